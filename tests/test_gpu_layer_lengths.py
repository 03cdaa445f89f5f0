"""The convolution and the scan at the strip and segment lengths that large calls get, and over more documents than a wave
looks through at once, against 64 bits.  The planned lengths are read from the workspaces, which hold a row a strip or segment."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda
from gated_delta_rule_41_amd import _lib

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
CODE = {F32: 0, BF16: 1}


def host(t):
    return t.detach().double().cpu().numpy()


class Normal:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, *shape, dtype=F32):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(dtype)


def cumulative(lens):
    return torch.tensor(ref.starts(lens), dtype=torch.int32, device="cuda")


def ragged(T, seed, shorts=(0, 1, 2, 3, 5, 0)):
    """A few long documents, short and empty ones between them and at both ends; T tokens."""
    rng = np.random.default_rng(seed)
    left = T - 2 * sum(shorts)
    cuts = np.sort(rng.integers(1, left, 3))
    longs = np.diff(np.concatenate([[0], cuts, [left]])).tolist()
    return [*shorts, *longs[:2], *shorts, *longs[2:], 0]


# ------------------------------------------------------------------ convolution
def conv_check(lens, C, W, dtype, channels, seed=0):
    normal, T, N = Normal(seed), sum(lens), len(lens)
    x, dy = normal(T, C, dtype=dtype), normal(T, C, dtype=dtype)
    w, b = normal(C, W, dtype=dtype), normal(C, dtype=dtype)
    state, dend = normal(N, W - 1, C, dtype=dtype), normal(N, W - 1, C, dtype=dtype)
    cu = cumulative(lens)
    y, end = kda.kda_conv_fwd(x, w, b, cu, state, out_dtype=F32)
    g = kda.kda_conv_bwd(x, w, b, dy, cu, state, dend, out_dtype=F32)
    ch = torch.tensor(channels, device="cuda")
    h = {n: host(t.index_select(d, ch)) for n, t, d in (("x", x, 1), ("w", w, 0), ("b", b, 0), ("state", state, 2), ("dy", dy, 1), ("dend", dend, 2))}
    want, last, bound = ref.conv_fwd(h["x"], h["w"], h["b"], h["state"], lens)
    assert (np.abs(host(y.index_select(1, ch)) - want) <= (bound + np.abs(want) * ref.U) * 1.01).all()
    assert (host(end.index_select(2, ch)) == last).all()
    want = ref.conv_bwd(h["x"], h["w"], h["b"], h["state"], lens, h["dy"], h["dend"])
    for n, d, half in (("dx", 1, ref.U), ("dw", 0, ref.U), ("db", 0, ref.U), ("dstate", 2, HALF[dtype])):
        value, off = want[n]
        assert (np.abs(host(g[n].index_select(d, ch)) - value) <= (off + np.abs(value) * half) * 1.01).all(), n
        assert torch.isfinite(g[n]).all(), n


def some(C, count=40):
    """The first and last channels and others between."""
    rng = np.random.default_rng(C)
    return sorted({0, min(7, C - 1), C - 1, max(C - 8, 0), max(C - 9, 0), *rng.integers(0, C, count).tolist()})


@pytest.mark.parametrize("T,C,dtype,strip", [(4500, 4096, BF16, 17), (16400, 4096, BF16, 64), (32800, 4096, BF16, 128), (33100, 4096, BF16, 65),
                                             (12500, 4099, BF16, 48), (11100, 12288, BF16, 65), (12000, 333, BF16, 30),
                                             (50000, 333, F32, 127), (9000, 4104, F32, 35), (1200000, 5, F32, 45)])
@pytest.mark.parametrize("W", [2, 4])
def test_convolution_strips(T, C, dtype, strip, W):
    need_gpu()
    lens = ragged(T, T)
    size = _lib.kda_conv_bwd_workspace_size(_lib.make_conv_config(C, W, CODE[dtype], 0, CODE[dtype]), T, len(lens))
    assert size == (T // strip + len(lens)) * (W + 1) * C * 4
    conv_check(lens, C, W, dtype, some(C))


def documents(N, seed):
    """Runs of empty ones, single tokens and short ones, a few long ones at the start, between and at the end."""
    rng = np.random.default_rng(seed)
    lens = rng.choice([0, 0, 0, 1, 1, 2, 3, 9], N)
    lens[N // 4:N // 3] = 0
    for at in (0, N // 2, N - 1):
        lens[at] = 150
    lens[rng.integers(0, N, 3)] = 61
    return lens.tolist()


@pytest.mark.parametrize("N", [64, 65, 66, 129, 4096, 4097, 70001])
@pytest.mark.parametrize("C,dtype,W", [(24, BF16, 4), (5, F32, 3)])
def test_convolution_over_many_documents(N, C, dtype, W):
    need_gpu()
    conv_check(documents(N, N), C, W, dtype, list(range(C)))


# ------------------------------------------------------------------ selective scan
GRADS = {"dx": "dx", "ddt": "ddt", "dA": "dA", "dB": "dB", "dC": "dC", "dD": "dD", "dz": "dz", "dbias": "ddt_bias", "dh0": "dS0"}
DIM = {"y": 1, "final": 1, "dx": 1, "ddt": 1, "dz": 1, "dA": 0, "dD": 0, "dbias": 0, "dh0": 1}


def check(got, want, most, count, dtype, name):
    """Every element within `count` roundings of its absolute sum, and the whole within the root of as many: they are independent."""
    assert got.dtype == dtype, name
    got = host(got)
    off = np.abs(got - want)
    assert (off <= (most * count * ref.U + np.abs(want) * HALF[dtype]) * 1.01 + 1e-37).all(), (name, (off / (most * ref.U + 1e-37)).max())
    assert np.linalg.norm(off) <= np.linalg.norm(most) * np.sqrt(count) * ref.U + np.linalg.norm(want) * HALF[dtype], name


def scan_check(lens, c, S, G, dtype, channels, segment, gated=True):
    """All outputs of `channels`; the others have x = 0 and dy = 0, so that they are in no sum for dB and dC."""
    normal, T, N = Normal(c + S), sum(lens), len(lens)
    d = {n: normal(T, c, dtype=dtype) for n in ("x", "raw", "dy")}
    d["z"] = normal(T, c, dtype=dtype) if gated else None
    ch = torch.tensor(channels, device="cuda")
    mask = torch.zeros(c, device="cuda", dtype=dtype)
    mask[ch] = 1
    d["x"] *= mask
    d["dy"] *= mask
    d.update(B=normal(T, G, S, dtype=dtype), C=normal(T, G, S, dtype=dtype), A=-torch.exp(normal(c, S)), D=normal(c), bias=normal(c) - 4,
             h0=normal(N, c, S), dh=normal(N, c, S))
    cu, kw = cumulative(lens), dict(D=d["D"], z=d["z"], dt_bias=d["bias"])
    args = [d[n] for n in ("x", "raw", "A", "B", "C")]
    y, final = kda.kda_selective_fwd(*args, cu, d["h0"], **kw)
    g = kda.kda_selective_bwd(*args, d["dy"], cu, d["h0"], d["dh"], **kw)
    per = c // G
    assert len(channels) % G == 0 and all(a // per == i // (len(channels) // G) for i, a in enumerate(channels))
    dims = {"x": 1, "raw": 1, "dy": 1, "z": 1, "A": 0, "D": 0, "bias": 0, "h0": 1, "dh": 1}
    h = {n: None if d[n] is None else host(d[n].index_select(k, ch)) for n, k in dims.items()}
    h.update(B=host(d["B"]), C=host(d["C"]), lens=lens)
    want, most = ref.selective(**h), ref.selective_absolute(**h)
    count = ref.selective_roundings(h["raw"], h["A"], h["bias"], lens, segment=segment)
    got = {"y": y, "final": final, **{n: g[k] for n, k in GRADS.items() if g[k] is not None}}
    for n, t in got.items():
        assert torch.isfinite(t).all(), n
        t = t.index_select(DIM[n], ch) if n in DIM else t
        # sums over all tokens, and over the waves of 64 channels
        more = T if n in ("dA", "dD", "dbias") else c // 64 if n in ("dB", "dC") else 0
        check(t, want[n], most[n], count + more, F32 if n in ("final", "dA", "dD", "dbias", "dh0") else dtype, n)


def spread(c, G, each):
    """`each` channels of every group, its first and last among them."""
    per, rng = c // G, np.random.default_rng(c)
    return [g * per + i for g in range(G) for i in [0, *sorted(1 + rng.choice(per - 2, each - 2, replace=False)), per - 1]]


def segment_length(T, N, c, S, G, dtype):
    """From the forward's workspace: a segment's states and sums of step sizes, each to 256 bytes."""
    size = _lib.kda_selective_fwd_workspace_size(_lib.make_selective_config(c, S, G, CODE[dtype], CODE[dtype]), T, N)
    slots = size // (c * 4 * (S + 1))
    assert size - slots * c * 4 * (S + 1) < 512
    return T // (slots - N), slots


@pytest.mark.parametrize("T,c,S,G,dtype,segment", [(2060, 16384, 16, 1, F32, 48), (4100, 16384, 16, 1, F32, 96), (4100, 16384, 8, 1, BF16, 96),
                                                   (4100, 16384, 32, 1, F32, 96), (6200, 16400, 16, 4, BF16, 156), (3000, 16390, 32, 2, F32, 72),
                                                   (2500, 32768, 8, 2, F32, 120)])
def test_scan_segments(T, c, S, G, dtype, segment):
    need_gpu()
    lens = ragged(T, T, (0, 1, 2, segment - 1, segment, segment + 1, 5, 0))
    length, slots = segment_length(T, len(lens), c, S, G, dtype)
    assert slots == T // segment + len(lens), length
    scan_check(lens, c, S, G, dtype, spread(c, G, 24 // G), segment)


@pytest.mark.parametrize("N", [64, 65, 66, 129, 4097, 9001])
@pytest.mark.parametrize("c,S,G,dtype,gated", [(24, 16, 1, F32, True), (10, 8, 2, BF16, False), (66, 32, 1, F32, False)])
def test_scan_over_many_documents(N, c, S, G, dtype, gated):
    need_gpu()
    lens = documents(N, N)
    scan_check(lens, c, S, G, dtype, list(range(c)), 64, gated)
