"""The documented forms in place against buffers of their own, bit for bit."""
import pytest

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda
from gated_delta_rule_41_amd import _lib

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CODE = {F32: 0, BF16: 1}


def p(t):
    return 0 if t is None else t.data_ptr()


def rand(*shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("C,dtype", [(64, BF16), (333, F32), (333, BF16), (12288, BF16), (2048, F32)])
def test_convolution_step_over_its_input(C, dtype):
    need_gpu()
    N, W = 37, 4
    x, w, state = rand(N, C, dtype=dtype, seed=1), rand(C, W, dtype=dtype, seed=2), rand(N, W - 1, C, dtype=dtype, seed=3)
    want, end = kda.kda_conv_decode(x, w, None, state)
    cfg = _lib.make_conv_config(C, W, CODE[dtype], CODE[dtype], CODE[dtype])
    assert _lib.kda_conv_decode_raw(cfg, N, p(x), p(w), 0, p(state), p(state), p(x), stream()) == 0
    assert torch.equal(x, want) and torch.equal(state, end)


def scan(lens, c, S, G, dtype):
    T = sum(lens)
    d = {n: rand(T, c, dtype=dtype, seed=i) for i, n in enumerate(("x", "dt", "z", "dy"))}
    d.update({n: rand(T, G, S, dtype=dtype, seed=9 + i) for i, n in enumerate(("B", "C"))})
    d.update(A=-rand(c, S, dtype=F32, seed=20).exp(), D=rand(c, dtype=F32, seed=21), bias=rand(c, dtype=F32, seed=22) - 3,
             h0=rand(len(lens), c, S, dtype=F32, seed=23), dh=rand(len(lens), c, S, dtype=F32, seed=24))
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    d["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    return d


# whole documents, many segments, groups that do not fill their waves
SCANS = [([5, 1, 0, 30], 72, 16, 1, BF16), ([1500, 7, 601], 200, 16, 2, F32), ([900, 0, 333], 130, 32, 2, BF16), ([700], 96, 8, 3, BF16),
         ([2500, 2500], 64, 16, 1, BF16)]


@pytest.mark.parametrize("lens,c,S,G,dtype", SCANS)
@pytest.mark.parametrize("over", ["x", "dt", "z"])
def test_scan_over_an_input(lens, c, S, G, dtype, over):
    need_gpu()
    d = scan(lens, c, S, G, dtype)
    T, N = sum(lens), len(lens)
    want, end = kda.kda_selective_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["cu"], d["h0"], D=d["D"], z=d["z"], dt_bias=d["bias"])
    cfg = _lib.make_selective_config(c, S, G, CODE[dtype], CODE[dtype])
    ws = torch.empty(_lib.kda_selective_fwd_workspace_size(cfg, T, N) + 16, dtype=torch.uint8, device="cuda")
    final, y = torch.empty_like(d["h0"]), d[over]
    assert _lib.kda_selective_fwd_raw(cfg, T, N, *(p(d[n]) for n in ("x", "dt", "A", "B", "C", "D", "z", "bias", "cu", "h0")), p(y), p(final),
                                      p(ws), ws.numel(), stream()) == 0
    assert torch.equal(y, want) and torch.equal(final, end)


@pytest.mark.parametrize("lens,c,S,G,dtype", SCANS)
@pytest.mark.parametrize("over", [("x", "dt", "z"), ("dy", "x", "dt"), ("dt", "z", "dy"), ("z", "dy", "x")])
def test_scan_backward_over_its_inputs(lens, c, S, G, dtype, over):
    need_gpu()
    d = scan(lens, c, S, G, dtype)
    T, N = sum(lens), len(lens)
    want = kda.kda_selective_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], d["cu"], d["h0"], d["dh"], D=d["D"], z=d["z"], dt_bias=d["bias"])
    cfg = _lib.make_selective_config(c, S, G, CODE[dtype], CODE[dtype])
    ws = torch.empty(_lib.kda_selective_bwd_workspace_size(cfg, T, N), dtype=torch.uint8, device="cuda")
    out = {n: torch.empty_like(t) for n, t in want.items()}
    out.update(zip(("dx", "ddt", "dz"), (d[n] for n in over)))
    assert _lib.kda_selective_bwd_raw(cfg, T, N, *(p(d[n]) for n in ("x", "dt", "A", "B", "C", "D", "z", "bias", "cu", "h0", "dy", "dh")),
                                      *(p(out[n]) for n in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")),
                                      p(ws), ws.numel(), stream()) == 0
    for n in want:
        assert torch.equal(out[n], want[n]), n


@pytest.mark.parametrize("c,S,G,dtype", [(64, 16, 1, BF16), (333, 16, 3, F32), (4096, 8, 1, BF16), (72, 32, 2, F32)])
@pytest.mark.parametrize("over", ["x", "dt", "z"])
def test_scan_step_over_an_input(c, S, G, dtype, over):
    need_gpu()
    N = 9
    d = scan([1] * N, c, S, G, dtype)
    want, end = kda.kda_selective_decode(d["x"], d["dt"], d["A"], d["B"], d["C"], d["h0"], D=d["D"], z=d["z"], dt_bias=d["bias"])
    cfg = _lib.make_selective_config(c, S, G, CODE[dtype], CODE[dtype])
    y = d[over]
    assert _lib.kda_selective_decode_raw(cfg, N, *(p(d[n]) for n in ("x", "dt", "A", "B", "C", "D", "z", "bias")), p(d["h0"]), p(d["h0"]), p(y),
                                         stream()) == 0
    assert torch.equal(y, want) and torch.equal(d["h0"], end)


# row ends in a thread's second group, in a wave of their own, rows read again, fewer than eight channels
WIDTHS = [5, 100, 333, 1000, 1025, 2049, 2561, 4096, 4099, 6137, 8200, 12281, 12289, 16377, 16384]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_over_its_inputs(C, dtype):
    """y over x, and s over the residual or over x with y elsewhere."""
    need_gpu()
    rows = 300
    x, r, w = rand(rows, C, dtype=dtype, seed=1), rand(rows, C, dtype=dtype, seed=2), rand(1, C, dtype=dtype, seed=3)[0]
    want, total = kda.kda_norm_fwd(x, w, r)
    alone, _ = kda.kda_norm_fwd(x, w)
    cfg = _lib.make_norm_config(C, *[CODE[dtype]] * 4)

    def call(x, r, y, s):
        assert _lib.kda_norm_fwd_raw(cfg, rows, p(x), p(r), p(w), p(y), p(s), 0, stream()) == 0
        return y, s

    a, b = x.clone(), r.clone()
    y, s = call(a, b, a, b)
    assert torch.equal(y, want) and torch.equal(s, total)
    a = x.clone()
    y, s = call(a, r, torch.empty_like(x), a)
    assert torch.equal(y, want) and torch.equal(s, total)
    a = x.clone()
    assert torch.equal(call(a, None, a, None)[0], alone)
    codes, _, scale = kda.kda_norm_fwd(x, w, r, out_dtype=torch.int8)
    cfg.out_dtype = _lib.KDA_I8
    a, got, got_scale = x.clone(), torch.empty_like(codes), torch.empty_like(scale)
    assert _lib.kda_norm_fwd_raw(cfg, rows, p(a), p(r), p(w), p(got), p(a), p(got_scale), stream()) == 0
    assert torch.equal(got, codes) and torch.equal(a, total) and torch.equal(got_scale, scale)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("over", ["dy", "ds"])
def test_norm_backward_over_a_gradient(C, dtype, over):
    """More rows than one turn of the workgroups takes: rows asked for early lie beside rows that are written."""
    need_gpu()
    rows = 20011 if C < 400 else 1700
    s, dy, ds = (rand(rows, C, dtype=dtype, seed=i) for i in range(3))
    w = rand(1, C, dtype=dtype, seed=3)[0]
    want = kda.kda_norm_bwd(s, w, dy, ds)
    cfg = _lib.make_norm_config(C, *[CODE[dtype]] * 4, eps=1e-6)
    ws = torch.empty(_lib.kda_norm_bwd_workspace_size(cfg, rows), dtype=torch.uint8, device="cuda")
    dx, dw = {"dy": dy, "ds": ds}[over], torch.empty_like(want["dw"])
    assert _lib.kda_norm_bwd_raw(cfg, rows, p(s), p(w), p(dy), p(ds), p(dx), p(dw), p(ws), ws.numel(), stream()) == 0
    assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"])
