"""The linear rule (kda_linear_fwd / _bwd / _decode) against the 64-bit token
recurrence of tests/linear_ref.py.

Tolerances, with M as defined there:
  * o, dq, dk, dv from fp32 inputs: a sum over the dk (or dv) channels and the
    tokens of a block (at most 128 + 128 + 128 terms), the decays' exponents
    (|G| <= 100 in the factors that matter, each rounded by 2^-24 of itself):
    512 half steps.
  * the same from bf16 inputs: two roundings to bf16 more (P or dP, and the
    state as it is read), each to its own terms: one 2^-8 of M.
  * states: fp32 terms in any order, 512 half steps, bf16 inputs or not.
  * dg: the crossing terms take two bf16 roundings in <S, dS>, 2^-7 of M; the row
    and column sums cancel in fp32, 512 half steps of everything summed.
  * an output stored in bf16: 2^-8 of the value more.
Over a whole output, with V as defined there, the norm of the error is at most
the same roundings times the norm of sqrt(V), with sqrt(512) < 32 half steps for
the sums.
"""
import numpy as np
import pytest

import linear_ref as ref
from linear_ref import BF16, F32

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu

STEPS, ROOT = 512 * F32, 32 * F32


def _say(msg):
    print(f"[gpu-linear] {msg}", flush=True)


def make(seed, lens, H, Hk, dk, dv, dtype, gate="token", strength=-2.0, s0=True):
    rng = np.random.default_rng([77, seed])
    T, N = int(sum(lens)), len(lens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rounded(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt)

    x = {"q": rounded(T, Hk, dk), "k": rounded(T, Hk, dk), "v": rounded(T, H, dv), "dO": rounded(T, H, dv)}
    shape = (H,) if gate == "head" else (T, H)
    x["g"] = torch.from_numpy(-np.log1p(np.exp(rng.standard_normal(shape) + strength)).astype(np.float32))
    x["s0"] = torch.from_numpy((0.1 * rng.standard_normal((N, H, dk, dv))).astype(np.float32)) if s0 else None
    x["dS"] = torch.from_numpy((0.1 * rng.standard_normal((N, H, dk, dv))).astype(np.float32)) if s0 else None
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    h = {n: None if t is None else t.float().numpy().astype(np.float64) for n, t in x.items()}
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return d, h, cu


def host(t):
    return t.detach().double().cpu().numpy()


def check(name, x, r, M, rel, stored=0.0, extra=0.0, V=None, whole=0.0):
    x = host(x)
    assert np.isfinite(x).all(), name
    if V is not None and x.size:
        off, most = np.linalg.norm(x - r), whole * np.sqrt(V.sum()) + stored * np.linalg.norm(r)
        _say(f"  {name}: the error's norm is {off / max(most, 1e-300):.3f} of its bound")
        assert off <= most, name
    bound = rel * M + stored * np.abs(r) + extra + 1e-30
    worst = float((np.abs(x - r) / bound).max()) if x.size else 0.0
    _say(f"  {name}: largest error is {worst:.3f} of its bound")
    assert worst <= 1.0, name


def check_fwd(d, h, cu, lens, dtype, out, scale, **kw):
    o, sf = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], out_dtype=out, scale=scale, **kw)
    torch.cuda.synchronize()
    r, rf, _ = ref.linear_fwd(h["q"], h["k"], h["v"], h["g"], lens, h["s0"], scale)
    M, Mf, _ = ref.linear_fwd(*ref.absolute(h["q"], h["k"], h["v"]), h["g"], lens, *ref.absolute(h["s0"]), abs(scale))
    V, Vf, _ = ref.linear_fwd(*ref.squared(h["q"], h["k"], h["v"]), 2 * h["g"], lens, *ref.squared(h["s0"]), scale ** 2)
    rounded = BF16 if dtype == "bf16" else 0
    check("o", o, r, M, STEPS + rounded, BF16 if out == torch.bfloat16 else 0, V=V, whole=ROOT + rounded)
    check("final", sf, rf, Mf, STEPS, V=Vf, whole=ROOT)
    return o, sf


def check_bwd(d, h, cu, lens, dtype, out, scale, **kw):
    gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], out_dtype=out, scale=scale, **kw)
    torch.cuda.synchronize()
    r = ref.linear_bwd(h["q"], h["k"], h["v"], h["g"], lens, h["dO"], h["s0"], h["dS"], scale)
    a = dict(zip(("q", "k", "v", "dO", "s0", "dS"), ref.absolute(*(h[n] for n in ("q", "k", "v", "dO", "s0", "dS")))))
    M = ref.linear_bwd(a["q"], a["k"], a["v"], h["g"], lens, a["dO"], a["s0"], a["dS"], abs(scale))
    a2 = dict(zip(("q", "k", "v", "dO", "s0", "dS"), ref.squared(*(h[n] for n in ("q", "k", "v", "dO", "s0", "dS")))))
    V = ref.linear_bwd(a2["q"], a2["k"], a2["v"], 2 * h["g"], lens, a2["dO"], a2["s0"], a2["dS"], scale ** 2)
    rounded = BF16 if dtype == "bf16" else 0
    stored = BF16 if out == torch.bfloat16 else 0
    for n in ("dq", "dk", "dv"):
        check(n, gr[n], r[n], M[n], STEPS + rounded, stored, V=V[n], whole=ROOT + rounded)
    check("dS0", gr["dS0"], r["dS0"], M["dS0"], STEPS, V=V["dS0"], whole=ROOT)
    # everything the row and column sums hold: a head's q . dq over the document (an upper bound for a block)
    R = d["v"].shape[1] // d["q"].shape[1]
    all_ = np.repeat((a["q"] * M["dq"]).sum((0, 2)), R) * 2
    check("dg", gr["dg"], r["dg"], M["dg"], STEPS + (2 * BF16 if dtype == "bf16" else 0), stored,
          STEPS * all_ * (len(lens) if d["g"].dim() == 1 else 1))
    return gr


CASES = [
    # lens, H, Hk, dk, dv, dtype, gate
    ([1], 1, 1, 64, 64, "f32", "token"),
    ([1], 2, 1, 128, 128, "bf16", "head"),
    ([5, 64, 65], 3, 3, 64, 128, "f32", "head"),
    ([0, 63, 0, 128, 1, 0], 2, 2, 128, 64, "f32", "token"),
    ([127, 128, 129, 1, 30], 4, 2, 128, 128, "bf16", "token"),
    ([257, 3], 6, 2, 64, 64, "bf16", "token"),
    ([200], 4, 1, 128, 64, "bf16", "head"),
    ([130, 40], 2, 2, 128, 128, "f32", "token"),
    ([33, 95, 2], 3, 1, 64, 128, "bf16", "token"),
]


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype,gate", CASES)
def test_forward(lens, H, Hk, dk, dv, dtype, gate):
    need_gpu()
    _say(f"forward {lens} H={H} Hk={Hk} {dk}x{dv} {dtype} {gate}")
    d, h, cu = make(1, lens, H, Hk, dk, dv, dtype, gate)
    for out in (torch.float32, torch.bfloat16):
        check_fwd(d, h, cu, lens, dtype, out, dk ** -0.5)


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype,gate", CASES)
def test_backward(lens, H, Hk, dk, dv, dtype, gate):
    need_gpu()
    _say(f"backward {lens} H={H} Hk={Hk} {dk}x{dv} {dtype} {gate}")
    d, h, cu = make(2, lens, H, Hk, dk, dv, dtype, gate)
    for out in (torch.float32, torch.bfloat16):
        check_bwd(d, h, cu, lens, dtype, out, dk ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H,Hk,dk,dv,gate", [
    ([1500, 1730], 2, 1, 64, 64, "token"),
    ([0, 3, 2600, 130, 0, 1024, 512, 513, 0], 1, 1, 64, 64, "head"),
    ([1100, 64], 2, 2, 128, 128, "token"),
    ([1700], 3, 1, 64, 128, "token"),
])
def test_segments(dtype, lens, H, Hk, dk, dv, gate):
    """Documents long enough to be cut into segments (128 tokens at these sizes), among short and empty ones."""
    need_gpu()
    _say(f"segments {lens} {dtype}")
    d, h, cu = make(3, lens, H, Hk, dk, dv, dtype, gate, -3.0)
    cfg = kda.linear._lib.make_linear_config(H, Hk, dk, dv)
    assert kda.linear._lib.kda_linear_fwd_workspace_size(cfg, sum(lens), len(lens)) > 0
    check_fwd(d, h, cu, lens, dtype, torch.float32, 0.125)
    check_bwd(d, h, cu, lens, dtype, torch.float32, 0.125)
    for n in ("s0", "dS"):
        d[n] = h[n] = None
    h["s0"] = h["dS"] = np.zeros((len(lens), H, dk, dv))
    check_fwd(d, h, cu, lens, dtype, torch.float32, 0.125)
    check_bwd(d, h, cu, lens, dtype, torch.float32, 0.125)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("short,long", [([0, 1, 2, 5, 9], [1290]), ([4, 3, 0, 2], [])])
def test_many_documents(dtype, short, long):
    """131 documents, one of them in segments, and 600 (more than are cut): looked up 64 at a time."""
    need_gpu()
    lens = (short * 65)[:70] + long + (short * 65)[:60] if long else short * 150
    _say(f"{len(lens)} documents {dtype}")
    d, h, cu = make(20, lens, 2, 1, 64, 64, dtype)
    sizes = kda.linear._lib.make_linear_config(2, 1, 64, 64), sum(lens), len(lens)
    assert sum(lens) > 1024 and (kda.linear._lib.kda_linear_fwd_workspace_size(*sizes) > 0) == bool(long)
    check_fwd(d, h, cu, lens, dtype, torch.float32, 0.125)
    check_bwd(d, h, cu, lens, dtype, torch.float32, 0.125)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H", [([129, 1, 200, 64, 0, 130, 65, 63], 32), ([8192], 64), ([2900] + [73, 64, 1] * 5, 16),
                                    ([256, 0, 128, 300, 1, 0, 384, 77], 64), ([40] * 50 + [0] * 13 + [700], 32),
                                    ([1024] * 8, 16), ([1024] * 3 + [1025, 1023] + [1024] * 3, 16)])
def test_many_heads(dtype, lens, H):
    """Enough walks that a workgroup of the state kernel takes 128 value columns, and that the forward's come in the order
    of their lengths (full segments, rests, equal ones, empty documents), and documents that the backward leaves whole
    until one is a token longer; some heads are compared, each with the
    reference and with a call for it alone."""
    need_gpu()
    _say(f"{H} heads {lens[:2]}... {dtype}")
    d, h, cu = make(21, lens, H, H, 64, 128, dtype)
    o, sf = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=0.125)
    gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125)
    torch.cuda.synchronize()
    for x in (o, sf, *gr.values()):
        assert bool(torch.isfinite(x).all())
    heads = [0, H // 2 + 1, H - 1] if sum(lens) < 1024 else [H - 1]
    for head in heads:
        # the same head alone: another plan, other kernels
        e = {n: t[:, head:head + 1].contiguous() for n, t in d.items()}
        eh = {n: t[:, head:head + 1] for n, t in h.items()}
        o1, sf1 = check_fwd(e, eh, cu, lens, dtype, torch.float32, 0.125)
        gr1 = check_bwd(e, eh, cu, lens, dtype, torch.float32, 0.125)
        # The inputs are independent, so the norm of sqrt(V) is about the output's own.  bf16: each side rounds P (or dP)
        # and the state once, 2^-8 each.
        for n, a, b in [("o", o, o1), ("final", sf, sf1)] + [(n, gr[n], gr1[n]) for n in ("dq", "dk", "dv", "dg", "dS0")]:
            a = a[:, head:head + 1].double()
            off, size = float((a - b.double()).norm()), float(b.double().norm())
            most = STEPS + (0 if dtype == "f32" or n in ("final", "dS0") else 4 * BF16)
            _say(f"  head {head} {n}: {off / size:.2e} of its norm from the head alone, at most {most:.2e}")
            assert off <= most * size, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H,Hk,dk,dv", [([130, 5], 8, 1, 64, 64), ([150], 9, 3, 128, 128), ([3] * 100 + [70], 6, 1, 64, 128)])
def test_divided_value_heads(dtype, lens, H, Hk, dk, dv):
    """A key head's value heads in several workgroups: 8 or 3 parts of one head, and 2 parts of three."""
    need_gpu()
    _say(f"{H}/{Hk} heads, {len(lens)} documents {dtype}")
    d, h, cu = make(22, lens, H, Hk, dk, dv, dtype)
    for out in (torch.float32, torch.bfloat16):
        check_bwd(d, h, cu, lens, dtype, out, 0.125)


def big(seed, T, N, H, Hk, dk, dv):
    """bf16 inputs made on the GPU, for sizes that numpy would take long over."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rounded(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    d = {"q": rounded(T, Hk, dk), "k": rounded(T, Hk, dk), "v": rounded(T, H, dv), "dO": rounded(T, H, dv)}
    d["g"] = -torch.nn.functional.softplus(torch.randn((T, H), generator=gen, device="cuda") - 2)
    d["s0"], d["dS"] = (0.1 * torch.randn((N, H, dk, dv), generator=gen, device="cuda") for _ in range(2))
    return d


def part(d, rows, docs, heads, keys):
    """The inputs of some rows, documents and heads, contiguous."""
    e = {n: d[n][rows][:, keys].contiguous() for n in ("q", "k")}
    e.update({n: d[n][rows][:, heads].contiguous() for n in ("v", "dO", "g")})
    e.update({n: d[n][docs][:, heads].contiguous() for n in ("s0", "dS")})
    return e, {n: host(t) for n, t in e.items()}


def test_most_heads():
    """32767 heads, the most there are: 32-bit row offsets of almost 2^31 bytes in the fp32 outputs."""
    need_gpu()
    T, H, dk, dv = 129, 32767, 64, 128
    d = big(31, T, 1, H, H, dk, dv)
    _say("most heads")
    o, sf = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], None, d["s0"], scale=0.125)
    gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], None, d["s0"], d["dS"], scale=0.125)
    torch.cuda.synchronize()
    heads = [0, 20001, 32766]
    e, h = part(d, slice(0, T), slice(0, 1), heads, heads)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    o1, sf1 = check_fwd(e, h, cu, [T], "bf16", torch.float32, 0.125)
    gr1 = check_bwd(e, h, cu, [T], "bf16", torch.float32, 0.125)
    # the plans differ only in the segments, which 129 tokens do not have: the same sums in the same order
    for n, a, b in [("o", o, o1), ("final", sf, sf1)] + [(n, gr[n], gr1[n]) for n in gr]:
        assert torch.equal(a[:, heads], b), n


def test_long_offsets():
    """131072 tokens x 128 heads of 128: more than 2^31 elements of v, o, dO and dv.  The last document is compared."""
    need_gpu()
    lens, H, Hk, dk, dv = [131000, 72], 128, 1, 64, 128
    d = big(32, sum(lens), 2, H, Hk, dk, dv)
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    _say("long offsets")
    o, sf = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=0.125, out_dtype=torch.bfloat16)
    gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125,
                            out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    rows = slice(lens[0], sum(lens))
    e, h = part(d, rows, slice(1, 2), slice(0, H), slice(0, 1))
    one = torch.tensor([0, lens[1]], dtype=torch.int32, device="cuda")
    o1, sf1 = check_fwd(e, h, one, lens[1:], "bf16", torch.bfloat16, 0.125)
    assert torch.equal(o[rows], o1) and torch.equal(sf[1:], sf1)
    gr1 = check_bwd(e, h, one, lens[1:], "bf16", torch.bfloat16, 0.125)
    for n in ("dv", "dg"):
        assert torch.equal(gr[n][rows], gr1[n]), n
    assert torch.equal(gr["dS0"][1:], gr1["dS0"])
    # the value heads of the one key head are divided among workgroups for 72 tokens, not for 131072: sums of 128 heads
    # in another order, then one rounding each
    for n in ("dq", "dk"):
        a, b = gr[n][rows].double(), gr1[n].double()
        assert float((a - b).norm()) <= (2 * BF16 + STEPS) * float(b.norm()), n


def test_decode_long_offsets():
    """More than 2^31 elements of state, in place."""
    need_gpu()
    N, H, d = 530, 256, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((N, H, d), generator=gen, device="cuda") for _ in range(3))
    g = -torch.rand((N, H), generator=gen, device="cuda")
    s = torch.randn((N, H, d, d), generator=gen, device="cuda")
    _say("decode, long offsets")
    want = [x[-1:] for x in kda.kda_linear_decode(*(x[-1:].clone() for x in (q, k, v, g)), s[-1:].clone())]
    o, s2 = kda.kda_linear_decode(q, k, v, g, s, out_state=s)
    torch.cuda.synchronize()
    assert s2 is s and torch.equal(o[-1:], want[0]) and torch.equal(s[-1:], want[1])


def test_strong_and_infinite_gates():
    """Gates of -8 a token, and -inf, which restarts the state at its token."""
    need_gpu()
    lens, H, Hk, dk, dv = [150, 70], 2, 2, 64, 64
    for dtype in ("f32", "bf16"):
        _say(f"strong gates {dtype}")
        d, h, cu = make(5, lens, H, Hk, dk, dv, dtype)
        g = np.full(h["g"].shape, -8.0, np.float32)
        g[::3] = -0.01
        g[40] = g[100, 1] = g[149] = g[150] = -np.inf
        g[41:60] = -200.0
        d["g"] = torch.from_numpy(g).cuda()
        h["g"] = np.maximum(g.astype(np.float64), -1e3)   # e^-1000 is zero in 64 bits too
        check_fwd(d, h, cu, lens, dtype, torch.float32, 1.0)
        check_bwd(d, h, cu, lens, dtype, torch.float32, 1.0)


def test_no_state_no_final():
    need_gpu()
    lens = [70, 129]
    d, h, cu = make(6, lens, 2, 1, 64, 64, "f32", s0=False)
    o, _ = check_fwd(d, h, cu, lens, "f32", torch.float32, 1.0)
    o2, none = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, output_final_state=False)
    assert none is None and torch.equal(o, o2)
    check_bwd(d, h, cu, lens, "f32", torch.float32, 1.0)
    gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, output_d_initial_state=False)
    assert gr["dS0"] is None


def test_equal_sequences_and_empty_stream():
    need_gpu()
    lens = [75, 75, 75]
    d, h, cu = make(7, lens, 2, 2, 64, 64, "f32")
    o, sf = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"])
    o2, sf2 = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], None, d["s0"], num_seqs=3)
    assert torch.equal(o, o2) and torch.equal(sf, sf2)
    # no tokens: states pass through, a gate per head has a zero gradient
    z, e = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.empty((0, 2, 64), device="cuda")
    s0, gh = d["s0"][:2].contiguous(), torch.full((2,), -0.1, device="cuda")
    o, sf = kda.kda_linear_fwd(e, e, e, gh, z, s0)
    gr = kda.kda_linear_bwd(e, e, e, gh, e, z, s0, s0)
    torch.cuda.synchronize()
    assert o.shape == (0, 2, 64) and torch.equal(sf, s0) and torch.equal(gr["dS0"], s0)
    assert torch.equal(gr["dg"], torch.zeros_like(gh))


def test_documents_do_not_touch_each_other():
    """NaN in one document (inputs, gate, state) leaves the others bitwise alone; so do rows behind the last one."""
    need_gpu()
    lens, H, Hk, dk, dv = [70, 65, 140], 2, 2, 64, 64
    d, h, cu = make(8, lens, H, Hk, dk, dv, "bf16")
    T, pad = sum(lens), 37
    clean = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"])
    cleang = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"])
    bad = {n: t.clone() for n, t in d.items()}
    for n in ("q", "k", "v", "g", "dO"):
        bad[n][70:135] = float("nan")
    bad["s0"][1], bad["dS"][1] = float("nan"), float("inf")
    o, sf = kda.kda_linear_fwd(bad["q"], bad["k"], bad["v"], bad["g"], cu, bad["s0"])
    gr = kda.kda_linear_bwd(bad["q"], bad["k"], bad["v"], bad["g"], bad["dO"], cu, bad["s0"], bad["dS"])
    torch.cuda.synchronize()
    for a, b in [(o, clean[0])] + [(gr[n], cleang[n]) for n in ("dq", "dk", "dv", "dg")]:
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[135:], b[135:])
    for a, b in ((sf, clean[1]), (gr["dS0"], cleang["dS0"])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    # a stream with room behind the last document: its rows are neither read nor written
    wide = {n: torch.cat([d[n], torch.full((pad,) + tuple(d[n].shape[1:]), float("nan"), device="cuda").to(d[n].dtype)])
            for n in ("q", "k", "v", "g", "dO")}
    lib = kda.linear._lib
    cfg = lib.make_linear_config(H, Hk, dk, dv)
    ow, sw = torch.full((T + pad, H, dv), 7.0, device="cuda"), torch.empty_like(sf)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.kda_linear_fwd_raw(cfg, T + pad, 3, *(wide[n].data_ptr() for n in ("q", "k", "v", "g")), cu.data_ptr(),
                                  d["s0"].data_ptr(), ow.data_ptr(), sw.data_ptr(), 0, 0, st) == 0
    outs = {n: torch.full(s, 7.0, device="cuda") for n, s in
            (("dq", (T + pad, Hk, dk)), ("dk", (T + pad, Hk, dk)), ("dv", (T + pad, H, dv)), ("dg", (T + pad, H)))}
    wsb = lib.kda_linear_bwd_workspace_size(cfg, T + pad, 3)
    ws, dS0 = torch.empty(wsb, dtype=torch.uint8, device="cuda"), torch.empty_like(sf)
    assert lib.kda_linear_bwd_raw(cfg, T + pad, 3, *(wide[n].data_ptr() for n in ("q", "k", "v", "g")), cu.data_ptr(),
                                  d["s0"].data_ptr(), wide["dO"].data_ptr(), d["dS"].data_ptr(),
                                  *(outs[n].data_ptr() for n in ("dq", "dk", "dv", "dg")), dS0.data_ptr(), ws.data_ptr(),
                                  wsb, st) == 0
    torch.cuda.synchronize()
    assert torch.equal(ow[:T], clean[0]) and torch.equal(sw, clean[1]) and bool((ow[T:] == 7.0).all())
    for n in outs:
        assert torch.equal(outs[n][:T], cleang[n]) and bool((outs[n][T:] == 7.0).all()), n
    assert torch.equal(dS0, cleang["dS0"])


def test_gradients_against_differences():
    """<dO, o> + <dS, final> is linear in each of q, k, v and the initial state: its difference along a direction is
    exact up to rounding.  Along g the step is small.  fp32 inputs; the losses are summed in 64 bits."""
    need_gpu()
    lens = [130, 61]
    for gate in ("token", "head"):
        d, h, cu = make(9, lens, 4, 2, 64, 64, "f32", gate)

        def loss(**kw):
            x = dict(d, **kw)
            o, sf = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["g"], cu, x["s0"], scale=0.125)
            return float((o.double() * d["dO"].double()).sum() + (sf.double() * d["dS"].double()).sum())

        gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125)
        # rounding of each loss: every output is off by up to ROOT sqrt(V), independently of the others; six deviations.
        # A step of at most 3 in one input makes no V more than 16 times larger.
        a = ref.squared(h["q"], h["k"], h["v"], h["s0"], h["dO"], h["dS"])
        V, Vf, _ = ref.linear_fwd(a[0], a[1], a[2], 2 * h["g"], lens, a[3], 0.125 ** 2)
        noise = 6 * ROOT * 4 * float(np.sqrt((V * a[4]).sum() + (Vf * a[5]).sum()))
        rng = torch.Generator(device="cuda").manual_seed(3)
        for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "dS0"), ("g", "dg")):
            u = torch.randn(d[n].shape, generator=rng, device="cuda")
            eps = 0.5 if n != "g" else 2.0 ** -8 if gate == "token" else 2.0 ** -11
            plus, minus = d[n] + eps * u, d[n] - eps * u
            du = (plus.double() - minus.double())     # the step that fp32 made of it
            diff = loss(**{n: plus}) - loss(**{n: minus})
            want = float((gr[gn].double() * du).sum())
            size = float((gr[gn].double() * du).abs().sum())
            tol = 2 * noise + STEPS * size
            if n == "g":
                # third order: a path over t tokens moves by e^x with x at most t steps (a fixed gate: all of them the
                # same way; gates per token: about sqrt(t)), x^3 / 6 of each term; terms beyond 32 tokens are small
                x = eps * float(u.abs().max()) * (32 if gate == "head" else 6)
                tol += x * x / 6 * size
            _say(f"{gate} d{n}: difference {diff:.6f}, gradient {want:.6f}, tolerance {tol:.6f}")
            assert abs(diff - want) <= tol, n


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("f32", 128, 128), ("bf16", 128, 128), ("bf16", 64, 128),
                                         ("bf16", 128, 64)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_decode(dtype, dk, dv, gate):
    need_gpu()
    N, H, Hk = 5, 4, 2
    d, h, _ = make(10, [1] * N, H, Hk, dk, dv, dtype, gate)
    r, rf, _ = ref.linear_fwd(h["q"], h["k"], h["v"], h["g"], [1] * N, h["s0"], 0.3)
    M, Mf, _ = ref.linear_fwd(*ref.absolute(h["q"], h["k"], h["v"]), h["g"], [1] * N, *ref.absolute(h["s0"]), 0.3)
    for out in (torch.float32, torch.bfloat16):
        o, s = kda.kda_linear_decode(d["q"], d["k"], d["v"], d["g"], d["s0"], out_dtype=out, scale=0.3)
        check("o", o, r, M, STEPS, BF16 if out == torch.bfloat16 else 0)
        check("state", s, rf, Mf, 8 * F32)
    keep = d["s0"].clone()
    o2, s2 = kda.kda_linear_decode(d["q"], d["k"], d["v"], d["g"], keep, out_state=keep, scale=0.3)
    assert s2 is keep and torch.equal(s2, s) and torch.equal(o2.to(torch.bfloat16), o)
    # zero state, and an empty batch
    o3, s3 = kda.kda_linear_decode(d["q"], d["k"], d["v"], d["g"], scale=0.3)
    o4, s4 = kda.kda_linear_decode(d["q"], d["k"], d["v"], d["g"], torch.zeros_like(d["s0"]), scale=0.3)
    assert torch.equal(o3, o4) and torch.equal(s3, s4)
    g0 = d["g"] if gate == "head" else d["g"][:0]
    o5, s5 = kda.kda_linear_decode(d["q"][:0], d["k"][:0], d["v"][:0], g0)
    torch.cuda.synchronize()
    assert o5.shape == (0, H, dv) and s5.shape == (0, H, dk, dv)


def test_prefill_then_decode():
    """The forward over a prefix and one decode step per further token equal the recurrence over the whole."""
    need_gpu()
    lens, steps, H, Hk, dk, dv = [90, 1, 130], 20, 4, 2, 128, 128
    total = [n + steps for n in lens]
    d, h, _ = make(11, total, H, Hk, dk, dv, "bf16")
    r, rf, _ = ref.linear_fwd(h["q"], h["k"], h["v"], h["g"], total, h["s0"], 0.1)
    M, Mf, _ = ref.linear_fwd(*ref.absolute(h["q"], h["k"], h["v"]), h["g"], total, *ref.absolute(h["s0"]), 0.1)
    start = np.concatenate([[0], np.cumsum(total)])[:-1]
    pre = np.concatenate([np.arange(s, s + n) for s, n in zip(start, lens)])
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    _, s = kda.kda_linear_fwd(*(d[n][pre].contiguous() for n in ("q", "k", "v", "g")), cu, d["s0"], scale=0.1)
    for t in range(steps):
        rows = start + np.array(lens) + t
        o, s = kda.kda_linear_decode(*(d[n][rows].contiguous() for n in ("q", "k", "v", "g")), s, out_state=s, scale=0.1)
        check(f"o of step {t}", o, r[rows], M[rows], STEPS)
    check("state", s, rf, Mf, STEPS)


def test_autograd_matches_direct_calls():
    need_gpu()
    lens = [100, 33]
    for gate in ("token", "head"):
        d, h, cu = make(12, lens, 4, 2, 64, 64, "bf16", gate)
        leaves = {n: d[n].clone().requires_grad_(True) for n in ("q", "k", "v", "g", "s0")}
        o, sf = kda.kda_linear(leaves["q"], leaves["k"], leaves["v"], leaves["g"], cu, leaves["s0"], scale=0.125)
        ((o * d["dO"].float()).sum() + (sf * d["dS"]).sum()).backward()
        o2, sf2 = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=0.125)
        gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125,
                                out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(sf, sf2)
        for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "dS0")):
            assert leaves[n].grad.dtype == leaves[n].dtype
            assert torch.equal(leaves[n].grad, gr[gn].to(leaves[n].dtype)), n
        # only one output in the loss
        leaves["q"].grad = None
        o, sf = kda.kda_linear(leaves["q"], d["k"], d["v"], d["g"], cu, scale=0.125)
        sf.sum().backward()
        assert torch.equal(leaves["q"].grad, torch.zeros_like(d["q"]))


def test_autograd_upstream_views_and_second_order():
    """Upstream gradients that are odd views of larger tensors; a second differentiation raises."""
    need_gpu()
    lens = [40, 9]
    d, h, cu = make(15, lens, 2, 2, 64, 64, "f32")
    gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125)
    leaves = {n: d[n].clone().requires_grad_(True) for n in ("q", "k", "v", "g", "s0")}
    o, sf = kda.kda_linear(leaves["q"], leaves["k"], leaves["v"], leaves["g"], cu, leaves["s0"], scale=0.125)
    one = torch.zeros(1, device="cuda", requires_grad=True)
    w = torch.cat([torch.zeros(1, device="cuda"), d["dO"].flatten(), d["dS"].flatten()])
    (torch.cat([one, o.flatten(), sf.flatten()]) * w).sum().backward()
    torch.cuda.synchronize()
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "dS0")):
        assert torch.equal(leaves[n].grad, gr[gn]), n
    o, _ = kda.kda_linear(leaves["q"], d["k"], d["v"], d["g"], cu, scale=0.125)
    (dq,) = torch.autograd.grad(o.square().sum(), leaves["q"], create_graph=True)
    with pytest.raises(RuntimeError):
        dq.sum().backward()


def test_scale_is_read_at_each_call():
    """A tensor as scale: its value counts, not its identity."""
    need_gpu()
    d, _, cu = make(16, [20], 1, 1, 64, 64, "f32")
    scale = torch.tensor(0.5)
    a, _ = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=scale)
    scale.mul_(2)
    b, _ = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(2 * a, b)


def test_repeatable_graph_streams():
    """Two calls agree bitwise; a captured forward, backward and decode replays bitwise, with eager work in between;
    calls on two streams at once equal the same calls in turn."""
    need_gpu()
    lens, H, Hk, dk, dv = [700, 64, 1300], 4, 2, 128, 128
    d, _, cu = make(13, lens, H, Hk, dk, dv, "bf16")
    e, _, _ = make(14, lens, H, Hk, dk, dv, "bf16")

    def call(x):
        o, sf = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["g"], cu, x["s0"], scale=0.1)
        gr = kda.kda_linear_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], cu, x["s0"], x["dS"], scale=0.1)
        od, sd = kda.kda_linear_decode(x["q"][:3], x["k"][:3], x["v"][:3], x["g"][:3], sf, scale=0.1)
        return [o, sf, od, sd] + [gr[n] for n in ("dq", "dk", "dv", "dg", "dS0")]

    want, other = call(d), call(e)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, call(d)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got2 = call(e)
    got1 = call(d)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got1)) and all(torch.equal(a, b) for a, b in zip(other, got2))
    x = {n: t.clone() for n, t in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(x)
    for rep, (src, ref_) in enumerate(((d, want), (e, other), (d, want), (d, want))):
        for n in x:
            x[n].copy_(src[n])
        junk = torch.randn(1 << 20, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        assert all(torch.equal(a, b) for a, b in zip(outs, ref_)), rep


def test_captured_autograd():
    """kda_linear and its backward in a graph: every replay equals the eager call, with eager calls in between."""
    need_gpu()
    lens = [300, 41]
    d, _, cu = make(17, lens, 4, 2, 64, 64, "bf16")
    e, _, _ = make(18, lens, 4, 2, 64, 64, "bf16")
    names = ("q", "k", "v", "g", "s0")

    def call(x, up):
        leaves = [x[n].detach().requires_grad_(True) for n in names]
        o, sf = kda.kda_linear(*leaves[:4], cu, leaves[4], scale=0.125)
        return [o.detach(), sf.detach()] + list(torch.autograd.grad([o, sf], leaves, up))

    up = [d["dO"].float(), d["dS"]]
    want = {id(x): call(x, up) for x in (d, e)}
    x = {n: d[n].clone() for n in names}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x, up)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(x, up)
    for src in (d, e, e, d):
        for n in names:
            x[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[id(src)]))
        assert all(torch.equal(a, b) for a, b in zip(call(src, up), want[id(src)]))
