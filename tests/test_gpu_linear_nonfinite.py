"""Infinities and NaN in the linear rule's inputs reach only what depends on them by the
recurrence: not the tokens before (o, dq), nor behind (dk, dv), not other columns, heads
or documents.  The packed calls do not say which of the two such a result is; decode and
commit keep a state's infinities.

The 64-bit reference runs on the same inputs.  Where it is finite, the result has to be
finite and within the bounds of tests/test_gpu_linear.py; where it is not, the result must
not be finite either.  Inside the bad token's 128-token block dg need not be finite.
"""
import numpy as np
import pytest

import linear_ref as ref
from linear_ref import BF16, F32

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda
from test_gpu_linear import STEPS, host, make

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _say(msg):
    print(f"[gpu-nonfinite] {msg}", flush=True)


def check(name, x, r, M, rel):
    x = host(x)
    fine = np.isfinite(r)
    assert np.array_equal(np.isfinite(x), fine), (name, int((np.isfinite(x) != fine).sum()), int((~fine).sum()))
    worst = float((np.abs(x[fine] - r[fine]) / (rel * M[fine] + 1e-30)).max()) if fine.any() else 0.0
    _say(f"  {name}: {int((~fine).sum())} of {fine.size} not finite, largest error of the others {worst:.3f} of its bound")
    assert worst <= 1.0, name
    return x


BAD = [
    # tensor, token, channel or None for a gate, value
    ("v", 0, 3, INF), ("v", 37, 63, -INF), ("v", 63, 0, NAN), ("v", 64, 20, INF), ("v", 100, 7, NAN), ("v", 149, 1, INF),
    ("k", 0, 5, INF), ("k", 20, 63, NAN), ("k", 90, 33, -INF),
    ("q", 3, 9, INF), ("q", 50, 40, NAN), ("q", 127, 0, -INF),
    ("g", 70, None, NAN),
]


def spoiled(d, h, tensor, token, channel, value):
    """The inputs with one value changed, in the last head."""
    d, h = dict(d), dict(h)
    at = (token, d[tensor].shape[1] - 1) + (() if channel is None else (channel,))
    d[tensor], h[tensor] = d[tensor].clone(), h[tensor].copy()
    d[tensor][at] = value
    h[tensor][at] = value
    return d, h


@pytest.mark.parametrize("dtype,H,Hk,dk,dv", [("bf16", 2, 2, 128, 128), ("bf16", 4, 2, 64, 64), ("f32", 2, 1, 64, 128)])
def test_forward(dtype, H, Hk, dk, dv):
    need_gpu()
    lens = [150, 70]
    d, h, cu = make(40, lens, H, Hk, dk, dv, dtype, strength=-3.0)
    clean, clean_final = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=0.125)
    rel = STEPS + (BF16 if dtype == "bf16" else 0)
    for bad in BAD:
        _say(f"forward {dtype} {H}/{Hk} {dk}x{dv}: {bad}")
        e, eh = spoiled(d, h, *bad)
        o, sf = kda.kda_linear_fwd(e["q"], e["k"], e["v"], e["g"], cu, e["s0"], scale=0.125)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            r, rf, _ = ref.linear_fwd(eh["q"], eh["k"], eh["v"], eh["g"], lens, eh["s0"], 0.125)
            M, Mf, _ = ref.linear_fwd(*ref.absolute(eh["q"], eh["k"], eh["v"]), eh["g"], lens, *ref.absolute(eh["s0"]), 0.125)
        check("o", o, r, M, rel)
        check("final", sf, rf, Mf, STEPS)
        # what comes before the token, and what belongs to others, is what it was to the last bit
        t = bad[1]
        assert torch.equal(o[:t], clean[:t]) and torch.equal(o[150:], clean[150:]) and torch.equal(sf[1], clean_final[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_in_segments(dtype):
    """The bad token in a segment of its own sum, in the last one, and in the first."""
    need_gpu()
    lens, H, dk, dv = [1500, 40], 2, 64, 64
    d, h, cu = make(41, lens, H, 1, dk, dv, dtype, strength=-5.0)
    cfg = kda.linear._lib.make_linear_config(H, 1, dk, dv)
    assert kda.linear._lib.kda_linear_fwd_workspace_size(cfg, sum(lens), 2) > 0
    clean, _ = kda.kda_linear_fwd(d["q"], d["k"], d["v"], d["g"], cu, d["s0"], scale=0.125)
    rel = STEPS + (BF16 if dtype == "bf16" else 0)
    for bad in (("v", 5, 3, INF), ("v", 700, 60, -INF), ("v", 1499, 0, NAN), ("k", 300, 2, INF), ("k", 1400, 63, -INF)):
        _say(f"forward in segments {dtype}: {bad}")
        e, eh = spoiled(d, h, *bad)
        o, sf = kda.kda_linear_fwd(e["q"], e["k"], e["v"], e["g"], cu, e["s0"], scale=0.125)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            r, rf, _ = ref.linear_fwd(eh["q"], eh["k"], eh["v"], eh["g"], lens, eh["s0"], 0.125)
            M, Mf, _ = ref.linear_fwd(*ref.absolute(eh["q"], eh["k"], eh["v"]), eh["g"], lens, *ref.absolute(eh["s0"]), 0.125)
        check("o", o, r, M, rel)
        check("final", sf, rf, Mf, STEPS)
        assert torch.equal(o[:bad[1]], clean[:bad[1]]) and torch.equal(o[1500:], clean[1500:])


def check_bwd(e, eh, cu, lens, dtype, bad):
    gr = kda.kda_linear_bwd(e["q"], e["k"], e["v"], e["g"], e["dO"], cu, e["s0"], e["dS"], scale=0.125)
    torch.cuda.synchronize()
    names = ("q", "k", "v", "dO", "s0", "dS")
    with np.errstate(all="ignore"):
        r = ref.linear_bwd(eh["q"], eh["k"], eh["v"], eh["g"], lens, eh["dO"], eh["s0"], eh["dS"], 0.125)
        a = dict(zip(names, ref.absolute(*(eh[n] for n in names))))
        M = ref.linear_bwd(a["q"], a["k"], a["v"], eh["g"], lens, a["dO"], a["s0"], a["dS"], 0.125)
    rel = STEPS + (BF16 if dtype == "bf16" else 0)
    for n in ("dq", "dk", "dv"):
        check(n, gr[n], r[n], M[n], rel)
    check("dS0", gr["dS0"], r["dS0"], M["dS0"], STEPS)
    dg = host(gr["dg"])
    outside = np.ones(dg.shape, bool)
    heads = dg.shape[1] // eh["q"].shape[1] if bad[0] in ("q", "k") else 1   # all that share the last key head
    outside[bad[1] // 128 * 128:bad[1] // 128 * 128 + 128, -heads:] = False
    assert np.array_equal(np.isfinite(dg)[outside], np.isfinite(r["dg"])[outside])
    assert not np.isfinite(dg)[~np.isfinite(r["dg"])].any()
    return gr


@pytest.mark.parametrize("dtype,H,Hk,dk,dv", [("bf16", 2, 2, 128, 128), ("bf16", 4, 2, 64, 64), ("f32", 2, 1, 64, 128)])
def test_backward(dtype, H, Hk, dk, dv):
    need_gpu()
    lens = [150, 70]
    d, h, cu = make(42, lens, H, Hk, dk, dv, dtype, strength=-3.0)
    clean = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125)
    for bad in [b for b in BAD if b[0] != "g"] + [("dO", 0, 1, INF), ("dO", 30, 63, NAN), ("dO", 31, 0, -INF), ("dO", 130, 5, INF)]:
        _say(f"backward {dtype} {H}/{Hk} {dk}x{dv}: {bad}")
        e, eh = spoiled(d, h, *bad)
        gr = check_bwd(e, eh, cu, lens, dtype, bad)
        t = bad[1]
        for n in ("dq", "dk", "dv", "dg"):
            assert torch.equal(gr[n][150:], clean[n][150:]), n
        assert torch.equal(gr["dq"][:t], clean["dq"][:t])
        if bad[0] in ("q", "dO"):
            assert torch.equal(gr["dk"][t + 1:], clean["dk"][t + 1:]) and torch.equal(gr["dv"][t + 1:], clean["dv"][t + 1:])


def test_backward_with_undivided_value_heads():
    """Enough workgroups that each takes all value heads of its key head in turn; the document with the bad value is
    compared with the reference, the others with a clean call."""
    need_gpu()
    length, N, H, Hk, dk, dv = 130, 70, 4, 2, 64, 64
    d, h, cu = make(43, [length] * N, H, Hk, dk, dv, "bf16", strength=-3.0)
    cfg = kda.linear._lib.make_linear_config(H, Hk, dk, dv)
    size = kda.linear._lib.kda_linear_bwd_workspace_size
    alone = kda.linear._lib.make_linear_config(H, H, dk, dv)
    assert size(cfg, length * N, N) == size(alone, length * N, N)   # no partial sums of dq and dk
    clean = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], scale=0.125)
    doc, lo = 33, 33 * length
    rows = slice(lo, lo + length)
    for tensor, token, channel, value in (("k", 17, 3, INF), ("q", 9, 4, NAN), ("dO", 40, 50, INF), ("v", 100, 0, NAN)):
        _say(f"undivided: {tensor} {token}")
        e, eh = spoiled(d, h, tensor, lo + token, channel, value)
        gr = kda.kda_linear_bwd(e["q"], e["k"], e["v"], e["g"], e["dO"], cu, e["s0"], e["dS"], scale=0.125)
        torch.cuda.synchronize()
        one = {n: (t[doc:doc + 1] if n in ("s0", "dS") else t[rows]) for n, t in eh.items()}
        with np.errstate(all="ignore"):
            r = ref.linear_bwd(one["q"], one["k"], one["v"], one["g"], [length], one["dO"], one["s0"], one["dS"], 0.125)
        for n in ("dq", "dk", "dv"):
            assert np.array_equal(np.isfinite(host(gr[n][rows])), np.isfinite(r[n])), n
            assert torch.equal(gr[n][:lo], clean[n][:lo]) and torch.equal(gr[n][lo + length:], clean[n][lo + length:]), n


def test_decode_and_commit_keep_infinities():
    """An infinity in v or the state stays one in the state, beside finite columns."""
    need_gpu()
    d, h, _ = make(44, [1] * 3, 2, 2, 64, 64, "bf16", strength=-3.0)
    for tensor, at, value in (("v", (1, 1, 5), INF), ("s0", (1, 1, 7, 5), -INF), ("k", (2, 1, 9), INF)):
        e, eh = ({n: None if t is None else t.copy() if isinstance(t, np.ndarray) else t.clone() for n, t in x.items()} for x in (d, h))
        e[tensor][at], eh[tensor][at] = value, value
        o, s = kda.kda_linear_decode(e["q"], e["k"], e["v"], e["g"], e["s0"], scale=0.3)
        par, acc = torch.full((3, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
        c = kda.kda_tree_commit(e["k"][:, None], e["v"][:, None], e["g"][:, None], None, par, acc, e["s0"])
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            r, rf, _ = ref.linear_fwd(eh["q"], eh["k"], eh["v"], eh["g"], [1] * 3, eh["s0"], 0.3)
            M, Mf, _ = ref.linear_fwd(*ref.absolute(eh["q"], eh["k"], eh["v"]), eh["g"], [1] * 3, *ref.absolute(eh["s0"]), 0.3)
        check("o", o, r, M, STEPS)
        for x in (s, c):
            y = check("state", x, rf, Mf, 8 * F32)
            assert np.array_equal(y[np.isinf(rf)], rf[np.isinf(rf)])
