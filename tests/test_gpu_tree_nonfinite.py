"""Infinite and very large states under a drafted tree: what the recurrence keeps finite or
infinite stays so, and other columns are what they were."""
import numpy as np
import pytest

import linear_ref as ref

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda
from test_gpu_tree import STEPS, bound, host, make

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [9, 40])
def test_infinite_and_largest_states(dtype, L):
    """Linear rule: o of a column with one infinity is that times q's sign, and one of fp32's largest values times a small
    q is a number, 2^-16 of which (two bf16 terms a side) and 512 half steps it may be off."""
    need_gpu()
    N, H, dk, dv = 2, 2, 64, 64
    d, h, rng = make(40, N, L, H, H, dk, dv, dtype, "linear", strength=-4.0)
    parent = [ref.random_tree(rng, L, 6) for _ in range(N)]
    par = torch.tensor(parent, dtype=torch.int32, device="cuda")
    clean = kda.kda_tree(d["q"], d["k"], d["v"], d["g"], None, par, d["s0"], scale=2.0 ** -10)
    for value in (INF, -INF, 3.4028e38, -3.4e38):
        print(f"[gpu-tree] state {value} {dtype}", flush=True)
        s, hs = d["s0"].clone(), h["s0"].copy()
        s[1, 1, 7, 5] = value
        hs[1, 1, 7, 5] = float(s[1, 1, 7, 5])
        o = kda.kda_tree(d["q"], d["k"], d["v"], d["g"], None, par, s, scale=2.0 ** -10)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            r, _ = ref.tree(h["q"], h["k"], h["v"], h["g"], None, parent, hs, 2.0 ** -10)
            M, _ = bound(dict(h, s0=hs), parent, 2.0 ** -10)
        x = host(o)
        same = np.ones(x.shape, bool)
        same[1, :, 1, 5] = False
        assert np.array_equal(x[same], host(clean)[same])
        y, ry, My = x[1, :, 1, 5], r[1, :, 1, 5], M[1, :, 1, 5]
        if np.isinf(value):
            assert np.isinf(ry).all() and np.array_equal(y, ry)
        else:
            assert np.isfinite(ry).all() and np.isfinite(y).all()
            assert (np.abs(y - ry) <= (STEPS + (3 * 2.0 ** -16 if dtype == "bf16" else 0)) * My).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norms_of_tiny_keys_and_queries(dtype):
    """eps = 0 and vectors of 1e-20, whose squares are below fp32's smallest normal number (about 2^-126): 64 of them add up
    in steps of 2^-149, so that a norm of 2^-127 and more is off by at most 64 * 2^-23 of itself, beside the bounds of
    tests/test_gpu_tree.py; tree and commit agree with decode steps."""
    need_gpu()
    N, L, H, d = 2, 7, 2, 64
    dev, h, rng = make(41, N, L, H, H, d, d, dtype, "delta")
    for n in ("q", "k"):
        dev[n] = (dev[n].float() * 1e-20).to(dev[n].dtype)
        h[n] = host(dev[n])
    parent = [list(range(-1, L - 1))] * N
    par = torch.tensor(parent, dtype=torch.int32, device="cuda")
    print(f"[gpu-tree] tiny keys {dtype}", flush=True)
    o = kda.kda_tree(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], par, dev["s0"], eps=0.0)
    acc = torch.full((N,), L - 1, dtype=torch.int32, device="cuda")
    c = kda.kda_tree_commit(dev["k"], dev["v"], dev["g"], dev["beta"], par, acc, dev["s0"], eps=0.0)
    s, outs = dev["s0"].clone(), []
    for t in range(L):
        x = [dev[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")]
        ot, s = kda.kda_decode(*x, s, out_state=s, eps=0.0)
        outs.append(ot)
    torch.cuda.synchronize()
    r, states = ref.tree(h["q"], h["k"], h["v"], h["g"], h["beta"], parent, h["s0"], eps=0.0)
    # the bound's own recurrence has eps = 1e-6: the same vectors at an ordinary size give the same directions
    M, Ms = bound(dict(h, q=h["q"] * 1e20, k=h["k"] * 1e20), parent, 1.0)
    tiny = 64 * 2.0 ** -23
    rel = STEPS + (3 * 2.0 ** -16 if dtype == "bf16" else 0) + L * 4 * tiny
    assert np.isfinite(host(o)).all() and (np.abs(host(o) - r) <= rel * M).all()
    assert (np.abs(host(o) - np.stack([host(x) for x in outs], 1)) <= rel * M).all()
    last = np.stack([states[n][L - 1] for n in range(N)])
    Ml = np.stack([Ms[n][L - 1] for n in range(N)])
    assert (np.abs(host(c) - last) <= (STEPS + L * 4 * tiny) * Ml).all()
    assert (np.abs(host(c) - host(s)) <= (STEPS + L * 4 * tiny) * Ml).all()
