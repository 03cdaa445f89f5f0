"""Trees of drafted tokens (kda_tree, kda_tree_commit) against the 64-bit token
recurrence along every path (tests/linear_ref.py).

Tolerances.  Linear rule: sums of non-negative terms in the bound M of
linear_ref (the recurrence on absolute values): the state product in two bf16
terms each (2^-16 of M, three products) or fp32, and fp32 sums of at most
dk + 64 terms: 512 half steps.  Delta rule: u is a difference, so M is the
recurrence with every minus turned to plus (v + S kh in place of v - S kh),
which bounds each path's terms; the norms, sigmoid and factors e^g add a few
half steps to each: 1024 in all.  A state needs no bf16 term: 1024 fp32 steps.
Over a whole output the roundings of independent terms add in squares: the
error's norm is at most sqrt(1024) = 32 half steps (and the 3 * 2^-16 of the
split product) of the output's own norm, twice for the delta rule's differences.
"""
import numpy as np
import pytest

import linear_ref as ref
from linear_ref import BF16, F32

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu

STEPS = 1024 * F32


def _say(msg):
    print(f"[gpu-tree] {msg}", flush=True)


def host(t):
    return t.detach().double().cpu().numpy()


def make(seed, N, L, H, Hk, dk, dv, dtype, rule, gate="token", strength=-2.0, s0=True):
    rng = np.random.default_rng([99, seed])
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rounded(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt)

    x = {"q": rounded(N, L, Hk, dk), "k": rounded(N, L, Hk, dk), "v": rounded(N, L, H, dv)}
    shape = (N, L, H, dk) if rule == "delta" else (H,) if gate == "head" else (N, L, H)
    x["g"] = torch.from_numpy(-np.log1p(np.exp(rng.standard_normal(shape) + strength)).astype(np.float32))
    x["g"] = x["g"].to(dt) if rule == "delta" else x["g"]
    x["beta"] = rounded(N, L, H) if rule == "delta" else None
    x["s0"] = torch.from_numpy((0.3 * rng.standard_normal((N, H, dk, dv))).astype(np.float32)) if s0 else None
    return ({n: None if t is None else t.cuda() for n, t in x.items()},
            {n: None if t is None else t.float().numpy().astype(np.float64) for n, t in x.items()}, rng)


def bound(h, parent, scale):
    """The recurrence with absolute values and every minus a plus: a bound of the sums behind each output."""
    a = dict(h)
    for n in ("q", "k", "v", "s0"):
        a[n] = None if h[n] is None else np.abs(h[n])
    if h["beta"] is None:
        return ref.tree(a["q"], a["k"], a["v"], a["g"], None, parent, a["s0"], abs(scale))
    N, L, H, dv = a["v"].shape
    dk = a["k"].shape[3]
    o, states = np.zeros((N, L, H, dv)), [[None] * L for _ in range(N)]
    k, q = (x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (a["k"], a["q"]))
    b = 1 / (1 + np.exp(-a["beta"]))
    for n in range(N):
        for i in range(L):
            p = parent[n][i]
            if p < -1 or p >= i or (p >= 0 and states[n][p] is None):
                continue
            S = states[n][p] if p >= 0 else (np.zeros((H, dk, dv)) if a["s0"] is None else a["s0"][n])
            S = np.exp(a["g"][n, i])[:, :, None] * S
            u = b[n, i][:, None] * (a["v"][n, i] + np.einsum("hk,hkv->hv", k[n, i], S))
            S = S + k[n, i][:, :, None] * u[:, None, :]
            o[n, i], states[n][i] = abs(scale) * np.einsum("hk,hkv->hv", q[n, i], S), S
    return o, states


def check(name, x, r, M, rel, stored=0.0):
    x = host(x)
    assert np.isfinite(x).all(), name
    if x.size:
        off, most = np.linalg.norm(x - r), (2 * (rel - STEPS + 32 * F32) + stored) * np.linalg.norm(r)
        _say(f"  {name}: the error's norm is {off / max(most, 1e-300):.3f} of its bound")
        assert off <= most, name
    worst = float((np.abs(x - r) / (rel * M + stored * np.abs(r) + 1e-30)).max()) if x.size else 0.0
    _say(f"  {name}: largest error is {worst:.3f} of its bound")
    assert worst <= 1.0, name


def check_tree(d, h, parent, dtype, scale, outs=(torch.float32, torch.bfloat16), accept=None):
    par = torch.tensor(parent, dtype=torch.int32, device="cuda")
    r, states = ref.tree(h["q"], h["k"], h["v"], h["g"], h["beta"], parent, h["s0"], scale)
    M, Ms = bound(h, parent, scale)
    rel = STEPS + (3 * 2.0 ** -16 if dtype == "bf16" else 0)
    for out in outs:
        o = kda.kda_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], par, d["s0"], out_dtype=out, scale=scale)
        torch.cuda.synchronize()
        assert o.dtype == out
        check("o", o, r, M, rel, BF16 if out == torch.bfloat16 else 0)
    N = len(parent)
    for acc in accept or []:
        a = torch.tensor(acc, dtype=torch.int32, device="cuda")
        s = kda.kda_tree_commit(d["k"], d["v"], d["g"], d["beta"], par, a, d["s0"])
        zero = np.zeros(tuple(s.shape[1:]))
        want, size = [], []
        for n in range(N):
            i = acc[n]
            ok = 0 <= i < len(parent[n]) and states[n][i] is not None
            base = zero if h["s0"] is None else h["s0"][n]
            want.append(states[n][i] if ok else base)
            size.append(Ms[n][i] if ok else np.abs(base) * 0)
        torch.cuda.synchronize()
        check(f"state {acc}", s, np.stack(want), np.stack(size), STEPS)
        if d["s0"] is not None:
            s2 = d["s0"].clone()
            assert kda.kda_tree_commit(d["k"], d["v"], d["g"], d["beta"], par, a, s2, out_state=s2) is s2
            torch.cuda.synchronize()
            assert torch.equal(s, s2)
    return r


CASES = [
    # rule, N, L, depth, H, Hk, dk, dv, dtype, gate
    ("delta", 1, 1, 1, 1, 1, 64, 64, "f32", "token"),
    ("delta", 2, 8, 4, 3, 3, 128, 128, "bf16", "token"),
    ("delta", 3, 16, 16, 2, 2, 128, 64, "f32", "token"),
    ("delta", 2, 17, 5, 2, 2, 64, 128, "bf16", "token"),
    ("delta", 2, 33, 9, 2, 2, 128, 128, "f32", "token"),
    ("delta", 2, 64, 8, 2, 2, 128, 128, "bf16", "token"),
    ("delta", 1, 64, 64, 1, 1, 64, 64, "bf16", "token"),
    ("delta", 1, 61, 7, 1, 1, 128, 64, "bf16", "token"),
    ("linear", 1, 1, 1, 2, 1, 128, 128, "bf16", "head"),
    ("linear", 3, 7, 3, 4, 2, 64, 64, "f32", "token"),
    ("linear", 2, 32, 6, 4, 1, 128, 128, "bf16", "token"),
    ("linear", 2, 50, 20, 2, 2, 128, 64, "f32", "head"),
    ("linear", 2, 64, 6, 2, 1, 64, 128, "bf16", "token"),
    ("linear", 2, 25, 4, 2, 2, 128, 64, "bf16", "token"),
]


@pytest.mark.parametrize("rule,N,L,depth,H,Hk,dk,dv,dtype,gate", CASES)
def test_tree_and_commit(rule, N, L, depth, H, Hk, dk, dv, dtype, gate):
    need_gpu()
    _say(f"{rule} N={N} L={L} depth={depth} H={H}/{Hk} {dk}x{dv} {dtype} {gate}")
    d, h, rng = make(1, N, L, H, Hk, dk, dv, dtype, rule, gate)
    parent = [ref.random_tree(rng, L, depth) for _ in range(N)]
    accept = [[L - 1] * N, [int(rng.integers(0, L)) for _ in range(N)], [-1] * N]
    check_tree(d, h, parent, dtype, 0.7, accept=accept)


@pytest.mark.parametrize("rule", ["delta", "linear"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shapes_of_trees(rule, dtype):
    """A chain of 64 (every node the ancestor of all later ones), 64 roots, a star, and no state."""
    need_gpu()
    L = 64
    chain, roots, star = list(range(-1, L - 1)), [-1] * L, [-1] + [0] * (L - 1)
    d, h, _ = make(2, 3, L, 1, 1, 64, 64, dtype, rule, strength=-3.0)
    _say(f"chain, roots, star: {rule} {dtype}")
    check_tree(d, h, [chain, roots, star], dtype, 1.0, accept=[[63, 63, 63], [40, 0, 5]])
    d["s0"] = h["s0"] = None
    check_tree(d, h, [star, chain, roots], dtype, 1.0, accept=[[63, 20, 1]])


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_absent_nodes_and_bad_parents(rule):
    """Absent nodes (their inputs NaN) give 0 and touch nothing; a parent that is not before its child, out of range or
    absent makes the node absent; an accept outside the tree or of an absent node copies the state."""
    need_gpu()
    N, L, H = 4, 20, 2
    d, h, rng = make(3, N, L, H, H, 64, 64, "f32", rule)
    parent = [ref.random_tree(rng, L, 5) for _ in range(N)]
    parent[0][12:] = [-2] * 8
    parent[1] = [-5] * L
    parent[2][4], parent[2][5], parent[2][6] = 4, 9, 1 << 30
    parent[2][7], parent[2][8] = 4, 7          # children of an absent node
    parent[3][0] = -(1 << 31)
    parent[3][1:] = [0] * 10 + [-1] * 9
    r, states = ref.tree(h["q"], h["k"], h["v"], h["g"], h["beta"], parent, h["s0"], 1.0)
    gone = torch.tensor([[s is None for s in row] for row in states], device="cuda")
    assert int(gone.sum()) >= 8 + L + 5 + 11
    for n in ("q", "k", "v", "g", "beta"):
        if d[n] is not None:
            d[n][gone] = float("nan")
    o_ref = check_tree(d, h, parent, "f32", 1.0, accept=[[11, 3, 3, 19], [12, L, 8, 0], [-1, -7, 1 << 30, -(1 << 31)]])
    o = kda.kda_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], torch.tensor(parent, dtype=torch.int32, device="cuda"), d["s0"])
    assert bool((o[gone] == 0).all()) and o_ref.shape == tuple(o.shape)
    s = kda.kda_tree_commit(d["k"], d["v"], d["g"], d["beta"], torch.tensor(parent, dtype=torch.int32, device="cuda"),
                            torch.tensor([12, L, 8, 0], dtype=torch.int32, device="cuda"), d["s0"])
    assert torch.equal(s, d["s0"])


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_strong_and_infinite_gates(rule):
    need_gpu()
    N, L, H = 2, 40, 2
    for dtype in ("f32", "bf16"):
        d, h, rng = make(4, N, L, H, H, 64, 64, dtype, rule)
        g = h["g"].astype(np.float32)
        g[:, ::3] = -8.0
        g[:, 7], g[:, 11] = -np.inf, -200.0
        if rule == "delta":
            g[:, 20, :, ::2] = 0.0
        d["g"] = torch.from_numpy(g).to(d["g"].dtype).cuda()
        h["g"] = np.maximum(g.astype(np.float64), -1e3)
        chain = list(range(-1, L - 1))
        check_tree(d, h, [chain, ref.random_tree(rng, L, 9)], dtype, 1.0, accept=[[L - 1, L - 1], [10, 13]])


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_long_offsets(rule):
    """More than 2^31 elements of state: the last sequence as in a call of its own."""
    need_gpu()
    N, L, H, d = 530, 3, 256, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn((N, L, H, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    g = -torch.rand((N, L, H, d) if rule == "delta" else (N, L, H), generator=gen, device="cuda")
    g = g.bfloat16() if rule == "delta" else g
    beta = torch.randn((N, L, H), generator=gen, device="cuda").bfloat16() if rule == "delta" else None
    s = torch.randn((N, H, d, d), generator=gen, device="cuda")
    par = torch.tensor([[-1, 0, 0]] * N, dtype=torch.int32, device="cuda")
    acc = torch.full((N,), 2, dtype=torch.int32, device="cuda")
    last = [None if x is None else x[-1:].clone() for x in (q, k, v, g, beta, par, acc, s)]
    _say(f"long offsets {rule}")
    want = kda.kda_tree(*last[:6], last[7]), kda.kda_tree_commit(*last[1:])
    o = kda.kda_tree(q, k, v, g, beta, par, s)
    assert kda.kda_tree_commit(k, v, g, beta, par, acc, s, out_state=s) is s
    torch.cuda.synchronize()
    assert torch.equal(o[-1:], want[0]) and torch.equal(s[-1:], want[1])


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_chain_equals_decode_steps(rule):
    """A chain's outputs and committed states are those of one decode step per token."""
    need_gpu()
    N, L, H = 3, 12, 4
    d, h, _ = make(5, N, L, H, H, 128, 128, "bf16", rule)
    parent = [list(range(-1, L - 1))] * N
    par = torch.tensor(parent, dtype=torch.int32, device="cuda")
    o = kda.kda_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], par, d["s0"])
    M, Ms = bound(h, parent, 1.0)
    s = d["s0"].clone()
    for t in range(L):
        x = [d[n][:, t].contiguous() for n in ("q", "k", "v", "g")]
        if rule == "delta":
            ot, s = kda.kda_decode(*x, d["beta"][:, t].contiguous(), s, out_state=s)
        else:
            ot, s = kda.kda_linear_decode(*x, s, out_state=s)
        check(f"node {t}", o[:, t], host(ot), M[:, t], STEPS + 3 * 2.0 ** -16)
        a = torch.full((N,), t, dtype=torch.int32, device="cuda")
        c = kda.kda_tree_commit(d["k"], d["v"], d["g"], d["beta"], par, a, d["s0"])
        check(f"state {t}", c, host(s), np.stack([Ms[n][t] for n in range(N)]), STEPS)


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_prefill_draft_commit_decode(rule):
    """The operators as a server strings them together, per round: outputs of a drafted tree, the accepted path
    committed in place, a decode step; against the recurrence over each sequence's accepted tokens."""
    need_gpu()
    lens, L, H, dk, dv, rounds = [70, 1, 131], 9, 2, 128, 128, 3
    N, T = len(lens), sum(lens)
    rng = np.random.default_rng(6)
    pre, hp, _ = make(6, 1, T, H, H, dk, dv, "bf16", rule, s0=False)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = [pre[n][0].contiguous() for n in ("q", "k", "v", "g")]
    if rule == "delta":
        _, s, _ = kda.kda_fwd(*x, pre["beta"][0].contiguous(), cu)
    else:
        _, s = kda.kda_linear_fwd(*x, cu)
    # from here the recurrence starts from the prefill's own state: the prefill has its own tests
    S, B = [list(host(s)), list(np.abs(host(s)))]
    for rnd in range(rounds):
        d, h, _ = make(7 + rnd, N, L, H, H, dk, dv, "bf16", rule, s0=False)
        h["s0"] = np.stack(S)
        parent = [ref.random_tree(rng, L, 4) for _ in range(N)]
        accept = [int(rng.integers(-1, L)) for _ in range(N)]
        par, acc = (torch.tensor(y, dtype=torch.int32, device="cuda") for y in (parent, accept))
        before = s.clone()
        o = kda.kda_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], par, s)
        assert torch.equal(s, before)
        s = kda.kda_tree_commit(d["k"], d["v"], d["g"], d["beta"], par, acc, s, out_state=s)
        r, states = ref.tree(h["q"], h["k"], h["v"], h["g"], h["beta"], parent, h["s0"])
        M, Ms = bound(dict(h, s0=np.stack(B)), parent, 1.0)
        check(f"round {rnd} o", o, r, M, STEPS + 3 * 2.0 ** -16)
        S = [states[n][a] if a >= 0 else S[n] for n, a in enumerate(accept)]
        B = [Ms[n][a] if a >= 0 else B[n] for n, a in enumerate(accept)]
        y, hy, _ = make(20 + rnd, N, 1, H, H, dk, dv, "bf16", rule, s0=False)
        tok = [y[n][:, 0].contiguous() for n in ("q", "k", "v", "g")]
        if rule == "delta":
            o, s = kda.kda_decode(*tok, y["beta"][:, 0].contiguous(), s, out_state=s)
        else:
            o, s = kda.kda_linear_decode(*tok, s, out_state=s)
        r, states = ref.tree(hy["q"], hy["k"], hy["v"], hy["g"], hy["beta"], [[-1]] * N, np.stack(S))
        M, Ms = bound(dict(hy, s0=np.stack(B)), [[-1]] * N, 1.0)
        check(f"round {rnd} token", o[:, None], r, M, STEPS)
        S, B = [states[n][0] for n in range(N)], [Ms[n][0] for n in range(N)]
        check(f"round {rnd} state", s, np.stack(S), np.stack(B), STEPS)


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_repeatable_graph_streams_and_empty(rule):
    need_gpu()
    N, L, H = 6, 40, 4
    d, _, rng = make(8, N, L, H, H, 128, 128, "bf16", rule)
    e, _, _ = make(9, N, L, H, H, 128, 128, "bf16", rule)
    for x in (d, e):
        x["parent"] = torch.tensor([ref.random_tree(rng, L, 7) for _ in range(N)], dtype=torch.int32, device="cuda")
        x["accept"] = torch.tensor([int(rng.integers(-1, L)) for _ in range(N)], dtype=torch.int32, device="cuda")

    def call(x):
        o = kda.kda_tree(x["q"], x["k"], x["v"], x["g"], x["beta"], x["parent"], x["s0"])
        s = kda.kda_tree_commit(x["k"], x["v"], x["g"], x["beta"], x["parent"], x["accept"], x["s0"])
        return o, s

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
    assert all(torch.equal(a, b) for a, b in zip(want + other, got1 + got2))
    x = {n: None if t is None else t.clone() for n, t in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(x)
    for src, ref_ in ((d, want), (e, other), (d, want)):
        for n in x:
            if x[n] is not None:
                x[n].copy_(src[n])
        torch.randn(1 << 20, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref_))
    z = {n: None if t is None else t[:0] for n, t in d.items()}
    o, s = call(z)
    torch.cuda.synchronize()
    assert o.shape[0] == 0 and s.shape[0] == 0
