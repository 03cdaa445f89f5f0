"""64-bit references of the linear rule and of drafted trees, token by token in
numpy, and the error bounds the GPU tests use.

Bounds.  Every output is a sum of products; M is the same sum with the absolute
value of every input, so rounding each term by a relative r moves an output by
at most r M.  One rounding is half a step: 2^-24 in fp32, 2^-8 in bf16.  A sum
of n fp32 terms in any order adds at most n half steps.  That bound holds for
every element and is wide.  Beside it stands one for the whole output: roundings
of independent terms add in squares, so with V the sum of the squared terms (the
same recurrence on squared inputs, with twice the gates) an output is off by
about r sqrt(V), and by sqrt(n) half steps of sqrt(V) for a sum of n terms.
"""
import numpy as np

F32, BF16 = 2.0 ** -24, 2.0 ** -8


def linear_fwd(q, k, v, g, lens, s0=None, scale=1.0):
    """q, k [T, Hk, dk], v [T, H, dv], g [T, H] or [H] -> (o [T, H, dv], final [N, H, dk, dv], states [T, ...])."""
    T, H, dv = v.shape
    R, dk = H // q.shape[1], q.shape[2]
    q, k = (np.repeat(x.astype(np.float64), R, 1) for x in (q, k))
    a = np.exp(np.broadcast_to(g.astype(np.float64), (T, H)))
    o, states, final = np.zeros((T, H, dv)), np.zeros((T, H, dk, dv)), np.zeros((len(lens), H, dk, dv))
    t = 0
    for n, length in enumerate(lens):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[n].astype(np.float64)
        for _ in range(length):
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t].astype(np.float64)[:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
            states[t] = S
            t += 1
        final[n] = S
    return o, final, states


def linear_bwd(q, k, v, g, lens, dO, s0=None, dSf=None, scale=1.0):
    T, H, dv = v.shape
    Hk, dk = q.shape[1:]
    R = H // Hk
    _, _, states = linear_fwd(q, k, v, g, lens, s0, scale)
    qe, ke = (np.repeat(x.astype(np.float64), R, 1) for x in (q, k))
    a = np.exp(np.broadcast_to(g.astype(np.float64), (T, H)))
    v, dO = v.astype(np.float64), dO.astype(np.float64)
    dq, dk_, dv_, dg = np.zeros((T, H, dk)), np.zeros((T, H, dk)), np.zeros((T, H, dv)), np.zeros((T, H))
    dS0 = np.zeros((len(lens), H, dk, dv))
    t0 = 0
    for n, length in enumerate(lens):
        dS = np.zeros((H, dk, dv)) if dSf is None else dSf[n].astype(np.float64)
        first = np.zeros((H, dk, dv)) if s0 is None else s0[n].astype(np.float64)
        for t in reversed(range(t0, t0 + length)):
            dS = dS + scale * qe[t][:, :, None] * dO[t][:, None, :]
            dq[t] = scale * np.einsum("hkv,hv->hk", states[t], dO[t])
            dk_[t] = np.einsum("hkv,hv->hk", dS, v[t])
            dv_[t] = np.einsum("hkv,hk->hv", dS, ke[t])
            before = states[t - 1] if t > t0 else first
            dg[t] = a[t] * (dS * before).sum((1, 2))
            dS = a[t][:, None, None] * dS
        dS0[n] = dS
        t0 += length
    dq, dk_ = (x.reshape(T, Hk, R, dk).sum(2) for x in (dq, dk_))
    return {"dq": dq, "dk": dk_, "dv": dv_, "dg": dg.sum(0) if g.ndim == 1 else dg, "dS0": dS0}


def absolute(*xs):
    return [None if x is None else np.abs(x) for x in xs]


def squared(*xs):
    return [None if x is None else x * x for x in xs]


def step(S, q, k, v, g, beta, scale=1.0, eps=1e-6):
    """One token of one sequence: S [H, dk, dv], q, k [H, dk], v [H, dv]; beta [H] for the delta rule, else None."""
    q, k, v = (None if x is None else x.astype(np.float64) for x in (q, k, v))
    if beta is not None:
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
        q = None if q is None else q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        S = np.exp(g.astype(np.float64))[:, :, None] * S
        b = 1.0 / (1.0 + np.exp(-beta.astype(np.float64)))
        v = b[:, None] * (v - np.einsum("hk,hkv->hv", k, S))
    else:
        S = np.exp(g.astype(np.float64))[:, None, None] * S
    S = S + k[:, :, None] * v[:, None, :]
    return (None if q is None else scale * np.einsum("hk,hkv->hv", q, S)), S


def tree(q, k, v, g, beta, parent, s0, scale=1.0, eps=1e-6):
    """o [N, L, H, dv] and the state after every node [N, L, H, dk, dv] (None for absent nodes)."""
    N, L, H, dv = v.shape
    dk = k.shape[3]
    R = H // k.shape[2]
    o, states = np.zeros((N, L, H, dv)), [[None] * L for _ in range(N)]
    for n in range(N):
        for i in range(L):
            p = parent[n][i]
            if p < -1 or p >= i or (p >= 0 and states[n][p] is None):
                continue
            S = states[n][p] if p >= 0 else (np.zeros((H, dk, dv)) if s0 is None else s0[n].astype(np.float64))
            gi = g if g.ndim == 1 else g[n, i]
            o[n, i], states[n][i] = step(S, np.repeat(q[n, i], R, 0), np.repeat(k[n, i], R, 0), v[n, i], gi,
                                         None if beta is None else beta[n, i], scale, eps)
    return o, states


def random_tree(rng, L, depth, roots=1):
    """parent [L] of a random tree with `roots` first nodes hanging on the state and paths of at most `depth` nodes."""
    parent, d = [], []
    for i in range(L):
        p = -1 if i < roots else int(rng.integers(-1, i))
        if p >= 0 and d[p] >= depth:
            p = parent[p]
        parent.append(p)
        d.append(1 if p < 0 else d[p] + 1)
    return parent
