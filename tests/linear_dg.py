"""Inputs, 64-bit gradient and tolerances of the linear rule's dg, shared by the GPU
test and by the check that those tolerances tell a wrong dg from a right one.

dg_t = e^{g_t} <dS_t, S_{t-1}>: over the pairs of a query i >= t (or the final state)
and a key j < t (or the initial state) it sums x = (scale q_i k_j decay)(dO_i v_j).
With V_t the sum of x^2 over the pairs and channels (the recurrence on squared inputs
with twice the gates), which is also about dg_t^2 where the inputs are independent:
  * bf16 inputs: the block's S and dS are rounded to bf16 once each, so an element of
    one of them moves dg_t by at most 2^-8 of what it carries: 2 * 2^-8 sqrt(V_t);
  * fp32 sums: sqrt(1024) half steps of sqrt(V_t), and as much of everything that the
    row and column sums of the token's own 128-token block hold, which cancel:
    B_t = sum over the block's queries of q . dq on squared inputs;
  * a dg stored in bf16: 2^-8 of the value.
The norm of the error over an output is at most these times the root of the summed V
and B.  A single element is a sum of many independent roundings, none larger than its
part: it passes six times its root with a probability of at most 2 e^-18 (Hoeffding).
A gate per head sums dg_t over the tokens: within a block they share S and dS, so the
roots add up there, and squares from block to block.
"""
import numpy as np

import linear_ref as ref
from linear_ref import BF16, F32

BLOCK, ROOT = 128, 32 * F32

CASES = [
    # lens, H, Hk, dk, dv, gate, initial and final states
    ([5, 64, 65], 3, 3, 64, 128, "head", True),
    ([0, 63, 0, 128, 1, 0], 2, 2, 128, 64, "token", True),
    ([127, 128, 129, 1, 30], 4, 2, 128, 128, "token", True),
    ([257, 3], 6, 2, 64, 64, "token", True),
    ([200], 4, 1, 128, 64, "head", True),
    ([130, 40], 2, 2, 128, 128, "token", True),
    ([33, 95, 2], 3, 1, 64, 128, "token", True),
    ([1500, 1730], 2, 1, 64, 64, "token", True),     # in segments from here on
    ([0, 3, 2600, 130, 0, 1024, 0], 1, 1, 64, 64, "head", True),
    ([1100, 64], 2, 2, 128, 128, "token", False),
    ([300, 900], 7, 1, 64, 64, "token", True),       # seven value heads to a key head
]


def rounded_to_bf16(x):
    """Round to nearest even, kept as float32."""
    u = x.astype(np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def make(seed, lens, H, Hk, dk, dv, dtype, gate, states):
    """float32 arrays, exact in `dtype`; s0 and dS are None without states.  Gates of about -0.004 a token leave about
    half of a state after a block, and the states are as large as a document makes them: what crosses a block counts."""
    rng = np.random.default_rng([78, seed])
    T, N = int(sum(lens)), len(lens)
    x = {n: rng.standard_normal(s).astype(np.float32)
         for n, s in (("q", (T, Hk, dk)), ("k", (T, Hk, dk)), ("v", (T, H, dv)), ("dO", (T, H, dv)))}
    if dtype == "bf16":
        x = {n: rounded_to_bf16(a) for n, a in x.items()}
    x["g"] = -np.log1p(np.exp(rng.standard_normal((H,) if gate == "head" else (T, H)) - 6.0)).astype(np.float32)
    for n in ("s0", "dS"):
        x[n] = (5.0 * rng.standard_normal((N, H, dk, dv))).astype(np.float32) if states else None
    return x


def _blocks(lens):
    at = 0
    for length in lens:
        for lo in range(at, at + length, BLOCK):
            yield slice(lo, min(lo + BLOCK, at + length))
        at += length


class Tolerance:
    """The gradient `r`, and what an output may be off by."""

    def __init__(self, x, lens, dtype, scale):
        h = {n: None if a is None else a.astype(np.float64) for n, a in x.items()}
        R = h["v"].shape[1] // h["q"].shape[1]
        for n in ("q", "k"):
            h[n] = np.repeat(h[n], R, 1)   # a key head for each value head: the same dg, and q . dq of each of them
        T, H = h["v"].shape[:2]
        g = np.broadcast_to(h["g"], (T, H))
        zero = np.zeros((len(lens), H, h["q"].shape[2], h["v"].shape[2]))
        s0, dS = (zero if h[n] is None else h[n] for n in ("s0", "dS"))
        self.tokens = ref.linear_bwd(h["q"], h["k"], h["v"], g, lens, h["dO"], s0, dS, scale)["dg"]
        q, k, v, dO, a, b = ref.squared(h["q"], h["k"], h["v"], h["dO"], s0, dS)
        sq = ref.linear_bwd(q, k, v, 2 * g, lens, dO, a, b, scale ** 2)
        rel = ROOT + (2 * BF16 if dtype == "bf16" else 0.0)
        var = np.zeros((T, H))
        for at in _blocks(lens):
            var[at] = rel ** 2 * sq["dg"][at] + ROOT ** 2 * (q[at] * sq["dq"][at]).sum((0, 2))
        self.per_head = h["g"].ndim == 1
        if self.per_head:
            self.r = self.tokens.sum(0)
            self.var = sum((np.sqrt(var[at]).sum(0) ** 2 for at in _blocks(lens)), np.zeros(H))
        else:
            self.r, self.var = self.tokens, var

    def norm(self, stored=0.0):
        return np.sqrt(self.var.sum()) + stored * np.linalg.norm(self.r)

    def element(self, stored=0.0):
        return 6 * np.sqrt(self.var) + stored * np.abs(self.r) + 1e-30

    def off(self, x, stored=0.0):
        """The error's norm and its largest element, each over its bound."""
        return (float(np.linalg.norm(x - self.r) / self.norm(stored)), float((np.abs(x - self.r) / self.element(stored)).max()))


def crossing(x, lens, scale):
    """The part of every dg_t that goes through both borders of its block: e^{G} <S, dS>, [T, H]."""
    T, H = x["v"].shape[:2]
    R = H // x["q"].shape[1]
    q, k = (np.repeat(x[n].astype(np.float64), R, 1) for n in ("q", "k"))
    v, dO = x["v"].astype(np.float64), x["dO"].astype(np.float64)
    a = np.exp(np.broadcast_to(x["g"].astype(np.float64), (T, H)))
    out, at = np.zeros((T, H)), 0
    for n, length in enumerate(lens):
        zero = np.zeros((H, q.shape[2], v.shape[2]))
        S = zero.copy() if x["s0"] is None else x["s0"][n].astype(np.float64)
        D = zero.copy() if x["dS"] is None else x["dS"][n].astype(np.float64)
        enter, leave = [], []
        blocks = [b for b in _blocks([length])]
        blocks = [slice(b.start + at, b.stop + at) for b in blocks]
        for b in blocks:
            enter.append(S)
            for t in range(b.start, b.stop):
                S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        for b in reversed(blocks):
            leave.append(D)
            for t in reversed(range(b.start, b.stop)):
                D = a[t][:, None, None] * (D + scale * q[t][:, :, None] * dO[t][:, None, :])
        for b, s, d in zip(blocks, enter, reversed(leave)):
            out[b] = a[b].prod(0) * (s * d).sum((1, 2))
        at += length
    return out
