"""Performance cases of the operators around the recurrences: the norm with the
residual's addition, the short causal convolution and the selective scan.

``listed()`` names the cases, ``draw(rng)`` gives further ones of the same
ranges, ``prepare(case, seed)`` makes a case's inputs on the GPU and
``run(state)`` is one pass: with ``own`` false in plain torch operations (32
bits), with ``own`` true through the package's entry points.  ``exact(case,
seed)`` is the same result from the definitions in 64 bits, and ``work(case)``
the bytes and operations a pass cannot do without.

The operators:

* norm: s = x + residual, y = s / sqrt(mean(s^2) + eps) * w over each row, in
  the input's type or in 8 bits with a scale a row; its backward;
* conv: y_t = silu(b + sum_j w_j x_{t-W+1+j}) for each channel over packed
  documents, the rows before a document from its state; its backward, and one
  decode step;
* selective: h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t, y_t = (C_t . h_t + D x_t)
  silu(z_t), for each channel with a state of S entries, dt = softplus(raw +
  bias); forward over packed documents, its backward, and one decode step.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


def listed():
    return [
        # a decode step's rows (256 sequences) on their way into an 8-bit product
        dict(op="norm", name="norm_step", dtype="bf16", out="int8", T=256, C=4096),
        # a serving step's packed prompts
        dict(op="norm", name="norm_prompt", dtype="bf16", out="same", T=16411, C=4096),
        # a training step of 4 x 8192 tokens, the residual stream's gradient passing through
        dict(op="norm_bwd", name="norm_train", dtype="bf16", T=32768, C=4096),
        # the next token of 256 sequences: the q, k and v channels of 32 heads of 128
        dict(op="conv_decode", name="conv_step", dtype="bf16", N=256, C=12288, W=4, bias=False),
        # packed prompts of very different lengths, the same channels
        dict(op="conv", name="conv_prompt", dtype="bf16", N=37, T=16411, spread=1.0, C=12288, W=4, bias=False),
        # a small fp32 training step over ragged documents with an odd number of channels
        dict(op="conv_bwd", name="conv_train_short", dtype="f32", N=3, T=1003, spread=1.0, C=333, W=3, bias=True),
        # a training step of 4 x 8192 tokens
        dict(op="conv_bwd", name="conv_train", dtype="bf16", N=4, T=32768, spread=0.0, C=4096, W=4, bias=True),
        # the next token of 256 sequences
        dict(op="sel_decode", name="selective_step", dtype="bf16", N=256, C=4096, S=16, G=1, gated=True),
        # packed prompts of very different lengths
        dict(op="sel", name="selective_prompt", dtype="bf16", N=37, T=16411, spread=1.0, C=4096, S=16, G=1, gated=True),
        # one long prompt of a small layer
        dict(op="sel", name="selective_long", dtype="bf16", N=1, T=131083, spread=0.0, C=512, S=16, G=1, gated=True),
        # a small fp32 training step over ragged documents, channels in two groups
        dict(op="sel_bwd", name="selective_train_short", dtype="f32", N=3, T=1003, spread=1.0, C=200, S=16, G=2, gated=False),
        # a training step of 4 x 4096 tokens
        dict(op="sel_bwd", name="selective_train", dtype="bf16", N=4, T=16384, spread=0.0, C=4096, S=16, G=1, gated=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _channels(rng, lo, hi):
    """Channels over the logarithm of the range, a multiple of 64, of 8 or any number."""
    c, step = _log(rng, lo, hi), rng.choice([64, 64, 8, 1])
    return max(step, c // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "conv", "conv_bwd", "conv_decode", "sel", "sel", "sel_bwd", "sel_bwd", "sel_decode"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    wide = 2 if c["dtype"] == "f32" else 1
    if op in ("norm", "norm_bwd"):
        c["C"] = _channels(rng, 100, 8192)
        c["T"] = _log(rng, 1, min(32768, (1 << 26) // wide // c["C"]))
        if op == "norm":
            c["out"] = rng.choice(["same", "same", "int8", "e4m3"])
        return c
    c["spread"] = rng.choice([0.5, 1.0])
    if op.startswith("conv"):
        c["C"], c["W"], c["bias"] = _channels(rng, 100, 12288), rng.choice([2, 3, 4, 4]), rng.choice([True, False])
        most = (1 << 26) // wide
    else:
        c["C"], c["S"], c["gated"] = _channels(rng, 64, 4096), rng.choice([8, 16, 16, 32]), rng.choice([True, False])
        c["G"] = rng.choice([g for g in (1, 1, 2, 4) if c["C"] % g == 0])
        most = (1 << (29 if op == "sel_bwd" else 30)) // c["S"] // wide
    if op.endswith("decode"):
        del c["spread"]
        c["N"] = _log(rng, 1, 256)
        return c
    c["T"] = _log(rng, 65, min(65536 if op == "sel" else 16384, most // c["C"]))
    c["N"] = min(_log(rng, 1, 64), c["T"])
    return c


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """N document lengths (each >= 1) that add up to T, lognormal with sigma `spread`; part of the case, not of the seed."""
    N, T = case["N"], case["T"]
    if case["spread"] == 0.0:
        return [T // N + (1 if i < T % N else 0) for i in range(N)]
    r = np.random.RandomState(2000 + N + T)
    w = np.exp(r.normal(0.0, case["spread"], N))
    n = 1 + np.floor((T - N) * w / w.sum()).astype(int)
    n[: T - int(n.sum())] += 1
    return [int(x) for x in n]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    op, C = case["op"], case["C"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = {"op": op, "dt": dt}
    rows = case["N"] if op.endswith("decode") else case["T"]
    if op in ("norm", "norm_bwd"):
        # the residual stream's rows differ in size, and some channels stand out
        size = (0.5 * normal(rows, 1)).exp() * (1 + 8 * (uniform(C) > 0.99).float())
        s["w"] = (1 + 0.1 * normal(C)).to(dt)
        s["x"] = normal(rows, C).to(dt)
        if op == "norm":
            s["residual"] = (normal(rows, C) * size).to(dt)
            s["out"] = {"same": dt, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["out"]]
        else:
            s["x"] = (s["x"] * size).to(dt)           # the sum that the forward left
            s["dy"], s["ds"] = normal(rows, C).to(dt), normal(rows, C).to(dt)
        return s
    N = case["N"]
    if not op.endswith("decode"):
        s["lens"] = _lengths(case)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(s["lens"])]), dtype=torch.int32, device="cuda")
    s["x"] = normal(rows, C).to(dt)
    if op.startswith("conv"):
        W = case["W"]
        s["w"] = ((2 * uniform(C, W) - 1) * W ** -0.5).to(dt)
        s["b"] = (0.1 * normal(C)).to(dt) if case["bias"] else None
        s["state"] = normal(N, W - 1, C).to(dt)
        if op == "conv_bwd":
            s["dy"], s["dstate"] = normal(rows, C).to(dt), normal(N, W - 1, C).to(dt)
        return s
    S, G = case["S"], case["G"]
    s["raw"] = (0.5 * normal(rows, C)).to(dt)
    # s["B"] and s["Cm"] write into and read from the states
    step = (math.log(1e-3) + uniform(C) * math.log(100.0)).exp()            # steps of 0.001 to 0.1
    s["bias"] = torch.log(torch.expm1(step))
    s["A"] = -torch.arange(1, S + 1, device="cuda", dtype=torch.float32) * (0.2 * normal(C, S)).exp()
    s["B"], s["Cm"] = normal(rows, G, S).to(dt), normal(rows, G, S).to(dt)
    s["D"] = 1 + 0.1 * normal(C)
    s["z"] = normal(rows, C).to(dt) if case["gated"] else None
    s["h0"] = 0.1 * normal(N, C, S)
    if op == "sel_bwd":
        s["dy"], s["dh"] = normal(rows, C).to(dt), 0.1 * normal(N, C, S)
    return s


# ------------------------------------------------------------------ plain forms: the norm
def _codes(p, amax, most):
    """The row's products in units of its scale: in 64 bits, as many lie next to a border between two codes."""
    return torch.where(amax > 0, p.double() * most / amax, 0.0)


def _e4m3(x):
    """Nearest e4m3 value, ties to even: 4 significant bits, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _plain_norm(s):
    total = (s["x"].float() + s["residual"].float()).to(s["dt"])
    x = total.float()
    rstd = 1 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
    p = x * s["w"].float()
    if s["out"] == s["dt"]:
        return {"y": (p * rstd).to(s["dt"]), "residual": total}
    most = 127.0 if s["out"] == torch.int8 else 448.0
    amax = p.abs().amax(1, keepdim=True)
    code = _codes(p, amax, most)
    code = code.round().float() if s["out"] == torch.int8 else _e4m3(code).float()
    scale = amax * rstd / most
    return {"y": code * scale, "residual": total, "scale": scale[:, 0]}


def _plain_norm_bwd(s):
    x, g = s["x"].float(), s["dy"].float()
    rstd = 1 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
    xh, wg = x * rstd, g * s["w"].float()
    dx = rstd * (wg - xh * (wg * xh).mean(1, keepdim=True)) + s["ds"].float()
    return {"dx": dx.to(s["dt"]), "dw": (g * xh).sum(0, dtype=torch.float64).float()}


# ------------------------------------------------------------------ plain forms: the convolution
def _rows(s):
    """Where row t - W + 1 + j stands among the rows [x, the states' rows]: [T, W]; and each token's document, start and end."""
    T, W = s["x"].shape[0], s["w"].shape[1]
    cu = s["cu"].long()
    t = torch.arange(T, device=cu.device)
    doc = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    start = cu[doc]
    at = t[:, None] - (W - 1) + torch.arange(W, device=cu.device)
    back = at - start[:, None]                                              # below 0: a row of the state
    return torch.where(back >= 0, at, T + doc[:, None] * (W - 1) + (W - 1) + back), doc


def _last_rows(s):
    """Where the rows of the final states stand among the rows [x, the states' rows]: [N, W - 1]."""
    T, W = s["x"].shape[0], s["w"].shape[1]
    cu = s["cu"].long()
    r = torch.arange(W - 1, device=cu.device)
    n = torch.arange(cu.numel() - 1, device=cu.device)
    back = (cu[1:] - cu[:-1])[:, None] - (W - 1) + r
    return torch.where(back >= 0, cu[:-1, None] + back, T + n[:, None] * (W - 1) + (W - 1) + back)


def _pre(s, taps):
    pre = (taps * s["w"].float().t()).sum(1)
    return pre if s["b"] is None else pre + s["b"].float()


def _plain_conv(s):
    ext = torch.cat([s["x"], s["state"].reshape(-1, s["x"].shape[1])])
    pre = _pre(s, ext[_rows(s)[0]].float())
    return (pre * pre.sigmoid()).to(s["dt"]), ext[_last_rows(s)]


def _plain_conv_bwd(s):
    T, C = s["x"].shape
    N, W = s["state"].shape[0], s["w"].shape[1]
    cu = s["cu"].long()
    at, doc = _rows(s)
    taps = torch.cat([s["x"], s["state"].reshape(-1, C)])[at].float()
    pre = _pre(s, taps)
    sig = pre.sigmoid()
    dpre = torch.cat([s["dy"].float() * sig * (1 + pre * (1 - sig)), torch.zeros(1, C, device=pre.device)])
    j = torch.arange(W, device=cu.device)
    to = torch.arange(T, device=cu.device)[:, None] + (W - 1) - j           # the token that reads row t by w_j
    grads = dpre[torch.where(to < cu[doc + 1][:, None], to, T)]
    dx = (grads * s["w"].float().t()).sum(1)
    to = torch.arange(W - 1, device=cu.device)[:, None] - j                 # likewise for the state's rows
    lens = (cu[1:] - cu[:-1])[:, None, None]
    to = torch.where((to >= 0) & (to < lens), cu[:-1, None, None] + to, T)
    dstate = (dpre[to] * s["w"].float().t()).sum(2)
    rows = torch.cat([dx, dstate.reshape(-1, C)])
    last = _last_rows(s).reshape(-1)
    rows[last] = rows[last] + s["dstate"].float().reshape(-1, C)
    dw = (taps * dpre[:T, None]).sum(0, dtype=torch.float64).t().float()
    out = {"dx": rows[:T].to(s["dt"]), "dw": dw, "dstate": rows[T:].reshape(N, W - 1, C).to(s["dt"])}
    if s["b"] is not None:
        out["db"] = dpre[:T].sum(0, dtype=torch.float64).float()
    return out


def _plain_conv_decode(s):
    ext = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = _pre(s, ext.float())
    return (pre * pre.sigmoid()).to(s["dt"]), ext[:, 1:].contiguous()


# ------------------------------------------------------------------ plain forms: the selective scan
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first dimension from zero: pairs first, then the rest between them."""
    T = a.shape[0]
    if T == 1:
        return b
    even = T // 2 * 2
    inner = _scan(a[1:even:2] * a[0:even:2], b[1:even:2] + a[1:even:2] * b[0:even:2])
    h = torch.empty_like(b)
    h[1:even:2] = inner
    h[0] = b[0]
    h[2::2] = b[2::2] + a[2::2] * inner[: (T - 1) // 2]
    return h


def _steps(s):
    """dt, x, B and C for each channel, and the decays, all fp32: [T, C], [T, C], [T, C, S]."""
    C, G = s["x"].shape[1], s["B"].shape[1]
    v = s["raw"].float() + s["bias"]
    dt = torch.where(v > 20, v, torch.log1p(v.clamp(max=20).exp()))
    B, Cc = (s[n].float().repeat_interleave(C // G, 1) for n in ("B", "Cm"))
    return v, dt, s["x"].float(), B, Cc, (dt[..., None] * s["A"]).exp()


def _states(s, u, B, a):
    """All states: every document starts with its own, behind a decay of zero."""
    first = s["cu"][:-1].long()
    b = u[..., None] * B
    b[first] += a[first] * s["h0"]
    cut = a.clone()
    cut[first] = 0
    return _scan(cut, b)


def _plain_sel(s):
    _, dt, x, B, Cc, a = _steps(s)
    h = _states(s, dt * x, B, a)
    y = (h * Cc).sum(2) + s["D"] * x
    if s["z"] is not None:
        y = y * s["z"].float() * s["z"].float().sigmoid()
    return y.to(s["dt"]), h[s["cu"][1:].long() - 1]


def _plain_sel_bwd(s):
    v, dt, x, B, Cc, a = _steps(s)
    T, C = x.shape
    G = s["B"].shape[1]
    first, last = s["cu"][:-1].long(), s["cu"][1:].long() - 1
    h = _states(s, dt * x, B, a)
    dy = s["dy"].float()
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = z.sigmoid()
        out["dz"] = (dy * ((h * Cc).sum(2) + s["D"] * x) * sig * (1 + z * (1 - sig))).to(s["dt"])
        dy = dy * z * sig
    e = dy[..., None] * Cc
    e[last] += s["dh"]
    ahead = torch.cat([a[1:], a[:1]])
    ahead[last] = 0
    e = _scan(ahead.flip(0), e.flip(0)).flip(0)                             # the gradient of every state
    out["dC"] = (h * dy[..., None]).reshape(T, G, C // G, -1).sum(2).to(s["dt"])
    before = torch.cat([h[:1], h[:-1]])
    before[first] = s["h0"]
    through = e * a
    out["dh0"] = through[first]
    through = through * before                                              # the gradient of dt A
    du = (e * B).sum(2)
    ddt = (through * s["A"]).sum(2) + du * x
    out["dB"] = (e * (dt * x)[..., None]).reshape(T, G, C // G, -1).sum(2).to(s["dt"])
    out["dA"] = (through * dt[..., None]).sum(0)
    draw_ = ddt * v.sigmoid()
    out["draw"] = draw_.to(s["dt"])
    out["dbias"] = draw_.sum(0, dtype=torch.float64).float()
    out["dx"] = (du * dt + s["D"] * dy).to(s["dt"])
    out["dD"] = (dy * x).sum(0, dtype=torch.float64).float()
    return out


def _plain_sel_decode(s):
    _, dt, x, B, Cc, a = _steps(s)
    h = a * s["h0"] + (dt * x)[..., None] * B
    y = (h * Cc).sum(2) + s["D"] * x
    if s["z"] is not None:
        y = y * s["z"].float() * s["z"].float().sigmoid()
    return y.to(s["dt"]), h


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import gated_delta_rule_41_amd as kda

    op = s["op"]
    if op == "norm":
        if s["out"] == s["dt"]:
            y, total = kda.kda_norm_fwd(s["x"], s["w"], s["residual"], eps=EPS)
            return {"y": y, "residual": total}
        y, total, scale = kda.kda_norm_fwd(s["x"], s["w"], s["residual"], eps=EPS, out_dtype=s["out"])
        return {"y": y.float() * scale[:, None], "residual": total, "scale": scale}
    if op == "norm_bwd":
        return kda.kda_norm_bwd(s["x"], s["w"], s["dy"], s["ds"], eps=EPS)
    if op == "conv":
        return kda.kda_conv_fwd(s["x"], s["w"], s["b"], s["cu"], s["state"], activation="silu")
    if op == "conv_bwd":
        d = kda.kda_conv_bwd(s["x"], s["w"], s["b"], s["dy"], s["cu"], s["state"], s["dstate"], activation="silu")
        return {n: x for n, x in d.items() if x is not None}
    if op == "conv_decode":
        return kda.kda_conv_decode(s["x"], s["w"], s["b"], s["state"], activation="silu")
    args = (s["x"], s["raw"], s["A"], s["B"], s["Cm"])
    kw = {"D": s["D"], "z": s["z"], "dt_bias": s["bias"], "softplus": True}
    if op == "sel":
        return kda.kda_selective_fwd(*args, s["cu"], s["h0"], **kw)
    if op == "sel_decode":
        return kda.kda_selective_decode(*args, s["h0"], **kw)
    d = kda.kda_selective_bwd(*args, s["dy"], s["cu"], s["h0"], s["dh"], **kw)
    names = {"dx": "dx", "draw": "ddt", "dA": "dA", "dB": "dB", "dC": "dC", "dD": "dD", "dz": "dz", "dbias": "ddt_bias", "dh0": "dS0"}
    return {n: d[m] for n, m in names.items() if d[m] is not None}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "conv": _plain_conv, "conv_bwd": _plain_conv_bwd,
            "conv_decode": _plain_conv_decode, "sel": _plain_sel, "sel_bwd": _plain_sel_bwd,
            "sel_decode": _plain_sel_decode}[state["op"]](state)


def work(case):
    op, C = case["op"], case["C"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        rows = case["T"]
        out = es * rows * C if case["out"] == "same" else rows * C + 4 * rows
        return {"bytes": 3 * es * rows * C + es * C + out, "flops": 6 * rows * C}
    if op == "norm_bwd":
        return {"bytes": es * (4 * case["T"] * C + C) + 4 * C, "flops": 12 * case["T"] * C}
    N = case["N"]
    if op.startswith("conv"):
        W = case["W"]
        state, weights = es * N * (W - 1) * C, C * (W + (1 if case["bias"] else 0))
        if op == "conv_bwd":
            return {"bytes": 3 * es * case["T"] * C + 3 * state + (es + 4) * weights, "flops": (6 * W + 8) * case["T"] * C}
        rows = N if op == "conv_decode" else case["T"]
        return {"bytes": 2 * es * rows * C + 2 * state + es * weights, "flops": (2 * W + 4) * rows * C}
    S, G = case["S"], case["G"]
    rows = N if op == "sel_decode" else case["T"]
    state, vectors = 4 * N * C * S, (3 + case["gated"]) * es * rows * C
    if op == "sel_bwd":
        return {"bytes": vectors + (2 + case["gated"]) * es * rows * C + 4 * es * rows * G * S + 3 * state + 4 * C * (2 * S + 4),
                "flops": 18 * rows * C * S}
    return {"bytes": vectors + 2 * es * rows * G * S + 2 * state + 4 * C * (S + 2), "flops": 6 * rows * C * S}


# ------------------------------------------------------------------ 64 bits
def _nearest_e4m3(x):
    """Halfway between two values goes to the one with the even last bit: they are multiples of eighths of a power of two."""
    _, e = torch.frexp(x)                                                   # x = m 2^e, m in [0.5, 1)
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-5) - 4)
    return (x / step).round() * step


def _exact_norm(s):
    x = (s["x"].double() + s["residual"].double()).to(s["dt"]).double()
    w = s["w"].double()
    norm = torch.sqrt((x * x).sum(1) / x.shape[1] + EPS)[:, None]
    if s["out"] == s["dt"]:
        return {"y": x / norm * w, "residual": x}
    most = 127.0 if s["out"] == torch.int8 else 448.0
    y = (x.float() * w.float()).double()            # the products are fp32 numbers by definition
    top = y.abs().max(1, keepdim=True)[0]
    unit = top / most
    code = y * most / top
    code = code.round() if s["out"] == torch.int8 else _nearest_e4m3(code)
    return {"y": code * (unit / norm), "residual": x, "scale": (unit / norm)[:, 0]}


def _exact_norm_bwd(s):
    x, w, g = s["x"].double(), s["w"].double(), s["dy"].double()
    C = x.shape[1]
    inv = (x.square().sum(1, keepdim=True) / C + EPS) ** -0.5
    dot = (g * w * x).sum(1, keepdim=True)
    return {"dx": inv * w * g - inv ** 3 / C * dot * x + s["ds"].double(), "dw": (g * x * inv).sum(0)}


def _exact_conv(s, backward):
    """Document by document, tap by tap."""
    W, w = s["w"].shape[1], s["w"].double()
    b = torch.zeros_like(w[:, 0]) if s["b"] is None else s["b"].double()
    ys, ends, dxs, dstates = [], [], [], []
    dw, db, lo = torch.zeros_like(w), torch.zeros_like(b), 0
    for n, length in enumerate(s["lens"]):
        hi = lo + length
        ext = torch.cat([s["state"][n], s["x"][lo:hi]]).double()
        pre = b.expand(length, -1).clone()
        for j in range(W):
            pre += ext[j:j + length] * w[:, j]
        sig = 1 / (1 + torch.exp(-pre))
        ys.append(pre * sig)
        ends.append(ext[length:])
        if backward:
            dpre = s["dy"][lo:hi].double() * (sig + pre * sig * (1 - sig))
            dext = torch.zeros_like(ext)
            dext[length:] += s["dstate"][n].double()
            for j in range(W):
                dext[j:j + length] += dpre * w[:, j]
                dw[:, j] += (dpre * ext[j:j + length]).sum(0)
            db += dpre.sum(0)
            dstates.append(dext[:W - 1])
            dxs.append(dext[W - 1:])
        lo = hi
    if not backward:
        return torch.cat(ys), torch.stack(ends)
    out = {"dx": torch.cat(dxs), "dw": dw, "dstate": torch.stack(dstates)}
    if s["b"] is not None:
        out["db"] = db
    return out


def _exact_conv_decode(s):
    ext = torch.cat([s["state"].double(), s["x"].double()[:, None]], 1)
    pre = (ext * s["w"].double().t()[None]).sum(1)
    pre = pre if s["b"] is None else pre + s["b"].double()
    return pre / (1 + torch.exp(-pre)), ext[:, 1:]


def _exact_sel(s, backward):
    """Token by token through the packed stream."""
    T, C = s["x"].shape
    G, S = s["B"].shape[1:]
    v = s["raw"].double() + s["bias"].double()
    dt = torch.nn.functional.softplus(v, threshold=50)
    x, A, D = s["x"].double(), s["A"].double(), s["D"].double()
    u = dt * x
    starts = {}
    lo = 0
    for n, length in enumerate(s["lens"]):
        starts[lo] = n
        lo += length
    B, Cc = s["B"].double(), s["Cm"].double()
    R = C // G
    h, keep = None, torch.empty(T, C, S, dtype=torch.float64, device="cuda") if backward else None
    y, final = torch.empty(T, C, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        if t in starts:
            if t:
                final.append(h)
            h = s["h0"][starts[t]].double()
        h = torch.exp(dt[t, :, None] * A) * h
        h = torch.addcmul(h.view(G, R, S), u[t].view(G, R, 1), B[t][:, None]).view(C, S)
        torch.matmul(h.view(G, R, S), Cc[t][:, :, None], out=y[t].view(G, R, 1))
        if backward:
            keep[t] = h
    final.append(h)
    y = y + D * x
    gate = None if s["z"] is None else s["z"].double() / (1 + torch.exp(-s["z"].double()))
    if not backward:
        return (y if gate is None else y * gate), torch.stack(final)
    out, dy = {}, s["dy"].double()
    if gate is not None:
        sig = 1 / (1 + torch.exp(-s["z"].double()))
        out["dz"] = dy * y * (sig + s["z"].double() * sig * (1 - sig))
        dy = dy * gate
    zero = torch.zeros(T, C, dtype=torch.float64, device="cuda")
    du, ddt, dA = zero.clone(), zero, torch.zeros_like(A)
    dB, dC = torch.empty_like(B), torch.empty_like(Cc)
    dh0, e = [None] * len(s["lens"]), None
    ends = {a + length - 1: n for (a, n), length in zip(sorted(starts.items()), s["lens"])}
    for t in reversed(range(T)):
        if t in ends:
            e = s["dh"][ends[t]].double()
        e = torch.addcmul(e.view(G, R, S), dy[t].view(G, R, 1), Cc[t][:, None]).view(C, S)
        before = s["h0"][starts[t]].double() if t in starts else keep[t - 1]
        dC[t] = (dy[t].view(G, 1, R) @ keep[t].view(G, R, S))[:, 0]
        dB[t] = (u[t].view(G, 1, R) @ e.view(G, R, S))[:, 0]
        du[t] = (e.view(G, R, S) @ B[t][:, :, None]).view(C)
        e = torch.exp(dt[t, :, None] * A) * e
        m = e * before
        ddt[t] = (m * A).sum(1)
        dA += m * dt[t, :, None]
        if t in starts:
            dh0[starts[t]] = e
    ddt = (ddt + du * x) / (1 + torch.exp(-v))
    out.update(dx=du * dt + D * dy, draw=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum(0), dbias=ddt.sum(0), dh0=torch.stack(dh0))
    return out


def _exact_sel_decode(s):
    N, C = s["x"].shape
    R = C // s["B"].shape[1]
    dt = torch.nn.functional.softplus(s["raw"].double() + s["bias"].double(), threshold=50)
    B, Cc = (s[n].double().repeat_interleave(R, 1) for n in ("B", "Cm"))
    h = torch.exp(dt[..., None] * s["A"].double()) * s["h0"].double() + (dt * s["x"].double())[..., None] * B
    y = (h * Cc).sum(2) + s["D"].double() * s["x"].double()
    if s["z"] is not None:
        y = y * s["z"].double() / (1 + torch.exp(-s["z"].double()))
    return y, h


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "conv_decode": _exact_conv_decode, "sel_decode": _exact_sel_decode,
            "conv": lambda s: _exact_conv(s, False), "conv_bwd": lambda s: _exact_conv(s, True),
            "sel": lambda s: _exact_sel(s, False), "sel_bwd": lambda s: _exact_sel(s, True)}[op](s)
