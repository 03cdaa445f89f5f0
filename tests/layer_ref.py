"""64-bit references of the norm, the short convolution and the selective scan,
token by token in numpy, and the error bounds the GPU tests use.

One rounding is half a step: u = 2^-24 in fp32, 2^-8 in bf16.  Functions called
*_bound return, for each output, what the fp32 arithmetic of the operator can be off by:
every term's count of roundings times u times the term's absolute value.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


# ------------------------------------------------------------------ norm
# Roundings of rstd: a sum of squares in which a term passes through at most 64 additions in a
# lane and 9 + 8 across lanes and waves (half of its relative error reaches rstd), then the
# mean, eps, root and quotient.
RSTD = (64 + 17) / 2 + 4


def norm_fwd(s, w, eps):
    rstd = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s * w * rstd, rstd


def norm_bwd(s, w, dy, ds, eps):
    _, rstd = norm_fwd(s, w, eps)
    xh, wg = s * rstd, dy * w
    dx = rstd * (wg - xh * (wg * xh).mean(1, keepdims=True)) + ds
    return dx, (dy * xh).sum(0)


def norm_bwd_bound(s, w, dy, ds, eps):
    _, rstd = norm_fwd(s, w, eps)
    xh, wg = np.abs(s * rstd), np.abs(dy * w)
    # rstd enters three times, the mean is a sum like rstd's, and five more operations
    dx = rstd * (wg + xh * (wg * xh).mean(1, keepdims=True)) * (3 * RSTD + 81 + 5) * U + np.abs(ds) * U
    return dx, (np.abs(dy) * xh).sum(0) * (s.shape[0] + RSTD + 20) * U


def codes(s, w, limit):
    """Codes as reals before rounding, from the fp32 products, and max|p|."""
    p = (s.astype(np.float32) * np.asarray(w, np.float32)).astype(np.float64)
    top = np.abs(p).max(1, keepdims=True)
    return np.where(top > 0, p * limit / np.where(top > 0, top, 1), 0.0), top


# ------------------------------------------------------------------ convolution
def conv_rows(x, state, lens):
    """For every document the rows of its state and its own."""
    at = starts(lens)
    return [np.concatenate([state[n], x[at[n]:at[n + 1]]]) for n in range(len(lens))]


def conv_fwd(x, w, b, state, lens, act=True):
    """(y, final state, bound of y) with w [C, W], state [N, W - 1, C]."""
    W = w.shape[1]
    ys, ends, off = [], [], []
    for rows in conv_rows(x, state, lens):
        T = len(rows) - (W - 1)
        pre = b + sum(rows[j:j + T] * w[:, j] for j in range(W))
        m = (np.abs(b) + sum(np.abs(rows[j:j + T] * w[:, j]) for j in range(W))) * (W + 1) * U
        ys.append(pre * sigmoid(pre) if act else pre)
        # |silu'| <= 1.1; the sigmoid's exponential, argument, sum, quotient and product: 16 half steps
        off.append(1.1 * m + 16 * U * np.maximum(np.abs(pre), 1) if act else m)
        ends.append(rows[T:])
    return np.concatenate(ys), np.stack(ends), np.concatenate(off)


def conv_bwd(x, w, b, state, lens, dy, dend, act=True):
    """{name: (gradient, bound)} for dx, dw, db, dstate."""
    W, at = w.shape[1], starts(lens)
    dx, dxm = np.zeros_like(x), np.zeros_like(x)
    dw, dwm, db, dbm = np.zeros_like(w), np.zeros_like(w), np.zeros(len(w)), np.zeros(len(w))
    dst, dstm = np.zeros_like(state), np.zeros_like(state)
    for n, rows in enumerate(conv_rows(x, state, lens)):
        T = lens[n]
        pre = b + sum(rows[j:j + T] * w[:, j] for j in range(W))
        m = (np.abs(b) + sum(np.abs(rows[j:j + T] * w[:, j]) for j in range(W))) * (W + 1) * U
        g = dy[at[n]:at[n + 1]]
        sig = sigmoid(pre)
        d = g * (sig * (1 + pre * (1 - sig))) if act else g
        dm = np.abs(g) * (0.5 * m + 16 * U) if act else 0 * g     # |silu''| <= 0.5
        ext, extm = np.zeros_like(rows), np.zeros_like(rows)
        ext[T:] += dend[n]
        extm[T:] += np.abs(dend[n]) * U
        for j in range(W):
            ext[j:j + T] += d * w[:, j]
            extm[j:j + T] += np.abs(w[:, j]) * (dm + np.abs(d) * (W + 1) * U)
            dw[:, j] += (d * rows[j:j + T]).sum(0)
            dwm[:, j] += (np.abs(rows[j:j + T]) * (dm + np.abs(d) * (len(x) + 20) * U)).sum(0)
        db += d.sum(0)
        dbm += (dm + np.abs(d) * (len(x) + 20) * U).sum(0)
        dst[n], dstm[n] = ext[:W - 1], extm[:W - 1]
        dx[at[n]:at[n + 1]], dxm[at[n]:at[n + 1]] = ext[W - 1:], extm[W - 1:]
    return {"dx": (dx, dxm), "dw": (dw, dwm), "db": (db, dbm), "dstate": (dst, dstm)}


# ------------------------------------------------------------------ selective scan
def selective(x, raw, A, B, C, D, z, bias, lens, h0, soft=True, dy=None, dh=None):
    """y, final states and, with dy and dh, all gradients, in 64 bits.  x, raw [T, c], A [c, S], B, C [T, G, S]."""
    T, c = x.shape
    R = c // B.shape[1]
    Bc, Cc = np.repeat(B, R, 1), np.repeat(C, R, 1)
    v = raw + bias
    dt = softplus(v) if soft else v
    a = np.exp(dt[:, :, None] * A)
    gate = z * sigmoid(z) if z is not None else np.ones_like(x)
    at = starts(lens)
    h, before = np.zeros((T,) + A.shape), np.zeros((T,) + A.shape)
    final = h0.copy()
    for n in range(len(lens)):
        for t in range(at[n], at[n + 1]):
            before[t] = final[n]
            final[n] = h[t] = a[t] * final[n] + (dt[t] * x[t])[:, None] * Bc[t]
    o = (h * Cc).sum(2) + D * x
    out = {"y": o * gate, "final": final}
    if dy is None:
        return out
    g = dy * gate
    e, dh0 = np.zeros_like(h), dh.copy()
    for n in range(len(lens)):
        for t in reversed(range(at[n], at[n + 1])):
            e[t] = g[t][:, None] * Cc[t] + dh0[n]
            dh0[n] = a[t] * e[t]
    du = (e * Bc).sum(2)
    m = e * a * before
    ddt = (m * A).sum(2) + du * x
    ddt = ddt * sigmoid(v) if soft else ddt
    groups = (T, B.shape[1], R, A.shape[1])
    out.update(dx=du * dt + D * g, ddt=ddt, dA=(m * dt[:, :, None]).sum(0), dB=(e * (dt * x)[:, :, None]).reshape(groups).sum(2),
               dC=(h * g[:, :, None]).reshape(groups).sum(2), dD=(g * x).sum(0), dbias=ddt.sum(0), dh0=dh0)
    if z is not None:
        s = sigmoid(z)
        out["dz"] = dy * o * s * (1 + z * (1 - s))
    return out


def selective_absolute(x, raw, A, B, C, D, z, bias, lens, h0, soft=True, dy=None, dh=None):
    """The same sums of absolute values (decays and step sizes as they are): what roundings are relative to."""
    T, c = x.shape
    v = raw + bias
    dt = softplus(v) if soft else v
    # silu and its derivative by their parts: |z| sig, sig (1 + |z| (1 - sig))
    ab = np.abs
    R = c // B.shape[1]
    Bc, Cc = np.repeat(ab(B), R, 1), np.repeat(ab(C), R, 1)
    a = np.exp(dt[:, :, None] * A)
    gate = ab(z) * sigmoid(z) if z is not None else np.ones_like(x)
    at = starts(lens)
    h, before = np.zeros((T,) + A.shape), np.zeros((T,) + A.shape)
    final = ab(h0)
    for n in range(len(lens)):
        for t in range(at[n], at[n + 1]):
            before[t] = final[n]
            final[n] = h[t] = a[t] * final[n] + ab(dt[t] * x[t])[:, None] * Bc[t]
    o = (h * Cc).sum(2) + ab(D * x)
    out = {"y": o * gate, "final": final}
    if dy is None:
        return out
    g = ab(dy) * gate
    e, dh0 = np.zeros_like(h), ab(dh)
    for n in range(len(lens)):
        for t in reversed(range(at[n], at[n + 1])):
            e[t] = g[t][:, None] * Cc[t] + dh0[n]
            dh0[n] = a[t] * e[t]
    du = (e * Bc).sum(2)
    m = e * a * before
    ddt = (m * ab(A)).sum(2) + du * ab(x)
    ddt = ddt * sigmoid(v) if soft else ddt
    groups = (T, B.shape[1], R, A.shape[1])
    out.update(dx=du * ab(dt) + ab(D) * g, ddt=ddt, dA=(m * ab(dt)[:, :, None]).sum(0),
               dB=(e * ab(dt * x)[:, :, None]).reshape(groups).sum(2), dC=(h * g[:, :, None]).reshape(groups).sum(2),
               dD=(g * ab(x)).sum(0), dbias=ddt.sum(0), dh0=dh0)
    if z is not None:
        s = sigmoid(z)
        out["dz"] = ab(dy) * o * s * (1 + ab(z) * (1 - s))
    return out


def selective_roundings(raw, A, bias, lens, soft=True, segment=64):
    """Roundings that a term passes through at most.  A decay's exponent has the step size's 6 half steps,
    A's product with log2 e, the product and, across a segment, a sum of its step sizes: 9 + segment
    half steps of the exponent, which add up to those of its document's sum; beside them each token takes
    the exponential's 2 and a multiply-add, and an output some 60 more (its sums over entries and lanes,
    gate and step size)."""
    v = raw + bias
    dt = softplus(v) if soft else np.abs(v)
    at = starts(lens)
    longest = max(lens) if len(lens) else 0
    sums = [np.abs(A).max(1) * dt[at[n]:at[n + 1]].sum(0) for n in range(len(lens)) if lens[n]]
    return (9 + segment) * (max(s.max() for s in sums) if sums else 0.0) + 3 * longest + 60
