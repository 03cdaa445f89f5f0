"""What stands around the recurrences in a layer: the norm with the residual's
addition, the short causal convolution, and the selective scan.  Marshalling only,
as in the package's ``__init__``: see include/kda.h for the layouts.

Inputs called x, dt, B, C and z may be parts of wider rows (a split projection):
their last dimensions have to be contiguous, rows may be further apart.  They begin
at a multiple of 16 bytes, and so does every row of B and C.  All other tensors are
contiguous.
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional

from . import _lib
from ._lib import KDA_ACT_NONE, KDA_ACT_SILU, KDA_BF16, KDA_E4M3, KDA_F32, KDA_I8, KDA_SELECTIVE_SOFTPLUS
from ._tensors import check as _check, dt_code as _dt_code, launch as _launch, ptr as _ptr, torch_module as _torch, upstream as _upstream

# Configs and workspace sizes depend on their arguments alone; made once for each set of them.
_norm_config = lru_cache(maxsize=256)(_lib.make_norm_config)
_conv_config = lru_cache(maxsize=256)(_lib.make_conv_config)
_selective_config = lru_cache(maxsize=256)(_lib.make_selective_config)


@lru_cache(maxsize=256)
def _workspace(size, make, sizes, *config):
    return size(make(*config), *sizes)


def _workspace_tensor(size, make, sizes, config, dev):
    torch = _torch()
    n = _workspace(size, make, sizes, *config)
    return (torch.empty(n, dtype=torch.uint8, device=dev) if n else None), n


def _gpu(t, name, dims):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("libkda runs on the GPU only: tensors must be on a cuda (HIP) device")


def _rows(t, name, shape, dtype, device):
    """A tensor whose rows may be further apart than they are long: the stride of its rows."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _check(t, name, shape, dtype, device)
    inner = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner:
            raise ValueError(f"{name}'s rows must be contiguous")
        inner *= size
    if shape[0] <= 1:
        return inner
    stride = t.stride()[0]
    if stride < inner:
        raise ValueError(f"{name}'s rows must not overlap")
    return stride


def _seqs(T, cu_seqlens, num_seqs, dev):
    if cu_seqlens is None:
        return 1 if num_seqs is None else int(num_seqs)
    if (cu_seqlens.dtype != _torch().int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor on the same device")
    N = cu_seqlens.numel() - 1
    if num_seqs is not None and int(num_seqs) != N:
        raise ValueError(f"num_seqs is {num_seqs}, but cu_seqlens holds {N} sequences")
    return N


def _is_float(dtype):
    torch = _torch()
    return dtype == torch.bfloat16 or dtype == torch.float32


# ------------------------------------------------------------------ norm
_CODES = {}


def _norm_out_code(dtype):
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: KDA_F32, torch.bfloat16: KDA_BF16, torch.int8: KDA_I8, torch.float8_e4m3fn: KDA_E4M3})
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _weight_code(weight, C, dev):
    if weight is None:
        return KDA_F32
    _check(weight, "weight", (C,), weight.dtype, dev)
    return _dt_code(weight.dtype)


def kda_norm_fwd(x, weight=None, residual=None, *, out_dtype=None, out_residual=None, eps: float = 1e-6):
    """Root-mean-square norm with the residual's addition: ``s = x + residual``,
    ``y = s * weight / sqrt(mean(s^2) + eps)`` over the last dimension.

    x ``[T, C]``; ``weight`` ``[C]`` (None: ones) fp32 or bf16; ``residual``
    ``[T, C]`` in x's type or fp32, or None (``s = x``).  s has the residual's type
    and the norm is of the rounded s.  y is in x's type unless ``out_dtype`` says
    otherwise.  Returns ``(y, s)``; ``out_residual`` takes s and may be ``residual``
    itself.  With ``out_dtype`` ``torch.int8`` or ``torch.float8_e4m3fn`` y holds
    codes and the call returns ``(y, s, scale)``, scale fp32 ``[T]``: the values are
    ``y * scale[:, None]``."""
    torch = _torch()
    _gpu(x, "x", 2)
    T, C = x.shape
    dev, dt = x.device, x.dtype
    _check(x, "x", (T, C), dt, dev)
    out_dtype = out_dtype or dt
    code = _norm_out_code(out_dtype)
    res_dtype = dt
    if residual is not None:
        res_dtype = residual.dtype if residual.dtype == torch.float32 else dt
        _check(residual, "residual", (T, C), res_dtype, dev)
    wcode = _weight_code(weight, C, dev)
    config = (C, _dt_code(dt), _dt_code(res_dtype), wcode, code, float(eps))
    y = torch.empty((T, C), dtype=out_dtype, device=dev)
    if residual is None:
        if out_residual is not None:
            raise ValueError("out_residual needs a residual")
        s = x
    elif out_residual is None:
        s = torch.empty_like(residual)
    else:
        _check(out_residual, "out_residual", (T, C), res_dtype, dev)
        s = out_residual
    scale = torch.empty(T, dtype=torch.float32, device=dev) if code > KDA_BF16 else None
    _launch(dev, _lib.kda_norm_fwd_raw, _norm_config(*config), T, _ptr(x), _ptr(residual), _ptr(weight), _ptr(y),
            _ptr(s if residual is not None else None), _ptr(scale))
    return (y, s) if scale is None else (y, s, scale)


def kda_norm_bwd(s, weight, dy, ds=None, *, out_dtype=None, eps: float = 1e-6):
    """Backward of kda_norm_fwd for the loss <dy, y> + <ds, s>, from the s that the
    forward returned.  dy ``[T, C]`` in x's type, ds in s's type or None.  Returns a
    dict with dx (the gradient of x and of the residual; s's type unless
    ``out_dtype`` says otherwise) and dw (fp32 ``[C]``; None without a weight)."""
    torch = _torch()
    _gpu(s, "s", 2)
    T, C = s.shape
    dev, rt, dt = s.device, s.dtype, dy.dtype
    _check(s, "s", (T, C), rt, dev)
    _check(dy, "dy", (T, C), dt, dev)
    _check(ds, "ds", (T, C), rt, dev)
    out_dtype = out_dtype or rt
    wcode = _weight_code(weight, C, dev)
    config = (C, _dt_code(dt), _dt_code(rt), wcode, _dt_code(out_dtype), float(eps))
    dx = torch.empty((T, C), dtype=out_dtype, device=dev)
    dw, ws, n = None, None, 0
    if weight is not None:
        dw = torch.empty(C, dtype=torch.float32, device=dev)
        ws, n = _workspace_tensor(_lib.kda_norm_bwd_workspace_size, _norm_config, (T,), config, dev)
    _launch(dev, _lib.kda_norm_bwd_raw, _norm_config(*config), T, _ptr(s), _ptr(weight), _ptr(dy), _ptr(ds), _ptr(dx), _ptr(dw),
            _ptr(ws), n)
    return {"dx": dx, "dw": dw}


# ------------------------------------------------------------------ short convolution
_ACTIVATIONS = {None: KDA_ACT_NONE, "silu": KDA_ACT_SILU}


def _conv_common(x, weight, bias, activation, out_dtype):
    _gpu(x, "x", 2)
    T, C = x.shape
    dev, dt = x.device, x.dtype
    stride = _rows(x, "x", (T, C), dt, dev)
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight must be [{C}, width], got shape {tuple(weight.shape)}")
    W = weight.shape[1]
    _check(weight, "weight", (C, W), weight.dtype, dev)
    _check(bias, "bias", (C,), weight.dtype, dev)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    config = (C, W, _dt_code(dt), _dt_code(out_dtype or dt), _dt_code(weight.dtype), _ACTIVATIONS[activation], stride)
    return config, T, C, W, dev, dt


def kda_conv_fwd(x, weight, bias=None, cu_seqlens=None, initial_state=None, *, num_seqs: Optional[int] = None,
                 activation: Optional[str] = "silu", out_dtype=None, output_final_state: bool = True):
    """Causal convolution of every channel with its own taps, over packed
    documents: ``y_t = act(bias + sum_j weight[:, j] x_{t - W + 1 + j})``.

    x ``[T, C]``; ``weight`` ``[C, W]``, W 2 to 4, and ``bias`` ``[C]`` or None, fp32
    or bf16; ``initial_state`` ``[N, W - 1, C]`` in x's type, the rows before each
    document, oldest first (None: zero).  Returns ``(y, final_state)``; y is in x's
    type unless ``out_dtype`` says otherwise.  ``num_seqs`` as in kda_fwd."""
    torch = _torch()
    config, T, C, W, dev, dt = _conv_common(x, weight, bias, activation, out_dtype)
    N = _seqs(T, cu_seqlens, num_seqs, dev)
    _check(initial_state, "initial_state", (N, W - 1, C), dt, dev)
    y = torch.empty((T, C), dtype=out_dtype or dt, device=dev)
    sf = torch.empty((N, W - 1, C), dtype=dt, device=dev) if output_final_state else None
    _launch(dev, _lib.kda_conv_fwd_raw, _conv_config(*config), T, N, _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens),
            _ptr(initial_state), _ptr(y), _ptr(sf))
    return y, sf


def kda_conv_bwd(x, weight, bias, dy, cu_seqlens=None, initial_state=None, d_final_state=None, *, num_seqs: Optional[int] = None,
                 activation: Optional[str] = "silu", out_dtype=None):
    """Backward of kda_conv_fwd for the loss <dy, y> + <d_final_state,
    final_state>, from the forward's inputs.  dy ``[T, C]`` in x's type.  Returns a
    dict with dx (x's type unless ``out_dtype`` says otherwise), dw and db (fp32;
    db None without a bias) and dstate (x's type; None without an initial state)."""
    torch = _torch()
    config, T, C, W, dev, dt = _conv_common(x, weight, bias, activation, out_dtype)
    N = _seqs(T, cu_seqlens, num_seqs, dev)
    _check(dy, "dy", (T, C), dt, dev)
    _check(initial_state, "initial_state", (N, W - 1, C), dt, dev)
    _check(d_final_state, "d_final_state", (N, W - 1, C), dt, dev)
    out = {
        "dx": torch.empty((T, C), dtype=out_dtype or dt, device=dev),
        "dw": torch.empty((C, W), dtype=torch.float32, device=dev),
        "db": torch.empty(C, dtype=torch.float32, device=dev) if bias is not None else None,
        "dstate": torch.empty_like(initial_state) if initial_state is not None else None,
    }
    ws, n = _workspace_tensor(_lib.kda_conv_bwd_workspace_size, _conv_config, (T, N), config, dev)
    _launch(dev, _lib.kda_conv_bwd_raw, _conv_config(*config), T, N, _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens),
            _ptr(initial_state), _ptr(dy), _ptr(d_final_state), _ptr(out["dx"]), _ptr(out["dw"]), _ptr(out["db"]), _ptr(out["dstate"]),
            _ptr(ws), n)
    return out


def kda_conv_decode(x, weight, bias=None, state=None, *, out_state=None, activation: Optional[str] = "silu", out_dtype=None):
    """One token per sequence of kda_conv_fwd: x ``[N, C]``, ``state``
    ``[N, W - 1, C]`` in x's type or None (zero); ``out_state`` may be ``state``
    itself.  Returns ``(y, out_state)``."""
    torch = _torch()
    config, N, C, W, dev, dt = _conv_common(x, weight, bias, activation, out_dtype)
    _check(state, "state", (N, W - 1, C), dt, dev)
    if out_state is None:
        out_state = torch.empty((N, W - 1, C), dtype=dt, device=dev)
    else:
        _check(out_state, "out_state", (N, W - 1, C), dt, dev)
    y = torch.empty((N, C), dtype=out_dtype or dt, device=dev)
    _launch(dev, _lib.kda_conv_decode_raw, _conv_config(*config), N, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(out_state),
            _ptr(y))
    return y, out_state


# ------------------------------------------------------------------ selective scan
def _selective_common(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype):
    torch = _torch()
    _gpu(x, "x", 2)
    T, channels = x.shape
    dev, t = x.device, x.dtype
    if A.dim() != 2:
        raise ValueError(f"A must have 2 dimensions, got shape {tuple(A.shape)}")
    if B.dim() != 3:
        raise ValueError(f"B must have 3 dimensions, got shape {tuple(B.shape)}")
    S, G = A.shape[1], B.shape[1]
    float32 = torch.float32
    _check(A, "A", (channels, S), float32, dev)
    _check(D, "D", (channels,), float32, dev)
    _check(dt_bias, "dt_bias", (channels,), float32, dev)
    strides = (_rows(x, "x", (T, channels), t, dev), _rows(dt, "dt", (T, channels), t, dev),
               _rows(z, "z", (T, channels), t, dev) if z is not None else 0,
               _rows(B, "B", (T, G, S), t, dev), _rows(C, "C", (T, G, S), t, dev))
    config = (channels, S, G, _dt_code(t), _dt_code(out_dtype or t), KDA_SELECTIVE_SOFTPLUS if softplus else 0, *strides)
    return config, T, channels, S, dev, t


def kda_selective_fwd(x, dt, A, B, C, cu_seqlens=None, initial_state=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                      num_seqs: Optional[int] = None, out_dtype=None, output_final_state: bool = True):
    """Selective scan over packed documents, a state of S entries for each channel:
    ``h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t``, ``y_t = (C_t . h_t + D x_t) silu(z_t)``
    with ``dt_t = softplus(dt_t + dt_bias)`` (``softplus=False``: without).

    x, dt, z ``[T, C]``; A fp32 ``[C, S]`` (negative), S 8, 16 or 32; B, C
    ``[T, G, S]`` with G dividing the channels (channel c reads group
    ``c // (channels // G)``); D and dt_bias fp32 ``[C]``; ``initial_state`` fp32
    ``[N, C, S]`` or None.  D, z and dt_bias may be None.  Returns
    ``(y, final_state)``; y is in x's type unless ``out_dtype`` says otherwise."""
    torch = _torch()
    config, T, channels, S, dev, t = _selective_common(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype)
    N = _seqs(T, cu_seqlens, num_seqs, dev)
    _check(initial_state, "initial_state", (N, channels, S), torch.float32, dev)
    y = torch.empty((T, channels), dtype=out_dtype or t, device=dev)
    sf = torch.empty((N, channels, S), dtype=torch.float32, device=dev) if output_final_state else None
    ws, n = _workspace_tensor(_lib.kda_selective_fwd_workspace_size, _selective_config, (T, N), config, dev)
    _launch(dev, _lib.kda_selective_fwd_raw, _selective_config(*config), T, N, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            _ptr(z), _ptr(dt_bias), _ptr(cu_seqlens), _ptr(initial_state), _ptr(y), _ptr(sf), _ptr(ws), n)
    return y, sf


def kda_selective_bwd(x, dt, A, B, C, dy, cu_seqlens=None, initial_state=None, dS_final=None, *, D=None, z=None, dt_bias=None,
                      softplus: bool = True, num_seqs: Optional[int] = None, out_dtype=None):
    """Backward of kda_selective_fwd for the loss <dy, y> + <dS_final,
    final_state>, from the forward's inputs.  dy ``[T, C]`` in x's type.  Returns a
    dict with dx, ddt (of dt as given), dB, dC, dz (x's type unless ``out_dtype`` says
    otherwise), dA, dD, ddt_bias and dS0 (fp32); what was None in the call is None."""
    torch = _torch()
    config, T, channels, S, dev, t = _selective_common(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype)
    N = _seqs(T, cu_seqlens, num_seqs, dev)
    _check(dy, "dy", (T, channels), t, dev)
    _check(initial_state, "initial_state", (N, channels, S), torch.float32, dev)
    _check(dS_final, "dS_final", (N, channels, S), torch.float32, dev)
    ot = out_dtype or t

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=dev)

    out = {
        "dx": empty(T, channels, dtype=ot),
        "ddt": empty(T, channels, dtype=ot),
        "dA": empty(channels, S),
        "dB": empty(*B.shape, dtype=ot),
        "dC": empty(*B.shape, dtype=ot),
        "dD": empty(channels) if D is not None else None,
        "dz": empty(T, channels, dtype=ot) if z is not None else None,
        "ddt_bias": empty(channels) if dt_bias is not None else None,
        "dS0": empty(N, channels, S) if initial_state is not None else None,
    }
    ws, n = _workspace_tensor(_lib.kda_selective_bwd_workspace_size, _selective_config, (T, N), config, dev)
    _launch(dev, _lib.kda_selective_bwd_raw, _selective_config(*config), T, N, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            _ptr(z), _ptr(dt_bias), _ptr(cu_seqlens), _ptr(initial_state), _ptr(dy), _ptr(dS_final),
            *(_ptr(out[k]) for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")), _ptr(ws), n)
    return out


def kda_selective_decode(x, dt, A, B, C, state=None, *, D=None, z=None, dt_bias=None, softplus: bool = True, out_state=None,
                         out_dtype=None):
    """One token per sequence of kda_selective_fwd on a resident fp32 state: x, dt,
    z ``[N, C]``, B, C ``[N, G, S]``, ``state`` ``[N, C, S]`` or None (zero);
    ``out_state`` may be ``state`` itself.  Returns ``(y, out_state)``."""
    torch = _torch()
    config, N, channels, S, dev, t = _selective_common(x, dt, A, B, C, D, z, dt_bias, softplus, out_dtype)
    _check(state, "state", (N, channels, S), torch.float32, dev)
    if out_state is None:
        out_state = torch.empty((N, channels, S), dtype=torch.float32, device=dev)
    else:
        _check(out_state, "out_state", (N, channels, S), torch.float32, dev)
    y = torch.empty((N, channels), dtype=out_dtype or t, device=dev)
    _launch(dev, _lib.kda_selective_decode_raw, _selective_config(*config), N, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            _ptr(z), _ptr(dt_bias), _ptr(state), _ptr(out_state), _ptr(y))
    return y, out_state


# ------------------------------------------------------------------ autograd
def _functions():
    """Autograd glue: the backwards run from the inputs (the norm's from the sum that it returns), so nothing else is kept."""
    torch = _torch()
    from torch.autograd.function import once_differentiable

    def grad(g, like):
        return _upstream(g.to(like.dtype)) if g is not None else torch.zeros_like(like, memory_format=torch.contiguous_format)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, residual, eps):
            y, s = kda_norm_fwd(x, weight, residual, eps=eps)
            ctx.save_for_backward(s, weight)
            ctx.set_materialize_grads(False)   # an output that the loss does not use has no gradient, not one of zeros
            ctx.eps, ctx.types = eps, (x.dtype, None if residual is None else residual.dtype)
            return (y, s) if residual is not None else y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, ds=None):
            s, weight = ctx.saved_tensors
            xt, rt = ctx.types
            dy = _upstream(dy.to(xt)) if dy is not None else torch.zeros(s.shape, dtype=xt, device=s.device)
            ds = _upstream(ds.to(s.dtype)) if ds is not None else None
            d = kda_norm_bwd(s, weight, dy, ds, eps=ctx.eps)
            dw = d["dw"].to(weight.dtype) if weight is not None else None
            return d["dx"].to(xt), dw, d["dx"] if rt is not None else None, None

    class Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, cu_seqlens, initial_state, num_seqs, activation):
            y, sf = kda_conv_fwd(x, weight, bias, cu_seqlens, initial_state, num_seqs=num_seqs, activation=activation)
            ctx.save_for_backward(x, weight, bias, cu_seqlens, initial_state)
            ctx.set_materialize_grads(False)
            ctx.num_seqs, ctx.activation = num_seqs, activation
            return y, sf

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dsf):
            x, weight, bias, cu, s0 = ctx.saved_tensors
            dsf = _upstream(dsf.to(x.dtype)) if dsf is not None else None
            d = kda_conv_bwd(x, weight, bias, grad(dy, x), cu, s0, dsf, num_seqs=ctx.num_seqs, activation=ctx.activation)
            db = d["db"].to(bias.dtype) if bias is not None else None
            return d["dx"], d["dw"].to(weight.dtype), db, None, d["dstate"], None, None

    class Selective(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, num_seqs, softplus):
            y, sf = kda_selective_fwd(x, dt, A, B, C, cu_seqlens, initial_state, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                                      num_seqs=num_seqs)
            ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state)
            ctx.set_materialize_grads(False)
            ctx.num_seqs, ctx.softplus = num_seqs, softplus
            return y, sf

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dsf):
            x, dt, A, B, C, D, z, dt_bias, cu, s0 = ctx.saved_tensors
            dsf = _upstream(dsf) if dsf is not None else None
            d = kda_selective_bwd(x, dt, A, B, C, grad(dy, x), cu, s0, dsf, D=D, z=z, dt_bias=dt_bias, softplus=ctx.softplus,
                                  num_seqs=ctx.num_seqs)
            return (d["dx"], d["ddt"], d["dA"], d["dB"], d["dC"], d["dD"], d["dz"], d["ddt_bias"], None, d["dS0"], None, None)

    return {"norm": Norm, "conv": Conv, "selective": Selective}


_FN = {}


def _fn(name):
    if not _FN:
        _FN.update(_functions())
    return _FN[name]


def kda_norm(x, weight=None, residual=None, *, eps: float = 1e-6):
    """kda_norm_fwd as a differentiable torch op: returns ``(y, s)``, or y alone
    without a residual.  Upstream gradients are cast to the types of x and s, and the
    weight's gradient, summed in fp32, is rounded to the weight's type.  A second
    differentiation is refused.

    In a captured graph use torch.autograd.grad, or leaves of which no eager graph
    is alive: torch ties a leaf's gradient accumulation to the stream of its first
    graph."""
    return _fn("norm").apply(x, weight, residual, eps)


def kda_conv(x, weight, bias=None, cu_seqlens=None, initial_state=None, *, num_seqs: Optional[int] = None,
             activation: Optional[str] = "silu"):
    """kda_conv_fwd as a differentiable torch op: returns ``(y, final_state)``, both
    in x's type.  Captured graphs and second differentiation as for kda_norm."""
    return _fn("conv").apply(x, weight, bias, cu_seqlens, initial_state, num_seqs, activation)


def kda_selective(x, dt, A, B, C, cu_seqlens=None, initial_state=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                  num_seqs: Optional[int] = None):
    """kda_selective_fwd as a differentiable torch op: returns ``(y, final_state)``,
    y in x's type.  Captured graphs and second differentiation as for kda_norm."""
    return _fn("selective").apply(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, num_seqs, softplus)
