"""The linear rule (linear attention with a decay for each head) and trees of
drafted tokens over the state, for both rules.  Marshalling only, as in the
package's ``__init__``: see include/kda.h for the layouts.
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional

from . import _lib
from ._lib import KDA_GATE_GRAD_F32, KDA_GATE_HEAD, KDA_GATE_TOKEN, KDA_RULE_DELTA, KDA_RULE_LINEAR, KDA_TREE_MAX_NODES
from ._tensors import check as _check, dt_code as _dt_code, launch as _launch, ptr as _ptr, torch_module as _torch

# Configs and workspace sizes depend on their arguments alone; made once for each set of them.
_linear_config = lru_cache(maxsize=256)(_lib.make_linear_config)
_tree_config = lru_cache(maxsize=256)(_lib.make_tree_config)


@lru_cache(maxsize=256)
def _linear_workspace(size, T, N, *config):
    return size(_linear_config(*config), T, N)


def _heads(q, k, v, lead_dims):
    """Shapes, device and dtype of q/k ``[..., Hk, dk]`` and v ``[..., H, dv]`` (q may be None)."""
    shape, vshape = k.shape, v.shape
    dims = lead_dims + 2
    if len(shape) != dims or len(vshape) != dims or (q is not None and q.dim() != dims):
        for name, t in (("q", q), ("k", k), ("v", v)):
            if t is not None and t.dim() != dims:
                raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    dev, dt, lead = k.device, k.dtype, tuple(shape[:-2])
    if not k.is_cuda:
        raise ValueError("libkda runs on the GPU only: tensors must be on a cuda (HIP) device")
    if q is not None:
        _check(q, "q", shape, dt, dev)
    _check(k, "k", shape, dt, dev)
    _check(v, "v", lead + vshape[-2:], dt, dev)
    return lead, vshape[-2], shape[-2], shape[-1], vshape[-1], dev, dt


def _gate(g, lead, H, dev):
    """fp32 gates ``[..., H]`` or ``[H]``."""
    float32 = _torch().float32
    if g.dim() == 1:
        _check(g, "g", (H,), float32, dev)
        return KDA_GATE_HEAD
    _check(g, "g", lead + (H,), float32, dev)
    return KDA_GATE_TOKEN


def _packed(q, k, v, g, cu_seqlens, num_seqs):
    torch = _torch()
    (T,), H, Hk, dk, dv, dev, dt = _heads(q, k, v, 1)
    gate = _gate(g, (T,), H, dev)
    if cu_seqlens is not None:
        if (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev
                or not cu_seqlens.is_contiguous()):
            raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor on the same device")
        N = cu_seqlens.numel() - 1
        if num_seqs is not None and int(num_seqs) != N:
            raise ValueError(f"num_seqs is {num_seqs}, but cu_seqlens holds {N} sequences")
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    return T, N, H, Hk, dk, dv, dev, dt, gate


def _check_dg_dtype(dg_dtype, out_dtype):
    if dg_dtype not in (None, out_dtype, _torch().float32):
        raise ValueError(f"dg_dtype must be torch.float32 or {out_dtype}, got {dg_dtype}")


def kda_linear_fwd(q, k, v, g, cu_seqlens=None, initial_state=None, *, num_seqs: Optional[int] = None, out_dtype=None,
                   scale: float = 1.0, output_final_state: bool = True):
    """Linear attention with a decay for each head, over packed documents:
    ``S_t = exp(g_t) S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t``.

    q, k ``[T, Hk, dk]``; v ``[T, H, dv]`` with Hk dividing H (head h reads
    query/key head ``h // (H // Hk)``); g fp32, the log-decay (<= 0), ``[T, H]``
    or ``[H]`` for a fixed decay; ``initial_state`` fp32 ``[N, H, dk, dv]`` or
    None.  Returns ``(o, final_state)``; o is fp32 unless ``out_dtype`` says
    otherwise.  ``num_seqs`` as in kda_fwd."""
    torch = _torch()
    T, N, H, Hk, dk, dv, dev, dt, gate = _packed(q, k, v, g, cu_seqlens, num_seqs)
    out_dtype = out_dtype or torch.float32
    _check(initial_state, "initial_state", (N, H, dk, dv), torch.float32, dev)
    config = (H, Hk, dk, dv, _dt_code(dt), _dt_code(out_dtype), gate, float(scale))
    o = torch.empty_like(v, dtype=out_dtype)
    sf = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if output_final_state else None
    wsb = _linear_workspace(_lib.kda_linear_fwd_workspace_size, T, N, *config)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _launch(dev, _lib.kda_linear_fwd_raw, _linear_config(*config), T, N, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(cu_seqlens),
            _ptr(initial_state), _ptr(o), _ptr(sf), _ptr(ws), wsb)
    return o, sf


def kda_linear_bwd(q, k, v, g, dO, cu_seqlens=None, initial_state=None, dS_final=None, *, num_seqs: Optional[int] = None,
                   out_dtype=None, dg_dtype=None, scale: float = 1.0, output_d_initial_state: bool = True):
    """Backward of kda_linear_fwd for the loss <dO, o> + <dS_final, final_state>,
    from the forward's inputs alone.  Returns a dict with dq, dk, dv, dg (the
    shapes of q, k, v, g; fp32 unless ``out_dtype`` says otherwise) and dS0
    (fp32, None unless requested).  ``dg_dtype=torch.float32`` keeps dg in g's own
    type beside a bf16 ``out_dtype``."""
    torch = _torch()
    T, N, H, Hk, dk, dv, dev, dt, gate = _packed(q, k, v, g, cu_seqlens, num_seqs)
    out_dtype = out_dtype or torch.float32
    dg_dtype = dg_dtype or out_dtype
    if dg_dtype != out_dtype:
        _check_dg_dtype(dg_dtype, out_dtype)
        gate |= KDA_GATE_GRAD_F32
    _check(dO, "dO", (T, H, dv), dt, dev)
    _check(initial_state, "initial_state", (N, H, dk, dv), torch.float32, dev)
    _check(dS_final, "dS_final", (N, H, dk, dv), torch.float32, dev)
    config = (H, Hk, dk, dv, _dt_code(dt), _dt_code(out_dtype), gate, float(scale))
    out = {
        "dq": torch.empty_like(q, dtype=out_dtype),
        "dk": torch.empty_like(k, dtype=out_dtype),
        "dv": torch.empty_like(v, dtype=out_dtype),
        "dg": torch.empty_like(g, dtype=dg_dtype),
        "dS0": torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if output_d_initial_state else None,
    }
    wsb = _linear_workspace(_lib.kda_linear_bwd_workspace_size, T, N, *config)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _launch(dev, _lib.kda_linear_bwd_raw, _linear_config(*config), T, N, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(cu_seqlens),
            _ptr(initial_state), _ptr(dO), _ptr(dS_final), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
            _ptr(out["dS0"]), _ptr(ws), wsb)
    return out


def kda_linear_decode(q, k, v, g, state=None, *, out_state=None, out_dtype=None, scale: float = 1.0):
    """One token per sequence of the linear rule on a resident fp32 state, as
    kda_decode: q, k ``[N, Hk, dk]``, v ``[N, H, dv]``, g fp32 ``[N, H]`` or
    ``[H]``, ``state`` ``[N, H, dk, dv]`` or None (zero).  ``out_state`` may be
    ``state`` itself.  Returns ``(o, out_state)``."""
    torch = _torch()
    (N,), H, Hk, dk, dv, dev, dt = _heads(q, k, v, 1)
    gate = _gate(g, (N,), H, dev)
    _check(state, "state", (N, H, dk, dv), torch.float32, dev)
    if out_state is None:
        out_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if state is None else torch.empty_like(state)
    else:
        _check(out_state, "out_state", (N, H, dk, dv), torch.float32, dev)
    out_dtype = out_dtype or torch.float32
    cfg = _linear_config(H, Hk, dk, dv, _dt_code(dt), _dt_code(out_dtype), gate, float(scale))
    o = torch.empty_like(v, dtype=out_dtype)
    _launch(dev, _lib.kda_linear_decode_raw, cfg, N, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state), _ptr(out_state), _ptr(o))
    return o, out_state


def _tree_common(q, k, v, g, beta, parent, state, out_dtype, eps, scale):
    torch = _torch()
    lead, H, Hk, dk, dv, dev, dt = _heads(q, k, v, 2)
    N, L = lead
    if not 1 <= L <= KDA_TREE_MAX_NODES:
        raise ValueError(f"a tree has 1 to {KDA_TREE_MAX_NODES} nodes, got {L}")
    if beta is None:
        rule, gate = KDA_RULE_LINEAR, _gate(g, lead, H, dev)
    else:
        rule, gate = KDA_RULE_DELTA, KDA_GATE_TOKEN
        if Hk != H:
            raise ValueError(f"the delta rule has as many key heads as value heads, got {Hk} and {H}")
        _check(g, "g", lead + (H, dk), dt, dev)
        _check(beta, "beta", lead + (H,), dt, dev)
    _check(parent, "parent", (N, L), torch.int32, dev)
    _check(state, "state", (N, H, dk, dv), torch.float32, dev)
    cfg = _tree_config(rule, H, Hk, dk, dv, L, _dt_code(dt), _dt_code(out_dtype), gate, float(eps), float(scale))
    return cfg, N, L, H, dk, dv, dev


def kda_tree(q, k, v, g, beta, parent, state=None, *, out_dtype=None, eps: float = 1e-6, scale: float = 1.0):
    """The outputs of a tree of drafted tokens over a recurrent state.

    Per sequence up to 64 nodes: q, k ``[N, L, Hk, dk]``, v ``[N, L, H, dv]``,
    ``parent`` int32 ``[N, L]`` (a node's parent, which comes before it; -1: the
    node follows the state; below -1: no node, its output is 0).  With ``beta``
    ``[N, L, H]`` and g ``[N, L, H, dk]`` the rule is kda_fwd's; with ``beta``
    None and g fp32 ``[N, L, H]`` or ``[H]`` it is kda_linear_fwd's.  ``state``
    fp32 ``[N, H, dk, dv]`` (None: zero) is read once and not changed.  Returns
    o ``[N, L, H, dv]``, fp32 unless ``out_dtype`` says otherwise."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    cfg, N, L, H, dk, dv, dev = _tree_common(q, k, v, g, beta, parent, state, out_dtype, eps, scale)
    o = torch.empty_like(v, dtype=out_dtype)
    _launch(dev, _lib.kda_tree_raw, cfg, N, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(parent), _ptr(state), _ptr(o))
    return o


def kda_tree_commit(k, v, g, beta, parent, accept, state=None, *, out_state=None, eps: float = 1e-6):
    """The state after the accepted path of a drafted tree: the recurrence over
    the nodes root .. ``accept[n]`` (int32 ``[N]``; -1 accepts nothing and copies
    the state).  The other arguments are kda_tree's.  ``out_state`` is a new
    tensor if None, or a given one, which may be ``state`` itself.  Returns it."""
    torch = _torch()
    cfg, N, L, H, dk, dv, dev = _tree_common(None, k, v, g, beta, parent, state, torch.float32, eps, 1.0)
    _check(accept, "accept", (N,), torch.int32, dev)
    if out_state is None:
        out_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if state is None else torch.empty_like(state)
    else:
        _check(out_state, "out_state", (N, H, dk, dv), torch.float32, dev)
    _launch(dev, _lib.kda_tree_commit_raw, cfg, N, _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(parent), _ptr(accept),
            _ptr(state), _ptr(out_state))
    return out_state


def _upstream(grad):
    """A gradient as the kernels take it: autograd may hand over a view of a larger tensor."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def _autograd_function():
    torch = _torch()
    from torch.autograd.function import once_differentiable

    class LinearFunction(torch.autograd.Function):
        """Autograd glue: the backward runs from the inputs, so nothing else is saved.
        Gradients flow to q, k, v, g and initial_state."""

        @staticmethod
        def forward(ctx, q, k, v, g, cu_seqlens, initial_state, num_seqs, scale, dg_dtype):
            o, sf = kda_linear_fwd(q, k, v, g, cu_seqlens, initial_state, num_seqs=num_seqs, scale=scale)
            ctx.save_for_backward(q, k, v, g, cu_seqlens, initial_state)
            ctx.set_materialize_grads(False)   # an output that the loss does not use has no gradient, not one of zeros
            ctx.num_seqs, ctx.scale, ctx.dg_dtype = num_seqs, scale, dg_dtype
            return o, sf

        @staticmethod
        @once_differentiable
        def backward(ctx, d_o, d_sf):
            q, k, v, g, cu_seqlens, s0 = ctx.saved_tensors
            d_o = _upstream((d_o if d_o is not None else torch.zeros_like(v)).to(q.dtype))
            d_sf = _upstream(d_sf) if d_sf is not None else None
            gr = kda_linear_bwd(q, k, v, g, d_o, cu_seqlens, s0, d_sf, num_seqs=ctx.num_seqs, out_dtype=q.dtype,
                                dg_dtype=ctx.dg_dtype, scale=ctx.scale, output_d_initial_state=s0 is not None)
            return gr["dq"], gr["dk"], gr["dv"], gr["dg"].to(g.dtype), None, gr["dS0"], None, None, None

    return LinearFunction


_FN = None


def kda_linear(q, k, v, g, cu_seqlens=None, initial_state=None, *, num_seqs: Optional[int] = None, scale: float = 1.0,
               dg_dtype=None):
    """kda_linear_fwd as a differentiable torch op: returns ``(o, final_state)``
    (fp32) and, under autograd, back-propagates through kda_linear_bwd.  The
    upstream gradient of o is cast to the input dtype, and the gradients of q,
    k, v and g are rounded to it; ``dg_dtype=torch.float32`` keeps g's as it is
    summed, which a fixed decay's gradient, a sum over all tokens, needs beside
    bf16 inputs.  A second differentiation is refused.

    In a captured graph use torch.autograd.grad, or leaves of which no eager graph
    is alive: torch ties a leaf's gradient accumulation to the stream of its first
    graph."""
    global _FN
    _check_dg_dtype(dg_dtype, q.dtype)
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(q, k, v, g, cu_seqlens, initial_state, num_seqs, scale, dg_dtype)
