"""ctypes binding of libkda (include/kda.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libkda.so.  PyTorch supplies device memory and the stream.  There is
no fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "kda.h")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_HIP = range(5)
KDA_F32, KDA_BF16 = 0, 1
KDA_FLAG_SAVE_FOR_BWD = 1
KDA_FLAG_SEQUENTIAL = 2
KDA_FLAG_STAGED = 4
# kda_stage (include/kda.h), in order
STAGES = ("G", "Akk", "Aqk", "T", "W", "Ut", "U", "S_in", "QG", "Ktil", "GamC")


class KdaConfig(ctypes.Structure):
    _fields_ = [
        ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("chunk", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("l2_eps", ctypes.c_float),
        ("scale", ctypes.c_float),
        ("flags", ctypes.c_uint32),
    ]


KDA_GATE_TOKEN, KDA_GATE_HEAD = 0, 1
KDA_GATE_GRAD_F32 = 0x100
KDA_RULE_DELTA, KDA_RULE_LINEAR = 0, 1
KDA_TREE_MAX_NODES = 64
KDA_I8, KDA_E4M3 = 2, 3   # outputs of kda_norm_fwd
KDA_NORM_MAX_CHANNELS, KDA_CONV_MAX_CHANNELS, KDA_SELECTIVE_MAX_CHANNELS = 16384, 1 << 20, 1 << 16
KDA_ACT_NONE, KDA_ACT_SILU = 0, 1
KDA_SELECTIVE_SOFTPLUS = 1


class KdaLinearConfig(ctypes.Structure):
    _fields_ = [
        ("H", ctypes.c_int32),
        ("Hk", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class KdaTreeConfig(ctypes.Structure):
    _fields_ = [
        ("rule", ctypes.c_int32),
        ("H", ctypes.c_int32),
        ("Hk", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("nodes", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("l2_eps", ctypes.c_float),
        ("scale", ctypes.c_float),
    ]


class KdaNormConfig(ctypes.Structure):
    _fields_ = [
        ("C", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("res_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class KdaConvConfig(ctypes.Structure):
    _fields_ = [
        ("C", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("x_stride", ctypes.c_int64),
    ]


class KdaSelectiveConfig(ctypes.Structure):
    _fields_ = [
        ("C", ctypes.c_int32),
        ("S", ctypes.c_int32),
        ("G", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("x_stride", ctypes.c_int64),
        ("dt_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64),
        ("b_stride", ctypes.c_int64),
        ("c_stride", ctypes.c_int64),
    ]


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libkda status {status}: {message}")
        self.status = status


_lib = None
_vp = ctypes.c_void_p


def header_functions() -> list[str]:
    """Names of the functions declared in include/kda.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kda_[a-z_]+)\s*\(", text)))


def load():
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    # One HIP runtime per process.  PyTorch ships its own libamdhip64 and
    # libhsa-runtime64; loading torch first makes libkda.so bind to those (same
    # soname) instead of pulling in a second copy from the ROCm install, and two
    # runtimes in one process compete for the device.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(LIB_PATH)
    cfgp = ctypes.POINTER(KdaConfig)
    lib.kda_config_init.argtypes = [cfgp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    lib.kda_config_init.restype = None
    lib.kda_stage_offset.argtypes = [cfgp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
    lib.kda_stage_offset.restype = ctypes.c_size_t
    for name in ("kda_saved_size", "kda_fwd_workspace_size", "kda_bwd_workspace_size"):
        fn = getattr(lib, name)
        fn.argtypes = [cfgp, ctypes.c_int64, ctypes.c_int32]
        fn.restype = ctypes.c_size_t
    lib.kda_fwd.argtypes = ([cfgp, ctypes.c_int64, ctypes.c_int32] + [_vp] * 10 + [ctypes.c_size_t, _vp]
                            + [ctypes.c_size_t, _vp])
    lib.kda_fwd.restype = ctypes.c_int
    lib.kda_fwd_static.argtypes = [cfgp, ctypes.c_int64, ctypes.c_int32] + [_vp] * 10 + [ctypes.c_size_t, _vp]
    lib.kda_fwd_static.restype = ctypes.c_int
    for name in ("kda_bwd", "kda_bwd_scan", "kda_bwd_grads"):
        fn = getattr(lib, name)
        fn.argtypes = ([cfgp, ctypes.c_int64, ctypes.c_int32] + [_vp] * 8 + [ctypes.c_size_t] + [_vp] * 9
                       + [ctypes.c_size_t, _vp])
        fn.restype = ctypes.c_int
    lib.kda_decode.argtypes = [cfgp, ctypes.c_int32] + [_vp] * 9
    lib.kda_decode.restype = ctypes.c_int
    lincfg, treecfg, i32, size = ctypes.POINTER(KdaLinearConfig), ctypes.POINTER(KdaTreeConfig), ctypes.c_int32, ctypes.c_size_t
    lib.kda_linear_config_init.argtypes = [lincfg] + [i32] * 4
    lib.kda_linear_config_init.restype = None
    for name in ("kda_linear_fwd_workspace_size", "kda_linear_bwd_workspace_size"):
        fn = getattr(lib, name)
        fn.argtypes = [lincfg, ctypes.c_int64, i32]
        fn.restype = size
    lib.kda_linear_fwd.argtypes = [lincfg, ctypes.c_int64, i32] + [_vp] * 9 + [size, _vp]
    lib.kda_linear_bwd.argtypes = [lincfg, ctypes.c_int64, i32] + [_vp] * 14 + [size, _vp]
    lib.kda_linear_decode.argtypes = [lincfg, i32] + [_vp] * 8
    lib.kda_tree_config_init.argtypes = [treecfg] + [i32] * 6
    lib.kda_tree_config_init.restype = None
    lib.kda_tree.argtypes = [treecfg, i32] + [_vp] * 9
    lib.kda_tree_commit.argtypes = [treecfg, i32] + [_vp] * 9
    for name in ("kda_linear_fwd", "kda_linear_bwd", "kda_linear_decode", "kda_tree", "kda_tree_commit"):
        getattr(lib, name).restype = ctypes.c_int
    i64, norm, conv, sel = ctypes.c_int64, *(ctypes.POINTER(c) for c in (KdaNormConfig, KdaConvConfig, KdaSelectiveConfig))
    for name, res, args in (
            ("kda_norm_config_init", None, [norm, i32]),
            ("kda_norm_fwd", i32, [norm, i64] + [_vp] * 7),
            ("kda_norm_bwd_workspace_size", size, [norm, i64]),
            ("kda_norm_bwd", i32, [norm, i64] + [_vp] * 7 + [size, _vp]),
            ("kda_conv_config_init", None, [conv, i32, i32]),
            ("kda_conv_fwd", i32, [conv, i64, i32] + [_vp] * 8),
            ("kda_conv_bwd_workspace_size", size, [conv, i64, i32]),
            ("kda_conv_bwd", i32, [conv, i64, i32] + [_vp] * 12 + [size, _vp]),
            ("kda_conv_decode", i32, [conv, i32] + [_vp] * 7),
            ("kda_selective_config_init", None, [sel, i32, i32, i32]),
            ("kda_selective_fwd_workspace_size", size, [sel, i64, i32]),
            ("kda_selective_bwd_workspace_size", size, [sel, i64, i32]),
            ("kda_selective_fwd", i32, [sel, i64, i32] + [_vp] * 13 + [size, _vp]),
            ("kda_selective_bwd", i32, [sel, i64, i32] + [_vp] * 22 + [size, _vp]),
            ("kda_selective_decode", i32, [sel, i32] + [_vp] * 12)):
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_last_error.argtypes = []
    lib.kda_last_error.restype = ctypes.c_char_p
    lib.kda_version.argtypes = []
    lib.kda_version.restype = ctypes.c_int32
    _lib = lib
    return lib


def make_config(H, dk, dv, in_dtype=KDA_BF16, out_dtype=KDA_F32, eps=1e-6, scale=1.0, flags=0):
    cfg = KdaConfig()
    load().kda_config_init(ctypes.byref(cfg), H, dk, dv)
    cfg.in_dtype, cfg.out_dtype = in_dtype, out_dtype
    cfg.l2_eps, cfg.scale, cfg.flags = eps, scale, flags
    return cfg


def check(status: int):
    if status != KDA_OK:
        lib = load()
        raise KdaError(status, f"{lib.kda_status_string(status).decode()}: {lib.kda_last_error().decode()}")


def kda_saved_size(cfg: KdaConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_saved_size(ctypes.byref(cfg), total_tokens, num_seqs))


def kda_fwd_workspace_size(cfg: KdaConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_fwd_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs))


def kda_stage_offset(cfg: KdaConfig, total_tokens: int, num_seqs: int, stage: int) -> int:
    return int(load().kda_stage_offset(ctypes.byref(cfg), total_tokens, num_seqs, stage))


def kda_bwd_workspace_size(cfg: KdaConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_bwd_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs))


def kda_fwd_raw(cfg, total_tokens, num_seqs, q, k, v, g, beta, cu_seqlens, initial_state, o,
                final_state, saved, saved_bytes, workspace, workspace_bytes, stream) -> int:
    """Direct call of kda_fwd with integer device addresses (0 = NULL); returns the status."""
    return load().kda_fwd(ctypes.byref(cfg), total_tokens, num_seqs, q, k, v, g, beta, cu_seqlens,
                          initial_state, o, final_state, saved, saved_bytes, workspace, workspace_bytes, stream)


KDA_STATIC_WORKSPACE_BYTES = 128 << 20


def kda_fwd_static_raw(cfg, total_tokens, num_seqs, q, k, v, g, beta, cu_seqlens, initial_state, o,
                       final_state, saved, saved_bytes, stream) -> int:
    """Direct call of kda_fwd_static (the forward on the library's static
    workspace) with integer device addresses (0 = NULL); returns the status."""
    return load().kda_fwd_static(ctypes.byref(cfg), total_tokens, num_seqs, q, k, v, g, beta, cu_seqlens,
                                 initial_state, o, final_state, saved, saved_bytes, stream)


BWD_ENTRY = {"all": "kda_bwd", "scan": "kda_bwd_scan", "grads": "kda_bwd_grads"}


def kda_bwd_raw(cfg, total_tokens, num_seqs, q, k, v, g, beta, cu_seqlens, initial_state, saved, saved_bytes,
                dO, dS_final, dq, dk, dv, dg, dbeta, d_initial_state, workspace, workspace_bytes,
                stream, stage: str = "all") -> int:
    """Direct call of kda_bwd (stage "all"), kda_bwd_scan ("scan") or kda_bwd_grads
    ("grads") with integer device addresses (0 = NULL); returns the status."""
    fn = getattr(load(), BWD_ENTRY[stage])
    return fn(ctypes.byref(cfg), total_tokens, num_seqs, q, k, v, g, beta, cu_seqlens, initial_state, saved,
              saved_bytes, dO, dS_final, dq, dk, dv, dg, dbeta, d_initial_state, workspace, workspace_bytes, stream)


def kda_decode_raw(cfg, num_seqs, q, k, v, g, beta, state_in, state_out, o, stream) -> int:
    """Direct call of kda_decode with integer device addresses (0 = NULL); returns the status."""
    return load().kda_decode(ctypes.byref(cfg), num_seqs, q, k, v, g, beta, state_in, state_out, o, stream)


# ---- the linear rule and drafted trees: direct calls with integer device addresses (0 = NULL)
def make_linear_config(H, Hk, dk, dv, in_dtype=KDA_BF16, out_dtype=KDA_F32, gate=KDA_GATE_TOKEN, scale=1.0):
    cfg = KdaLinearConfig()
    load().kda_linear_config_init(ctypes.byref(cfg), H, Hk, dk, dv)
    cfg.in_dtype, cfg.out_dtype, cfg.gate, cfg.scale = in_dtype, out_dtype, gate, scale
    return cfg


def make_tree_config(rule, H, Hk, dk, dv, nodes, in_dtype=KDA_BF16, out_dtype=KDA_F32, gate=KDA_GATE_TOKEN, eps=1e-6,
                     scale=1.0):
    cfg = KdaTreeConfig()
    load().kda_tree_config_init(ctypes.byref(cfg), rule, H, Hk, dk, dv, nodes)
    cfg.in_dtype, cfg.out_dtype, cfg.gate, cfg.l2_eps, cfg.scale = in_dtype, out_dtype, gate, eps, scale
    return cfg


def kda_linear_fwd_workspace_size(cfg: KdaLinearConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_linear_fwd_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs))


def kda_linear_bwd_workspace_size(cfg: KdaLinearConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_linear_bwd_workspace_size(ctypes.byref(cfg), total_tokens, num_seqs))


def kda_linear_fwd_raw(cfg, total_tokens, num_seqs, q, k, v, g, cu_seqlens, initial_state, o, final_state, workspace,
                       workspace_bytes, stream) -> int:
    return load().kda_linear_fwd(ctypes.byref(cfg), total_tokens, num_seqs, q, k, v, g, cu_seqlens, initial_state, o,
                                 final_state, workspace, workspace_bytes, stream)


def kda_linear_bwd_raw(cfg, total_tokens, num_seqs, q, k, v, g, cu_seqlens, initial_state, dO, dS_final, dq, dk, dv, dg,
                       d_initial_state, workspace, workspace_bytes, stream) -> int:
    return load().kda_linear_bwd(ctypes.byref(cfg), total_tokens, num_seqs, q, k, v, g, cu_seqlens, initial_state, dO,
                                 dS_final, dq, dk, dv, dg, d_initial_state, workspace, workspace_bytes, stream)


def kda_linear_decode_raw(cfg, num_seqs, q, k, v, g, state_in, state_out, o, stream) -> int:
    return (_lib or load()).kda_linear_decode(cfg, num_seqs, q, k, v, g, state_in, state_out, o, stream)


def kda_tree_raw(cfg, num_seqs, q, k, v, g, beta, parent, state, o, stream) -> int:
    return (_lib or load()).kda_tree(cfg, num_seqs, q, k, v, g, beta, parent, state, o, stream)


def kda_tree_commit_raw(cfg, num_seqs, k, v, g, beta, parent, accept, state_in, state_out, stream) -> int:
    return (_lib or load()).kda_tree_commit(cfg, num_seqs, k, v, g, beta, parent, accept, state_in, state_out, stream)


# ---- the norm, the short convolution and the selective scan: direct calls with integer device addresses (0 = NULL)
def make_norm_config(C, in_dtype=KDA_BF16, res_dtype=KDA_BF16, weight_dtype=KDA_BF16, out_dtype=KDA_BF16, eps=1e-6):
    cfg = KdaNormConfig()
    load().kda_norm_config_init(ctypes.byref(cfg), C)
    cfg.in_dtype, cfg.res_dtype, cfg.weight_dtype, cfg.out_dtype, cfg.eps = in_dtype, res_dtype, weight_dtype, out_dtype, eps
    return cfg


def make_conv_config(C, width, in_dtype=KDA_BF16, out_dtype=KDA_BF16, weight_dtype=KDA_BF16, activation=KDA_ACT_SILU, x_stride=0):
    cfg = KdaConvConfig()
    load().kda_conv_config_init(ctypes.byref(cfg), C, width)
    cfg.in_dtype, cfg.out_dtype, cfg.weight_dtype, cfg.activation, cfg.x_stride = in_dtype, out_dtype, weight_dtype, activation, x_stride
    return cfg


def make_selective_config(C, S, G=1, in_dtype=KDA_BF16, out_dtype=KDA_BF16, flags=KDA_SELECTIVE_SOFTPLUS, x_stride=0, dt_stride=0,
                          z_stride=0, b_stride=0, c_stride=0):
    cfg = KdaSelectiveConfig()
    load().kda_selective_config_init(ctypes.byref(cfg), C, S, G)
    cfg.in_dtype, cfg.out_dtype, cfg.flags, cfg.x_stride, cfg.dt_stride = in_dtype, out_dtype, flags, x_stride, dt_stride
    cfg.z_stride, cfg.b_stride, cfg.c_stride = z_stride, b_stride, c_stride
    return cfg


def kda_norm_bwd_workspace_size(cfg: KdaNormConfig, rows: int) -> int:
    return int(load().kda_norm_bwd_workspace_size(cfg, rows))


def kda_conv_bwd_workspace_size(cfg: KdaConvConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_conv_bwd_workspace_size(cfg, total_tokens, num_seqs))


def kda_selective_fwd_workspace_size(cfg: KdaSelectiveConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_selective_fwd_workspace_size(cfg, total_tokens, num_seqs))


def kda_selective_bwd_workspace_size(cfg: KdaSelectiveConfig, total_tokens: int, num_seqs: int) -> int:
    return int(load().kda_selective_bwd_workspace_size(cfg, total_tokens, num_seqs))


def kda_norm_fwd_raw(cfg, rows, x, residual, weight, y, s, scale, stream) -> int:
    return (_lib or load()).kda_norm_fwd(cfg, rows, x, residual, weight, y, s, scale, stream)


def kda_norm_bwd_raw(cfg, rows, s, weight, dy, ds, dx, dweight, workspace, workspace_bytes, stream) -> int:
    return (_lib or load()).kda_norm_bwd(cfg, rows, s, weight, dy, ds, dx, dweight, workspace, workspace_bytes, stream)


def kda_conv_fwd_raw(cfg, total_tokens, num_seqs, x, weight, bias, cu_seqlens, initial_state, y, final_state, stream) -> int:
    return (_lib or load()).kda_conv_fwd(cfg, total_tokens, num_seqs, x, weight, bias, cu_seqlens, initial_state, y, final_state, stream)


def kda_conv_bwd_raw(cfg, total_tokens, num_seqs, x, weight, bias, cu_seqlens, initial_state, dy, d_final_state, dx, dweight, dbias,
                     d_initial_state, workspace, workspace_bytes, stream) -> int:
    return (_lib or load()).kda_conv_bwd(cfg, total_tokens, num_seqs, x, weight, bias, cu_seqlens, initial_state, dy, d_final_state, dx,
                                         dweight, dbias, d_initial_state, workspace, workspace_bytes, stream)


def kda_conv_decode_raw(cfg, num_seqs, x, weight, bias, state_in, state_out, y, stream) -> int:
    return (_lib or load()).kda_conv_decode(cfg, num_seqs, x, weight, bias, state_in, state_out, y, stream)


def kda_selective_fwd_raw(cfg, total_tokens, num_seqs, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, y, final_state,
                          workspace, workspace_bytes, stream) -> int:
    return (_lib or load()).kda_selective_fwd(cfg, total_tokens, num_seqs, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, y,
                                              final_state, workspace, workspace_bytes, stream)


def kda_selective_bwd_raw(cfg, total_tokens, num_seqs, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, dy, dS_final, dx, ddt,
                          dA, dB, dC, dD, dz, ddt_bias, d_initial_state, workspace, workspace_bytes, stream) -> int:
    return (_lib or load()).kda_selective_bwd(cfg, total_tokens, num_seqs, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, dy,
                                              dS_final, dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_initial_state, workspace,
                                              workspace_bytes, stream)


def kda_selective_decode_raw(cfg, num_seqs, x, dt, A, B, C, D, z, dt_bias, state_in, state_out, y, stream) -> int:
    return (_lib or load()).kda_selective_decode(cfg, num_seqs, x, dt, A, B, C, D, z, dt_bias, state_in, state_out, y, stream)
