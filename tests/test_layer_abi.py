"""The norm's, the short convolution's and the selective scan's C ABI and binding
without a GPU: sizes, refusals (every call fails its checks before any HIP call), and
the 64-bit references of tests/layer_ref.py against differences."""
import ctypes

import numpy as np
import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")

import gated_delta_rule_41_amd as kda
from gated_delta_rule_41_amd import _lib
from gated_delta_rule_41_amd._lib import (KDA_BF16, KDA_E4M3, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_F32,
                                          KDA_I8)

BASE = 1 << 40


def _err():
    return _lib.load().kda_last_error().decode()


class Call:
    """One entry point with distinct fake addresses for its pointers (never dereferenced: every call below fails its checks)."""

    def __init__(self, fn, make, names, optional=(), sizes=("T",), ws=None, **cfg):
        self.fn, self.make, self.names, self.optional, self.sizes, self.ws, self.cfg = fn, make, names, optional, sizes, ws, cfg

    def __call__(self, T=128, N=2, wsb=None, cfg=None, **kw):
        c = self.make(**self.cfg)
        for n, x in (cfg or {}).items():
            setattr(c, n, x)
        a = {n: 0 if n in self.optional else BASE + (i << 34) for i, n in enumerate(self.names)}
        a.update({n: x for n, x in kw.items()})
        size = [T, N][:len(self.sizes)] if self.sizes != ("N",) else [N]
        tail = []
        if self.ws:
            tail = [self.ws(c, *size) if wsb is None else wsb]
        return self.fn(c, *size, *(a[n] for n in self.names), *tail, 0)

    def at(self, name):
        return BASE + (self.names.index(name) << 34)


NORM = dict(C=64)
CONV = dict(C=64, width=4)
SEL = dict(C=64, S=16, G=2)
norm_fwd = Call(_lib.kda_norm_fwd_raw, _lib.make_norm_config, ("x", "residual", "weight", "y", "s", "scale"), ("scale",), **NORM)
norm_bwd = Call(_lib.kda_norm_bwd_raw, _lib.make_norm_config, ("s", "weight", "dy", "ds", "dx", "dweight", "workspace"), ("ds",),
                ws=_lib.kda_norm_bwd_workspace_size, **NORM)
conv_fwd = Call(_lib.kda_conv_fwd_raw, _lib.make_conv_config, ("x", "weight", "bias", "cu_seqlens", "initial_state", "y", "final_state"),
                ("bias",), ("T", "N"), **CONV)
conv_bwd = Call(_lib.kda_conv_bwd_raw, _lib.make_conv_config,
                ("x", "weight", "bias", "cu_seqlens", "initial_state", "dy", "d_final_state", "dx", "dweight", "dbias", "d_initial_state",
                 "workspace"), ("bias", "dbias"), ("T", "N"), _lib.kda_conv_bwd_workspace_size, **CONV)
conv_decode = Call(_lib.kda_conv_decode_raw, _lib.make_conv_config, ("x", "weight", "bias", "state_in", "state_out", "y"), ("bias",), ("N",),
                   **CONV)
SEL_IN = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
sel_fwd = Call(_lib.kda_selective_fwd_raw, _lib.make_selective_config,
               SEL_IN + ("cu_seqlens", "initial_state", "y", "final_state", "workspace"), (), ("T", "N"),
               _lib.kda_selective_fwd_workspace_size, **SEL)
sel_bwd = Call(_lib.kda_selective_bwd_raw, _lib.make_selective_config,
               SEL_IN + ("cu_seqlens", "initial_state", "dy", "dS_final", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias",
                         "d_initial_state", "workspace"), (), ("T", "N"), _lib.kda_selective_bwd_workspace_size, **SEL)
sel_decode = Call(_lib.kda_selective_decode_raw, _lib.make_selective_config, SEL_IN + ("state_in", "state_out", "y"), (), ("N",), **SEL)
ALL = {"norm_fwd": norm_fwd, "norm_bwd": norm_bwd, "conv_fwd": conv_fwd, "conv_bwd": conv_bwd, "conv_decode": conv_decode,
       "sel_fwd": sel_fwd, "sel_bwd": sel_bwd, "sel_decode": sel_decode}


@pytest.mark.parametrize("name", ALL)
def test_pointers_are_checked(name):
    call = ALL[name]
    may_be_null = {"residual", "weight" if name.startswith("norm") else "", "s" if name == "norm_fwd" else "", "bias", "cu_seqlens",
                   "initial_state", "final_state", "d_final_state", "dbias", "d_initial_state", "D", "z", "dt_bias", "state_in",
                   "dS_final", "dD", "ddt_bias", "ds", "scale", "dweight" if name == "norm_bwd" else ""}
    for p in call.names:
        assert call(**{p: BASE + 8}) == KDA_ERR_INVALID_ARG and "aligned" in _err(), p
        if p not in may_be_null and p != "workspace":
            assert call(**{p: 0}) == KDA_ERR_INVALID_ARG and _err().startswith(p), p


@pytest.mark.parametrize("name", ALL)
def test_null_configs_are_refused(name):
    call = ALL[name]
    n = len(call.names)
    fn = getattr(_lib.load(), call.fn.__name__[:-4])
    sizes = [128, 2][:len(call.sizes)] if call.sizes != ("N",) else [2]
    tail = [0, None] if call.ws else [None]
    assert fn(None, *sizes, *([None] * n), *tail) == KDA_ERR_INVALID_ARG
    if call.ws:
        assert getattr(_lib.load(), call.ws.__name__)(None, *sizes) == 0
    for init in ("norm", "conv", "selective"):
        getattr(_lib.load(), f"kda_{init}_config_init")(*([None] + [1] * {"norm": 1, "conv": 2, "selective": 3}[init]))


def test_norm_configs():
    for call in (norm_fwd, norm_bwd):
        for change, status in ((dict(C=0), KDA_ERR_INVALID_ARG), (dict(C=_lib.KDA_NORM_MAX_CHANNELS + 1), KDA_ERR_UNSUPPORTED),
                               (dict(in_dtype=2), KDA_ERR_INVALID_ARG), (dict(res_dtype=-1), KDA_ERR_INVALID_ARG),
                               (dict(weight_dtype=9), KDA_ERR_INVALID_ARG), (dict(out_dtype=4), KDA_ERR_INVALID_ARG),
                               (dict(eps=-1.0), KDA_ERR_INVALID_ARG), (dict(eps=float("nan")), KDA_ERR_INVALID_ARG),
                               (dict(in_dtype=KDA_F32, res_dtype=KDA_BF16), KDA_ERR_UNSUPPORTED)):
            assert call(cfg=change) == status, change
            assert _err()
        assert call(T=-1) == KDA_ERR_INVALID_ARG and call(T=1 << 30) == KDA_ERR_UNSUPPORTED
        assert _lib.kda_norm_bwd_workspace_size(_lib.make_norm_config(0), 5) == 0
    assert norm_bwd(cfg=dict(out_dtype=KDA_I8)) == KDA_ERR_INVALID_ARG
    for code in (KDA_I8, KDA_E4M3):
        assert norm_fwd(cfg=dict(out_dtype=code)) == KDA_ERR_INVALID_ARG and _err().startswith("scale")
    assert norm_fwd(cfg=dict(res_dtype=KDA_F32), residual=0) == KDA_ERR_INVALID_ARG and "res_dtype" in _err()
    need = _lib.kda_norm_bwd_workspace_size(_lib.make_norm_config(64), 128)
    assert need > 0 and norm_bwd(wsb=need - 1) == KDA_ERR_WORKSPACE
    assert norm_bwd(workspace=0) == KDA_ERR_INVALID_ARG


def test_norm_overlaps():
    half = 128 * 64      # bytes of half a tensor
    for a in ("x", "residual", "weight", "s"):
        off = 16 if a == "weight" else half
        assert norm_fwd(y=norm_fwd.at(a) + off) == KDA_ERR_INVALID_ARG and "overlap" in _err()
    for a in ("x", "residual"):
        assert norm_fwd(s=norm_fwd.at(a) + half) == KDA_ERR_INVALID_ARG and "overlap" in _err()
    # equal addresses, but of another type
    assert norm_fwd(cfg=dict(out_dtype=KDA_F32), y=norm_fwd.at("x")) == KDA_ERR_INVALID_ARG
    assert norm_fwd(cfg=dict(res_dtype=KDA_F32), s=norm_fwd.at("x")) == KDA_ERR_INVALID_ARG
    assert norm_fwd(y=norm_fwd.at("residual")) == KDA_ERR_INVALID_ARG
    for a in ("x", "residual", "y", "s"):
        assert norm_fwd(cfg=dict(out_dtype=KDA_I8), scale=norm_fwd.at(a)) == KDA_ERR_INVALID_ARG
    assert norm_bwd(dx=norm_bwd.at("s")) == KDA_ERR_INVALID_ARG
    assert norm_bwd(dx=norm_bwd.at("dy") + half) == KDA_ERR_INVALID_ARG
    assert norm_bwd(dweight=norm_bwd.at("dx")) == KDA_ERR_INVALID_ARG


def test_conv_configs():
    for call in (conv_fwd, conv_bwd, conv_decode):
        for change, status in ((dict(C=0), KDA_ERR_INVALID_ARG), (dict(C=_lib.KDA_CONV_MAX_CHANNELS + 1), KDA_ERR_UNSUPPORTED), (dict(width=1), KDA_ERR_UNSUPPORTED),
                               (dict(width=5), KDA_ERR_UNSUPPORTED), (dict(in_dtype=2), KDA_ERR_INVALID_ARG),
                               (dict(out_dtype=3), KDA_ERR_INVALID_ARG), (dict(weight_dtype=-1), KDA_ERR_INVALID_ARG),
                               (dict(activation=2), KDA_ERR_INVALID_ARG), (dict(x_stride=63), KDA_ERR_INVALID_ARG),
                               (dict(x_stride=-64), KDA_ERR_INVALID_ARG)):
            assert call(cfg=change) == status, change
    for call in (conv_fwd, conv_bwd):
        assert call(T=-1) == KDA_ERR_INVALID_ARG and call(T=1 << 31) == KDA_ERR_INVALID_ARG and call(N=0) == KDA_ERR_INVALID_ARG
        assert call(T=101, N=2, cu_seqlens=0) == KDA_ERR_INVALID_ARG
    assert conv_decode(N=-1) == KDA_ERR_INVALID_ARG and conv_decode(N=1 << 30) == KDA_ERR_UNSUPPORTED
    need = _lib.kda_conv_bwd_workspace_size(_lib.make_conv_config(64, 4), 128, 2)
    assert need > 0 and conv_bwd(wsb=need - 1) == KDA_ERR_WORKSPACE
    assert _lib.kda_conv_bwd_workspace_size(_lib.make_conv_config(64, 4), -1, 2) == 0


def test_conv_overlaps():
    assert conv_fwd(final_state=conv_fwd.at("initial_state")) == KDA_ERR_INVALID_ARG and "overlap" in _err()
    assert conv_fwd(y=conv_fwd.at("x")) == KDA_ERR_INVALID_ARG
    assert conv_fwd(cfg=dict(x_stride=128), y=conv_fwd.at("x") + 128 * 127 * 2) == KDA_ERR_INVALID_ARG
    assert conv_bwd(dx=conv_bwd.at("dy")) == KDA_ERR_INVALID_ARG and conv_bwd(dx=conv_bwd.at("x")) == KDA_ERR_INVALID_ARG
    for a in ("initial_state", "d_final_state"):
        assert conv_bwd(d_initial_state=conv_bwd.at(a)) == KDA_ERR_INVALID_ARG
    assert conv_decode(state_out=conv_decode.at("state_in") + 16) == KDA_ERR_INVALID_ARG and "overlap" in _err()


def test_selective_configs():
    for call in (sel_fwd, sel_bwd, sel_decode):
        for change, status in ((dict(C=0), KDA_ERR_INVALID_ARG), (dict(G=0), KDA_ERR_INVALID_ARG), (dict(G=3), KDA_ERR_INVALID_ARG),
                               (dict(C=_lib.KDA_SELECTIVE_MAX_CHANNELS + 2), KDA_ERR_UNSUPPORTED), (dict(S=64), KDA_ERR_UNSUPPORTED), (dict(S=12), KDA_ERR_UNSUPPORTED),
                               (dict(in_dtype=2), KDA_ERR_INVALID_ARG), (dict(out_dtype=2), KDA_ERR_INVALID_ARG),
                               (dict(flags=2), KDA_ERR_INVALID_ARG), (dict(x_stride=63), KDA_ERR_INVALID_ARG),
                               (dict(dt_stride=1), KDA_ERR_INVALID_ARG), (dict(z_stride=-1), KDA_ERR_INVALID_ARG),
                               (dict(b_stride=31), KDA_ERR_INVALID_ARG), (dict(c_stride=36), KDA_ERR_UNSUPPORTED)):
            assert call(cfg=change) == status, change
    for call in (sel_fwd, sel_bwd):
        assert call(T=-1) == KDA_ERR_INVALID_ARG and call(T=1 << 31) == KDA_ERR_INVALID_ARG and call(N=0) == KDA_ERR_INVALID_ARG
        assert call(T=101, N=2, cu_seqlens=0) == KDA_ERR_INVALID_ARG
        assert call(T=100, N=1 << 25) == KDA_ERR_UNSUPPORTED
    assert sel_decode(N=-1) == KDA_ERR_INVALID_ARG and sel_decode(N=1 << 30) == KDA_ERR_UNSUPPORTED
    cfg = _lib.make_selective_config(64, 16, 2)
    need = _lib.kda_selective_bwd_workspace_size(cfg, 128, 2)
    assert need > 0 and sel_bwd(wsb=need - 1) == KDA_ERR_WORKSPACE
    need = _lib.kda_selective_fwd_workspace_size(cfg, 4096, 2)
    assert need > 0 and sel_fwd(T=4096, wsb=need - 1) == KDA_ERR_WORKSPACE
    # a stream of one segment needs none
    assert _lib.kda_selective_fwd_workspace_size(cfg, 12, 1) == 0
    for T, N in ((-1, 1), (1 << 31, 1), (128, 0)):
        assert _lib.kda_selective_fwd_workspace_size(cfg, T, N) == 0 and _lib.kda_selective_bwd_workspace_size(cfg, T, N) == 0


def test_selective_overlaps():
    assert sel_fwd(final_state=sel_fwd.at("initial_state")) == KDA_ERR_INVALID_ARG and "overlap" in _err()
    for a in ("initial_state", "dS_final"):
        assert sel_bwd(d_initial_state=sel_bwd.at(a) + 64) == KDA_ERR_INVALID_ARG
    assert sel_decode(state_out=sel_decode.at("state_in") + 16) == KDA_ERR_INVALID_ARG and "overlap" in _err()


def test_config_structs_match_the_header():
    c = _lib.KdaNormConfig()
    _lib.load().kda_norm_config_init(ctypes.byref(c), 7)
    assert (c.C, c.in_dtype, c.res_dtype, c.weight_dtype, c.out_dtype) == (7, 0, 0, 0, 0) and abs(c.eps - 1e-6) < 1e-12
    c = _lib.KdaConvConfig()
    _lib.load().kda_conv_config_init(ctypes.byref(c), 7, 3)
    assert [getattr(c, n) for n, _ in c._fields_] == [7, 3, 0, 0, 0, 1, 0]
    c = _lib.KdaSelectiveConfig()
    _lib.load().kda_selective_config_init(ctypes.byref(c), 8, 16, 2)
    assert [getattr(c, n) for n, _ in c._fields_] == [8, 16, 2, 0, 0, 1, 0, 0, 0, 0, 0]


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, A, B = torch.zeros(5, 8), torch.zeros(8, 16), torch.zeros(5, 1, 16)
    w = torch.zeros(8, 4)
    for call in (lambda: kda.kda_norm_fwd(x), lambda: kda.kda_norm_bwd(x, None, x), lambda: kda.kda_conv_fwd(x, w),
                 lambda: kda.kda_conv_bwd(x, w, None, x), lambda: kda.kda_conv_decode(x, w), lambda: kda.kda_selective_fwd(x, x, A, B, B),
                 lambda: kda.kda_selective_bwd(x, x, A, B, B, x), lambda: kda.kda_selective_decode(x, x, A, B, B)):
        with pytest.raises(ValueError, match="GPU only"):
            call()
    with pytest.raises(ValueError, match="dimensions"):
        kda.kda_norm_fwd(x[0])
    with pytest.raises(ValueError, match="dimensions"):
        kda.kda_conv_fwd(x[None], w)


def _rows(stride, shape=(4, 6)):
    return torch.zeros(4, 40)[:, :shape[1]].as_strided(shape, stride)


def test_binding_row_strides():
    from gated_delta_rule_41_amd.layer import _rows as rows

    cpu, f32 = torch.device("cpu"), torch.float32
    assert rows(_rows((9, 1)), "x", (4, 6), f32, cpu) == 9
    assert rows(torch.zeros(4, 2, 3), "x", (4, 2, 3), f32, cpu) == 6
    assert rows(torch.zeros(4, 6)[:1], "x", (1, 6), f32, cpu) == 6
    assert rows(torch.zeros(0, 6), "x", (0, 6), f32, cpu) == 6
    for bad in ((0, 1), (5, 1), (9, 2)):
        with pytest.raises(ValueError):
            rows(_rows(bad), "x", (4, 6), f32, cpu)
    with pytest.raises(ValueError, match="shape"):
        rows(torch.zeros(4, 5), "x", (4, 6), f32, cpu)
    with pytest.raises(TypeError):
        rows(torch.zeros(4, 6).double(), "x", (4, 6), f32, cpu)


# ------------------------------------------------------------------ the references against differences
def _difference(f, x, i, step=1e-5):
    lo, hi = x.copy(), x.copy()
    lo.flat[i] -= step
    hi.flat[i] += step
    return (f(hi) - f(lo)) / (2 * step)


def test_norm_reference():
    rng = np.random.default_rng(1)
    s, w, dy, ds = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    dx, dw = ref.norm_bwd(s, w, dy, ds, 1e-3)
    for i in range(15):
        want = _difference(lambda v: (ref.norm_fwd(v, w, 1e-3)[0] * dy).sum() + (v * ds).sum(), s, i)
        assert abs(dx.flat[i] - want) < 1e-8
    for i in range(5):
        assert abs(dw[i] - _difference(lambda v: (ref.norm_fwd(s, v, 1e-3)[0] * dy).sum(), w, i)) < 1e-8


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_reference(W):
    rng = np.random.default_rng(W)
    lens, C = [4, 0, 1, 2], 3
    a = dict(x=rng.normal(size=(7, C)), w=rng.normal(size=(C, W)), b=rng.normal(size=C), state=rng.normal(size=(4, W - 1, C)))
    dy, dend = rng.normal(size=(7, C)), rng.normal(size=(4, W - 1, C))
    grads = ref.conv_bwd(a["x"], a["w"], a["b"], a["state"], lens, dy, dend)
    for n, name in (("x", "dx"), ("w", "dw"), ("b", "db"), ("state", "dstate")):
        def loss(v):
            y, end, _ = ref.conv_fwd(**{**a, n: v}, lens=lens)
            return (y * dy).sum() + (end * dend).sum()
        for i in range(a[n].size):
            assert abs(grads[name][0].flat[i] - _difference(loss, a[n], i)) < 1e-8, (name, i)


@pytest.mark.parametrize("gated,soft", [(True, True), (False, False)])
def test_selective_reference(gated, soft):
    rng = np.random.default_rng(7)
    lens, c, S, G, T = [3, 0, 1], 4, 8, 2, 4
    a = dict(x=rng.normal(size=(T, c)), raw=rng.normal(size=(T, c)) if soft else np.abs(rng.normal(size=(T, c))),
             A=-np.exp(rng.normal(size=(c, S))), B=rng.normal(size=(T, G, S)), C=rng.normal(size=(T, G, S)), D=rng.normal(size=c),
             z=rng.normal(size=(T, c)) if gated else None, bias=rng.normal(size=c), h0=rng.normal(size=(3, c, S)))
    dy, dh = rng.normal(size=(T, c)), rng.normal(size=(3, c, S))
    out = ref.selective(**a, lens=lens, soft=soft, dy=dy, dh=dh)
    bound = ref.selective_absolute(**a, lens=lens, soft=soft, dy=dy, dh=dh)
    for n, x in out.items():
        assert (np.abs(x) <= bound[n] * (1 + 1e-12)).all(), n
    names = {"x": "dx", "raw": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "bias": "dbias", "h0": "dh0"}
    for n, name in names.items():
        if a[n] is None:
            continue

        def loss(v):
            o = ref.selective(**{**a, n: v}, lens=lens, soft=soft)
            return (o["y"] * dy).sum() + (o["final"] * dh).sum()
        for i in range(a[n].size):
            assert abs(out[name].flat[i] - _difference(loss, a[n], i)) < 1e-7, (name, i)
