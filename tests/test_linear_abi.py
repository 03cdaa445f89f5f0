"""The linear rule's and the drafted trees' C ABI and binding without a GPU: sizes,
refusals (every call fails its checks before any HIP call), and the 64-bit
references of tests/linear_ref.py against closed forms and differences."""
import ctypes

import numpy as np
import pytest

import linear_ref as ref

torch = pytest.importorskip("torch")

import gated_delta_rule_41_amd as kda
from gated_delta_rule_41_amd import _lib
from gated_delta_rule_41_amd._lib import (KDA_BF16, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_F32,
                                          KDA_GATE_HEAD, KDA_RULE_DELTA, KDA_RULE_LINEAR)

FAKE = 0x10000


def _err():
    return _lib.load().kda_last_error().decode()


def lin(H=2, Hk=2, dk=64, dv=64, **kw):
    cfg = _lib.make_linear_config(H, Hk, 64, 64)
    cfg.dk, cfg.dv = dk, dv
    for n, x in kw.items():
        setattr(cfg, n, x)
    return cfg


def fwd(cfg, T=128, N=1, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, cu=0, s0=0, o=FAKE, sf=0, ws=0, wsb=0)
    a.update(kw)
    return _lib.kda_linear_fwd_raw(cfg, T, N, *(a[n] for n in ("q", "k", "v", "g", "cu", "s0", "o", "sf", "ws", "wsb")), 0)


def bwd(cfg, T=128, N=1, **kw):
    names = ("q", "k", "v", "g", "cu", "s0", "dO", "dS", "dq", "dk", "dv", "dg", "dS0", "ws", "wsb")
    a = dict.fromkeys(names, FAKE)
    a.update(cu=0, s0=0, dS=0, dS0=0, wsb=_lib.kda_linear_bwd_workspace_size(cfg, T, N) if cfg and T >= 0 and N > 0 else 0)
    a.update(kw)
    return _lib.kda_linear_bwd_raw(cfg, T, N, *(a[n] for n in names), 0)


def decode(cfg, N=3, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, si=0, so=FAKE, o=FAKE)
    a.update(kw)
    return _lib.kda_linear_decode_raw(cfg, N, *(a[n] for n in ("q", "k", "v", "g", "si", "so", "o")), 0)


def tree_cfg(rule=KDA_RULE_DELTA, nodes=8, **kw):
    cfg = _lib.make_tree_config(rule, 2, 2, 64, 64, nodes)
    for n, x in kw.items():
        setattr(cfg, n, x)
    return cfg


def tree(cfg, N=3, **kw):
    names = ("q", "k", "v", "g", "beta", "parent", "state", "o")
    a = dict.fromkeys(names, FAKE)
    a.update(kw)
    return _lib.kda_tree_raw(cfg, N, *(a[n] for n in names), 0)


def commit(cfg, N=3, **kw):
    names = ("k", "v", "g", "beta", "parent", "accept", "si", "so")
    a = dict.fromkeys(names, FAKE)
    a.update(kw)
    return _lib.kda_tree_commit_raw(cfg, N, *(a[n] for n in names), 0)


BAD_HEADS = [(dict(H=0), KDA_ERR_INVALID_ARG), (dict(Hk=0), KDA_ERR_INVALID_ARG), (dict(H=3), KDA_ERR_INVALID_ARG),
             (dict(dk=96), KDA_ERR_UNSUPPORTED), (dict(dv=32), KDA_ERR_UNSUPPORTED), (dict(in_dtype=7), KDA_ERR_INVALID_ARG),
             (dict(out_dtype=-1), KDA_ERR_INVALID_ARG), (dict(gate=2), KDA_ERR_INVALID_ARG),
             (dict(scale=float("nan")), KDA_ERR_INVALID_ARG)]


@pytest.mark.parametrize("change,status", BAD_HEADS)
def test_configs_are_refused(change, status):
    for call, cfg in ((fwd, lin(**change)), (bwd, lin(**change)), (decode, lin(**change)),
                      (tree, tree_cfg(KDA_RULE_LINEAR, **change)), (commit, tree_cfg(KDA_RULE_LINEAR, **change))):
        assert call(cfg) == status, call
        assert _err()
    assert _lib.kda_linear_fwd_workspace_size(lin(**change), 4096, 1) == 0
    assert _lib.kda_linear_bwd_workspace_size(lin(**change), 4096, 1) == 0


def test_null_configs_are_refused():
    lib = _lib.load()
    assert lib.kda_linear_fwd(None, 1, 1, *([None] * 9), 0, None) == KDA_ERR_INVALID_ARG
    assert lib.kda_linear_bwd(None, 1, 1, *([None] * 14), 0, None) == KDA_ERR_INVALID_ARG
    assert lib.kda_linear_decode(None, 1, *([None] * 8)) == KDA_ERR_INVALID_ARG
    assert lib.kda_tree(None, 1, *([None] * 9)) == KDA_ERR_INVALID_ARG
    assert lib.kda_tree_commit(None, 1, *([None] * 9)) == KDA_ERR_INVALID_ARG
    assert lib.kda_linear_fwd_workspace_size(None, 1, 1) == 0 and lib.kda_linear_bwd_workspace_size(None, 1, 1) == 0
    lib.kda_linear_config_init(None, 1, 1, 64, 64)
    lib.kda_tree_config_init(None, 0, 1, 1, 64, 64, 1)


def test_forward_and_backward_refuse_bad_arguments():
    cfg = lin()
    for call in (fwd, bwd):
        assert call(cfg, T=-1) == KDA_ERR_INVALID_ARG
        assert call(cfg, T=1 << 31) == KDA_ERR_INVALID_ARG
        assert call(cfg, N=0) == KDA_ERR_INVALID_ARG
        assert call(cfg, T=100, N=3) == KDA_ERR_INVALID_ARG
        assert call(cfg, T=(1 << 31) - 64, N=1) == KDA_ERR_UNSUPPORTED
        for name in ("q", "k", "v", "g"):
            assert call(cfg, **{name: 0}) == KDA_ERR_INVALID_ARG and _err().startswith(name + " ")
            assert call(cfg, **{name: FAKE + 4}) == KDA_ERR_INVALID_ARG and "aligned" in _err()
        for name in ("cu", "s0"):
            assert call(cfg, **{name: FAKE + 8}) == KDA_ERR_INVALID_ARG
    assert fwd(cfg, o=0) == KDA_ERR_INVALID_ARG and fwd(cfg, sf=FAKE + 2) == KDA_ERR_INVALID_ARG
    for name in ("dO", "dq", "dk", "dv", "dg"):
        assert bwd(cfg, **{name: 0}) == KDA_ERR_INVALID_ARG
    for name in ("dS", "dS0"):
        assert bwd(cfg, **{name: FAKE + 2}) == KDA_ERR_INVALID_ARG
    need = _lib.kda_linear_bwd_workspace_size(cfg, 128, 1)
    assert need > 0 and bwd(cfg, wsb=need - 1) == KDA_ERR_WORKSPACE and bwd(cfg, ws=0) == KDA_ERR_INVALID_ARG
    # a long document of few heads is cut into segments, which need a workspace; many heads need none
    need = _lib.kda_linear_fwd_workspace_size(cfg, 8192, 1)
    assert need > 0
    assert fwd(cfg, T=8192, ws=FAKE, wsb=need - 1) == KDA_ERR_WORKSPACE
    assert fwd(cfg, T=8192, ws=0, wsb=need) == KDA_ERR_INVALID_ARG
    assert _lib.kda_linear_fwd_workspace_size(lin(H=1024, Hk=1024), 8192, 1) == 0
    assert _lib.kda_linear_fwd_workspace_size(cfg, 128, 1) == 0
    # sizes that the calls refuse need no workspace either
    for T, N in ((-1, 1), (1 << 31, 1), (1 << 62, 1), ((1 << 31) - 64, 1), (128, 0), (128, -1)):
        assert _lib.kda_linear_fwd_workspace_size(cfg, T, N) == 0 and _lib.kda_linear_bwd_workspace_size(cfg, T, N) == 0
    # many value heads on one key head: the partial gradients stay a few times the gradients themselves
    for H in (8192, 8191):
        shared = _lib.kda_linear_bwd_workspace_size(lin(H=H, Hk=1), 256, 1)
        assert 0 < shared <= 1.05 * _lib.kda_linear_bwd_workspace_size(lin(H=H, Hk=H), 256, 1)
    big = lin(H=1 << 30, Hk=1 << 30)
    assert _lib.kda_linear_bwd_workspace_size(big, 1 << 20, 1) == 0 and fwd(big) == KDA_ERR_UNSUPPORTED


def test_packed_calls_refuse_overlapping_states():
    """The walks read and write states in one launch, so none of these may share memory, in place included."""
    cfg = lin()
    state, nbytes = 1 << 30, 3 * 2 * 64 * 64 * 4
    for other in (state, state + 16, state + nbytes - 16, state - nbytes + 16):
        for T in (129, 12288):   # whole documents and cut ones
            size = _lib.kda_linear_fwd_workspace_size(cfg, T, 3)
            assert fwd(cfg, T=T, N=3, s0=state, sf=other, ws=FAKE, wsb=size) == KDA_ERR_INVALID_ARG
            assert "overlap" in _err()
            for name in ("s0", "dS"):
                assert bwd(cfg, T=T, N=3, dS0=state, **{name: other}) == KDA_ERR_INVALID_ARG, name
                assert "overlap" in _err()


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_sizes_up_to_the_documented_limit(dk, dv):
    """(total_tokens / 128 + num_seqs + 8) * H below 2^21, whatever the head sizes."""
    cfg = lin(dk=dk, dv=dv)
    N = 1 << 19
    T = ((1 << 20) - 1 - 8 - N) * 128
    assert _lib.kda_linear_bwd_workspace_size(cfg, T, N) > 0
    assert _lib.kda_linear_bwd_workspace_size(cfg, T + 128, N) == 0 and "too large" in _err()
    assert _lib.kda_linear_bwd_workspace_size(cfg, 600000, 600000) > 0
    assert fwd(cfg, T=T + 128, N=N) == KDA_ERR_UNSUPPORTED and bwd(cfg, T=T + 128, N=N) == KDA_ERR_UNSUPPORTED


def test_prime_numbers_of_value_heads_are_divided():
    """Few workgroups' worth of tokens with 7 or 127 value heads to a key head: partial sums of dq and dk for each."""
    for T, H, Hk in ((1152, 28, 4), (1024, 127, 1)):
        whole = _lib.kda_linear_bwd_workspace_size(lin(H=H, Hk=H), T, 1)
        assert _lib.kda_linear_bwd_workspace_size(lin(H=H, Hk=Hk), T, 1) == whole + 2 * T * H * 64 * 4, (T, H)


def test_dg_in_fp32_is_a_bit_of_the_gate():
    flag = _lib.KDA_GATE_GRAD_F32
    for gate in (0, KDA_GATE_HEAD):
        a, b = lin(gate=gate), lin(gate=gate | flag)
        for T, N in ((128, 1), (8192, 3)):
            assert _lib.kda_linear_bwd_workspace_size(b, T, N) == _lib.kda_linear_bwd_workspace_size(a, T, N) > 0
            assert _lib.kda_linear_fwd_workspace_size(b, T, N) == _lib.kda_linear_fwd_workspace_size(a, T, N)
        # each call gets as far as its pointers
        for call in (fwd, bwd, decode):
            assert call(b, q=0) == KDA_ERR_INVALID_ARG and _err().startswith("q ")
    for gate in (2 | flag, flag << 1, -1):
        for call in (fwd, bwd, decode):
            assert call(lin(gate=gate)) == KDA_ERR_INVALID_ARG and "gate" in _err()
    for call in (tree, commit):
        assert call(tree_cfg(KDA_RULE_LINEAR, gate=flag)) == KDA_ERR_INVALID_ARG


def test_decode_refuses_bad_arguments():
    cfg = lin()
    assert decode(cfg, N=-1) == KDA_ERR_INVALID_ARG
    assert decode(cfg, N=1 << 30) == KDA_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "g", "so", "o"):
        assert decode(cfg, **{name: 0}) == KDA_ERR_INVALID_ARG
        assert decode(cfg, **{name: FAKE + 4}) == KDA_ERR_INVALID_ARG
    assert decode(cfg, si=FAKE + 16) == KDA_ERR_INVALID_ARG and "overlap" in _err()
    assert decode(cfg, si=FAKE + 2) == KDA_ERR_INVALID_ARG


def test_trees_refuse_bad_arguments():
    for call in (tree, commit):
        for nodes in (0, -1, 65):
            assert call(tree_cfg(nodes=nodes)) == KDA_ERR_UNSUPPORTED
        assert call(tree_cfg(rule=2)) == KDA_ERR_INVALID_ARG
        assert call(tree_cfg(Hk=1)) == KDA_ERR_UNSUPPORTED                      # delta rule: no shared key heads
        assert call(tree_cfg(gate=KDA_GATE_HEAD)) == KDA_ERR_UNSUPPORTED
        assert call(tree_cfg(l2_eps=-1.0)) == KDA_ERR_INVALID_ARG
        assert call(tree_cfg(l2_eps=float("inf"))) == KDA_ERR_INVALID_ARG
        assert call(tree_cfg(), N=-1) == KDA_ERR_INVALID_ARG
        assert call(tree_cfg(), N=1 << 30) == KDA_ERR_UNSUPPORTED
        for name in ("k", "v", "g", "beta", "parent"):
            assert call(tree_cfg(), **{name: 0}) == KDA_ERR_INVALID_ARG and _err().startswith(name + " ")
            assert call(tree_cfg(), **{name: FAKE + 4}) == KDA_ERR_INVALID_ARG
    assert tree(tree_cfg(), q=0) == KDA_ERR_INVALID_ARG and tree(tree_cfg(), o=0) == KDA_ERR_INVALID_ARG
    assert commit(tree_cfg(), accept=0) == KDA_ERR_INVALID_ARG and commit(tree_cfg(), so=0) == KDA_ERR_INVALID_ARG
    assert commit(tree_cfg(), si=FAKE + 64) == KDA_ERR_INVALID_ARG and "overlap" in _err()


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q, v, g = torch.zeros(5, 2, 64), torch.zeros(5, 2, 64), torch.zeros(5, 2)
    with pytest.raises(ValueError, match="GPU only"):
        kda.kda_linear_fwd(q, q, v, g)
    with pytest.raises(ValueError, match="GPU only"):
        kda.kda_linear_decode(q, q, v, g)
    with pytest.raises(ValueError, match="GPU only"):
        kda.kda_tree(q[None], q[None], v[None], g[None], None, torch.zeros(1, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        kda.kda_tree(q, q, v, g, None, torch.zeros(1, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        kda.kda_linear_fwd(q[0], q, v, g)


def test_config_structs_match_the_header():
    """The defaults that the init functions write, read back through the binding's structs."""
    cfg = _lib.KdaLinearConfig()
    _lib.load().kda_linear_config_init(ctypes.byref(cfg), 6, 3, 128, 64)
    assert [getattr(cfg, n) for n, _ in cfg._fields_] == [6, 3, 128, 64, KDA_F32, KDA_F32, 0, 1.0]
    cfg = _lib.KdaTreeConfig()
    _lib.load().kda_tree_config_init(ctypes.byref(cfg), 1, 6, 3, 128, 64, 9)
    got = [getattr(cfg, n) for n, _ in cfg._fields_]
    assert got[:9] == [1, 6, 3, 128, 64, 9, KDA_F32, KDA_F32, 0] and abs(got[9] - 1e-6) < 1e-12 and got[10] == 1.0
    assert KDA_BF16 == 1


# ------------------------------------------------------------------ the references themselves
def _random(seed, lens, H=4, Hk=2, dk=3, dv=5, gate="token"):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    x = dict(q=rng.standard_normal((T, Hk, dk)), k=rng.standard_normal((T, Hk, dk)), v=rng.standard_normal((T, H, dv)),
             g=-np.abs(rng.standard_normal((T, H) if gate == "token" else H)), s0=rng.standard_normal((N, H, dk, dv)))
    return x, rng.standard_normal((T, H, dv)), rng.standard_normal((N, H, dk, dv))


def test_reference_forward_against_the_sum_over_pairs():
    lens = [4, 1, 6]
    x, _, _ = _random(1, lens)
    o, final, _ = ref.linear_fwd(x["q"], x["k"], x["v"], x["g"], lens, x["s0"], 0.5)
    lo = 0
    for n, length in enumerate(lens):
        for h in range(4):
            for i in range(lo, lo + length):
                want = 0.5 * np.exp(x["g"][lo:i + 1, h].sum()) * x["q"][i, h // 2] @ x["s0"][n, h]
                for j in range(lo, i + 1):
                    want = want + 0.5 * np.exp(x["g"][j + 1:i + 1, h].sum()) * (x["q"][i, h // 2] @ x["k"][j, h // 2]) * x["v"][j, h]
                assert np.allclose(o[i, h], want, rtol=1e-12, atol=1e-12)
        lo += length


@pytest.mark.parametrize("gate", ["token", "head"])
def test_reference_backward_against_differences(gate):
    lens = [5, 3]
    x, dO, dS = _random(2, lens, gate=gate)
    gr = ref.linear_bwd(x["q"], x["k"], x["v"], x["g"], lens, dO, x["s0"], dS, 0.5)

    def loss(**kw):
        y = dict(x, **kw)
        o, final, _ = ref.linear_fwd(y["q"], y["k"], y["v"], y["g"], lens, y["s0"], 0.5)
        return (o * dO).sum() + (final * dS).sum()

    rng = np.random.default_rng(3)
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "dS0")):
        u = rng.standard_normal(x[n].shape)
        diff = (loss(**{n: x[n] + 1e-5 * u}) - loss(**{n: x[n] - 1e-5 * u})) / 2e-5
        assert abs(diff - (gr[gn] * u).sum()) <= 1e-6 * (1 + np.abs(gr[gn] * u).sum()), n


def test_reference_tree_of_one_path_is_the_recurrence():
    rng = np.random.default_rng(4)
    N, L, H, d = 1, 6, 2, 4
    q, k, v = (rng.standard_normal((N, L, H, d)) for _ in range(3))
    g, s0 = -np.abs(rng.standard_normal((N, L, H))), rng.standard_normal((N, H, d, d))
    parent = [[-1, 0, 0, 1, -1, 3]]
    o, states = ref.tree(q, k, v, g, None, parent, s0)
    path = [0, 1, 3, 5]
    o2, final, _ = ref.linear_fwd(q[0, path], k[0, path], v[0, path], g[0, path], [4], s0)
    assert np.allclose(o[0, path], o2, rtol=1e-13) and np.allclose(states[0][5], final[0], rtol=1e-13)
    # delta rule: beta -> 0 leaves pure decay
    gd = -np.abs(rng.standard_normal((N, L, H, d)))
    _, states = ref.tree(q, k, v, gd, np.full((N, L, H), -700.0), parent, s0)
    assert np.allclose(states[0][5][:, :, 0], np.exp(gd[0, path].sum(0)) * s0[0, :, :, 0], rtol=1e-13)
