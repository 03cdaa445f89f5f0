"""The selective scan against 64 bits: types, states, groups, documents, gradients, single tokens, extreme decays."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
GRADS = {"dx": "dx", "ddt": "ddt", "dA": "dA", "dB": "dB", "dC": "dC", "dD": "dD", "dz": "dz", "dbias": "ddt_bias", "dh0": "dS0"}


def host(t):
    return t.detach().double().cpu().numpy()


def make(lens, c, S, G, dtype, seed=0, gated=True):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, dt=dtype):
        return torch.randn(*shape, generator=gen).to(dt).cuda()

    T, N = sum(lens), len(lens)
    d = {"x": normal(T, c), "raw": normal(T, c), "A": -torch.exp(normal(c, S, dt=F32)), "B": normal(T, G, S), "C": normal(T, G, S),
         "D": normal(c, dt=F32), "z": normal(T, c) if gated else None, "bias": normal(c, dt=F32) - 3, "h0": normal(N, c, S, dt=F32),
         "dy": normal(T, c), "dh": normal(N, c, S, dt=F32)}
    d["cu"] = torch.tensor(ref.starts(lens), dtype=torch.int32, device="cuda")
    return d


def fwd(d, cu="cu", **kw):
    return kda.kda_selective_fwd(d["x"], d["raw"], d["A"], d["B"], d["C"], d["cu"] if cu else None, d["h0"], D=d["D"], z=d["z"],
                                 dt_bias=d["bias"], **kw)


def bwd(d, cu="cu", **kw):
    return kda.kda_selective_bwd(d["x"], d["raw"], d["A"], d["B"], d["C"], d["dy"], d["cu"] if cu else None, d["h0"], d["dh"], D=d["D"],
                                 z=d["z"], dt_bias=d["bias"], **kw)


def exact(d, lens, soft=True, backward=True):
    h = {n: None if x is None else host(x) for n, x in d.items() if n != "cu"}
    a = dict(x=h["x"], raw=h["raw"], A=h["A"], B=h["B"], C=h["C"], D=h["D"], z=h["z"], bias=h["bias"], lens=lens, h0=h["h0"], soft=soft)
    if backward:
        a.update(dy=h["dy"], dh=h["dh"])
    return ref.selective(**a), ref.selective_absolute(**a), ref.selective_roundings(h["raw"], h["A"], h["bias"], lens, soft)


def check(got, want, most, count, dtype, name):
    """Every element within `count` roundings of its absolute sum, and the whole within the root of as many: they are independent."""
    assert got.dtype == dtype, name
    got = host(got)
    off = np.abs(got - want)
    assert (off <= (most * count * ref.U + np.abs(want) * HALF[dtype]) * 1.01 + 1e-37).all(), (name, (off / (most * ref.U + 1e-37)).max())
    assert np.linalg.norm(off) <= np.linalg.norm(most) * np.sqrt(count) * ref.U + np.linalg.norm(want) * HALF[dtype], name


LENS = [[1], [7], [8], [64], [65, 0, 1, 200], [0, 0, 17], [130, 3, 129, 64, 1]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("c,S,G,dtype", [(64, 16, 1, BF16), (200, 16, 2, F32), (1, 8, 1, F32), (96, 8, 3, BF16), (72, 32, 1, BF16), (130, 32, 2, F32),
                                         (8, 16, 8, BF16), (300, 16, 1, F32)])
@pytest.mark.parametrize("gated", [True, False])
def test_forward_and_backward(lens, c, S, G, dtype, gated):
    need_gpu()
    d = make(lens, c, S, G, dtype, S, gated)
    want, most, count = exact(d, lens)
    y, final = fwd(d)
    check(y, want["y"], most["y"], count, dtype, "y")
    check(final, want["final"], most["final"], count, F32, "final")
    y32, _ = fwd(d, out_dtype=F32)
    check(y32, want["y"], most["y"], count, F32, "y32")
    g = bwd(d)
    for n, name in GRADS.items():
        if n == "dz" and not gated:
            assert g[name] is None
            continue
        check(g[name], want[n], most[n], count + (sum(lens) if n in ("dA", "dD", "dbias") else 0),
              F32 if n in ("dA", "dD", "dbias", "dh0") else dtype, n)


@pytest.mark.parametrize("soft", [True, False])
def test_absent_arguments_and_equal_documents(soft):
    need_gpu()
    lens = [70, 70]
    d = make(lens, 80, 16, 1, F32)
    d["raw"] = d["raw"] if soft else d["raw"].abs() * 0.1
    d["bias"], d["D"], d["z"] = torch.zeros_like(d["bias"]), torch.zeros_like(d["D"]), None
    d["h0"], d["dh"] = torch.zeros_like(d["h0"]), torch.zeros_like(d["dh"])
    y, final = fwd(d, softplus=soft)
    g = bwd(d, softplus=soft)
    want, most, count = exact(d, lens, soft)
    check(y, want["y"], most["y"], count, F32, "y")
    for n in ("dx", "ddt", "dA", "dB", "dC", "dh0"):
        check(g[GRADS[n]], want[n], most[n], count + 140, F32, n)
    args = d["x"], d["raw"], d["A"], d["B"], d["C"]
    y2, final2 = kda.kda_selective_fwd(*args, num_seqs=2, softplus=soft)
    assert torch.equal(y, y2) and torch.equal(final, final2)
    y2, none = kda.kda_selective_fwd(*args, num_seqs=2, softplus=soft, output_final_state=False)
    assert torch.equal(y, y2) and none is None
    g2 = kda.kda_selective_bwd(*args, d["dy"], num_seqs=2, softplus=soft)
    for n in ("dx", "ddt", "dA", "dB", "dC"):
        assert torch.equal(g[n], g2[n]), n
    assert all(g2[n] is None for n in ("dD", "dz", "ddt_bias", "dS0"))


def test_empty_stream():
    need_gpu()
    d = make([0, 0, 0], 72, 16, 1, BF16)
    y, final = fwd(d)
    assert y.shape == (0, 72) and torch.equal(final, d["h0"])
    g = bwd(d)
    assert torch.equal(g["dS0"], d["dh"]) and (g["dA"] == 0).all() and (g["dD"] == 0).all() and (g["ddt_bias"] == 0).all()


@pytest.mark.parametrize("lens,c,S,G", [([5000], 64, 16, 1), ([3000, 1, 700, 0, 1299], 192, 8, 1), ([2500, 2500], 130, 32, 2)])
def test_many_segments(lens, c, S, G):
    """Long documents in many segments: the carry goes over more of them than it loads at once."""
    need_gpu()
    d = make(lens, c, S, G, F32)
    d["bias"] -= 2      # slow decays, so that states reach across segments
    want, most, count = exact(d, lens)
    y, final = fwd(d)
    check(y, want["y"], most["y"], count, F32, "y")
    check(final, want["final"], most["final"], count, F32, "final")
    g = bwd(d)
    for n, name in GRADS.items():
        check(g[name], want[n], most[n], count + (sum(lens) if n in ("dA", "dD", "dbias") else 0), F32, n)


def test_segments_change_only_rounding():
    """Wide layers are cut less: the same channels alone and among 4096 agree to rounding, and repeated calls to the bit."""
    need_gpu()
    lens = [1500, 548]
    d = make(lens, 4096, 16, 1, BF16)
    part = {n: x for n, x in d.items()}
    for n in ("x", "raw", "z", "dy"):
        part[n] = d[n][:, :64].contiguous()
    part.update(A=d["A"][:64], D=d["D"][:64], bias=d["bias"][:64], h0=d["h0"][:, :64].contiguous(), dh=d["dh"][:, :64].contiguous())
    want, most, count = exact(part, lens)
    y, final = fwd(d)
    again, _ = fwd(d)
    assert torch.equal(y, again)
    check(y[:, :64], want["y"], most["y"], count, BF16, "y")
    check(final[:, :64], want["final"], most["final"], count, F32, "final")
    g, same = bwd(d), bwd(d)
    for n, name in GRADS.items():
        assert torch.equal(g[name], same[name]), n
        if n not in ("dB", "dC"):
            x = g[name]
            x = x[:64] if n in ("dA", "dD", "dbias") else x[:, :64]
            check(x, want[n], most[n], count + (2048 if n in ("dA", "dD", "dbias") else 0), F32 if n in ("dA", "dD", "dbias", "dh0") else BF16, n)


def test_rows_of_wider_tensors():
    """x and z as halves of one projection, dt, B and C as parts of another."""
    need_gpu()
    T, c, S = 150, 96, 16
    lens = [100, 50]
    d = make(lens, c, S, 1, BF16)
    xz = torch.cat([d["x"], d["z"]], 1)
    rest = torch.cat([d["raw"], d["B"].view(T, S), d["C"].view(T, S)], 1)
    wide = dict(d, x=xz[:, :c], z=xz[:, c:], raw=rest[:, :c], B=rest[:, None, c:c + S], C=rest[:, None, c + S:])
    assert all(torch.equal(a, b) for a, b in zip(fwd(d), fwd(wide)))
    g, w = bwd(d), bwd(wide)
    assert all(torch.equal(g[n], w[n]) for n in g)
    args = [[v[n][:2] for n in ("x", "raw", "B", "C")] + [v["z"][:2]] for v in (d, wide)]
    outs = [kda.kda_selective_decode(x, r, d["A"], B, C, d["h0"], z=z) for x, r, B, C, z in args]
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("c,S,G,dtype", [(64, 16, 1, BF16), (333, 16, 3, F32), (4096, 8, 1, BF16), (72, 32, 2, F32), (1, 8, 1, BF16)])
def test_decode(c, S, G, dtype):
    """A step against 64 bits, in place too, and a run of steps as a prompt's continuation."""
    need_gpu()
    N = 5
    d = make([1] * N, c, S, G, dtype)
    want, most, count = exact(d, [1] * N, backward=False)
    args = d["x"], d["raw"], d["A"], d["B"], d["C"]
    kw = dict(D=d["D"], z=d["z"], dt_bias=d["bias"])
    y, state = kda.kda_selective_decode(*args, d["h0"], **kw)
    check(y, want["y"], most["y"], count, dtype, "y")
    check(state, want["final"], most["final"], count, F32, "state")
    own = d["h0"].clone()
    y2, same = kda.kda_selective_decode(*args, own, out_state=own, **kw)
    assert same is own and torch.equal(y, y2) and torch.equal(own, state)
    y0, s0 = kda.kda_selective_decode(*args)
    y1, s1 = kda.kda_selective_decode(*args, torch.zeros_like(state), D=torch.zeros_like(d["D"]), dt_bias=torch.zeros_like(d["bias"]))
    assert torch.equal(y0, y1) and torch.equal(s0, s1)
    lens = [12, 9]
    d = make(lens, c, S, G, dtype, 3)
    want, most, count = exact(d, lens, backward=False)
    at, state = ref.starts(lens), d["h0"].clone()
    short = dict(d, cu=torch.tensor([0, 7, 11], dtype=torch.int32, device="cuda"))
    pick = list(range(7)) + list(range(12, 16))
    for n in ("x", "raw", "B", "C", "z"):
        short[n] = d[n][pick].contiguous()
    y, state = fwd(short)
    for t in range(5):
        rows = [7 + t, 16 + t]
        y, state = kda.kda_selective_decode(d["x"][rows], d["raw"][rows], d["A"], d["B"][rows], d["C"][rows], state, D=d["D"],
                                            z=d["z"][rows], dt_bias=d["bias"])
        check(y, want["y"][rows], most["y"][rows], count, dtype, "y")
    check(state, want["final"], most["final"], count, F32, "state")
    y, _ = kda.kda_selective_decode(d["x"][:0], d["raw"][:0], d["A"], d["B"][:0], d["C"][:0])
    assert y.shape == (0, c)


def test_step_sizes():
    """softplus and its derivative over fp32's range: steps of 1e-30 to 1e4, where 1 + e rounds and where e overflows."""
    need_gpu()
    c = 512
    raw = torch.linspace(-80, 80, c, device="cuda")[None].repeat(2, 1).contiguous()
    one = torch.ones(2, c, device="cuda")
    B = torch.ones(2, 1, 8, device="cuda") / 8
    A = torch.zeros(c, 8, device="cuda")
    y, _ = kda.kda_selective_fwd(one, raw, A, B, B * 8)
    dt = ref.softplus(host(raw))
    # the state is the sum of the steps: the exponential, sum, logarithm, correction and quotient, 6 half steps and 2 of
    # the exponent's rounding a unit of its size
    rel = (10 + 2.9 * np.abs(host(raw))) * ref.U
    assert (np.abs(host(y) - np.cumsum(dt, 0)) <= np.cumsum(dt, 0) * (rel + 4 * ref.U)).all()
    g = kda.kda_selective_bwd(one, raw, A, B, B * 8, one)
    want = np.array([[2.0], [1.0]]) * ref.sigmoid(host(raw))
    assert (np.abs(host(g["ddt"]) - want) <= want * (rel + 4 * ref.U)).all()


def test_extreme_decays():
    """A of zero keeps a state, a huge one drops it at once."""
    need_gpu()
    lens = [300]
    d = make(lens, 64, 16, 1, F32)
    d["A"][:, 0], d["A"][:, 1] = 0.0, -1e30
    d["A"][:, 2] = -1e-30
    want, most, _ = exact(d, lens)
    rest = d["A"].clone()
    rest[:, 1] = -1
    count = ref.selective_roundings(host(d["raw"]), host(rest), host(d["bias"]), lens)
    y, final = fwd(d)
    check(y, want["y"], most["y"], count, F32, "y")
    check(final, want["final"], most["final"], count, F32, "final")
    g = bwd(d)
    for n, name in GRADS.items():
        check(g[name], want[n], most[n], count + 300, F32, n)


def test_nonfinite_values_stay_where_they_belong():
    need_gpu()
    lens = [100, 80, 90]
    d = make(lens + [40], 128, 16, 1, F32)
    d.update(cu=d["cu"][:4].contiguous(), h0=d["h0"][:3].contiguous(), dh=d["dh"][:3].contiguous())
    for n in ("x", "raw", "z", "B", "C", "dy"):     # rows behind the last document
        d[n][270:] = float("nan")
    y, final = fwd(d)
    assert torch.isfinite(y[:270]).all() and torch.isfinite(final).all()
    g = bwd(d)
    assert all(torch.isfinite(g[n][:270] if g[n].shape[0] == 310 else g[n]).all() for n in g)
    for n in ("x", "raw"):                         # one channel of the second document, from its token 20 on
        e = {k: v.clone() for k, v in d.items()}
        e[n][120, 7] = float("nan")
        y2, final2 = fwd(e)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[120:180, 7] = True
        assert torch.isnan(y2[bad]).all() and torch.equal(y2[:270][~bad[:270]], y[:270][~bad[:270]])
        assert torch.isnan(final2[1, 7]).all()
        final2[1, 7] = final[1, 7]
        assert torch.equal(final2, final)
    e = {k: v.clone() for k, v in d.items()}
    e["dy"][120, 7] = float("nan")                  # reaches that channel's earlier tokens, and its own dC
    g2 = bwd(e)
    rows = [t for t in range(270) if not 100 <= t <= 120]
    for n in ("dx", "ddt", "dz"):
        assert torch.equal(g2[n][rows], g[n][rows])
        assert torch.equal(g2[n][:270, :7], g[n][:270, :7]) and torch.equal(g2[n][:270, 8:], g[n][:270, 8:])
    for n in ("dB", "dC"):
        assert torch.equal(g2[n][rows], g[n][rows])
    assert torch.equal(g2["dA"][:7], g["dA"][:7]) and torch.isnan(g2["dA"][7]).any()
    assert torch.equal(g2["dS0"][0], g["dS0"][0]) and torch.equal(g2["dS0"][2], g["dS0"][2])
    e = {k: v.clone() for k, v in d.items()}
    e["h0"][1, 5, 3] = float("inf")
    y2, final2 = fwd(e)
    assert not torch.isfinite(y2[100, 5]) and torch.equal(y2[:270, :5], y[:270, :5]) and torch.equal(y2[:270, 6:], y[:270, 6:])
    assert torch.equal(y2[:100], y[:100]) and torch.equal(y2[180:270], y[180:270])


@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("gated", [True, False])
def test_infinity_at_a_documents_last_token(S, gated):
    """x_T is in no other token's gradient and not in dA, which has h_T only through later tokens: there are none."""
    need_gpu()
    lens = [100, 7, 9, 1, 6]
    d = make(lens, 70, S, 1, F32, S, gated)
    y, final = fwd(d)
    g = bwd(d)
    last = (np.cumsum(lens) - 1).tolist()
    e = dict(d, x=d["x"].clone())
    e["x"][last, 5] = float("inf")
    y2, final2 = fwd(e)
    g2 = bwd(e)
    rest = [t for t in range(sum(lens)) if t not in last]
    assert torch.equal(y2[rest], y[rest]) and not torch.isfinite(y2[last, 5]).any() and not torch.isfinite(final2[:, 5]).any()
    for n in ("dx", "ddt", "dz", "dB", "dC"):
        if g[n] is not None:
            assert torch.equal(g2[n][rest], g[n][rest]), n
    for n in ("dA", "dS0", "dx"):
        assert torch.equal(g2[n], g[n]), n
    assert torch.equal(g2["dD"][:5], g["dD"][:5]) and torch.equal(g2["dD"][6:], g["dD"][6:]) and not torch.isfinite(g2["dD"][5])
    assert not torch.isfinite(g2["ddt"][last, 5]).any()


def test_rows_behind_the_documents_are_left():
    need_gpu()
    lens, T = [40, 37], 90
    d = make(lens + [13], 72, 16, 1, BF16)
    cu = d["cu"][:3].contiguous()
    from gated_delta_rule_41_amd import _lib
    lib = _lib.load()
    cfg = _lib.make_selective_config(72, 16)
    p = {n: x.data_ptr() for n, x in d.items()}
    out = {n: torch.full((T, 72), 7.0, dtype=BF16, device="cuda") for n in ("y", "dx", "ddt", "dz")}
    out.update({n: torch.full((T, 16), 7.0, dtype=BF16, device="cuda") for n in ("dB", "dC")})
    small = {n: torch.empty(72 * 16, device="cuda") for n in ("dA", "dD", "dbias")}
    ws = torch.empty(_lib.kda_selective_bwd_workspace_size(cfg, T, 2), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    head = (cfg, T, 2, p["x"], p["raw"], p["A"], p["B"], p["C"], p["D"], p["z"], p["bias"], cu.data_ptr(), p["h0"])
    assert lib.kda_selective_fwd(*head, out["y"].data_ptr(), None, ws.data_ptr(), ws.numel(), stream) == 0
    assert lib.kda_selective_bwd(*head, p["dy"], None, out["dx"].data_ptr(), out["ddt"].data_ptr(), small["dA"].data_ptr(),
                                 out["dB"].data_ptr(), out["dC"].data_ptr(), small["dD"].data_ptr(), out["dz"].data_ptr(),
                                 small["dbias"].data_ptr(), None, ws.data_ptr(), ws.numel(), stream) == 0
    conv = _lib.make_conv_config(72, 4)
    w = torch.ones(72, 4, dtype=BF16, device="cuda")
    cy, cdx, dw = (torch.full((T, 72), 7.0, dtype=t, device="cuda") for t in (BF16, BF16, F32))
    ws2 = torch.empty(_lib.kda_conv_bwd_workspace_size(conv, T, 2), dtype=torch.uint8, device="cuda")
    assert lib.kda_conv_fwd(conv, T, 2, p["x"], w.data_ptr(), None, cu.data_ptr(), None, cy.data_ptr(), None, stream) == 0
    assert lib.kda_conv_bwd(conv, T, 2, p["x"], w.data_ptr(), None, cu.data_ptr(), None, p["dy"], None, cdx.data_ptr(), dw.data_ptr(), None,
                            None, ws2.data_ptr(), ws2.numel(), stream) == 0
    torch.cuda.synchronize()
    for n, x in dict(out, cy=cy, cdx=cdx).items():
        assert (x[77:] == 7).all() and not (x[:77] == 7).all(1).any(), n


def test_long_offsets():
    """Rows behind 2^31 elements, a document that reaches across them."""
    need_gpu()
    T, c = 540000, 4096
    cu = torch.tensor([0, T - 1000, T], dtype=torch.int32, device="cuda")
    small = make([1000], c, 16, 1, BF16)
    zero = torch.zeros(T, c, dtype=BF16, device="cuda")
    vectors = {}
    for n in ("x", "raw"):
        vectors[n] = zero.clone()
        vectors[n][-1000:] = small[n]
    B, C = (torch.zeros(T, 1, 16, dtype=BF16, device="cuda") for _ in range(2))
    B[-1000:], C[-1000:] = small["B"], small["C"]
    h0 = torch.cat([torch.zeros_like(small["h0"]), small["h0"]])
    y, final = kda.kda_selective_fwd(vectors["x"], vectors["raw"], small["A"], B, C, cu, h0, dt_bias=small["bias"])
    want, last = kda.kda_selective_fwd(small["x"], small["raw"], small["A"], small["B"], small["C"], None, small["h0"], dt_bias=small["bias"])
    assert (y[:-1000] == 0).all() and (final[0] == 0).all()
    # cut into other segments: equal to fp32 rounding, so bf16 values differ by at most one step
    assert (y[-1000:].float() - want.float()).abs().max() <= want.float().abs().max() * 2.0 ** -7
    assert torch.allclose(final[1], last[0], rtol=0, atol=float(last.abs().max()) * 2.0 ** -16)


def test_autograd():
    need_gpu()
    lens = [70, 1, 9]
    d = make(lens, 40, 16, 1, F32)
    names = ("x", "raw", "A", "B", "C", "D", "z", "bias", "h0")
    leaf = {n: d[n].clone().requires_grad_() for n in names}
    y, final = kda.kda_selective(leaf["x"], leaf["raw"], leaf["A"], leaf["B"], leaf["C"], d["cu"], leaf["h0"], D=leaf["D"], z=leaf["z"],
                                 dt_bias=leaf["bias"])
    ((y * d["dy"]).sum() + (final * d["dh"]).sum()).backward()
    g = bwd(d)
    for n, k in zip(names, ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")):
        assert torch.equal(leaf[n].grad, g[k]), n
    # one output unused, arguments absent, an upstream gradient that is a view
    y, final = kda.kda_selective(leaf["x"], leaf["raw"], leaf["A"], leaf["B"], leaf["C"], d["cu"])
    gA, = torch.autograd.grad(final.sum(), leaf["A"], retain_graph=True)
    assert torch.isfinite(gA).all()
    wide = torch.randn(80, 41, device="cuda")
    gx, = torch.autograd.grad(y, leaf["x"], wide[:, 1:], retain_graph=True)
    hx, = torch.autograd.grad(y, leaf["x"], wide[:, 1:].contiguous())
    assert torch.equal(gx, hx)


def test_refusals():
    need_gpu()
    d = make([6], 64, 16, 1, BF16)
    args = [d[n] for n in ("x", "raw", "A", "B", "C")]

    def call(i, value, **kw):
        return kda.kda_selective_fwd(*(value if j == i else a for j, a in enumerate(args)), **kw)

    with pytest.raises(TypeError):
        call(2, d["A"].to(BF16))
    with pytest.raises(TypeError):
        call(1, d["raw"].float())
    with pytest.raises(ValueError, match="shape"):
        call(3, d["B"][:, :, :8])
    with pytest.raises(ValueError, match="dimensions"):
        call(3, d["B"][:, 0])
    with pytest.raises(kda.KdaError, match="S must"):
        kda.kda_selective_fwd(*args[:2], d["A"][:, :4].contiguous(), d["B"][..., :4].contiguous(), d["C"][..., :4].contiguous())
    with pytest.raises(kda.KdaError, match="16 bytes"):
        call(3, torch.zeros(6, 1, 20, dtype=BF16, device="cuda")[..., :16])
    with pytest.raises(kda.KdaError, match="divide"):
        kda.kda_selective_fwd(*args[:3], *(torch.zeros(6, 3, 16, dtype=BF16, device="cuda") for _ in range(2)))
    with pytest.raises(ValueError, match="shape"):
        call(0, args[0], initial_state=d["h0"][:, :8].contiguous())
