"""The norm with the residual's addition against 64 bits: types, sizes, 8-bit codes, extreme rows, gradients."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def host(t):
    return t.detach().double().cpu().numpy()


def rand(rows, C, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, C, generator=gen) * scale).to(dtype).cuda()


# every width of a row's threads, rows of eight channels and odd ones, one channel, one row
SIZES = [(1, 1), (3, 7), (5, 64), (2, 333), (9, 512), (7, 1000), (4, 1024), (6, 1032), (3, 2048), (257, 2056), (5, 4096), (3, 4099), (2, 8192),
         (2, 8200), (9, 100), (20, 128), (11, 200), (8, 256), (2, 12001), (1, 16384)]


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32)])
def test_forward(rows, C, types):
    need_gpu()
    xt, rt, wt = types
    x, r = rand(rows, C, xt, C), rand(rows, C, rt, C + 1, 2.0)
    w = (1 + 0.2 * rand(1, C, F32, C + 2)[0]).to(wt)
    y, s = kda.kda_norm_fwd(x, w, r, eps=EPS)
    total = (x.float() + r.float()).to(rt)
    assert s.dtype == rt and torch.equal(s, total)
    want, _ = ref.norm_fwd(host(total), host(w), EPS)
    assert y.dtype == xt
    # rstd's roundings and two products, then the output's own
    tol = np.abs(want) * ((ref.RSTD + 2) * ref.U + HALF[xt]) * 1.01
    assert (np.abs(host(y) - want) <= tol).all()
    # without a residual, without a weight, other output types
    y, s = kda.kda_norm_fwd(x, eps=EPS, out_dtype=F32)
    assert s is x and y.dtype == F32
    want, _ = ref.norm_fwd(host(x), 1.0, EPS)
    assert (np.abs(host(y) - want) <= np.abs(want) * (ref.RSTD + 3) * ref.U * 1.01).all()


@pytest.mark.parametrize("rows,C", [(1, 1), (3, 7), (9, 512), (2, 333), (40, 1032), (33, 4096), (3, 4099), (2, 8200), (2, 12001), (1, 16384)])
@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("out", [torch.int8, torch.float8_e4m3fn])
def test_codes(rows, C, types, out):
    """Codes are exact: nearest to the real quotient, ties to even, so they have to be equal."""
    need_gpu()
    xt, rt = types
    x, r = rand(rows, C, xt, C + 3), rand(rows, C, rt, C + 4)
    w = (1 + 0.2 * rand(1, C, F32, C + 5)[0]).to(xt)
    y, s, scale = kda.kda_norm_fwd(x, w, r, eps=EPS, out_dtype=out)
    assert y.dtype == out and scale.dtype == F32 and scale.shape == (rows,)
    limit = 127 if out == torch.int8 else 448
    real, top = ref.codes(s.float().cpu().numpy(), w.float().cpu().numpy(), limit)
    if out == torch.int8:
        want = np.rint(real)
    else:
        # 4 significant bits, steps of 2^-9 below 2^-6; the 64-bit quotient's own rounding is 2^-53
        step = np.exp2(np.maximum(np.frexp(real)[1], -5) - 4.0)
        want = np.rint(real / step) * step
    assert (host(y.float()) == want).all()
    _, rstd = ref.norm_fwd(host(s), 1.0, EPS)
    want = (top * rstd / limit)[:, 0]
    assert (np.abs(host(scale) - want) <= want * (ref.RSTD + 2) * ref.U * 1.01).all()


@pytest.mark.parametrize("out,limit", [(torch.int8, 127), (torch.float8_e4m3fn, 448)])
def test_codes_on_borders(out, limit):
    """Rows whose quotients lie on and next to the borders between codes: halves of the largest's 127th or 448th parts."""
    need_gpu()
    k = torch.arange(-4 * limit, 4 * limit + 1, dtype=torch.float32)
    x = torch.stack([k / 4, torch.nextafter(k / 4, k * 100), torch.nextafter(k / 4, 0 * k), k / 4 * 2 ** -140, k / 4 * 2.0 ** 100]).cuda()
    y, _, _ = kda.kda_norm_fwd(x, out_dtype=out, eps=0.0)
    real, _ = ref.codes(x.cpu().numpy(), 1.0, limit)
    if out == torch.int8:
        want = np.rint(real)
    else:
        step = np.exp2(np.maximum(np.frexp(real)[1], -5) - 4.0)
        want = np.rint(real / step) * step
    got = host(y.float())
    assert (got == want).all(), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("C", [512, 4096, 333])
def test_extreme_rows(C):
    """Zeros, the largest and smallest values, infinities and NaN: each row by itself."""
    need_gpu()
    x = rand(8, C, F32, 11)
    x[1] = 0
    x[2] = x[2].sign() * 3e38
    x[3] *= 1e-42
    x[4, 5] = float("inf")
    x[5, 6] = float("nan")
    x[6] *= 1e30
    y, _ = kda.kda_norm_fwd(x, eps=1e-12)
    want, _ = ref.norm_fwd(host(x), 1.0, 1e-12)
    fine = [0, 1, 2, 3, 6, 7]
    # the largest rows' rstd is a number below fp32's normal range, held in steps of 2^-149
    tol = np.abs(want) * (ref.RSTD + 3) * ref.U * 1.01 + np.abs(host(x)) * 2.0 ** -149
    assert (np.abs(host(y) - want)[fine] <= tol[fine]).all()
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[4]).all()
    for out in (torch.int8, torch.float8_e4m3fn):
        codes, _, scale = kda.kda_norm_fwd(x, eps=1e-12, out_dtype=out)
        assert scale[1] == 0 and (codes[1].float() == 0).all()
        assert torch.isnan(scale[4:6]).all() and torch.isfinite(scale[fine]).all()
        back = host(codes.float()) * host(scale)[:, None]
        step = np.abs(want).max(1, keepdims=True) / 127 / 2 if out == torch.int8 else np.abs(want) * 2.0 ** -4 + np.abs(want).max(1, keepdims=True) * 2.0 ** -10 / 448
        assert (np.abs(back - want)[fine] <= (step * 1.001 + tol)[fine]).all()


@pytest.mark.parametrize("C", [64, 333, 4096])
def test_zero_rows_without_eps(C):
    """0 / 0 in the formula: values are NaN, as the formula has them; the row's codes and its scale are zeros."""
    need_gpu()
    x = rand(3, C, BF16, 1)
    x[1] = 0
    y, _ = kda.kda_norm_fwd(x, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()
    for out in (torch.int8, torch.float8_e4m3fn):
        codes, _, scale = kda.kda_norm_fwd(x, eps=0.0, out_dtype=out)
        assert scale[1] == 0 and (codes[1].float() == 0).all() and (scale[[0, 2]] > 0).all()


@pytest.mark.parametrize("C", [64, 1000, 4096, 8200, 12001])
@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_rows_whose_squares_leave_the_range(C, eps):
    """Rows of 2^-110 to 2^126: their squares are zeros, of few bits, or infinite in fp32."""
    need_gpu()
    powers = [-110, -90, -70, -64, -60, -50, -40, 0, 60, 64, 100, 124]
    x = rand(len(powers), C, F32, 3).clamp(-3.9, 3.9) * torch.tensor([2.0 ** p for p in powers], device="cuda")[:, None]
    w = 1 + 0.2 * rand(1, C, F32, 4)[0]
    y, _ = kda.kda_norm_fwd(x, w, eps=eps)
    eps = float(np.float32(eps))
    want, rstd = ref.norm_fwd(host(x), host(w), eps)
    # a product may fall below the normal range, where it is held in steps of 2^-149
    assert (np.abs(host(y) - want) <= (np.abs(want) * (ref.RSTD + 3) * ref.U + 2.0 ** -149) * 1.01).all()
    for out, limit in ((torch.int8, 127), (torch.float8_e4m3fn, 448)):
        _, _, scale = kda.kda_norm_fwd(x, w, eps=eps, out_dtype=out)
        top = ref.codes(x.cpu().numpy(), w.cpu().numpy(), limit)[1]
        want = (top * rstd / limit)[:, 0]
        assert (np.abs(host(scale) - want) <= want * (ref.RSTD + 3) * ref.U * 1.01).all()
    dy, ds = rand(len(powers), C, F32, 5), rand(len(powers), C, F32, 6)
    d = kda.kda_norm_bwd(x, w, dy, ds, eps=eps)
    args = host(x), host(w), host(dy), host(ds), eps
    (dx, dw), (dxm, dwm) = ref.norm_bwd(*args), ref.norm_bwd_bound(*args)
    assert (np.abs(host(d["dx"]) - dx) <= (dxm + np.abs(dx) * ref.U + 2.0 ** -149) * 1.01).all()
    assert (np.abs(host(d["dw"]) - dw) <= (dwm + 2.0 ** -149 * len(powers)) * 1.01).all()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
def test_gradients_of_both_terms_do_not_share_memory(types):
    need_gpu()
    x, r = rand(3, 64, types[0], 1).requires_grad_(), rand(3, 64, types[1], 2).requires_grad_()
    y, s = kda.kda_norm(x, None, r, eps=EPS)
    (y.sum() + s.sum()).backward()
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    kept = r.grad.clone()
    x.grad.zero_()
    assert torch.equal(r.grad, kept)


def test_in_place_and_no_rows():
    need_gpu()
    for C in (64, 333, 4096):
        x, r = rand(5, C, BF16, 1), rand(5, C, BF16, 2)
        w = rand(1, C, BF16, 3)[0]
        y, s = kda.kda_norm_fwd(x, w, r)
        r2 = r.clone()
        y2, s2 = kda.kda_norm_fwd(x, w, r2, out_residual=r2)
        assert s2 is r2 and torch.equal(y, y2) and torch.equal(s, r2)
    y, s = kda.kda_norm_fwd(x[:0], w, r[:0])
    assert y.shape == (0, 4096)
    d = kda.kda_norm_bwd(s, w, y)
    assert d["dx"].shape == (0, 4096) and (d["dw"] == 0).all()


@pytest.mark.parametrize("rows,C", [(1, 1), (3, 7), (70, 64), (2, 333), (9, 512), (7, 1000), (1100, 1032), (5, 4096), (3, 4099), (2, 8192), (2, 8200),
                                    (40, 100), (70, 128), (33, 200), (2, 12001), (1, 16384)])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32)])
def test_backward(rows, C, types):
    need_gpu()
    xt, rt, wt = types
    s, dy, ds = rand(rows, C, rt, C), rand(rows, C, xt, C + 1), rand(rows, C, rt, C + 2)
    w = (1 + 0.2 * rand(1, C, F32, C + 3)[0]).to(wt)
    for up in (ds, None):
        d = kda.kda_norm_bwd(s, w, dy, up, eps=EPS)
        args = (host(s), host(w), host(dy), host(up) if up is not None else np.zeros((rows, C)), EPS)
        dx, dw = ref.norm_bwd(*args)
        dxm, dwm = ref.norm_bwd_bound(*args)
        assert d["dx"].dtype == rt and d["dw"].dtype == F32
        assert (np.abs(host(d["dx"]) - dx) <= (dxm + np.abs(dx) * HALF[rt]) * 1.01).all()
        assert (np.abs(host(d["dw"]) - dw) <= dwm * 1.01).all()
    d = kda.kda_norm_bwd(s, None, dy, None, eps=EPS, out_dtype=F32)
    dx, _ = ref.norm_bwd(host(s), 1.0, host(dy), 0.0, EPS)
    dxm, _ = ref.norm_bwd_bound(host(s), 1.0, host(dy), np.zeros((rows, C)), EPS)
    assert d["dw"] is None and (np.abs(host(d["dx"]) - dx) <= (dxm + np.abs(dx) * ref.U) * 1.01).all()


@pytest.mark.parametrize("rows,C", [(5, 2), (5, 8), (9000, 9), (17, 15), (40, 130), (9000, 320), (33, 377), (9, 384), (2500, 640), (2100, 761), (2100, 1280),
                                    (9, 1529), (1100, 2560), (600, 5120), (7, 6137), (300, 10240), (3, 12281)])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32)])
def test_backward_of_every_split(rows, C, types):
    """Each number of threads and groups a row, with rows for more than one turn, with ends of less than eight channels."""
    test_backward(rows, C, types)


def test_autograd():
    need_gpu()
    x, r, w = rand(6, 96, F32, 1).requires_grad_(), rand(6, 96, F32, 2).requires_grad_(), rand(1, 96, F32, 3)[0].requires_grad_()
    dy, ds = rand(6, 96, F32, 4), rand(6, 96, F32, 5)
    y, s = kda.kda_norm(x, w, r, eps=EPS)
    ((y * dy).sum() + (s * ds).sum()).backward()
    d = kda.kda_norm_bwd(s.detach(), w.detach(), dy, ds, eps=EPS)
    assert torch.equal(x.grad, d["dx"]) and torch.equal(r.grad, d["dx"]) and torch.equal(w.grad, d["dw"])
    # against differences, along a direction: the loss is smooth, a step of 2^-7 leaves its third derivative
    def loss(e):
        v, _ = ref.norm_fwd(host(x) + host(r) + e * host(dy), host(w), EPS)
        return (v * host(dy)).sum() + ((host(x) + host(r) + e * host(dy)) * host(ds)).sum()
    want = (loss(2.0 ** -10) - loss(-2.0 ** -10)) * 2.0 ** 9
    got = (host(x.grad) * host(dy)).sum()
    assert abs(got - want) <= 1e-4 * np.abs(host(x.grad) * host(dy)).sum()
    # only one output used, a single input's gradient, mixed types
    xb = rand(6, 96, BF16, 1).requires_grad_()
    y, s = kda.kda_norm(xb, w.detach(), r.detach(), eps=EPS)
    assert s.dtype == F32
    g, = torch.autograd.grad(s.sum(), xb)
    assert g.dtype == BF16 and (g == 1).all()
    y = kda.kda_norm(xb)
    g, = torch.autograd.grad(y.float().sum(), xb)
    assert torch.isfinite(g).all()


def test_refusals():
    need_gpu()
    x = rand(4, 64, BF16, 1)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_norm_fwd(x[:, ::2])
    with pytest.raises(TypeError):
        kda.kda_norm_fwd(x, residual=x.half())
    with pytest.raises(TypeError):
        kda.kda_norm_fwd(x.half())
    with pytest.raises(TypeError):
        kda.kda_norm_fwd(x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out_residual"):
        kda.kda_norm_fwd(x, out_residual=x)
    big = torch.zeros(4 * 64 + 8, dtype=BF16, device="cuda")
    with pytest.raises(kda.KdaError, match="overlaps"):
        kda.kda_norm_fwd(big[:256].view(4, 64), residual=x, out_residual=big[8:].view(4, 64))
    with pytest.raises(ValueError, match="shape"):
        kda.kda_norm_fwd(x, weight=x[0, :32])
    with pytest.raises(kda.KdaError, match="too large"):
        kda.kda_norm_fwd(torch.zeros(1, 16385, device="cuda"))

