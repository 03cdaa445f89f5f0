"""The norm over rows of every kind: fewer than eight channels, ends of every length, in place, more rows than 2^23."""
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


def rand(rows, C, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, C, generator=gen, device="cuda").to(dtype)


def check_backward(s, w, dy, ds, **kw):
    """dx and dw within the roundings of their sums, dx rounded once."""
    d = kda.kda_norm_bwd(s, w, dy, ds, eps=EPS, **kw)
    args = host(s), host(w) if w is not None else 1.0, host(dy), host(ds) if ds is not None else np.zeros(s.shape), EPS
    (dx, dw), (dxm, dwm) = ref.norm_bwd(*args), ref.norm_bwd_bound(*args)
    assert (np.abs(host(d["dx"]) - dx) <= (dxm + np.abs(dx) * HALF[d["dx"].dtype]) * 1.01).all()
    if w is None:
        assert d["dw"] is None
    else:
        assert (np.abs(host(d["dw"]) - dw) <= dwm * 1.01).all()


@pytest.mark.parametrize("C", range(1, 8))
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("wt", [BF16, F32, None])
def test_rows_of_fewer_than_eight_channels(C, xt, rt, wt):
    """Read element by element, the weights of either type too: each channel has its own."""
    need_gpu()
    w = (1 + rand(1, C, F32, 7)[0]).to(wt) if wt else None
    for rows in (1, 16, 17, 20011):
        x, r, ds = rand(rows, C, xt, C), rand(rows, C, rt, C + 10), rand(rows, C, rt, C + 20)
        y, s = kda.kda_norm_fwd(x, w, r, eps=EPS)
        assert torch.equal(s, (x.float() + r.float()).to(rt))
        want, _ = ref.norm_fwd(host(s), host(w) if wt else 1.0, EPS)
        assert (np.abs(host(y) - want) <= np.abs(want) * ((ref.RSTD + 2) * ref.U + HALF[xt]) * 1.01).all()
        check_backward(s, w, x, ds)
        check_backward(s, w, x, None, out_dtype=F32)


@pytest.mark.parametrize("whole", [8, 120, 248, 376, 504, 760, 1016, 1528, 2040, 4088, 6136, 8184, 12280])
def test_backward_with_ends_of_every_length(whole):
    """fp32, the widths around each change of a row's threads and groups, more rows than one turn takes."""
    need_gpu()
    rows = 20011 if whole < 400 else 2100 if whole < 1600 else 7
    if whole < 400:
        rows //= 1 + whole // 64
    for C in range(whole + 1, whole + 8):
        s, dy, ds = (rand(rows, C, F32, C + i) for i in range(3))
        check_backward(s, 1 + rand(1, C, F32, C + 3)[0], dy, ds)


def test_more_rows_than_2_to_the_23():
    """262144 tokens of 32 heads and some more: their last rows as those rows alone."""
    need_gpu()
    rows, last, C = 262144 * 32 + 21, 40, 128
    x, w = rand(last, C, BF16, 1), 1 + rand(1, C, F32, 2)[0]
    big = torch.zeros(rows, C, dtype=BF16, device="cuda")
    big[-last:] = x
    y, _ = kda.kda_norm_fwd(big, w, eps=EPS)
    want, _ = kda.kda_norm_fwd(x, w, eps=EPS)
    assert torch.equal(y[-last:], want) and not y[:-last].any()
    del y
    d = kda.kda_norm_bwd(big, w, big, eps=EPS)
    small = kda.kda_norm_bwd(x, w, x, eps=EPS)
    assert torch.equal(d["dx"][-last:], small["dx"]) and not d["dx"][:-last].any()
    _, dwm = ref.norm_bwd_bound(host(x), host(w), host(x), np.zeros(x.shape), EPS)
    assert (np.abs(host(d["dw"]) - host(small["dw"])) <= 2 * dwm).all()
