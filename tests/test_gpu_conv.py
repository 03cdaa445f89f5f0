"""The short causal convolution against 64 bits: types, widths, documents, states, strides, gradients, single tokens."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def host(t):
    return t.detach().double().cpu().numpy()


def make(lens, C, W, dtype, seed=0, wt=None):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, dt=dtype):
        return torch.randn(*shape, generator=gen).to(dt).cuda()

    T, N = sum(lens), len(lens)
    d = {"x": normal(T, C), "w": normal(C, W, dt=wt or dtype), "b": normal(C, dt=wt or dtype),
         "state": normal(N, W - 1, C), "dy": normal(T, C), "dend": normal(N, W - 1, C)}
    d["cu"] = torch.tensor(ref.starts(lens), dtype=torch.int32, device="cuda")
    return d


def check(got, want, bound, dtype):
    assert got.dtype == dtype
    assert (np.abs(host(got) - want) <= (bound + np.abs(want) * HALF[dtype]) * 1.01).all()


# empty, single-token and long documents; strips of 8 tokens end inside and at documents' ends
LENS = [[1], [5], [8], [17, 0, 1, 2, 3, 40], [0, 0, 9], [300, 1, 127], [64, 64]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,dtype,wt", [(64, BF16, BF16), (333, F32, F32), (8, BF16, F32), (1, F32, F32), (100, BF16, BF16), (2080, F32, F32)])
@pytest.mark.parametrize("act", ["silu", None])
def test_forward_and_backward(lens, W, C, dtype, wt, act):
    need_gpu()
    d = make(lens, C, W, dtype, W, wt)
    h = {n: host(x) for n, x in d.items()}
    y, end = kda.kda_conv_fwd(d["x"], d["w"], d["b"], d["cu"], d["state"], activation=act)
    want, last, bound = ref.conv_fwd(h["x"], h["w"], h["b"], h["state"], lens, act is not None)
    check(y, want, bound, dtype)
    assert end.dtype == dtype and (host(end) == last).all()
    g = kda.kda_conv_bwd(d["x"], d["w"], d["b"], d["dy"], d["cu"], d["state"], d["dend"], activation=act)
    want = ref.conv_bwd(h["x"], h["w"], h["b"], h["state"], lens, h["dy"], h["dend"], act is not None)
    for n, t in (("dx", dtype), ("dw", F32), ("db", F32), ("dstate", dtype)):
        check(g[n], *want[n], t)


@pytest.mark.parametrize("C,dtype", [(4099, BF16), (4104, BF16), (14003, F32)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_eight_channels_a_thread(C, dtype, W):
    """Larger calls: eight channels a thread, the last of a row's threads moved back, strips of 16 to 64 tokens."""
    need_gpu()
    lens = [700, 1, 0, 130, 64, 2, 303]
    d = make(lens, C, W, dtype)
    h = {n: host(x) for n, x in d.items()}
    y, end = kda.kda_conv_fwd(d["x"], d["w"], d["b"], d["cu"], d["state"], out_dtype=F32)
    want, last, bound = ref.conv_fwd(h["x"], h["w"], h["b"], h["state"], lens)
    check(y, want, bound, F32)
    assert (host(end) == last).all()
    g = kda.kda_conv_bwd(d["x"], d["w"], d["b"], d["dy"], d["cu"], d["state"], d["dend"], out_dtype=F32)
    want = ref.conv_bwd(h["x"], h["w"], h["b"], h["state"], lens, h["dy"], h["dend"])
    for n, t in (("dx", F32), ("dw", F32), ("db", F32), ("dstate", dtype)):
        check(g[n], *want[n], t)


def test_strip_lengths_change_nothing():
    """64 tokens a strip in one call, fewer in calls that carry the state on: the same bits."""
    need_gpu()
    d = make([11001], 12288, 4, BF16)
    y, end = kda.kda_conv_fwd(d["x"], d["w"], d["b"], d["cu"], d["state"])
    state, parts = d["state"], []
    for x in d["x"].split(1001):
        part, state = kda.kda_conv_fwd(x, d["w"], d["b"], None, state)
        parts.append(part)
    assert torch.equal(y, torch.cat(parts)) and torch.equal(end, state)
    g = kda.kda_conv_bwd(d["x"], d["w"], d["b"], d["dy"], d["cu"], d["state"], d["dend"])
    at = 10000
    last = kda.kda_conv_bwd(d["x"][at:], d["w"], d["b"], d["dy"][at:], None, d["x"][None, at - 3:at].contiguous(), d["dend"])
    assert torch.equal(g["dx"][at:], last["dx"])


def test_absent_arguments_and_equal_documents():
    need_gpu()
    d = make([12, 12, 12], 72, 4, F32)
    zero = torch.zeros_like(d["state"])
    full = kda.kda_conv_fwd(d["x"], d["w"], torch.zeros_like(d["b"]), d["cu"], zero)
    y, end = kda.kda_conv_fwd(d["x"], d["w"], num_seqs=3)
    assert torch.equal(y, full[0]) and torch.equal(end, full[1])
    y, end = kda.kda_conv_fwd(d["x"], d["w"], num_seqs=3, output_final_state=False)
    assert torch.equal(y, full[0]) and end is None
    full = kda.kda_conv_bwd(d["x"], d["w"], torch.zeros_like(d["b"]), d["dy"], d["cu"], zero, zero)
    g = kda.kda_conv_bwd(d["x"], d["w"], None, d["dy"], num_seqs=3)
    assert torch.equal(g["dx"], full["dx"]) and torch.equal(g["dw"], full["dw"]) and g["db"] is None and g["dstate"] is None
    y, end = kda.kda_conv_fwd(d["x"][:0], d["w"], d["b"], None, d["state"], num_seqs=3)
    assert y.shape == (0, 72) and torch.equal(end, d["state"])
    g = kda.kda_conv_bwd(d["x"][:0], d["w"], d["b"], d["dy"][:0], None, d["state"], d["dend"], num_seqs=3)
    assert torch.equal(g["dstate"], d["dend"]) and (g["dw"] == 0).all() and (g["db"] == 0).all()


@pytest.mark.parametrize("gap", [8, 24, 3])
def test_rows_of_a_wider_tensor(gap):
    """x as part of a projection's rows; a gap that is no multiple of eight takes one channel at a time."""
    need_gpu()
    wide = torch.randn(50, 64 + gap, device="cuda").to(BF16)
    d = make([30, 20], 64, 4, BF16)
    for off in ([0, 8] if gap > 8 else [0]):
        x = wide[:, off:off + 64]
        for call in (lambda v: kda.kda_conv_fwd(v, d["w"], d["b"], d["cu"], d["state"])[0],
                     lambda v: kda.kda_conv_bwd(v, d["w"], d["b"], d["dy"], d["cu"], d["state"])["dx"],
                     lambda v: kda.kda_conv_bwd(v, d["w"], d["b"], d["dy"], d["cu"], d["state"])["dw"],
                     lambda v: kda.kda_conv_decode(v[:2], d["w"], d["b"], d["state"])[0]):
            a, b = call(x), call(x.contiguous())
            assert torch.equal(a, b)


@pytest.mark.parametrize("C,dtype,W", [(64, BF16, 4), (333, F32, 3), (12288, BF16, 2), (1, BF16, 4)])
def test_decode_continues_a_prompt(C, dtype, W):
    """Single tokens after a prompt equal the prompt with those tokens, bit for bit, in place too."""
    need_gpu()
    lens = [9, 1, 4]
    d = make(lens, C, W, dtype)
    more = make([5, 5, 5], C, W, dtype, 9)["x"].view(3, 5, C)
    _, state = kda.kda_conv_fwd(d["x"], d["w"], d["b"], d["cu"], d["state"])
    at = ref.starts(lens)
    joined = torch.cat([torch.cat([d["x"][at[n]:at[n + 1]], more[n]]) for n in range(3)])
    long = torch.tensor(ref.starts([14, 6, 9]), dtype=torch.int32, device="cuda")
    want, end = kda.kda_conv_fwd(joined, d["w"], d["b"], long, d["state"])
    ends = ref.starts([14, 6, 9])[1:]
    for t in range(5):
        y, new = kda.kda_conv_decode(more[:, t].contiguous(), d["w"], d["b"], state)
        again, same = kda.kda_conv_decode(more[:, t].contiguous(), d["w"], d["b"], state, out_state=state)
        assert same is state and torch.equal(y, again) and torch.equal(new, state)
        assert torch.equal(y, want[[e - 5 + t for e in ends]])
    assert torch.equal(state, end)
    y, _ = kda.kda_conv_decode(more[:, 0].contiguous(), d["w"])
    zero, _ = kda.kda_conv_decode(more[:, 0].contiguous(), d["w"], torch.zeros_like(d["b"]), torch.zeros_like(state))
    assert torch.equal(y, zero)


def test_documents_and_rows_behind_them():
    """NaN in one document, and in the rows behind the last one, stays there; those rows of the outputs are left alone."""
    need_gpu()
    lens, C = [20, 33, 11], 64
    d = make(lens + [16], C, 4, BF16)
    cu = d["cu"][:4].contiguous()
    state = d["state"][:3].contiguous()
    clean, _ = kda.kda_conv_fwd(d["x"], d["w"], d["b"], cu, state)
    x = d["x"].clone()
    x[30] = float("nan")
    x[64:] = float("nan")
    y, end = kda.kda_conv_fwd(x, d["w"], d["b"], cu, state)
    assert torch.isnan(y[30:34]).all()
    keep = [t for t in range(64) if not 30 <= t < 34]
    assert torch.equal(y[keep], clean[keep]) and torch.isfinite(end).all()
    g = kda.kda_conv_bwd(d["x"], d["w"], d["b"], d["dy"], cu, state)
    dy = d["dy"].clone()
    dy[64:] = float("nan")
    dy[30, 3] = float("inf")
    h = kda.kda_conv_bwd(d["x"], d["w"], d["b"], dy, cu, state)
    keep = [t for t in range(64) if not 27 <= t <= 30]
    assert torch.equal(h["dx"][keep], g["dx"][keep]) and torch.equal(h["dx"][27:31, 4:], g["dx"][27:31, 4:])
    assert torch.equal(h["dw"][4:], g["dw"][4:]) and not torch.isfinite(h["dw"][3]).all()


def test_autograd():
    need_gpu()
    d = make([7, 1, 12], 40, 4, F32)
    leaves = [d[n].clone().requires_grad_() for n in ("x", "w", "b", "state")]
    y, end = kda.kda_conv(leaves[0], leaves[1], leaves[2], d["cu"], leaves[3])
    ((y * d["dy"]).sum() + (end * d["dend"]).sum()).backward()
    g = kda.kda_conv_bwd(d["x"], d["w"], d["b"], d["dy"], d["cu"], d["state"], d["dend"])
    for leaf, n in zip(leaves, ("dx", "dw", "db", "dstate")):
        assert torch.equal(leaf.grad, g[n])
    y, end = kda.kda_conv(leaves[0], leaves[1], None, d["cu"])
    gx, = torch.autograd.grad(end.sum(), leaves[0])
    # the last rows of every document, and nothing else
    want = torch.zeros_like(gx)
    want[[4, 5, 6, 7, 17, 18, 19]] = 1
    assert torch.equal(gx, want)


def test_refusals():
    need_gpu()
    d = make([6], 64, 4, BF16)
    with pytest.raises(kda.KdaError, match="width"):
        kda.kda_conv_fwd(d["x"], torch.zeros(64, 5, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="activation"):
        kda.kda_conv_fwd(d["x"], d["w"], activation="relu")
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_conv_fwd(d["x"].t().contiguous().t(), d["w"])
    with pytest.raises(ValueError, match="overlap"):
        kda.kda_conv_fwd(d["x"][:1].expand(6, 64), d["w"])
    with pytest.raises(kda.KdaError, match="aligned"):
        kda.kda_conv_fwd(torch.zeros(6, 72, dtype=BF16, device="cuda")[:, 4:68], d["w"])
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.kda_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"].long())
    with pytest.raises(TypeError):
        kda.kda_conv_fwd(d["x"], d["w"], d["b"].float())
    with pytest.raises(TypeError):
        kda.kda_conv_fwd(d["x"], d["w"], initial_state=d["state"].float())


def test_long_offsets():
    """Rows behind 2^31 elements of x."""
    need_gpu()
    C, T = 8192, 270000
    x = torch.zeros(T, C, dtype=BF16, device="cuda")
    x[-40:] = torch.randn(40, C, device="cuda").to(BF16)
    d = make([1], C, 4, BF16)
    cu = torch.tensor([0, T - 37, T], dtype=torch.int32, device="cuda")
    y, end = kda.kda_conv_fwd(x, d["w"], None, cu)
    want, last = kda.kda_conv_fwd(x[-37:].contiguous(), d["w"], None)
    assert torch.equal(y[-37:], want) and torch.equal(end[1], last[0])
    g = kda.kda_conv_bwd(x, d["w"], None, y, cu)
    want = kda.kda_conv_bwd(x[-37:].contiguous(), d["w"], None, want)
    assert torch.equal(g["dx"][-37:], want["dx"])
