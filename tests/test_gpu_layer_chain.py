"""The norm, the convolution and the recurrences together, as a layer and a server use them: prompts and steps, gradients,
captured graphs, other streams, several calls at once."""
import numpy as np
import pytest

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Layer:
    """Residual + norm, projections, convolution, selective scan; a KDA layer's q, k and v through the same convolution."""

    def __init__(self, width=128, inner=192, S=16, dtype=F32):
        gen = torch.Generator().manual_seed(5)

        def normal(*shape, dt=dtype, scale=1.0):
            return (torch.randn(*shape, generator=gen) * scale).to(dt).cuda()

        self.inner, self.S = inner, S
        self.norm = 1 + 0.1 * normal(width)
        self.w_in = normal(width, 2 * inner, scale=width ** -0.5)
        self.taps, self.bias = normal(inner, 4, scale=0.5), normal(inner, scale=0.1)
        self.w_x = normal(inner, inner + 2 * S, scale=inner ** -0.5)
        self.dt_bias = normal(inner, dt=F32) - 3
        self.A = -torch.exp(normal(inner, S, dt=F32))
        self.D = normal(inner, dt=F32)
        self.w_out = normal(inner, width, scale=inner ** -0.5)

    def params(self):
        return [self.norm, self.w_in, self.taps, self.bias, self.w_x, self.dt_bias, self.A, self.D, self.w_out]

    def prompt(self, x, residual, cu, conv_state, state, train=False):
        norm, conv, scan = (kda.kda_norm, kda.kda_conv, kda.kda_selective) if train else (
            kda.kda_norm_fwd, kda.kda_conv_fwd, kda.kda_selective_fwd)
        y, residual = norm(x, self.norm, residual)
        xz = y @ self.w_in
        u, conv_state = conv(xz[:, :self.inner], self.taps, self.bias, cu, conv_state)
        dt, B, C = (u @ self.w_x).split([self.inner, self.S, self.S], 1)
        y, state = scan(u, dt, self.A, B[:, None], C[:, None], cu, state, D=self.D, z=xz[:, self.inner:], dt_bias=self.dt_bias)
        return y @ self.w_out, residual, conv_state, state

    def step(self, x, residual, conv_state, state):
        y, residual = kda.kda_norm_fwd(x, self.norm, residual)
        xz = y @ self.w_in
        u, _ = kda.kda_conv_decode(xz[:, :self.inner], self.taps, self.bias, conv_state, out_state=conv_state)
        dt, B, C = (u @ self.w_x).split([self.inner, self.S, self.S], 1)
        y, _ = kda.kda_selective_decode(u, dt, self.A, B[:, None], C[:, None], state, D=self.D, z=xz[:, self.inner:],
                                        dt_bias=self.dt_bias, out_state=state)
        return y @ self.w_out, residual


def stream(lens, width=128, dtype=F32, seed=3):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    x, r = (torch.randn(T, width, generator=gen).to(dtype).cuda() for _ in range(2))
    return x, r, torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def test_steps_continue_a_prompt():
    need_gpu()
    layer = Layer()
    lens = [90, 1, 33]
    x, r, cu = stream([n + 4 for n in lens])
    start = cu[:-1].tolist()
    want, _, cs, ss = layer.prompt(x, r, cu, None, None)
    pick = [t for s, n in zip(start, lens) for t in range(s, s + n)]
    _, _, conv_state, state = layer.prompt(x[pick], r[pick], stream(lens)[2], None, None)
    for i in range(4):
        rows = [s + n + i for s, n in zip(start, lens)]
        y, _ = layer.step(x[rows], r[rows], conv_state, state)
        # fp32 throughout; the matrix products dominate: 192 terms each, four of them in a row
        assert torch.allclose(y, want[rows], rtol=0, atol=float(want.abs().max()) * 4 * 192 * 2.0 ** -24 * 4)
    # the state's projections' rounding passes through a product of 128 and the convolution
    assert torch.allclose(conv_state, cs, rtol=0, atol=float(cs.abs().max()) * 128 * 2.0 ** -24 * 4)
    assert torch.allclose(state, ss, rtol=0, atol=float(ss.abs().max()) * 4 * 192 * 2.0 ** -24 * 4)


def test_gradients_of_the_layer():
    """The layer's gradients along a direction against differences of its loss in 64 bits."""
    need_gpu()
    import layer_ref as ref

    layer = Layer()
    lens = [70, 3, 20]
    x, r, cu = stream(lens)
    params = layer.params()
    for p in params:
        p.requires_grad_()
    x.requires_grad_()
    y, res, _, _ = layer.prompt(x, r, cu, None, None, train=True)
    up, up_r = stream(lens, seed=8)[:2]
    ((y * up).sum() + (res * up_r).sum()).backward()
    gen = np.random.default_rng(0)
    host = [p.detach().double().cpu().numpy() for p in params + [x]]
    dirs = [gen.normal(size=p.shape) * np.abs(p).mean() for p in host]
    rr, uy, ur = (t.double().cpu().numpy() for t in (r, up, up_r))

    def loss(e):
        norm, w_in, taps, bias, w_x, dt_bias, A, D, w_out, xx = (p + e * d for p, d in zip(host, dirs))
        s = xx + rr
        yy, _ = ref.norm_fwd(s, norm, 1e-6)
        xz = yy @ w_in
        u, _, _ = ref.conv_fwd(xz[:, :192], taps, bias, np.zeros((3, 3, 192)), lens)
        p = u @ w_x
        o = ref.selective(u, p[:, :192], A, p[:, None, 192:208], p[:, None, 208:], D, xz[:, 192:], dt_bias, lens, np.zeros((3, 192, 16)))
        return ((o["y"] @ w_out) * uy).sum() + (s * ur).sum()

    grads = [p.grad.double().cpu().numpy() for p in params + [x]]
    got = sum((g * d).sum() for g, d in zip(grads, dirs))
    size = sum(np.abs(g * d).sum() for g, d in zip(grads, dirs))
    # Richardson's step takes the third derivative out; what is left is fp32 rounding of the gradients
    d1, d2 = ((loss(e) - loss(-e)) / (2 * e) for e in (2.0 ** -12, 2.0 ** -13))
    assert abs(got - (4 * d2 - d1) / 3) <= size * 1000 * 2.0 ** -24, (got, d1, d2, size)


def test_convolution_before_kda():
    """q, k and v of a KDA layer from one convolution over their joined channels."""
    need_gpu()
    lens, H, dk = [100, 28], 2, 64
    T, C = 128, 3 * H * dk
    gen = torch.Generator().manual_seed(2)
    qkv = torch.randn(T, C, generator=gen).to(BF16).cuda()
    taps = torch.randn(C, 4, generator=gen).to(BF16).cuda()
    cu = stream(lens)[2]
    mixed, _ = kda.kda_conv_fwd(qkv, taps, None, cu)
    q, k, v = (t.reshape(T, H, dk).contiguous() for t in mixed.split(H * dk, 1))
    g = -torch.rand(T, H, dk, generator=gen).to(BF16).cuda() * 0.1
    beta = torch.randn(T, H, generator=gen).to(BF16).cuda()
    o, state, _ = (*kda.kda_fwd(q, k, v, g, beta, cu), None)[:3]
    assert torch.isfinite(o).all() and o.shape == (T, H, dk)
    parts = [kda.kda_conv_fwd(t.contiguous(), w.contiguous(), None, cu)[0] for t, w in zip(qkv.split(H * dk, 1), taps.split(H * dk))]
    assert torch.equal(torch.cat(parts, 1), mixed)


def test_eight_bit_rows_feed_an_integer_product():
    """Codes and scales stand for the norm: a product of the codes is the product of the values to one fp32 rounding."""
    need_gpu()
    x, r, _ = stream([64], 256, BF16)
    y, _ = kda.kda_norm_fwd(x, None, r, out_dtype=F32)
    codes, _, scale = kda.kda_norm_fwd(x, None, r, out_dtype=torch.int8)
    w = torch.randint(-127, 128, (256, 32), device="cuda")
    product = (codes.double() @ w.double()) * scale.double()[:, None]
    # half a code's step for each of the row's values, once for each weight
    assert ((product - y.double() @ w.double()).abs() <= scale.double()[:, None] * 0.5001 * w.double().abs().sum(0)).all()


def _graph_case(dtype=BF16):
    layer = Layer(dtype=dtype)
    lens = [300, 1, 211]
    x, r, cu = stream(lens, dtype=dtype)
    return layer, x, r, cu


def test_captured_prompts_and_steps():
    """Two captured graphs with workspaces of their own, replayed in turn with eager work and waits between."""
    need_gpu()
    layer, x, r, cu = _graph_case()
    N = 3
    cs, ss = torch.zeros(N, 3, 192, dtype=BF16, device="cuda"), torch.zeros(N, 192, 16, device="cuda")
    x2, r2 = torch.empty_like(x), torch.empty_like(r)
    xs, rs = x[:N].clone(), r[:N].clone()

    def prompt():
        return layer.prompt(x2, r2, cu, None, None)

    def step():
        return layer.step(xs, rs, cs, ss)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2.copy_(x), r2.copy_(r)
        prompt(), step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out = prompt()
    with torch.cuda.graph(g2):
        one = step()
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        x2.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        r2.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        want = prompt()
        cs.copy_(want[2]), ss.copy_(want[3])
        wy, _ = step()
        after = cs.clone(), ss.clone()
        cs.copy_(want[2]), ss.copy_(want[3])
        for t in out:
            t.zero_()
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert torch.equal(one[0], wy) and torch.equal(cs, after[0]) and torch.equal(ss, after[1])


def test_captured_backward():
    need_gpu()
    layer, x, r, cu = _graph_case(F32)
    dt, B, C, z = x[:, :96].contiguous(), x[:, None, :16].contiguous(), x[:, None, 16:32].contiguous(), r[:, :96].contiguous()
    u, A, D, bias = r[:, 16:112].contiguous(), layer.A[:96], layer.D[:96], layer.dt_bias[:96]
    taps = layer.taps[:96].contiguous()

    def grads():
        a = kda.kda_selective_bwd(u, dt, A, B, C, z, cu, D=D, z=z, dt_bias=bias)
        b = kda.kda_conv_bwd(u, taps, None, z, cu)
        c = kda.kda_norm_bwd(x, layer.norm, r, x)
        return [t for d in (a, b, c) for t in d.values() if t is not None]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        grads()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = grads()
    for i in range(3):
        u.normal_(), z.normal_(), dt.normal_()
        want = grads()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_streams_at_once():
    """Calls on two streams at the same time, each with its own workspace, give what they give alone."""
    need_gpu()
    layer, x, r, cu = _graph_case()
    want = layer.prompt(x, r, cu, None, None)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(layer.prompt(x, r, cu, None, None))
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
