"""dg of the linear rule against 64 bits, within the tolerances of tests/linear_dg.py,
which tests/test_linear_dg_bounds.py shows to reject wrong ones."""
import numpy as np
import pytest

import linear_dg
from linear_ref import BF16

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[gpu-dg] {msg}", flush=True)


def on_gpu(x, lens, dtype):
    d = {n: None if a is None else torch.from_numpy(a).cuda() for n, a in x.items()}
    if dtype == "bf16":
        d.update({n: d[n].bfloat16() for n in ("q", "k", "v", "dO")})
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return d, cu


def host(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(linear_dg.CASES)))
def test_dg(case, dtype):
    need_gpu()
    lens, H, Hk, dk, dv, gate, states = linear_dg.CASES[case]
    _say(f"{lens} {H}/{Hk} {dk}x{dv} {gate} {dtype}")
    x = linear_dg.make(case, lens, H, Hk, dk, dv, dtype, gate, states)
    tol = linear_dg.Tolerance(x, lens, dtype, dk ** -0.5)
    d, cu = on_gpu(x, lens, dtype)
    for out in (torch.float32, torch.bfloat16):
        gr = kda.kda_linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"], out_dtype=out, scale=dk ** -0.5)
        torch.cuda.synchronize()
        norm, element = tol.off(host(gr["dg"]), BF16 if out == torch.bfloat16 else 0.0)
        _say(f"  {out}: the error's norm is {norm:.3f} of its bound, its largest element {element:.3f}")
        assert norm <= 1.0 and element <= 1.0


@pytest.mark.parametrize("gate", ["token", "head"])
def test_dg_in_its_own_type(gate):
    """Beside bf16 outputs dg may stay in fp32, the type of g: the same values as beside fp32 outputs, through the call
    and through autograd."""
    need_gpu()
    _say(f"own type, {gate}")
    lens = [300, 41]
    x = linear_dg.make(60, lens, 4, 2, 64, 64, "bf16", gate, True)
    d, cu = on_gpu(x, lens, "bf16")
    args = d["q"], d["k"], d["v"], d["g"], d["dO"], cu, d["s0"], d["dS"]
    want = kda.kda_linear_bwd(*args, scale=0.125)["dg"]
    rounded = kda.kda_linear_bwd(*args, scale=0.125, out_dtype=torch.bfloat16)
    gr = kda.kda_linear_bwd(*args, scale=0.125, out_dtype=torch.bfloat16, dg_dtype=torch.float32)
    torch.cuda.synchronize()
    assert gr["dg"].dtype == torch.float32 and torch.equal(gr["dg"], want)
    assert rounded["dg"].dtype == torch.bfloat16 and torch.equal(rounded["dg"], want.bfloat16())
    for n in ("dq", "dk", "dv", "dS0"):
        assert torch.equal(gr[n], rounded[n]), n
    for dg_dtype, grad in ((None, want.bfloat16().float()), (torch.bfloat16, want.bfloat16().float()), (torch.float32, want)):
        g = d["g"].clone().requires_grad_(True)
        o, sf = kda.kda_linear(d["q"], d["k"], d["v"], g, cu, d["s0"], scale=0.125, dg_dtype=dg_dtype)
        ((o * d["dO"].float()).sum() + (sf * d["dS"]).sum()).backward()
        torch.cuda.synchronize()
        assert g.grad.dtype == torch.float32 and torch.equal(g.grad, grad)
    with pytest.raises(ValueError, match="dg_dtype"):
        kda.kda_linear(d["q"], d["k"], d["v"], d["g"], cu, dg_dtype=torch.float16)
    with pytest.raises(ValueError, match="dg_dtype"):
        kda.kda_linear_bwd(*args, dg_dtype=torch.bfloat16)
