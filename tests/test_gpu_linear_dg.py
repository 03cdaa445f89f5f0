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
