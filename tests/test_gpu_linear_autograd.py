"""kda_linear under autograd where the loss uses one of its outputs."""
import pytest

import linear_dg

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda
from test_gpu_linear_dg import on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("used", ["o", "final_state"])
def test_loss_on_one_output(used, monkeypatch):
    """The backward gets no dS_final (a state for every document) for a loss on o alone, and the gradients are those of
    the direct call."""
    need_gpu()
    lens = [300, 41]
    d, cu = on_gpu(linear_dg.make(61, lens, 4, 2, 64, 64, "bf16", "token", True), lens, "bf16")
    calls, direct = [], kda.linear.kda_linear_bwd

    def watched(q, k, v, g, dO, cu_seqlens, initial_state, dS_final, **kw):
        calls.append((dO, dS_final))
        return direct(q, k, v, g, dO, cu_seqlens, initial_state, dS_final, **kw)

    monkeypatch.setattr(kda.linear, "kda_linear_bwd", watched)
    leaves = {n: d[n].clone().requires_grad_(True) for n in ("q", "k", "v", "g", "s0")}
    o, sf = kda.kda_linear(*(leaves[n] for n in ("q", "k", "v", "g")), cu, leaves["s0"], scale=0.125)
    if used == "o":
        (o * d["dO"].float()).sum().backward()
        dO, dS = d["dO"], None
    else:
        (sf * d["dS"]).sum().backward()
        dO, dS = torch.zeros_like(d["dO"]), d["dS"]
    want = direct(d["q"], d["k"], d["v"], d["g"], dO, cu, d["s0"], dS, scale=0.125, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    (got_dO, got_dS), = calls
    assert torch.equal(got_dO, dO) and (got_dS is None if dS is None else torch.equal(got_dS, dS))
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "dS0")):
        assert torch.equal(leaves[n].grad, want[gn].to(leaves[n].dtype)), n
