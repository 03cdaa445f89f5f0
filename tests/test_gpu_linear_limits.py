"""The linear rule at sizes near its limits."""
import pytest

from gpu_util import need_gpu, torch

import gated_delta_rule_41_amd as kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,Hk", [(1152, 28, 4), (1024, 127, 1)])
def test_prime_numbers_of_value_heads(T, H, Hk):
    """7 and 127 value heads to a key head, each in a workgroup of its own: dq and dk are the sums of what every value head
    gives with a key head of its own.  fp32: both sides add the same terms, 32 half steps of the root of their squares
    each (tests/linear_ref.py), which for independent inputs is the result's norm; dv and dg do not change."""
    need_gpu()
    R = H // Hk
    gen = torch.Generator(device="cuda").manual_seed(42)
    q, k = (torch.randn((T, Hk, 64), generator=gen, device="cuda") for _ in range(2))
    v, dO = (torch.randn((T, H, 64), generator=gen, device="cuda") for _ in range(2))
    g = -0.1 * torch.rand((T, H), generator=gen, device="cuda")
    print(f"[gpu-linear] {T} tokens, {H} heads on {Hk}", flush=True)
    got = kda.kda_linear_bwd(q, k, v, g, dO, scale=0.125)
    one = kda.kda_linear_bwd(q.repeat_interleave(R, 1), k.repeat_interleave(R, 1), v, g, dO, scale=0.125)
    torch.cuda.synchronize()
    assert torch.equal(got["dv"], one["dv"]) and torch.equal(got["dg"], one["dg"])
    for n in ("dq", "dk"):
        want = one[n].double().view(T, Hk, R, 64).sum(2)
        off = float((got[n].double() - want).norm() / want.norm())
        print(f"[gpu-linear]   {n}: {off:.2e}", flush=True)
        assert off <= 2 * 32 * 2.0 ** -24, n


def test_many_documents_of_one_token():
    """530000 documents x 2 heads of 128 x 128, more than 2^20 states: with no state before, o = scale (q . k) v,
    dv = scale (q . k) dO and dg = 0.  bf16 products are exact in fp32, and 128 of them add up with at most 128 half steps
    (2^-17) of their absolute sum M.  P and the result are rounded to bf16 once each: (1 + 2^-8)^2 - 1 = 2^-7 + 2^-16 of
    the value, and 2^-17 (1 + 2^-7) of M: at most 2^-7 of the value and 2^-15 of M.  dg is the difference of a row and a
    column sum of one product each, both fp32: 2 (2^-17 + 2^-17 + 2^-22) of its absolute terms, at most 2^-14."""
    need_gpu()
    N, H, d = 530000, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(41)
    q, k, v, dO = (torch.randn((N, H, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    g = torch.full((N, H), -0.1, device="cuda")
    print("[gpu-linear] one-token documents, forward", flush=True)
    o, none = kda.kda_linear_fwd(q, k, v, g, num_seqs=N, scale=0.5, out_dtype=torch.bfloat16, output_final_state=False)
    torch.cuda.synchronize()
    assert none is None
    P = 0.5 * (q.double() * k.double()).sum(2, keepdim=True)
    M = 0.5 * (q.double() * k.double()).abs().sum(2, keepdim=True)

    def check(name, x, b):
        worst = float(((x.double() - P * b.double()).abs() / ((2.0 ** -7 * P.abs() + 2.0 ** -15 * M) * b.double().abs() + 1e-30)).max())
        print(f"[gpu-linear]   {name}: largest error is {worst:.3f} of its bound", flush=True)
        assert worst <= 1.0, name

    check("o", o, v)
    print("[gpu-linear] one-token documents, backward", flush=True)
    gr = kda.kda_linear_bwd(q, k, v, g, dO, num_seqs=N, scale=0.5, out_dtype=torch.bfloat16, output_d_initial_state=False)
    torch.cuda.synchronize()
    check("dv", gr["dv"], dO)
    A = (M * (dO.double() * v.double()).abs().sum(2, keepdim=True))[:, :, 0]
    assert bool((gr["dg"].double().abs() <= 2.0 ** -14 * A).all())
    del gr
    torch.cuda.empty_cache()
