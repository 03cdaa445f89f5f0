"""The tolerances of tests/linear_dg.py reject a wrong gradient of the gates, in every case
and type that the GPU test runs: none, half of it, its negative, one without the terms
that cross a whole block, one of the token before."""
import numpy as np
import pytest

import linear_dg
from linear_ref import BF16


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(linear_dg.CASES)))
def test_wrong_gradients_are_rejected(case, dtype):
    lens, H, Hk, dk, dv, gate, states = linear_dg.CASES[case]
    x = linear_dg.make(case, lens, H, Hk, dk, dv, dtype, gate, states)
    tol = linear_dg.Tolerance(x, lens, dtype, dk ** -0.5)
    cross = linear_dg.crossing(x, lens, dk ** -0.5)
    # the crossing terms are part of the gradient: with S and dS at the borders taken as given they add up to it
    assert np.abs(cross).max() > 0
    shifted = np.roll(tol.tokens, 1, 0)
    if tol.per_head:
        cross = cross.sum(0)
    wrong = {"none": 0 * tol.r, "half": tol.r / 2, "negative": -tol.r, "no crossing": tol.r - cross}
    if not tol.per_head:
        wrong["token before"] = shifted
    for stored in (0.0, BF16):
        assert tol.off(tol.r, stored) == (0.0, 0.0)
        for name, y in wrong.items():
            norm, element = tol.off(y, stored)
            assert norm > 2.0, (name, norm, element)
        # and they are not wider than they say: an error of the bf16 roundings' size is near the bound
        if dtype == "bf16" and not tol.per_head:
            y = tol.r + np.sqrt(tol.var) * np.random.default_rng(case).choice([-1.0, 1.0], tol.r.shape)
            assert tol.off(y)[0] <= 1.0 + 1e-9


def test_the_gradient_against_differences():
    """The 64-bit dg that the tolerances are for, along random directions of g."""
    lens = [5, 3]
    rng = np.random.default_rng(5)
    import linear_ref as ref
    x = linear_dg.make(50, lens, 4, 2, 3, 5, "f32", "token", True)
    tol = linear_dg.Tolerance(x, lens, "f32", 0.5)

    def loss(g):
        o, final, _ = ref.linear_fwd(x["q"], x["k"], x["v"], g, lens, x["s0"], 0.5)
        return (o * x["dO"]).sum() + (final * x["dS"]).sum()

    g = x["g"].astype(np.float64)
    for _ in range(3):
        u = rng.standard_normal(g.shape)
        diff = (loss(g + 1e-5 * u) - loss(g - 1e-5 * u)) / 2e-5
        assert abs(diff - (tol.r * u).sum()) <= 1e-6 * (1 + np.abs(tol.r * u).sum())


def test_rounding_to_bf16_is_torchs():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(6).standard_normal(4096).astype(np.float32)
    assert np.array_equal(linear_dg.rounded_to_bf16(x), torch.from_numpy(x).bfloat16().float().numpy())
