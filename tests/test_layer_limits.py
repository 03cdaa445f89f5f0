"""The sizes that the norm, the short convolution and the selective scan take and refuse, without a GPU."""
import pytest

from test_layer_abi import BASE, _err, norm_bwd, norm_fwd

from gated_delta_rule_41_amd import _lib
from gated_delta_rule_41_amd._lib import KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("C,most", [(1, 16 * (2 ** 24 - 1)), (128, 16 * (2 ** 24 - 1)), (129, 8 * (2 ** 24 - 1)), (256, 8 * (2 ** 24 - 1)),
                                    (257, 4 * (2 ** 24 - 1)), (1024, 4 * (2 ** 24 - 1)), (1025, 2 ** 24 - 1), (8192, 2 ** 24 - 1),
                                    (8193, 2 ** 23 - 1), (16384, 2 ** 23 - 1)])
def test_rows_of_the_norm(C, most):
    """As many rows as a launch of that width covers: 262144 tokens of 32 heads of 128 among them."""
    cfg = _lib.make_norm_config(C)
    assert _lib.kda_norm_bwd_workspace_size(cfg, most) > 0 and _lib.kda_norm_bwd_workspace_size(cfg, most + 1) == 0
    for call, first in ((norm_fwd, "x"), (norm_bwd, "s")):
        assert call(T=most, cfg=dict(C=C), **{first: BASE + 8}) == KDA_ERR_INVALID_ARG and "aligned" in _err()
        for rows in (most + 1, 2 ** 62, 2 ** 63 - 1):
            assert call(T=rows, cfg=dict(C=C), **{first: BASE + 8}) == KDA_ERR_UNSUPPORTED and "too large" in _err()
