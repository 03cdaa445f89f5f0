"""Outputs of the short convolution and the selective scan lie in memory of their own, but for the documented
forms in place: every pair of an output and another argument, without a GPU."""
import pytest

from test_layer_abi import ALL, _err, conv_decode, sel_bwd, sel_decode, sel_fwd

from gated_delta_rule_41_amd._lib import KDA_ERR_INVALID_ARG, KDA_ERR_WORKSPACE, KDA_F32

OUT = {"conv_fwd": ("y", "final_state"), "conv_bwd": ("dx", "dweight", "dbias", "d_initial_state"), "conv_decode": ("state_out", "y"),
       "sel_fwd": ("y", "final_state"),
       "sel_bwd": ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "d_initial_state"), "sel_decode": ("state_out", "y")}
# outputs that may be an input themselves
IN_PLACE = {"conv_fwd": {}, "conv_bwd": {}, "conv_decode": {"state_out": ("state_in",), "y": ("x",)},
            "sel_fwd": {"y": ("x", "dt", "z")}, "sel_bwd": {n: ("x", "dt", "z", "dy") for n in ("dx", "ddt", "dz")},
            "sel_decode": {"state_out": ("state_in",), "y": ("x", "dt", "z")}}


@pytest.mark.parametrize("name,out", [(n, o) for n, outs in OUT.items() for o in outs])
def test_outputs_share_no_memory(name, out):
    call = ALL[name]
    every = {n: call.at(n) for n in call.names}      # the ones that may be absent too
    assert set(OUT[name]) < set(every)
    for other in call.names:
        if other in (out, "workspace"):
            continue
        for off in (0, -16):                         # itself, and its first bytes
            if off == 0 and other in IN_PLACE[name].get(out, ()):
                continue
            assert call(**{**every, out: call.at(other) + off}) == KDA_ERR_INVALID_ARG, (other, off)
            assert "overlap" in _err(), (other, off, _err())


def test_in_place_needs_equal_rows():
    """Another type, or rows with gaps: a row of the output lies over other rows of the input."""
    for call, out, ins, strides in ((conv_decode, "y", ("x",), ("x_stride",)), (sel_decode, "y", ("x", "dt", "z"), ("x_stride", "dt_stride", "z_stride")),
                                    (sel_fwd, "y", ("x", "dt", "z"), ("x_stride", "dt_stride", "z_stride")),
                                    (sel_bwd, "dx", ("x", "dt", "z"), ("x_stride", "dt_stride", "z_stride"))):
        for name, stride in zip(ins, strides):
            assert call(cfg={"out_dtype": KDA_F32}, **{out: call.at(name)}) == KDA_ERR_INVALID_ARG and "overlap" in _err()
            assert call(cfg={stride: 72}, **{out: call.at(name)}) == KDA_ERR_INVALID_ARG and "overlap" in _err()


def test_in_place_is_accepted():
    """Such calls get as far as the workspace."""
    for name, outs in IN_PLACE.items():
        call = ALL[name]
        if call.ws:
            for out, ins in outs.items():
                for other in ins:
                    assert call(T=4096, wsb=0, **{out: call.at(other)}) == KDA_ERR_WORKSPACE, (out, other, _err())
    # dz is not used without z
    assert sel_bwd(wsb=0, z=0, dz=sel_bwd.at("dx")) == KDA_ERR_WORKSPACE
