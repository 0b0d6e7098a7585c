"""Serving calls that have nothing to do, at the C ABI (see test_serving_abi_cpu for the stand-ins)."""
import transformer_linear_layer_gb300 as tll
from test_serving_abi_cpu import at, ctx, needs_no_gpu, plan, rotary  # noqa: F401


@needs_no_gpu
def test_a_rotation_of_nothing_in_place_reaches_no_device(ctx):  # noqa: F811
    for form in ("forward", "backward"):
        assert rotary(ctx, form, r=plan(0, turns=None), y=at(0)) == tll.OK
        assert rotary(ctx, form, r=plan(0, turns=None), N=1, y=at(0), ldy=500) == tll.OK
        assert rotary(ctx, form, r=plan(0, turns=None)) == tll.ERR_CUDA           # a copy
        assert rotary(ctx, form, r=plan(2), y=at(0)) == tll.ERR_CUDA
        assert rotary(ctx, form, r=plan(0, turns=None), y=at(0), ldy=200) == tll.ERR_ARG
