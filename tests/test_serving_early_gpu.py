"""Early start at level 2 around the serving calls: a call that runs a kernel lets later calls read what older ones wrote,
one that runs none does not (see test_early_outputs_gpu)."""
import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_early_outputs_gpu import plain, setup  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_rotation_of_nothing_orders_nothing(setup):  # noqa: F811
    call, x, y, isolated, early, s, ctx, w = setup
    z = torch.randn(4, 2, 64, device="cuda")
    positions = torch.arange(4, device="cuda")
    none, some = tll.Rotary(0), tll.Rotary(64)
    torch.cuda.synchronize()
    kept = z.clone()

    def turn(r):
        with torch.cuda.stream(s):
            tll.rotary_forward(z, positions, r, out=z, ctx=ctx)

    call(x[2], y[2])
    call(x[0], y[3])
    turn(none)
    assert call(y[2], y[20]) == isolated  # y[2]'s call may still run
    call(x[2], y[2])
    call(x[0], y[3])
    turn(some)
    assert call(y[2], y[21]) == early     # the rotation has waited for it
    torch.cuda.synchronize()
    want = plain(plain(x[2], w).bfloat16(), w)
    for out in (y[20], y[21]):
        assert float((out.float() - want).norm() / want.norm()) < 1e-2
    assert not torch.equal(z, kept)
