"""Rows of very many heads: taken up to the documented number, refused beyond (the CPU tests have the other limits)."""
import pytest
import torch

import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,fits", [(65535, True), (65536, False)])
def test_many_wide_heads(heads, fits):
    D = 200
    buf = torch.randn(heads * D + 8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    aligned, odd = (buf[i:i + heads * D].view(1, heads, D) for i in (0, 1))
    positions, r = torch.tensor([77], device="cuda"), tll.Rotary(64)
    whole = tll.rotary_forward(aligned.contiguous(), positions, r)  # 16 bytes at a time: many heads a block
    assert whole.shape == (1, heads, D) and torch.equal(whole[:, :, 64:], aligned[:, :, 64:])
    if not fits:
        with pytest.raises(tll.LinError) as e:
            tll.rotary_forward(odd, positions, r)  # an element at a time: a head a block
        assert e.value.status == tll.ERR_UNSUPPORTED
        return
    got = tll.rotary_forward(odd, positions, r)
    want = torch.cat([tll.rotary_forward(h.contiguous(), positions, r) for h in odd.split(1000, 1)], 1)
    assert torch.equal(got, want)
