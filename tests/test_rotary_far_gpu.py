"""Rotary positions far out, against angles from the plan's frequencies in exact arithmetic."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import serving_turns as exact
import transformer_linear_layer_gb300 as tll
from test_rotary_gpu import host, matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 1, 2 ** 40, 2 ** 50, 2 ** 54])
def test_far_positions(far, interleaved):
    """To the usual bound and the table's own error, |p| 2^-62 radians, of |x_a| + |x_b|."""
    N, H, D = 9, 2, 64
    x = matrix(N, H, D, H * D, torch.float32)
    places = [far, -far, far - 1, far // 3, -(far // 7), far - 12345, 1, 0, far // 2 + 1]
    positions = torch.tensor(places, device="cuda")
    r = tll.Rotary(64, interleaved=interleaved, scaling="ntk", factor=2.0)
    theta = exact.angles(places, r.frequencies)
    for sign, call in ((1, tll.rotary_forward), (-1, tll.rotary_backward)):
        want = ref.rotate(host(x), theta, 64, interleaved, 1.0, sign)
        tol = ref.rotate_tol(host(x), want, 64, interleaved, 1.0, ref.HALF["fp32"])
        off = np.array([abs(p) * 2.0 ** -62 for p in places])[:, None, None]
        for i in range(32):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
            tol[:, :, [a, b]] += (off * (np.abs(host(x))[:, :, [a]] + np.abs(host(x))[:, :, [b]]))
        assert np.all(np.abs(host(call(x, positions, r)) - want) <= tol)
