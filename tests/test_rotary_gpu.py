"""Rotary positions on the GPU against the formulas in float64 (serving_ref)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu
NAMES = {torch.float32: "fp32", torch.bfloat16: "bf16"}


def host(t):
    return t.double().cpu().numpy()


def matrix(N, H, D, ld, dtype, seed=0, offset=0):
    """N x H x D heads in rows of ld, the first `offset` elements into a buffer of NaN."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((N * ld + offset + 64,), float("nan"), dtype=dtype, device="cuda")
    x = buf.as_strided((N, H, D), (ld, D, 1), offset)
    x.copy_(torch.randn(N, H, D, generator=g).to(dtype))
    return x


def spread(N, dtype, far):
    g = torch.Generator().manual_seed(N)
    p = torch.randint(-far, far + 1, (N,), generator=g)
    p[0] = far
    return p.to(dtype).cuda()


def check(got, x, positions, r, sign, dtype):
    theta = ref.angles(positions.tolist(), r.turns.tolist())
    scale = float(np.float32(r.scale))
    want = ref.rotate(host(x), theta, r.dim, r.interleaved, scale, sign)
    tol = ref.rotate_tol(host(x), want, r.dim, r.interleaved, scale, ref.HALF[NAMES[dtype]])
    tol[:, :, r.dim:] = 0  # copied
    err = np.abs(host(got) - want)
    assert np.all(err <= tol), (err.max(), (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,D,rot,ld,offset", [
    (1, 1, 64, 64, 64, 0), (1, 24, 64, 64, 2304, 0), (5, 3, 64, 32, 192, 0), (700, 24, 64, 64, 2304, 8),
    (33, 5, 80, 20, 408, 0), (17, 2, 128, 96, 259, 0), (9, 4, 64, 64, 256, 3), (3, 1, 2, 2, 2, 0), (4, 7, 6, 0, 42, 0),
    (2, 3, 256, 256, 768, 0), (2, 130, 128, 128, 130 * 128, 0), (6, 2, 65, 64, 130, 0), (2, 1, 1024, 1024, 1024, 0)])
def test_parity(dtype, interleaved, N, H, D, rot, ld, offset):
    x = matrix(N, H, D, ld, dtype, offset=offset)
    for kind, far in ((torch.int32, 100000), (torch.int64, 2 ** 50)):
        positions = spread(N, kind, far)
        r = tll.Rotary(rot, interleaved=interleaved, scaling="yarn", factor=4.0, original_length=2048)
        check(tll.rotary_forward(x, positions, r), x, positions, r, 1, dtype)
        check(tll.rotary_backward(x, positions, r), x, positions, r, -1, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (32, False), (20, True)])
def test_in_place_and_strided_outputs(dtype, rot, interleaved):
    """The q and k columns of a qkv matrix in place; v, the padding and the other rows stay."""
    N, H, D = 77, 6, 64
    ld = 3 * 3 * D + 8
    r = tll.Rotary(rot, interleaved=interleaved)
    positions = torch.arange(N, device="cuda")
    qkv = matrix(N, 9, D, ld, dtype)
    whole = qkv.as_strided((N, ld), (ld, 1), 0).clone()
    want = tll.rotary_forward(qkv[:, :H], positions, r)
    out = matrix(N, 9, D, ld, dtype, seed=1)
    kept = out.clone()
    assert tll.rotary_forward(qkv[:, :H], positions, r, out=out[:, 3:]).data_ptr() == out[:, 3:].data_ptr()
    assert torch.equal(out[:, 3:], want) and torch.equal(out[:, :3], kept[:, :3])
    tll.rotary_forward(qkv[:, :H], positions, r, out=qkv[:, :H])
    assert torch.equal(qkv[:, :H], want)
    after = qkv.as_strided((N, ld), (ld, 1), 0)
    assert torch.equal(after[:, H * D:].nan_to_num(7.0), whole[:, H * D:].nan_to_num(7.0))


def test_gradient_is_the_adjoint_and_meets_differences():
    N, H, D = 11, 3, 64
    r = tll.Rotary(48, interleaved=True, scale=1.5)
    x, g = matrix(N, H, D, H * D, torch.float32), matrix(N, H, D, H * D, torch.float32, seed=1)
    positions = spread(N, torch.int64, 10 ** 6)
    y, dx = tll.rotary_forward(x, positions, r), tll.rotary_backward(g, positions, r)
    # <R x, g> = <x, R' g>, each side of 2112 products off by 8 * 2^-24 of its terms' sizes
    left, right = (host(y) * host(g)).sum(), (host(x) * host(dx)).sum()
    size = 1.5 * 2 * (np.abs(host(x)).sum(2, keepdims=True) * np.abs(host(g))).sum()
    assert abs(left - right) <= 16 * ref.FP32_HALF * size
    # differences along a few coordinates; the operator is linear, so h = 1 has no error of its own
    for n, h, d in ((0, 0, 0), (3, 1, 17), (10, 2, 47), (10, 2, 63)):
        up = x.clone()
        up[n, h, d] += 1.0
        diff = (host(tll.rotary_forward(up, positions, r)) - host(y))
        assert abs((diff * host(g)).sum() - host(dx)[n, h, d]) <= 64 * ref.FP32_HALF * 1.5 * (3 + np.abs(host(g)[n, h]).max()) * 4


def test_odd_values_reach_their_own_pair_only():
    x = matrix(4, 2, 64, 128, torch.bfloat16)
    positions = torch.arange(4, device="cuda")
    r = tll.Rotary(32)
    clean = tll.rotary_forward(x, positions, r)
    y = x.clone()
    y[1, 1, 3], y[2, 0, 20], y[3, 1, 40] = float("nan"), float("inf"), -float("inf")
    got = tll.rotary_forward(y, positions, r)
    touched = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    touched[1, 1, [3, 19]] = touched[2, 0, [4, 20]] = touched[3, 1, 40] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert got[1, 1, [3, 19]].isnan().all() and not got[2, 0, [4, 20]].isfinite().any() and got[3, 1, 40] == -float("inf")


def test_nothing_to_do():
    r = tll.Rotary(64)
    empty = torch.empty(0, 4, 64, device="cuda")
    assert tll.rotary_forward(empty, torch.empty(0, dtype=torch.int64, device="cuda"), r).shape == (0, 4, 64)


def test_graph_and_streams():
    x = matrix(300, 24, 64, 2304, torch.bfloat16)
    positions = torch.arange(300, device="cuda")
    r = tll.Rotary(64)
    want = tll.rotary_forward(x, positions, r)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tll.rotary_forward(x, positions, r, out=out)
    positions.add_(5)
    later = tll.rotary_forward(x, positions, r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, later) and not torch.equal(later, want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = tll.rotary_forward(x, positions, r, stream=other)
    other.synchronize()
    assert torch.equal(got, later)
