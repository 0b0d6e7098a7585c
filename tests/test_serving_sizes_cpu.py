"""Sizes past what the serving kernels' 32-bit arithmetic holds are refused, at the C ABI (with test_serving_abi_cpu's
stand-ins) and in the binding (with stand-ins of tensors: the real ones would fill the GPU)."""
import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_serving_abi_cpu import append, attention, at, batch, cache, ctx, needs_no_gpu, rotary  # noqa: F401


def wide(n):
    """A batch of n tokens whose rows overlap nothing: operands 2^45 bytes apart."""
    return dict(b=batch(tokens=n), q=at(0) + (1 << 45), out=at(0) + (1 << 46), lse=None)


@needs_no_gpu
def test_the_most_tokens(ctx):  # noqa: F811
    for max_new in (1, 1000):
        assert attention(ctx, max_new=max_new, **wide(1 << 28)) == tll.ERR_CUDA  # past the checks
        assert attention(ctx, max_new=max_new, **wide((1 << 28) + 1)) == tll.ERR_UNSUPPORTED
        assert attention(ctx, max_new=max_new, **wide((1 << 31) - 1)) == tll.ERR_UNSUPPORTED


def test_the_most_sequences(ctx):  # noqa: F811
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        assert append(ctx, b=batch(sequences=n)) == tll.ERR_UNSUPPORTED
        assert attention(ctx, b=batch(sequences=n)) == tll.ERR_UNSUPPORTED
    assert attention(ctx, b=batch(sequences=(1 << 24) + 1)) == tll.ERR_UNSUPPORTED


class Huge:
    """What the binding asks of a CUDA tensor, without its memory."""

    is_cuda = True

    def __init__(self, shape, dtype, strides=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda:0")
        strides = strides or [1] * len(shape)
        for i in range(len(shape) - 2, -1, -1):
            strides[i] = strides[i + 1] * shape[i + 1]
        self.strides = tuple(strides)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 40


def test_the_binding_counts_in_32_bits():
    big, bf16, i32 = 2 ** 32 + 5, torch.bfloat16, torch.int32
    for shape in ((big, 1, 64), (2, big, 64), (1, 1, big)):
        with pytest.raises(ValueError):
            tll._check_heads(Huge(shape, bf16), bf16, "x")
    assert tll._check_heads(Huge((2 ** 31 - 1, 1, 64), bf16), bf16, "x") == (2 ** 31 - 1, 1, 64, 64)
    with pytest.raises(ValueError):
        tll.KVCache(Huge((big, 1, 8, 64), bf16), Huge((big, 1, 8, 64), bf16))
    with pytest.raises(ValueError):
        tll.KVBatch(Huge((2,), i32), Huge((1,), i32), Huge((1, big), i32))
    with pytest.raises(ValueError):
        tll.KVBatch(Huge((big + 1,), i32), Huge((big,), i32), Huge((big, 1), i32))
    assert tll.KVBatch(Huge((2,), i32), Huge((1,), i32), Huge((1, 9), i32)).sequences == 1


@needs_no_gpu
def test_the_widest_rows(ctx):  # noqa: F811
    far = dict(y=at(0) + (1 << 45), N=2, D=1024)
    most, less = 1 << 17, (1 << 17) + 1
    for form in ("forward", "backward"):
        assert rotary(ctx, form, H=most, ldx=1 << 30, ldy=1 << 30, **far) == tll.ERR_CUDA  # past the checks
        assert rotary(ctx, form, H=less, ldx=1 << 30, ldy=1 << 30, **far) == tll.ERR_UNSUPPORTED
        assert rotary(ctx, form, H=3, ldx=(1 << 30) + 1, ldy=1 << 30, **far) == tll.ERR_UNSUPPORTED
    many = cache(heads=512, ps=512 * 16 * 64)
    assert attention(ctx, c=many, H=65536, ldq=1 << 22, ldo=1 << 22) == tll.ERR_UNSUPPORTED
    assert append(ctx, H=(1 << 21) + 1, ldq=1 << 28, ldqo=1 << 28, c=many, ldk=1 << 15, ldv=1 << 15) == tll.ERR_UNSUPPORTED
