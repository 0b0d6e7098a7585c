"""Refusals of the training and evaluation entries, at the C ABI and in the
binding, without a GPU: every check stands before the device is touched. The
context is a block of zeros (the checks read only plain values of it); a call
that passes them all reaches the device and returns LIN_ERR_CUDA."""
import ctypes

import pytest
import torch

import transformer_linear_layer_gb300 as tll

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would run")
BASE = 1 << 40  # addresses that are compared, never read


def at(n):
    return BASE + (n << 32)


@pytest.fixture()
def ctx():
    return ctypes.create_string_buffer(4096)


def attention(ctx, **k):
    a = dict(B=2, T=5, H=3, D=64, qkv=at(0), out=at(1), lse=at(2), dout=at(3), dqkv=at(4), causal=1, scale=0.0)
    a.update(k)
    return tll.library().lin_attention_backward(ctx, a["B"], a["T"], a["H"], a["D"], a["qkv"], a["out"], a["lse"],
                                                a["dout"], a["dqkv"], a["causal"], a["scale"], None)


def logprobs(ctx, **k):
    a = dict(R=3, V=100, z=at(0), ld=100, zt=tll.TYPE_BF16, tok=at(1), tt=tll.TYPE_INT64, tau=1.0, top=4, lp=at(2),
             ent=at(3), lse=at(4), tl=at(5), ti=at(6))
    a.update(k)
    return tll.library().lin_token_logprobs(ctx, a["R"], a["V"], a["z"], a["ld"], a["zt"], a["tok"], a["tt"], a["tau"],
                                            a["top"], a["lp"], a["ent"], a["lse"], a["tl"], a["ti"], None)


def distill(ctx, form, **k):
    a = dict(R=3, V=100, K=8, z=at(0), ld=100, zt=tll.TYPE_FP32, ids=at(1), it=tll.TYPE_INT32, t=at(2),
             tt=tll.TYPE_BF16, tau=2.0, loss=at(3), lse=at(4), w=at(5), dz=at(6), ldd=100)
    a.update(k)
    head = (ctx, a["R"], a["V"], a["K"], a["z"], a["ld"], a["zt"], a["ids"], a["it"], a["t"], a["tt"], a["tau"])
    lib = tll.library()
    if form == "forward":
        return lib.lin_distill_forward(*head, a["loss"], a["lse"], None)
    if form == "backward":
        return lib.lin_distill_backward(*head, a["lse"], a["w"], a["dz"], a["ldd"], None)
    return lib.lin_distill_forward_backward(*head, a["w"], a["loss"], a["dz"], a["ldd"], None)


@needs_no_gpu
def test_good_calls_pass_the_checks(ctx):
    assert attention(ctx) == tll.ERR_CUDA
    assert logprobs(ctx) == tll.ERR_CUDA
    for form in ("forward", "backward", "both"):
        assert distill(ctx, form) == tll.ERR_CUDA
    assert distill(ctx, "both", dz=at(0)) == tll.ERR_CUDA              # in place
    assert distill(ctx, "both", w=None, loss=None) == tll.ERR_CUDA
    assert distill(ctx, "forward", K=0, ids=None, t=None, lse=None) == tll.ERR_CUDA
    assert logprobs(ctx, tok=None, lp=None, ent=None, lse=None) == tll.ERR_CUDA
    assert logprobs(ctx, top=0, tl=None, ti=None) == tll.ERR_CUDA


def test_nothing_to_do(ctx):
    for k in ({"B": 0}, {"T": 0}, {"H": 0}):
        assert attention(ctx, **k) == tll.OK
    assert logprobs(ctx, R=0) == tll.OK
    assert logprobs(ctx, tok=None, lp=None, ent=None, lse=None, top=0) == tll.OK
    for form in ("forward", "backward", "both"):
        assert distill(ctx, form, R=0) == tll.OK


@pytest.mark.parametrize("bad", [{"B": -1}, {"T": -1}, {"H": -1}, {"D": -1}, {"causal": 2}, {"scale": -1.0},
                                 {"scale": float("nan")}, {"scale": float("inf")}, {"scale": 1e-39}, {"qkv": None},
                                 {"out": None}, {"lse": None}, {"dout": None}, {"dqkv": None}, {"dqkv": at(0)},
                                 {"dqkv": at(3) - 16}])
def test_attention_backward_arguments(ctx, bad):
    assert attention(ctx, **bad) == tll.ERR_ARG
    assert attention(None) == tll.ERR_ARG


def test_attention_backward_other_refusals(ctx):
    assert attention(ctx, D=128) == tll.ERR_UNSUPPORTED
    assert attention(ctx, B=1 << 20, T=1 << 20) == tll.ERR_UNSUPPORTED
    for name, n in (("qkv", 8), ("out", 8), ("dout", 4), ("dqkv", 2), ("lse", 2)):
        i = ["qkv", "out", "lse", "dout", "dqkv"].index(name)
        assert attention(ctx, **{name: at(i) + n}) == tll.ERR_ALIGN


@pytest.mark.parametrize("bad", [{"R": -1}, {"V": -1}, {"V": 0}, {"ld": 99}, {"zt": 2}, {"zt": 9}, {"tt": 0}, {"tau": 0.0},
                                 {"tau": -1.0}, {"tau": float("nan")}, {"tau": float("inf")}, {"tau": 1e-40}, {"z": None},
                                 {"tok": None}, {"lp": None}, {"top": -1}, {"top": 64, "V": 63, "ld": 63}, {"tl": None},
                                 {"ti": None}, {"lp": at(0)}, {"ent": at(2)}, {"ti": at(5) + 8}, {"lse": at(1)}])
def test_token_logprobs_arguments(ctx, bad):
    assert logprobs(ctx, **bad) == tll.ERR_ARG
    assert logprobs(None) == tll.ERR_ARG


def test_token_logprobs_other_refusals(ctx):
    assert logprobs(ctx, top=65) == tll.ERR_UNSUPPORTED
    assert logprobs(ctx, V=(1 << 30) + 1, ld=(1 << 30) + 1) == tll.ERR_UNSUPPORTED
    assert logprobs(ctx, R=(1 << 27) + 1) == tll.ERR_UNSUPPORTED
    for k in ({"z": at(0) + 1}, {"tok": at(1) + 4}, {"lp": at(2) + 2}, {"ti": at(6) + 1}):
        assert logprobs(ctx, **k) == tll.ERR_ALIGN


@pytest.mark.parametrize("form", ["forward", "backward", "both"])
@pytest.mark.parametrize("bad", [{"R": -1}, {"K": -1}, {"V": 0}, {"ld": 99}, {"zt": 3}, {"it": 1}, {"tt": 2}, {"tau": 0.0},
                                 {"z": None}, {"ids": None}, {"t": None}])
def test_distill_arguments(ctx, form, bad):
    assert distill(ctx, form, **bad) == tll.ERR_ARG
    assert distill(None, form) == tll.ERR_ARG


def test_distill_other_refusals(ctx):
    assert distill(ctx, "forward", loss=None) == tll.ERR_ARG
    assert distill(ctx, "backward", lse=None) == tll.ERR_ARG
    assert distill(ctx, "backward", w=None) == tll.ERR_ARG
    for form in ("backward", "both"):
        assert distill(ctx, form, dz=None) == tll.ERR_ARG
        assert distill(ctx, form, ldd=99) == tll.ERR_ARG
        assert distill(ctx, form, dz=at(0) + 4) == tll.ERR_ARG              # over the logits, not in place
        assert distill(ctx, form, dz=at(0), ldd=104) == tll.ERR_ARG         # nor with other rows
        assert distill(ctx, form, dz=at(6) + 2) == tll.ERR_ALIGN
        assert distill(ctx, form, K=257) == tll.ERR_UNSUPPORTED
    assert distill(ctx, "forward", loss=at(4)) == tll.ERR_ARG
    assert distill(ctx, "forward", ids=at(1) + 2) == tll.ERR_ALIGN


def test_the_binding_takes_gpu_tensors_only():
    z = torch.zeros(2, 10)
    ids = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        tll.token_logprobs(z)
    with pytest.raises(ValueError):
        tll.distill_forward(z, ids, torch.zeros(2, 3))
    with pytest.raises(ValueError):
        tll.attention_backward(torch.zeros(2, 192).bfloat16(), torch.zeros(2, 64).bfloat16(), torch.zeros(1, 1, 2),
                               torch.zeros(2, 64).bfloat16(), 1, 2, 1)


@pytest.mark.parametrize("scale", [1e-38, 1e-35, 7.8e-31, 1.3e30, 3e38])
def test_attention_backward_scales_that_fp32_statistics_cannot_carry(ctx, scale):
    """lse / scale and the score that stands for "sees no key" have to be finite."""
    assert attention(ctx, scale=scale) == tll.ERR_ARG


@needs_no_gpu
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 100])
def test_attention_backward_takes_scales_up_to_that(ctx, scale):
    assert attention(ctx, scale=scale) == tll.ERR_CUDA


@pytest.mark.parametrize("tau", [3e-39, 4.2e-39])
def test_temperatures_whose_base_2_factor_overflows(ctx, tau):
    """1 / tau is finite, log2(e) / tau is not."""
    assert logprobs(ctx, tau=tau) == tll.ERR_ARG
    for form in ("forward", "backward", "both"):
        assert distill(ctx, form, tau=tau) == tll.ERR_ARG
