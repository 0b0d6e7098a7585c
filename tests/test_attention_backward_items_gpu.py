"""lin_attention_backward where its blocks take several work items each: more items
than SMs, causal and full, with several chains of dq sums and with one, against the
float64 formulas (on the GPU, a head at a time; the bound per output is
training_ref.attention_backward's); and where another stream's kernel keeps some of
the blocks from running."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

import training_ref as ref
import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def inputs(B, T, H, causal, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    C = 64 * H
    qkv = torch.randn(B * T, 3 * C, generator=g, device="cuda")
    qkv[:, :2 * C] *= 1.2
    qkv = qkv.bfloat16()
    dout = (torch.randn(B * T, C, generator=g, device="cuda") * 0.1).bfloat16()
    out, lse = tll.attention_forward(qkv, B, T, H, causal=causal, with_lse=True)
    return qkv, out, lse, dout


def check(got, qkv, out, lse, dout, B, T, H, causal, scale=0.125):
    C = 64 * H
    half, single = ref.BF16_HALF, ref.FP32_HALF
    seen = torch.ones(T, T, dtype=torch.bool, device="cuda").tril_() if causal else None
    for b in range(B):
        rows = slice(b * T, (b + 1) * T)
        for h in range(H):
            at = [slice(n * C + 64 * h, n * C + 64 * h + 64) for n in range(3)]
            q, k, v = (qkv[rows, c].double() for c in at)
            o, do = out[rows, at[0]].double(), dout[rows, at[0]].double()
            p = torch.exp(q @ k.T * scale - lse[b, h].double()[:, None])
            if causal:
                p = torch.where(seen, p, 0.0)
            dp = do @ v.T - (do * o).sum(1, keepdim=True)
            ds = p * dp
            want = [scale * ds @ k, scale * ds.T @ q, p.T @ do]
            size = q.abs().max() * k.abs().max() * 64 * scale + lse[b, h].abs().max().double()
            rel = 16 * single * (size + 8)
            parts = do.abs() @ v.abs().T + (o.abs() * do.abs()).sum(1, keepdim=True)
            eds = half * ds.abs() + p * (rel * dp.abs() + 32 * single * parts) + 64 * single * ds.abs()
            ep = p * (half + rel + 64 * single)
            errs = [scale * eds @ k.abs(), scale * eds.T @ q.abs(), ep.T @ do.abs()]
            for name, c, w, e in zip(("dq", "dk", "dv"), at, want, errs):
                bound = 1.02 * (e + half * (w.abs() + e)) + 1e-30
                off = (got[rows, c].double() - w).abs() / bound
                assert bool((off <= 1).all()), (name, b, h, int(off.argmax()) // 64, float(off.max()))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,T,H,workspace", [
    (8, 520, 12, 0),            # 480 items, two chains a head
    (8, 520, 12, 18 << 20),     # the same items, one chain
    (8, 520, 12, 9 << 20),      # two launches and a rest
    (1, 4153, 6, 0),            # 198 items of up to 33 steps
    (40, 200, 16, 0),           # 1280 items of one and two steps
    (20, 129, 16, 0)])          # 640, a block of one token among each two
def test_blocks_take_several_items(B, T, H, workspace, causal):
    ctx = tll.Context(0, workspace) if workspace else tll.default_context(0)
    x = inputs(B, T, H, causal)
    got = tll.attention_backward(*x, B, T, H, causal=causal, ctx=ctx)
    ctx.check()
    check(got, *x, B, T, H, causal)
    for _ in range(3):
        assert torch.equal(tll.attention_backward(*x, B, T, H, causal=causal, ctx=ctx), got)
    ctx.check()


@pytest.fixture(scope="module")
def hold(tmp_path_factory):
    """hold(blocks, ns, stream): blocks that each keep an SM's shared memory for ns."""
    so = str(tmp_path_factory.mktemp("hold") / "libhold.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-Xcompiler", "-fPIC", "-o", so,
                    os.path.join(HERE, "hold_sms.cu")], check=True)
    lib = ctypes.CDLL(so)
    lib.hold_sms.argtypes = [ctypes.c_int, ctypes.c_ulonglong, ctypes.c_void_p]
    return lambda blocks, ns, stream: lib.hold_sms(blocks, ns, stream.cuda_stream)


@pytest.mark.parametrize("left", [-1, 40, 3])
@pytest.mark.parametrize("B,T,H,causal", [(1, 1500, 20, True), (2, 700, 16, False)])
def test_blocks_that_cannot_run_hold_up_no_other(hold, B, T, H, causal, left):
    """Another stream's kernel keeps all SMs but `left` (or one SM) for 1.5 s: the call
    is right, and done before that kernel, on the SMs that it leaves."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctx = tll.Context(0, 24 << 20)  # one or two chains, so that items wait for items
    x = inputs(B, T, H, causal)
    want = tll.attention_backward(*x, B, T, H, causal=causal, ctx=ctx)
    check(want, *x, B, T, H, causal)
    got = torch.empty_like(want)
    other, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    assert hold(1 if left < 0 else sms - left, 1_500_000_000, other) == 0
    done.record(other)
    time.sleep(0.05)  # its blocks are in place
    tll.attention_backward(*x, B, T, H, causal=causal, dqkv=got, ctx=ctx)
    torch.cuda.current_stream().synchronize()
    assert not done.query(), "the SMs were not held throughout"
    torch.cuda.synchronize()
    ctx.check()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [100, 300])
@pytest.mark.parametrize("scale", [2.0 ** -98, 2.0 ** -100])
def test_queries_that_see_no_key_at_tiny_scales(T, scale):
    """lse = -inf takes no part in dv at a scale where the scores hardly differ."""
    B, H, C = 2, 2, 128
    qkv, out, lse, dout = inputs(B, T, H, False)
    out, lse = tll.attention_forward(qkv, B, T, H, causal=False, scale=scale, with_lse=True)
    lse[:, :, ::3] = -torch.inf
    got = tll.attention_backward(qkv, out, lse, dout, B, T, H, causal=False, scale=scale)
    tll.default_context(0).check()
    assert bool(got.isfinite().all())
    p = torch.exp(-lse.double())
    p[:, :, ::3] = 0
    do = dout.double().view(B, T, H, 64).transpose(1, 2)
    want = torch.einsum("bhi,bhid->bhd", p, do)  # every key's dv
    bound = torch.einsum("bhi,bhid->bhd", p * (ref.BF16_HALF + 2.0 ** -16), do.abs())
    bound = 1.02 * (bound + ref.BF16_HALF * (want.abs() + bound)) + 1e-30
    dv = got[:, 2 * C:].double().view(B, T, H, 64).transpose(1, 2)
    assert bool(((dv - want[:, :, None]).abs() <= bound[:, :, None]).all())


@pytest.mark.parametrize("T", [100, 300])
def test_the_output_of_a_query_that_sees_no_key_does_not_matter(T):
    """lse = -inf: its out may be 0 / 0, and reaches no gradient."""
    qkv, out, lse, dout = inputs(2, T, 2, False)
    lse[:, :, ::3] = -torch.inf
    want = tll.attention_backward(qkv, out, lse, dout, 2, T, 2, causal=False)
    out.view(2, T, 128)[:, ::3] = float("nan")
    got = tll.attention_backward(qkv, out, lse, dout, 2, T, 2, causal=False)
    tll.default_context(0).check()
    assert bool(got.isfinite().all()) and torch.equal(got, want)
