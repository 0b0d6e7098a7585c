"""GPU parity of lin_attention_backward against the float64 formulas. The bound
per output counts the roundings of the kernel's arithmetic (training_ref.
attention_backward): p and ds to bf16 (2^-8 each) before the products that take
them, the output to bf16, and fp32 for everything else."""
import numpy as np
import pytest
import torch

import training_ref as ref
import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu


def inputs(B, T, H, causal, scale=None, sharp=1.2, seed=0, ctx=None):
    g = torch.Generator().manual_seed(seed)
    C = 64 * H
    qkv = torch.randn(B * T, 3 * C, generator=g)
    qkv[:, :2 * C] *= sharp
    qkv = qkv.bfloat16().cuda()
    dout = (torch.randn(B * T, C, generator=g) * 0.1).bfloat16().cuda()
    out, lse = tll.attention_forward(qkv, B, T, H, causal=causal, scale=scale, with_lse=True, ctx=ctx)
    return qkv, out, lse, dout


def host(t):
    return t.double().cpu().numpy()


def check(B, T, H, causal, scale=None, ctx=None, **k):
    qkv, out, lse, dout = inputs(B, T, H, causal, scale, ctx=ctx, **k)
    got = tll.attention_backward(qkv, out, lse, dout, B, T, H, causal=causal, scale=scale, ctx=ctx)
    (ctx or tll.default_context(0)).check()
    want, bound = ref.attention_backward(host(qkv), host(out), host(lse), host(dout), B, T, H, causal,
                                         0.125 if scale is None else scale, bounds=True)
    err = np.abs(host(got) - want)
    worst = np.unravel_index(np.argmax(err / bound), err.shape)
    assert np.all(err <= bound), (worst, host(got)[worst], want[worst], bound[worst])
    return got


# one block, ragged blocks, one token, several key blocks, several chains of partial sums
CASES = [(1, 1, 1, True), (3, 1, 2, False), (2, 5, 2, True), (4, 77, 3, True), (2, 127, 2, False), (1, 128, 3, True),
         (1, 128, 1, False), (2, 129, 2, True), (2, 200, 2, False), (1, 256, 2, True), (1, 257, 3, False),
         (2, 300, 3, True), (1, 700, 2, False), (1, 1153, 1, True)]


@pytest.mark.parametrize("B,T,H,causal", CASES)
def test_matches_the_formulas(B, T, H, causal):
    check(B, T, H, causal)


@pytest.mark.parametrize("T", [96, 300])
def test_scale_and_peaked_rows(T):
    check(2, T, 2, True, scale=0.31, sharp=2.5)
    check(1, T, 2, False, scale=0.02, sharp=0.3)


def test_gpt2_batch():
    check(4, 128, 12, True, seed=5)


@pytest.mark.parametrize("T,workspace", [(300, 1 << 20), (700, 1 << 20), (400, 5 << 18)])
def test_small_workspaces_take_several_launches(T, workspace):
    """Fewer heads a launch and one chain of sums: the same bound holds."""
    ctx = tll.Context(0, workspace)
    check(2, T, 3, True, ctx=ctx)
    check(1, T, 3, False, ctx=ctx)


def test_refuses_a_workspace_without_room_for_one_head():
    ctx = tll.Context(0, 256 << 10)
    qkv, out, lse, dout = inputs(1, 1024, 1, True)
    with pytest.raises(tll.LinError) as e:
        tll.attention_backward(qkv, out, lse, dout, 1, 1024, 1, ctx=ctx)
    assert e.value.status == tll.ERR_WORKSPACE
    check(1, 100, 2, True, ctx=ctx)  # one block needs none


@pytest.mark.parametrize("B,T,H,causal", [(8, 128, 4, True), (2, 640, 6, True), (1, 900, 5, False)])
def test_repeats_bit_for_bit(B, T, H, causal):
    qkv, out, lse, dout = inputs(B, T, H, causal)
    first = tll.attention_backward(qkv, out, lse, dout, B, T, H, causal=causal)
    for _ in range(4):
        assert torch.equal(tll.attention_backward(qkv, out, lse, dout, B, T, H, causal=causal), first)


@pytest.mark.parametrize("T", [100, 200])
def test_queries_that_see_no_key(T):
    """lse = -inf: the query takes part in no gradient, and its own is zero."""
    qkv, out, lse, dout = inputs(2, T, 2, False)
    lse[:, :, ::3] = -torch.inf
    got = host(tll.attention_backward(qkv, out, lse, dout, 2, T, 2, causal=False))
    want, bound = ref.attention_backward(host(qkv), host(out), host(lse), host(dout), 2, T, 2, False, 0.125, bounds=True)
    assert np.all(np.abs(got - want) <= bound)
    assert np.all(got.reshape(2, T, 384)[:, ::3, :128] == 0)


@pytest.mark.parametrize("T", [70, 130])
def test_sequences_do_not_touch(T):
    """A block that reaches past its sequence's end takes nothing from the next."""
    qkv, out, lse, dout = inputs(3, T, 2, True)
    want = tll.attention_backward(qkv, out, lse, dout, 3, T, 2)
    for t in (qkv, out, dout):
        t.view(3, T, -1)[1] = float("nan")
    lse[1] = float("nan")
    got = tll.attention_backward(qkv, out, lse, dout, 3, T, 2)
    for b in (0, 2):
        assert torch.equal(got.view(3, T, -1)[b], want.view(3, T, -1)[b])
    assert got.view(3, T, -1)[1].isnan().any()


@pytest.mark.parametrize("T", [100, 200])
def test_future_gradients_do_not_reach_earlier_queries(T):
    """Causal: inf in a later query's dout leaves the earlier queries' dq alone."""
    qkv, out, lse, dout = inputs(1, T, 1, True)
    want = tll.attention_backward(qkv, out, lse, dout, 1, T, 1)
    dout[T - 1] = float("inf")
    got = tll.attention_backward(qkv, out, lse, dout, 1, T, 1)
    assert torch.equal(got[:T - 1, :64], want[:T - 1, :64])


@pytest.mark.parametrize("B,T,H", [(2, 100, 3), (1, 400, 2)])
def test_in_a_graph_and_on_another_stream(B, T, H):
    qkv, out, lse, dout = inputs(B, T, H, True)
    want = tll.attention_backward(qkv, out, lse, dout, B, T, H)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ctx = tll.Context(0)
    got = torch.empty_like(qkv)
    with torch.cuda.stream(s):
        tll.attention_backward(qkv, out, lse, dout, B, T, H, dqkv=got, ctx=ctx)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tll.attention_backward(qkv, out, lse, dout, B, T, H, dqkv=got, ctx=ctx)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    ctx.check()


def test_next_to_other_calls_of_the_library():
    """The workspace's counters and sums are left as other calls need them."""
    torch.manual_seed(0)
    x, w = torch.randn(128, 768, device="cuda"), torch.randn(768, 768, device="cuda")
    ctx = tll.Context(0)
    y = tll.forward(x, w, precision="fp32", ctx=ctx)
    qkv, out, lse, dout = inputs(2, 500, 4, True)
    want = tll.attention_backward(qkv, out, lse, dout, 2, 500, 4, ctx=ctx)
    for _ in range(3):
        assert torch.equal(tll.forward(x, w, precision="fp32", ctx=ctx), y)
        assert torch.equal(tll.attention_backward(qkv, out, lse, dout, 2, 500, 4, ctx=ctx), want)
    ctx.check()


def test_binding_refusals():
    qkv, out, lse, dout = inputs(1, 8, 2, True)
    with pytest.raises(ValueError):
        tll.attention_backward(qkv, out, lse, dout, 1, 8, 3)
    with pytest.raises(ValueError):
        tll.attention_backward(qkv.float(), out, lse, dout, 1, 8, 2)
    with pytest.raises(ValueError):
        tll.attention_backward(qkv, out, lse.double(), dout, 1, 8, 2)
    with pytest.raises(tll.LinError) as e:
        tll.attention_backward(qkv, out, lse, dout, 1, 8, 2, dqkv=qkv)
    assert e.value.status == tll.ERR_ARG
