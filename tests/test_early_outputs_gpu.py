"""Early start at level 2: an input that a call before the previous one writes is not
read early, although it lies outside the previous call's output (that older call may
still run, since its successor lets others start before its own wait). Seen in the
plan: a call that reads early narrows its split, one that does not keeps the table's."""
import pytest
import torch

import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu
N = 4096


@pytest.fixture()
def setup():
    s = torch.cuda.Stream()
    ctx = tll.Context(0)
    ctx.set_option(tll.OPT_EARLY_START, tll.EARLY_ALL)
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(N, N, device="cuda", generator=g).bfloat16() * 0.02
    x = [torch.randn(16, N, device="cuda", generator=g).bfloat16() for _ in range(3)]
    y = [torch.zeros(16, N, device="cuda", dtype=torch.bfloat16) for _ in range(80)]
    torch.cuda.synchronize()

    def call(a, out):
        with torch.cuda.stream(s):
            tll.forward(a, w, precision="bf16", out=out, ctx=ctx)
        return ctx.last_plan().splits

    with torch.cuda.stream(s):
        tll.token_logprobs(w[:1].float(), ctx=ctx)  # (a stream of torch's pool may have had calls)
    isolated = tll.plan_query(ctx.sm_count, 16, N, N, "bf16").splits
    call(x[0], y[0])
    early = call(x[1], y[1])
    assert early < isolated, "the shape does not tell an early read"
    yield call, x, y, isolated, early, s, ctx, w
    torch.cuda.synchronize()
    ctx.check()


def plain(a, w):
    return a.float() @ w.float().T


@pytest.mark.parametrize("between", [0, 1, 5])
def test_an_older_calls_output_is_not_read_early(setup, between):
    call, x, y, isolated, early, s, ctx, w = setup
    call(x[2], y[2])
    for k in range(between):
        assert call(x[k % 2], y[3 + k]) == early
    assert call(y[2], y[20]) == isolated
    assert call(x[0], y[21]) == early  # and the calls after it are early again
    torch.cuda.synchronize()
    want = plain(plain(x[2], w).bfloat16(), w)
    assert float((y[20].float() - want).norm() / want.norm()) < 1e-2


def test_a_list_that_overflows_loses_no_output(setup):
    call, x, y, isolated, early, s, ctx, w = setup
    call(x[2], y[2])
    for k in range(3, 79):
        call(x[k % 2], y[k])
    call(y[2], y[79])
    torch.cuda.synchronize()
    want = plain(plain(x[2], w).bfloat16(), w)
    assert float((y[79].float() - want).norm() / want.norm()) < 1e-2


def test_after_a_call_that_orders_older_outputs_are_done(setup):
    call, x, y, isolated, early, s, ctx, w = setup
    call(x[2], y[2])
    z = torch.randn(4, 1000, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for op in (lambda: tll.token_logprobs(z, top=3, ctx=ctx), lambda: tll.distill_forward(z, ids, z[:, :2].contiguous(), ctx=ctx),
               lambda: tll.distill_forward_backward(z, ids, z[:, :2].contiguous(), ctx=ctx)):
        call(x[2], y[2])
        with torch.cuda.stream(s):
            op()
        assert call(y[2], y[22]) == early
    torch.cuda.synchronize()
    want = plain(plain(x[2], w).bfloat16(), w)
    assert float((y[22].float() - want).norm() / want.norm()) < 1e-2


def test_level_1_and_the_default_keep_their_plans(setup):
    call, x, y, isolated, early, s, ctx, w = setup
    for level in (tll.EARLY_WEIGHTS, tll.EARLY_NONE):
        ctx.set_option(tll.OPT_EARLY_START, level)
        call(x[2], y[2])
        call(x[0], y[3])
        assert call(y[2], y[4]) == isolated
        assert call(x[1], y[5]) == isolated
