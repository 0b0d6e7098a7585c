"""Which stream the memory of a call with ``stream=`` belongs to: the one that its kernels run on. torch hands a freed
block out again at once on the stream that it was taken on, with what still runs there."""
import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_paged_attention_gpu import fill, queries
from test_paged_cache_gpu import make

pytestmark = pytest.mark.gpu


def setup(H=4, Hkv=2, D=64):
    cache, batch, starts, N = make([1, 2], [300, 200], Hkv, D, 16, "heads")
    fill(cache, batch, [300, 200])
    return cache, batch, queries(N, H, D), N


def test_the_default_streams_handle_names_the_default_stream(monkeypatch):
    """A call on stream 0 from within another stream: its workspace comes from the default stream's memory."""
    cache, batch, q, N = setup()
    want = tll.paged_attention(q, cache, batch)
    taken, scratch = [], tll._scratch
    monkeypatch.setattr(tll, "_scratch", lambda *a: taken.append(scratch(*a)) or taken[-1])
    size = tll.paged_attention_workspace(cache, batch, N, 4)
    torch.cuda.synchronize()
    mine = torch.empty(size, dtype=torch.uint8, device="cuda")
    place = mine.data_ptr()
    del mine
    side = torch.cuda.Stream()
    for zero in (0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream):
        taken.clear()
        with torch.cuda.stream(side):
            out = tll.paged_attention(q, cache, batch, stream=zero)
        torch.cuda.synchronize()
        assert [t.data_ptr() for t in taken] == [place]
        assert torch.equal(out, want)


def calls():
    """name, call(stream) with a result (or several) of its own."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, 256, generator=g).bfloat16().cuda()
    w = torch.randn(256, 256, generator=g).bfloat16().cuda()
    w32, gamma = w.float(), torch.ones(256, device="cuda")
    qkv = torch.randn(2 * 70, 3 * 128, generator=g).bfloat16().cuda()
    a, lse = tll.attention_forward(qkv, 2, 70, 2, with_lse=True)
    z = torch.randn(5, 1000, generator=g).cuda()
    ids = torch.zeros(5, 2, dtype=torch.int64, device="cuda")
    teacher, tokens = z[:, :2].contiguous(), ids[:, 0].contiguous()
    loss, zl = tll.distill_forward(z, ids, teacher)
    cache, batch, q, N = setup()
    r, positions = tll.Rotary(64), torch.arange(N, device="cuda")
    k = torch.randn(N, 2, 64, generator=g).bfloat16().cuda()
    return {
        "forward": lambda s: tll.forward(x, w, stream=s),
        "forward_plan": lambda s: tll.forward_plan(tll.plan_query(152, 64, 256, 256), x, w, stream=s),
        "forward_residual": lambda s: tll.forward_residual(x, w, x, stream=s),
        "fold_layernorm": lambda s: tll.fold_layernorm(w32, gamma, stream=s),
        "backward_data": lambda s: tll.backward_data(x, w, stream=s),
        "backward_data_gelu": lambda s: tll.backward_data_gelu(x, w, x, stream=s),
        "backward_weight": lambda s: tll.backward_weight(x, x, db=True, stream=s),
        "gelu_backward": lambda s: tll.gelu_backward(x, x, stream=s),
        "attention_forward": lambda s: tll.attention_forward(qkv, 2, 70, 2, with_lse=True, stream=s),
        "attention_backward": lambda s: tll.attention_backward(qkv, a, lse, a, 2, 70, 2, stream=s),
        "token_logprobs": lambda s: tll.token_logprobs(z, tokens, top=3, stream=s),
        "distill_forward": lambda s: tll.distill_forward(z, ids, teacher, stream=s),
        "distill_backward": lambda s: tll.distill_backward(z, ids, teacher, zl, loss, stream=s),
        "distill_forward_backward": lambda s: tll.distill_forward_backward(z, ids, teacher, stream=s),
        "rotary_forward": lambda s: tll.rotary_forward(q, positions, r, stream=s),
        "rotary_backward": lambda s: tll.rotary_backward(q, positions, r, stream=s),
        "cache_append": lambda s: tll.cache_append(q, k, k, cache, batch, rotary=r, stream=s),
        "paged_attention": lambda s: tll.paged_attention(q, cache, batch, with_lse=True, stream=s),
    }


def tensors(result):
    return [t for t in (result if isinstance(result, tuple) else (result,)) if t is not None]


@pytest.mark.parametrize("name", sorted([
    "forward", "forward_plan", "forward_residual", "fold_layernorm", "backward_data", "backward_data_gelu", "backward_weight",
    "gelu_backward", "attention_forward", "attention_backward", "token_logprobs", "distill_forward", "distill_backward",
    "distill_forward_backward", "rotary_forward", "rotary_backward", "cache_append", "paged_attention"]))
def test_results_are_memory_of_the_calls_stream(name):
    call = calls()[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    # blocks that the current stream has freed, and may still be using, are not written by another
    freed = [torch.empty_like(t) for t in want for _ in range(4)]
    places = {t.data_ptr() for t in freed}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del freed
    for s in (side, side.cuda_stream):
        got = tensors(call(s))
        assert not places & {t.data_ptr() for t in got}
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and a result that the current stream is still at work with when it is let go is not written either
    held = {t.data_ptr() for t in got}
    torch.cuda._sleep(200_000_000)
    del got
    again = tensors(call(side))
    assert not held & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_the_legacy_streams_handle_is_the_default_stream():
    cache, batch, q, N = setup()
    want = tll.paged_attention(q, cache, batch)
    torch.cuda.synchronize()
    assert tll._torch_stream(1, q.device) == torch.cuda.default_stream()
    out = tll.paged_attention(q, cache, batch, stream=1)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("name", ["forward", "rotary_forward", "cache_append", "paged_attention"])
def test_calls_on_a_given_stream_in_a_capture(name):
    """On the captured stream itself, and on one that is forked from it and joined: the results are the graph's memory."""
    call = calls()[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    s, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        first = tensors(call(s))
        side.wait_stream(s)
        second = tensors(call(side))
        s.wait_stream(side)
    for t in first + second:
        t.fill_(0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in (first, second):
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
