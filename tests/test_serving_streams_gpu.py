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
