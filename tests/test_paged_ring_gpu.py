"""Attention on the tensor cores where one group of a block often has no keys of its own while the other has many: tiles
that the second group has no tokens of, or fewer keys (causal), before and behind full ones. Results against
serving_ref, and the same every time."""
import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_paged_attention_gpu import check, fill, queries
from test_paged_cache_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,held", [
    ([40, 100, 3], [2500, 1900, 3000]), ([65, 1, 129, 2], [1400, 2100, 700, 2600]), ([33] * 6, [1200 + 150 * i for i in range(6)])])
def test_groups_of_unequal_work(new, held, causal, D):
    H, Hkv = 16, 4  # 32 tokens a group
    cache, batch, starts, N = make(new, held, Hkv, D, 16, "heads")
    fill(cache, batch, held)
    q = queries(N, H, D)
    out, lse = tll.paged_attention(q, cache, batch, causal=causal, max_new=max(new), with_lse=True)
    tll.default_context(0).check()
    check(out, lse, q, cache, batch, starts, held, causal, D ** -0.5)
    got = [tll.paged_attention(q, cache, batch, causal=causal, max_new=max(new), with_lse=True) for _ in range(100)]
    tll.default_context(0).check()
    assert all(torch.equal(a, out) and torch.equal(b, lse) for a, b in got)
