"""Threads that call on the default stream at the same time, with one cache and items that are cut between blocks: every
result is the one that a thread alone gets, bit for bit."""
import threading

import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_paged_attention_gpu import fill, queries
from test_paged_cache_gpu import make

pytestmark = pytest.mark.gpu


def test_threads_on_the_default_stream():
    H, Hkv, D = 16, 2, 128
    new, held = [1] * 6, [900 + 90 * i for i in range(6)]
    cache, batch, starts, N = make(new, held, Hkv, D, 16, "heads")
    fill(cache, batch, held)
    # calls of one, three and six sequences, by either kernel
    calls = []
    for n, hint in ((1, 1), (3, 100), (6, 1), (6, 100)):
        part = tll.KVBatch(batch.q_start[:n + 1], batch.kv_len[:n], batch.block_table[:n])
        calls.append((queries(n, H, D, seed=n + hint), part, hint))
    want = [tll.paged_attention(q, cache, b, max_new=h, with_lse=True) for q, b, h in calls]
    tll.default_context(0).check()
    got, errors = [[] for _ in calls], []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            q, b, h = calls[i]
            start.wait()
            for _ in range(300):
                got[i].append(tll.paged_attention(q, cache, b, max_new=h, with_lse=True))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    tll.default_context(0).check()
    assert not errors
    for (out, lse), results in zip(want, got):
        assert len(results) == 300
        assert all(torch.equal(a, out) and torch.equal(b, lse) for a, b in results)
