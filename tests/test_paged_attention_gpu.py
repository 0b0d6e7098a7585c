"""Attention of new tokens over a paged cache against serving_ref (float64).

Bound of an output: probabilities are rounded to bf16 for the product with V (half a step,
2^-8, of sum_j p_ij |v_j|) and the output once (2^-8 of its value); scores, exponentials and
sums in fp32 add less than 5 % of that at these sizes, and 1e-5. lse: fp32 scores of at
most 128 products and the hardware's exponentials and logarithm, 1e-4 of 1 + |lse|."""
import ctypes

import numpy as np
import pytest
import torch

import serving_ref as ref
import transformer_linear_layer_gb300 as tll
from test_paged_cache_gpu import host, make

pytestmark = pytest.mark.gpu
NAN = float("nan")


def fill(cache, batch, held, seed=3, spread=1.0):
    """Keys and values in the held slots; the others stay NaN."""
    g = torch.Generator().manual_seed(seed)
    table = batch.block_table.cpu()
    for b, n in enumerate(held):
        n = min(n, table.shape[1] * cache.page_size)
        for i in range(0, max(n, 0), cache.page_size):
            k = min(cache.page_size, n - i)
            for c in (cache.k, cache.v):
                x = torch.randn(cache.heads, k, cache.head_dim, generator=g)
                c[table[b, i // cache.page_size], :, :k] = (x * spread).bfloat16().cuda()


def queries(N, H, D, seed=4, spread=1.5, ld=None):
    g = torch.Generator().manual_seed(seed)
    q = (spread * torch.randn(N, H, D, generator=g)).bfloat16().cuda()
    if ld is None:
        return q
    buf = torch.full((N, ld), NAN, dtype=torch.bfloat16, device="cuda")
    buf[:, :H * D] = q.reshape(N, -1)
    return buf[:, :H * D].unflatten(1, (H, D))


def check(got, lse, q, cache, batch, starts, held, causal, scale):
    want, wl, size = ref.attention(host(q), host(cache.k), host(cache.v), starts, held,
                                   batch.block_table.cpu().numpy(), cache.page_size, causal, scale)
    live = ~np.isnan(want)
    tol = 1.05 * 2.0 ** -8 * (size + np.abs(want)) + 1e-5
    err = np.abs(host(got) - want)
    assert np.isfinite(host(got)[live]).all()
    assert np.all(err[live] <= tol[live]), (err[live].max(), (err / tol)[live].max())
    if lse is not None:
        rows = ~np.isnan(wl)
        a, b = host(lse)[rows], wl[rows]
        assert np.array_equal(np.isinf(a), np.isinf(b))
        fin = np.isfinite(b)
        assert np.all(np.abs(a[fin] - b[fin]) <= 1e-4 * (1 + np.abs(b[fin])))


CASES = [
    # new, held, H, Hkv, D, page
    ([1], [1], 1, 1, 64, 8), ([1], [1000], 12, 12, 64, 16), ([1], [777], 8, 2, 128, 64),
    ([1] * 5, [1, 15, 16, 17, 300], 4, 4, 64, 16), ([1] * 70, [(37 * i) % 500 + 1 for i in range(70)], 6, 2, 64, 32),
    ([1, 0, 4, 2], [9, 0, 100, 2], 15, 5, 64, 8), ([3], [3], 4, 1, 128, 128), ([1], [5000], 16, 1, 128, 256),
    ([16], [130], 2, 2, 64, 16), ([7, 33], [64, 33], 10, 2, 64, 16), ([1, 65, 1, 130], [70, 65, 1, 400], 8, 4, 128, 16),
    ([200], [200], 3, 3, 64, 32), ([129, 5], [1000, 5], 5, 1, 128, 64), ([1], [64], 32, 1, 64, 8),
    ([2, 1], [65, 128], 32, 1, 128, 16), ([300], [301], 7, 1, 64, 16), ([257], [700], 4, 2, 128, 8),
    ([1] * 3, [2000, 3, 1], 2, 1, 64, 4096), ([1, 3], [70, 400], 128, 1, 128, 16), ([2], [300], 96, 2, 64, 32),
    ([500, 3, 256], [1500, 3, 256], 2, 1, 128, 32), ([255, 1], [300, 4000], 6, 2, 64, 16),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,held,H,Hkv,D,page", CASES)
def test_parity(new, held, H, Hkv, D, page, causal):
    order = ("heads", "tokens", "pairs")[(len(new) + H + page) % 3]
    cache, batch, starts, N = make(new, held, Hkv, D, page, order)
    fill(cache, batch, held)
    q = queries(N, H, D)
    for max_new in (None, max(new), 1, 10 ** 6):
        out, lse = tll.paged_attention(q, cache, batch, causal=causal, max_new=max_new, with_lse=True)
        tll.default_context(0).check()
        check(out, lse, q, cache, batch, starts, held, causal, D ** -0.5)
    for _ in range(5):
        again = tll.paged_attention(q, cache, batch, causal=causal, max_new=max_new)
        assert torch.equal(again, out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_new", [1, 10 ** 6])
def test_rows_that_see_nothing(D, max_new):
    """Sequences that hold nothing, fewer keys than new tokens, or a length below zero."""
    new, held = [3, 5, 2, 1, 40], [0, 2, -7, 9, 20]
    cache, batch, starts, N = make(new, held, 2, D, 8, "heads")
    fill(cache, batch, held)
    q = queries(N, 4, D)
    out, lse = tll.paged_attention(q, cache, batch, max_new=max_new, with_lse=True)
    check(out, lse, q, cache, batch, starts, held, True, D ** -0.5)
    assert (out[:6] == 0).all() and (lse[:6] == -float("inf")).all() and (out[8:10] == 0).all()
    out, lse = tll.paged_attention(q, cache, batch, causal=False, max_new=max_new, with_lse=True)
    check(out, lse, q, cache, batch, starts, held, False, D ** -0.5)


@pytest.mark.parametrize("max_new", [1, 10 ** 6])
def test_rows_of_no_sequence_and_pages_that_are_none(max_new):
    H, Hkv, D, page = 4, 2, 64, 16
    cache, batch, _, _ = make([4, 6, 1], [40, 20, 70], Hkv, D, page, "heads")
    fill(cache, batch, [40, 20, 70])
    starts = [2, 6, 12, 13]
    batch.q_start.copy_(torch.tensor(starts))
    batch.block_table[0, 1], batch.block_table[2, 3] = cache.pages, -(2 ** 31)
    N = 16
    q = queries(N, H, D)
    out = torch.full((N, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, H), 5.0, device="cuda")
    tll.paged_attention(q, cache, batch, out=out, lse=lse, max_new=max_new)
    check(out, lse, q, cache, batch, starts, [40, 20, 70], True, D ** -0.5)
    for x in (out, lse):
        assert (x[:2] == 5).all() and (x[13:] == 5).all()
    # longer than the table: what the table holds; not ascending: nothing out of range
    batch.kv_len.fill_(2 ** 31 - 1)
    tll.paged_attention(q, cache, batch, causal=False, out=out, max_new=max_new)
    batch.q_start.copy_(torch.tensor([7, 3, 19, 1]))
    tll.paged_attention(q, cache, batch, out=out, max_new=max_new)
    torch.cuda.synchronize()


@pytest.mark.parametrize("max_new", [1, 10 ** 6])
def test_strides_scale_and_odd_values(max_new):
    H, Hkv, D, page = 6, 3, 64, 32
    new, held = [2, 1, 40], [100, 64, 90]
    cache, batch, starts, N = make(new, held, Hkv, D, page, "tokens")
    fill(cache, batch, held)
    q = queries(N, H, D, ld=H * D + 24)
    out = torch.full((N, H * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, :H * D].unflatten(1, (H, D))
    for scale in (2.0, 1e-3):
        tll.paged_attention(q, cache, batch, scale=scale, out=view, max_new=max_new)
        check(view, None, q, cache, batch, starts, held, True, float(np.float32(scale)))
        assert (out[:, H * D:] == 5).all()
    clean = tll.paged_attention(q, cache, batch, max_new=max_new)
    # one sequence's odd values stay in it, and in their key head
    page_id = int(batch.block_table[1, 0])
    cache.k[page_id, 1, 3], cache.v[page_id, 1, 3] = float("nan"), float("inf")
    got = tll.paged_attention(q, cache, batch, max_new=max_new)
    touched = torch.zeros(N, H, dtype=torch.bool, device="cuda")
    touched[2, 2:4] = True
    assert torch.equal(got[~touched], clean[~touched]) and not got[touched].isfinite().any()
    # scores of -inf throughout a row: like a row that sees no key; far scores: no overflow
    cache.k[page_id, 1, 3], cache.v[page_id, 1, 3] = 1.0, 1.0
    big = queries(N, H, D, spread=300.0)
    big_out, lse = tll.paged_attention(big, cache, batch, with_lse=True, max_new=max_new)
    check(big_out, lse, big, cache, batch, starts, held, True, D ** -0.5)


def test_long_context_and_many_parts():
    """Items cut over many blocks, offsets past 2^31 bytes, one head."""
    new, held = [1, 1], [70001, 33000]
    cache, batch, starts, N = make(new, held, 1, 128, 64, "heads", spare=200000)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache.k.normal_(generator=g)
    cache.v.normal_(generator=g)
    q = queries(N, 3, 128)
    for max_new in (1, 10 ** 6):
        out, lse = tll.paged_attention(q, cache, batch, with_lse=True, max_new=max_new)
        tll.default_context(0).check()
        for b in range(2):
            pages = batch.block_table[b, :-(-held[b] // 64)].long()
            k, v = (c[pages][:, 0].flatten(0, 1)[:held[b]].double().cpu() for c in (cache.k, cache.v))
            s = q[b].double().cpu() @ k.T * 128 ** -0.5
            want = torch.softmax(s, 1) @ v
            size = torch.softmax(s, 1) @ v.abs()
            assert ((out[b].double().cpu() - want).abs() <= 1.05 * 2.0 ** -8 * (size + want.abs()) + 1e-5).all()
            assert (lse[b].double().cpu() - torch.logsumexp(s, 1)).abs().max() <= 1e-3


@pytest.mark.parametrize("max_new", [1, 10 ** 6])
def test_graphs_follow_lengths_and_run_side_by_side(max_new):
    """Two graphs of one context, replayed on two streams at once, after lengths have changed."""
    H, Hkv, D, page = 8, 2, 64, 16
    sets = []
    for seed in (0, 1):
        new, held = [1] * 9 + [30], [900 + 40 * i for i in range(10)]
        cache, batch, starts, N = make(new, held, Hkv, D, page, "heads", seed=seed)
        fill(cache, batch, held, seed=seed)
        q = queries(N, H, D, seed=seed)
        out, lse = torch.empty_like(q), torch.empty(N, H, device="cuda")
        tll.paged_attention(q, cache, batch, out=out, lse=lse, max_new=max_new)
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            for _ in range(20):
                tll.paged_attention(q, cache, batch, out=out, lse=lse, max_new=max_new)
        sets.append((g, torch.cuda.Stream(), out, lse, q, cache, batch, starts, [h - 5 for h in held]))
    for g, s, out, lse, q, cache, batch, starts, held in sets:
        batch.kv_len.sub_(5)
        out.fill_(NAN)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s, *_ in sets:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    tll.default_context(0).check()
    for g, s, out, lse, q, cache, batch, starts, held in sets:
        check(out, lse, q, cache, batch, starts, held, True, D ** -0.5)


def test_workspaces_and_streams():
    new, held = [1] * 4, [300] * 4
    cache, batch, starts, N = make(new, held, 4, 64, 16, "heads")
    fill(cache, batch, held)
    q = queries(N, 4, 64)
    want = tll.paged_attention(q, cache, batch)
    size = tll.paged_attention_workspace(cache, batch, N, 4)
    own = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert torch.equal(tll.paged_attention(q, cache, batch, workspace=own), want)
    with pytest.raises(tll.LinError) as e:
        tll.paged_attention(q, cache, batch, workspace=own[:size - 1])
    assert e.value.status == tll.ERR_WORKSPACE
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    for stream in (s, s.cuda_stream):
        out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        tll.paged_attention(q, cache, batch, out=out, stream=stream)
        s.synchronize()
        assert torch.equal(out, want)
    # the context's own workspace, from C
    ctx = tll.default_context(0)
    out.zero_()
    rc = tll.library().lin_paged_attention(ctx.handle, cache._ref, batch._ref(N), 4, q.data_ptr(), 256, out.data_ptr(),
                                           256, None, 1, 0.0, 0, None, 0,
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == tll.OK
    ctx.check()
    assert torch.equal(out, want)
    small = tll.Context(0, 1 << 17)
    assert tll.library().lin_paged_attention(small.handle, cache._ref, batch._ref(N), 4, q.data_ptr(), 256,
                                             out.data_ptr(), 256, None, 1, 0.0, 0, None, 0, None) == tll.ERR_WORKSPACE


def test_the_default_streams_workspace_is_its_own():
    """Calls on the default stream share the cache's workspace, growing with what they need; calls on another
    stream at the same time do not touch it."""
    new, held = [1] * 6, [700 + 90 * i for i in range(6)]
    cache, batch, starts, N = make(new, held, 2, 128, 16, "heads")
    fill(cache, batch, held)
    q = queries(N, 16, 128)
    hints = (1, 100, 1, 100)
    want = [tll.paged_attention(q, cache, batch, max_new=h).clone() for h in hints]
    small = cache._workspace.numel()
    assert small >= tll.paged_attention_workspace(cache, batch, N, 16, 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = {0: [], 1: []}
    for _ in range(30):
        for h in hints:
            got[0].append(tll.paged_attention(q, cache, batch, max_new=h))
            with torch.cuda.stream(side):
                got[1].append(tll.paged_attention(q, cache, batch, max_new=h))
    torch.cuda.synchronize()
    assert cache._workspace.numel() == small
    for outs in got.values():
        for i, out in enumerate(outs):
            assert torch.equal(out, want[i % 4])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [-600.0, 600.0])
def test_scores_of_minus_infinity_before_far_ones(D, far):
    """The first 130 keys of each sequence score -inf for every query; the others lie far below, or far above, zero,
    where an exponential against anything but their own maximum is 0 or inf."""
    new, held = [60, 1, 3], [400, 140, 131]
    cache, batch, starts, N = make(new, held, 2, D, 16, "heads")
    fill(cache, batch, held)
    for b, n in enumerate(held):
        for p in range(n):
            page_id, slot = int(batch.block_table[b, p // 16]), p % 16
            cache.k[page_id, :, slot, 0] = float("-inf") if p < 130 else far / 4
    q = queries(N, 4, D)
    q[:, :, 0] = 4.0 * D ** 0.5
    for max_new in (1, 10 ** 6):
        out, lse = tll.paged_attention(q, cache, batch, max_new=max_new, with_lse=True)
        for b, n in enumerate(held):
            for i in range(new[b]):
                at = n - new[b] + i + 1
                row = starts[b] + i
                for h in range(4):
                    if at <= 130:
                        assert (out[row, h] == 0).all() and lse[row, h] == -float("inf")
                        continue
                    ids = batch.block_table[b, torch.arange(130, at, device="cuda") // 16].long()
                    slots = torch.arange(130, at, device="cuda") % 16
                    k, v = (c[ids, h // 2, slots].double() for c in (cache.k, cache.v))
                    s = k @ q[row, h].double() * D ** -0.5
                    want, size = torch.softmax(s, 0) @ v, torch.softmax(s, 0) @ v.abs()
                    # scores near 600 in fp32, and their product with log2 e: 4 half steps of 2^-24 * 900, once for the
                    # probability and once for the sum, on top of the usual bound
                    tol = 1.05 * 2.0 ** -8 * (size + want.abs()) + 8 * 2.0 ** -24 * 900 * size + 1e-5
                    assert ((out[row, h].double() - want).abs() <= tol).all()
                    assert (lse[row, h].double() - torch.logsumexp(s, 0)).abs() <= 1e-4 * (1 + abs(far))


@pytest.mark.parametrize("max_new", [1, 10 ** 6])
def test_sequences_that_share_pages(max_new):
    """A common prefix of two pages, one page twice in a table, and columns of a wider table."""
    new, held = [2, 1, 40], [50, 37, 64]
    cache, batch, starts, N = make(new, held, 2, 64, 16, "heads")
    fill(cache, batch, held)
    table = batch.block_table
    wide = torch.full((3, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    wide[1, :2] = table[0, :2]
    wide[2, 3] = table[2, 0]
    shared = tll.KVBatch(batch.q_start, batch.kv_len, wide[:, :table.shape[1]])
    q = queries(N, 6, 64)
    for causal in (True, False):
        out, lse = tll.paged_attention(q, cache, shared, causal=causal, max_new=max_new, with_lse=True)
        check(out, lse, q, cache, shared, starts, held, causal, 0.125)


def test_batches_keep_their_arrays():
    cache, batch, _, _ = make([1, 1], [20, 30], 2, 64, 16, "heads")
    with pytest.raises(AttributeError):
        batch.kv_len = batch.kv_len + 1
    with pytest.raises(AttributeError):
        cache.k = cache.v
    batch.kv_len += 1  # in place: what the kernels read
    assert batch.kv_len.tolist() == [21, 31]
