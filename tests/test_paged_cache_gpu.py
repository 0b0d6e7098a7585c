"""The append of new keys and values to a paged cache against serving_ref."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu


def host(t):
    return t.double().cpu().numpy()


def make(new, held, Hkv, D, page, order, seed=0, spare=2, N=None):
    """A cache of scattered pages (unused slots NaN) and the batch over it."""
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-h // page)) for h in held]
    total, width = sum(need) + spare, max(need + [1])
    shape = {"heads": (total, Hkv, page, D), "tokens": (total, page, Hkv, D), "pairs": (total, 2, Hkv, page, D)}[order]
    if order == "pairs":
        kv = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        k, v = kv[:, 0], kv[:, 1]
    else:
        k, v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if order == "tokens":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
    ids = torch.randperm(total, generator=g).int()
    table = torch.full((len(new), width + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    table = table.cuda()[:, :width]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    batch = tll.KVBatch(torch.from_numpy(starts).cuda(), torch.tensor(held, dtype=torch.int32, device="cuda"), table)
    return tll.KVCache(k, v), batch, starts, N or int(starts[-1])


def qkv(N, H, Hkv, D, seed=1, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, (H + 2 * Hkv) * D + pad, generator=g).bfloat16().cuda()
    x = x[:, :(H + 2 * Hkv) * D].unflatten(1, (-1, D))
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def check(cache, before, batch, starts, held, q, q_out, k, v, r, positions=None):
    table = batch.block_table.cpu().numpy()
    N = k.shape[0]
    at = ref.places(starts, held, N)
    pos = [p[1] if p else 0 for p in at] if positions is None else positions
    kr, tol = host(k), np.zeros(k.shape)
    if r is not None:
        theta, scale = ref.angles(pos, r.turns.tolist()), float(np.float32(r.scale))
        kr = ref.rotate(host(k), theta, r.dim, r.interleaved, scale)
        tol = ref.rotate_tol(host(k), kr, r.dim, r.interleaved, scale, ref.HALF["bf16"])
        if q is not None:
            want = ref.rotate(host(q), theta, r.dim, r.interleaved, scale)
            live = np.array([p is not None for p in at])
            qt = ref.rotate_tol(host(q), want, r.dim, r.interleaved, scale, ref.HALF["bf16"])
            assert np.all(np.abs(host(q_out) - want)[live] <= qt[live])
    wk, wv, wrote = ref.append(*before, kr, host(v), starts, held, table, cache.page_size)
    wt, _, _ = ref.append(np.zeros_like(wk), np.zeros_like(wk), tol, tol, starts, held, table, cache.page_size)
    gk, gv = host(cache.k), host(cache.v)
    assert np.array_equal(np.isnan(gk), np.isnan(wk)) and np.array_equal(np.isnan(gv), np.isnan(wv))
    assert np.all(np.abs(gk - wk)[wrote] <= wt[wrote]) and np.array_equal(gv[wrote], wv[wrote])
    assert np.array_equal(gk[~wrote], wk[~wrote], equal_nan=True)
    return wrote


@pytest.mark.parametrize("order", ["heads", "tokens", "pairs"])
@pytest.mark.parametrize("new,held,H,Hkv,D,page,rot,interleaved", [
    ([1], [1], 1, 1, 64, 8, 64, False), ([1] * 40, [3 * i + 1 for i in range(40)], 12, 12, 64, 16, 64, False),
    ([5, 0, 17, 1], [5, 9, 40, 33], 6, 2, 128, 32, 64, True), ([130], [700], 5, 5, 64, 256, 20, True),
    ([3, 64, 2], [3, 64, 2], 8, 1, 128, 64, 128, False), ([0, 0, 7], [0, 4, 7], 2, 2, 64, 8, 0, False)])
def test_append(order, new, held, H, Hkv, D, page, rot, interleaved):
    cache, batch, starts, N = make(new, held, Hkv, D, page, order)
    before = host(cache.k), host(cache.v)
    q, k, v = qkv(N, H, Hkv, D)
    r = tll.Rotary(rot, interleaved=interleaved, scaling="linear", factor=2.0)
    q_out = tll.cache_append(q, k, v, cache, batch, rotary=r)
    wrote = check(cache, before, batch, starts, held, q, q_out, k, v, r)
    assert wrote.any()


def test_without_rotation_and_with_given_positions():
    new, held = [4, 9], [20, 9]
    for positions in (None, torch.arange(13, device="cuda") * 1000 - 5, torch.arange(13, device="cuda").int()):
        cache, batch, starts, N = make(new, held, 3, 64, 16, "heads")
        before = host(cache.k), host(cache.v)
        q, k, v = qkv(N, 6, 3, 64, pad=3)  # odd strides: element by element
        if positions is None:
            assert tll.cache_append(None, k, v, cache, batch) is None
            check(cache, before, batch, starts, held, None, None, k, v, None)
        else:
            r = tll.Rotary(64)
            got = tll.cache_append(q, k, v, cache, batch, rotary=r, positions=positions)
            check(cache, before, batch, starts, held, q, got, k, v, r, positions.tolist())


def test_queries_in_place_in_the_qkv_matrix():
    new, held = [33, 1], [33, 50]
    cache, batch, starts, N = make(new, held, 2, 64, 16, "heads")
    q, k, v = qkv(N, 4, 2, 64)
    kept = k.clone(), v.clone()
    r = tll.Rotary(64)
    want = tll.cache_append(q, k, v, cache, batch, rotary=r)
    once = cache.k.clone()
    assert tll.cache_append(q, k, v, cache, batch, rotary=r, q_out=q) is q
    assert torch.equal(q, want) and torch.equal(k, kept[0]) and torch.equal(v, kept[1])
    assert torch.equal(cache.k.nan_to_num(9.0), once.nan_to_num(9.0))


def test_rows_and_places_that_are_none():
    """Rows before the first and behind the last sequence, a sequence longer than its
    table, one shorter than its new tokens, and entries that are no pages."""
    Hkv, D, page = 2, 64, 8
    cache, batch, _, _ = make([4, 6, 3], [4, 20, 9], Hkv, D, page, "heads")
    starts, held = [2, 6, 12, 15], [4, 2, 9]           # the second holds fewer than its 6 new tokens
    q_start, kv_len = batch.q_start, batch.kv_len
    q_start.copy_(torch.tensor(starts)), kv_len.copy_(torch.tensor(held))
    batch.block_table[2, 0] = cache.pages               # not a page
    batch.block_table[0, 0] = -5
    before = host(cache.k), host(cache.v)
    N = 20
    q, k, v = qkv(N, 4, Hkv, D)
    r = tll.Rotary(64)
    q_out = torch.full((N, 4, D), 5.0, dtype=torch.bfloat16, device="cuda")
    tll.cache_append(q, k, v, cache, batch, rotary=r, q_out=q_out)
    wrote = check(cache, before, batch, starts, held, q, q_out, k, v, r)
    assert wrote.sum() == (2 + 1) * Hkv * D             # two of the second's, the last of the third's (position 8)
    assert (q_out[:2] == 5).all() and (q_out[15:] == 5).all()
    kv_len.fill_(2 ** 31 - 1)                           # far past the table: nothing is stored
    now = cache.k.clone()
    tll.cache_append(q, k, v, cache, batch, rotary=r, q_out=q_out)
    assert torch.equal(cache.k.nan_to_num(9.0), now.nan_to_num(9.0))
    q_start.copy_(torch.tensor([7, 3, 19, 1]))          # not ascending: nothing out of range
    tll.cache_append(q, k, v, cache, batch, rotary=r, q_out=q_out)
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """A cache whose last page starts past 2^32 elements."""
    page_stride, pages, Hkv, D, page = 1 << 28, 18, 2, 64, 8
    buf = torch.empty(page_stride * (pages - 1) + 2 * Hkv * page * D, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((pages, Hkv, page, D), (page_stride, page * D, D, 1), 0)
    v = buf.as_strided((pages, Hkv, page, D), (page_stride, page * D, D, 1), Hkv * page * D)
    cache = tll.KVCache(k, v)
    table = torch.tensor([[17, 0]], dtype=torch.int32, device="cuda")
    batch = tll.KVBatch(torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                        torch.tensor([9], dtype=torch.int32, device="cuda"), table)
    q, nk, nv = qkv(3, 2, Hkv, D)
    tll.cache_append(None, nk, nv, cache, batch)
    for i, (page_id, slot) in enumerate(((17, 6), (17, 7), (0, 0))):
        assert torch.equal(k[page_id, :, slot], nk[i]) and torch.equal(v[page_id, :, slot], nv[i])
    del buf, k, v, cache


def test_graph_follows_the_batch():
    new, held = [1, 1, 1], [5, 17, 30]
    cache, batch, starts, N = make(new, held, 2, 64, 16, "heads", spare=8)
    batch.block_table.copy_(torch.arange(6).reshape(3, 2))
    q, k, v = qkv(N, 4, 2, 64)
    r = tll.Rotary(64)
    q_out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tll.cache_append(q, k, v, cache, batch, rotary=r, q_out=q_out)
    for step in range(3):
        before = host(cache.k), host(cache.v)
        g.replay()
        torch.cuda.synchronize()
        check(cache, before, batch, starts, [h + step for h in held], q, q_out, k, v, r)
        batch.kv_len.add_(1)
