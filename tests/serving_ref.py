"""Rotary positions, the append to a paged cache and attention over it, from their
formulas in float64 numpy, one token at a time. Test infrastructure."""
import math

import numpy as np

FP32_HALF = 2.0 ** -24
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def angles(positions, turns):
    """Exact angle in [0, 2 pi) of each position and pair: integers modulo one turn."""
    out = np.empty((len(positions), len(turns)))
    for i, p in enumerate(positions):
        for j, t in enumerate(turns):
            out[i, j] = ((int(p) * (int(t) % (1 << 64))) % (1 << 64)) / 2.0 ** 64
    return 2 * math.pi * out


def rotate(x, theta, rot, interleaved, scale, sign=1):
    """x: N x H x D; theta: N x rot/2."""
    y = np.array(x, dtype=np.float64)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = np.cos(theta[:, i])[:, None] * scale, sign * np.sin(theta[:, i])[:, None] * scale
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, a] * s + x[:, :, b] * c
    return y


def rotate_tol(x, y, rot, interleaved, scale, half):
    """Cosine and sine: the angle (at most pi/4 after quarters are taken off) rounded to
    fp32, and 2 units of the last place of the function, 5 * 2^-24 in all, one more half step for
    the scale; the product and the sum another each (7 in all, of |x_a| + |x_b|), then the
    type's rounding."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    size = np.zeros_like(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        size[:, :, a] = size[:, :, b] = x[:, :, a] + x[:, :, b]
    return 7 * FP32_HALF * abs(scale) * size + half * np.abs(y) + 1e-37


def places(q_start, kv_len, N):
    """(sequence, position) of each row, None for a row of no sequence."""
    out = [None] * N
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            out[q_start[b] + i] = (b, kv_len[b] - n + i)
    return out


def append(k_pages, v_pages, k, v, q_start, kv_len, table, page_size):
    """k_pages, v_pages (pages x heads x page_size x D) with the rows stored, and
    which slots were written."""
    k_pages, v_pages = np.array(k_pages, dtype=np.float64), np.array(v_pages, dtype=np.float64)
    wrote = np.zeros(k_pages.shape, dtype=bool)
    for n, at in enumerate(places(q_start, kv_len, k.shape[0])):
        if at is None:
            continue
        b, p = at
        if not 0 <= p < table.shape[1] * page_size:
            continue
        page = table[b, p // page_size]
        if not 0 <= page < k_pages.shape[0]:
            continue
        k_pages[page, :, p % page_size], v_pages[page, :, p % page_size] = k[n], v[n]
        wrote[page, :, p % page_size] = True
    return k_pages, v_pages, wrote


def attention(q, k_pages, v_pages, q_start, kv_len, table, page_size, causal, scale):
    """out, lse and the bound's size sum_j p_ij |v_j| of each row (NaN for rows of no sequence)."""
    N, H, D = q.shape
    Hkv = k_pages.shape[1]
    G = H // Hkv
    out, size = np.full((N, H, D), np.nan), np.full((N, H, D), np.nan)
    lse = np.full((N, H), np.nan)
    for b in range(len(kv_len)):
        n, held = q_start[b + 1] - q_start[b], max(0, min(kv_len[b], table.shape[1] * page_size))
        if n == 0:
            continue
        K, V = np.zeros((Hkv, held, D)), np.zeros((Hkv, held, D))
        for p in range(held):
            page = table[b, p // page_size]
            if 0 <= page < k_pages.shape[0]:  # a page that is none reads as zeros
                K[:, p], V[:, p] = k_pages[page, :, p % page_size], v_pages[page, :, p % page_size]
        rows = slice(q_start[b], q_start[b + 1])
        at = np.arange(kv_len[b] - n, kv_len[b])
        seen = np.arange(held)[None, :] <= at[:, None] if causal else np.ones((n, held), dtype=bool)
        for h in range(H):
            s = np.where(seen, np.nan_to_num(q[rows, h] @ K[h // G].T, nan=np.nan) * scale, -np.inf)
            m = s.max(1, initial=-np.inf)
            e = np.exp(s - np.where(np.isfinite(m), m, 0)[:, None])
            total = e.sum(1)
            with np.errstate(divide="ignore", invalid="ignore"):
                lse[rows, h] = np.where(total > 0, m + np.log(total), -np.inf)
                prob = np.where(total[:, None] > 0, e / total[:, None], 0)
            out[rows, h], size[rows, h] = prob @ V[h // G], prob @ np.abs(V[h // G])
    return out, lse, size
