"""The training and evaluation operators written out in float64 (numpy), for the
tests: attention's backward pass, distillation from a teacher's top logits and
token log probabilities. Plain sums over explicit arrays, nothing blocked."""
from __future__ import annotations

import numpy as np

BF16_HALF = 2.0 ** -8    # half a step of a bf16 value, relative to it
FP32_HALF = 2.0 ** -24


def heads(x, B, T, H):
    """(B*T) x C to B x H x T x 64."""
    return np.asarray(x, dtype=np.float64).reshape(B, T, H, -1).transpose(0, 2, 1, 3)


def rows(x):
    """Back: B x H x T x 64 to (B*T) x C."""
    B, H, T, D = x.shape
    return x.transpose(0, 2, 1, 3).reshape(B * T, H * D)


def attention_forward(qkv, B, T, H, causal, scale):
    C = qkv.shape[1] // 3
    q, k, v = (heads(qkv[:, i * C:(i + 1) * C], B, T, H) for i in range(3))
    s = np.einsum("bhid,bhjd->bhij", q, k) * scale
    if causal:
        s = np.where(np.tril(np.ones((T, T), dtype=bool)), s, -np.inf)
    m = s.max(-1, keepdims=True)
    lse = (m + np.log(np.exp(s - m).sum(-1, keepdims=True)))[..., 0]
    p = np.exp(s - lse[..., None])
    return rows(np.einsum("bhij,bhjd->bhid", p, v)), lse


def attention_backward(qkv, out, lse, dout, B, T, H, causal, scale, bounds=False):
    """dqkv, and with `bounds` an array of what each output may be off by for p
    and ds rounded to bf16, fp32 products and sums, and the output's rounding."""
    C = qkv.shape[1] // 3
    q, k, v = (heads(qkv[:, i * C:(i + 1) * C], B, T, H) for i in range(3))
    o, do = heads(out, B, T, H), heads(dout, B, T, H)
    s = np.einsum("bhid,bhjd->bhij", q, k) * scale
    lse = np.asarray(lse, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        p = np.exp(s - lse[..., None])
    p = np.where(np.isneginf(lse)[..., None], 0.0, p)
    if causal:
        p = np.where(np.tril(np.ones((T, T), dtype=bool)), p, 0.0)
    delta = (o * do).sum(-1, keepdims=True)
    dp = np.einsum("bhid,bhjd->bhij", do, v)
    ds = p * (dp - delta)
    grads = [scale * np.einsum("bhij,bhjd->bhid", ds, k), scale * np.einsum("bhij,bhid->bhjd", ds, q),
             np.einsum("bhij,bhid->bhjd", p, do)]
    dqkv = np.concatenate([rows(g) for g in grads], axis=1)
    if not bounds:
        return dqkv
    # p: an exponent's argument is right to a few units of 2^-23 of its largest
    # term, then bf16; ds: fp32 of p, dp and delta, then bf16; the sums fp32.
    size = np.abs(q).max() * np.abs(k).max() * q.shape[-1] * scale + np.abs(np.where(np.isfinite(lse), lse, 0)).max()
    rel = 16 * FP32_HALF * (size + 8)
    aq, ak, ado = np.abs(q), np.abs(k), np.abs(do)
    parts = np.einsum("bhid,bhjd->bhij", ado, np.abs(v)) + (np.abs(o) * ado).sum(-1, keepdims=True)
    eds = BF16_HALF * np.abs(ds) + p * (rel * np.abs(dp - delta) + 32 * FP32_HALF * parts)
    ep = p * (BF16_HALF + rel)
    n = 64 * FP32_HALF
    errs = [scale * (np.einsum("bhij,bhjd->bhid", eds + n * np.abs(ds), ak)),
            scale * (np.einsum("bhij,bhid->bhjd", eds + n * np.abs(ds), aq)),
            np.einsum("bhij,bhid->bhjd", ep + n * p, ado)]
    bound = np.concatenate([rows(e) for e in errs], axis=1)
    return dqkv, 1.02 * (bound + BF16_HALF * (np.abs(dqkv) + bound)) + 1e-30


def log_softmax(z, tau):
    z = np.asarray(z, dtype=np.float64) / tau
    m = z.max(-1, keepdims=True)
    base = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        # less the maximum first: at a mask of the type's lowest value lse itself
        # has no digits left for the logarithm
        logs = np.log(np.exp(z - base).sum(-1, keepdims=True))
        lse = base + logs
        return np.where(np.isneginf(lse), -np.inf, (z - base) - logs), lse[:, 0]


def token_logprobs(z, tokens, top, tau):
    """(logprob, entropy, lse, top log probabilities, top ids)."""
    lp, lse = log_softmax(z, tau)
    p = np.exp(lp)
    entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(-1)
    order = np.argsort(-np.where(np.isnan(z), -np.inf, np.asarray(z, dtype=np.float64)), axis=-1, kind="stable")[:, :top]
    tokens = np.asarray(tokens)
    picked = np.take_along_axis(lp, np.clip(tokens, 0, z.shape[1] - 1)[:, None], axis=1)[:, 0]
    picked = np.where(tokens < 0, 0.0, np.where(tokens >= z.shape[1], np.nan, picked))
    return picked, entropy, lse, np.take_along_axis(lp, order, axis=1), order


def distill(z, ids, teacher, weight, tau):
    """(loss, lse, dz)."""
    R, V = z.shape
    lp, lse = log_softmax(z, tau)
    loss, dz = np.zeros(R), np.zeros((R, V))
    for r in range(R):
        if (ids[r] >= V).any():
            loss[r], dz[r] = np.nan, np.nan
            continue
        held = ids[r] >= 0
        t = np.asarray(teacher[r], dtype=np.float64)[held] / tau
        if t.size == 0 or np.all(np.isneginf(t)):
            continue
        q = np.exp(t - t.max())
        q /= q.sum()
        target = np.zeros(V)
        np.add.at(target, ids[r][held], q)
        on = q > 0
        loss[r] = tau ** 2 * (q[on] * (np.log(q[on]) - lp[r, ids[r][held][on]])).sum()
        if weight[r] != 0:
            dz[r] = weight[r] * tau * (np.exp(lp[r]) - target)
    return loss, lse, dz


def sum_error(V):
    """Relative error of a sum of V positive fp32 terms in chains of a few hundred
    additions, each term an exponential right to 2^-21."""
    return (V / 64 + 64) * FP32_HALF + 2.0 ** -21
