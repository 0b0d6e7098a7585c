"""The float64 references of the training operators, pinned by central
differences, by torch's autograd and by closed forms (no GPU)."""
import numpy as np
import pytest
import torch

import training_ref as ref


@pytest.mark.parametrize("B,T,H,causal,scale", [(1, 5, 2, True, 0.125), (2, 4, 1, False, 0.3), (1, 1, 1, True, 0.125)])
def test_attention_backward_matches_differences(B, T, H, causal, scale):
    rng = np.random.default_rng(T)
    C = 64 * H
    qkv, g = rng.normal(size=(B * T, 3 * C)), rng.normal(size=(B * T, C))
    out, lse = ref.attention_forward(qkv, B, T, H, causal, scale)
    dqkv = ref.attention_backward(qkv, out, lse, g, B, T, H, causal, scale)
    for _ in range(40):
        i, j = rng.integers(B * T), rng.integers(3 * C)
        h = 1e-5
        e = np.zeros_like(qkv)
        e[i, j] = h
        f = [(ref.attention_forward(qkv + s * e, B, T, H, causal, scale)[0] * g).sum() for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * h) - dqkv[i, j]) <= 1e-7 * (1 + abs(dqkv[i, j]))


def test_attention_backward_matches_autograd():
    B, T, H, C = 2, 7, 3, 192
    torch.manual_seed(0)
    qkv = torch.randn(B * T, 3 * C, dtype=torch.float64, requires_grad=True)
    g = torch.randn(B * T, C, dtype=torch.float64)
    q, k, v = (qkv[:, i * C:(i + 1) * C].reshape(B, T, H, 64).transpose(1, 2) for i in range(3))
    o = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True)
    o.transpose(1, 2).reshape(B * T, C).backward(g)
    x = qkv.detach().numpy()
    out, lse = ref.attention_forward(x, B, T, H, True, 0.125)
    got = ref.attention_backward(x, out, lse, g.numpy(), B, T, H, True, 0.125)
    np.testing.assert_allclose(got, qkv.grad.numpy(), rtol=0, atol=1e-12)


def test_attention_backward_of_a_query_that_sees_nothing():
    rng = np.random.default_rng(3)
    qkv, g = rng.normal(size=(3, 192)), rng.normal(size=(3, 64))
    out, lse = ref.attention_forward(qkv, 1, 3, 1, False, 0.125)
    lse[0, 0, 1] = -np.inf
    dqkv = ref.attention_backward(qkv, out, lse, g, 1, 3, 1, False, 0.125)
    assert np.all(dqkv[1, :64] == 0) and np.all(np.isfinite(dqkv))


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.5])
def test_distill_matches_differences(tau):
    rng = np.random.default_rng(1)
    R, V, K = 4, 11, 5
    z = rng.normal(size=(R, V)) * 2
    ids = rng.integers(0, V, size=(R, K))
    ids[0, 3:] = -1        # padding
    ids[1, 1] = ids[1, 0]  # the same token twice
    ids[2] = -1            # no entry
    t, w = rng.normal(size=(R, K)), rng.random(R)
    loss, lse, dz = ref.distill(z, ids, t, w, tau)
    assert loss[2] == 0 and np.all(dz[2] == 0)
    h = 1e-6
    for r in range(R):
        for j in range(V):
            e = np.zeros_like(z)
            e[r, j] = h
            f = [(w * ref.distill(z + s * e, ids, t, w, tau)[0]).sum() for s in (1, -1)]
            assert abs((f[0] - f[1]) / (2 * h) - dz[r, j]) <= 1e-7


def test_distill_is_zero_where_student_and_teacher_agree():
    """The loss over all tokens of a vocabulary is tau^2 KL, 0 at the teacher."""
    rng = np.random.default_rng(2)
    z = rng.normal(size=(3, 9))
    ids = np.tile(np.arange(9), (3, 1))
    loss, _, dz = ref.distill(z, ids, z + 4.0, np.ones(3), 1.7)
    np.testing.assert_allclose(loss, 0, atol=1e-14)
    np.testing.assert_allclose(dz, 0, atol=1e-14)


def test_token_logprobs_against_torch():
    torch.manual_seed(0)
    z = torch.randn(6, 13, dtype=torch.float64) * 3
    tokens = np.array([0, 12, -1, 5, 13, 3])
    lp, ent, lse, tl, ti = ref.token_logprobs(z.numpy(), tokens, 4, 0.8)
    want = torch.log_softmax(z / 0.8, -1)
    np.testing.assert_allclose(lse, torch.logsumexp(z / 0.8, -1).numpy(), atol=1e-13)
    np.testing.assert_allclose(ent, torch.distributions.Categorical(logits=z / 0.8).entropy().numpy(), atol=1e-12)
    v, i = torch.topk(want, 4)
    assert np.array_equal(ti, i.numpy())
    np.testing.assert_allclose(tl, v.numpy(), atol=1e-13)
    assert lp[2] == 0 and np.isnan(lp[4]) and abs(lp[0] - want[0, 0].item()) < 1e-13


def test_token_logprobs_ties_and_masks():
    z = np.array([[1.0, 2.0, 2.0, -np.inf], [-np.inf] * 4, [0.0, -0.0, 0.0, -1.0]])
    _, ent, lse, tl, ti = ref.token_logprobs(z, [0, 0, 0], 4, 1.0)
    assert ti.tolist() == [[1, 2, 0, 3], [0, 1, 2, 3], [0, 1, 2, 3]]
    assert np.isneginf(lse[1]) and ent[1] == 0 and np.all(np.isneginf(tl[1])) and np.isneginf(tl[0, 3])
