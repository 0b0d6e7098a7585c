"""GPU parity of the operators on logits against the float64 formulas.

Bounds. A term of a softmax's sum is exp2((z - m) c): the difference, c and the
product are each within half a step, so the argument d is off by 3 * 2^-24 |d|
and the hardware exponential by 2^-22; a sum of V terms in chains of a few hundred
additions by sum_error(V). Log probabilities are then within sum_error(V) +
4 * 2^-24 |value|, probabilities within twice that relative, outputs of bf16 one
more 2^-8."""
import numpy as np
import pytest
import torch

import training_ref as ref
import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu
INF = float("inf")


def host(t):
    return t.double().cpu().numpy()


def logits(R, V, ld, dtype, seed=0, offset=0, spread=3.0):
    """R x V logits, rows ld apart, the first `offset` elements into a buffer of NaN."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((R * ld + 64,), float("nan"), dtype=dtype, device="cuda")
    z = buf.as_strided((R, V), (ld, 1), offset)
    z.copy_((torch.randn(R, V, generator=g) * spread).to(dtype))
    return z


def close(got, want, tol, what):
    got, want, tol = host(got), np.asarray(want, dtype=np.float64), np.broadcast_to(tol, np.shape(want))
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), what
    err = np.where(odd, 0, np.abs(np.where(odd, 0, got) - np.where(odd, 0, want)))
    assert np.all((err <= tol) | odd), (what, err.max(), np.nanmax(err / np.maximum(tol, 1e-300)))


def log_tol(V, want):
    return ref.sum_error(V) + 4 * ref.FP32_HALF * np.where(np.isfinite(want), np.abs(want), 0)


def check_logprobs(z, tokens, top, tau):
    tau = float(np.float32(tau))
    r = tll.token_logprobs(z, tokens, top=top, temperature=tau)
    tll.default_context(0).check()
    tok = np.full(z.shape[0], -1) if tokens is None else host(tokens).astype(np.int64)
    lp, ent, lse, tlp, ti = ref.token_logprobs(host(z), tok, top, tau)
    V = z.shape[1]
    assert np.array_equal(host(r.top_ids), ti)
    close(r.lse, lse, log_tol(V, lse), "lse")
    # the entropy adds the terms' own values: each to the sums' error
    close(r.entropy, ent, 2 * ref.sum_error(V) * (1 + np.nan_to_num(ent)) + 1e-6, "entropy")
    size = np.abs(np.where(np.isfinite(host(z)), host(z), 0)).max() / tau
    close(r.top_logprob, tlp, log_tol(V, tlp) + 4 * ref.FP32_HALF * size, "top")
    if tokens is None:
        assert r.logprob is None
    else:
        close(r.logprob, lp, log_tol(V, lp) + 4 * ref.FP32_HALF * size, "logprob")


SHAPES = [  # R, V, row stride, offset: one row, odd and aligned vocabularies, rows that start anywhere
    (1, 50257, 50257, 0), (1, 1, 1, 0), (3, 7, 9, 1), (5, 300, 300, 0), (2, 1025, 1030, 3), (40, 4001, 4001, 0),
    (200, 2048, 2048, 0), (19, 50257, 50304, 0), (700, 777, 777, 5), (3, 131072, 131072, 0)]


@pytest.mark.parametrize("R,V,ld,offset", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_token_logprobs(R, V, ld, offset, dtype):
    z = logits(R, V, ld, dtype, seed=R + V, offset=offset)
    tokens = torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(1)).cuda()
    if R > 2:
        tokens[1] = -100
    check_logprobs(z, tokens, min(20, V), 1.0)
    check_logprobs(z, tokens.int(), min(64, V), 0.7)
    check_logprobs(z, None, min(1, V), 3.0)
    check_logprobs(z, tokens, 0, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V", [(3, 50257), (200, 4001), (2, 130), (1, 64), (170, 300)])
@pytest.mark.parametrize("kind", ["all_masked", "constant", "few", "quantised", "zeros", "lowest", "lowest_few"])
def test_ties_and_masks(dtype, R, V, kind):
    """More equal values than the top holds (lowest index first), rows whose mask
    leaves nothing or little, masks of -inf and of the type's lowest value."""
    g = torch.Generator().manual_seed(7)
    z = torch.randn(R, V, generator=g).cuda()
    low = torch.finfo(dtype).min
    few = (torch.rand(R, V, generator=g) < 10 / V).cuda()
    z = {"all_masked": torch.full_like(z, -INF), "constant": torch.full_like(z, 1.5), "few": z.masked_fill(~few, -INF),
         "quantised": z.round(), "zeros": torch.where(few, 0.0, -0.0), "lowest": torch.full_like(z, low),
         "lowest_few": z.masked_fill(~few, low)}[kind].to(dtype)
    for top in (1, 20, 64):
        if top <= V:
            check_logprobs(z, None, top, 1.0)


def test_not_a_number_and_infinity_stay_in_their_row():
    z = logits(6, 5000, 5000, torch.float32)
    z[1, 77], z[3, 4999], z[4] = float("nan"), INF, -INF
    tokens = torch.tensor([3, 3, 5000, 3, 3, 4999], device="cuda")
    r = tll.token_logprobs(z, tokens, top=5)
    lp = host(r.logprob)
    assert np.isnan(lp[[1, 2, 3]]).all() and np.isfinite(lp[[0, 5]]).all() and np.isneginf(lp[4])
    assert np.isnan(host(r.lse)[[1, 3]]).all() and np.isfinite(host(r.lse)[[0, 2, 5]]).all()
    assert host(r.entropy)[4] == 0 and np.isfinite(host(r.top_logprob)[[0, 2, 5]]).all()
    assert 77 not in r.top_ids[1].tolist()


@pytest.mark.parametrize("offset", [1e4, -3e5])
def test_an_offset_common_to_a_row_changes_nothing(offset):
    """fp32 logits that are whole multiples of a step survive the offset exactly."""
    z = (logits(4, 3001, 3001, torch.float32) * 32).round() / 32
    a, b = tll.token_logprobs(z, top=8), tll.token_logprobs(z + offset, top=8)
    assert torch.equal(a.top_ids, b.top_ids) and torch.equal(a.top_logprob, b.top_logprob)
    assert torch.equal(a.entropy, b.entropy)


def test_rows_past_four_gigabytes():
    R, V = 20000, 131072
    z = torch.empty(R, V, dtype=torch.bfloat16, device="cuda").normal_()
    tokens = torch.full((R,), 131071, device="cuda")
    r = tll.token_logprobs(z, tokens, top=4)
    pick = torch.tensor([0, 9999, 16383, 16384, 19998, 19999], device="cuda")
    part = tll.token_logprobs(z[pick].contiguous(), tokens[pick], top=4)
    assert torch.equal(r.top_ids[pick], part.top_ids)
    want = ref.token_logprobs(host(z[pick]), np.full(6, 131071), 4, 1.0)
    assert np.array_equal(host(r.top_ids[pick]), want[4])
    close(r.lse[pick], want[2], log_tol(V, want[2]), "lse")
    close(r.logprob[pick], want[0], log_tol(V, want[0]) + 1e-5, "logprob")


# ------------------------------------------------------------------ distillation

def teacher(R, V, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (R, K), generator=g)
    if K > 3:
        ids[:, 3::4] = ids[:, :1]          # tokens that appear more than once
    t = torch.randn(R, K, generator=g) * 2
    w = torch.rand(R, generator=g)
    if R > 2:
        ids[1] = -1                        # no entry at all
        ids[0, K // 2] = -7                # padding among entries
    if R > 4:
        t[3] = -INF                        # entries without weight
        t[4, 0] = -INF
        w[2] = 0.0
    if R > 30:
        ids[7, 0] = V                      # past the vocabulary
    return ids.cuda(), t.cuda(), w.cuda()


def check_distill(z, ids, t, w, tau, exact_bf16=True):
    tau = float(np.float32(tau))
    V = z.shape[1]
    loss, lse, dz = ref.distill(host(z), host(ids).astype(np.int64), host(t), host(w), tau)
    size = np.abs(host(z)).max() / tau + np.abs(np.where(np.isfinite(host(t)), host(t), 0)).max() / tau
    rel = ref.sum_error(V) + 8 * ref.FP32_HALF * size
    loss_tol = tau * tau * rel * 4 + 8 * ref.FP32_HALF * np.abs(loss)
    # p and q each to rel, their difference to a half step of fp32, the output's own rounding
    p = np.exp(ref.log_softmax(host(z), tau)[0])
    g = np.abs(host(w))[:, None] * tau
    out = ref.BF16_HALF if z.dtype == torch.bfloat16 else ref.FP32_HALF
    dz_tol = 1.01 * (2 * rel * g * (p + np.abs(np.where(g > 0, dz / np.where(g > 0, g, 1), 0)) ) + out * np.abs(dz)) + 1e-37
    dz_tol = np.where(np.isnan(dz_tol), 0, dz_tol)
    got, got_lse = tll.distill_forward(z, ids, t, temperature=tau)
    close(got, loss, loss_tol, "loss")
    close(got_lse, lse, log_tol(V, lse), "lse")
    back = tll.distill_backward(z, ids, t, got_lse, w, temperature=tau)
    # lse itself is rounded to fp32: every p of the row moves with it
    close(back, dz, dz_tol + 4 * ref.FP32_HALF * np.abs(np.nan_to_num(lse))[:, None] * g * p, "backward")
    both_loss, both = tll.distill_forward_backward(z, ids, t, weight=w, temperature=tau)
    close(both_loss, loss, loss_tol, "loss of both")
    close(both, dz, dz_tol, "gradient of both")
    tll.default_context(0).check()
    return both


DISTILL = [  # R, V, row stride, offset, K
    (1, 50257, 50257, 0, 16), (1, 1, 1, 0, 1), (3, 7, 9, 1, 5), (5, 300, 300, 0, 256), (40, 4001, 4001, 0, 33),
    (9, 50257, 50304, 0, 64), (333, 777, 777, 5, 4), (160, 20011, 20011, 0, 8), (3, 131072, 131072, 0, 100)]


@pytest.mark.parametrize("R,V,ld,offset,K", DISTILL)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill(R, V, ld, offset, K, dtype):
    z = logits(R, V, ld, dtype, seed=R + V, offset=offset)
    ids, t, w = teacher(R, V, K)
    check_distill(z, ids, t, w, 1.0)
    check_distill(z, ids.int(), t.bfloat16(), w, 2.5)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 262145), (torch.bfloat16, 500003)])
def test_distill_of_rows_larger_than_a_cluster_holds(dtype, V):
    z = logits(5, V, V, dtype)
    ids, t, w = teacher(5, V, 12)
    check_distill(z, ids, t, w, 1.0)
    check_logprobs(z, None, 10, 1.0)


@pytest.mark.parametrize("R,V,ld", [(300, 5003, 5003), (6, 50257, 50304), (2, 500003, 500003)])
def test_distill_in_place_and_into_other_rows(R, V, ld):
    z = logits(R, V, ld, torch.bfloat16)
    ids, t, w = teacher(R, V, 24)
    loss, want = tll.distill_forward_backward(z, ids, t, weight=w)
    out = torch.full((R, V + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    tll.distill_forward_backward(z, ids, t, weight=w, out=out[:, 1:V + 1])
    assert torch.equal(out[:, 1:V + 1].nan_to_num(99), want.nan_to_num(99))
    assert (out[:, 0] == 7).all() and (out[:, V + 1:] == 7).all()
    lse = tll.distill_forward(z, ids, t)[1]
    back = tll.distill_backward(z, ids, t, lse, w)
    copy = z.clone()
    tll.distill_backward(copy, ids, t, lse, w, out=copy)
    assert torch.equal(copy.nan_to_num(99), back.nan_to_num(99))
    tll.distill_forward_backward(z, ids, t, weight=w, out=z)  # rows ld apart, NaN between them
    assert torch.equal(z.nan_to_num(99), want.nan_to_num(99))


def test_distill_ignores_logits_of_rows_without_weight():
    z = logits(6, 999, 999, torch.float32)
    ids, t, w = teacher(6, 999, 8)
    w[5] = 0.0
    z[1], z[5, 3] = -INF, float("nan")     # a row without entries, a row of weight 0
    _, dz = tll.distill_forward_backward(z, ids, t, weight=w)
    assert (dz[[1, 2, 3, 5]] == 0).all() and torch.isfinite(dz).all()


def test_distill_masked_student():
    """-inf among the student's logits: no probability, no gradient there."""
    z = logits(4, 2000, 2000, torch.float32)
    ids, t, w = teacher(1, 2000, 8, seed=4)
    ids, t, w = ids.repeat(4, 1), t.repeat(4, 1), w.repeat(4)
    banned = torch.ones(2000, dtype=torch.bool, device="cuda")
    banned[ids[0]] = False
    z[:, banned & (torch.arange(2000, device="cuda") % 2 == 0)] = -INF
    loss, dz = tll.distill_forward_backward(z, ids, t, weight=w)
    want = ref.distill(host(z), host(ids).astype(int), host(t), host(w), 1.0)
    close(loss, want[0], 1e-5, "loss")
    close(dz, want[2], 1e-6, "gradient")
    assert (dz[z == -INF] == 0).all()


def test_repeats_bit_for_bit_in_graphs_and_on_other_streams():
    z = logits(400, 6001, 6001, torch.bfloat16)
    ids, t, w = teacher(400, 6001, 16)
    tokens = torch.randint(0, 6001, (400,), device="cuda")
    one = z[:3]

    def run():
        return (*tll.distill_forward_backward(z, ids, t, weight=w), *tll.token_logprobs(z, tokens, top=9),
                *tll.distill_forward(z, ids, t), *tll.token_logprobs(one, tokens[:3], top=9),
                *tll.distill_forward_backward(one, ids[:3], t[:3]))

    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a.nan_to_num(9), b.nan_to_num(9)) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = run()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.nan_to_num(9), b.nan_to_num(9)) for a, b in zip(got, want))


def test_binding_refusals():
    z = logits(3, 50, 50, torch.float32)
    ids, t, w = teacher(1, 50, 4)
    ids, t, w = ids.repeat(3, 1), t.repeat(3, 1), w.repeat(3)
    for bad in (lambda: tll.token_logprobs(z.half()), lambda: tll.token_logprobs(z, torch.zeros(3, device="cuda")),
                lambda: tll.distill_forward(z, ids.float(), t), lambda: tll.distill_forward(z, ids, t.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: tll.token_logprobs(z.t()), lambda: tll.token_logprobs(z, top=51),
                lambda: tll.token_logprobs(z, torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: tll.distill_forward(z, ids[:2], t[:2]), lambda: tll.distill_forward(z, ids, t[:, :3]),
                lambda: tll.distill_forward_backward(z, ids, t, weight=w[:2]),
                lambda: tll.distill_forward_backward(z, ids, t, out=z.bfloat16()),
                lambda: tll.distill_backward(z, ids, t, w.double(), w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tll.LinError) as e:
        tll.token_logprobs(z, temperature=0.0)
    assert e.value.status == tll.ERR_ARG
    many = torch.zeros(3, 257, dtype=torch.int32, device="cuda")
    with pytest.raises(tll.LinError) as e:
        tll.distill_forward(z, many, many.float())
    assert e.value.status == tll.ERR_UNSUPPORTED
