"""Distillation where its persistent blocks and clusters take many rows each, and on
rows whose logits lie far from zero, against the float64 formulas (evaluated on the
GPU, some rows at a time).

Bounds. The exponential of a logit's distance d from its row's maximum is right to
3 * 2^-24 |d| + 2^-22 (difference, scale and product each to half a step; the hardware
exponential), a sum of V of them to training_ref.sum_error(V). So p is within
sum_error(V) + 4 * 2^-24 min(|d|, 110) relative (further below it is 0 in fp32).
lin_distill_backward may take p from the fp32 lse it is given where |lse| is at most
512 (bf16) or 64 (fp32): two more half steps of such an lse."""
import pytest
import torch

import training_ref as ref
import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu
INF = float("inf")


def make(R, V, K, dtype, seed=0, pad=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((R, V + pad), float("nan"), dtype=dtype, device="cuda")
    z = buf[:, :V]
    for r in range(0, R, 256):
        z[r:r + 256] = (torch.randn(z[r:r + 256].shape, generator=g, device="cuda") * spread).to(dtype)
    ids = torch.randint(0, V, (R, K), generator=g, device="cuda")
    if K > 3:
        ids[:, 3] = ids[:, 0]                  # a token twice
    t = torch.randn(R, K, generator=g, device="cuda") * 2
    w = torch.rand(R, generator=g, device="cuda")
    # padding, no entry, no weight and a bad id all along the rows
    ids[2::11, K // 2] = -1
    ids[5::37] = -1
    w[7::41] = 0.0
    if R > 60:
        ids[59::97, 0] = V
    return z, ids, t, w


def check_rows(z, ids, t, w, tau, got, want_loss=None, lse=None):
    """Gradient `got` (and losses) of all rows; `lse` where the gradient came from one."""
    tau = float(torch.tensor(tau, dtype=torch.float32))
    R, V = z.shape
    half = ref.BF16_HALF if z.dtype == torch.bfloat16 else ref.FP32_HALF
    limit = 512 if z.dtype == torch.bfloat16 else 64
    n = max(1, (1 << 24) // V)
    for r in range(0, R, n):
        x, i, ti, wi = (a[r:r + n] for a in (z, ids, t, w))
        d = x.double() / tau
        d = d - torch.clamp(d.amax(1, keepdim=True), min=-1e300)  # (a row of -inf is not made here)
        p = torch.exp(d)
        logs = torch.log(p.sum(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        held = (i >= 0) & (i < V)
        q = torch.softmax(torch.where(held, ti.double() / tau, -INF), 1).nan_to_num(0.0)
        at = i.clamp(0, V - 1)
        target = torch.zeros_like(p).scatter_add_(1, at, q)
        live = held.any(1) & (wi != 0)
        g = torch.where(live, wi.double() * tau, 0.0)[:, None]
        dz = g * (p - target)
        bad = (i >= V).any(1)
        rel = ref.sum_error(V) + 4 * ref.FP32_HALF * torch.clamp(-d, max=110.0)
        if lse is not None:
            rel = rel + 2 * ref.FP32_HALF * torch.clamp(lse[r:r + n].double().abs(), max=limit)[:, None]
        relq = ref.sum_error(V) + 8 * ref.FP32_HALF * 16
        tol = 1.01 * (g * (rel * p + relq * target + 4 * ref.FP32_HALF * (p + target)) + half * dz.abs()) + 1e-37
        off = (got[r:r + n].double() - dz).abs()
        ok = (off <= tol) | bad[:, None]
        assert bool(ok.all()), (r + int((~ok).any(1).nonzero()[0]), float((off / tol)[~ok].max()))
        assert bool(got[r:r + n][bad & (wi != 0)].isnan().all())
        assert bool((got[r:r + n][~live & ~bad] == 0).all())
        if want_loss is not None:
            logp = d.gather(1, at) - logs
            logq = torch.log(q)
            term = torch.where(q > 0, q * (logq - logp), 0.0)
            loss = tau * tau * term.sum(1)
            size = torch.where(q > 0, q * (logq.abs() + logp.abs()), 0.0).sum(1)
            ltol = tau * tau * (2 * ref.sum_error(V) + 16 * ref.FP32_HALF * (size + 8)) + 4 * ref.FP32_HALF * loss.abs()
            lo = want_loss[r:r + n].double()
            assert bool((((lo - loss).abs() <= ltol) | bad).all()), float(((lo - loss).abs() / ltol)[~bad].max())
            assert bool(lo[bad].isnan().all())


def check_all(z, ids, t, w, tau):
    loss, lse = tll.distill_forward(z, ids, t, temperature=tau)
    back = tll.distill_backward(z, ids, t, lse, w, temperature=tau)
    both_loss, both = tll.distill_forward_backward(z, ids, t, weight=w, temperature=tau)
    tll.default_context(0).check()
    check_rows(z, ids, t, w, tau, both, both_loss)
    check_rows(z, ids, t, w, tau, back, loss, lse)
    # in place, from a copy that lies like the logits
    def copy():
        if z.stride(0) == z.shape[1]:
            return z.clone()
        b = torch.full((z.shape[0], z.stride(0)), float("nan"), dtype=z.dtype, device="cuda")[:, :z.shape[1]]
        return b.copy_(z)
    c = copy()
    tll.distill_backward(c, ids, t, lse, w, temperature=tau, out=c)
    assert torch.equal(c.nan_to_num(9), back.nan_to_num(9))
    c = copy()
    tll.distill_forward_backward(c, ids, t, weight=w, temperature=tau, out=c)
    assert torch.equal(c.nan_to_num(9), both.nan_to_num(9))
    for _ in range(2):
        assert torch.equal(tll.distill_backward(z, ids, t, lse, w, temperature=tau).nan_to_num(9), back.nan_to_num(9))
        again = tll.distill_forward_backward(z, ids, t, weight=w, temperature=tau)
        assert torch.equal(again[1].nan_to_num(9), both.nan_to_num(9))
        assert torch.equal(again[0].nan_to_num(9), both_loss.nan_to_num(9))
    tll.default_context(0).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V,K,pad", [(9001, 517, 12, 0), (6000, 5003, 33, 5), (3000, 20011, 8, 0)])
def test_many_rows_a_block(R, V, K, pad, dtype):
    """Tens of rows a block: its rings of chunks and of teacher entries come round."""
    check_all(*make(R, V, K, dtype, seed=V, pad=pad), 1.5)


@pytest.mark.parametrize("dtype,R,V", [
    (torch.float32, 300, 60001), (torch.float32, 260, 128001),   # loss and gradient: clusters hold a row
    (torch.bfloat16, 300, 128001),
    (torch.float32, 170, 330001), (torch.bfloat16, 170, 700001)])  # the gradient alone takes clusters too
def test_many_rows_a_cluster(dtype, R, V):
    check_all(*make(R, V, 20, dtype, seed=R), 1.0)


def far(z, kinds):
    """Rows in turn moved by an offset, or made of one value."""
    low = torch.finfo(z.dtype).min
    for n, kind in enumerate(kinds):
        rows = z[n::len(kinds)]
        if kind == "lowest":
            rows.fill_(low)
        elif kind == "constant":
            rows.fill_(1e4)
        else:
            rows.copy_((rows.float() + kind).to(z.dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V", [(40, 3001), (1000, 777), (5, 50257), (40, 50257)])
@pytest.mark.parametrize("tau", [1.0, 0.3])
def test_rows_far_from_zero(R, V, dtype, tau):
    """Offsets common to a row (an lse without digits left for the probabilities), and a
    mask of the type's lowest value on all of it."""
    z, ids, t, w = make(R, V, 8, dtype, seed=3)
    far(z, [0.0, 60.0, -500.0, 1e4, -3e5, "lowest", "constant", 2e7])
    check_all(z, ids, t, w, tau)


@pytest.mark.parametrize("dtype,R,V", [(torch.float32, 170, 330001), (torch.bfloat16, 12, 131072)])
def test_clusters_with_rows_far_from_zero(dtype, R, V):
    z, ids, t, w = make(R, V, 8, dtype, seed=4)
    far(z, [0.0, -3e5, 0.0, "lowest", 1e4])
    check_all(z, ids, t, w, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V", [(30, 777), (3, 50257)])
@pytest.mark.parametrize("tau", [1.0, 0.3, 2.0])
def test_loss_where_the_student_masks_a_teachers_token(R, V, dtype, tau):
    """A mask of the type's lowest value costs its finite amount (inf only where the
    loss itself passes fp32), one of -inf costs inf."""
    tau = float(torch.tensor(tau, dtype=torch.float32))
    z, ids, t, _ = make(R, V, 6, dtype, seed=9)
    ids[:] = torch.arange(6, device="cuda") * (V // 7)
    t[:] = torch.tensor([4.0, 1.0, 0.0, -2.0, 3.0, 2.0], device="cuda")
    low = torch.finfo(dtype).min
    z[:, ids[0, 2]] = low
    z[1::3, ids[0, 3]] = low
    z[2::3, ids[0, 1]] = -INF
    d = z.double() / tau
    d = d - d.amax(1, keepdim=True)
    logp = (d - torch.log(torch.exp(d).sum(1, keepdim=True))).gather(1, ids)
    logq = torch.log_softmax(t.double() / tau, 1)
    loss = (tau * tau * (logq.exp() * (logq - logp)).sum(1)).float()  # (past fp32: inf)
    rel = 2 * ref.sum_error(V) + 64 * ref.FP32_HALF
    got, _ = tll.distill_forward(z, ids, t, temperature=tau)
    both, dz = tll.distill_forward_backward(z, ids, t, temperature=tau)
    assert torch.equal(got.isinf(), loss.isinf()) and bool(loss[2::3].isinf().all())
    if tau <= 1:
        assert bool(loss[::3].isfinite().all())
    fine = loss.isfinite()
    assert bool(((got - loss).abs() <= rel * loss.abs())[fine].all())
    assert bool(((both - loss).abs() <= rel * loss.abs())[fine].all()) and torch.equal(both.isinf(), loss.isinf())
    assert bool(dz.isfinite().all())
