"""Refusals of the rotary, append and paged attention entries, at the C ABI and in
the binding, without a GPU: every check stands before the device is touched. The
context is a block of zeros (the checks read only plain values of it); a call that
passes them all reaches the device and returns LIN_ERR_CUDA."""
import ctypes
import math

import pytest
import torch

import serving_ref as ref
import transformer_linear_layer_gb300 as tll

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would run")
BASE = 1 << 40  # addresses that are compared, never read


def at(n):
    return BASE + (n << 34)


@pytest.fixture()
def ctx():
    return ctypes.create_string_buffer(4096)


def plan(dim=64, layout=0, scale=1.0, turns=at(9)):
    return tll.RotaryPlan(dim, layout, scale, turns)


def rotary(ctx, form="forward", r=None, **k):
    a = dict(N=5, H=3, D=64, x=at(0), ldx=192, y=at(1), ldy=192, t=tll.TYPE_BF16, pos=at(2), pt=tll.TYPE_INT64)
    a.update(k)
    call = getattr(tll.library(), "lin_rotary_" + form)
    return call(ctx, a["N"], a["H"], a["D"], a["x"], a["ldx"], a["y"], a["ldy"], a["t"], a["pos"], a["pt"],
                ctypes.byref(plan() if r is None else r), None)


def cache(**k):
    a = dict(k=at(10), v=at(11), pages=50, page_size=16, heads=2, head_dim=64, ps=2 * 16 * 64, hs=16 * 64, ts=64)
    a.update(k)
    return tll.KVCachePlan(a["k"], a["v"], a["pages"], a["page_size"], a["heads"], a["head_dim"], a["ps"], a["hs"], a["ts"])


def batch(**k):
    a = dict(sequences=3, tokens=7, q_start=at(12), kv_len=at(13), table=at(14), table_pages=9, stride=9)
    a.update(k)
    return tll.KVBatchPlan(a["sequences"], a["tokens"], a["q_start"], a["kv_len"], a["table"], a["table_pages"], a["stride"])


def append(ctx, c=None, b=None, r=None, rot=True, **k):
    a = dict(H=4, q=at(0), ldq=256, qo=at(1), ldqo=256, k=at(2), ldk=128, v=at(3), ldv=128, pos=None, pt=tll.TYPE_INT32)
    a.update(k)
    return tll.library().lin_cache_append(ctx, ctypes.byref(c or cache()), ctypes.byref(b or batch()), a["H"], a["q"],
                                          a["ldq"], a["qo"], a["ldqo"], a["k"], a["ldk"], a["v"], a["ldv"], a["pos"],
                                          a["pt"], ctypes.byref(r or plan()) if rot else None, None)


def attention(ctx, c=None, b=None, **k):
    a = dict(H=4, q=at(0), ldq=256, out=at(1), ldo=256, lse=at(2), causal=1, scale=0.0, max_new=1, ws=at(3), size=1 << 28)
    a.update(k)
    return tll.library().lin_paged_attention(ctx, ctypes.byref(c or cache()), ctypes.byref(b or batch()), a["H"], a["q"],
                                             a["ldq"], a["out"], a["ldo"], a["lse"], a["causal"], a["scale"],
                                             a["max_new"], a["ws"], a["size"], None)


@needs_no_gpu
def test_good_calls_pass_the_checks(ctx):
    for form in ("forward", "backward"):
        assert rotary(ctx, form) == tll.ERR_CUDA
        assert rotary(ctx, form, y=at(0)) == tll.ERR_CUDA                           # in place
        assert rotary(ctx, form, r=plan(0, turns=None)) == tll.ERR_CUDA
        assert rotary(ctx, form, ldx=400, y=at(0) + 2 * 192, ldy=400) == tll.ERR_CUDA  # columns of one matrix
        assert rotary(ctx, form, N=1, ldx=192, y=at(0), ldy=500) == tll.ERR_CUDA
    assert append(ctx) == tll.ERR_CUDA
    assert append(ctx, qo=at(0)) == tll.ERR_CUDA
    assert append(ctx, rot=False, H=0, q=None, qo=None) == tll.ERR_CUDA
    assert append(ctx, H=0, q=None, qo=None, pos=at(4)) == tll.ERR_CUDA
    # q, k and v as columns of one matrix, q rotated in place
    assert append(ctx, q=at(0), ldq=512, qo=at(0), ldqo=512, k=at(0) + 512, ldk=512, v=at(0) + 768, ldv=512) == tll.ERR_CUDA
    # k and v as halves of one tensor of pages
    assert append(ctx, c=cache(v=at(10) + 2 * 2048, ps=4096)) == tll.ERR_CUDA
    assert append(ctx, c=cache(hs=64, ts=128)) == tll.ERR_CUDA                     # token-major pages
    assert append(ctx, c=cache(pages=1, heads=1, ps=3, hs=5, ts=64)) == tll.ERR_CUDA
    for k in ({}, {"lse": None}, {"max_new": 0}, {"max_new": 1000}, {"H": 2, "ldq": 128, "ldo": 136}, {"causal": 0},
              {"H": 256, "ldq": 16384, "ldo": 16384}):
        assert attention(ctx, **k) == tll.ERR_CUDA, k


def test_nothing_to_do(ctx):
    assert rotary(ctx, N=0) == tll.OK and rotary(ctx, H=0) == tll.OK and rotary(ctx, D=0, r=plan(0)) == tll.OK
    for b in (batch(tokens=0), batch(sequences=0)):
        assert append(ctx, b=b) == tll.OK
        assert attention(ctx, b=b) == tll.OK
    assert attention(ctx, H=0) == tll.OK


@pytest.mark.parametrize("status,bad", [
    (tll.ERR_ARG, {"N": -1}), (tll.ERR_ARG, {"H": -1}), (tll.ERR_ARG, {"D": -1}), (tll.ERR_ARG, {"x": None}),
    (tll.ERR_ARG, {"y": None}), (tll.ERR_ARG, {"pos": None}), (tll.ERR_ARG, {"ldx": 191}), (tll.ERR_ARG, {"ldy": 191}),
    (tll.ERR_ARG, {"t": 2}), (tll.ERR_ARG, {"pt": 1}), (tll.ERR_ARG, {"y": at(0) + 2}), (tll.ERR_ARG, {"y": at(0), "ldy": 200}),
    (tll.ERR_ARG, {"y": at(2) - 8}), (tll.ERR_ARG, {"y": at(9)}), (tll.ERR_ARG, {"r": plan(63)}),
    (tll.ERR_ARG, {"r": plan(66)}), (tll.ERR_ARG, {"r": plan(-2)}), (tll.ERR_ARG, {"r": plan(layout=2)}),
    (tll.ERR_ARG, {"r": plan(scale=float("inf"))}), (tll.ERR_ARG, {"r": plan(turns=None)}),
    (tll.ERR_ARG, {"ldx": 300, "y": at(0) + 2 * 150, "ldy": 300}),
    (tll.ERR_ALIGN, {"x": at(0) + 1}), (tll.ERR_ALIGN, {"pos": at(2) + 4}), (tll.ERR_ALIGN, {"t": 0, "y": at(1) + 2}),
    (tll.ERR_ALIGN, {"r": plan(turns=at(9) + 4)}), (tll.ERR_UNSUPPORTED, {"D": 2048, "ldx": 9000, "ldy": 9000}),
    (tll.ERR_UNSUPPORTED, {"ldx": 1 << 40})])
def test_rotary_arguments(ctx, status, bad):
    for form in ("forward", "backward"):
        assert rotary(ctx, form, **bad) == status
    assert tll.library().lin_rotary_forward(None, 5, 3, 64, at(0), 192, at(1), 192, 1, at(2), 3, ctypes.byref(plan()),
                                            None) == tll.ERR_ARG
    assert tll.library().lin_rotary_forward(ctx, 5, 3, 64, at(0), 192, at(1), 192, 1, at(2), 3, None, None) == tll.ERR_ARG


CACHES = [
    (tll.ERR_ARG, dict(pages=0)), (tll.ERR_ARG, dict(heads=0)), (tll.ERR_ARG, dict(k=None)), (tll.ERR_ARG, dict(v=None)),
    (tll.ERR_ARG, dict(v=at(10))), (tll.ERR_ARG, dict(v=at(10) + 64)), (tll.ERR_ARG, dict(ts=32)),
    (tll.ERR_ARG, dict(ps=1024)), (tll.ERR_ARG, dict(hs=512)), (tll.ERR_ARG, dict(ts=-64)), (tll.ERR_ARG, dict(ps=0)),
    (tll.ERR_ALIGN, dict(k=at(10) + 8)), (tll.ERR_ALIGN, dict(ts=68, hs=2000, ps=4000)),
    (tll.ERR_ALIGN, dict(hs=1028, ps=2060)), (tll.ERR_ALIGN, dict(ps=2052)), (tll.ERR_UNSUPPORTED, dict(page_size=12)),
    (tll.ERR_UNSUPPORTED, dict(page_size=4)), (tll.ERR_UNSUPPORTED, dict(page_size=8192)),
    (tll.ERR_UNSUPPORTED, dict(head_dim=96)), (tll.ERR_UNSUPPORTED, dict(heads=1 << 20)),
    (tll.ERR_UNSUPPORTED, dict(ps=1 << 45)), (tll.ERR_UNSUPPORTED, dict(pages=2, ps=1 << 40))]
BATCHES = [
    (tll.ERR_ARG, dict(sequences=-1)), (tll.ERR_ARG, dict(tokens=-1)), (tll.ERR_ARG, dict(q_start=None)),
    (tll.ERR_ARG, dict(kv_len=None)), (tll.ERR_ARG, dict(table=None)), (tll.ERR_ARG, dict(table_pages=-1)),
    (tll.ERR_ARG, dict(stride=8)), (tll.ERR_ALIGN, dict(q_start=at(12) + 2)), (tll.ERR_ALIGN, dict(kv_len=at(13) + 2)),
    (tll.ERR_ALIGN, dict(table=at(14) + 2)), (tll.ERR_UNSUPPORTED, dict(table_pages=(1 << 26) + 1, stride=1 << 27)),
    (tll.ERR_UNSUPPORTED, dict(stride=1 << 40))]


@pytest.mark.parametrize("status,bad", CACHES)
def test_caches(ctx, status, bad):
    assert append(ctx, c=cache(**bad)) == status
    assert attention(ctx, c=cache(**bad)) == status


@pytest.mark.parametrize("status,bad", BATCHES)
def test_batches(ctx, status, bad):
    assert append(ctx, b=batch(**bad)) == status
    assert attention(ctx, b=batch(**bad)) == status


@pytest.mark.parametrize("status,bad", [
    (tll.ERR_ARG, {"H": -1}), (tll.ERR_ARG, {"q": None}), (tll.ERR_ARG, {"qo": None}), (tll.ERR_ARG, {"k": None}),
    (tll.ERR_ARG, {"v": None}), (tll.ERR_ARG, {"ldq": 255}), (tll.ERR_ARG, {"ldqo": 255}), (tll.ERR_ARG, {"ldk": 127}),
    (tll.ERR_ARG, {"ldv": 127}), (tll.ERR_ARG, {"rot": False}), (tll.ERR_ARG, {"H": 0}), (tll.ERR_ARG, {"r": plan(66)}),
    (tll.ERR_ARG, {"pos": at(4), "pt": 0}), (tll.ERR_ARG, {"qo": at(0) + 2}), (tll.ERR_ARG, {"qo": at(2)}),
    (tll.ERR_ARG, {"qo": at(3) + 4}), (tll.ERR_ARG, {"k": at(10)}), (tll.ERR_ARG, {"v": at(11) + 64}),
    (tll.ERR_ARG, {"q": at(10) + 16}), (tll.ERR_ARG, {"qo": at(11)}), (tll.ERR_ARG, {"qo": at(12)}),
    (tll.ERR_ARG, {"qo": at(13)}), (tll.ERR_ARG, {"qo": at(14)}), (tll.ERR_ARG, {"qo": at(9)}),
    (tll.ERR_ARG, {"pos": at(10)}), (tll.ERR_ALIGN, {"k": at(2) + 1}), (tll.ERR_ALIGN, {"pos": at(4) + 2}),
    (tll.ERR_UNSUPPORTED, {"ldk": 1 << 40})])
def test_append_arguments(ctx, status, bad):
    assert append(ctx, **bad) == status
    assert append(None) == tll.ERR_ARG


@pytest.mark.parametrize("status,bad", [
    (tll.ERR_ARG, {"H": -1}), (tll.ERR_ARG, {"H": 3}), (tll.ERR_ARG, {"q": None}), (tll.ERR_ARG, {"out": None}),
    (tll.ERR_ARG, {"ldq": 248}), (tll.ERR_ARG, {"ldo": 248}), (tll.ERR_ARG, {"causal": 2}), (tll.ERR_ARG, {"scale": -1.0}),
    (tll.ERR_ARG, {"scale": float("nan")}), (tll.ERR_ARG, {"scale": float("inf")}), (tll.ERR_ARG, {"scale": 1e-35}), (tll.ERR_ARG, {"scale": 1e35}),
    (tll.ERR_ARG, {"max_new": -1}),
    (tll.ERR_ARG, {"out": at(0)}), (tll.ERR_ARG, {"out": at(10)}), (tll.ERR_ARG, {"out": at(11) + 64}),
    (tll.ERR_ARG, {"out": at(12)}), (tll.ERR_ARG, {"out": at(14)}), (tll.ERR_ARG, {"lse": at(1)}),
    (tll.ERR_ARG, {"lse": at(0) + 4}), (tll.ERR_ARG, {"lse": at(13)}), (tll.ERR_ARG, {"ws": at(0)}),
    (tll.ERR_ARG, {"ws": at(1)}), (tll.ERR_ARG, {"ws": at(10)}), (tll.ERR_ARG, {"ws": at(2) - 16}),
    (tll.ERR_ALIGN, {"q": at(0) + 8}), (tll.ERR_ALIGN, {"out": at(1) + 2}), (tll.ERR_ALIGN, {"ldq": 260}),
    (tll.ERR_ALIGN, {"ldo": 257}), (tll.ERR_ALIGN, {"lse": at(2) + 2}), (tll.ERR_ALIGN, {"ws": at(3) + 8}),
    (tll.ERR_UNSUPPORTED, {"H": 2 * 130, "ldq": 16640, "ldo": 16640}), (tll.ERR_UNSUPPORTED, {"ldq": 1 << 40})])
def test_attention_arguments(ctx, status, bad):
    assert attention(ctx, **bad) == status
    assert attention(None) == tll.ERR_ARG


def test_workspace_sizes(ctx):
    size = ctypes.c_size_t()
    ask = lambda c, b, H, n: tll.library().lin_paged_attention_workspace(  # noqa: E731
        ctx, None if c is None else ctypes.byref(c), None if b is None else ctypes.byref(b), H, n, ctypes.byref(size))
    assert ask(cache(), None, 4, 1) == tll.OK
    assert ask(cache(), batch(), 4, 0) == tll.OK
    assert ask(cache(), None, 4, 0) == tll.ERR_ARG          # nothing to go by
    assert ask(None, batch(), 4, 1) == tll.ERR_ARG
    assert ask(cache(), None, 3, 1) == tll.ERR_ARG
    assert ask(cache(), None, 4, -1) == tll.ERR_ARG
    assert ask(cache(head_dim=80), None, 4, 1) == tll.ERR_UNSUPPORTED
    assert ask(cache(), None, 2 * 129, 1) == tll.ERR_UNSUPPORTED
    assert tll.library().lin_paged_attention_workspace(None, ctypes.byref(cache()), None, 4, 1, ctypes.byref(size)) == tll.ERR_ARG
    assert tll.library().lin_paged_attention_workspace(ctx, ctypes.byref(cache()), None, 4, 1, None) == tll.ERR_ARG


def test_turns_are_the_frequencies_modulo_one_turn():
    values = [0.0, 1.0, -1.0, 2 * math.pi, 1e-9, -1e-30, 500.25, 10000.0 ** -0.5, 7.0 * math.pi]
    turns = (ctypes.c_ulonglong * len(values))()
    freq = (ctypes.c_double * len(values))(*values)
    assert tll.library().lin_rotary_turns(freq, len(values), turns) == tll.OK
    for f, t in zip(values, turns):
        want = (f / (2 * math.pi)) % 1.0
        off = abs(t / 2.0 ** 64 - want)
        # the quotient is rounded to 53 bits, once
        assert min(off, 1 - off) <= 2.0 ** -52 * max(1.0, abs(f)), f
    freq[3] = float("inf")
    assert tll.library().lin_rotary_turns(freq, len(values), turns) == tll.ERR_ARG
    assert tll.library().lin_rotary_turns(None, 1, turns) == tll.ERR_ARG
    assert tll.library().lin_rotary_turns(freq, -1, turns) == tll.ERR_ARG
    assert tll.library().lin_rotary_turns(None, 0, None) == tll.OK


def test_scaled_frequencies():
    """Each scaling at its ends: the fastest pair, the slowest, and what a ramp leaves between."""
    plain = tll.Rotary(64, device="cpu").frequencies
    assert plain[0] == 1.0 and plain[31] == pytest.approx(10000.0 ** (-62 / 64), rel=1e-12)
    linear = tll.Rotary(64, scaling="linear", factor=4.0, device="cpu").frequencies
    assert linear == pytest.approx([f / 4 for f in plain], rel=1e-12)
    ntk = tll.Rotary(64, scaling="ntk", factor=4.0, device="cpu").frequencies
    assert ntk[0] == 1.0 and ntk[31] == pytest.approx(plain[31] / 4, rel=1e-9)
    r = tll.Rotary(64, scaling="yarn", factor=8.0, original_length=2048, device="cpu")
    assert r.scale == pytest.approx(0.1 * math.log(8) + 1)
    for f, g in zip(plain, r.frequencies):
        turns = 2048 * f / (2 * math.pi)
        keep = min(1, max(0, (turns - 1) / 31))
        assert g == pytest.approx(f * keep + f / 8 * (1 - keep), rel=1e-12)
    assert r.frequencies[0] == 1.0 and r.frequencies[31] == pytest.approx(plain[31] / 8, rel=1e-12)
    own = tll.Rotary(4, frequencies=[0.5, 0.25], scale=2.0, device="cpu")
    assert own.frequencies == [0.5, 0.25] and own.scale == 2.0
    assert own.turns.tolist()[1] == pytest.approx(0.25 / (2 * math.pi) * 2 ** 64, rel=1e-12)
    theta = ref.angles([4], tll.Rotary(2, frequencies=[1.0], device="cpu").turns.tolist())
    assert theta[0, 0] == pytest.approx(4.0, abs=1e-12)


@pytest.mark.parametrize("bad", [dict(dim=63), dict(dim=-2), dict(dim=64, scaling="cubic"), dict(dim=64, scaling="linear", factor=0.5),
                                 dict(dim=64, base=0.0), dict(dim=64, scaling="yarn", factor=2.0),
                                 dict(dim=64, scaling="yarn", factor=2.0, original_length=100, fast=1.0, slow=1.0),
                                 dict(dim=64, frequencies=[1.0])])
def test_plans_that_are_none(bad):
    with pytest.raises(ValueError):
        tll.Rotary(**bad, device="cpu")
    with pytest.raises(tll.LinError):
        tll.Rotary(2, frequencies=[float("nan")], device="cpu")


def test_the_binding_refuses_tensors_that_are_not_on_the_gpu():
    r = tll.Rotary(64, device="cpu")
    with pytest.raises(ValueError):
        tll.rotary_forward(torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int64), r)
    with pytest.raises(ValueError):
        tll.KVCache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        tll.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32))


def test_plans_keep_what_the_library_was_given():
    plan = tll.Rotary(64, device="cpu")
    with pytest.raises(AttributeError):
        plan.scale = 2.0
    with pytest.raises(AttributeError):
        plan.turns = plan.turns.clone()
    plan.turns += 0  # in place: the same tensor
    assert plan.scale == 1.0 and plan._plan.turns == plan.turns.data_ptr()
