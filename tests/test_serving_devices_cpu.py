"""A context of another device than the tensors' is refused (its kernels would run there, on addresses of the other)."""
import types

import pytest
import torch

import transformer_linear_layer_gb300 as tll
from test_paged_threads_cpu import caches, stand_ins


def test_contexts_of_another_device(monkeypatch):
    lib = stand_ins(monkeypatch)
    monkeypatch.setattr(tll, "_check_positions", lambda *a: tll.TYPE_INT64)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    for call in ("lin_rotary_forward", "lin_rotary_backward", "lin_cache_append"):
        setattr(lib, call, lambda *a, call=call: lib.launches.append(call) or tll.OK)
    cache, = caches(1)
    cache.__dict__["heads"] = 4
    batch = types.SimpleNamespace(index=0, sequences=1, _ref=lambda n: None)
    rotary = types.SimpleNamespace(index=0, _ref=None)
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    here, there = (types.SimpleNamespace(device=d, _h=None) for d in (0, 1))
    entries = (lambda c: tll.rotary_forward(x, x, rotary, out=x.clone(), ctx=c),
               lambda c: tll.rotary_backward(x, x, rotary, out=x.clone(), ctx=c),
               lambda c: tll.cache_append(x, x, x, cache, batch, rotary=rotary, q_out=x.clone(), ctx=c),
               lambda c: tll.paged_attention(x, cache, batch, max_new=1, out=x.clone(), ctx=c))
    for entry in entries:
        with pytest.raises(ValueError):
            entry(there)
    assert not lib.launches
    for entry in entries:
        entry(here)
        entry(None)
    assert len(lib.launches) == 6 + 2 * 2
    monkeypatch.undo()
    with pytest.raises(ValueError):
        tll.paged_attention_workspace(cache, None, 1, 4, 1, ctx=there)
