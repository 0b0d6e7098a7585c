"""Paged attention from several threads on the default stream, with the library's call replaced by one that notes who is
in it: the two kernels of a call that uses the shared workspace are enqueued before another call's."""
import threading
import time
import types

import pytest
import torch

import transformer_linear_layer_gb300 as tll


class Library:
    """lin_paged_attention's place in the binding: two launches with a pause between, as threads see them."""

    def __init__(self):
        self.launches = []  # (workspace, call)

    def lin_paged_attention(self, *args):
        workspace, call = args[12], threading.get_ident()
        self.launches.append((workspace, call))
        time.sleep(0.001)
        self.launches.append((workspace, call))
        return tll.OK


def stand_ins(monkeypatch, raw=0):
    lib = Library()
    monkeypatch.setattr(tll, "_loaded", lambda: lib)
    monkeypatch.setattr(tll, "_context", lambda index: types.SimpleNamespace(_h=None, device=index))
    monkeypatch.setattr(tll, "_raw_stream", lambda stream, index: raw)
    monkeypatch.setattr(tll, "_check_heads", lambda t, *rest: (*t.shape, t.stride(0)))
    monkeypatch.setattr(tll, "paged_attention_workspace", lambda *a: 4096)
    return lib


def caches(n):
    out = []
    for _ in range(n):
        c = tll.KVCache.__new__(tll.KVCache)
        c.__dict__.update(index=0, head_dim=64, device=torch.device("cpu"), _sizes={}, _ref=None, _workspace=None)
        out.append(c)
    return out


def test_calls_of_two_threads_do_not_mix_their_launches(monkeypatch):
    lib = stand_ins(monkeypatch)
    cache, = caches(1)
    batch = types.SimpleNamespace(index=0, sequences=1, _ref=lambda n: None)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)

    def work():
        for _ in range(10):
            tll.paged_attention(q, cache, batch, max_new=1, out=torch.empty_like(q))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(lib.launches) == 60 and len({w for w, _ in lib.launches}) == 1
    assert all(a == b for a, b in zip(lib.launches[::2], lib.launches[1::2]))


def test_caches_of_a_device_share_one_workspace(monkeypatch):
    """A model has a cache a layer: what calls on the default stream keep does not grow with their number."""
    lib = stand_ins(monkeypatch)
    batch = types.SimpleNamespace(index=0, sequences=1, _ref=lambda n: None)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    layers = caches(5)
    for c in layers:
        tll.paged_attention(q, c, batch, max_new=1, out=torch.empty_like(q))
    assert len({w for w, _ in lib.launches}) == 1
    assert len({c._workspace.data_ptr() for c in layers}) == 1


def test_a_workspace_must_hold_what_its_shape_says(monkeypatch):
    """One byte expanded, or every other byte: the kernels would write past the tensor's memory."""
    lib = stand_ins(monkeypatch)
    cache, = caches(1)
    batch = types.SimpleNamespace(index=0, sequences=1, _ref=lambda n: None)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            tll.paged_attention(q, cache, batch, max_new=1, out=torch.empty_like(q), workspace=bad)
    assert not lib.launches
    good = torch.empty(1024, dtype=torch.float32)
    tll.paged_attention(q, cache, batch, max_new=1, out=torch.empty_like(q), workspace=good)
    assert lib.launches == [(good.data_ptr(), threading.get_ident())] * 2
