"""Host logic of KVCache8 without a GPU: the C entry points are recorded, not called."""
import contextlib
import ctypes
import os
import re
import types

import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from moe_ffn_layer_gb300 import kv_cache
from moe_ffn_layer_gb300.kv_cache import KVCache8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Recorder:
    """Stands in for the library: the size query is the library's own, the launches are kept."""

    def __init__(self, real):
        self.entered = []
        self.calls, self.at = [], []                   # and the device that each was called on
        self.device = -1                               # the current one; the caches' is a CPU tensor's, -1
        self.moe_kv_attention_workspace_bytes = real.moe_kv_attention_workspace_bytes
        for name in ("moe_kv_append", "moe_kv_attention", "moe_kv_evict"):
            setattr(self, name, lambda *args, name=name: self.keep(name, args))

    def keep(self, name, args):
        self.calls.append((name, args))
        self.at.append(self.device)
        return 0

    def on_stream(self, stream):
        self.entered.append(stream.cuda_stream)        # as torch does: a stream object, no handle
        return contextlib.nullcontext()

    @contextlib.contextmanager
    def on(self, device):
        was, self.device = self.device, device
        yield
        self.device = was


@pytest.fixture
def calls(monkeypatch):
    """A recorder in the library's place, on stream 0 of a machine that may have no GPU."""
    build_mod.build()
    rec = Recorder(B.lib())
    monkeypatch.setattr(B, "_lib", rec)
    monkeypatch.setattr(kv_cache, "_current", lambda device: 0)
    monkeypatch.setattr(kv_cache, "_capturing", lambda: False, raising=False)
    monkeypatch.setattr(kv_cache, "_device", lambda: rec.device, raising=False)
    monkeypatch.setattr(torch.cuda, "device", rec.on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.cuda, "stream", rec.on_stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: types.SimpleNamespace(cuda_stream=handle))
    return rec


def make(pages=8, Hkv=2, D=64, P=16):
    return KVCache8(pages, Hkv, D, P, device="cpu")


def attend(cache, max_len, Hq=4, B_=1, **kw):
    q = torch.zeros(B_, Hq, cache.head_dim, dtype=torch.bfloat16)
    width = -(-max_len // cache.page)
    return cache.attend(q, torch.zeros(B_, width, dtype=torch.int32), torch.ones(B_, dtype=torch.int32),
                        torch.arange(B_ + 1, dtype=torch.int32), 1, max_len, **kw)


def ws_of(call):
    """(address, bytes) of the workspace that an attention call was given."""
    return call[1][14:16]


def test_counter_bytes_are_the_headers():
    header = open(os.path.join(ROOT, "include", "moe_ffn.h")).read()
    assert int(re.search(r"#define MOE_KV_COUNTER_BYTES (\d+)", header).group(1)) == B.KV_COUNTER_BYTES
    cache = make()
    assert B.moe_kv_attention_workspace_bytes(cache.dims, 4, 1, 1, 1, 64, 0) >= B.KV_COUNTER_BYTES


def test_captured_calls_have_workspaces_of_their_own(calls, monkeypatch):
    """None is the stream's, none is kept for a later call, and each starts with its counters zero."""
    cache = make()
    attend(cache, 64)
    warm = ws_of(calls.calls[-1])
    held, zero = [], []

    def keep(name, args):
        held.append(args)
        zero.append(ctypes.string_at(args[14], B.KV_COUNTER_BYTES).count(0) == B.KV_COUNTER_BYTES)
        return 0

    monkeypatch.setattr(kv_cache, "_capturing", lambda: True, raising=False)
    monkeypatch.setattr(calls, "moe_kv_attention", lambda *args: keep("moe_kv_attention", args))
    attend(cache, 64)
    attend(cache, 64)
    assert all(args[14] != warm[0] for args in held) and all(zero)
    monkeypatch.setattr(kv_cache, "_capturing", lambda: False, raising=False)
    attend(cache, 64)
    assert held[-1][14] == warm[0]                     # the stream's own again

    cold = make()
    monkeypatch.setattr(kv_cache, "_capturing", lambda: True, raising=False)
    attend(cold, 64)
    assert not cold._ws                                # the first call of a stream, captured: nothing to hand on


def test_a_growing_length_seldom_allocates(calls):
    """A decode loop with weights, max_len one more each step: the workspace holds scores by max_len."""
    cache = make(Hkv=8, D=128, P=64)
    w = torch.zeros(2, 8, 5000)
    for L in range(1, 4001):
        attend(cache, L, Hq=32, B_=2, weights=w)
        assert ws_of(calls.calls[-1])[1] >= B.moe_kv_attention_workspace_bytes(cache.dims, 32, 2, 2, 1, L, 1)
    given = [ws_of(c) for c in calls.calls]
    assert sum(a != b for a, b in zip(given, given[1:])) <= 3      # the parts' fixed 5 MB cover most of the growth
    big = torch.zeros(2, 8, 1 << 20)
    del calls.calls[:]
    for L in range(100_000, 110_000, 10):
        attend(cache, L, Hq=32, B_=2, weights=big)
    given = [ws_of(c) for c in calls.calls]
    assert sum(a != b for a, b in zip(given, given[1:])) <= 1


def test_calls_of_other_sizes_from_another_thread_in_between(calls):
    """Whatever another thread's call leaves in the cache between this call's steps, its workspace is its own size's."""

    class Interrupted(KVCache8):
        @property
        def _need(self):
            return (None, 0)

        @_need.setter
        def _need(self, value):
            pass                                       # another thread's sizes, smaller ones, take its place at once

    cache = Interrupted(8, 2, 64, 16, device="cpu")
    attend(cache, 64)
    assert ws_of(calls.calls[-1])[1] >= B.moe_kv_attention_workspace_bytes(cache.dims, 4, 1, 1, 1, 64, 0)


def test_evict_refuses_a_destination_on_another_device(calls):
    cache, dst = make(), make()
    args = (torch.zeros(1, 2, 16), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32), 16, 4, 0, 0,
            torch.zeros(1, 1, dtype=torch.int32))
    cache.evict(*args, dst=dst)
    assert len(calls.calls) == 1
    dst.device, dst._dev = torch.device("cuda", 1), 1
    with pytest.raises(ValueError, match="dst"):
        cache.evict(*args, dst=dst)
    assert len(calls.calls) == 1


@pytest.mark.parametrize("device", [-1, 0, 3])
def test_calls_are_made_on_the_caches_device(calls, device):
    """Whatever device is current; it is current again afterwards."""
    cache = make()
    calls.device = device
    new = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, one = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cache.append(new, new, table, one, torch.arange(2, dtype=torch.int32))
    attend(cache, 16)
    cache.evict(torch.zeros(1, 2, 16), table, one, 16, 4, 0, 0, table)
    assert [name for name, _ in calls.calls] == ["moe_kv_append", "moe_kv_attention", "moe_kv_evict"]
    assert calls.at == [-1, -1, -1] and calls.device == device


@pytest.mark.parametrize("stream", [77, types.SimpleNamespace(cuda_stream=77)])
def test_streams_are_given_as_objects_or_handles(calls, stream):
    """What a call allocates is allocated on its stream, however that is named."""
    cache = make()
    attend(cache, 16, stream=stream)
    table, one = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cache.evict(torch.zeros(1, 2, 16), table, one, 16, 4, 0, 0, table, stream=stream)
    assert [args[-1] for _, args in calls.calls] == [77, 77]
    assert calls.entered == [77, 77, 77] and list(cache._ws) == [77]   # out, the workspace, the eviction's outputs
