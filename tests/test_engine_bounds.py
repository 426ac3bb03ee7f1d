"""How the engine keeps the key bounds, on the host: which stream each piece of work
goes to and which calls bring the bounds up to date, with the library's calls and the
streams recorded instead of run."""
import contextlib

import numpy as np
import pytest
import torch

from _lib import library, pkv
from paged_kv_cache_259_gb300 import engine

NB, HQ, HKV, D, BS = 12, 4, 2, 64, 16
BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


class Recorder:
    """What was done, in order: (name, stream, arguments)."""

    def __init__(self, monkeypatch):
        self.log, self.stack = [], ["current"]
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stack[-1])
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

        @contextlib.contextmanager
        def on(stream):
            self.stack.append(stream)
            try:
                yield
            finally:
                self.stack.pop()

        monkeypatch.setattr(torch.cuda, "stream", on)
        for name in ("zeros", "zeros_like", "full", "arange"):
            real = getattr(torch, name)

            def fill(*a, _real=real, _name=name, **k):
                self.log.append((_name, self.stack[-1], a))
                return _real(*a, **k)

            monkeypatch.setattr(engine.torch, name, fill)

    def call(self, name):
        def fn(*a, stream=None, **k):
            self.log.append((name, self.stack[-1] if stream is None else stream, a))
        return fn

    def named(self, name):
        return [e for e in self.log if e[0] == name]


@pytest.fixture
def rec(monkeypatch):
    library()
    r = Recorder(monkeypatch)
    monkeypatch.setattr(engine, "update_key_bounds", r.call("update"))
    return r


class FakeStream:
    def __init__(self, name):
        self.name, self.cuda_stream, self.synced = name, 0, 0

    def synchronize(self):
        self.synced += 1


def new_cache(**over):
    return engine.PagedKVCache(NB, HQ, HKV, D, BS, BF, range(NB), device="cpu", **over)


def test_bounds_made_on_first_use_are_filled_on_the_stream_that_uses_them(rec):
    s = FakeStream("side")
    rec.stack[0] = FakeStream("current")
    cache, tables, lens = new_cache(), torch.zeros(1, 2, dtype=I32), torch.ones(1, dtype=I32)
    rec.log.clear()
    cache.refresh_key_bounds(tables, lens, stream=s)
    assert cache.key_bounds is not None and rec.named("update")
    assert [e for e in rec.log if e[1] is not s] == []
