"""How the engine keeps the key bounds, on the host: which stream each piece of work
goes to and which calls bring the bounds up to date, with the library's calls and the
streams recorded instead of run."""
import contextlib
import ctypes

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
        """A library call, or a bound one, that records itself."""
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


def step_args(B=2, width=4, K=3):
    """Host tensors of a sparse step, to be called with the library's calls recorded."""
    plan = {"pairs": torch.zeros(0, 2, dtype=I64), "slots": torch.zeros(B, dtype=I64),
            "tables": torch.zeros(B, width, dtype=I32), "lens": torch.ones(B, dtype=I32)}
    q, kv = torch.zeros(B, HQ, D, dtype=BF), torch.zeros(B, HKV, D, dtype=BF)
    pos = torch.zeros(B, dtype=I32)
    return dict(q=q, k_new=kv, v_new=kv.clone(), dev_plan=plan, positions=pos, first=pos.clone(),
                rotary=engine.Rotary(torch.zeros(8, 2, D // 2)), selected=torch.zeros(B, HKV, K, dtype=I32),
                out=torch.empty_like(q), scale=0.1)


def covered(updates):
    """Blocks whose bounds the recorded updates take whole: (block, tokens seen)."""
    seen = {}
    for _, _, (_, _, tables, lens, first, *_) in updates:
        for row, n, f in zip(tables.tolist(), lens.tolist(), first.tolist()):
            for j in range(f // BS, -(-n // BS)) if f < n else ():
                seen[row[j]] = min(BS, n - j * BS)
    return seen


@pytest.mark.parametrize("blocks", [1, NB, (1 << 16) + 3])
def test_enabling_takes_the_bounds_of_every_block(rec, blocks):
    s = FakeStream("side")
    cache = engine.PagedKVCache(blocks, 1, 1, 16, 16, BF, range(blocks), device="cpu")
    cache.enable_key_bounds(s)
    assert covered(rec.named("update")) == {i: 16 for i in range(blocks)}
    assert all(e[1] is s for e in rec.log[-3:]) and s.synced == 1
    n = len(rec.log)
    assert cache.enable_key_bounds() is cache.key_bounds and len(rec.log) == n


def test_a_sparse_step_on_a_cache_without_bounds_takes_them_first(rec, monkeypatch):
    s = FakeStream("side")
    cache, a = new_cache(), step_args()
    for name in ("bind_rotary_and_cache", "bind_update_key_bounds", "bind_select_blocks",
                 "bind_paged_attention_decode_sparse"):
        monkeypatch.setattr(engine, name, lambda *x, name=name: rec.call(name[5:]))
    cache.sparse_step(**a, stream=s)
    order = [e[0] for e in rec.log if e[0] not in ("arange", "full", "zeros", "zeros_like")]
    assert order == ["update", "rotary_and_cache", "update_key_bounds", "select_blocks",
                     "paged_attention_decode_sparse"]
    assert set(covered(rec.named("update"))) == set(range(NB))


def test_bounds_are_not_made_while_a_graph_is_captured(rec, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    cache = new_cache()
    with pytest.raises(RuntimeError, match="before capturing"):
        cache.enable_key_bounds()
    assert getattr(cache, "key_bounds", None) is None and not rec.named("update")


# --------------------------------------------------- every write keeps them up
@pytest.fixture
def kept(rec, monkeypatch):
    """A cache that keeps bounds, the library's calls recorded."""
    for name in ("reshape_and_cache", "copy_blocks", "swap_blocks", "paged_prefill_step"):
        monkeypatch.setattr(engine, name, rec.call(name))
    monkeypatch.setattr(engine, "bind_paged_decode_step", lambda *a: lambda s, **k: rec.log.append(("step", s, a)))
    rec.stack[0] = FakeStream("current")
    cache = new_cache()
    cache.key_bounds = torch.zeros(pkv.key_bounds_shape(NB, HKV, D), dtype=BF)
    return cache


def seq_table(cache, s):
    n = cache.bm.seq_len(s)
    return cache.bm.build_tables([s], -(-n // BS))[0][0].tolist(), n


def last(rec, name):
    """The index of the last record of this name (-1: none)."""
    return max((i for i, e in enumerate(rec.log) if e[0] == name), default=-1)


def test_load_takes_the_bounds_of_every_block(kept, rec):
    kept.load(torch.zeros(NB, HKV, BS, D), torch.zeros(NB, HKV, BS, D))
    assert covered(rec.named("update")) == {i: BS for i in range(NB)}
    assert last(rec, "update") > last(rec, "reshape_and_cache")


def test_copies_move_the_bounds_with_their_blocks(kept):
    for i in range(NB):
        kept.key_bounds[i] = i
    kept.apply_copies([(0, 5), (1, 6), (5, 7), (2, 1), (NB, 3), (4, -1)])      # the last two are not blocks
    want = list(range(NB))
    want[5], want[6], want[7], want[1] = 0, 1, 0, 2
    assert kept.key_bounds[:, 0, 0, 0].tolist() == want


@pytest.mark.parametrize("n", [1, BS, BS + 1, 3 * BS])
def test_decode_steps_take_the_bounds_of_the_last_block(kept, rec, n):
    s = FakeStream("side")
    kept.bm.add_seq(0)
    kept.bm.append_n(0, n - 1)
    plan = kept.plan_step([0]).host_tensors(pin=False)
    q, kv = torch.zeros(1, HQ, D, dtype=BF), torch.zeros(1, HKV, D, dtype=BF)
    kept.step(q, kv, kv, plan, torch.empty_like(q), 0.1, stream=s)
    table, _ = seq_table(kept, 0)
    assert covered(rec.named("update")) == {table[(n - 1) // BS]: (n - 1) % BS + 1}
    assert rec.log[last(rec, "update")][1] is s and last(rec, "update") > last(rec, "step")


def test_prefill_steps_take_the_bounds_of_the_chunks_blocks(kept, rec):
    s = FakeStream("side")
    chunks, before = [BS + 3, 1, 0], [BS - 2, 0, 5]
    for i, n in enumerate(before):
        kept.bm.add_seq(i)
        kept.bm.append_n(i, n)
    plan = kept.plan_prefill([0, 1, 2], chunks)
    T = sum(chunks)
    q, kv = torch.zeros(T, HQ, D, dtype=BF), torch.zeros(T, HKV, D, dtype=BF)
    out = torch.empty_like(q)
    assert kept.prefill_step(q, kv, kv, plan.host_tensors(pin=False), out, 0.1, plan.max_query_len, s) is out
    t = [seq_table(kept, i)[0] for i in range(3)]
    assert covered(rec.named("update")) == {t[0][0]: BS, t[0][1]: BS, t[0][2]: 1, t[1][0]: 1}
    assert rec.log[last(rec, "update")][1] is s and last(rec, "update") > last(rec, "paged_prefill_step")


def test_swapped_in_sequences_get_their_bounds(kept, rec, monkeypatch):
    s = FakeStream("side")
    kept.bm = pkv.BlockManager(NB, BS, range(NB), num_host_blocks=8)
    kept.host_k = kept.host_v = None
    for i, n in enumerate([2 * BS + 1, 4]):
        kept.bm.add_seq(i)
        kept.bm.append_n(i, n)
    kept.swap_out([0, 1])
    assert not rec.named("update")
    kept.swap_in([0, 1], s)
    t = [seq_table(kept, i)[0] for i in range(2)]
    assert covered(rec.named("update")) == {t[0][0]: BS, t[0][1]: BS, t[0][2]: 1, t[1][0]: 4}
    assert rec.log[last(rec, "update")][1] is s and last(rec, "update") > last(rec, "swap_blocks")


def test_nothing_is_updated_where_no_bounds_are_kept(kept, rec):
    kept.key_bounds = None
    kept.load(torch.zeros(NB, HKV, BS, D), torch.zeros(NB, HKV, BS, D))
    kept.apply_copies([(0, 5)])
    kept.bm.add_seq(0)
    q, kv = torch.zeros(1, HQ, D, dtype=BF), torch.zeros(1, HKV, D, dtype=BF)
    kept.step(q, kv, kv, kept.plan_step([0]).host_tensors(pin=False), torch.empty_like(q), 0.1)
    assert not rec.named("update")


# ------------------------------------------------- refused before anything runs
class Launches:
    """The library with its packed calls and its block copy recorded, not run."""

    def __init__(self, lib):
        self.lib, self.ran = lib, []

    def __getattr__(self, name):
        if name == "pkv_bound_call":
            return lambda call, addr, n, stream: self.ran.append(call) or 0
        if name in ("copy_blocks", "paged_attention_prefill"):
            return lambda *a: self.ran.append(name) or 0
        return getattr(self.lib, name)


@pytest.fixture
def host_step(monkeypatch):
    """A cache whose steps take host tensors; what they would launch is recorded."""
    ran = Launches(library())
    monkeypatch.setattr(pkv, "load_library", lambda: ran)

    def host(t, what, contiguous=True):                    # the check of the device left out
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        return t

    monkeypatch.setattr(pkv, "_cuda", host)
    monkeypatch.setattr(pkv, "_current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_raw_stream", lambda idx: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream("current"))
    return ran


def prefill_args(D=128):
    """Host tensors of a prompt step of 2 sequences of 3 and 2 tokens."""
    B, T = 2, 5
    plan = {"pairs": torch.zeros(1, 2, dtype=I64), "slots": torch.zeros(T, dtype=I64),
            "tables": torch.zeros(B, 4, dtype=I32), "lens": torch.ones(B, dtype=I32),
            "query_start": torch.tensor([0, 3, 5], dtype=I32)}
    q, kv = torch.zeros(T, HQ, D, dtype=BF), torch.zeros(T, HKV, D, dtype=BF)
    return dict(q=q, k_new=kv, v_new=kv.clone(), dev_plan=plan, positions=torch.zeros(T, dtype=I32),
                first=torch.zeros(B, dtype=I32), rotary=engine.Rotary(torch.zeros(8, 2, D // 2)),
                out=torch.empty_like(q), scale=0.1, max_query_len=3)


def cache_of(D=D, dtype=BF, bs=BS):
    c = engine.PagedKVCache(NB, HQ, HKV, D, bs, dtype, range(NB), device="cpu")
    c.key_bounds = torch.zeros(pkv.key_bounds_shape(NB, HKV, D), dtype=pkv.key_bounds_dtype(dtype))
    return c


WS = torch.zeros(1 << 16, dtype=torch.uint8)


def fused(T, D):
    """q of a fused projection: rows of all heads."""
    return torch.zeros(T, HQ + 2 * HKV, D, dtype=BF)[:, :HQ]


@pytest.mark.parametrize("over", [
    dict(), dict(q=fused(2, D)), dict(workspace=WS[:64]), dict(workspace=None), dict(first_blocks=3),
    dict(scale=float("nan")), dict(out=torch.zeros(2, HQ, D)), dict(selected=torch.zeros(2, HQ, 2, dtype=I32)),
    dict(k_scale=2.0),
    dict(out=torch.zeros(2 * HQ * D + 1, dtype=BF)[1:].view(2, HQ, D)),       # rows not on 16 bytes
], ids=lambda o: "-".join(o) or "good")
def test_a_refused_sparse_step_has_run_nothing(host_step, over):
    a = step_args()
    a["dev_plan"]["pairs"] = torch.zeros(1, 2, dtype=I64)
    a.update(workspace=WS)
    a.update(over)
    if not over:
        cache_of().sparse_step(**a)
        assert host_step.ran == ["copy_blocks", 0, 1, 2, 3]
        return
    with pytest.raises((ValueError, TypeError, pkv.PagedKVError)):
        cache_of().sparse_step(**a)
    assert host_step.ran == []


@pytest.mark.parametrize("cache,over", [
    (dict(D=128), dict()), (dict(D=128), dict(q=fused(5, 128))), (dict(D=128), dict(scale=float("inf"))),
    (dict(D=128), dict(max_query_len=-1)), (dict(D=128), dict(out=torch.zeros(4, HQ, 128, dtype=BF))),
    (dict(D=128, dtype=torch.uint8), dict()), (dict(D=64), dict()),
    (dict(D=128), dict(out=torch.zeros(5 * HQ * 128 + 1, dtype=BF)[1:].view(5, HQ, 128))),
], ids=lambda o: "-".join(f"{k}" for k in o) or "none")
def test_a_refused_prefill_step_has_run_nothing(host_step, cache, over):
    """Caches that the prefill attention does not have among them: E4M3, heads of 64."""
    a = prefill_args(cache["D"])
    a.update(over)
    if cache == dict(D=128) and not over:
        cache_of(**cache).rotary_prefill_step(**a)
        assert host_step.ran == ["copy_blocks", 0, 1, 4]
        return
    with pytest.raises((ValueError, pkv.PagedKVError)):
        cache_of(**cache).rotary_prefill_step(**a)
    assert host_step.ran == []


def test_checked_calls_return_what_the_calls_return():
    """pkv_bound_check on good arguments and on one error of each kind, for each call."""
    lib, f32, at = library(), lambda x: np.float32(x).view(np.uint32).item(), ctypes.addressof
    sections = (ctypes.c_int32 * 1)(32)

    def check(call, *args):
        a = (ctypes.c_uint64 * len(args))(*[x & 0xffffffffffffffff for x in args])
        return lib.pkv_bound_check(call, at(a), len(a))

    P = 0x1000
    rotary = lambda q=P, R=64, cache=1, ks=1.0: check(
        0, 0x2000, q, *[P] * 7, at(sections), 1, 256, 256, 128, 128, 3, 4, 2, 64, R, 0, 16, 8, 64, 1, cache,
        f32(ks), f32(1.0))
    assert (rotary(), rotary(q=0), rotary(q=P + 8), rotary(R=24), rotary(cache=0), rotary(ks=2.0)) == \
        (0, -1, -1, -2, -2, -1)
    bounds = lambda k=P, D=64: check(1, k, *[P] * 4, 3, 5, 8, 2, D, 16, 1, 1)
    assert (bounds(), bounds(k=0), bounds(D=24)) == (0, -1, -2)
    select = lambda ws=P, n=1 << 20, D=64: check(2, *[P] * 5, 3, 5, 8, 4, 2, D, 16, 4, 1, 1, 1, ws, n)
    assert (select(), select(ws=0), select(n=64), select(D=96)) == (0, -1, -1, -2)
    sparse = lambda q=P, bs=16, kv=1: check(3, P, q, *[P] * 5, 3, 5, 8, 4, 4, 2, 64, bs, f32(0.1), 1, kv, f32(1.0),
                                            f32(1.0))
    assert (sparse(), sparse(q=P + 2), sparse(bs=48), sparse(kv=0)) == (0, -1, -2, -2)
    prefill = lambda q=P, B=3, n=7, Hq=4, D=128, bs=16, kv=1, scale=0.1, kp=P: check(
        4, P, q, kp, P, P, P, P, B, n, 5, 8, Hq, 2, D, bs, f32(scale), 1, kv)
    assert (prefill(), prefill(q=0), prefill(q=P + 8), prefill(kp=0), prefill(n=-1), prefill(Hq=3),
            prefill(scale=float("nan"))) == (0, -1, -1, -1, -1, -1, -1)
    assert (prefill(D=64), prefill(bs=48), prefill(kv=2)) == (-2, -2, -2)
    assert (prefill(B=0), prefill(n=0), prefill(B=0, kp=0), prefill(B=0, D=64)) == (0, 0, 0, -2)
    assert check(4, P) == -1 and check(5, P) == -1 and lib.pkv_bound_check(0, None, 28) == -1
