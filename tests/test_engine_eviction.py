"""The engine's side of caches of bounded size, on the host: what its calls are given and what it
refuses before anything changes, with the library's calls recorded instead of run."""
import numpy as np
import pytest
import torch

from _lib import library
from paged_kv_cache_259_gb300 import engine

NB, HQ, HKV, D, BS = 80, 4, 2, 64, 16
BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


class NoStream:
    def __init__(self, *a):
        pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        pass


@pytest.fixture
def calls(monkeypatch):
    """(name, arguments) of the library's calls that a step binds and runs; no streams."""
    library()
    monkeypatch.setattr(torch.cuda, "stream", NoStream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    log = []
    for name in ("copy_blocks", "reshape_and_cache", "rotary_and_cache", "norm_rotary_and_cache", "update_key_bounds",
                 "paged_attention_decode_weighed", "weigh_prefill_tokens", "select_tokens", "keep_tokens",
                 "paged_attention_prefill", "select_blocks", "paged_attention_decode_sparse"):
        monkeypatch.setattr(engine, "bind_" + name, lambda *a, name=name: lambda s=None: log.append((name, a)))
    return log


def cache(head_dim=D, block_size=BS, num_blocks=NB, **kw):
    return engine.PagedKVCache(num_blocks, HQ, HKV, head_dim, block_size, BF, range(num_blocks), device="cpu", **kw)


def filled(c, lens):
    for s, n in enumerate(lens):
        c.bm.add_seq(s)
        c.bm.append_n(s, n)


def rows_of(n):
    q, kv = torch.zeros(n, HQ, D, dtype=BF), torch.zeros(n, HKV, D, dtype=BF)
    return q, kv, kv.clone()


# ------------------------------------------------- rows of token weights of any size
@pytest.mark.parametrize("block_size", [16, 32])
@pytest.mark.parametrize("max_tokens", [1, 50, 1000, 1024])
@pytest.mark.parametrize("max_seqs", [1, 3])
def test_rows_hold_the_whole_blocks_of_the_longest_sequence(calls, max_tokens, block_size, max_seqs):
    """The calls want a place for every slot of the table; a sequence of max_tokens has that
    many rounded up to whole blocks."""
    c = cache(block_size=block_size)
    W = c.enable_token_weights(max_seqs, max_tokens)
    assert W.shape == (max_seqs, HKV, -(-max_tokens // 4) * 4) and c.enable_token_weights(9, 9) is W
    filled(c, [max_tokens - 1])
    plan = c.plan_step([0], group_prefixes=False)
    assert plan.lens.tolist() == [max_tokens]
    dev, rows = plan.device_tensors("cpu"), c.weight_rows([0])
    q, k, v = rows_of(1)
    c.weighed_step(q, k, v, dev, rows, torch.empty_like(q), 0.1, None)
    c.weigh_prompt(q, dict(dev, query_start=torch.zeros(2, dtype=I32)), rows, 0.1, 1, None)
    given = [a[{"paged_attention_decode_weighed": 1, "weigh_prefill_tokens": 0}[name]] for name, a in calls
             if name != "reshape_and_cache"]
    if max_tokens > 1:
        keep = c.plan_keep([0], 1)
        c.keep_step(keep.device_tensors("cpu"), rows, 1)
        given += [a[1] for name, a in calls[-2:]]
        assert keep.tables.shape == plan.tables.shape
    assert len(given) == (4 if max_tokens > 1 else 2)
    for t in given:
        assert t.is_contiguous() and t.shape[2] >= plan.tables.shape[1] * block_size
        t[:, :, 0] = 5.0
        assert (W[:, :, 0] == 5).all()                     # the same weights
        t.zero_()


def test_a_fork_copies_the_whole_row(calls):
    c = cache()
    c.enable_token_weights(2, 50)
    c.weight_rows([0])
    c.weight_storage.fill_(3.0)
    c.fork_weight_row(0, 1)
    assert (c.weight_storage == 3).all()
    c.drop_weight_rows([1])
    c.weight_rows([2])
    assert (c.weight_storage[1] == 0).all()


# ------------------------------------------------------------- evictions as planned
@pytest.mark.parametrize("other", [16, 31, 33, 40, 0])
def test_another_number_than_the_plan_has_is_refused(calls, other):
    """The manager counts the planned tokens: fewer would leave slots that nobody filled."""
    c = cache()
    c.enable_token_weights(2, 128)
    filled(c, [100, 70])
    plan = c.plan_keep([0, 1], 32)
    dev, rows = plan.device_tensors("cpu"), c.weight_rows([0, 1])
    with pytest.raises(ValueError, match="num_kept"):
        c.keep_step(dev, rows, other)
    assert calls == []
    kept = c.keep_step(dev, rows, 32)                      # the plan still stands
    assert kept.shape == (2, HKV, 32) and [name for name, _ in calls] == ["select_tokens", "keep_tokens"]


def host_state(c, ids):
    return (c.bm.free_list(), [(c.bm.block_table(s), c.bm.seq_len(s), c.bm.is_kept(s)) for s in ids])


@pytest.mark.parametrize("first,last", [(33, 0), (0, 33), (20, 13), (-1, 5), (5, -1), (1 << 31, 1 << 31)])
def test_ends_that_cannot_be_kept_are_refused_before_the_plan(calls, first, last):
    c = cache()
    c.enable_token_weights(2, 128)
    filled(c, [100, 70])
    before = host_state(c, [0, 1])
    with pytest.raises(ValueError, match="first_tokens"):
        c.plan_keep([0, 1], 32, first, last)
    assert host_state(c, [0, 1]) == before and c.plan_keep([0, 1], 32, 20, 12) is not None


@pytest.mark.parametrize("head_dim,block_size", [(24, 16), (528, 16), (64, 24), (64, 8)])
def test_a_cache_that_cannot_be_moved_is_refused_before_the_plan(calls, head_dim, block_size):
    c = cache(head_dim=head_dim, block_size=block_size)
    filled(c, [100])
    before = host_state(c, [0])
    with pytest.raises(ValueError, match="multiples of 16"):
        c.plan_keep([0], 32)
    assert host_state(c, [0]) == before


def test_a_sequence_longer_than_its_weights_is_refused_before_the_plan(calls):
    c = cache()
    c.enable_token_weights(2, 50)                          # whole blocks: 64
    filled(c, [64, 65])
    before = host_state(c, [0, 1])
    with pytest.raises(ValueError, match="token weights"):
        c.plan_keep([0, 1], 32)
    assert host_state(c, [0, 1]) == before
    assert c.plan_keep([0], 32).lens.tolist() == [64]


def test_the_plans_ends_are_those_of_the_step(calls):
    c = cache()
    c.enable_token_weights(1, 128)
    filled(c, [100])
    dev, rows = c.plan_keep([0], 32, 4, 20).device_tensors("cpu"), c.weight_rows([0])
    c.keep_step(dev, rows, 32)
    c.keep_step(dev, rows, 32, 1, 2)
    c.keep_step(dev, rows, 32, last_tokens=7)
    assert [a[4:] for name, a in calls if name == "select_tokens"] == [(4, 20), (1, 2), (4, 7)]


# ----------------------------------------------------------------- beam search
def beams(c, n, rows):
    """n beams of one prompt; those in ``rows`` have token weights, all 10 + their number."""
    c.bm.add_seq(0)
    c.bm.append_n(0, 20)
    for s in range(1, n):
        c.bm.fork(0, s)
    for s in rows:
        c.weight_storage[c.weight_rows([s]).tolist()] = 10.0 + s


@pytest.mark.parametrize("parents", [[0, 1, 2, 3], [3, 2, 1, 0], [1, 1, 1, 1], [2, 0, 2, 0], [0, 0, 3, 3], [2], []])
@pytest.mark.parametrize("max_seqs", [4, 7])
def test_new_beams_take_their_parents_weights(calls, parents, max_seqs):
    """With no more rows than there are beams, too."""
    c = cache()
    W = c.enable_token_weights(max_seqs, 50)
    beams(c, 4, range(4))
    new = list(range(10, 10 + len(parents)))
    c.bm.beam_step(range(4), parents, new)
    rows = c.beam_weight_rows(range(4), parents, new)
    assert rows.dtype == I32 and len(set(rows.tolist())) == len(new)
    assert rows.tolist() == c.weight_rows(new).tolist()
    for r, p in zip(rows.tolist(), parents):
        assert (c.weight_storage[r] == 10 + p).all() and (W[r] == 10 + p).all()
    left = c.weight_rows(range(20, 20 + max_seqs - len(new)))      # the old beams' rows are free
    assert sorted(rows.tolist() + left.tolist()) == list(range(max_seqs))


def test_beams_without_weights_and_ids_used_before(calls):
    c = cache()
    c.enable_token_weights(4, 50)
    beams(c, 3, [1])
    c.weight_storage[c.weight_rows([11]).tolist()] = 7.0           # of a sequence that is long gone
    c.bm.beam_step(range(3), [1, 0, 1], [10, 11, 12])
    rows = c.beam_weight_rows(range(3), [1, 0, 1], [10, 11, 12]).tolist()
    assert [c.weight_storage[r].unique().tolist() for r in rows] == [[11.0], [0.0], [11.0]]
    assert len(c.weight_rows([30])) == 1 and len(set(rows)) == 3


def test_beams_are_handed_over_all_or_none(calls):
    c = cache()
    c.enable_token_weights(3, 50)
    beams(c, 2, range(2))
    c.weight_rows([9])
    before = c.weight_storage.clone(), c.weight_rows([0, 1, 9]).tolist()
    with pytest.raises(RuntimeError, match="rows free"):
        c.beam_weight_rows([0, 1], [0, 0, 1], [10, 11, 12])
    for old, parents, new in (([0, 1], [0], [10, 11]), ([0, 1], [2], [10]), ([0, 1], [-1], [10]), ([0, 1], [0, 1], [10, 10]),
                              ([0, 1], [0], [1]), ([0, 0], [0], [10])):
        with pytest.raises(ValueError):
            c.beam_weight_rows(old, parents, new)
    assert torch.equal(c.weight_storage, before[0]) and c.weight_rows([0, 1, 9]).tolist() == before[1]
    with pytest.raises(RuntimeError, match="enable"):
        cache().beam_weight_rows([0], [0], [1])


# ------------------------------------------------------------- steps that rotate
def test_a_rotated_step_without_a_rotary_is_refused(calls, monkeypatch):
    """Only a weighed step has a form without the rotation: the others would attend with
    unrotated keys."""
    monkeypatch.setattr(engine.PagedKVCache, "enable_key_bounds", lambda self, stream=None: None)
    c = cache()
    filled(c, [30])
    plan = c.plan_step([0], group_prefixes=False).device_tensors("cpu")
    q, k, v = rows_of(1)
    pos = torch.zeros(1, dtype=I32)
    with pytest.raises(TypeError, match="rotary"):
        c.rotary_prefill_step(q, k, v, dict(plan, query_start=torch.zeros(2, dtype=I32)), pos, pos, None, q, 0.1, 1)
    with pytest.raises(TypeError, match="rotary"):
        c.sparse_step(q, k, v, plan, pos, pos, None, torch.zeros(1, HKV, 2, dtype=I32), q, 0.1)
    assert calls == []
    c.enable_token_weights(1, 64)
    c.weighed_step(q, k, v, plan, c.weight_rows([0]), q, 0.1, None)
    assert [name for name, _ in calls] == ["reshape_and_cache", "paged_attention_decode_weighed"]


@pytest.mark.parametrize("what", ["dtype", "aligned k", "aligned v"])
def test_an_unrotated_step_checks_its_append_before_the_copies(calls, what):
    c = cache()
    filled(c, [20])
    c.bm.fork(0, 1)
    c.enable_token_weights(2, 64)
    plan = c.plan_step([0, 1], group_prefixes=False)
    assert len(plan.pairs) == 1                            # a copy of the shared block
    q, k, v = rows_of(2)
    odd = torch.zeros(2 * HKV * D + 1, dtype=BF)[1:].view(2, HKV, D)
    bad = {"dtype": (k.float(), v.float()), "aligned k": (odd, v), "aligned v": (k, odd)}[what]
    dev, rows = plan.device_tensors("cpu"), c.weight_rows([0, 1])
    with pytest.raises((TypeError, ValueError)):
        c.weighed_step(q, *bad, dev, rows, q, 0.1, None)
    assert calls == []
    c.weighed_step(q, k, v, dev, rows, q, 0.1, None)
    assert [name for name, _ in calls] == ["copy_blocks", "reshape_and_cache", "paged_attention_decode_weighed"]


def test_an_unrotated_step_of_an_e4m3_cache_takes_either_type(calls):
    c = engine.PagedKVCache(NB, HQ, HKV, D, BS, torch.uint8, range(NB), device="cpu")
    filled(c, [20])
    c.enable_token_weights(1, 64)
    plan, rows = c.plan_step([0], group_prefixes=False).device_tensors("cpu"), c.weight_rows([0])
    q, k, v = rows_of(1)
    c.weighed_step(q, k, v, plan, rows, q, 0.1, None)
    c.weighed_step(q, k.float(), v.float(), plan, rows, q, 0.1, None)
    with pytest.raises(TypeError):
        c.weighed_step(q, k.half(), v.half(), plan, rows, q, 0.1, None)
    assert len(calls) == 4


def test_an_unrotated_step_without_rows_is_refused_as_the_binding_does(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", NoStream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    c = cache()
    filled(c, [20])
    c.enable_token_weights(1, 64)
    plan, rows = c.plan_step([0], group_prefixes=False).device_tensors("cpu"), c.weight_rows([0])
    q, k, v = rows_of(1)
    for bad in ((None, v), (k, None)):
        with pytest.raises(TypeError, match="must be a tensor"):
            c.weighed_step(q, *bad, plan, rows, q, 0.1, None)
