"""bm_plan_keep and the engine's eviction plans on the host: blocks taken and released, all or
nothing, sharing, prefix caching, swapping."""
import ctypes

import numpy as np
import pytest
import torch

from _lib import library, pkv
from paged_kv_cache_259_gb300 import engine

BS = 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    return library()


def manager(blocks=20, **kw):
    return pkv.BlockManager(blocks, BS, list(range(blocks)), **kw)


def filled(bm, lens):
    for s, n in enumerate(lens):
        bm.add_seq(s)
        bm.append_n(s, n)


def state(bm, ids):
    return ([bm.block_table(s) for s in ids], [bm.seq_len(s) for s in ids], bm.free_list(),
            [bm.refcount(b) for b in range(bm.num_blocks)], [bm.is_kept(s) for s in ids])


def test_fresh_blocks_come_before_the_old_ones_return():
    bm = manager()
    filled(bm, [13, 9])                                    # blocks 0-3, 4-6
    tables, lens, kept = bm.plan_keep([1, 0], 6)
    assert tables.tolist() == [[4, 5, 6, -1], [0, 1, 2, 3]] and lens.tolist() == [9, 13]
    assert kept.tolist() == [[7, 8], [9, 10]]
    assert bm.block_table(0) == [9, 10] and bm.block_table(1) == [7, 8]
    assert bm.seq_len(0) == bm.seq_len(1) == 6
    assert bm.free_list() == list(range(11, 20)) + [4, 5, 6, 0, 1, 2, 3]
    assert bm.is_kept(0) and bm.is_kept(1)
    slot, cow = bm.append_slot(0)                          # goes on behind the kept tokens
    assert (slot, cow) == (10 * BS + 2, None)
    bm.free_seq(0)
    bm.free_seq(1)
    assert sorted(bm.free_list()) == list(range(20))


def test_one_token_kept_and_a_whole_number_of_blocks():
    bm = manager()
    filled(bm, [2, 9])
    assert bm.plan_keep([0], 1)[2].tolist() == [[4]] and bm.seq_len(0) == 1
    assert bm.plan_keep([1], 8)[2].shape == (1, 2) and bm.seq_len(1) == 8
    assert bm.append_slot(1)[0] % BS == 0                  # a new block


def test_shared_blocks_stay_with_the_others():
    bm = manager()
    filled(bm, [10])
    bm.fork(0, 1)
    bm.plan_keep([0], 5)
    assert bm.block_table(1) == [0, 1, 2] and [bm.refcount(b) for b in range(3)] == [1, 1, 1]
    assert not bm.is_kept(1) and bm.is_kept(0)
    assert bm.append_slot(1) == (2 * BS + 2, None)         # the child owns its last block alone now
    bm.fork(0, 2)
    assert bm.is_kept(2)                                   # a fork of what has dropped tokens


@pytest.mark.parametrize("ids,kept,status", [
    ([0, 9], 3, -4), ([0, 0], 3, -1), ([0], 13, -1), ([0], 14, -1), ([1, 0], 9, -1), ([0], 0, -1), ([0, 1, 2], 8, -5),
    ([2, 3], 3, -1),
])
def test_refusals_change_nothing(ids, kept, status):
    bm = manager(17, num_host_blocks=4)
    filled(bm, [13, 9, 20, 4])                             # 4 + 3 + 5 + 1 blocks: 4 left
    bm.swap_out(3)                                         # and 5
    before = state(bm, [0, 1, 2])
    with pytest.raises(pkv.PagedKVError) as e:
        bm.plan_keep(ids, kept, max_blocks=8)
    assert e.value.status == status
    assert state(bm, [0, 1, 2]) == before


def test_narrow_buffers_and_bad_arguments():
    bm = manager()
    filled(bm, [13])
    before = state(bm, [0])
    for kw in (dict(max_blocks=3), dict(max_blocks=1)):
        with pytest.raises(pkv.PagedKVError):
            bm.plan_keep([0], 5, **kw)
    i32 = lambda n: (ctypes.c_int32 * n)()
    one = (ctypes.c_int64 * 1)(0)
    lib = library()
    assert lib.bm_plan_keep(bm._h, one, 1, 5, 4, 1, i32(4), i32(1), i32(1)) == -1     # two blocks
    assert lib.bm_plan_keep(bm._h, None, 1, 5, 4, 2, i32(4), i32(1), i32(2)) == -1
    assert lib.bm_plan_keep(bm._h, one, 1, 5, 4, 2, None, i32(1), i32(2)) == -1
    assert lib.bm_plan_keep(bm._h, one, -1, 5, 4, 2, i32(4), i32(1), i32(2)) == -1
    assert lib.bm_plan_keep(None, one, 1, 5, 4, 2, i32(4), i32(1), i32(2)) == -1
    assert lib.bm_plan_keep(bm._h, None, 0, 5, 4, 2, None, None, None) == 0
    assert lib.bm_is_kept(bm._h, 7, (ctypes.c_int * 1)()) == -4
    assert state(bm, [0]) == before


def test_prefix_caching_registers_nothing_behind_kept_tokens():
    bm = manager(prefix_caching=True)
    prompt = list(range(100, 111))
    assert bm.add_seq_prompt(0, prompt) == 0
    bm.append_tokens(0, prompt)
    assert bm.cache_stats()[2] == 2                        # two full blocks of known tokens
    bm.plan_keep([0], 3)
    bm.append_tokens(0, list(range(50, 64)))               # fills four blocks
    assert bm.cache_stats()[2:] == (2, 2)                  # the old ones, evictable; no new one
    assert bm.add_seq_prompt(1, prompt) == 8               # and still found
    bm.free_seq(0)
    bm.free_seq(1)
    assert bm.num_free() + bm.cache_stats()[3] == 20


def test_fresh_blocks_may_be_evicted_ones():
    bm = manager(6, prefix_caching=True)
    bm.add_seq_prompt(0, list(range(8)))
    bm.append_tokens(0, list(range(8)))
    bm.free_seq(0)                                         # two cached, evictable
    filled(bm, [])
    bm.add_seq(1)
    bm.append_n(1, 15)                                     # the four others
    tables, _, kept = bm.plan_keep([1], 5)
    assert sorted(kept[0]) == [0, 1] and sorted(tables[0]) == [2, 3, 4, 5]
    assert bm.cache_stats()[2:] == (0, 0)


def test_swapped_and_back():
    bm = manager(num_host_blocks=8)
    filled(bm, [13])
    bm.plan_keep([0], 6)
    bm.swap_out(0)
    with pytest.raises(pkv.PagedKVError):
        bm.plan_keep([0], 2)
    bm.swap_in(0)
    assert bm.seq_len(0) == 6 and bm.is_kept(0)


# --------------------------------------------------------------------- the engine
def cache(**kw):
    return engine.PagedKVCache(20, 4, 2, 64, 16, torch.bfloat16, range(20), device="cpu", **kw)


def test_engine_plans_only_what_has_outgrown_the_budget():
    c = cache()
    for s, n in enumerate((40, 32, 33)):
        c.bm.add_seq(s)
        c.bm.append_n(s, n)
    plan = c.plan_keep([0, 1, 2, 2], 32)
    assert plan.seq_ids.tolist() == [0, 2] and plan.lens.tolist() == [40, 33] and plan.kept_tables.shape == (2, 2)
    assert c.plan_keep([0, 1, 2], 32) is None
    t = plan.device_tensors("cpu")
    assert t["kept_tables"].tolist() == [c.bm.block_table(0), c.bm.block_table(2)]


def test_engine_does_not_recompute_what_dropped_tokens():
    c = cache()
    for s in (0, 1):
        c.bm.add_seq(s)
        c.bm.append_n(s, 40)
    c.plan_keep([1], 16)
    free = c.bm.free_list()
    with pytest.raises(ValueError, match="swap it out"):
        c.preempt_by_recompute([0, 1])
    assert c.bm.free_list() == free and c.bm.seq_len(0) == 40
    assert c.preempt_by_recompute([0]) == {0: 40}


class NoStream:
    def __init__(self, *a):
        pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        pass


def test_engine_weight_rows(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", NoStream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    c = cache()
    with pytest.raises(RuntimeError, match="enable"):
        c.weight_rows([0])
    W = c.enable_token_weights(3, 50)
    assert W.shape == (3, 2, 52) and c.enable_token_weights(3, 50) is W
    W.fill_(7.0)
    rows = c.weight_rows([5, 6, 5]).tolist()
    assert rows[0] == rows[2] != rows[1] and (W[rows] == 0).all()
    W[rows[0]] = 3.0
    assert c.weight_rows([5]).tolist() == rows[:1] and (W[rows[0]] == 3).all()      # kept
    with pytest.raises(RuntimeError, match="rows free"):
        c.weight_rows([7, 8])
    assert c.fork_weight_row(5, 7).tolist() != rows[:1] and (W == 3).all(-1).all(-1).sum() == 2
    c.drop_weight_rows([5, 99])
    assert c.weight_rows([8]).tolist() == rows[:1] and (W[rows[0]] == 0).all()
