"""The engine with caches of bounded size where its limits are: rows of token weights of any
number of tokens, used to the last one, each step against float64 on the pool's own values."""
import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import eviction as oev
from test_gpu_engine_eviction import Loop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def on_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


def loop(max_tokens, max_seqs=6, **kw):
    """A serving loop whose rows of token weights hold ``max_tokens``."""
    x = Loop(**kw)
    x.c.token_weights = None
    x.c.enable_token_weights(max_seqs, max_tokens)
    assert x.c.token_weights.shape[2] == -(-max_tokens // 4) * 4
    return x


@pytest.mark.parametrize("max_tokens", [50, 97, 99])
def test_every_token_that_the_rows_hold(max_tokens):
    """Prompts and steps up to max_tokens, which end inside a block, and an eviction from there."""
    x = loop(max_tokens, seed=max_tokens)
    x.prompts([0, 1], [max_tokens, max_tokens - 3], 8)
    for _ in range(3):
        x.decode([1])
    assert x.c.bm.seq_len(0) == x.c.bm.seq_len(1) == max_tokens
    x.evict([0, 1], 20, 2, 5)
    for _ in range(max_tokens - 20):
        x.decode([1, 0])
    assert x.c.bm.seq_len(0) == max_tokens
    x.evict([1], 33, 0, 1)
    assert pkv.get_device_error() == 0


def test_refused_eviction_changes_nothing_and_can_be_repeated():
    x = loop(128, seed=1, bounds=True)
    x.prompts([0, 1], [100, 61], 0)
    c = x.c
    rows = c.weight_rows([0, 1])
    before, weights = [x.cached(s) for s in (0, 1)], c.token_weights.cpu().numpy()
    dev = c.plan_keep([0, 1], 32, 3, 8).device_tensors("cuda")
    pools = [t.clone() for t in (c.k_pool, c.v_pool, c.weight_storage, c.key_bounds)]
    for bad in (dict(num_kept=31), dict(first_tokens=30), dict(last_tokens=-1), dict(rows=rows[:1]), dict(rows=rows.long()),
                dict(kept=torch.empty(2, 2, 31, dtype=torch.int32, device="cuda")),
                dict(kept=torch.empty(2, 2, 32, device="cuda")), dict(dev_plan=dict(dev, kept_tables=dev["kept_tables"][:, :1].contiguous()))):
        a = dict(dev_plan=dev, rows=rows, num_kept=32)
        a.update(bad)
        with pytest.raises((ValueError, TypeError, pkv.PagedKVError)):
            c.keep_step(**a)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pools, (c.k_pool, c.v_pool, c.weight_storage, c.key_bounds)))
    kept = c.keep_step(dev, rows, 32).cpu().numpy()
    for b, s in enumerate((0, 1)):
        k, v = x.cached(s)
        for h in range(2):
            t = kept[b, h]
            assert t.tolist() == oev.select(weights[c._weight_rows[s], h], len(before[b][0][h]), 32, 3, 8)
            assert np.array_equal(k[h], before[b][0][h, t]) and np.array_equal(v[h], before[b][1][h, t])
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("side", [False, True])
def test_beam_search_at_a_budget(side):
    """Beams hand their token weights on; with no row more than there are beams."""
    x = loop(96, max_seqs=3, seed=11 + side, stream=torch.cuda.Stream() if side else None)
    x.prompts([0], [41], 4)
    ids = [0, 1, 2]
    for s in ids[1:]:
        x.c.bm.fork(0, s)
        x.c.fork_weight_row(0, s, x.stream)
        x.pos[s], x.W[s] = x.pos[0], x.W[0].copy()
    for step, parents in enumerate(([0, 1, 2], [2, 2, 0], [1, 0, 1], [0, 0, 0], [2, 1, 0])):
        for _ in range(4):
            x.decode(ids, decay=0.99)
        new = [100 * (step + 1) + i for i in range(3)]
        x.c.bm.beam_step(ids, parents, new)
        rows = x.c.beam_weight_rows(ids, parents, new, x.stream)
        torch.cuda.synchronize()
        assert rows.tolist() == x.c.weight_rows(new).tolist()
        for p, s in zip(parents, new):
            x.pos[s], x.W[s] = x.pos[ids[p]], x.W[ids[p]].copy()
            x.check_weights(s)
        ids = new
        if step % 2:
            x.evict(ids, 40, 2, 6)
    x.decode(ids)
    assert pkv.get_device_error() == 0
