"""The engine with caches of bounded size: prompts with normalised and rotated heads, their token
weights, decode steps that add to them, evictions, forks and swapping between, each step against
float64 on the pool's own values."""
import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import attention as oatt
from oracle import eviction as oev
from oracle import fp8_e4m3 as ofp8
from oracle import long_context as olc
from paged_kv_cache_259_gb300 import engine

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS = 8, 2, 128, 16
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
SCALE = D ** -0.5


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


class Loop:
    """A serving loop's state and its float64 shadow: the weights of every sequence."""

    def __init__(self, cache=BF, blocks=64, norm=True, seed=0, stream=None, bounds=False):
        self.rng = np.random.default_rng(seed)
        self.c = engine.PagedKVCache(blocks, HQ, HKV, D, BS, cache, range(blocks), "cuda", num_host_blocks=32)
        self.c.k_pool.zero_()
        self.c.v_pool.zero_()
        self.ks, self.vs = (0.02, 0.02) if cache == U8 else (1.0, 1.0)
        self.c.enable_token_weights(6, 512)
        if bounds:
            self.c.enable_key_bounds()
        w = [torch.from_numpy(1 + 0.2 * self.rng.standard_normal(D)).to(BF).cuda() for _ in range(2)]
        self.rotary = engine.Rotary(pkv.rotary_table(2048, D, device="cuda"), q_norm=w[0] if norm else None,
                                    k_norm=w[1] if norm else None)
        self.pos, self.W, self.stream = {}, {}, stream

    def rows(self, n):
        x = torch.from_numpy(self.rng.standard_normal((n, HQ + 2 * HKV, D)).astype(np.float32)).to(BF).cuda()
        q, k, v = x.split([HQ, HKV, HKV], 1)
        torch.cuda.synchronize()
        return q.contiguous(), k, v

    def cached(self, sid):
        """K and V ``[Hkv, L, D]`` of a sequence as the pool holds them."""
        out = []
        t = np.arange(self.c.bm.seq_len(sid))
        table = np.asarray(self.c.bm.block_table(sid))
        for view, scale in ((self.c.k_view(), self.ks), (self.c.v_view(), self.vs)):
            x = view.cpu()
            f = ofp8.e4m3_decode(x.numpy()) * float(np.float32(scale)) if x.dtype == U8 else oatt.widen(x)
            out.append(f[table[t // BS], :, t % BS].transpose(1, 0, 2))
        return out

    def check_weights(self, sid):
        got = self.c.token_weights[self.c._weight_rows[sid]].double().cpu().numpy()
        n = self.c.bm.seq_len(sid)
        # sums of weights of at most 1 each; a logit's error of D + 16 float32 steps of about 64, twice
        assert np.allclose(got[:, :n], self.W[sid], rtol=2e-4, atol=1e-6), np.abs(got[:, :n] - self.W[sid]).max()

    def prompts(self, ids, lens, window):
        for s in ids:
            if s not in self.pos:
                self.c.bm.add_seq(s)
                self.pos[s] = 0
                self.W[s] = np.zeros((HKV, 0))
        plan = self.c.plan_prefill(ids, lens)
        pos = np.concatenate([self.pos[s] + np.arange(n) for s, n in zip(ids, lens)]).astype(np.int32)
        q, k, v = self.rows(sum(lens))
        dev, out = plan.device_tensors("cuda"), torch.empty_like(q)
        rows = self.c.weight_rows(ids, self.stream)
        ws = self.c.weigh_workspace(len(ids), plan.max_query_len, window)
        first = torch.from_numpy(engine.first_changed(plan)).cuda()
        positions = torch.from_numpy(pos).cuda()
        torch.cuda.synchronize()
        self.c.rotary_prefill_step(q, k, v, dev, positions, first, self.rotary, out, SCALE, plan.max_query_len, self.stream)
        self.c.weigh_prompt(q, dev, rows, SCALE, plan.max_query_len, ws, window=window, stream=self.stream)
        torch.cuda.synchronize()
        qf, at = oatt.widen(q.cpu()), 0
        for s, n in zip(ids, lens):
            kf, _ = self.cached(s)
            L, w = kf.shape[1], min(window or n, n)
            G = HQ // HKV
            new = []
            for h in range(HKV):
                p = oev.prompt_weights(qf[at + n - w:at + n, h * G:(h + 1) * G], kf[h], SCALE).sum((0, 1))
                before = np.concatenate([self.W[s][h], np.zeros(n)])
                new.append(oev.updated(before, p, n, 1.0))
            self.W[s] = np.stack(new)
            assert self.W[s].shape[1] == L
            self.pos[s] += n
            at += n
            self.check_weights(s)

    def decode(self, ids, decay=1.0, rotated=True):
        plan = self.c.plan_step(ids, group_prefixes=False)
        q, k, v = self.rows(len(ids))
        dev, out = plan.device_tensors("cuda"), torch.empty_like(q)
        rows = self.c.weight_rows(ids, self.stream)
        ws = self.c.weighed_workspace(len(ids), plan.tables.shape[1])
        pos = torch.tensor([self.pos[s] for s in ids], dtype=I32).cuda()
        first = torch.from_numpy(engine.first_changed(plan)).cuda()
        torch.cuda.synchronize()
        self.c.weighed_step(q, k, v if rotated else v.contiguous(), dev, rows, out, SCALE, ws, decay, positions=pos, first=first,
                            rotary=self.rotary, k_scale=self.ks, v_scale=self.vs, stream=self.stream)
        torch.cuda.synchronize()
        qf, of, G = oatt.widen(q.cpu()), oatt.widen(out.cpu()), HQ // HKV
        for b, s in enumerate(ids):
            kf, vf = self.cached(s)
            new = []
            for h in range(HKV):
                p = oev.decode_weights(qf[b, h * G:(h + 1) * G], kf[h], SCALE)
                ref = p @ vf[h]
                assert np.all(np.abs(of[b, h * G:(h + 1) * G] - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + 1e-3)
                new.append(oev.updated(np.concatenate([self.W[s][h], [0.0]]), p.sum(0), 1, decay))
            self.W[s] = np.stack(new)
            self.pos[s] += 1
            self.check_weights(s)
        assert pkv.get_device_error() == 0

    def evict(self, ids, budget, first, last):
        before = {s: self.cached(s) for s in ids}
        weights = {s: self.c.token_weights[self.c._weight_rows[s]].cpu().numpy() for s in ids}
        lens = {s: self.c.bm.seq_len(s) for s in ids}
        plan = self.c.plan_keep(ids, budget)
        over = [s for s in ids if lens[s] > budget]
        assert (plan is None) == (not over)
        if plan is None:
            return
        assert plan.seq_ids.tolist() == over
        dev, rows = plan.device_tensors("cuda"), self.c.weight_rows(over, self.stream)
        torch.cuda.synchronize()
        kept = self.c.keep_step(dev, rows, budget, first, last, stream=self.stream)
        torch.cuda.synchronize()
        assert pkv.get_device_error() == 0
        for b, s in enumerate(over):
            new = []
            k, v = self.cached(s)
            for h in range(HKV):
                t = kept[b, h].cpu().numpy()
                assert t.tolist() == oev.select(weights[s][h], lens[s], budget, first, last)
                assert np.array_equal(k[h], before[s][0][h, t]) and np.array_equal(v[h], before[s][1][h, t])
                new.append(self.W[s][h, t])
            self.W[s] = np.stack(new)
            self.check_weights(s)
        for s in set(ids) - set(over):
            assert np.array_equal(self.cached(s)[0], before[s][0])

    def check_bounds(self):
        k = oatt.widen(self.c.k_view().cpu())
        got = self.c.key_bounds.double().cpu().numpy()
        for s in self.pos:
            for j, blk in enumerate(self.c.bm.block_table(s)):
                n = min(BS, self.c.bm.seq_len(s) - j * BS)
                for h in range(HKV):
                    assert np.array_equal(got[blk, h], olc.key_bounds(k[blk, h], n))


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("window", [0, 8])
def test_loop_at_a_budget(side, window):
    """Prompts longer and shorter than the budget, then decode steps with an eviction whenever a
    sequence is a block over it."""
    x = Loop(stream=torch.cuda.Stream() if side else None, bounds=True, seed=window)
    x.prompts([0, 1, 2], [150, 30, 97], window)
    x.evict([0, 1, 2], 64, 4, 16)
    x.check_bounds()
    for step in range(40):
        x.decode([0, 1, 2] if step % 3 else [2, 0], decay=1.0 if step % 2 else 0.98)
        if max(x.c.bm.seq_len(s) for s in (0, 1, 2)) >= 64 + BS:
            x.evict([0, 1, 2], 64, 4, 16)
            x.check_bounds()
    assert x.pos[0] == 150 + 40 and x.c.bm.seq_len(0) <= 64 + BS
    x.prompts([1], [21], window)                           # another turn of a conversation
    x.decode([0, 1])


@pytest.mark.parametrize("cache", [BF, U8])
def test_loop_forks_and_swaps(cache):
    x = Loop(cache=cache, norm=False, seed=3)
    for s, n in ((0, 45), (1, 70)):
        x.c.bm.add_seq(s)
        x.pos[s], x.W[s] = 0, np.zeros((HKV, 0))
        for _ in range(n // 15):
            x.decode([s])
    x.c.bm.fork(0, 2)
    x.c.fork_weight_row(0, 2)
    x.pos[2], x.W[2] = x.pos[0], x.W[0].copy()
    x.decode([0, 1, 2])                                    # copy-on-write of the shared block
    x.c.swap_out([1])
    for _ in range(16):
        x.decode([2, 0])
    x.evict([0, 2], 12, 1, 3)
    torch.cuda.synchronize()
    x.c.swap_in([1])
    x.decode([1, 2, 0])
    x.c.bm.free_seq(2)
    x.c.drop_weight_rows([2])
    x.evict([0], 1, 0, 1)
    x.decode([0, 1])


def test_step_captured_and_replayed():
    """A weighed step in a graph, its plan rewritten in place between replays."""
    x = Loop(seed=9)
    x.prompts([0, 1], [33, 50], 4)
    c = x.c
    plan = c.plan_step([0, 1], max_blocks=8, group_prefixes=False)
    dev = plan.device_tensors("cuda")
    q, k, v = x.rows(2)
    q0, out = q.clone(), torch.empty_like(q)
    rows, ws = c.weight_rows([0, 1]), c.weighed_workspace(2, 8)
    pos = torch.tensor([x.pos[0], x.pos[1]], dtype=I32).cuda()
    first = torch.from_numpy(engine.first_changed(plan)).cuda()
    run = lambda: c.weighed_step(q, k, v, dev, rows, out, SCALE, ws, positions=pos, first=first, rotary=x.rotary)
    before = c.token_weights.clone()
    torch.cuda.synchronize()
    run()
    torch.cuda.synchronize()
    want = out.clone(), c.token_weights.clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    q.copy_(q0)
    c.token_weights.copy_(before)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(c.token_weights, want[1])
    # the next step, through the same graph
    plan = c.plan_step([0, 1], max_blocks=8, group_prefixes=False)
    assert not len(plan.pairs)
    for name, t in plan.device_tensors("cuda").items():
        if name != "pairs":
            dev[name].copy_(t)
    pos += 1
    first += 1
    q.copy_(q0)
    g.replay()
    torch.cuda.synchronize()
    after = out.clone(), c.token_weights.clone()
    q.copy_(q0)
    c.token_weights.copy_(want[1])
    run()
    torch.cuda.synchronize()
    assert torch.equal(out, after[0]) and torch.equal(c.token_weights, after[1])
    assert pkv.get_device_error() == 0


def test_refused_step_changes_nothing():
    x = Loop(seed=5)
    x.prompts([0], [40], 0)
    c = x.c
    plan = c.plan_step([0], group_prefixes=False)
    dev = plan.device_tensors("cuda")
    q, k, v = x.rows(1)
    rows, pos = c.weight_rows([0]), torch.tensor([40], dtype=I32).cuda()
    first = torch.from_numpy(engine.first_changed(plan)).cuda()
    kept = q.clone(), c.k_pool.clone(), c.token_weights.clone()
    bad = [dict(decay=1.5), dict(workspace=torch.empty(64, dtype=U8, device="cuda")), dict(scale=float("nan"))]
    for over in bad:
        a = dict(scale=SCALE, workspace=c.weighed_workspace(1, plan.tables.shape[1]), decay=1.0)
        a.update(over)
        with pytest.raises((ValueError, pkv.PagedKVError)):
            c.weighed_step(q, k, v, dev, rows, torch.empty_like(q), a["scale"], a["workspace"], a["decay"], positions=pos,
                           first=first, rotary=x.rotary)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, (q, c.k_pool, c.token_weights)))
