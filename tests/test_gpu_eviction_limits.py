"""The cache eviction operators where sizes, streams and orders are extreme: offsets past 2^31
elements and 2^32 bytes, calls at once on two streams, replays with rewritten inputs, scales of
zero and below, groups of any size, batches of empty sequences. Where a case only differs in place
from a small one (which blocks, which row, which part of q), its results are the small one's bits."""
import math

import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import eviction as oev

pytestmark = pytest.mark.gpu
BF, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
HKV, D, BS = 2, 128, 16


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    assert pkv.get_device_error() == 0
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


def pools(NB, dtype, hkv=HKV, d=D, bs=BS):
    ks, vs = pkv.pool_shapes(NB, hkv, bs, d, dtype)
    return torch.zeros(ks, dtype=dtype, device="cuda"), torch.zeros(vs, dtype=dtype, device="cuda")


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def decode_ws(B, Hq, d, bs, blocks):
    return torch.empty(pkv.weighed_decode_workspace_size(B, Hq, d, bs, blocks), dtype=U8, device="cuda")


def prompt_ws(B, Hq, most, window=0):
    return torch.empty(pkv.weigh_prefill_workspace_size(B, Hq, most, window), dtype=U8, device="cuda")


# ------------------------------------------------------------------------- offsets
@pytest.mark.parametrize("dtype", [BF, U8])
def test_blocks_past_four_gib(dtype):
    """Every operator with blocks at the end of pools of more than 2^32 bytes, against the same
    blocks at the beginning of small ones."""
    per = HKV * BS * D * (1 if dtype == U8 else 2)
    NB = (1 << 32) // per + 3000
    lens, K = [300, 33], 100
    tables = np.full((2, 20), -1, dtype=np.int32)
    tables[0, :19], tables[1, :3] = np.arange(19), np.arange(19, 22)
    fresh = np.arange(22, 36, dtype=np.int32).reshape(2, 7)
    n, used = 36, 36
    content = torch.randint(0, 120, (2, n * per), generator=gen(1), device="cuda", dtype=U8) if dtype == U8 else \
        randn(1, 2, n * per // 2).view(U8)
    q, k, v = randn(2, 2, 8, D), randn(3, 2, HKV, D), randn(4, 2, HKV, D)
    qc = randn(5, 20, 8, D)
    qw, kw = randn(6, D), randn(7, D)
    turns = randn(8, 400, 2, D // 2, dtype=F32)
    ks, vs = (0.05, 0.04) if dtype == U8 else (1.0, 1.0)

    def run(NB, move):
        kp, vp = pools(NB, dtype)
        at = move(np.arange(used))
        for pool, c in ((kp, content[0]), (vp, content[1])):
            pool.view(U8).view(NB, per)[torch.from_numpy(at).cuda()] = c.view(n, per)
        t = ints(np.where(tables < 0, -1, move(np.maximum(tables, 0))).tolist())
        f = ints(move(fresh).tolist())
        slots = torch.tensor([int(move(np.array(tables[b, (m - 1) // BS]))) * BS + (m - 1) % BS for b, m in enumerate(lens)],
                             dtype=I64, device="cuda")
        ln, W, out, q_out = ints(lens), torch.zeros(2, HKV, 320, device="cuda"), torch.empty_like(q), torch.empty_like(q)
        pkv.norm_rotary_and_cache(q_out, q, k, v, qw, kw, kp, vp, slots, ints([299, 32]), turns, k_scale=ks, v_scale=vs)
        pkv.paged_attention_decode_weighed(out, W, None, q, kp, vp, t, ln, 0.05, k_scale=ks, v_scale=vs,
                                           workspace=decode_ws(2, 8, D, BS, 20))
        if dtype == BF:
            pkv.weigh_prefill_tokens(W, None, qc, kp, t, ln, ints([0, 15, 20]), 0.05, 15, workspace=prompt_ws(2, 8, 15))
        kept = torch.empty(2, HKV, K, dtype=I32, device="cuda")
        pkv.select_tokens(kept, W, None, ln, 4, 8)
        pkv.keep_tokens(kept, W, None, kp, vp, t, f, ln)
        at = torch.from_numpy(at).cuda()
        return [q_out, out, W, kept] + [p.view(U8).view(NB, per)[at] for p in (kp, vp)]

    small = run(n, lambda x: x)
    big = run(NB, lambda x: NB - 1 - 61 * x)
    assert all(torch.equal(a, b) for a, b in zip(small, big))


def test_weight_rows_past_two_gi():
    """Rows of token weights at offsets of more than 2^31 elements."""
    max_tokens, rows = 1 << 20, 1100
    W = torch.empty(rows, HKV, max_tokens, device="cuda")
    assert W.numel() > 1 << 31
    small = torch.zeros(2, HKV, max_tokens, device="cuda")
    at = ints([rows - 1, rows - 3])
    W[rows - 3:].zero_()
    kp, vp = pools(40, BF)
    kp.copy_(randn(1, *kp.shape)), vp.copy_(randn(2, *vp.shape))
    tables, ln, q, qc = ints([list(range(20)), list(range(20, 40))]), ints([300, 200]), randn(3, 2, 8, D), randn(4, 20, 8, D)
    lists = []
    fresh = ints([[0], [1]])
    for w, r in ((small, None), (W, at)):
        k1, v1 = kp.clone(), vp.clone()
        pkv.paged_attention_decode_weighed(torch.empty_like(q), w, r, q, k1, v1, tables, ln, 0.1,
                                           workspace=decode_ws(2, 8, D, BS, 20))
        pkv.weigh_prefill_tokens(w, r, qc, k1, tables, ln, ints([0, 15, 20]), 0.1, 15, workspace=prompt_ws(2, 8, 15))
        kept = torch.empty(2, HKV, 16, dtype=I32, device="cuda")
        pkv.select_tokens(kept, w, r, ln, 2, 2)
        pkv.keep_tokens(kept, w, r, k1, v1, tables, fresh, ln)
        lists.append(kept)
    assert torch.equal(*lists)
    assert torch.equal(small[0], W[rows - 1]) and torch.equal(small[1], W[rows - 3])
    assert (W[rows - 2] == 0).all()


def test_logits_past_two_gi():
    """A workspace whose logits pass 2^31 elements: many sequences under wide tables."""
    B, Hq, blocks = 300, 8, 65536
    assert B * Hq * blocks * BS > 1 << 31
    kp, vp = pools(8, BF, 1)
    kp.copy_(randn(1, *kp.shape)), vp.copy_(randn(2, *vp.shape))
    q, ln = randn(3, B, Hq, D), torch.full((B,), 100, dtype=I32, device="cuda")
    ln[5] = 0
    narrow = torch.arange(7, dtype=I32, device="cuda").expand(B, 7).contiguous()
    wide = torch.full((B, blocks), -1, dtype=I32, device="cuda")
    wide[:, :7] = narrow
    got = []
    for t in (narrow, wide):
        W, out = torch.zeros(B, 1, t.shape[1] * BS, device="cuda"), torch.empty_like(q)
        pkv.paged_attention_decode_weighed(out, W, None, q, kp, vp, t, ln, 0.1, workspace=decode_ws(B, Hq, D, BS, t.shape[1]))
        got.append((out, W[:, :, :112].clone()))
    # the same sums in another order: float32 steps of numbers below 8 (weights), a bf16 step
    assert (got[0][1] - got[1][1]).abs().max() <= 8 * 128 * 2.0 ** -24
    assert (got[0][0].float() - got[1][0].float()).abs().max() <= 2.0 ** -7 * got[0][0].abs().max()
    assert (got[1][0][5] == 0).all()


def test_queries_past_two_gi():
    """Rows of q at offsets of more than 2^31 elements, in the append and in a prompt's chunk."""
    T, Hq = 135_000, 128
    assert (T - 8) * Hq * D > 1 << 31
    q = torch.zeros(T, Hq, D, dtype=BF, device="cuda")
    q[-8:] = randn(1, 8, Hq, D)
    k, v = torch.zeros(T, 1, D, dtype=BF, device="cuda"), torch.zeros(T, 1, D, dtype=BF, device="cuda")
    k[-8:], v[-8:] = randn(2, 8, 1, D), randn(3, 8, 1, D)
    qw, kw, turns = randn(4, D), randn(5, D), randn(6, 50, 2, D // 2, dtype=F32)
    tables, ln = ints([[0, 1, 2]]), ints([40])
    got = []
    for n in (8, T):
        kp, vp = pools(4, BF, 1)
        kp.copy_(randn(7, *kp.shape)), vp.copy_(randn(8, *vp.shape))
        slots = torch.full((n,), -1, dtype=I64, device="cuda")
        slots[-8:] = torch.arange(32, 40, device="cuda")
        pos = torch.zeros(n, dtype=I32, device="cuda")
        pos[-8:] = torch.arange(32, 40, device="cuda")
        q_out = torch.zeros_like(q[-n:])
        pkv.norm_rotary_and_cache(q_out, q[-n:], k[-n:], v[-n:], qw, kw, kp, vp, slots, pos, turns)
        W = torch.zeros(1, 1, 48, device="cuda")
        pkv.weigh_prefill_tokens(W, None, q_out, kp, tables, ln, ints([n - 8, n]), 0.1, 8, workspace=prompt_ws(1, Hq, 8))
        got.append((q_out[-8:].clone(), kp, vp, W))
        assert (q_out[:-8] == 0).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # a weight is off by twice its logit's error: (D + 16) steps of 2^-23 of magnitudes that add up to
    # less than 400, times the scale
    assert abs(float(got[0][3].sum()) - 8 * Hq) <= 8 * Hq * 2.0 ** -9


# ------------------------------------------------------------------------- streams and replays
class Batch:
    """A weighed step and a prompt's weights, with buffers of their own."""

    def __init__(self, seed, lens, chunks, Hq=8, window=0):
        self.lens, B, blocks = lens, len(lens), -(-max(lens) // BS)
        self.kp, self.vp = pools(B * blocks, BF)
        self.kp.copy_(randn(seed, *self.kp.shape)), self.vp.copy_(randn(seed + 1, *self.vp.shape))
        self.tables = torch.arange(B * blocks, dtype=I32, device="cuda").view(B, blocks)
        self.ln, self.q = ints(lens), randn(seed + 2, B, Hq, D)
        self.start = ints(np.concatenate([[0], np.cumsum(chunks)]).tolist())
        self.qc, self.most, self.window = randn(seed + 3, sum(chunks), Hq, D), max(chunks), window
        self.W, self.out = torch.zeros(B, HKV, blocks * BS, device="cuda"), torch.zeros_like(self.q)
        self.ws, self.wp = decode_ws(B, Hq, D, BS, blocks), prompt_ws(B, Hq, self.most, window)
        self.kept = torch.zeros(B, HKV, 40, dtype=I32, device="cuda")

    def step(self, stream=None):
        pkv.weigh_prefill_tokens(self.W, None, self.qc, self.kp, self.tables, self.ln, self.start, 0.1, self.most,
                                 self.window, 0.9, self.wp, stream=stream)
        pkv.paged_attention_decode_weighed(self.out, self.W, None, self.q, self.kp, self.vp, self.tables, self.ln, 0.1, 0.9,
                                           workspace=self.ws, stream=stream)
        pkv.select_tokens(self.kept, self.W, None, self.ln, 4, 4, stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.W, self.out, self.kept)]


def test_two_streams_at_once():
    a, b = Batch(10, [2000, 900, 77], [200, 900, 5]), Batch(20, [300] * 20, [30] * 20, window=8)
    for x in (a, b):
        x.step()
    want = [x.results() for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for x in (a, b):
            x.W.zero_()
        torch.cuda.synchronize()
        for x, s in zip((a, b), streams):
            x.step(s)
        for x, w in zip((a, b), want):
            assert all(torch.equal(p, q) for p, q in zip(x.results(), w))


@pytest.mark.parametrize("window", [0, 8])
def test_prompt_replayed_with_other_lengths(window):
    """A graph of the calls replayed with lengths, chunks and tables rewritten in place."""
    x = Batch(30, [1500, 700, 320], [60, 700, 8], window=window)
    x.step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.step()
    for lens, chunks in (([1500, 700, 320], [60, 700, 8]), ([33, 0, 1400], [33, 0, 700]), ([1, 2, 3], [0, 0, 0]),
                         ([999, 1000, 1001], [1, 2, 500])):
        x.ln.copy_(ints(lens))
        x.start.copy_(ints(np.concatenate([[0], np.cumsum(chunks)]).tolist()))
        x.tables.copy_(x.tables.flip(0))
        x.W.zero_(), x.out.zero_()
        x.step()
        want = x.results()
        x.W.zero_(), x.out.zero_(), x.kept.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(x.results(), want)), lens


def test_empty_batch_is_in_order():
    """Rows of an empty batch are zero for whatever follows on the stream: a step that is launched
    while the one before it ends sees them."""
    kp, vp = pools(4, BF)
    kp.copy_(randn(1, *kp.shape)), vp.copy_(randn(2, *vp.shape))
    B = 512
    q = randn(3, B, 8, D)
    tables, none, one = torch.zeros(B, 1, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda"), \
        torch.full((B,), 16, dtype=I32, device="cuda")
    W, out, out2 = torch.zeros(B, HKV, BS, device="cuda"), torch.empty_like(q), torch.empty_like(q)
    ws, ws2 = decode_ws(B, 8, D, BS, 1), decode_ws(B, 8, D, BS, 1)
    want = torch.empty_like(q)
    pkv.paged_attention_decode_weighed(want, W, None, torch.zeros_like(q), kp, vp, tables, one, 0.1, workspace=ws)
    for _ in range(50):
        out.fill_(math.nan)
        pkv.paged_attention_decode_weighed(out, W, None, q, kp, vp, tables, none, 0.1, workspace=ws)
        pkv.paged_attention_decode_weighed(out2, W, None, out, kp, vp, tables, one, 0.1, workspace=ws2)
        assert torch.equal(out2, want)


# ------------------------------------------------------------------------- scales and groups
@pytest.mark.parametrize("dtype,group", [(BF, 1), (BF, 4), (U8, 1), (U8, 8), (F32, 2)])
def test_decode_scales_of_zero_and_below(dtype, group):
    act = F32 if dtype == F32 else BF
    kp, vp = pools(12, dtype)
    for i, p in enumerate((kp, vp)):
        if dtype == U8:
            p.copy_(torch.randint(0, 120, p.shape, generator=gen(i), device="cuda", dtype=U8))
        else:
            p.copy_(randn(i, *p.shape, dtype=dtype))
    ks, vs = (0.01, 0.02) if dtype == U8 else (1.0, 1.0)
    tables, ln, q = ints([list(range(12))]), ints([177]), randn(3, 1, HKV * group, D, dtype=act)

    def run(q, scale):
        W, out = torch.zeros(1, HKV, 192, device="cuda"), torch.empty_like(q)
        pkv.paged_attention_decode_weighed(out, W, None, q, kp, vp, tables, ln, scale, 1.0, ks, vs,
                                           decode_ws(1, HKV * group, D, BS, 12))
        return out, W

    a, b = run(q, -0.1), run(-q, 0.1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    out, W = run(q, 0.0)
    even = group / 177
    assert (W[:, :, :177] - even).abs().max() <= even * 2.0 ** -18 and (W[:, :, 177:] == 0).all()
    _, vv = pkv.pool_views(kp, vp)
    assert torch.isfinite(out).all()


def test_prompt_scales_of_zero_and_below():
    x = Batch(40, [300, 140], [20, 140])

    def run(q, scale):
        W = torch.zeros_like(x.W)
        pkv.weigh_prefill_tokens(W, None, q, x.kp, x.tables, x.ln, x.start, scale, x.most, workspace=x.wp)
        return W

    assert torch.equal(run(x.qc, -0.1), run(-x.qc, 0.1))
    # a scale of zero: every token that a query sees has the same weight, of each of 4 heads
    W = run(x.qc, 0.0).cpu().numpy()
    for b, (n, c) in enumerate(((300, 20), (140, 140))):
        want = np.zeros(x.W.shape[2])
        for i in range(c):
            want[:n - c + i + 1] += 4.0 / (n - c + i + 1)
        assert np.abs(W[b] - want).max() <= 2.0 ** -16 * want.max()
    tiny = run(x.qc, 2.0 ** -100).cpu().numpy()
    assert np.abs(tiny - W).max() <= 2.0 ** -16 * W.max()


@pytest.mark.parametrize("G,Hkv", [(3, 2), (7, 1), (48, 1), (127, 1), (128, 2)])
def test_prompt_groups_of_any_size(G, Hkv):
    """Rows of a tile that belong to many queries, a query's heads in two tiles, padding rows."""
    d, lens, chunks = 64, [190, 60, 0, 33], [9, 60, 0, 1]
    kp, vp = pools(40, BF, Hkv, d)
    kp.copy_(randn(1, *kp.shape))
    views, _ = pkv.pool_views(kp, vp)
    views = views.double().cpu().numpy()
    tables = np.random.default_rng(G).permutation(40)[:4 * 12 - 8].reshape(4, 10)
    tables = np.concatenate([tables, np.full((4, 2), -1)], 1).astype(np.int32)
    tables[0, 10:12] = [tables[1, 8], tables[1, 9]]
    q = randn(2, sum(chunks), G * Hkv, d)
    start = np.concatenate([[0], np.cumsum(chunks)])
    W = torch.full((4, Hkv, 192), 3.0, device="cuda")
    for window in (0, 2):
        W.fill_(3.0)
        pkv.weigh_prefill_tokens(W, None, q, kp, torch.from_numpy(tables).cuda(), ints(lens), ints(start.tolist()), 0.125, 60,
                                 window, 0.5, workspace=prompt_ws(4, G * Hkv, 60, window))
        got, qd = W.double().cpu().numpy(), q.double().cpu().numpy()
        for b, (n, c) in enumerate(zip(lens, chunks)):
            w = min(window or c, c)
            for h in range(Hkv):
                want = np.full(192, 3.0)
                if c:
                    t = np.arange(n)
                    k = views[tables[b][t // BS], h, t % BS]
                    p = oev.prompt_weights(qd[start[b + 1] - w:start[b + 1], h * G:(h + 1) * G], k, 0.125).sum((0, 1))
                    want[:n] = oev.updated(want, p, c, 0.5)
                # a weight is off by twice its logit's error: 80 steps of 2^-23 of magnitudes that add up to
                # less than 100, times the scale: 2^-12
                assert (np.abs(got[b, h] - want) <= 2.0 ** -9 * want + 1e-30).all(), (b, h, np.abs(got[b, h] - want).max())


def test_prompt_of_many_sequences():
    """More sequences than a warp's lanes, empty chunks among them, rows in any order."""
    B = 75
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 200, B)]
    chunks = [int(rng.integers(0, n + 1)) if i % 3 else 0 for i, n in enumerate(lens)]
    kp, vp = pools(B * 13, BF)
    kp.copy_(randn(1, *kp.shape))
    tables = torch.arange(B * 13, dtype=I32, device="cuda").view(B, 13)
    q = randn(2, sum(chunks), 4, D)
    start = np.concatenate([[0], np.cumsum(chunks)])
    rows = ints(rng.permutation(B).tolist())
    W = torch.zeros(B, HKV, 208, device="cuda")
    pkv.weigh_prefill_tokens(W, rows, q, kp, tables, ints(lens), ints(start.tolist()), 0.1, max(chunks),
                             workspace=prompt_ws(B, 4, max(chunks)))
    for b in range(B):                                     # each one alone
        one = torch.zeros(1, HKV, 208, device="cuda")
        n = chunks[b]
        if n == 0:
            assert (W[rows[b]] == 0).all()
            continue
        pkv.weigh_prefill_tokens(one, None, q[start[b]:start[b + 1]], kp, tables[b:b + 1], ints(lens[b:b + 1]), ints([0, n]),
                                 0.1, max(1, n), workspace=prompt_ws(1, 4, max(1, n)))
        # the same weights, added in another order
        assert (one[0] - W[rows[b]]).abs().max() <= 2.0 ** -18 * max(1.0, float(one.max()))


def test_rotary_with_one_norm_is_refused():
    from paged_kv_cache_259_gb300.engine import PagedKVCache, Rotary
    cache = PagedKVCache(8, 4, 2, 128, 16, BF, list(range(8)), "cuda")
    cache.k_pool.zero_()
    cache.bm.add_seq(0)
    plan = cache.plan_step([0]).device_tensors("cuda")
    q, k, v = randn(1, 1, 4, 128), randn(2, 1, 2, 128), randn(3, 1, 2, 128)
    cache.enable_token_weights(1, 16)
    rows, before = cache.weight_rows([0]), q.clone()
    rot = Rotary(randn(4, 10, 2, 64, dtype=F32), q_norm=randn(5, 128))
    with pytest.raises(TypeError):
        cache.weighed_step(q, k, v, plan, rows, torch.empty_like(q), 0.1, cache.weighed_workspace(1, plan["tables"].shape[1]),
                           positions=ints([0]), rotary=rot)
    assert torch.equal(q, before) and (cache.k_pool == 0).all()
