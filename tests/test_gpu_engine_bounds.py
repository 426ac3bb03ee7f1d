"""The engine's key bounds on a GPU: whatever order a user's calls come in, the bounds
of every block that a sparse step scores are those of its filled slots (exact)."""
import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import attention as oatt
from oracle import long_context as olc
from paged_kv_cache_259_gb300 import engine

pytestmark = pytest.mark.gpu
BF, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
HQ, HKV, D, BS = 8, 2, 128, 16


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


def new_cache(NB=80, cache=BF, seed=0, **over):
    return engine.PagedKVCache(NB, HQ, HKV, D, BS, cache, np.random.default_rng(seed).permutation(NB), "cuda", **over)


def values(rng, *shape, dtype=BF):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def rotary():
    return engine.Rotary(pkv.rotary_table(4096, D, device="cuda"))


def sparse_step(cache, ids, rng, K=4, act=BF, stream=None):
    """One sparse decode step of the sequences; checks its choice of blocks against the
    oracle on bounds taken from the pool's own values."""
    plan = cache.plan_step(ids, group_prefixes=False)
    q, k, v = (values(rng, len(ids), h, D, dtype=act).cuda() for h in (HQ, HKV, HKV))
    sel = torch.empty(len(ids), HKV, K, dtype=I32, device="cuda")
    ws = cache.select_workspace(len(ids), plan.tables.shape[1])
    args = (plan.device_tensors("cuda"), torch.from_numpy((plan.lens - 1).astype(np.int32)).cuda(),
            torch.from_numpy(engine.first_changed(plan)).cuda(), rotary(), sel, torch.empty_like(q), D ** -0.5)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    cache.sparse_step(q, k, v, *args, first_blocks=1, last_blocks=1, workspace=ws, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    check_bounds(cache, plan.tables, plan.lens)
    want = olc.select_blocks(q.double().cpu().numpy(), cache.key_bounds.double().cpu().numpy(), plan.tables,
                             plan.lens, BS, HKV, K, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)
    assert pkv.get_device_error() == 0
    return plan


def check_bounds(cache, tables, lens):
    k = oatt.widen(cache.k_view().cpu()).reshape(cache.num_blocks, HKV, BS, D)
    got = cache.key_bounds.double().cpu().numpy()
    for row, L in zip(tables, lens):
        for j in range(-(-int(L) // BS)):
            for h in range(HKV):
                assert np.array_equal(got[row[j], h], olc.key_bounds(k[row[j], h], min(BS, L - j * BS))), (j, h)


def filled(cache, lens, rng, **load):
    """Sequences of these lengths over values loaded into every slot."""
    cache.load(*(values(rng, cache.num_blocks, HKV, BS, D, dtype=F32 if cache.k_pool.dtype == U8 else cache.k_pool.dtype)
                 for _ in range(2)), **load)
    for s, n in enumerate(lens):
        cache.bm.add_seq(s)
        cache.bm.append_n(s, n)
    return list(range(len(lens)))


@pytest.mark.parametrize("cache", [BF, U8, F32])
@pytest.mark.parametrize("side", [False, True])
def test_sparse_step_on_a_cache_filled_without_bounds(cache, side):
    """The first sparse step takes the bounds of all that is cached, on its own stream
    (the current one kept busy)."""
    rng = np.random.default_rng(1)
    c = new_cache(cache=cache)
    ids = filled(c, [300, 161, 16, 15, 1], rng)
    s = torch.cuda.Stream() if side else None
    if side:
        torch.cuda.synchronize()
        x = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            x = x @ x
    sparse_step(c, ids, rng, act=F32 if cache == F32 else BF, stream=s)
    sparse_step(c, ids[1:], rng, act=F32 if cache == F32 else BF, stream=s)


def test_bounds_of_a_pool_of_more_blocks_than_one_launch_row():
    """70,000 blocks: the second row of the launch is shorter."""
    NB = 70000
    c = engine.PagedKVCache(NB, 1, 1, 16, 16, BF, range(NB), "cuda")
    c.k_pool.normal_()
    kb = c.enable_key_bounds()
    k = c.k_view()
    want = torch.stack([k.float().amin(2), k.float().amax(2)], 2)
    assert torch.equal(kb.float(), want)


def decode_args(cache, ids, rng):
    plan = cache.plan_step(ids, group_prefixes=False)
    q, k, v = (values(rng, len(ids), h, D).cuda() for h in (HQ, HKV, HKV))
    return plan, (q, k, v, plan.device_tensors("cuda"), torch.empty_like(q), D ** -0.5)


@pytest.mark.parametrize("side", [False, True])
def test_bounds_follow_every_write_of_the_cache(side):
    """Prompts, decode steps, copies, swapping and loads between sparse steps: each
    sparse step's choice is the oracle's on the pool's own values."""
    rng = np.random.default_rng(2)
    s = torch.cuda.Stream() if side else None
    c = new_cache(num_host_blocks=40)
    c.enable_key_bounds()
    for i in range(3):
        c.bm.add_seq(i)
    chunks = [130, 47, 16]
    plan = c.plan_prefill([0, 1, 2], chunks)
    q, k, v = (values(rng, sum(chunks), h, D).cuda() for h in (HQ, HKV, HKV))
    torch.cuda.synchronize()
    c.prefill_step(q, k, v, plan.device_tensors("cuda"), torch.empty_like(q), D ** -0.5, plan.max_query_len, s)
    torch.cuda.synchronize()
    check_bounds(c, plan.tables, plan.lens)
    sparse_step(c, [0, 1, 2], rng, stream=s)
    c.bm.fork(0, 7)                                        # the next step copies its last block
    for _ in range(18):                                    # over a block border
        plan, a = decode_args(c, [0, 1, 2, 7], rng)
        torch.cuda.synchronize()
        c.step(*a, workspace=c.workspace(4, plan.tables.shape[1]), stream=s)
        torch.cuda.synchronize()
    check_bounds(c, plan.tables, plan.lens)
    sparse_step(c, [0, 1, 2, 7], rng, stream=s)
    torch.cuda.synchronize()
    c.swap_out([0, 2], s)
    c.swap_in([2, 0], s)
    torch.cuda.synchronize()
    sparse_step(c, [0, 1, 2], rng, stream=s)
    torch.cuda.synchronize()
    c.swap_out([1], copy_engines=True)
    c.swap_in([1], copy_engines=True)
    sparse_step(c, [1, 7], rng)
    c.load(*(values(rng, c.num_blocks, HKV, BS, D) for _ in range(2)))
    sparse_step(c, [0, 1, 2, 7], rng, stream=s)
    torch.cuda.synchronize()
    table = c.bm.build_tables([0], 12)[0][0]
    c.apply_copies([(int(table[1]), int(table[2])), (int(table[2]), int(table[3]))], stream=s)
    sparse_step(c, [0], rng, stream=s)


def test_bounds_follow_a_live_decode_pipeline():
    rng = np.random.default_rng(3)
    c = new_cache()
    ids = filled(c, [60, 31, 200], rng)
    c.enable_key_bounds()
    q, k, v = (values(rng, 3, h, D) for h in (HQ, HKV, HKV))
    pipe = engine.LiveDecodePipeline(c, ids, q, k, v, torch.empty_like(q), 16, group_prefixes=False)
    outs = [torch.empty_like(q).pin_memory() for _ in range(6)]
    ws = c.workspace(3, 16)
    for i in range(6):
        views = pipe.host_inputs()
        for name, h in (("q", HQ), ("k_new", HKV), ("v_new", HKV)):
            views[name].copy_(values(rng, 3, h, D))
        _, done = pipe.submit(outs[i], D ** -0.5, workspace=ws)
        assert pipe.last_counts[0] == 0 and pipe.last_plan_us > 0
    done.synchronize()
    tables, lens = c.bm.build_tables(ids, 16)
    assert list(lens) == [66, 37, 206]
    check_bounds(c, tables, lens)
    sparse_step(c, ids, rng)


def test_a_refused_step_leaves_q_and_the_cache_as_they_were():
    """q as a view of a fused projection, and a workspace that is too small: refused before
    q is turned in place, so the step can be tried again."""
    rng = np.random.default_rng(4)
    c = new_cache()
    ids = filled(c, [200, 90], rng)
    c.enable_key_bounds()
    plan = c.plan_step(ids, group_prefixes=False)
    x = values(rng, 2, HQ + 2 * HKV, D).cuda()
    q, k, v = x.split([HQ, HKV, HKV], 1)
    sel, out = torch.empty(2, HKV, 4, dtype=I32, device="cuda"), torch.zeros(2, HQ, D, dtype=BF, device="cuda")
    a = (plan.device_tensors("cuda"), torch.from_numpy((plan.lens - 1).astype(np.int32)).cuda(),
         torch.from_numpy(engine.first_changed(plan)).cuda(), rotary(), sel, out, D ** -0.5)
    ws = c.select_workspace(2, plan.tables.shape[1])
    before = [t.clone() for t in (x, c.k_pool, c.v_pool, c.key_bounds)]
    for q_, kw in ((q, dict(workspace=ws)), (q.contiguous(), dict(workspace=ws[:64])), (q.contiguous(), {})):
        keep = q_.clone()
        with pytest.raises((ValueError, pkv.PagedKVError)):
            c.sparse_step(q_, k, v, *a, **kw)
        torch.cuda.synchronize()
        assert torch.equal(q_, keep)
    assert all(torch.equal(t, b) for t, b in zip((x, c.k_pool, c.v_pool, c.key_bounds), before))
    q = q.contiguous()
    c.sparse_step(q, k, v, *a, workspace=ws)               # k and v as views
    check_bounds(c, plan.tables, plan.lens)
    assert pkv.get_device_error() == 0 and bool(out.any())


def test_a_refused_prompt_step_leaves_q_and_the_cache_as_they_were():
    rng = np.random.default_rng(5)
    c = new_cache(cache=U8)                                # the prefill attention has bf16 caches
    c.load(*(values(rng, c.num_blocks, HKV, BS, D, dtype=F32) for _ in range(2)))
    c.bm.add_seq(0)
    plan = c.plan_prefill([0], [40])
    q, k, v = (values(rng, 40, h, D).cuda() for h in (HQ, HKV, HKV))
    before = [t.clone() for t in (q, c.k_pool, c.v_pool)]
    with pytest.raises(pkv.PagedKVError):
        c.rotary_prefill_step(q, k, v, plan.device_tensors("cuda"), torch.arange(40, dtype=I32, device="cuda"),
                              torch.zeros(1, dtype=I32, device="cuda"), rotary(), torch.empty_like(q), 0.1, 40)
    torch.cuda.synchronize()
    assert all(torch.equal(t, b) for t, b in zip((q, c.k_pool, c.v_pool), before))


def test_a_captured_sparse_step_replays():
    """The engine's sparse step captured once and replayed for three steps of one batch,
    its plan, positions and inputs rewritten in place; the same steps run eagerly."""
    rng = np.random.default_rng(6)
    runs = []
    for graph in (False, True):
        step_rng = np.random.default_rng(7)
        c = new_cache(seed=3)
        ids = filled(c, [300, 161, 31], np.random.default_rng(8))
        c.enable_key_bounds()
        width, B = 24, len(ids)
        dev = {"pairs": torch.empty(0, 2, dtype=I64, device="cuda"), "slots": torch.empty(B, dtype=I64, device="cuda"),
               "tables": torch.empty(B, width, dtype=I32, device="cuda"), "lens": torch.empty(B, dtype=I32, device="cuda")}
        q, k, v = (torch.empty(B, h, D, dtype=BF, device="cuda") for h in (HQ, HKV, HKV))
        pos, first = (torch.empty(B, dtype=I32, device="cuda") for _ in range(2))
        sel, out = torch.empty(B, HKV, 5, dtype=I32, device="cuda"), torch.empty_like(q)
        ws, rot, g = c.select_workspace(B, width), rotary(), None
        results = []
        for _ in range(3):
            plan = c.plan_step(ids, width, group_prefixes=False)
            for name in ("slots", "tables", "lens"):
                dev[name].copy_(torch.from_numpy(getattr(plan, name)))
            for t, h in ((q, HQ), (k, HKV), (v, HKV)):
                t.copy_(values(step_rng, B, h, D))
            pos.copy_(torch.from_numpy((plan.lens - 1).astype(np.int32)))
            first.copy_(pos)
            run = lambda: c.sparse_step(q, k, v, dev, pos, first, rot, sel, out, D ** -0.5, workspace=ws)
            if graph and g is None:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    run()
            g.replay() if graph else run()
            torch.cuda.synchronize()
            check_bounds(c, plan.tables, plan.lens)
            results.append([t.clone() for t in (q, sel, out)])
        runs.append(results)
    for a, b in zip(*runs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert pkv.get_device_error() == 0
