"""The cache eviction operators on a GPU against the oracle (float64), at the sizes, masks and
orders where they can go wrong. Tolerances count the roundings that are made: see ``logit_error``
and each check."""
import math

import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import attention as oatt
from oracle import eviction as oev
from oracle import fp8_e4m3 as ofp8
from oracle import long_context as olc

pytestmark = pytest.mark.gpu
BF, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
KINDS = {"f32": (F32, F32), "bf16": (BF, BF), "e4m3": (BF, U8), "f32-e4m3": (F32, U8)}
KS, VS = 0.05, 0.04                                        # E4M3 scales
OUT_OF_RANGE = -4
U = 2.0 ** -24                                             # half a float32 step
HALF = {F32: 2.0 ** -24, BF: 2.0 ** -8}


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


def rng_of(*key):
    return np.random.default_rng([abs(int(k)) for k in key])


def normal(rng, shape, dtype, by=1.0):
    return torch.from_numpy((by * rng.standard_normal(shape)).astype(np.float32)).to(dtype)


def random_views(rng, NB, Hkv, bs, D, cache):
    def one(scale):
        x = rng.standard_normal((NB, Hkv, bs, D)).astype(np.float32)
        return torch.from_numpy(ofp8.e4m3_quantize(x, scale)) if cache == U8 else torch.from_numpy(x).to(cache)
    return one(KS), one(VS)


def values(view, scale):
    """A plain cache view as float64 values."""
    if view.dtype == U8:
        return ofp8.e4m3_decode(view.numpy()) * float(np.float32(scale))
    return oatt.widen(view)


def tables_of(rng, lens, bs, NB, width=None):
    blocks = [-(-n // bs) for n in lens]
    t = np.full((len(lens), width or max(1, max(blocks))), -1, dtype=np.int32)
    ids = rng.permutation(NB)
    at = 0
    for b, n in enumerate(blocks):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, ids[at:]


def rows_of(view, table, h, n, bs):
    t = np.arange(n)
    return view[table[t // bs], h, t % bs]


def cuda(x):
    return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()


def weights_of(rng, rows, Hkv, cap):
    return np.exp(2 * rng.standard_normal((rows, Hkv, cap))).astype(np.float32)


# ---------------------------------------------------------- norm_rotary_and_cache
def norm_case(kind, T, Hq, Hkv, D, bs, R, axes, interleaved, how, per_head, seed=0, f32_weights=False, eps=1e-6):
    rng = rng_of(seed, T, D, R, Hq)
    act, cache = KINDS[kind]
    NB = -(-(T + 8) // bs) + 3
    P = 97
    if how == "random":
        slots = rng.permutation(NB * bs)[:T].astype(np.int64)
        slots[rng.random(T) < 0.15] = -1
    else:
        at = np.arange(T) + 3
        slots = rng.permutation(NB)[at // bs].astype(np.int64) * bs + at % bs
    pos = rng.integers(0, P, (axes, T)).astype(np.int32)
    half = R // 2
    sections = [half] if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    table = rng.standard_normal((P, 2, half)).astype(np.float32)
    gain = np.exp(rng.standard_normal((Hq + 2 * Hkv, 1)))
    x = torch.from_numpy((rng.standard_normal((T, Hq + 2 * Hkv, D)) * gain).astype(np.float32)).to(act)
    wt = F32 if f32_weights else act
    qw, kw = (normal(rng, (h, D) if per_head else (D,), wt) for h in (Hq, Hkv))
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    return dict(x=x, Hq=Hq, Hkv=Hkv, qw=qw, kw=kw, kv=kv, vv=vv, slots=slots, pos=pos, sections=sections, table=table,
                act=act, cache=cache, interleaved=interleaved, bs=bs, eps=eps,
                scales=(KS, VS) if cache == U8 else (1.0, 1.0))


def norm_gpu(c, strided=False, in_place=False, stream=None, x=None):
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    split = [c["Hq"], c["Hkv"], c["Hkv"]]
    q, k, v = (c["x"] if x is None else x).cuda().split(split, 1)
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = q if in_place else torch.full(q.shape, 7.0, dtype=c["act"], device="cuda")
    pos = c["pos"][0] if len(c["pos"]) == 1 else c["pos"]
    pkv.norm_rotary_and_cache(q_out, q, k, v, c["qw"].cuda(), c["kw"].cuda(), kp, vp, cuda(c["slots"]), cuda(pos),
                              cuda(c["table"]), eps=c["eps"], sections=c["sections"], interleaved=c["interleaved"],
                              k_scale=c["scales"][0], v_scale=c["scales"][1], stream=stream)
    return q_out, kp, vp


def check_norm(c, q_out, kp, vp, untouched=None):
    """Against float64: the result's own rounding, and the float32 steps before it -- the sum of D
    squares (each partial sum one rounding, log2 of them deep where the lanes meet: D / 16 + 40 is
    above any of the orders), a root (2 steps), two products, and the rotation's three: all relative
    to the pair's magnitude."""
    live = c["slots"] >= 0
    cos, sin = olc.turns(c["pos"], c["table"], c["sections"])
    D = c["x"].shape[2]
    R = 2 * cos.shape[1]
    steps = (D / 16 + 40) * U
    a, b = olc.pair_dims(R, c["interleaved"])

    def expect(x, w):
        y = oev.normed(oatt.widen(x), oatt.widen(w), c["eps"])
        size = np.abs(y).copy()                            # what the rotation's steps are relative to
        both = np.abs(y[..., a]) + np.abs(y[..., b])
        both *= np.maximum(np.abs(cos), np.abs(sin))[:, None]
        size[..., a], size[..., b] = both, both
        return olc.rotate_f64(y, cos, sin, c["interleaved"]), size * steps

    q_ref, q_slack = expect(c["x"][:, :c["Hq"]], c["qw"])
    got = oatt.widen(q_out.cpu())
    assert (np.abs(got - q_ref) <= HALF[c["act"]] * np.abs(q_ref) * (1 + 2 * HALF[c["act"]]) + q_slack + 1e-38)[live].all()
    if untouched is not None:
        assert (got[~live] == untouched[~live]).all()
    k_view, v_view = (t.cpu() for t in pkv.pool_views(kp, vp))
    s = c["slots"][live]
    at = (s // c["bs"], slice(None), s % c["bs"])
    k_ref, k_slack = expect(c["x"][:, c["Hq"]:c["Hq"] + c["Hkv"]], c["kw"])
    k_ref, k_slack = k_ref[live], k_slack[live]
    if c["cache"] == U8:
        scale = float(np.float32(c["scales"][0]))
        want = np.clip(k_ref / scale, -448, 448)
        have = ofp8.e4m3_decode(k_view.numpy())[at]
        assert (np.abs(have - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + k_slack / scale).all()
        v_want = torch.from_numpy(ofp8.e4m3_quantize(c["x"].float().numpy()[live][:, c["Hq"] + c["Hkv"]:], c["scales"][1]))
    else:
        have = oatt.widen(k_view)[at]
        half = HALF[c["cache"]]
        assert (np.abs(have - k_ref) <= half * np.abs(k_ref) * (1 + 2 * half) + k_slack + 1e-38).all()
        v_want = c["x"][live][:, c["Hq"] + c["Hkv"]:].to(c["cache"])
    assert torch.equal(v_view[at], v_want)
    # nothing else was written
    rest = torch.ones(k_view.shape[0], k_view.shape[2], dtype=torch.bool)
    rest[s // c["bs"], s % c["bs"]] = False
    for view, before in ((k_view, c["kv"]), (v_view, c["vv"])):
        assert torch.equal(view.permute(0, 2, 1, 3)[rest], before.permute(0, 2, 1, 3)[rest])


NORM = [
    # kind, T, Hq, Hkv, D, bs, R, axes, interleaved, slots, per head, strided
    ("bf16", 1, 4, 1, 128, 16, 128, 1, False, "chunk", False, False),
    ("bf16", 37, 8, 2, 128, 16, 128, 3, False, "random", True, True),
    ("bf16", 65, 4, 4, 64, 32, 32, 1, True, "chunk", False, True),
    ("bf16", 9, 3, 3, 80, 16, 64, 2, False, "random", True, False),
    ("bf16", 21, 2, 1, 256, 16, 256, 1, False, "chunk", False, True),
    ("bf16", 13, 2, 2, 512, 16, 128, 1, True, "random", True, False),
    ("bf16", 11, 4, 2, 16, 16, 16, 1, False, "random", False, False),
    ("bf16", 7, 5, 5, 32, 48, 16, 1, False, "chunk", True, False),
    ("e4m3", 50, 8, 2, 128, 32, 64, 1, True, "random", False, True),
    ("e4m3", 19, 4, 4, 96, 16, 96, 4, False, "chunk", True, False),
    ("f32", 23, 4, 2, 128, 16, 128, 2, True, "random", True, True),
    ("f32", 33, 6, 3, 64, 16, 64, 1, False, "chunk", False, False),
    ("f32-e4m3", 17, 4, 1, 112, 16, 48, 1, False, "random", False, True),
]


@pytest.mark.parametrize("case", NORM)
@pytest.mark.parametrize("f32_weights", [False, True])
def test_norm(case, f32_weights):
    c = norm_case(*case[:11], f32_weights=f32_weights)
    q_out, kp, vp = norm_gpu(c, strided=case[11])
    check_norm(c, q_out, kp, vp, untouched=np.full(q_out.shape, 7.0))


def test_norm_many_tokens_and_heads():
    """Warps that walk over several heads, with weights of their own, uneven shares."""
    c = norm_case("bf16", 2500, 20, 5, 64, 16, 64, 1, False, "chunk", True)
    check_norm(c, *norm_gpu(c, strided=True))


def test_norm_in_place_and_on_another_stream():
    c = norm_case("bf16", 37, 8, 2, 128, 16, 64, 1, False, "random", False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    q_out, kp, vp = norm_gpu(c, strided=True, in_place=True, stream=s)
    torch.cuda.synchronize()
    check_norm(c, q_out, kp, vp, untouched=oatt.widen(c["x"][:, :8]))


def test_norm_of_zero_tiny_and_huge_heads():
    """A zero head stays zero under a positive eps; magnitudes are taken out whatever they are."""
    c = norm_case("f32", 6, 2, 1, 64, 16, 64, 1, False, "chunk", False)
    x = c["x"].clone()
    x[0] = 0.0
    x[1] *= 1e-12
    x[2] *= 1e15
    c["x"] = x
    check_norm(c, *norm_gpu(c))
    c["eps"] = 0.0                                         # without eps: the definition's 0 / 0 in the zero head
    q_out, _, _ = norm_gpu(c)
    assert q_out[0].isnan().all() and q_out[1:].isfinite().all()


def test_norm_skips_bad_slots_and_positions():
    c = norm_case("bf16", 12, 4, 2, 128, 16, 128, 1, False, "chunk", False)
    NB = c["kv"].shape[0]
    c["slots"][3] = NB * c["bs"]
    c["pos"][0, 5] = 97
    c["pos"][0, 6] = -1
    q_out, kp, vp = norm_gpu(c)
    assert pkv.get_device_error() == OUT_OF_RANGE
    c["slots"][[3, 5, 6]] = -1
    c["pos"][:] = np.clip(c["pos"], 0, 96)
    check_norm(c, q_out, kp, vp, untouched=np.full(q_out.shape, 7.0))


def test_norm_of_nothing():
    c = norm_case("bf16", 1, 4, 2, 64, 16, 64, 1, False, "chunk", False)
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")
    pkv.norm_rotary_and_cache(e(0, 4, 64), e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), c["qw"].cuda(), c["kw"].cuda(), kp, vp,
                              e(0, dt=I64), e(0, dt=I32), cuda(c["table"]))
    assert torch.equal(pkv.pool_views(kp, vp)[0].cpu(), c["kv"])


# ------------------------------------------------- paged_attention_decode_weighed
def logit_error(q, k, scale):
    """How far a logit may be off: products of 16-bit numbers are exact, of float32 rounded once, and
    their sums go through at most D + 8 additions of a float32 step each (a tensor core may cut
    where it adds: a whole step, 2 U) of the row's largest sum of magnitudes; then the scale."""
    D = q.shape[-1]
    return float((np.abs(q) @ np.abs(k).T).max(initial=0.0)) * scale * (D + 16) * 2 * U


def decode_case(kind, lens, Hq, Hkv, D, bs, seed=0, width=None, decay=1.0, gain=2.0, spare=2):
    rng = rng_of(seed, Hq, Hkv, D, bs, len(lens), max(lens))
    act, cache = KINDS[kind]
    NB = sum(-(-n // bs) for n in lens) + spare
    tables, free = tables_of(rng, lens, bs, NB, width)
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    cap = tables.shape[1] * bs + 4
    weights = weights_of(rng, len(lens) + 2, Hkv, cap)
    rows = rng.permutation(len(lens) + 2)[:len(lens)].astype(np.int32)
    q = normal(rng, (len(lens), Hq, D), act, gain)
    ks, vs = (KS, VS) if cache == U8 else (1.0, 1.0)
    return dict(q=q, kv=kv, vv=vv, tables=tables, lens=np.asarray(lens, dtype=np.int32), weights=weights, rows=rows,
                ks=ks, vs=vs, scale=1.0 / math.sqrt(D), bs=bs, decay=decay, act=act, free=free)


def decode_gpu(c, rows="given", stream=None, calls=1):
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    q, W, tables = c["q"].cuda(), cuda(c["weights"].copy()), cuda(c["tables"])
    out = torch.full_like(q, 7.0)
    B, Hq, D = q.shape
    ws = torch.full((pkv.weighed_decode_workspace_size(B, Hq, D, c["bs"], tables.shape[1]),), 255, dtype=U8, device="cuda")
    r = cuda(c["rows"]) if rows == "given" else None
    for _ in range(calls):
        pkv.paged_attention_decode_weighed(out, W, r, q, kp, vp, tables, cuda(c["lens"]), c["scale"], c["decay"], c["ks"],
                                           c["vs"], ws, stream=stream)
    return out, W


def check_decode(c, out, W, rows=None, missing=(), skip=(), calls=1, error=0):
    """``missing``: (sequence, token) without a block; ``skip``: sequences whose weights stay."""
    torch.cuda.synchronize()
    rows = c["rows"] if rows is None else rows
    B, Hq, D = c["q"].shape
    Hkv = c["kv"].shape[1]
    G = Hq // Hkv
    kf, vf, q = values(c["kv"], c["ks"]), values(c["vv"], c["vs"]), oatt.widen(c["q"])
    want = c["weights"].astype(np.float64)
    slack = np.zeros_like(want)
    o_got = oatt.widen(out.cpu())
    for b, n in enumerate(c["lens"]):
        gone = [t for s, t in missing if s == b]
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            k, v = (rows_of(f, np.maximum(c["tables"][b], 0), h, n, c["bs"]) for f in (kf, vf))
            p = oev.decode_weights(q[b, heads], k, c["scale"], gone) if n else np.zeros((G, 0))
            # a weight: twice the logit's error (numerator and sum), two exponentials of 2^-22, a sum
            # of n weights in runs of n / 8 or less, products
            eps = 2 * logit_error(q[b, heads], k, c["scale"]) + 2.0 ** -20 + (n / 8 + 64) * U
            ref = p @ v
            # the weights that multiply V are two 16-bit numbers: 2^-16 of each
            tol = (eps + 2.0 ** -15) * (p @ np.abs(v)) + HALF[c["act"]] * np.abs(ref) * 1.01 + 1e-30
            assert (np.abs(o_got[b, heads] - ref) <= tol).all(), (b, h, np.abs(o_got[b, heads] - ref).max())
            if b in skip or n == 0:
                continue
            for _ in range(calls):
                want[rows[b], h, :n] = oev.updated(want[rows[b], h], p.sum(0), 1, c["decay"])
                slack[rows[b], h, :n] += eps * p.sum(0) + 3 * U * want[rows[b], h, :n] + 1e-36
    got = W.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= slack).all(), np.abs(got - want).max()   # untouched places: equal
    assert pkv.get_device_error() == error


DECODE = [
    # kind, lens, Hq, Hkv, D, bs
    ("bf16", [1], 4, 1, 128, 16), ("bf16", [0, 1, 16, 17, 31, 32, 33], 8, 2, 128, 16),
    ("bf16", [700, 5, 0, 130], 8, 8, 64, 16), ("bf16", [257, 511], 8, 1, 64, 32), ("bf16", [333, 64, 15], 4, 2, 128, 32),
    ("bf16", [1100, 2], 10, 5, 128, 16),
    ("e4m3", [0, 1, 16, 17, 31, 32, 33, 48], 8, 2, 128, 16), ("e4m3", [900, 47, 18], 8, 8, 128, 16),
    ("e4m3", [301, 95], 16, 2, 64, 16), ("e4m3", [301, 31, 1], 4, 1, 64, 32), ("e4m3", [200, 77], 8, 4, 128, 32),
    ("f32", [0, 1, 15, 16, 17], 4, 4, 64, 16), ("f32", [300, 33], 8, 2, 128, 32), ("f32", [513, 7], 8, 1, 128, 16),
    ("f32", [130, 260], 2, 1, 64, 32),
]


@pytest.mark.parametrize("case", DECODE)
@pytest.mark.parametrize("decay", [1.0, 0.75])
def test_decode(case, decay):
    c = decode_case(*case, decay=decay)
    check_decode(c, *decode_gpu(c))


@pytest.mark.parametrize("kind,lens,Hq,Hkv,D,bs", [
    ("bf16", [9000, 2050], 8, 2, 128, 16), ("e4m3", [8200], 4, 1, 128, 16), ("f32", [2500], 2, 2, 64, 16)])
def test_decode_long(kind, lens, Hq, Hkv, D, bs):
    """Many partitions of a row, the last one short."""
    c = decode_case(kind, lens, Hq, Hkv, D, bs)
    check_decode(c, *decode_gpu(c))


def test_decode_many_sequences_of_one_partition():
    c = decode_case("bf16", [1 + (7 * i) % 45 for i in range(300)], 16, 8, 64, 16)
    check_decode(c, *decode_gpu(c))


def test_decode_default_rows_and_several_calls():
    c = decode_case("bf16", [40, 100, 3], 8, 2, 128, 16, decay=0.5)
    check_decode(c, *decode_gpu(c, rows=None, calls=3), rows=np.arange(3), calls=3)


def test_decode_decay_zero_forgets():
    c = decode_case("bf16", [40, 100], 8, 2, 128, 16, decay=0.0)
    c["weights"][:] = 1e30
    check_decode(c, *decode_gpu(c))


@pytest.mark.parametrize("kind,bs", [("bf16", 16), ("e4m3", 16), ("e4m3", 32), ("f32", 16)])
def test_decode_bad_table_entries(kind, bs):
    """Tokens of a block outside the pool get no weight: the first block, two in a row, the last."""
    c = decode_case(kind, [200, 100], 8, 2, 64, bs)
    NB = c["kv"].shape[0]
    last = (200 - 1) // bs
    missing = []
    for j, bad in ((0, NB), (3, -1), (4, 1 << 30), (last, -7)):
        c["tables"][0, j] = bad
        missing += [(0, t) for t in range(j * bs, min(200, (j + 1) * bs))]
    out, W = decode_gpu(c)
    c["tables"] = np.where((c["tables"] < 0) | (c["tables"] >= NB), 0, c["tables"])
    check_decode(c, out, W, missing=missing, error=OUT_OF_RANGE)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
def test_decode_wide_float32_blocks(Hq, Hkv):
    """32 float32 tokens of 128 dims, which are read by halves: lengths that end in either half, blocks
    outside the pool, a length that the table does not hold, slots past the sequence holding anything."""
    c = decode_case("f32", [15, 16, 17, 31, 32, 33, 300, 100, 64], Hq, Hkv, 128, 32)
    clean = c["kv"].clone(), c["vv"].clone()
    for b, n in enumerate(c["lens"][:6]):
        blk = c["tables"][b, (n - 1) // 32]
        c["kv"][blk, :, (n - 1) % 32 + 1:] = math.nan
        c["vv"][blk, :, (n - 1) % 32 + 1:] = math.inf
    NB = c["kv"].shape[0]
    missing = []
    for b, j, bad in ((6, 0, NB), (6, 4, -1), (6, 9, 1 << 30), (7, 3, -7)):
        c["tables"][b, j] = bad
        missing += [(b, t) for t in range(j * 32, min(c["lens"][b], (j + 1) * 32))]
    c["tables"][8, 2:] = c["tables"][8, 0]
    c["lens"][8] = 5000                                    # clamped to the table's width
    out, W = decode_gpu(c)
    c["lens"][8] = c["tables"].shape[1] * 32
    c["kv"], c["vv"] = clean
    c["tables"] = np.where((c["tables"] < 0) | (c["tables"] >= NB), 0, c["tables"])
    check_decode(c, out, W, missing=missing, error=OUT_OF_RANGE)


def test_decode_every_block_bad():
    c = decode_case("e4m3", [40], 4, 2, 64, 16)
    c["tables"][:] = -1
    out, W = decode_gpu(c)
    check_decode(c, out, W, missing=[(0, t) for t in range(40)], error=OUT_OF_RANGE)
    assert (out == 0).all()


def test_decode_bad_lengths_are_clamped():
    c = decode_case("bf16", [33, 48], 4, 2, 64, 16)
    held = c["lens"].copy()
    c["lens"][:] = [-5, 1000]
    out, W = decode_gpu(c)
    c["lens"][:] = [0, held[1]]                            # the table's three blocks
    check_decode(c, out, W, error=OUT_OF_RANGE)


def test_decode_bad_and_repeated_rows():
    """Outputs are whole; the second sequence of a row and those without one leave the weights."""
    c = decode_case("bf16", [33, 50, 20, 41, 7], 8, 2, 64, 16)
    c["rows"][:] = [4, 7, 4, -1, 0]
    out, W = decode_gpu(c)
    check_decode(c, out, W, skip=(1, 2, 3), error=OUT_OF_RANGE)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4])
def test_decode_infinite_and_nan_logits(kind, G):
    """-inf keys beside finite ones get no weight; all -inf: zero row, no weight; a NaN or +inf logit
    makes the head's output and weights NaN."""
    Hkv, D, bs, lens = 1, 64, 16, [40, 40, 40, 40]
    c = decode_case(kind, lens, G * Hkv, Hkv, D, bs)
    c["q"][:] = 0.25
    c["q"][..., 1:] = 0
    kv = c["kv"]
    kv[:, :, :, 0] = 1.0
    of = lambda b, t: (c["tables"][b, t // bs], 0, t % bs, 0)
    kv[of(0, 3)] = kv[of(0, 39)] = -math.inf
    for t in range(40):
        kv[of(1, t)] = -math.inf
    kv[of(2, 17)] = math.inf
    kv[of(3, 39)] = math.nan
    kv[..., 1:] = 0
    out, W = decode_gpu(c)
    out, W = out.cpu().float(), W.cpu().numpy()
    assert out[0].isfinite().all() and (out[1] == 0).all() and out[2].isnan().all() and out[3].isnan().all()
    r = c["rows"]
    before = c["weights"]
    p = np.full(40, G / 38.0)
    p[[3, 39]] = 0.0
    assert np.allclose(W[r[0], 0, :40], oev.updated(before[r[0], 0], p, 1, 1.0), rtol=1e-5, atol=0)
    assert np.array_equal(W[r[1], 0, :39], before[r[1], 0, :39]) and W[r[1], 0, 39] == 0
    assert np.isnan(W[r[2], 0, :40]).all() and np.isnan(W[r[3], 0, :40]).all()
    assert np.array_equal(W[r[2], 0, 40:], before[r[2], 0, 40:])


def test_decode_unwritten_slots_may_hold_anything():
    for kind in ("bf16", "f32"):
        c = decode_case(kind, [35, 17], 4, 1, 64, 16)
        clean = c["kv"].clone(), c["vv"].clone()
        for b, n in enumerate(c["lens"]):
            blk = c["tables"][b, (n - 1) // 16]
            c["kv"][blk, :, n % 16:] = math.nan
            c["vv"][blk, :, n % 16:] = math.inf
        out, W = decode_gpu(c)
        c["kv"], c["vv"] = clean
        check_decode(c, out, W)


def test_decode_queries_of_any_magnitude():
    """An E4M3 cache's products are f16: queries far from 1 are brought into its range."""
    for by in (1e-20, 1e-3, 3e4):
        c = decode_case("e4m3", [70, 33], 8, 2, 128, 16, gain=by)
        c["scale"] = 0.1 / max(by, 1e-3) if by > 1 else 1.0 / by * 0.1
        check_decode(c, *decode_gpu(c))


def test_decode_result_does_not_depend_on_the_row_or_batch():
    """The same sequence alone and in a batch gives the same weights, and a call twice the same bits."""
    c = decode_case("bf16", [520, 130, 77], 8, 2, 128, 16)
    out1, W1 = decode_gpu(c)
    out2, W2 = decode_gpu(c)
    assert torch.equal(out1, out2) and torch.equal(W1, W2)


# ----------------------------------------------------------- weigh_prefill_tokens
def prompt_case(lens, chunks, Hq, Hkv, D, bs, window=0, decay=1.0, seed=0, width=None):
    c = decode_case("bf16", lens, Hq, Hkv, D, bs, seed=seed, decay=decay, width=width)
    rng = rng_of(seed, 5, sum(chunks), Hq)
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    c.update(q=normal(rng, (max(1, start[-1]), Hq, D), BF, 2.0), start=start, chunks=chunks, window=window,
             most=max(chunks))
    return c


def prompt_gpu(c, rows="given", stream=None):
    kp, _ = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    q, W = c["q"].cuda(), cuda(c["weights"].copy())
    n = pkv.weigh_prefill_workspace_size(len(c["lens"]), q.shape[1], c["most"], c["window"])
    ws = torch.full((max(16, n),), 255, dtype=U8, device="cuda")
    pkv.weigh_prefill_tokens(W, cuda(c["rows"]) if rows == "given" else None, q, kp, cuda(c["tables"]), cuda(c["lens"]),
                             cuda(c["start"]), c["scale"], c["most"], c["window"], c["decay"], ws, stream=stream)
    return W


def check_prompt(c, W, rows=None, missing=(), skip=(), error=0):
    torch.cuda.synchronize()
    rows = c["rows"] if rows is None else rows
    Hq, D = c["q"].shape[1:]
    Hkv = c["kv"].shape[1]
    G = Hq // Hkv
    kf, q = values(c["kv"], 1.0), oatt.widen(c["q"])
    want = c["weights"].astype(np.float64)
    slack = np.zeros_like(want)
    for b, n in enumerate(c["lens"]):
        C = c["chunks"][b]
        if b in skip or C == 0:
            continue
        w = min(c["window"] or C, C)
        end = c["start"][b + 1]
        gone = [t for s, t in missing if s == b]
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            k = rows_of(kf, np.maximum(c["tables"][b], 0), h, n, c["bs"])
            qs = q[end - w:end, heads]
            gained = oev.prompt_weights(qs, k, c["scale"], gone).sum((0, 1))
            # as a decode's weight; the row's logarithm costs 2^-22 and a rounding of a number below
            # 64; then w * G weights added in runs of a quarter
            eps = 2 * logit_error(qs.reshape(-1, D), k, c["scale"]) + 2.0 ** -18 + (n / 4 + w * G / 4 + 64) * U
            want[rows[b], h, :n] = oev.updated(want[rows[b], h], gained, C, c["decay"])
            slack[rows[b], h, :n] = eps * gained + 3 * U * want[rows[b], h, :n] + 1e-36
    got = W.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= slack).all(), np.abs(got - want).max()
    assert pkv.get_device_error() == error


PROMPT = [
    # lens, chunks, Hq, Hkv, D, bs, window
    ([1], [1], 1, 1, 128, 16, 0), ([5, 20], [5, 1], 4, 2, 128, 16, 0), ([128, 129], [128, 2], 4, 4, 64, 16, 0),
    ([300, 17, 40], [7, 0, 40], 8, 2, 128, 16, 0), ([260, 513], [260, 100], 4, 1, 128, 32, 0),
    ([700, 90], [64, 90], 8, 2, 128, 16, 32), ([1000, 33, 5], [200, 33, 5], 8, 1, 64, 32, 16),
    ([400], [400], 6, 2, 128, 16, 0), ([333], [150], 5, 1, 128, 16, 1), ([150, 150], [150, 3], 12, 1, 64, 16, 64),
    ([2100], [50], 4, 4, 128, 16, 8), ([130], [130], 1, 1, 64, 16, 130),
]


@pytest.mark.parametrize("case", PROMPT)
@pytest.mark.parametrize("decay", [1.0, 0.75])
def test_prompt(case, decay):
    c = prompt_case(*case[:6], window=case[6], decay=decay)
    check_prompt(c, prompt_gpu(c))


def test_prompt_many_key_tiles_and_heads():
    """Several key tiles a CTA in the second pass, several splits in the first."""
    c = prompt_case([5000, 4700, 130, 3000] * 2, [40] * 8, 8, 8, 64, 16, window=16)
    check_prompt(c, prompt_gpu(c))


def test_prompt_default_rows_and_stream():
    c = prompt_case([140, 60], [30, 60], 4, 2, 128, 16, window=8)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    W = prompt_gpu(c, rows=None, stream=s)
    check_prompt(c, W, rows=np.arange(2))


def test_prompt_bad_table_entries():
    for window in (0, 8):
        c = prompt_case([400, 100], [60, 100], 4, 2, 128, 16, window=window)
        NB = c["kv"].shape[0]
        missing = []
        for j, bad in ((0, -1), (9, NB), (24, 1 << 30)):   # first, in the middle, the last: within the chunk
            c["tables"][0, j] = bad
            missing += [(0, t) for t in range(16 * j, min(400, 16 * j + 16))]
        W = prompt_gpu(c)
        c["tables"] = np.where((c["tables"] < 0) | (c["tables"] >= NB), 0, c["tables"])
        check_prompt(c, W, missing=missing, error=OUT_OF_RANGE)


def test_prompt_bad_sequences_are_left():
    """A chunk longer than its sequence, a length past the table, more queries than announced, rows
    outside the weights, a row twice."""
    lens, chunks = [50, 60, 70, 80, 90, 40], [20, 30, 10, 12, 10, 10]
    for window in (0, 4):
        c = prompt_case(lens, chunks, 4, 2, 64, 16, window=window)
        c["lens"][0] = 15
        c["lens"][2] = 1000
        c["most"] = 25
        c["rows"][3:] = [6, 8, 6]
        W = prompt_gpu(c)
        check_prompt(c, W, skip=(0, 1, 2, 4, 5), error=OUT_OF_RANGE)


def test_prompt_offsets_out_of_order():
    c = prompt_case([50, 60], [20, 30], 4, 2, 64, 16)
    c["start"][:] = [0, -1, 50]                            # the first chunk negative, the second before q
    c["most"] = 51
    W = prompt_gpu(c)
    check_prompt(c, W, skip=(0, 1), error=OUT_OF_RANGE)


def test_prompt_infinite_and_nan_logits():
    lens, chunks = [200, 200, 200], [3, 3, 3]
    c = prompt_case(lens, chunks, 2, 1, 64, 16)
    c["q"][:] = 0
    c["q"][..., 0] = 0.25
    kv = c["kv"]
    kv[:] = 0
    of = lambda b, t: (c["tables"][b, t // 16], 0, t % 16, 0)
    kv[of(0, 5)] = -math.inf
    for t in range(200):
        kv[of(1, t)] = -math.inf
    kv[of(2, 199)] = math.nan                              # the last token: only the last query sees it
    W = prompt_gpu(c).cpu().numpy()
    r, before = c["rows"], c["weights"]
    p = np.zeros(200)
    for i in range(3):
        p[:198 + i] += 2.0 / (197 + i)
    p[5] = 0
    assert np.allclose(W[r[0], 0, :200], oev.updated(before[r[0], 0], p, 3, 1.0), rtol=1e-5, atol=0)
    assert np.array_equal(W[r[1], 0, :197], before[r[1], 0, :197]) and (W[r[1], 0, 197:200] == 0).all()
    assert np.isnan(W[r[2], 0, :200]).all()


def test_prompt_of_nothing_and_unwritten_slots():
    c = prompt_case([37, 20], [0, 0], 4, 2, 64, 16)
    c["most"] = 4
    check_prompt(c, prompt_gpu(c))
    c = prompt_case([37, 129], [5, 9], 4, 2, 64, 16)
    clean = c["kv"].clone()
    for b, n in enumerate(c["lens"]):
        c["kv"][c["tables"][b, (n - 1) // 16], :, n % 16:] = math.nan
    W = prompt_gpu(c)
    c["kv"] = clean
    check_prompt(c, W)


# ------------------------------------------------------------------ select_tokens
def select_gpu(W, rows, lens, K, first, last):
    kept = torch.full((len(lens), W.shape[1], K), -9, dtype=I32, device="cuda")
    pkv.select_tokens(kept, cuda(W), None if rows is None else cuda(np.asarray(rows, dtype=np.int32)),
                      cuda(np.asarray(lens, dtype=np.int32)), first, last)
    return kept.cpu().numpy()


def check_select(W, rows, lens, K, first, last):
    got = select_gpu(W, rows, lens, K, first, last)
    for b, n in enumerate(lens):
        for h in range(W.shape[1]):
            want = oev.select(W[b if rows is None else rows[b], h], n, K, first, last)
            assert got[b, h].tolist() == want, (b, h)


@pytest.mark.parametrize("lens,K,first,last", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2, 1, 0], 1, 1, 0), ([2, 3], 1, 0, 1), ([5, 4, 3, 0], 4, 1, 2),
    ([100, 64, 65, 63], 64, 0, 0), ([100, 64, 65], 64, 64, 0), ([100, 64, 65], 64, 0, 64), ([100, 99], 64, 30, 34),
    ([1000, 513, 40], 100, 4, 16), ([5000, 4097, 3], 1234, 4, 64), ([9001], 9000, 0, 0), ([9001], 1, 0, 0),
    ([20000, 16385, 11], 4096, 4, 256), ([33333], 77, 3, 0),
])
def test_select(lens, K, first, last):
    rng = rng_of(K, first, last, len(lens), max(lens))
    cap = -(-max(lens) // 4) * 4 + 8
    W = weights_of(rng, len(lens) + 1, 3, cap)
    W[:, 1] = np.round(W[:, 1])                            # many equal ones
    W[:, 2, ::3] = 0.0
    rows = rng.permutation(len(lens) + 1)[:len(lens)]
    check_select(W, rows, lens, K, first, last)
    check_select(W, None, lens, K, first, last)


def test_select_long_rows():
    """Rows past what a cluster's shared memory holds are read again in every pass."""
    rng = rng_of(77)
    n = 400_000
    W = weights_of(rng, 1, 2, n)
    W[0, 1] = np.floor(W[0, 1])
    check_select(W, None, [n - 3], 5000, 4, 100)


@pytest.mark.parametrize("cap,lens", [
    (32768, [32768, 16385, 20001, 700]), (32772, [32772, 32769, 32768, 5]), (65540, [65537, 65540, 32769, 32768]),
    (131076, [131073, 65000, 40000]), (262148, [262145, 131077, 32768]), (600_000, [262_149, 599_999, 262_144]),
])
def test_select_by_several_ctas(cap, lens):
    """Each size of CTA and cluster, and rows of it that need fewer than it has; equal weights on
    both sides of the CTAs' borders."""
    rng = rng_of(cap, len(lens))
    W = weights_of(rng, len(lens), 2, cap)
    W[:, 1] = np.floor(4 * W[:, 1]) / 4
    W[0, 1] = 1.0
    for K, first, last in ((500, 4, 30), (4000, 0, 0)):
        check_select(W, None, lens, K, first, last)


@pytest.mark.parametrize("cap", [12000, 20000, 40000])
def test_select_many_rows_of_every_length(cap):
    """More rows than one wave holds, short and long ones, bad lengths and rows among them: every list
    is written, once."""
    rng = rng_of(cap, 9)
    B, K, first, last = 110, 300, 2, 7
    lens = rng.integers(0, 8193, B)
    lens[:9] = [0, 1, K, 8191, 8192, 8193, cap - 1, cap, 9000]
    lens[9:12] = [cap + 5, -3, 8000]
    W = np.floor(50 * rng.standard_normal((B, 3, cap))).astype(np.float32)
    rows = rng.permutation(B).astype(np.int32)
    rows[11] = B
    got = select_gpu(W, rows, lens.astype(np.int32), K, first, last)
    assert pkv.get_device_error() == OUT_OF_RANGE
    for b in range(B):
        n = 0 if rows[b] == B else min(max(lens[b], 0), cap)
        for h in range(3):
            if n <= K:
                want = np.concatenate([np.arange(n), np.full(K - n, -1)])
            else:
                t = np.arange(first, n - last)
                best = t[np.lexsort((t, -W[rows[b], h, t]))][:K - first - last]
                want = np.sort(np.concatenate([np.arange(first), best, np.arange(n - last, n)]))
            assert np.array_equal(got[b, h], want), (b, h, n)


def test_select_one_value_and_extremes():
    n = 3000
    W = np.zeros((4, 2, n), dtype=np.float32)
    W[0] = 2.5                                             # all equal
    W[1, :, ::2] = -0.0                                    # 0 and -0 are equal
    W[2, 0, 100:200] = np.nan
    W[2, 0, 300:310] = np.inf
    W[2, 0, 400] = -np.inf
    W[2, 1] = -np.arange(n)                                # negative numbers
    W[3, 0] = np.float32(1e-45) * (np.arange(n) % 7)       # subnormal ones
    W[3, 1] = np.float32(3.4e38) * ((np.arange(n) % 5) - 2) / 2
    check_select(W, None, [n] * 4, 105, 0, 0)
    check_select(W, None, [n, n - 1, n - 2, n - 3], 700, 9, 33)


def test_select_does_not_look_past_the_sequence():
    W = np.full((1, 1, 64), np.inf, dtype=np.float32)
    W[0, 0, :30] = np.arange(30)
    check_select(W, None, [30], 10, 0, 0)


def test_select_bad_lengths_and_rows():
    W = weights_of(rng_of(3), 3, 2, 64)
    got = select_gpu(W, [1, 3, -1, 1], [90, 20, 20, -4], 8, 1, 1)
    assert pkv.get_device_error() == OUT_OF_RANGE
    for h in range(2):
        assert got[0, h].tolist() == oev.select(W[1, h], 64, 8, 1, 1)
    assert (got[1:] == -1).all()
    check_select(W, [2, 2, 1], [40, 30, 64], 8, 1, 1)      # a row twice


# -------------------------------------------------------------------- keep_tokens
def keep_case(kind, lens, K, Hkv, D, bs, seed=0, counts=None):
    rng = rng_of(seed, K, D, bs, Hkv, len(lens))
    act, cache = KINDS[kind]
    width = -(-K // bs)
    NB = sum(-(-n // bs) for n in lens) + width * len(lens) + 2
    tables, free = tables_of(rng, lens, bs, NB)
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    W = weights_of(rng, len(lens) + 2, Hkv, tables.shape[1] * bs)
    rows = rng.permutation(len(lens) + 2)[:len(lens)].astype(np.int32)
    kept = np.full((len(lens), Hkv, K), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            m = min(n, K) if counts is None else min(n, counts[h % len(counts)])
            kept[b, h, :m] = np.sort(rng.permutation(n)[:m])
    return dict(kv=kv, vv=vv, tables=tables, fresh=free[:width * len(lens)].reshape(len(lens), width).astype(np.int32),
                weights=W, rows=rows, kept=kept, lens=np.asarray(lens, dtype=np.int32), bs=bs)


def keep_gpu(c, weights=True, rows="given"):
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    W = cuda(c["weights"].copy())
    pkv.keep_tokens(cuda(c["kept"]), W if weights else None, cuda(c["rows"]) if rows == "given" and weights else None, kp, vp,
                    cuda(c["tables"]), cuda(c["fresh"]), cuda(c["lens"]))
    return kp, vp, W


def check_keep(c, kp, vp, W, skip=(), rows=None, weights=True, lost=(), error=0):
    """``skip``: (sequence, head, place) that stay; ``lost``: sequences whose weights stay."""
    rows = c["rows"] if rows is None else rows
    want_k, want_v, want_w = c["kv"].clone(), c["vv"].clone(), c["weights"].copy()
    bs = c["bs"]
    for b in range(len(c["lens"])):
        for h in range(c["kept"].shape[1]):
            for i, t in enumerate(c["kept"][b, h]):
                if t < 0 or (b, h, i) in skip:
                    continue
                src, dst = c["tables"][b, t // bs], c["fresh"][b, i // bs]
                want_k[dst, h, i % bs] = c["kv"][src, h, t % bs]
                want_v[dst, h, i % bs] = c["vv"][src, h, t % bs]
                if weights and b not in lost:
                    want_w[rows[b], h, i] = c["weights"][rows[b], h, t]
    k, v = (t.cpu() for t in pkv.pool_views(kp, vp))
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert np.array_equal(W.cpu().numpy(), want_w)
    assert pkv.get_device_error() == error


@pytest.mark.parametrize("kind,lens,K,Hkv,D,bs", [
    ("bf16", [1], 1, 1, 128, 16), ("bf16", [40, 33, 5], 20, 2, 128, 16), ("bf16", [200, 0, 100], 65, 3, 64, 32),
    ("bf16", [300], 300, 2, 80, 48), ("e4m3", [40, 33, 5], 20, 2, 128, 16), ("e4m3", [500, 129], 100, 2, 64, 32),
    ("e4m3", [70], 33, 1, 16, 16), ("f32", [40, 33, 5], 21, 2, 128, 16), ("f32", [150, 3], 70, 1, 512, 16),
    ("bf16", [5000, 4500], 4100, 1, 64, 16),
])
def test_keep(kind, lens, K, Hkv, D, bs):
    c = keep_case(kind, lens, K, Hkv, D, bs)
    check_keep(c, *keep_gpu(c))


def test_keep_without_weights_default_rows_uneven_heads():
    c = keep_case("bf16", [100, 60], 50, 2, 64, 16, counts=[50, 13])
    check_keep(c, *keep_gpu(c, weights=False), weights=False)
    check_keep(c, *keep_gpu(c, rows=None), rows=np.arange(2))


def test_keep_runs_and_everything():
    """A prefix, a suffix, everything: whole rows of V move at once."""
    for pick in (range(0, 64), range(36, 100), range(20, 84)):
        c = keep_case("bf16", [100], 64, 2, 128, 16)
        c["kept"][0, :] = np.asarray(pick)
        check_keep(c, *keep_gpu(c))


def test_keep_bad_entries_are_skipped():
    c = keep_case("bf16", [100, 90, 80], 40, 2, 64, 16)
    skip = set()

    def bad(b, h, i, t, also=()):
        c["kept"][b, h, i] = t
        skip.add((b, h, i))
        skip.update((b, h, j) for j in also)

    c["kept"][0, 0] = np.arange(40) * 2
    bad(0, 0, 3, 100, also=(4,))                           # past the sequence; the next one is not above it
    bad(0, 0, 20, 38)                                      # not above the entry before (38)
    bad(0, 0, 30, -5, also=(31,))                          # no padding's sign; the next one behind a negative
    c["kept"][1, 1] = np.arange(40) + 10
    bad(1, 1, 25, -1, also=(26,))                          # padding, then an entry
    out = keep_gpu(c)
    check_keep(c, *out, skip=skip, error=OUT_OF_RANGE)


def test_keep_entry_below_its_index():
    c = keep_case("bf16", [100], 8, 1, 64, 16)
    c["kept"][0, 0] = [3, 9, 20, 30, 2, 3, 50, 60]         # 2 not above 30; 3 above 2 but below its index 5
    check_keep(c, *keep_gpu(c), skip={(0, 0, 4), (0, 0, 5)}, error=OUT_OF_RANGE)


def test_keep_bad_blocks_and_rows():
    c = keep_case("e4m3", [100, 90, 80], 40, 2, 64, 16)
    NB = c["kv"].shape[0]
    c["tables"][0, 2] = NB
    c["fresh"][1, 1] = -1
    c["rows"][:] = [2, 2, 9]
    out = keep_gpu(c)
    skip = {(0, h, i) for h in range(2) for i, t in enumerate(c["kept"][0, h]) if t // 16 == 2}
    skip |= {(1, h, i) for h in range(2) for i in range(16, 32)}
    want = c["weights"].copy()
    for h in range(2):                                     # a row's weights move whatever its blocks
        want[2, h, :40] = c["weights"][2, h, c["kept"][0, h]]
    kp, vp, W = out
    assert np.array_equal(W.cpu().numpy(), want)
    check_keep(c, kp, vp, cuda(c["weights"]), skip=skip, weights=False, error=OUT_OF_RANGE)


# ------------------------------------------------------------------- all together
def test_captured_and_replayed():
    """The calls of a step captured into a graph and replayed with inputs rewritten in place."""
    c = decode_case("bf16", [300, 120], 8, 2, 128, 16, spare=20)
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    q, W0, tables, lens, rows = c["q"].cuda(), cuda(c["weights"]), cuda(c["tables"]), cuda(c["lens"]), cuda(c["rows"])
    W, out = W0.clone(), torch.empty_like(q)
    ws = torch.empty(pkv.weighed_decode_workspace_size(2, 8, 128, 16, tables.shape[1]), dtype=U8, device="cuda")
    kept = torch.empty(2, 2, 64, dtype=I32, device="cuda")
    fresh = cuda(c["free"][:8].reshape(2, 4).astype(np.int32))
    k1, v1 = kp.clone(), vp.clone()
    calls = [pkv.bind_paged_attention_decode_weighed(out, W, rows, q, k1, v1, tables, lens, c["scale"], workspace=ws),
             pkv.bind_select_tokens(kept, W, rows, lens, 2, 8),
             pkv.bind_keep_tokens(kept, W, rows, k1, v1, tables, fresh, lens)]

    def step():
        for f in calls:
            f()

    def reset():
        W.copy_(W0)
        k1.copy_(kp)
        v1.copy_(vp)

    reset()
    step()
    want = [t.clone() for t in (out, W, kept, k1, v1)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        reset()
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        reset()
        g.replay()
        for got, w in zip((out, W, kept, k1, v1), want):
            assert torch.equal(got, w)
    # another query, another length
    q2 = torch.randn(q.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF)
    q.copy_(q2)
    lens.copy_(torch.tensor([290, 64], dtype=I32))
    reset()
    g.replay()
    got = [t.clone() for t in (out, W, kept, k1, v1)]
    reset()
    step()
    for a, b in zip(got, (out, W, kept, k1, v1)):
        assert torch.equal(a, b)


def test_kept_tokens_attend_as_the_whole_cache_does_without_the_others():
    """Evicting tokens and decoding over the kept ones is decoding over the kept ones of the whole."""
    c = decode_case("bf16", [400], 8, 2, 128, 16, spare=20)
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    kept = torch.empty(1, 2, 100, dtype=I32, device="cuda")
    W, rows, lens = cuda(c["weights"]), cuda(c["rows"]), cuda(c["lens"])
    pkv.select_tokens(kept, W, rows, lens, 4, 16)
    fresh = cuda(c["free"][:7].reshape(1, 7).astype(np.int32))
    pkv.keep_tokens(kept, W, rows, kp, vp, cuda(c["tables"]), fresh, lens)
    q = c["q"].cuda()
    out = torch.empty_like(q)
    pkv.paged_attention_decode(out, q, kp, vp, fresh, torch.tensor([100], dtype=I32, device="cuda"), c["scale"])
    kf, vf, qf = oatt.widen(c["kv"]), oatt.widen(c["vv"]), oatt.widen(c["q"])
    got = oatt.widen(out.cpu())
    for h in range(2):
        t = kept.cpu().numpy()[0, h]
        k, v = (rows_of(f, c["tables"][0], h, 400, 16)[t] for f in (kf, vf))
        p = oev.decode_weights(qf[0, 4 * h:4 * h + 4], k, c["scale"])
        ref = p @ v
        # the decode's weights are one bf16 number each (2^-8), its output another
        tol = 2.0 ** -8 * 1.1 * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(ref) * 1.01 + 1e-4
        assert (np.abs(got[0, 4 * h:4 * h + 4] - ref) <= tol).all()
