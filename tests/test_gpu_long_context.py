"""The long-context operators on a GPU against the oracle (float64): the rotated
append (stored bits), the key bounds (exact), the choice of blocks (exact) and
the attention over chosen blocks (tolerances from the roundings it makes), each
at the sizes, masks and orders where it can go wrong, then together as a serving
loop runs them."""
import math

import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import attention as oatt
from oracle import fp8_e4m3 as ofp8
from oracle import long_context as olc
from paged_kv_cache_259_gb300 import engine

pytestmark = pytest.mark.gpu
BF, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
KINDS = {"f32": (F32, F32), "bf16": (BF, BF), "e4m3": (BF, U8), "f32-e4m3": (F32, U8)}


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


def rng_of(*key):
    return np.random.default_rng(list(key))


def normal(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def f64(t):
    return oatt.widen(t)


def random_views(rng, NB, Hkv, bs, D, cache):
    """Filled plain [NB, Hkv, bs, D] K and V (CPU); E4M3 caches: codes of N(0, 1) / 0.05."""
    def one():
        x = rng.standard_normal((NB, Hkv, bs, D)).astype(np.float32)
        if cache == U8:
            return torch.from_numpy(ofp8.e4m3_quantize(x, 0.05))
        return torch.from_numpy(x).to(cache)
    return one(), one()


def tables_of(rng, lens, bs, NB, width=None):
    """Block tables over a random order of the pool's blocks, -1 past each sequence."""
    blocks = [-(-n // bs) for n in lens]
    t = np.full((len(lens), width or max(1, max(blocks))), -1, dtype=np.int32)
    ids = rng.permutation(NB)[:sum(blocks)]
    at = 0
    for b, n in enumerate(blocks):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


# ------------------------------------------------------------ rotary_and_cache
def rotary_case(kind, T, Hq, Hkv, D, bs, R, axes, interleaved, how, seed, strided=False):
    """Inputs (CPU) and the oracle's results. ``how``: 'random' slots with padding,
    'chunk' consecutive slots from an odd offset, 'reverse' the same backwards."""
    rng = rng_of(seed, T, D, R)
    act, cache = KINDS[kind]
    NB = -(-(T + 8) // bs) + 3
    P = 97
    if how == "random":
        slots = rng.permutation(NB * bs)[:T].astype(np.int64)
        slots[rng.random(T) < 0.15] = -1
    else:
        order = rng.permutation(NB)
        at = np.arange(T) + 3
        slots = order[at // bs].astype(np.int64) * bs + at % bs
        if how == "reverse":
            slots = slots[::-1].copy()
    pos = rng.integers(0, P, (axes, T)).astype(np.int32)
    half = R // 2
    sections = [half] if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    table = rng.standard_normal((P, 2, half)).astype(np.float32)     # any numbers: the operator's input
    x = normal(rng, (T, Hq + 2 * Hkv, D), act)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    ks, vs = (0.05, 0.04) if cache == U8 else (1.0, 1.0)
    cos, sin = olc.turns(pos, table, sections)
    live = slots >= 0
    # the oracle: float32 rotation, then one rounding
    qr = torch.from_numpy(olc.rotate_f32(q.float().numpy(), cos, sin, interleaved))
    kr = olc.rotate_f32(k.float().numpy(), cos, sin, interleaved)
    q_ref = torch.full((T, Hq, D), 7.0, dtype=act)
    q_ref[live] = qr.to(act)[live]
    enc = (lambda y, s: torch.from_numpy(ofp8.e4m3_quantize(y, s))) if cache == U8 else \
        (lambda y, s: torch.from_numpy(np.ascontiguousarray(y)).to(cache))
    k_ref, v_ref = kv.clone(), vv.clone()
    s = torch.from_numpy(slots[live])
    k_ref[s // bs, :, s % bs] = enc(kr[live], ks)
    v_ref[s // bs, :, s % bs] = enc(v.float().numpy()[live], vs)
    return dict(q=q, k=k, v=v, x=x, kv=kv, vv=vv, slots=slots, pos=pos, sections=sections, table=table,
                ks=ks, vs=vs, q_ref=q_ref, k_ref=k_ref, v_ref=v_ref, cos=cos, sin=sin, act=act, live=live,
                interleaved=interleaved)


def rotary_gpu(c, strided=False, in_place=False, stream=None):
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    Hq, Hkv = c["q"].shape[1], c["k"].shape[1]
    if strided:
        q, k, v = c["x"].cuda().split([Hq, Hkv, Hkv], 1)
    else:
        q, k, v = (t.contiguous().cuda() for t in (c["q"], c["k"], c["v"]))
    q_out = q if in_place else torch.full(q.shape, 7.0, dtype=c["act"], device="cuda")
    pos = c["pos"][0] if c["pos"].shape[0] == 1 else c["pos"]
    args = (q_out, q, k, v, kp, vp, torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(pos).cuda(),
            torch.from_numpy(c["table"]).cuda())
    kw = dict(sections=c["sections"], interleaved=c["interleaved"], k_scale=c["ks"], v_scale=c["vs"])
    if stream is None:
        pkv.rotary_and_cache(*args, **kw)
    else:
        stream.wait_stream(torch.cuda.current_stream())
        pkv.rotary_and_cache(*args, **kw, stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
    return q_out, kp, vp


def check_rotary(c, q_out, kp, vp):
    k, v = (t.cpu() for t in pkv.pool_views(kp, vp))
    as_bits = (lambda t: t.view(torch.int16) if t.dtype == BF else t.view(I32) if t.dtype == F32 else t)
    assert torch.equal(as_bits(k), as_bits(c["k_ref"])), "K pool"
    assert torch.equal(as_bits(v), as_bits(c["v_ref"])), "V pool"
    assert torch.equal(as_bits(q_out.cpu().contiguous()), as_bits(c["q_ref"])), "q"


ROTARY = [
    # kind, T, Hq, Hkv, D, bs, R, axes, interleaved, slots, strided
    ("bf16", 1, 4, 1, 128, 16, 128, 1, False, "chunk", False),
    ("bf16", 7, 8, 8, 64, 16, 64, 1, False, "random", True),
    ("bf16", 64, 8, 2, 128, 16, 128, 1, False, "random", True),
    ("bf16", 301, 8, 2, 128, 16, 128, 3, False, "chunk", True),
    ("bf16", 40, 5, 5, 128, 32, 64, 2, True, "chunk", False),
    ("bf16", 33, 2, 1, 80, 16, 48, 4, False, "reverse", False),      # head_dim not a multiple of 64
    ("bf16", 9, 2, 2, 16, 16, 16, 1, True, "chunk", False),          # one unit of 16 dims
    ("e4m3", 1, 4, 4, 64, 32, 32, 1, True, "chunk", False),
    ("e4m3", 129, 8, 2, 128, 16, 128, 1, False, "chunk", True),
    ("e4m3", 50, 4, 4, 64, 16, 64, 2, False, "random", False),
    ("e4m3", 65, 4, 4, 112, 32, 16, 1, True, "reverse", False),
    ("f32-e4m3", 21, 2, 1, 64, 16, 32, 1, False, "chunk", False),
    ("f32", 1, 2, 2, 64, 16, 64, 1, False, "chunk", False),
    ("f32", 70, 4, 2, 128, 16, 64, 3, True, "chunk", True),
    ("f32", 31, 3, 1, 96, 32, 96, 1, False, "random", False),
    ("bf16", 3000, 4, 2, 64, 16, 64, 1, False, "chunk", True),       # warps that walk several heads
    ("bf16", 2600, 16, 8, 128, 16, 128, 2, True, "chunk", False),
]


@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("in_place", [False, True])
def test_rotary_and_cache_bits(case, in_place):
    """q_out, both pools bit for bit (every other slot as it was); skipped rows of
    q_out as they were."""
    *a, strided = case
    c = rotary_case(*a, seed=11)
    got = rotary_gpu(c, strided, in_place)
    if in_place:
        c["q_ref"][~c["live"]] = c["q"][~c["live"]]
    check_rotary(c, *got)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind,half_step", [("f32", 2 ** -24), ("bf16", 2 ** -8)])
def test_rotary_error_against_64_bits(kind, half_step):
    """x1 c - x2 s: three float32 roundings of at most 2^-24 (|x1 c| + |x2 s|) each
    (the difference is no larger), then half a step of the result's type."""
    c = rotary_case(kind, 77, 8, 2, 128, 16, 96, 1, False, "chunk", seed=5)
    q_out, _, _ = rotary_gpu(c)
    x = c["q"].double().numpy()
    ref = olc.rotate_f64(x, c["cos"], c["sin"], False)
    mag = olc.rotate_f64(np.abs(x), np.abs(c["cos"]), np.abs(c["sin"]), False)
    a, b = olc.pair_dims(96, False)
    mag[..., a] += 2 * np.abs(x[..., b]) * np.abs(c["sin"])[:, None]       # |x1 c| + |x2 s|
    err = np.abs(q_out.double().cpu().numpy() - ref)
    f32_err = 3 * 2.0 ** -24 * mag
    assert np.all(err <= f32_err + (half_step if kind != "f32" else 0) * (np.abs(ref) + f32_err))


def test_rotary_skips_and_flags_bad_slots_and_positions():
    c = rotary_case("bf16", 20, 4, 2, 64, 16, 64, 2, False, "chunk", seed=3)
    NB, bs = c["kv"].shape[0], 16
    bad = [2, 9, 13]
    s = c["slots"][bad]
    c["slots"] = c["slots"].copy()
    c["slots"][2] = NB * bs                                # one past the pool
    c["pos"] = c["pos"].copy()
    c["pos"][0, 9], c["pos"][1, 13] = -1, 97               # before and one past the table
    for i, sl in zip(bad, s):
        c["q_ref"][i] = 7.0
        c["k_ref"][sl // bs, :, sl % bs] = c["kv"][sl // bs, :, sl % bs]
        c["v_ref"][sl // bs, :, sl % bs] = c["vv"][sl // bs, :, sl % bs]
    check_rotary(c, *rotary_gpu(c))
    assert pkv.get_device_error() == -4
    assert pkv.get_device_error() == 0


def test_rotary_far_slots_pass_32_bits():
    """A pool of over 2^31 elements: the slots of its last block."""
    Hkv, bs, D = 8, 32, 128
    NB = 2 ** 31 // (Hkv * bs * D) + 9
    ks, vs = pkv.pool_shapes(NB, Hkv, bs, D, U8)
    kp, vp = torch.zeros(ks, dtype=U8, device="cuda"), torch.zeros(vs, dtype=U8, device="cuda")
    T = 11
    slots = torch.arange(NB * bs - T, NB * bs, dtype=I64, device="cuda")
    q = torch.randn(T, 8, D, device="cuda").to(BF)
    k, v = torch.randn_like(q), torch.randn_like(q)
    table = pkv.rotary_table(T, D, device="cuda")
    pkv.rotary_and_cache(torch.empty_like(q), q, k, v, kp, vp, slots,
                         torch.arange(T, dtype=I32, device="cuda"), table)
    kk, vv = pkv.pool_views(kp[-1:], vp[-1:])
    cos, sin = olc.turns(np.arange(T)[None], table.cpu().numpy(), [D // 2])
    kr = ofp8.e4m3_quantize(olc.rotate_f32(k.float().cpu().numpy(), cos, sin, False), 1.0)
    vr = ofp8.e4m3_quantize(v.float().cpu().numpy(), 1.0)
    assert np.array_equal(kk[0, :, bs - T:].cpu().numpy().transpose(1, 0, 2), kr)
    assert np.array_equal(vv[0, :, bs - T:].cpu().numpy().transpose(1, 0, 2), vr)
    assert int(kp[:-1].any()) == 0 and int(vp[:-1].any()) == 0
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("scale", [0.037, 1.0, 3.0, 1e-35, 3e-39, 2e33, 0.7 * 2.0 ** -40])
@pytest.mark.parametrize("src", [BF, F32])
def test_rotary_e4m3_codes_at_rounding_borders(scale, src):
    """Values whose quotient by the scale lies on or next to the midpoints between
    E4M3 codes, in the subnormal range, at saturation and zero: the codes are those of
    the IEEE quotient."""
    s = np.float32(scale)
    mags = ofp8._MAGNITUDES
    mid = np.concatenate([(mags[1:] + mags[:-1]) / 2, mags, [448.0, 463.9, 464.0, 480.0, 1e6, 0.0]]).astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        x = (mid * s).astype(np.float32)
        x = np.concatenate([np.nextafter(np.nextafter(x, np.float32(-np.inf)), np.float32(-np.inf))] +
                           [np.nextafter(x, np.float32(-np.inf)), x, np.nextafter(x, np.float32(np.inf))])
    x = x[torch.isfinite(torch.from_numpy(x).to(src)).numpy()]     # an infinity turns its partner into NaN
    x = np.concatenate([x, -x])
    x = np.resize(x, -(-len(x) // 64) * 64).reshape(-1, 1, 64)
    t = torch.from_numpy(x).to(src)
    T = t.shape[0]
    NB = -(-T // 16)
    ks, vs = pkv.pool_shapes(NB, 1, 16, 64, U8)
    kp, vp = torch.zeros(ks, dtype=U8, device="cuda"), torch.zeros(vs, dtype=U8, device="cuda")
    table = torch.zeros(1, 2, 8, device="cuda")
    table[:, 0] = 1.0                                      # no turn
    q = t.cuda()
    pkv.rotary_and_cache(torch.empty_like(q), q, q, q, kp, vp, torch.arange(T, dtype=I64, device="cuda"),
                         torch.zeros(T, dtype=I32, device="cuda"), table, k_scale=float(s), v_scale=float(s))
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ofp8.e4m3_encode(np.clip(t.float().numpy() / s, -1e30, 1e30)))
    zero = want & 0x7f == 0                                # 0 x 1 - 0 x 0: the sign of a zero is the sum's
    for pool in pkv.pool_views(kp, vp):
        got = pool.cpu().permute(0, 2, 1, 3).reshape(-1, 1, 64)[:T]
        assert torch.equal(torch.where(zero, got & 0x7f, got), torch.where(zero, want & 0x7f, want))


def test_rotary_no_tokens():
    c = rotary_case("bf16", 4, 2, 1, 64, 16, 64, 1, False, "chunk", seed=1)
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    e = lambda h: torch.empty(0, h, 64, dtype=BF, device="cuda")
    pkv.rotary_and_cache(e(2), e(2), e(1), e(1), kp, vp, torch.empty(0, dtype=I64, device="cuda"),
                         torch.empty(0, dtype=I32, device="cuda"), torch.from_numpy(c["table"]).cuda())
    assert torch.equal(pkv.pool_views(kp, vp)[0].cpu(), c["kv"])


# ----------------------------------------------------------- update_key_bounds
def bounds_ref(kv, before, tables, lens, first, bs):
    out = before.double().numpy().copy()
    k = f64(kv).reshape(kv.shape)
    for b, L in enumerate(lens):
        for j in range(first[b] // bs, -(-L // bs)) if first[b] < L else ():
            for h in range(kv.shape[1]):
                out[tables[b, j], h] = olc.key_bounds(k[tables[b, j], h], min(bs, L - j * bs))
    return out


BOUNDS = [
    # kind, lens, new tokens, Hkv, D, bs
    ("bf16", [1], [1], 1, 64, 16),
    ("bf16", [33, 16, 17, 400, 0], [1, 1, 1, 1, 0], 5, 128, 16),
    ("bf16", [500, 31, 32], [500, 15, 32], 2, 128, 32),
    ("bf16", [40, 40], [7, 0], 3, 80, 16),
    ("e4m3", [1, 90, 48], [1, 50, 16], 2, 64, 16),
    ("e4m3", [257], [100], 4, 128, 32),
    ("e4m3", [20], [20], 1, 16, 16),
    ("f32", [70, 5], [70, 2], 2, 64, 16),
    ("f32", [129], [1], 3, 128, 32),
]


@pytest.mark.parametrize("hint", [None, 0, 1])
@pytest.mark.parametrize("case", BOUNDS, ids=lambda c: f"{c[0]}-{c[1]}-{c[3]}x{c[4]}x{c[5]}")
def test_key_bounds_exact(case, hint):
    """Every changed block's bounds, every other row as it was; the launch hint
    (the true count, unknown, too small) changes nothing."""
    kind, lens, new, Hkv, D, bs = case
    rng = rng_of(21, D, bs, len(lens))
    cache = KINDS[kind][1]
    NB = sum(-(-n // bs) for n in lens) + 3
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    tables = tables_of(rng, lens, bs, NB)
    first = np.array(lens, np.int32) - np.array(new, np.int32)
    before = normal(rng, (NB, Hkv, 2, D), pkv.key_bounds_dtype(cache))
    kb = before.cuda()
    pkv.update_key_bounds(pkv.pools_from_views(kv.cuda(), vv.cuda())[0], kb, torch.from_numpy(tables).cuda(),
                          torch.tensor(lens, dtype=I32).cuda(), torch.from_numpy(first).cuda(),
                          max(new) if hint is None else hint)
    assert np.array_equal(kb.double().cpu().numpy(), bounds_ref(kv, before, tables, lens, first, bs))
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_key_bounds_keep_nan_and_infinity_and_ignore_unfilled_slots(kind):
    rng = rng_of(22)
    cache = KINDS[kind][1]
    kv, vv = random_views(rng, 2, 1, 16, 64, cache)
    nan = 0x7f if cache == U8 else math.nan
    kv[0, 0, 3, 5] = nan                                   # filled: the bound is NaN
    kv[1, 0, 9:, :] = nan                                  # past the length: not seen
    if cache != U8:
        kv[0, 0, 2, 7], kv[0, 0, 4, 8] = math.inf, -math.inf
    tables = np.array([[0, 1]], np.int32)
    kb = torch.zeros(2, 1, 2, 64, dtype=pkv.key_bounds_dtype(cache), device="cuda")
    pkv.update_key_bounds(pkv.pools_from_views(kv.cuda(), vv.cuda())[0], kb, torch.from_numpy(tables).cuda(),
                          torch.tensor([25], dtype=I32).cuda(), torch.zeros(1, dtype=I32).cuda())
    ref = bounds_ref(kv, kb.cpu() * 0, tables, [25], [0], 16)
    got = kb.double().cpu().numpy()
    assert np.isnan(got[0, 0, :, 5]).all() and np.isnan(got).sum() == 2
    assert np.array_equal(got, ref, equal_nan=True)


def test_key_bounds_flag_bad_entries_and_lengths():
    rng = rng_of(23)
    kv, vv = random_views(rng, 4, 2, 16, 64, BF)
    kp = pkv.pools_from_views(kv.cuda(), vv.cuda())[0]
    kb = torch.zeros(4, 2, 2, 64, dtype=BF, device="cuda")
    run = lambda t, n, f: pkv.update_key_bounds(kp, kb, torch.tensor(t, dtype=I32).cuda(),
                                                torch.tensor(n, dtype=I32).cuda(),
                                                torch.tensor(f, dtype=I32).cuda())
    run([[1, 4, 2]], [48], [0])                            # block 4 of 4: skipped
    assert pkv.get_device_error() == -4
    got = kb.double().cpu().numpy()
    ref = bounds_ref(kv, kb.cpu() * 0, np.array([[1, 2]]), [32], [0], 16)
    assert np.array_equal(got, ref)
    run([[1, 0, 2]], [49], [48])                           # longer than the table
    assert pkv.get_device_error() == -4
    run([[1, 0, 2]], [-3], [0])
    assert pkv.get_device_error() == -4
    run([[1, 0, 2]], [3], [-1])
    assert pkv.get_device_error() == -4


# ---------------------------------------------------------------- select_blocks
def select_gpu(q, bounds, tables, lens, bs, Hkv, K, F, W, workspace=True, fill=-7):
    sel = torch.full((q.shape[0], Hkv, K), fill, dtype=I32, device="cuda")
    t = torch.as_tensor(tables).cuda()
    ws = torch.full((pkv.select_blocks_workspace_size(len(lens), Hkv, t.shape[1]),), 255, dtype=U8,
                    device="cuda") if workspace else None     # scratch needs no clearing
    pkv.select_blocks(sel, q.cuda(), bounds.cuda(), t, torch.tensor(lens, dtype=I32).cuda(), bs, F, W, ws)
    return sel.cpu().numpy()


def check_select(q, bounds, tables, lens, bs, Hkv, K, F, W):
    ref = olc.select_blocks(q.double().numpy(), bounds.double().numpy(), tables, lens, bs, Hkv, K, F, W)
    got = select_gpu(q, bounds, tables, lens, bs, Hkv, K, F, W)
    assert np.array_equal(got, ref)
    assert pkv.get_device_error() == 0


def key_like_bounds(rng, NB, Hkv, D, dtype):
    mid, wide = rng.standard_normal((NB, Hkv, D)), np.abs(rng.standard_normal((NB, Hkv, D))) + 0.5
    return torch.from_numpy(np.stack([mid - wide, mid + wide], 2).astype(np.float32)).to(dtype)


SELECT = [
    # dtype, lens, Hq, Hkv, D, bs, K, first, last
    (BF, [1], 1, 1, 64, 16, 1, 0, 0),
    (BF, [0, 5, 160, 161, 700, 1600], 8, 2, 128, 16, 10, 1, 1),
    (BF, [2000, 999, 3], 8, 1, 64, 32, 7, 0, 3),
    (BF, [4000, 77], 6, 2, 128, 16, 33, 1, 0),             # 3 query heads a kv head
    (BF, [40000, 12345], 4, 4, 128, 16, 200, 1, 2),
    (BF, [3000], 16, 2, 64, 16, 3, 1, 2),                  # forced blocks only
    (BF, [3000], 16, 2, 64, 16, 4, 0, 0),
    (F32, [3000, 100], 8, 2, 64, 16, 20, 1, 1),
    (F32, [9000], 7, 1, 128, 32, 50, 0, 1),
    (BF, [16 * 5000], 8, 2, 64, 16, 64, 1, 2),             # the 1024-thread selection
]


@pytest.mark.parametrize("case", SELECT, ids=lambda c: f"{str(c[0])[6:]}-{c[1]}-{c[2:]}")
def test_select_blocks_exact(case):
    dt, lens, Hq, Hkv, D, bs, K, F, W = case
    rng = rng_of(31, D, K, len(lens))
    NB = sum(-(-n // bs) for n in lens) + 2
    q = normal(rng, (len(lens), Hq, D), dt)
    check_select(q, key_like_bounds(rng, NB, Hkv, D, dt), tables_of(rng, lens, bs, NB), lens, bs, Hkv, K, F, W)


def test_select_long_row_scores_from_global_memory():
    """60,000 blocks: more scores than a CTA keeps in shared memory; logical blocks
    share 300 physical ones, so most scores are tied and the index decides."""
    rng = rng_of(32)
    n, NB, D = 60000, 300, 64
    tables = rng.integers(0, NB, (1, n)).astype(np.int32)
    q = normal(rng, (1, 2, D), BF)
    check_select(q, key_like_bounds(rng, NB, 1, D, BF), tables, [n * 16], 16, 1, 1000, 1, 1)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K", [3, 100, 258, 259])
def test_select_long_rows_from_few_likely_blocks(dt, K):
    """Rows of more blocks than a CTA's threads keep, looked at through a lower bound of
    the last place's score: rows of every length beside each other, scores in any order,
    rising (the likely blocks all at the end) and mostly tied (too many likely ones)."""
    rng = rng_of(34, K)
    lens, NB, D = [16 * 20001, 16 * 8192 + 1, 16 * 3000, 16 * 700 - 3, 16 * 258, 5], 20100, 64
    q = normal(rng, (len(lens), 4, D), dt)
    b = key_like_bounds(rng, NB, 2, D, dt)
    tables = np.stack([rng.permutation(NB)[:20001] for _ in lens]).astype(np.int32)
    check_select(q, b, tables, lens, 16, 2, K, 1, 1)
    c = torch.full_like(b, 0.5)
    c *= (1 + torch.arange(NB) / NB).to(dt)[:, None, None, None]
    check_select(q.abs(), c, np.arange(20001, dtype=np.int32)[None].repeat(len(lens), 0), lens, 16, 2, K, 1, 1)
    tied = torch.full_like(b, 0.25)
    tied[7000:7010] = 1
    check_select(q.abs(), tied, tables, lens, 16, 2, K, 0, 0)


@pytest.mark.parametrize("B,blocks,Hkv,D", [(2, 15000, 1, 64), (3, 9000, 2, 128), (40, 1500, 1, 128), (40, 700, 4, 64),
                                            (129, 400, 3, 64), (300, 300, 4, 128), (1024, 140, 2, 64),
                                            (1025, 140, 2, 64)])
def test_select_ragged_batches(B, blocks, Hkv, D):
    """Rows of every length beside each other: empty, listed whole, full; several stages a
    CTA, more rows than fit at once."""
    rng = rng_of(35, B)
    NB, K = 500, 12
    lens = rng.integers(0, blocks * 16 + 1, B)
    lens[rng.integers(0, B, B // 4)] = rng.integers(0, K * 16 + 20, B // 4)
    lens[0], lens[B - 1] = blocks * 16, rng.integers(0, 2) * blocks * 16
    q = normal(rng, (B, 2 * Hkv, D), BF)
    tables = rng.integers(0, NB, (B, blocks)).astype(np.int32)
    check_select(q, key_like_bounds(rng, NB, Hkv, D, BF), tables, lens.tolist(), 16, Hkv, K, 1, 2)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n", [300, 3000])
def test_select_equal_scores_take_the_lower_index(dt, n):
    """Every block's bounds are one set of numbers in another order and q is
    constant: exact scores are equal, float32 sums differ in their last bits.
    300 blocks are ranked from a list, 3,000 by bisection."""
    rng = rng_of(33, n)
    D = 128
    base = normal(rng, (D,), dt).abs() + 0.1
    bounds = torch.stack([torch.stack([-base[torch.from_numpy(rng.permutation(D))],
                                       base[torch.from_numpy(rng.permutation(D))]]) for _ in range(n)])[:, None]
    q = torch.full((1, 2, D), 1.5, dtype=dt)
    got = select_gpu(q, bounds, np.arange(n, dtype=np.int32)[None], [n * 16], 16, 1, 40, 1, 1)
    assert got[0, 0].tolist() == list(range(39)) + [n - 1]


@pytest.mark.parametrize("n", [200, 2500])
def test_select_scores_that_differ_below_float32(n):
    """Scores 2^12 + j 2^-26 (j a random order): equal in float32, distinct in 64
    bits; the largest j win."""
    rng = rng_of(34, n)
    D = 64
    j = rng.permutation(n)
    bounds = torch.zeros(n, 1, 2, D, dtype=F32)
    bounds[:, 0, 1, 0] = 2.0 ** 12
    bounds[:, 0, 1, 33] = torch.from_numpy((j * 2.0 ** -26).astype(np.float32))
    q = torch.ones(1, 1, D, dtype=F32)
    got = select_gpu(q, bounds, np.arange(n, dtype=np.int32)[None], [n * 16], 16, 1, 25, 0, 0)
    assert got[0, 0].tolist() == sorted(np.argsort(-j)[:25].tolist())


def test_select_rounding_window_random():
    """bf16 bounds that cancel: scores near zero from terms near 2^10, so hundreds of
    blocks lie within the float32 rounding of one another."""
    rng = rng_of(35)
    n, D = 4000, 128
    x = rng.standard_normal((n, 1, D)).astype(np.float32) * 1024
    x[..., 1::2] = -x[..., 0::2] + rng.standard_normal((n, 1, D // 2)) * 2.0 ** -6
    b = torch.from_numpy(np.stack([x, x], 2)).to(BF)
    q = torch.ones(1, 4, D, dtype=BF)
    check_select(q, b, rng.permutation(n).astype(np.int32)[None], [n * 16], 16, 1, 100, 1, 1)


@pytest.mark.parametrize("what", ["zero q", "zero bounds", "nan block", "inf blocks", "nan q", "huge", "tiny", "zero q, inf block", "outlier"])
@pytest.mark.parametrize("n", [500, 5000])
@pytest.mark.parametrize("dt", [BF, F32])
def test_select_degenerate_values(what, n, dt):
    rng = rng_of(36, n)
    D = 64
    q, b = normal(rng, (1, 4, D), dt), key_like_bounds(rng, n, 2, D, dt)
    if what == "zero q":
        q.zero_()
    elif what == "zero bounds":
        b.zero_()
    elif what == "nan block":
        b[37, 0, 1, 9] = math.nan
    elif what == "inf blocks":
        b[41, 0, 1, 9], b[17, 1, 0, 3], b[n - 9, 0, :, 2] = math.inf, -math.inf, math.inf
    elif what == "nan q":
        q[0, 1, 5] = math.nan
    elif what == "zero q, inf block":                      # 0 x inf: that block first
        q.zero_()
        b[60, 0, 0, 1] = math.inf
    elif what == "outlier":                                # one score stretches the range
        b[90, 0, 1] = 3e5
        b[91, 0, 1] = 1e3
    elif what == "huge":                                   # float32 sums overflow, exact ones do not
        q, b = (q.float() * 1e19).to(dt), (b.float() * 1e19).to(dt)
    else:                                                  # float32 products vanish
        q, b = (q.float() * 1e-25).to(dt), (b.float() * 1e-25).to(dt)
    check_select(q, b, rng.permutation(n).astype(np.int32)[None], [n * 16 - 3], 16, 2, 30, 1, 1)


def test_select_without_scores_needs_no_workspace():
    rng = rng_of(37)
    q, b = normal(rng, (2, 4, 64), BF), key_like_bounds(rng, 40, 2, 64, BF)
    t = tables_of(rng, [100, 250], 16, 40)                 # at most 16 blocks
    got = select_gpu(q, b, t, [100, 250], 16, 2, 16, 1, 1, workspace=False)
    assert got[0, 0].tolist() == list(range(7)) + [-1] * 9 and got[1, 1].tolist() == list(range(16))


def test_select_flags_bad_entries_and_lengths():
    rng = rng_of(38)
    q, b = normal(rng, (1, 2, 64), BF), key_like_bounds(rng, 50, 1, 64, BF)
    t = np.arange(40, dtype=np.int32)[None].copy()
    t[0, 7], t[0, 21] = -1, 50
    got = select_gpu(q, b, t, [40 * 16], 16, 1, 20, 1, 1)
    assert pkv.get_device_error() == -4
    ok = [j for j in range(1, 39) if j not in (7, 21)]     # bad blocks rank last
    s = olc.block_scores(q[0].double().numpy(), b[np.array(ok), 0].double().numpy())
    want = sorted([0, 39] + [ok[i] for i in np.argsort(-s, kind="stable")[:18]])
    assert got[0, 0].tolist() == want
    t[0, 3:38] = 99                                        # fewer good blocks than places
    got = select_gpu(q, b, t, [40 * 16], 16, 1, 20, 1, 1)
    assert pkv.get_device_error() == -4
    assert got[0, 0].tolist() == [0, 1, 2] + list(range(3, 18)) + [38, 39]
    t = np.arange(40, dtype=np.int32)[None].copy()
    t[0, [2, 3, 5]] = 50
    got = select_gpu(q, torch.zeros_like(b), t, [40 * 16], 16, 1, 8, 1, 1)   # all scores are zero
    assert pkv.get_device_error() == -4 and got[0, 0].tolist() == [0, 1, 4, 6, 7, 8, 9, 39]
    got = select_gpu(q, b, np.arange(40, dtype=np.int32)[None], [40 * 16 + 1], 16, 1, 40, 0, 0)
    assert pkv.get_device_error() == -4 and got[0, 0].tolist() == list(range(40))
    got = select_gpu(q, b, np.arange(40, dtype=np.int32)[None], [-1], 16, 1, 4, 0, 0)
    assert pkv.get_device_error() == -4 and got[0, 0].tolist() == [-1] * 4


# ------------------------------------------------ paged_attention_decode_sparse
def random_lists(rng, lens, bs, Hkv, K, fill=1.0):
    """Random ascending lists; ``fill``: the share of min(K, blocks) that is listed."""
    out = np.full((len(lens), Hkv, K), -1, np.int32)
    for b, L in enumerate(lens):
        n = -(-L // bs)
        for h in range(Hkv):
            m = int(round(min(K, n) * fill))
            out[b, h, :m] = np.sort(rng.permutation(n)[:m])
    return out


def sparse_tolerance(kind, G, ref, mag, logit, tokens, vmax, out_half):
    """What the roundings allow. Logits: sums of D products, every operation off by
    at most 2^-23 of the magnitudes (the tensor core truncates), (D + 8) of them,
    and that much relative error in every weight, twice (weight and sum). Weights:
    bf16 caches with query groups round them to bf16 (2^-8), E4M3 caches always to f16
    (2^-11, and 2^-25 where they are subnormal). Sums over the tokens and the merges: 2^-24 an
    operation, (tokens + 64). Last, half a step of the result."""
    D = ref.shape[-1]
    w = 0.0
    if G > 1 or kind == "e4m3":
        w = {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}[kind]
    rel = w + 2 * (D + 8) * 2.0 ** -23 * logit[..., None] + (tokens + 64) * 2.0 ** -23
    sub = tokens * 2.0 ** -25 * vmax if kind == "e4m3" else 0.0
    return rel * mag + sub + out_half * (np.abs(ref) + rel * mag)


def sparse_case(kind, lens, Hq, Hkv, D, bs, K, seed, fill=1.0, qgain=1.5):
    rng = rng_of(seed, D, bs, K, len(lens))
    act, cache = KINDS[kind]
    NB = sum(-(-n // bs) for n in lens) + 2
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    ks, vs = (0.05, 0.045) if cache == U8 else (1.0, 1.0)
    q = normal(rng, (len(lens), Hq, D), act) * qgain
    return dict(kind=kind, lens=lens, q=q, kv=kv, vv=vv, tables=tables_of(rng, lens, bs, NB), bs=bs,
                sel=random_lists(rng, lens, bs, Hkv, K, fill), ks=ks, vs=vs, scale=D ** -0.5)


def sparse_gpu(c, out=None):
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    q = c["q"].cuda()
    out = torch.full_like(q, math.nan) if out is None else out
    pkv.paged_attention_decode_sparse(out, q, kp, vp, torch.from_numpy(c["tables"]).cuda(),
                                      torch.tensor(c["lens"], dtype=I32).cuda(),
                                      torch.from_numpy(c["sel"]).cuda(), c["scale"], c["ks"], c["vs"])
    return out


def check_sparse(c, got, sel=None):
    ks, vs = np.float32(c["ks"]), np.float32(c["vs"])
    k, v = (f64(x).reshape(x.shape) for x in (c["kv"], c["vv"]))
    sel = c["sel"] if sel is None else sel
    ref, mag, logit = olc.sparse_decode(c["q"].double().numpy(), k, v, c["tables"], c["lens"], sel, c["scale"],
                                        c["bs"], float(ks), float(vs), with_bound=True)
    G = c["q"].shape[1] // c["kv"].shape[1]
    half = 2.0 ** -24 if c["q"].dtype == F32 else 2.0 ** -8
    vals = np.abs(v[np.isfinite(v)])
    tol = sparse_tolerance(c["kind"], G, ref, mag, logit, sel.shape[2] * c["bs"],
                           float(vs) * (vals.max() if vals.size else 0), half)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


SPARSE = [
    # kind, lens, Hq, Hkv, D, bs, K
    ("bf16", [1], 1, 1, 64, 16, 1),
    ("bf16", [0, 1, 16, 17, 300, 1000], 8, 2, 128, 16, 9),
    ("bf16", [900, 33, 0], 8, 1, 64, 32, 12),
    ("bf16", [2000, 40], 4, 2, 128, 32, 40),
    ("bf16", [5000, 3000], 5, 5, 128, 16, 128),
    ("bf16", [6000], 4, 1, 128, 16, 300),
    ("e4m3", [1], 4, 1, 128, 16, 3),
    ("e4m3", [0, 1, 16, 17, 31, 700], 8, 2, 128, 16, 9),
    ("e4m3", [2500, 1300, 15], 8, 1, 64, 16, 64),
    ("e4m3", [2500, 20], 8, 4, 128, 32, 33),
    ("e4m3", [400, 90], 3, 3, 64, 16, 7),
    ("f32", [0, 1, 500], 4, 4, 64, 16, 5),
    ("f32", [700, 90], 8, 2, 128, 32, 17),
    ("f32", [3000], 8, 1, 64, 16, 100),
]


@pytest.mark.parametrize("fill", [1.0, 0.6])
@pytest.mark.parametrize("case", SPARSE, ids=lambda c: f"{c[0]}-{c[1]}-{c[2:]}")
def test_sparse_decode(case, fill):
    kind, *a = case
    c = sparse_case(kind, *a, seed=41, fill=fill)
    check_sparse(c, sparse_gpu(c))
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind,B,Hq,Hkv", [("bf16", 80, 32, 8), ("e4m3", 70, 8, 8), ("f32", 130, 8, 8)])
def test_sparse_decode_many_rows_is_one_part_a_row(kind, B, Hq, Hkv):
    c = sparse_case(kind, [3 + 7 * b for b in range(B)], Hq, Hkv, 64, 16, 12, seed=42)
    check_sparse(c, sparse_gpu(c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (64, 32), (128, 32)])
def test_sparse_decode_one_row_shared_by_a_cluster(kind, G, D, bs):
    """Lists for clusters of 2, 4 and 8 CTAs with a row each; rows of every number of
    parts: none, one, fewer than warps, as many, several stages each."""
    for K in (17, 40, 70, 130):
        lens = [K * bs + 5, (K // 2) * bs - 1, 2 * bs, 1, 0, 9 * bs + 7]
        c = sparse_case(kind, lens, 2 * G, 2, D, bs, K, seed=44)
        check_sparse(c, sparse_gpu(c))
    assert pkv.get_device_error() == 0


def test_sparse_decode_sharp_logits():
    """Logits over +-60: one token takes nearly all the weight, late or early."""
    for kind in ("bf16", "e4m3", "f32"):
        c = sparse_case(kind, [3000, 700], 8, 2, 128, 16, 64, seed=43, qgain=20.0)
        check_sparse(c, sparse_gpu(c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("bs", [16, 32])
def test_sparse_with_every_block_listed_is_the_decode(kind, bs):
    """Both are within their tolerance of the oracle on the same tokens."""
    lens = [1, 130, 512, 777]
    c = sparse_case(kind, lens, 8, 2, 128, bs, -(-777 // bs), seed=44)
    check_sparse(c, sparse_gpu(c))
    kp, vp = pkv.pools_from_views(c["kv"].cuda(), c["vv"].cuda())
    q = c["q"].cuda()
    full = pkv.paged_attention_decode(torch.empty_like(q), q, kp, vp, torch.from_numpy(c["tables"]).cuda(),
                                      torch.tensor(lens, dtype=I32).cuda(), c["scale"], c["ks"], c["vs"])
    check_sparse(c, full)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("G", [1, 4])
def test_sparse_unfilled_slots_and_unlisted_blocks_are_not_seen(kind, G):
    """NaN (E4M3: the NaN code) and infinities past the length and in unlisted blocks."""
    c = sparse_case(kind, [75, 9], 2 * G, 2, 64, 16, 3, seed=45)
    c["sel"][0] = [[0, 2, 4], [1, 4, -1]]
    c["sel"][1] = [[0, -1, -1], [-1, -1, -1]]
    bad = 0x7f if kind == "e4m3" else math.nan
    for x in (c["kv"], c["vv"]):
        for b, L in enumerate(c["lens"]):
            last = c["tables"][b, L // 16]
            x[last, :, L % 16:] = bad
        for h, js in ((0, (1, 3)), (1, (0, 2, 3))):
            for j in js:
                x[c["tables"][0, j], h] = bad
        x[c["tables"][1, 0], 1] = bad
    got = sparse_gpu(c)
    assert not torch.isnan(got).any()
    check_sparse(c, got)
    assert float(got[1, G:].abs().max()) == 0.0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("K", [6, 40])
def test_sparse_bad_entries_are_flagged_and_skipped(kind, K):
    c = sparse_case(kind, [100, 100, 100, 640], 4, 1, 64, 16, K, seed=46)
    good = np.full_like(c["sel"], -1)
    c["sel"][:] = -1
    c["sel"][0, 0, :4] = [0, 2, 2, 5]                      # repeated
    good[0, 0, :3] = [0, 2, 5]
    c["sel"][1, 0, :4] = [1, 3, 7, 9]                      # past the sequence (7 blocks)
    good[1, 0, :2] = [1, 3]
    c["sel"][2, 0, :5] = [0, -1, 3, 4, -1]                 # 3 is directly behind padding
    good[2, 0, :2] = [0, 4]
    c["sel"][3, 0, :4] = good[3, 0, :4] = [0, 1, 20, 39]
    got = sparse_gpu(c)
    assert pkv.get_device_error() == -4
    check_sparse(c, got, good)
    # a block id outside the pool: its tokens get no weight
    c["sel"], good = good, good.copy()
    c["tables"] = c["tables"].copy()
    c["tables"][1, 1] = c["kv"].shape[0]
    good[1, 0, :2] = [3, -1]
    got = sparse_gpu(c)
    assert pkv.get_device_error() == -4
    check_sparse(c, got, good)
    # a length the table cannot hold is clamped
    c["lens"] = [100, 0, 0, 640 + 1]
    got = sparse_gpu(c)
    assert pkv.get_device_error() == -4
    c["lens"][3] = 640
    check_sparse(c, got, good)


def test_sparse_leaves_rows_behind_the_batch():
    c = sparse_case("bf16", [100, 40], 4, 2, 64, 16, 4, seed=47)
    whole = torch.full((5, 4, 64), 3.0, dtype=BF, device="cuda")
    check_sparse(c, sparse_gpu(c, whole[:2]))
    assert bool((whole[2:] == 3.0).all())


# ------------------------------------------------------------- streams, graphs
def step_state(seed, B=6, Hq=8, Hkv=2, D=128, bs=16, K=12, kind="bf16"):
    """A batch in mid-generation: device tensors of one decode step, rotated append
    to attention."""
    rng = rng_of(seed)
    act, cache = KINDS[kind]
    lens = [int(n) for n in rng.integers(1, 900, B)]
    NB = sum(-(-n // bs) for n in lens) + 2
    kv, vv = random_views(rng, NB, Hkv, bs, D, cache)
    tables = tables_of(rng, lens, bs, NB)
    kp, vp = pkv.pools_from_views(kv.cuda(), vv.cuda())
    s = dict(kp=kp, vp=vp, tables=torch.from_numpy(tables).cuda(), lens=torch.tensor(lens, dtype=I32).cuda(),
             q=normal(rng, (B, Hq, D), act).cuda(), k=normal(rng, (B, Hkv, D), act).cuda(),
             v=normal(rng, (B, Hkv, D), act).cuda(), table=pkv.rotary_table(1000, D, device="cuda"),
             ks=0.05 if cache == U8 else 1.0, K=K, scale=D ** -0.5, bs=bs)
    at = np.array(lens) - 1
    s["slots"] = torch.from_numpy(tables[np.arange(B), at // bs].astype(np.int64) * bs + at % bs).cuda()
    s["pos"] = torch.from_numpy(at.astype(np.int32)).cuda()
    s["kb"] = torch.zeros(NB, Hkv, 2, D, dtype=pkv.key_bounds_dtype(cache), device="cuda")
    pkv.update_key_bounds(kp, s["kb"], s["tables"], s["lens"], torch.zeros_like(s["lens"]))
    s["qr"], s["out"] = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    s["sel"] = torch.empty(B, Hkv, K, dtype=I32, device="cuda")
    s["ws"] = torch.empty(pkv.select_blocks_workspace_size(B, Hkv, tables.shape[1]), dtype=U8, device="cuda")
    return s


def step_calls(s, stream=None):
    pkv.rotary_and_cache(s["qr"], s["q"], s["k"], s["v"], s["kp"], s["vp"], s["slots"], s["pos"], s["table"],
                         k_scale=s["ks"], v_scale=s["ks"], stream=stream)
    pkv.update_key_bounds(s["kp"], s["kb"], s["tables"], s["lens"], s["pos"], 1, stream=stream)
    pkv.select_blocks(s["sel"], s["qr"], s["kb"], s["tables"], s["lens"], s["bs"], 1, 1, s["ws"], stream=stream)
    pkv.paged_attention_decode_sparse(s["out"], s["qr"], s["kp"], s["vp"], s["tables"], s["lens"], s["sel"],
                                      s["scale"], s["ks"], s["ks"], stream=stream)


RESULTS = ("qr", "kp", "vp", "kb", "sel", "out")


def bits(s):
    return [s[k].clone().view(torch.uint8) for k in RESULTS]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_step_captured_replayed_and_on_other_streams(kind):
    """The same bits from the default stream, another stream, a captured graph
    replayed with new inputs in place, and two graphs in turn that share every
    buffer but run in order."""
    ref = step_state(51, kind=kind)
    step_calls(ref)
    want = bits(ref)
    s = step_state(51, kind=kind)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    step_calls(s, other)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(s), want))
    # captured on other values, replayed on these
    s = step_state(51, kind=kind)
    keep = {k: s[k].clone() for k in ("q", "k", "v")}
    graphs = []
    for _ in range(2):
        for k in keep:
            s[k].normal_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step_calls(s)
        graphs.append(g)
    for k in keep:
        s[k].copy_(keep[k])
    for g in (graphs[0], graphs[1], graphs[0]):
        for k in RESULTS[:1] + RESULTS[4:]:
            s[k].zero_()
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(s), want))
    assert pkv.get_device_error() == 0


def test_two_steps_at_once_with_workspaces_of_their_own():
    alone = [step_state(61 + i, B=4 + 3 * i) for i in range(2)]
    for s in alone:
        step_calls(s)
    want = [bits(s) for s in alone]
    both = [step_state(61 + i, B=4 + 3 * i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(both, streams):
            step_calls(s, st)
    torch.cuda.synchronize()
    for s, w in zip(both, want):
        assert all(torch.equal(a, b) for a, b in zip(bits(s), w))


def test_results_do_not_change_from_run_to_run():
    s = step_state(71, B=9)
    step_calls(s)
    want = bits(s)
    for _ in range(20):
        step_calls(s)
        assert all(torch.equal(a, b) for a, b in zip(bits(s), want))


# --------------------------------------------------------- together, as served
@pytest.mark.parametrize("kind,axes,interleaved", [("bf16", 1, False), ("bf16", 3, True), ("e4m3", 1, False)])
def test_serving_loop_against_the_oracle(kind, axes, interleaved):
    """Prompts prefilled (bf16) or appended (E4M3), one sequence forked, then decode
    steps through the engine; every step's pools, bounds and choice bit for bit and
    its attention within tolerance. The oracle keeps its own cache."""
    rng = rng_of(81, axes)
    act, cache = KINDS[kind]
    Hq, Hkv, D, bs, NB, K, R = 8, 2, 128, 16, 120, 6, 96
    sc = 0.05 if cache == U8 else 1.0
    eng = engine.PagedKVCache(NB, Hq, Hkv, D, bs, cache, rng.permutation(NB), "cuda")
    eng.k_pool.zero_(), eng.v_pool.zero_()
    eng.enable_key_bounds()
    half = R // 2
    sections = [half] if axes == 1 else [16, 16, 16]
    table = pkv.rotary_table(600, R)
    rot = engine.Rotary(table.cuda(), sections, interleaved)
    okv = {n: torch.zeros(NB, Hkv, bs, D, dtype=cache) for n in "kv"}
    kb = np.zeros((NB, Hkv, 2, D))
    enc = (lambda y: torch.from_numpy(ofp8.e4m3_quantize(y, sc))) if cache == U8 else \
        (lambda y: torch.from_numpy(y).to(cache))

    def append(plan, pos, q, k, v):
        """The oracle's half of an append; returns the rotated query."""
        for a, d in plan.pairs:
            for n in "kv":
                okv[n][d] = okv[n][a]
        cos, sin = olc.turns(pos, table.numpy(), sections)
        sl = torch.from_numpy(plan.slots)
        okv["k"][sl // bs, :, sl % bs] = enc(olc.rotate_f32(k.float().numpy(), cos, sin, interleaved))
        okv["v"][sl // bs, :, sl % bs] = enc(v.float().numpy())
        first, kk = engine.first_changed(plan), f64(okv["k"]).reshape(NB, Hkv, bs, D)
        for b, L in enumerate(plan.lens):
            for j in range(first[b] // bs, -(-L // bs)):
                for h in range(Hkv):
                    kb[plan.tables[b, j], h] = olc.key_bounds(kk[plan.tables[b, j], h], min(bs, L - j * bs))
        return torch.from_numpy(olc.rotate_f32(q.float().numpy(), cos, sin, interleaved)).to(act)

    def check_cache():
        assert torch.equal(eng.k_view().cpu().view(U8), okv["k"].view(U8))
        assert torch.equal(eng.v_view().cpu().view(U8), okv["v"].view(U8))
        assert np.array_equal(eng.key_bounds.double().cpu().numpy(), kb)

    def inputs(T):
        return (normal(rng, (T, h, D), act) for h in (Hq, Hkv, Hkv))

    def dev(plan, pos):
        return (plan.device_tensors("cuda"), torch.from_numpy(pos).cuda(),
                torch.from_numpy(engine.first_changed(plan)).cuda(), rot)

    prompts = [200, 37, 1]
    for i in range(3):
        eng.bm.add_seq(i)
    plan = eng.plan_prefill([0, 1, 2], prompts)
    T = sum(prompts)
    pos = rng.integers(0, 600, (axes, T)).astype(np.int32) if axes > 1 else \
        np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)
    q, k, v = inputs(T)
    if cache == U8:                                        # chunked prefill attention is bf16 only
        d, p, f, _ = dev(plan, pos)
        qd = q.cuda()
        eng._rotated_append(qd, k.cuda(), v.cuda(), d, p, f, rot, max(prompts), sc, sc, None)
        assert torch.equal(qd.cpu(), append(plan, pos, q, k, v))
    else:
        out, qd = torch.empty(T, Hq, D, dtype=act, device="cuda"), q.cuda()
        eng.rotary_prefill_step(qd, k.cuda(), v.cuda(), *dev(plan, pos), out, D ** -0.5, plan.max_query_len)
        qr = append(plan, pos, q, k, v)
        assert torch.equal(qd.cpu(), qr)
        ref = oatt.paged_prefill(qr, okv["k"], okv["v"], plan.tables, plan.lens, plan.query_start, D ** -0.5, bs)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert np.all(err <= 2e-2 + 2e-2 * np.abs(ref))    # the prefill's own tolerance
    check_cache()
    eng.bm.fork(0, 3)                                      # shares a partial last block
    ids = [0, 1, 2, 3]
    for step in range(4):
        plan = eng.plan_step(ids, group_prefixes=False)
        assert len(plan.pairs) == (1 if step == 0 else 0)
        pos = rng.integers(0, 600, (axes, 4)).astype(np.int32) if axes > 1 else (plan.lens - 1).astype(np.int32)
        q, k, v = inputs(4)
        qd, out = q.cuda(), torch.full((4, Hq, D), math.nan, dtype=act, device="cuda")
        sel = torch.empty(4, Hkv, K, dtype=I32, device="cuda")
        eng.sparse_step(qd, k.cuda(), v.cuda(), *dev(plan, pos), sel, out, D ** -0.5, 1, 2, sc, sc,
                        eng.select_workspace(4, plan.tables.shape[1]))
        qr = append(plan, pos, q, k, v)
        assert torch.equal(qd.cpu(), qr)
        check_cache()
        want = olc.select_blocks(qr.double().numpy(), kb, plan.tables, plan.lens, bs, Hkv, K, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want)
        check_sparse(dict(kind=kind, lens=[int(n) for n in plan.lens], q=qr, kv=okv["k"], vv=okv["v"],
                          tables=plan.tables, bs=bs, sel=want, ks=sc, vs=sc, scale=D ** -0.5), out)
    # bounds from scratch are the bounds kept step by step
    before = eng.key_bounds.clone()
    eng.refresh_key_bounds(torch.from_numpy(plan.tables).cuda(), torch.from_numpy(plan.lens).cuda())
    assert torch.equal(eng.key_bounds, before)
    assert pkv.get_device_error() == 0
