"""paged_attention_decode_sparse where its arithmetic or its split of the work can go
wrong: infinite and NaN logits, weights far below the largest, queries outside fp16's
range, rows shared by several CTAs. Against the definition in float64."""
import math

import numpy as np
import pytest
import torch

from _lib import library, pkv
from test_gpu_long_context import BF, F32, I32, U8, f64, rng_of, sparse_case, sparse_gpu, tables_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


def definition(c):
    """(out, sum_t p_t |V_t|, largest sum_d |q_d K_td| scale) of a case in float64: logits of
    -infinity have no weight, a NaN or +infinite one makes the row NaN, no weight at all a
    zero row."""
    q, (k, v) = c["q"].double().numpy(), (f64(x).reshape(x.shape) for x in (c["kv"], c["vv"]))
    B, Hq, D = q.shape
    Hkv, bs = k.shape[1], c["bs"]
    ks, vs = float(np.float32(c["ks"])), float(np.float32(c["vs"]))
    out, mag, logit = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hq))
    for b, L in enumerate(c["lens"]):
        for h in range(Hkv):
            t = [t for j in c["sel"][b, h] if j >= 0 for t in range(j * bs, min(L, (j + 1) * bs))]
            if not t:
                continue
            t = np.array(t)
            ids = c["tables"][b][t // bs]
            K, V = k[ids, h, t % bs], v[ids, h, t % bs]
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                with np.errstate(invalid="ignore"):
                    x = (K * q[b, g]).sum(1) * (ks * c["scale"])
                if np.isnan(x).any() or (x == np.inf).any():
                    out[b, g] = np.nan
                    continue
                fine = np.isfinite(x)
                if not fine.any():
                    continue
                p = np.exp(x[fine] - x[fine].max())
                p /= p.sum()
                out[b, g], mag[b, g] = p @ V[fine] * vs, p @ np.abs(V[fine]) * vs
                logit[b, g] = (np.abs(K[fine]) @ np.abs(q[b, g])).max() * ks * c["scale"]
    return out, mag, logit


def check(c, got):
    """Logits: sums of D products, (D + 8) roundings of 2^-23 of the magnitudes, in the
    weight and in their sum; 2^-22 for a power of two and 2^-23 a token and merge for the
    sums. Weights of tensor-core products are two 16-bit numbers: 2^-16 of themselves off
    in bf16, 2^-22 in f16 and, lifted by 2^14, 2^-39 of the largest. Half a step of the
    result (2^-8; float32 2^-24)."""
    ref, mag, logit = definition(c)
    kind, D, G = c["kind"], ref.shape[-1], c["q"].shape[1] // c["kv"].shape[1]
    tokens = c["sel"].shape[2] * c["bs"]
    w = {"f32": 0.0, "bf16": 2.0 ** -16 if G > 1 else 0.0, "e4m3": 2.0 ** -22}[kind]
    rel = w + 2 * (D + 8) * 2.0 ** -23 * logit[..., None] + (tokens + 64) * 2.0 ** -23 + 2.0 ** -21
    tiny = tokens * 2.0 ** -39 * 448 * float(np.float32(c["vs"])) if kind == "e4m3" else 0.0
    half = 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    err = rel * mag + tiny
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~np.isnan(ref)
    off, tol = np.abs(got - ref)[fine], (err + half * (np.abs(ref) + err))[fine]
    assert np.all(off <= tol), f"worst {np.max(off / np.maximum(tol, 1e-300)):.3g} of the tolerance"


# ------------------------------------------------------------ infinite and NaN logits
# rows that one warp holds, that warps of a CTA share, that a cluster shares (few rows: by
# pushes; many: by its own merge)
SPLITS = [(1, 2), (3, 9), (2, 40), (1, 130), (70, 40)]


def with_keys(kind, G, B, K, bad, where, D=64, bs=16, Hkv=2):
    """Sequences whose last block holds one token; its key (where = 'last'), the first
    token's ('first') or all of a middle block's ('block') get ``bad`` in dim 5, which q
    meets with positive numbers in every head but the first of the last sequence."""
    c = sparse_case(kind, [(K - 1) * bs + 1] * B, Hkv * G, Hkv, D, bs, K, seed=91)
    c["q"][:, :, 5] = c["q"][:, :, 5].abs() + 0.25
    for b in range(B):
        t = c["tables"][b]
        if where == "last":
            c["kv"][t[K - 1], :, 0, 5] = bad
        elif where == "first":
            c["kv"][t[0], :, 0, 5] = bad
        else:
            c["kv"][t[(K - 1) // 2], :, :, 5] = bad
    return c


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("where", ["last", "first", "block"])
@pytest.mark.parametrize("B,K", SPLITS)
def test_keys_at_minus_infinity_have_no_weight(kind, G, where, B, K):
    c = with_keys(kind, G, B, K, -math.inf, where)
    c["q"][B - 1, 0, 5] = -1.0                             # +infinity: that row is NaN
    check(c, sparse_gpu(c))
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4])
def test_rows_whose_logits_are_all_minus_infinity_are_zero(kind, G):
    for B, K in SPLITS[:4]:
        c = with_keys(kind, G, B, K, -math.inf, "last")
        c["kv"][c["tables"][0][:K], :, :, 5] = -math.inf
        got = sparse_gpu(c)
        assert bool((got[0] == 0).all())
        check(c, got)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("where", ["last", "block"])
@pytest.mark.parametrize("B,K", SPLITS)
def test_a_nan_key_makes_its_row_nan(kind, G, where, B, K):
    c = with_keys(kind, G, B, K, 0x7f if kind == "e4m3" else math.nan, where)
    if B > 1:                                              # and no other row
        c["sel"][1] = np.where(np.arange(K) < K // 2 - 1, np.arange(K), -1)
    check(c, sparse_gpu(c))
    assert pkv.get_device_error() == 0


# ------------------------------------------------------------ queries of any magnitude
@pytest.mark.parametrize("gain", [1e-36, 1e-30, 2.0 ** -20, 1e-4, 2e4, 1e6, 1e30])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_e4m3_queries_of_any_magnitude(gain, G):
    """The products run in f16; bf16 queries past 65504 and below 2^-14 keep their bits, each
    head by its own scale (head 0 is 2^30 times smaller, with its logits near zero)."""
    for B, K in SPLITS[:4]:
        c = sparse_case("e4m3", [K * 16 - 5] * B, 2 * G, 2, 64, 16, K, seed=92)
        c["q"] = (c["q"].float() * gain).to(BF)
        if G > 1:
            c["q"][:, 0] = (c["q"][:, 0].float() * 2.0 ** -30).to(BF)
        c["scale"] = 0.125 / gain
        check(c, sparse_gpu(c))
    assert pkv.get_device_error() == 0


def test_e4m3_queries_of_mixed_magnitude():
    """Elements 2^-14 of their head's largest, below f16's normal range as they stand:
    their keys are the ones that differ."""
    c = sparse_case("e4m3", [64 * 16], 4, 1, 64, 16, 64, seed=93)
    c["q"] = c["q"] * 2.0 ** -24
    c["q"][:, :, 7] = 2.0 ** -10
    c["kv"][:, :, :, 7] = 0x38                             # 1.0 in every key
    c["scale"] = 2.0 ** 16 / c["ks"]
    check(c, sparse_gpu(c))


# ------------------------------------------------------------------------ weights
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bits", [9, 14.4, 20, 25.4, 30])
def test_a_flat_tail_of_small_weights_counts(kind, G, bits):
    """One token of weight 1 with values 0 beside tokens of 2^-bits with values 448, and
    half of them with 1 - 2^-8 of that: the output is the tail alone."""
    for K in (3, 64, 130):
        c = sparse_case(kind, [K * 32] * 2, 2 * G, 2, 64, 32, K, seed=94)
        one, top = (0x38, 0x7e) if kind == "e4m3" else (1.0, 448.0)
        c["kv"].fill_(0)
        c["vv"].fill_(top)
        c["vv"][:, :, ::2] = 0x7d if kind == "e4m3" else 446.0
        c["q"].zero_()
        c["q"][:, :, 3] = 1.0
        c["ks"] = c["vs"] = 1.0
        c["scale"] = bits * math.log(2.0)
        first = c["tables"][:, 0]
        c["kv"][first, :, 5, 3], c["vv"][first, :, 5] = one, 0
        check(c, sparse_gpu(c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [2, 4, 8])
def test_weights_are_those_of_float32(kind, G):
    """Values that cancel: tokens of +448 and -448 in turn under nearly equal weights, so
    that the output is far smaller than the values and weights of one 16-bit number would
    be off by more than everything else allows."""
    c = sparse_case(kind, [32] * 64, 2 * G, 2, 128, 16, 2, seed=95, qgain=0.05)
    top = (0x7e, 0xfe) if kind == "e4m3" else (448.0, -448.0)
    c["vv"][:, :, ::2], c["vv"][:, :, 1::2] = top
    check(c, sparse_gpu(c))


# ----------------------------------------------- many rows, shared by clusters of CTAs
def many_rows(kind, G, D, bs, B, K, how, seed=96, Hkv=8):
    """B sequences of 8 kv heads on the GPU: ragged lengths and lists, an empty sequence, one
    of a single token, empty lists. ``how``: 'ragged', or 'one long' among sequences of
    one or two blocks."""
    g = torch.Generator(device="cuda").manual_seed(seed + B + K + G)
    act, cache = {"f32": (F32, F32), "bf16": (BF, BF), "e4m3": (BF, U8)}[kind]
    n, NB = 3 * K, 700
    def pool(shape):
        x = torch.randn(shape, generator=g, device="cuda")
        return (x / 0.05).to(torch.float8_e4m3fn).view(U8) if kind == "e4m3" else x.to(cache)
    ks, vs = pkv.pool_shapes(NB, Hkv, bs, D, cache)
    c = dict(kind=kind, kp=pool(ks), vp=pool(vs), bs=bs, scale=D ** -0.5, ks=0.05 if kind == "e4m3" else 1.0,
             q=(torch.randn(B, Hkv * G, D, generator=g, device="cuda") * 1.5).to(act))
    c["vs"] = c["ks"]
    lens = torch.randint(1, n * bs + 1, (B,), generator=g, device="cuda")
    if how == "one long":
        lens = torch.randint(1, 2 * bs + 1, (B,), generator=g, device="cuda")
        lens[B // 2] = n * bs
    lens[1], lens[B - 3], lens[B - 1] = 0, 1, n * bs
    c["lens"] = lens.to(I32)
    c["tables"] = torch.randint(0, NB, (B, n), generator=g, device="cuda").to(I32)
    blocks = (lens + bs - 1) // bs
    rank = torch.rand(B, Hkv, n, generator=g, device="cuda")
    rank[torch.arange(n, device="cuda").expand(B, Hkv, n) >= blocks[:, None, None]] = 2.0
    take = torch.randint(0, K + 1, (B, Hkv), generator=g, device="cuda")
    take[torch.rand(B, Hkv, generator=g, device="cuda") < 0.5] = K
    order = rank.argsort(-1)[..., :K]
    listed = (torch.arange(K, device="cuda") < take[..., None]) & (rank.gather(-1, order) < 1.5)
    sel = torch.where(listed, order, n).sort(-1).values
    c["sel"] = torch.where(sel < n, sel, -1).to(I32)
    return c


def many_definition(c):
    """(out, sum_t p_t |V_t|, largest sum_d |q_d K_td| scale) in float64, on the GPU."""
    B, Hkv, K = c["sel"].shape
    bs, (Hq, D) = c["bs"], c["q"].shape[1:]
    G, ks, vs = Hq // Hkv, float(np.float32(c["ks"])), float(np.float32(c["vs"]))
    val = lambda t: (t.view(torch.float8_e4m3fn) if t.dtype == U8 else t).double()
    out, mag = torch.zeros(2, B, Hkv, G, D, dtype=torch.float64, device="cuda")
    logit = torch.zeros(B, Hkv, G, dtype=torch.float64, device="cuda")
    k, v = pkv.pool_views(c["kp"], c["vp"])                # [NB, Hkv, bs, D]
    heads = torch.arange(Hkv, device="cuda")[:, None]
    for b in range(B):
        j = c["sel"][b].long()
        ids = c["tables"][b].long()[j.clamp(min=0)]
        K_, V_ = (val(x[ids, heads]).reshape(Hkv, K * bs, D) for x in (k, v))
        at = j[..., None] * bs + torch.arange(bs, device="cuda")
        seen = ((j[..., None] >= 0) & (at < c["lens"][b])).reshape(Hkv, 1, K * bs)
        q = c["q"][b].double().reshape(Hkv, G, D)
        x = (q @ K_.transpose(1, 2) * (ks * c["scale"])).masked_fill(~seen, -math.inf)
        p = torch.where(seen.any(-1, keepdim=True), torch.softmax(x, -1), 0.0).nan_to_num(0.0)
        out[b], mag[b] = p @ V_ * vs, p @ V_.abs() * vs
        logit[b] = (q.abs() @ K_.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(-1) * (ks * c["scale"])
    return out.reshape(B, Hq, D), mag.reshape(B, Hq, D), logit.reshape(B, Hq)


def check_many(c):
    q = c["q"]
    got = torch.full_like(q, math.nan)
    pkv.paged_attention_decode_sparse(got, q, c["kp"], c["vp"], c["tables"], c["lens"], c["sel"], c["scale"], c["ks"],
                                      c["vs"])
    ref, mag, logit = many_definition(c)
    kind, D, G = c["kind"], q.shape[2], q.shape[1] // c["kp"].shape[1]
    tokens = c["sel"].shape[2] * c["bs"]
    w = {"f32": 0.0, "bf16": 2.0 ** -16 if G > 1 else 0.0, "e4m3": 2.0 ** -22}[kind]     # as in check
    err = (w + 2 * (D + 8) * 2.0 ** -23 * logit[..., None] + (tokens + 64) * 2.0 ** -23 + 2.0 ** -21) * mag
    if kind == "e4m3":
        err += tokens * 2.0 ** -39 * 448 * c["vs"]
    tol = err + (2.0 ** -24 if kind == "f32" else 2.0 ** -8) * (ref.abs() + err)
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol.clamp(min=1e-300)).nan_to_num(9e9).max()):.3g} of the tolerance"
    assert pkv.get_device_error() == 0
    return got


# Batches of 8 kv heads whose rows make clusters of 2 (20, 24, 80), 4 (40, 64, 115) and 8
# (30, 70) on 152 SMs with three CTAs each, or a CTA a row (50)
@pytest.mark.parametrize("B", [20, 24, 30, 40, 50, 64, 70, 80, 115])
@pytest.mark.parametrize("kind,G,D,bs", [("bf16", 1, 128, 16), ("bf16", 4, 128, 32), ("bf16", 8, 128, 16),
                                         ("e4m3", 1, 128, 16), ("e4m3", 4, 128, 16), ("e4m3", 8, 64, 32),
                                         ("f32", 1, 128, 32), ("f32", 8, 128, 16), ("f32", 8, 128, 32)])
def test_rows_shared_by_clusters(kind, G, D, bs, B):
    for K, how in ((64, "ragged"), (128, "one long")):
        check_many(many_rows(kind, G, D, bs, B, K, how))


@pytest.mark.parametrize("kind,G,D,bs", [("bf16", 4, 128, 16), ("e4m3", 4, 128, 16), ("f32", 1, 64, 32)])
def test_rows_shared_by_clusters_repeat_their_bits(kind, G, D, bs):
    c = many_rows(kind, G, D, bs, 64, 64, "ragged")
    want = check_many(c)
    for _ in range(10):
        got = torch.empty_like(want)
        pkv.paged_attention_decode_sparse(got, c["q"], c["kp"], c["vp"], c["tables"], c["lens"], c["sel"], c["scale"],
                                          c["ks"], c["vs"])
        assert torch.equal(got, want)


def test_rows_shared_by_clusters_with_infinite_and_nan_keys():
    """What crosses the merge of several CTAs: a row of -infinite logits alone, one with some,
    one with a NaN; the others as without them."""
    for kind, G in (("bf16", 4), ("f32", 1)):
        c = many_rows(kind, G, 128, 16, 64, 64, "ragged", seed=97)
        want = check_many(c)
        full = torch.nonzero((c["sel"][:, 0] >= 0).all(-1) & (c["sel"][:, 0] < 100).any(-1))[:, 0][:3].tolist()
        k, v = pkv.pool_views(c["kp"], c["vp"])
        NB = k.shape[0]
        k = torch.cat([k, k[:3]])                          # blocks of their own
        k[NB:, :, :, 5], k[NB + 1, :, 1:, 5] = -math.inf, 0.0
        k[NB + 2, :, 3, 7] = math.nan
        c["kp"], c["vp"] = pkv.pools_from_views(k, torch.cat([v, v[:3]]))
        c["q"][:, :, 5] = c["q"][:, :, 5].abs() + 0.1
        before = check_many(c)
        for b, blk in zip(full, (NB, NB + 1, NB + 2)):
            j = c["sel"][b, 0]
            c["tables"][b, (j if blk == NB else j[30:31]).long()] = blk
        got = torch.empty_like(want)
        pkv.paged_attention_decode_sparse(got, c["q"], c["kp"], c["vp"], c["tables"], c["lens"], c["sel"], c["scale"],
                                          c["ks"], c["vs"])
        assert bool((got[full[0], :G] == 0).all()) and bool(got[full[1]].isfinite().all())
        assert bool(got[full[2], :G].isnan().all())
        others = [b for b in range(64) if b not in full]
        assert torch.equal(got[others], before[others])
    assert pkv.get_device_error() == 0


# ------------------------------------------------------------------------ bound calls
def test_bound_calls_are_called_again_and_on_other_streams():
    """Each of the four bound calls, kept and called many times: on the current stream, on two
    others in turn and at once (each with its own buffers), with new inputs in place."""
    from test_gpu_long_context import bits, step_calls, step_state

    def bind(s):
        return [pkv.bind_rotary_and_cache(s["qr"], s["q"], s["k"], s["v"], s["kp"], s["vp"], s["slots"], s["pos"],
                                          s["table"]),
                pkv.bind_update_key_bounds(s["kp"], s["kb"], s["tables"], s["lens"], s["pos"], 1),
                pkv.bind_select_blocks(s["sel"], s["qr"], s["kb"], s["tables"], s["lens"], s["bs"], 1, 1, s["ws"]),
                pkv.bind_paged_attention_decode_sparse(s["out"], s["qr"], s["kp"], s["vp"], s["tables"], s["lens"],
                                                       s["sel"], s["scale"])]

    ref, s, t = (step_state(51) for _ in range(3))
    inputs = [{k: torch.randn_like(s[k]) for k in ("q", "k", "v")} for _ in range(3)]
    calls, others = bind(s), bind(t)
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    for i, stream in enumerate(streams + streams):
        for k, x in inputs[i % 3].items():
            for state in (ref, s, t):
                state[k].copy_(x)
        step_calls(ref)
        torch.cuda.synchronize()
        for c, o in zip(calls, others):
            c(stream)
            o(streams[(i + 1) % 3])
        torch.cuda.synchronize()
        for state in (s, t):
            assert all(torch.equal(a, b) for a, b in zip(bits(state), bits(ref)))
    assert pkv.get_device_error() == 0
