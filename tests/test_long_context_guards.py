"""The long-context operators without a GPU: refusals of the C entries and of the
binding (before any pointer reaches a kernel), the rotary table, and the oracle's
own definitions against hand-worked cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import long_context as olc

B, HQ, HKV, D, BS, NB, MB, T, K = 3, 4, 2, 64, 16, 8, 5, 7, 4
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def lib():
    return library()


# ------------------------------------------------------------------ C entries
SOME = ctypes.c_void_p(0x1000)


def c_rotary(sections=(32,), axes=1, strides=(256, 256, 128, 128), T=T, Hq=HQ, Hkv=HKV, D=D, R=64,
             bs=BS, NB=NB, P=64, src=1, cache=1, ks=1.0, vs=1.0, ptrs=None, sec_ptr=True):
    a = ptrs or [ctypes.c_void_p(0x2000)] + [SOME] * 8
    sec = (ctypes.c_int32 * len(sections))(*sections) if sec_ptr else None
    return library().rotary_and_cache(*a, sec, axes, *strides, T, Hq, Hkv, D, R, 0, bs, NB, P, src,
                                      cache, ks, vs, None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), -1), (dict(Hq=3), -1), (dict(R=80), -1), (dict(P=0), -1), (dict(axes=0), -1),
    (dict(sec_ptr=False), -1), (dict(sections=(31,)), -1), (dict(sections=(33, -1), axes=2), -1),
    (dict(strides=(255, 256, 128, 128)), -1),           # shorter than a row
    (dict(strides=(260, 256, 128, 128)), -1),           # rows not on 16 bytes
    (dict(strides=(256, 256, 128, 0)), -1),             # one row for all tokens
    (dict(strides=(264, 256, 128, 128), ptrs=[SOME] * 9), -1),   # in place, rows elsewhere
    (dict(ks=2.0), -1), (dict(cache=2, ks=0.0), -1), (dict(cache=2, vs=math.inf), -1),
    (dict(ptrs=[None] + [SOME] * 8), -1), (dict(ptrs=[SOME] * 8 + [None]), -1),
    (dict(ptrs=[ctypes.c_void_p(0x1008)] + [SOME] * 8), -1),
    (dict(R=24, sections=(12,)), -2), (dict(bs=24), -2),
    (dict(sections=(8, 8, 8, 4, 4), axes=5), -2), (dict(src=0, cache=1), -2), (dict(src=2, cache=2), -2),
    (dict(T=0, ptrs=[None] * 9), 0),                    # nothing to do
])
def test_rotary_entry_refuses_before_any_cuda_call(over, status):
    assert c_rotary(**over) == status


def c_bounds(ptrs=None, B=B, MB=MB, NB=NB, Hkv=HKV, D=D, bs=BS, new=1, kv=1):
    return library().update_key_bounds(*(ptrs or [SOME] * 5), B, MB, NB, Hkv, D, bs, new, kv, None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(B=65536), -1), (dict(MB=0), -1), (dict(new=-1), -1), (dict(D=24), -2),
    (dict(bs=8), -2), (dict(kv=3), -2), (dict(ptrs=[None] + [SOME] * 4), -1),
    (dict(ptrs=[SOME, ctypes.c_void_p(0x1004)] + [SOME] * 3), -1), (dict(MB=1 << 28), -1),
    (dict(B=0, ptrs=[None] * 5), 0),
])
def test_bounds_entry_refuses_before_any_cuda_call(over, status):
    assert c_bounds(**over) == status


def c_select(ptrs=None, B=B, MB=MB, NB=NB, Hq=HQ, Hkv=HKV, D=D, bs=BS, K=K, F=1, W=1, dt=1,
             ws=SOME, ws_bytes=1 << 20):
    return library().select_blocks(*(ptrs or [SOME] * 5), B, MB, NB, Hq, Hkv, D, bs, K, F, W, dt, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(K=0), -1), (dict(F=-1), -1), (dict(F=3, W=2), -1), (dict(Hq=3), -1), (dict(bs=0), -1),
    (dict(ws=None), -1), (dict(ws_bytes=64), -1), (dict(ws=ctypes.c_void_p(0x1004)), -1),
    (dict(ptrs=[SOME, ctypes.c_void_p(0x1004)] + [SOME] * 3), -1), (dict(ptrs=[None] + [SOME] * 4), -1),
    (dict(D=96), -2), (dict(Hq=18), -2), (dict(dt=2), -2), (dict(MB=(1 << 19) + 1), -2),
    (dict(B=0, ptrs=[None] * 5), 0),
])
def test_select_entry_refuses_before_any_cuda_call(over, status):
    assert c_select(**over) == status


def test_select_workspace_covers_scores_maxima_and_exact_keys():
    # 5 blocks pad to 16: 16 float32 scores, one maximum, 16 keys of 8 bytes a row
    assert library().select_blocks_workspace_size(3, 2, 5) == 6 * (16 * 12 + 4)
    assert library().select_blocks_workspace_size(0, 2, 5) == 0


def c_sparse(ptrs=None, B=B, MB=MB, NB=NB, K=K, Hq=HQ, Hkv=HKV, D=D, bs=BS, scale=0.1, qd=1, kv=1,
             ks=1.0, vs=1.0):
    return library().paged_attention_decode_sparse(*(ptrs or [SOME] * 7), B, MB, NB, K, Hq, Hkv, D, bs,
                                                   scale, qd, kv, ks, vs, None)


@pytest.mark.parametrize("over,status", [
    (dict(K=0), -1), (dict(B=-1), -1), (dict(Hq=5), -1), (dict(scale=math.nan), -1), (dict(ks=2.0), -1),
    (dict(kv=2, vs=-1.0), -1), (dict(ptrs=[SOME] * 6 + [None]), -1),
    (dict(ptrs=[ctypes.c_void_p(0x1008)] + [SOME] * 6), -1),
    (dict(Hq=6), -2), (dict(D=96), -2), (dict(bs=48), -2), (dict(qd=0, kv=1), -2), (dict(qd=0, kv=2), -2),
    (dict(B=0, ptrs=[None] * 7), 0),
])
def test_sparse_entry_refuses_before_any_cuda_call(over, status):
    assert c_sparse(**over) == status


def test_packed_call_is_the_call():
    """pkv_bound_call refuses another number of arguments or an unknown call, and
    passes every argument on: the statuses of the calls' own checks come back."""
    lib = library()
    f32 = lambda x: ctypes.c_uint32.from_buffer_copy(ctypes.c_float(x)).value
    u64 = lambda *a: (ctypes.c_uint64 * len(a))(*[x & 0xffffffffffffffff for x in a])
    call = lambda c, a: lib.pkv_bound_call(c, ctypes.addressof(a), len(a), None)
    sections = (ctypes.c_int32 * 1)(32)

    def rotary(T=T, R=64, stride=256, ks=1.0, sec=ctypes.addressof(sections), cache=1):
        return u64(*[0x1000] * 9, sec, 1, stride, 256, 128, 128, T, HQ, HKV, D, R, 0, BS, NB, 64, 1, cache,
                   f32(ks), f32(1.0))

    assert call(0, rotary(T=0)) == 0
    assert call(0, rotary(T=-1)) == -1                     # a sign survives
    assert call(0, rotary(stride=-256)) == -1
    assert call(0, rotary(R=24)) == -2
    assert call(0, rotary(ks=2.0)) == -1                   # a float does
    assert call(0, rotary(T=0, ks=2.0, cache=2)) == 0
    assert call(0, rotary(sec=0)) == -1                    # a pointer does
    assert call(0, u64(*list(rotary())[:-1])) == -1        # one argument short
    assert call(1, u64(*[0] * 5, 0, MB, NB, HKV, D, BS, 1, 1)) == 0
    assert call(1, u64(*[0] * 5, 0, MB, NB, HKV, 24, BS, 1, 1)) == -2
    assert call(2, u64(*[0] * 5, 0, MB, NB, HQ, HKV, D, BS, K, 1, 1, 1, 0, 0)) == 0
    assert call(2, u64(*[0] * 5, 0, MB, NB, HQ, HKV, D, BS, K, 3, 2, 1, 0, 0)) == -1
    assert call(3, u64(*[0] * 7, 0, MB, NB, K, HQ, HKV, D, BS, f32(0.1), 1, 1, f32(1.0), f32(1.0))) == 0
    assert call(3, u64(*[0] * 7, 0, MB, NB, K, HQ, HKV, D, BS, f32(math.nan), 1, 1, f32(1.0), f32(1.0))) == -1
    assert call(4, rotary(T=0)) == -1 and lib.pkv_bound_call(0, None, 28, None) == -1


# -------------------------------------------------------------------- binding
def pools(dtype=BF):
    ks, vs = pkv.pool_shapes(NB, HKV, BS, D, dtype)
    return torch.empty(ks, dtype=dtype), torch.empty(vs, dtype=dtype)


def rotary_args(**over):
    kp, vp = pools()
    a = dict(q_out=torch.empty(T, HQ, D, dtype=BF), q=torch.empty(T, HQ, D, dtype=BF),
             k=torch.empty(T, HKV, D, dtype=BF), v=torch.empty(T, HKV, D, dtype=BF), k_pool=kp, v_pool=vp,
             slot_mapping=torch.zeros(T, dtype=I64), positions=torch.zeros(T, dtype=I32),
             cos_sin=torch.zeros(16, 2, D // 2))
    a.update(over)
    return a


@pytest.mark.parametrize("over,exc", [
    (dict(q=torch.empty(T, HQ * D, dtype=BF)), ValueError),
    (dict(q_out=torch.empty(T, HQ, D)), ValueError),
    (dict(k=torch.empty(T - 1, HKV, D, dtype=BF)), ValueError),
    (dict(v=torch.empty(T, HKV, D)), ValueError),
    (dict(slot_mapping=torch.zeros(T, dtype=I32)), TypeError),
    (dict(positions=torch.zeros(T, dtype=I64)), TypeError),
    (dict(positions=torch.zeros(T + 1, dtype=I32)), ValueError),
    (dict(positions=torch.zeros(3, T, dtype=I32)), ValueError),                # no sections
    (dict(positions=torch.zeros(2, T, dtype=I32), sections=[16, 15]), ValueError),
    (dict(sections=[40, -8], positions=torch.zeros(2, T, dtype=I32)), ValueError),
    (dict(cos_sin=torch.zeros(16, 2, D // 2, dtype=torch.float64)), TypeError),
    (dict(cos_sin=torch.zeros(16, D)), ValueError),
    (dict(q=torch.empty(T, D, HQ, dtype=BF).transpose(1, 2)), ValueError),     # heads not contiguous
    (dict(q_out=torch.empty(1, HQ, D, dtype=BF).expand(T, HQ, D)), ValueError),
    (dict(k_pool=torch.empty(NB, HKV, BS, D, dtype=BF)), ValueError),
    ({}, TypeError),                                                           # on the host
])
def test_rotary_binding_refuses(over, exc):
    with pytest.raises(exc):
        pkv.rotary_and_cache(**rotary_args(**over))


def bounds_args(**over):
    a = dict(k_pool=pools()[0], key_bounds=torch.empty(NB, HKV, 2, D, dtype=BF),
             block_tables=torch.zeros(B, MB, dtype=I32), seq_lens=torch.zeros(B, dtype=I32),
             first_changed=torch.zeros(B, dtype=I32))
    a.update(over)
    return a


@pytest.mark.parametrize("over,exc", [
    (dict(key_bounds=torch.empty(NB, HKV, D, dtype=BF)), ValueError),
    (dict(key_bounds=torch.empty(NB - 1, HKV, 2, D, dtype=BF)), ValueError),
    (dict(key_bounds=torch.empty(NB, HKV, 2, D)), TypeError),
    (dict(first_changed=torch.zeros(B + 1, dtype=I32)), ValueError),
    (dict(first_changed=torch.zeros(B, dtype=I64)), TypeError),
    (dict(block_tables=torch.zeros(B + 1, MB, dtype=I32)), ValueError),
    (dict(k_pool=torch.empty(NB, HKV, BS, D, dtype=BF)), ValueError),
    ({}, TypeError),
])
def test_bounds_binding_refuses(over, exc):
    with pytest.raises(exc):
        pkv.update_key_bounds(**bounds_args(**over))


def select_args(**over):
    a = dict(selected=torch.empty(B, HKV, K, dtype=I32), q=torch.empty(B, HQ, D, dtype=BF),
             key_bounds=torch.empty(NB, HKV, 2, D, dtype=BF), block_tables=torch.zeros(B, MB, dtype=I32),
             seq_lens=torch.zeros(B, dtype=I32), block_size=BS)
    a.update(over)
    return a


@pytest.mark.parametrize("over,exc", [
    (dict(selected=torch.empty(B, HKV, K, dtype=I64)), TypeError),
    (dict(selected=torch.empty(B, HKV * K, dtype=I32)), ValueError),
    (dict(selected=torch.empty(B + 1, HKV, K, dtype=I32)), ValueError),
    (dict(key_bounds=torch.empty(NB, HKV + 1, 2, D, dtype=BF)), ValueError),
    (dict(key_bounds=torch.empty(NB, HKV, 2, D)), TypeError),
    (dict(q=torch.empty(B, HQ, D)), TypeError),                                # bounds of another type
    (dict(seq_lens=torch.zeros(B + 1, dtype=I32)), ValueError),
    ({}, TypeError),
])
def test_select_binding_refuses(over, exc):
    with pytest.raises(exc):
        pkv.select_blocks(**select_args(**over))


@pytest.mark.parametrize("over,exc", [
    (dict(selected=torch.empty(B, HKV, K, dtype=I64)), TypeError),
    (dict(selected=torch.empty(B, HQ, K, dtype=I32)), ValueError),
    (dict(selected=torch.empty(B, K, dtype=I32)), ValueError),
    (dict(q=torch.empty(B, HQ, 2 * D, dtype=BF), out=torch.empty(B, HQ, 2 * D, dtype=BF)), ValueError),
    ({}, TypeError),
])
def test_sparse_binding_refuses(over, exc):
    kp, vp = pools()
    a = dict(out=torch.empty(B, HQ, D, dtype=BF), q=torch.empty(B, HQ, D, dtype=BF), k_pool=kp, v_pool=vp,
             block_tables=torch.zeros(B, MB, dtype=I32), seq_lens=torch.zeros(B, dtype=I32),
             selected=torch.empty(B, HKV, K, dtype=I32), scale=0.1)
    a.update(over)
    with pytest.raises(exc):
        pkv.paged_attention_decode_sparse(**a)


# --------------------------------------------------------------- host helpers
def test_rotary_table_is_right_at_far_positions():
    """Within one float32 rounding (2^-24 of a value of at most 1, doubled for the
    float64 sine's argument) of the angle formed exactly as a rational multiple."""
    P, R = 1 << 20, 64
    t = pkv.rotary_table(P, R, base=10000.0)
    assert t.shape == (P, 2, R // 2) and t.dtype == F32
    for p in (0, 1, 777, P - 1):
        for i in (0, 1, 31):
            angle = p * 10000.0 ** (-2.0 * i / R)
            assert abs(t[p, 0, i].item() - math.cos(angle)) <= 2 ** -23
            assert abs(t[p, 1, i].item() - math.sin(angle)) <= 2 ** -23
    half = pkv.rotary_table(9, R, stretch=2.0)
    assert torch.equal(half[8], pkv.rotary_table(5, R)[4])
    for bad in ((0, 64, 1e4, 1.0), (8, 63, 1e4, 1.0), (8, 64, 0.0, 1.0), (8, 64, 1e4, 0.0)):
        with pytest.raises(ValueError):
            pkv.rotary_table(*bad)


def test_first_changed_of_plans():
    from paged_kv_cache_259_gb300 import engine
    z = np.zeros(0)
    lens = np.array([1, 40, 17], dtype=np.int32)
    assert list(engine.first_changed(engine.StepPlan(z, z, z, z, lens))) == [0, 39, 16]
    plan = engine.PrefillPlan(z, np.array([1, 40, 5], dtype=np.int64), z, z, z, lens, z)
    f = engine.first_changed(plan)
    assert list(f) == [0, 0, 12] and f.dtype == np.int32


# ---------------------------------------------------------------- oracle pins
def test_oracle_rotation_by_a_quarter_turn():
    cos, sin = np.zeros((1, 2), np.float32), np.ones((1, 2), np.float32)
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    assert olc.rotate_f64(x, cos, sin, False).tolist() == [[[-3.0, -4.0, 1.0, 2.0, 9.0]]]
    assert olc.rotate_f32(x, cos, sin, True).tolist() == [[[-2.0, 1.0, -4.0, 3.0, 9.0]]]


def test_oracle_turns_take_each_axis_its_section():
    table = np.arange(10 * 2 * 3, dtype=np.float32).reshape(10, 2, 3)
    cos, sin = olc.turns(np.array([[1, 4], [7, 9]]), table, [1, 2])
    assert cos.tolist() == [[table[1, 0, 0], table[7, 0, 1], table[7, 0, 2]],
                            [table[4, 0, 0], table[9, 0, 1], table[9, 0, 2]]]
    assert sin[1, 2] == table[9, 1, 2]


def test_oracle_score_bounds_every_key_of_the_block():
    rng = np.random.default_rng(0)
    for _ in range(50):
        k, q = rng.standard_normal((16, 8)), rng.standard_normal((4, 8))
        n = int(rng.integers(1, 17))
        s = olc.block_scores(q, olc.key_bounds(k, n)[None])[0]
        assert s >= (q @ k[:n].T).max() - 1e-12
    one = olc.block_scores(q, olc.key_bounds(k, 1)[None])[0]      # one key: the logit itself
    assert abs(one - (q @ k[0]).max()) < 1e-12
    assert np.isinf(olc.block_scores(q, np.full((1, 2, 8), np.nan))[0])


def test_oracle_select_ties_forced_blocks_and_short_rows():
    s = np.array([9.0, 1, 5, 5, 7, 5, 0, 0])
    assert olc.select(s, 4, 0, 0).tolist() == [0, 2, 3, 4]         # tie of 5s: the lower indices
    assert olc.select(s, 4, 1, 2).tolist() == [0, 4, 6, 7]
    assert olc.select(s, 3, 1, 2).tolist() == [0, 6, 7]            # nothing left to score
    assert olc.select(s[:3], 4, 1, 2).tolist() == [0, 1, 2]
    assert olc.select(s[:0], 4, 1, 2).tolist() == []
