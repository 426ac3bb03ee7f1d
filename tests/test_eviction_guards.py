"""The cache eviction operators without a GPU: refusals of the C entries and of the binding
(before any pointer reaches a kernel), and the oracle's definitions against hand-worked cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

from _lib import library, pkv
from oracle import eviction as oev

B, HQ, HKV, D, BS, NB, MB, T, K, ROWS, CAP = 3, 4, 2, 64, 16, 8, 5, 7, 4, 6, 80
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
SOME, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module", autouse=True)
def lib():
    return library()


def at(n, i, value):
    a = [SOME] * n
    a[i] = value
    return a


# ------------------------------------------------------------------ C entries
def c_norm(ptrs=None, strides=(256, 256, 128, 128), steps=(0, 0), T=T, Hq=HQ, Hkv=HKV, D=D, R=64, bs=BS, src=1,
           cache=1, wdt=1, eps=1e-6, ks=1.0, vs=1.0, sections=(32,), sec_ptr=True):
    a = ptrs or [ctypes.c_void_p(0x2000)] + [SOME] * 10
    sec = (ctypes.c_int32 * len(sections))(*sections) if sec_ptr else None
    return library().norm_rotary_and_cache(*a, sec, len(sections), *strides, *steps, T, Hq, Hkv, D, R, 0, bs, NB, 64,
                                           src, cache, wdt, eps, ks, vs, None)


@pytest.mark.parametrize("over,status", [
    (dict(eps=-1e-6), -1), (dict(eps=math.nan), -1), (dict(eps=math.inf), -1), (dict(steps=(60, 0)), -1),
    (dict(steps=(0, 68)), -1), (dict(steps=(-64, 0)), -1), (dict(steps=(0, 1 << 33)), -1),
    (dict(ptrs=at(11, 4, None)), -1), (dict(ptrs=at(11, 5, None)), -1), (dict(ptrs=at(11, 4, ODD)), -1),
    (dict(ptrs=at(11, 5, ctypes.c_void_p(0x1008))), -1),
    (dict(wdt=2), -2), (dict(src=0, cache=0, wdt=1, strides=(256, 256, 128, 128)), -2),
    (dict(D=528, R=64, Hq=1, Hkv=1, strides=(528,) * 4), -2),
    # rotary_and_cache's own
    (dict(T=-1), -1), (dict(Hq=3), -1), (dict(R=80), -1), (dict(sec_ptr=False), -1), (dict(sections=(31,)), -1),
    (dict(strides=(255, 256, 128, 128)), -1), (dict(ks=2.0), -1), (dict(cache=2, vs=0.0), -1),
    (dict(ptrs=at(11, 0, None)), -1), (dict(bs=24), -2), (dict(src=0, cache=1), -2),
    (dict(T=0, ptrs=[None] * 11), 0), (dict(T=0, steps=(64, 64)), 0),
])
def test_norm_entry_refuses_before_any_cuda_call(over, status):
    assert c_norm(**over) == status


def c_decode(ptrs=None, B=B, MB=MB, NB=NB, rows=ROWS, cap=CAP, Hq=HQ, Hkv=HKV, D=D, bs=BS, scale=0.1, decay=1.0,
             qd=1, kv=1, ks=1.0, vs=1.0, ws=SOME, ws_bytes=1 << 30):
    return library().paged_attention_decode_weighed(*(ptrs or [SOME] * 8), B, MB, NB, rows, cap, Hq, Hkv, D, bs, scale,
                                                    decay, qd, kv, ks, vs, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(B=65536), -1), (dict(MB=0), -1), (dict(NB=0), -1), (dict(rows=0), -1), (dict(Hq=5), -1),
    (dict(cap=79), -1), (dict(cap=76), -1), (dict(cap=82), -1), (dict(ptrs=at(8, 2, None), rows=2), -1),
    (dict(scale=math.nan), -1), (dict(decay=-0.1), -1), (dict(decay=1.1), -1), (dict(decay=math.nan), -1),
    (dict(ks=2.0), -1), (dict(kv=2, vs=0.0), -1), (dict(kv=2, ks=math.inf), -1),
    (dict(ptrs=at(8, 0, None)), -1), (dict(ptrs=at(8, 1, None)), -1), (dict(ptrs=at(8, 1, ODD)), -1),
    (dict(ptrs=at(8, 3, ctypes.c_void_p(0x1008))), -1), (dict(ptrs=at(8, 5, ODD)), -1), (dict(ptrs=at(8, 7, None)), -1),
    (dict(ws=None), -1), (dict(ws=ODD), -1), (dict(ws_bytes=1 << 10), -1), (dict(MB=1 << 27, cap=1 << 30), -1),
    (dict(Hq=6), -2), (dict(Hq=32), -2), (dict(D=96), -2), (dict(bs=48, cap=240), -2), (dict(qd=0, kv=1), -2),
    (dict(qd=0, kv=2), -2), (dict(B=40000), -2),
    (dict(B=0, ptrs=[None] * 8), 0),
])
def test_decode_entry_refuses_before_any_cuda_call(over, status):
    assert c_decode(**over) == status


def c_prompt(ptrs=None, B=B, most=7, window=0, MB=MB, NB=NB, rows=ROWS, cap=CAP, Hq=HQ, Hkv=HKV, D=D, bs=BS,
             scale=0.1, decay=1.0, qd=1, kv=1, ws=SOME, ws_bytes=1 << 30):
    return library().weigh_prefill_tokens(*(ptrs or [SOME] * 7), B, most, window, MB, NB, rows, cap, Hq, Hkv, D, bs,
                                          scale, decay, qd, kv, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(most=-1), -1), (dict(window=-1), -1), (dict(MB=0), -1), (dict(rows=0), -1),
    (dict(Hq=3), -1), (dict(cap=76), -1), (dict(cap=82), -1), (dict(ptrs=at(7, 1, None), rows=2), -1),
    (dict(scale=math.inf), -1), (dict(decay=2.0), -1), (dict(decay=math.nan), -1),
    (dict(ptrs=at(7, 0, None)), -1), (dict(ptrs=at(7, 0, ODD)), -1), (dict(ptrs=at(7, 2, ODD)), -1),
    (dict(ptrs=at(7, 3, ODD)), -1), (dict(ptrs=at(7, 6, None)), -1), (dict(ws=None), -1), (dict(ws=ODD), -1),
    (dict(ws_bytes=64), -1), (dict(MB=1 << 27, cap=1 << 30), -1),
    (dict(D=96), -2), (dict(bs=48, cap=240), -2), (dict(qd=0, kv=0), -2), (dict(kv=2), -2),
    (dict(Hq=129, Hkv=1), -2), (dict(B=40000), -2), (dict(MB=1 << 21, cap=1 << 25), -2),
    (dict(B=0, ptrs=[None] * 7), 0), (dict(most=0, ptrs=[None] * 7), 0),
])
def test_prompt_entry_refuses_before_any_cuda_call(over, status):
    assert c_prompt(**over) == status


def c_select(ptrs=None, B=B, Hkv=HKV, rows=ROWS, cap=CAP, K=K, F=1, N=1):
    return library().select_tokens(*(ptrs or [SOME] * 4), B, Hkv, rows, cap, K, F, N, None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(B=65536), -1), (dict(Hkv=0), -1), (dict(rows=0), -1), (dict(cap=0), -1), (dict(cap=82), -1),
    (dict(K=0), -1), (dict(F=-1), -1), (dict(N=-1), -1), (dict(F=3, N=2), -1), (dict(F=5, N=0), -1),
    (dict(ptrs=at(4, 2, None), rows=2), -1), (dict(ptrs=at(4, 0, None)), -1), (dict(ptrs=at(4, 1, ODD)), -1),
    (dict(ptrs=at(4, 3, None)), -1), (dict(B=65535, Hkv=65535), -2), (dict(cap=(1 << 30) + 4), -2),
    (dict(B=0, ptrs=[None] * 4), 0),
])
def test_select_entry_refuses_before_any_cuda_call(over, status):
    assert c_select(**over) == status


def c_keep(ptrs=None, B=B, K=K, MB=MB, MK=1, NB=NB, rows=ROWS, cap=CAP, Hkv=HKV, D=D, bs=BS, kv=1):
    return library().keep_tokens(*(ptrs or [SOME] * 8), B, K, MB, MK, NB, rows, cap, Hkv, D, bs, kv, None)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -1), (dict(K=0), -1), (dict(K=17), -1), (dict(MB=0), -1), (dict(MK=0), -1), (dict(NB=0), -1),
    (dict(Hkv=0), -1), (dict(rows=0), -1), (dict(cap=76), -1), (dict(cap=82), -1),
    (dict(ptrs=at(8, 2, None), rows=2), -1), (dict(ptrs=at(8, 1, ODD)), -1), (dict(ptrs=at(8, 0, None)), -1),
    (dict(ptrs=at(8, 3, ODD)), -1), (dict(ptrs=at(8, 4, None)), -1), (dict(ptrs=at(8, 6, None)), -1),
    (dict(MB=1 << 28), -1), (dict(D=24), -2), (dict(D=528), -2), (dict(bs=24, cap=120), -2), (dict(kv=3), -2),
    (dict(B=65535, Hkv=65535), -2), (dict(B=0, ptrs=[None] * 8), 0),
])
def test_keep_entry_refuses_before_any_cuda_call(over, status):
    assert c_keep(**over) == status


def test_workspaces():
    lib = library()
    assert lib.weighed_decode_workspace_size(0, 4, 64, 16, 5) == 0
    # 80 tokens pad to 96; at most 4096 partitions of 8 heads and one a head
    assert lib.weighed_decode_workspace_size(3, 4, 64, 16, 5) == 4 * (12 * 96 + (8 * 4096 + 12) * 66)
    assert lib.weighed_decode_workspace_size(64, 64, 128, 16, 1 << 14) > 4 << 30     # beyond 32 bits
    assert lib.weigh_prefill_workspace_size(2, 4, 0, 0) == 0 and lib.weigh_prefill_workspace_size(2, 4, 5, -1) == 0
    assert lib.weigh_prefill_workspace_size(2, 4, 9, 0) == lib.weigh_prefill_workspace_size(2, 4, 9, 11)
    assert lib.weigh_prefill_workspace_size(2, 4, 9, 3) < lib.weigh_prefill_workspace_size(2, 4, 9, 0)


# -------------------------------------------------------------------- binding
def base():
    ks, vs = pkv.pool_shapes(NB, HKV, BS, D, BF)
    return dict(k_pool=torch.empty(ks, dtype=BF), v_pool=torch.empty(vs, dtype=BF),
                token_weights=torch.empty(ROWS, HKV, CAP), weight_rows=torch.empty(B, dtype=I32),
                block_tables=torch.empty(B, MB, dtype=I32), seq_lens=torch.empty(B, dtype=I32))


def norm_args(**over):
    p = base()
    a = dict(q_out=torch.empty(T, HQ, D, dtype=BF), q=torch.empty(T, HQ, D, dtype=BF),
             k=torch.empty(T, HKV, D, dtype=BF), v=torch.empty(T, HKV, D, dtype=BF), q_weight=torch.empty(D, dtype=BF),
             k_weight=torch.empty(HKV, D, dtype=BF), k_pool=p["k_pool"], v_pool=p["v_pool"],
             slot_mapping=torch.empty(T, dtype=I64), positions=torch.empty(T, dtype=I32),
             cos_sin=torch.empty(64, 2, 32))
    a.update(over)
    return a


def decode_args(**over):
    a = base()
    a.update(out=torch.empty(B, HQ, D, dtype=BF), q=torch.empty(B, HQ, D, dtype=BF), scale=0.1)
    a.update(over)
    return a


def prompt_args(**over):
    a = base()
    del a["v_pool"]
    a.update(q=torch.empty(T, HQ, D, dtype=BF), query_start=torch.empty(B + 1, dtype=I32), scale=0.1, max_query_len=4)
    a.update(over)
    return a


def select_args(**over):
    p = base()
    a = {k: p[k] for k in ("token_weights", "weight_rows", "seq_lens")}
    a["kept"] = torch.empty(B, HKV, K, dtype=I32)
    a.update(over)
    return a


def keep_args(**over):
    a = base()
    a.update(kept=torch.empty(B, HKV, K, dtype=I32), kept_tables=torch.empty(B, 1, dtype=I32))
    a.update(over)
    return a


E = torch.empty
REFUSED = [
    ("norm", norm_args, [
        (dict(q_weight=E(D + 1, dtype=BF)), ValueError), (dict(k_weight=E(HQ, D, dtype=BF)), ValueError),
        (dict(q_weight=E(1, HQ, D, dtype=BF)), ValueError), (dict(q_weight=E(D)), TypeError),
        (dict(q_weight=E(D, dtype=torch.float16), k_weight=E(D, dtype=torch.float16)), TypeError),
        (dict(q_weight=E(2 * D, dtype=BF)[::2]), ValueError), (dict(q=None), TypeError), (dict(k_weight=None), TypeError),
        (dict(slot_mapping=E(T, dtype=I32)), TypeError), (dict(k=E(T, HKV, D + 16, dtype=BF)), ValueError),
        (dict(sections=[16, 16]), ValueError)]),
    ("decode", decode_args, [
        (dict(token_weights=E(ROWS, HKV, CAP, dtype=BF)), TypeError), (dict(token_weights=E(ROWS, HKV + 1, CAP)), ValueError),
        (dict(token_weights=E(ROWS, CAP)), ValueError), (dict(weight_rows=E(B, dtype=I64)), TypeError),
        (dict(weight_rows=E(B + 1, dtype=I32)), ValueError), (dict(weight_rows=None, token_weights=E(B - 1, HKV, CAP)), ValueError),
        (dict(out=E(B, HQ, D)), ValueError), (dict(seq_lens=E(B, dtype=I64)), TypeError), (dict(token_weights=None), TypeError)]),
    ("prompt", prompt_args, [
        (dict(token_weights=E(ROWS, HKV, CAP, dtype=BF)), TypeError), (dict(weight_rows=E(B - 1, dtype=I32)), ValueError),
        (dict(q=E(T, HQ, D + 16, dtype=BF)), ValueError), (dict(query_start=E(B, dtype=I32)), ValueError),
        (dict(query_start=E(B + 1, dtype=I64)), TypeError), (dict(block_tables=E(B + 1, MB, dtype=I32)), ValueError),
        (dict(k_pool=E(2, 2)), ValueError)]),
    ("select", select_args, [
        (dict(kept=E(B, HKV, K, dtype=I64)), TypeError), (dict(kept=E(B, HKV + 1, K, dtype=I32)), ValueError),
        (dict(seq_lens=E(B + 1, dtype=I32)), ValueError), (dict(token_weights=E(ROWS, HKV, CAP).double()), TypeError),
        (dict(weight_rows=E(B, 1, dtype=I32)), ValueError)]),
    ("keep", keep_args, [
        (dict(kept=E(B, HKV + 1, K, dtype=I32)), ValueError), (dict(kept_tables=E(B + 1, 1, dtype=I32)), ValueError),
        (dict(kept_tables=E(B, 1, dtype=I64)), TypeError), (dict(v_pool=E(2, 2)), ValueError),
        (dict(token_weights=E(ROWS, HKV + 1, CAP)), ValueError), (dict(seq_lens=E(B + 2, dtype=I32)), ValueError)]),
]
CALLS = {"norm": "norm_rotary_and_cache", "decode": "paged_attention_decode_weighed", "prompt": "weigh_prefill_tokens",
         "select": "select_tokens", "keep": "keep_tokens"}


@pytest.mark.parametrize("op,make,over,error", [(o, m, d, e) for o, m, cases in REFUSED for d, e in cases])
def test_binding_refuses(op, make, over, error):
    with pytest.raises(error):
        getattr(pkv, CALLS[op])(**make(**over))


@pytest.mark.parametrize("op,make", [(o, m) for o, m, _ in REFUSED])
def test_binding_wants_gpu_tensors(op, make):
    with pytest.raises(TypeError, match="CUDA"):           # every other check passed
        getattr(pkv, CALLS[op])(**make())


def test_token_weights_shape():
    assert pkv.token_weights_shape(3, 2, 77) == (3, 2, 80)


# --------------------------------------------------------------------- oracle
def test_oracle_norm_by_hand():
    y = oev.normed([[3.0, 4.0]], [1.0, 2.0], 0.0)          # mean square 12.5
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]], rtol=1e-15)


def test_oracle_weights_by_hand():
    k = np.array([[0.0], [math.log(2.0)], [math.log(5.0)]])
    assert np.allclose(oev.decode_weights([[1.0]], k, 1.0), [[1 / 8, 2 / 8, 5 / 8]])
    assert np.allclose(oev.decode_weights([[1.0]], k, 1.0, missing=[1]), [[1 / 6, 0, 5 / 6]])
    p = oev.prompt_weights([[[1.0]], [[1.0]]], k, 1.0)     # the first of two queries sees two tokens
    assert np.allclose(p[:, 0], [[1 / 3, 2 / 3, 0], [1 / 8, 2 / 8, 5 / 8]])
    assert np.allclose(oev.updated([4.0, 4.0, 9.0, 9.0], np.array([1.0, 1.0, 1.0]), 1, 0.5), [3.0, 3.0, 1.0])
    assert np.array_equal(oev.softmax([-np.inf, -np.inf]), [0.0, 0.0])
    assert np.isnan(oev.softmax([0.0, np.inf])).all() and np.isnan(oev.softmax([0.0, np.nan])).all()


def test_oracle_select_by_hand():
    w = np.array([0.0, 5.0, 1.0, 5.0, 1.0, 9.0])
    assert oev.select(w, 6, 3, 0, 0) == [1, 3, 5]
    assert oev.select(w, 6, 3, 1, 1) == [0, 1, 5]
    assert oev.select(w, 6, 4, 0, 0) == [1, 2, 3, 5]       # equal: the lower token
    assert oev.select(w, 4, 5, 1, 1) == [0, 1, 2, 3, -1]
    assert oev.select([1.0, np.nan, 7.0, -np.inf], 4, 2, 0, 0) == [1, 3]
