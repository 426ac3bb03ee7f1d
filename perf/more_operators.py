"""Cases of the cache eviction operators: the append with normalised and rotated heads,
decode attention that adds up the weight every cached token gets, the same weights
from a prompt's last queries, the choice of the tokens to keep, and their move into
fresh blocks.

``run`` computes one pass either in plain torch (``own`` false) or with the
framework's calls (``own`` true), on the same state. The pools have the library's
layout: K ``[NB, Hkv, bs/8, D/X, 8, X]`` and V ``[NB, Hkv, bs/X, D/8, 8, X]`` with X
elements in 16 bytes. Token weights are ``[rows, Hkv, max_tokens]`` float32; sequence
b's are row ``rows[b]``.
"""
import math

import torch

own = False

TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
         "e4m3": (torch.bfloat16, torch.uint8)}      # (activations, cache)
ELT = {"f32": 4, "bf16": 2, "e4m3": 1}
K_SCALE, V_SCALE = 0.037, 0.041                     # E4M3 caches: value = code * scale
F8 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a 64-sequence batch: q, k, v are views of the fused projection, one
        # weight vector for all heads of q, one for k
        {"name": "norm rotary decode 64", "op": "norm", "type": "bf16", "seqs": 64, "tokens": 1, "len": 32768,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "R": 128, "axes": 1, "interleaved": False, "fused": True,
         "per_head": False},
        # a prompt with image tokens (time, height, width), 16 sequences' chunks of 512, weights of each head
        {"name": "norm rotary chunk 8192 3 axes", "op": "norm", "type": "bf16", "seqs": 16, "tokens": 512, "len": 4096,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "R": 128, "axes": 3, "interleaved": False, "fused": True,
         "per_head": True},
        # one conversation whose cache is held at 4096 tokens: latency
        {"name": "weighed decode 1 x 4096", "op": "decode", "type": "bf16", "seqs": 1, "len": 4096, "decay": 1.0,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # a batch of them, quantised, older weights fading
        {"name": "weighed decode 64 x 4096 e4m3", "op": "decode", "type": "e4m3", "seqs": 64, "len": 4096,
         "decay": 0.999, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # multi-head attention, ragged lengths
        {"name": "weighed decode 32 x 8192 mha", "op": "decode", "type": "bf16", "seqs": 32, "len": 8192, "decay": 1.0,
         "Hq": 40, "Hkv": 40, "D": 128, "bs": 16},
        # float32, small heads, an empty sequence
        {"name": "weighed decode f32 3 x 500", "op": "decode", "type": "f32", "seqs": 3, "len": 500, "decay": 1.0,
         "Hq": 8, "Hkv": 8, "D": 64, "bs": 32},
        # long prompts just prefilled, weighed by their last 32 queries
        {"name": "weigh prompt 4 x 32768 last 32", "op": "prompt", "type": "bf16", "seqs": 4, "chunk": 512,
         "len": 32768, "window": 32, "decay": 1.0, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # every query of a chunk counts; eight query heads a kv head
        {"name": "weigh chunk 4 x 2048", "op": "prompt", "type": "bf16", "seqs": 4, "chunk": 2048, "len": 4096,
         "window": 0, "decay": 1.0, "Hq": 32, "Hkv": 4, "D": 128, "bs": 16},
        # one long conversation to a small cache
        {"name": "select 4096 of 1 x 131072", "op": "select", "seqs": 1, "len": 131072, "K": 4096, "first": 4,
         "last": 256, "Hkv": 8, "bs": 16},
        # a batch's regular trim: half of each ragged cache
        {"name": "select 4096 of 64 x 8192", "op": "select", "seqs": 64, "len": 8192, "K": 4096, "first": 4,
         "last": 64, "Hkv": 8, "bs": 16},
        # what was kept of a quantised cache moves, odd counts
        {"name": "keep 999 of 3 x 2011 e4m3", "op": "keep", "type": "e4m3", "seqs": 3, "len": 2011, "K": 999,
         "Hkv": 8, "D": 128, "bs": 32},
        # a batch's regular trim
        {"name": "keep 4096 of 64 x 8192", "op": "keep", "type": "bf16", "seqs": 64, "len": 8192, "K": 4096,
         "Hkv": 8, "D": 128, "bs": 16},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "decode", "prompt", "select", "keep"])
    kind = rng.choice(["bf16", "bf16", "e4m3", "f32"])
    D, bs = rng.choice([64, 128]), rng.choice([16, 32])
    G, Hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if op == "norm":
        D = rng.choice([64, 128, 128, 80, 256])
        tokens = rng.choice([1, _log(rng, 2, 900)])
        R = rng.choice([D, D, D // 4 // 16 * 16 or 16])
        return {"op": op, "type": kind, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "bs": bs,
                "seqs": _log(rng, 1, max(1, min(200, 4096 // tokens))), "tokens": tokens,
                "len": tokens + _log(rng, 1, 16384), "R": R, "axes": rng.choice([1, 1, 2, 3]) if R >= 32 else 1,
                "interleaved": rng.random() < 0.4, "fused": rng.random() < 0.6, "per_head": rng.random() < 0.4}
    if op == "decode":
        seqs = _log(rng, 1, 64)
        return {"op": op, "type": kind, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "bs": bs, "seqs": seqs,
                "len": _log(rng, 1, min(131072, (1 << 18) // seqs)), "decay": rng.choice([1.0, 0.95])}
    if op == "prompt":
        seqs = _log(rng, 1, 4)
        chunk = _log(rng, 1, 2048)
        window = rng.choice([0, _log(rng, 1, 64)])
        more = 2048 if window == 0 else 30000
        return {"op": op, "type": "bf16", "Hq": G * min(Hkv, 4), "Hkv": min(Hkv, 4), "D": D, "bs": bs, "seqs": seqs,
                "chunk": chunk, "len": chunk + _log(rng, 1, more), "window": window, "decay": rng.choice([1.0, 0.95])}
    seqs = _log(rng, 1, 64)
    length = _log(rng, 2, min(131072, (1 << 19) // seqs))
    K = _log(rng, 1, length)
    if op == "select":
        first = rng.randint(0, min(K, 8))
        return {"op": op, "seqs": seqs, "len": length, "K": K, "first": first,
                "last": rng.randint(0, min(K - first, 300)), "Hkv": Hkv, "bs": bs}
    return {"op": op, "type": kind, "seqs": seqs, "len": length, "K": K, "Hkv": Hkv, "D": D, "bs": bs}


def _lens(c):
    """The sequences' lengths, from the case alone: the longest first, then spread
    over (0, len] (over its upper part where caches are held near one size); the last
    one empty where the attention has three or more."""
    low = max(c.get("tokens", 1), c.get("chunk", 1))
    spread = [(0.6180339887498949 * i) % 1.0 or 1.0 for i in range(c["seqs"])]
    if c["op"] in ("select", "keep"):
        spread = [1.0 - 0.5 * (1.0 - x) for x in spread]
    lens = [max(low, int(c["len"] * x)) for x in spread]
    if c["op"] == "decode" and c["seqs"] >= 3:
        lens[-1] = 0
    return lens


def _chunks(c):
    """The new tokens of each sequence of a prompt step, ragged."""
    return [max(1, int(c["chunk"] * ((0.7548776662466927 * i) % 1.0 or 1.0))) for i in range(c["seqs"])]


def _watched(c):
    """The queries of each chunk that count."""
    return [min(n, c["window"] or n) for n in _chunks(c)]


def work(c):
    lens, Hkv = _lens(c), c["Hkv"]
    if c["op"] == "norm":
        Hq, D, act = c["Hq"], c["D"], 2 if c["type"] != "f32" else 4
        T = c["seqs"] * c["tokens"]
        rows = len({n - 1 - t for n in lens for t in range(c["tokens"])}) if c["axes"] == 1 else c["len"] // 256 + 33
        weights = (Hq + Hkv if c["per_head"] else 2) * D * act
        return {"bytes": T * D * ((2 * Hq + 2 * Hkv) * act + 2 * Hkv * ELT[c["type"]]) + T * (8 + 4 * c["axes"]) +
                rows * c["R"] * 4 + weights,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * c["R"])}
    if c["op"] == "decode":
        Hq, D, act = c["Hq"], c["D"], 2 if c["type"] != "f32" else 4
        tokens, blocks = sum(lens), sum(-(-n // c["bs"]) for n in lens)
        return {"bytes": tokens * Hkv * (2 * D * ELT[c["type"]] + 8) + 4 * blocks + c["seqs"] * (2 * Hq * D * act + 8),
                "flops": 4 * tokens * Hq * D}
    if c["op"] == "prompt":
        seen = watched = 0
        for L, n in zip(lens, _watched(c)):
            seen += n * L - n * (n - 1) // 2
            watched += n
        return {"bytes": sum(lens) * Hkv * (2 * c["D"] + 8) + sum(-(-n // c["bs"]) for n in lens) * 4 +
                watched * c["Hq"] * c["D"] * 2 + 12 * c["seqs"],
                "flops": 2 * seen * c["Hq"] * c["D"]}
    kept = sum(min(n, c["K"]) for n in lens) * Hkv
    if c["op"] == "select":
        read = sum(n for n in lens if n > c["K"]) * Hkv
        return {"bytes": read * 4 + c["seqs"] * (Hkv * c["K"] * 4 + 8), "flops": read}
    return {"bytes": kept * (4 * c["D"] * ELT[c["type"]] + 12) + sum(-(-n // c["bs"]) for n in lens) * 4, "flops": 0}


# ------------------------------------------------------------- what a program has
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _pools(c, NB, g, keys_only=False):
    """Filled pools of the library's layout: N(0, 1) values, for E4M3 the codes' bytes."""
    X, D, bs = 16 // ELT[c["type"]], c["D"], c["bs"]

    def fill(shape):
        if c["type"] != "e4m3":
            return torch.randn(shape, generator=g, device="cuda", dtype=TYPES[c["type"]][1])
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        return x.mul_(1.0 / K_SCALE).to(F8).view(torch.uint8)

    k = fill((NB, c["Hkv"], bs // 8, D // X, 8, X))
    return k, None if keys_only else fill((NB, c["Hkv"], bs // X, D // 8, 8, X))


def _tables(blocks, ids):
    """Block tables of sequences of these block counts, from a list of block ids."""
    tables = torch.full((len(blocks), max(1, max(blocks))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        tables[b, :n] = ids[at:at + n]
        at += n
    return tables


def _weights(c, lens, g):
    """Accumulated weights as steps leave them: a few heavy tokens, many light ones, ties."""
    cap = -(-max(max(lens), 1) // c["bs"]) * c["bs"]
    shape = (len(lens) + 2, c["Hkv"], cap)
    w = torch.exp(2.0 * torch.randn(shape, generator=g, device="cuda") - 3.0)
    same = torch.rand(shape, generator=g, device="cuda") < 0.3
    w = torch.where(same, torch.round(w * 64.0) / 64.0, w)
    rows = torch.randperm(shape[0], generator=g, device="cuda")[:len(lens)].to(torch.int32)
    return w, rows


def prepare(c, seed):
    g, lens = _gen(seed), _lens(c)
    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    blocks = [-(-n // c["bs"]) for n in lens]
    fresh = [-(-min(n, c["K"]) // c["bs"]) for n in lens] if c["op"] == "keep" else []
    total = sum(blocks) + sum(fresh)
    NB = total + total // 16 + 2
    if c["op"] != "select":
        ids = torch.randperm(NB, generator=g, device="cuda")[:total].to(torch.int32)
        s["tables"] = _tables(blocks, ids)
        s["scales"] = (K_SCALE, V_SCALE) if c["type"] == "e4m3" else (1.0, 1.0)
        s["k_pool"], s["v_pool"] = _pools(c, NB, g, keys_only=c["op"] == "prompt")
    if c["op"] == "norm":
        _prepare_norm(s, c, lens, g)
        return s
    s["weights"], s["rows"] = _weights(c, lens, g)
    if c["op"] == "decode":
        s["q"] = _normal((c["seqs"], c["Hq"], c["D"]), g, TYPES[c["type"]][0]) * 2.0
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(c["D"])
    elif c["op"] == "prompt":
        chunks = _chunks(c)
        start = [0]
        for n in chunks:
            start.append(start[-1] + n)
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["q"] = _normal((start[-1], c["Hq"], c["D"]), g, torch.bfloat16) * 2.0
        s["scale"] = 1.0 / math.sqrt(c["D"])
        s["max_chunk"], s["watched"] = max(chunks), max(_watched(c))
    else:
        s["kept"] = torch.full((c["seqs"], c["Hkv"], c["K"]), -1, dtype=torch.int32, device="cuda")
        if c["op"] == "keep":
            s["fresh"] = _tables(fresh, ids[sum(blocks):])
            # the choice of a random score: min(L, K) positions of every kv head, ascending
            cap = s["weights"].shape[-1]
            t = torch.arange(cap, device="cuda")
            score = torch.rand((c["seqs"], c["Hkv"], cap), generator=g, device="cuda")
            score = score.masked_fill(t >= s["lens"][:, None, None], -1.0)
            top = score.topk(min(c["K"], cap), -1)
            chosen = torch.where(top.values >= 0, top.indices, cap).sort(-1).values
            s["kept"][..., :chosen.shape[-1]] = torch.where(chosen < cap, chosen, -1).to(torch.int32)
    return s


def _prepare_norm(s, c, lens, g):
    act = TYPES[c["type"]][0]
    Hq, Hkv, D, bs, n, T = c["Hq"], c["Hkv"], c["D"], c["bs"], c["tokens"], c["seqs"] * c["tokens"]
    at = (s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")).reshape(-1)
    seq = torch.arange(c["seqs"], device="cuda").repeat_interleave(n)
    s["slots"] = s["tables"][seq, at // bs].long() * bs + at % bs
    if c["axes"] == 1:
        s["positions"] = at.to(torch.int32)
    else:   # time advances by frames of 16 x 16 patches
        grid = [at // 256, at // 16 % 16, at % 16]
        s["positions"] = torch.stack(grid[:c["axes"]]).to(torch.int32)
    half, rest = c["R"] // 2, c["R"] // 2 // c["axes"]
    s["sections"] = [half - rest * (c["axes"] - 1)] + [rest] * (c["axes"] - 1)
    angle = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    s["cos_sin"] = torch.stack([angle.cos(), angle.sin()], 1).float()
    # a projection's heads: of different magnitude, a few strong channels
    gain = torch.exp(0.7 * torch.randn((Hq + 2 * Hkv, 1), generator=g, device="cuda")).repeat(1, D)
    gain[:, ::max(1, D // 4)] *= 4.0
    qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda") * gain).to(act)
    s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
    if not c["fused"]:
        s["q"], s["k"], s["v"] = s["q"].contiguous(), s["k"].contiguous(), s["v"].contiguous()
    of = (lambda h: (h, D)) if c["per_head"] else (lambda h: (D,))
    s["q_weight"] = (1.0 + 0.2 * torch.randn(of(Hq), generator=g, device="cuda")).to(act)
    s["k_weight"] = (1.0 + 0.2 * torch.randn(of(Hkv), generator=g, device="cuda")).to(act)
    s["q_out"] = torch.empty((T, Hq, D), dtype=act, device="cuda")


# ------------------------------------------------------------------- one pass
def _bound_call(s, bind):
    """A serving loop checks and binds its buffers once and launches on them many times."""
    if "call" not in s:
        s["call"] = bind()
    s["call"]()


def run(s):
    op = s["case"]["op"]
    if op == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    if op == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    if op == "prompt":
        return _own_prompt(s) if own else _plain_prompt(s)
    if op == "select":
        return _own_select(s) if own else _plain_select(s)
    return _own_keep(s) if own else _plain_keep(s)


def _as_values(pool):
    return pool.view(F8) if pool.dtype == torch.uint8 else pool


def _own_norm(s):
    import paged_kv_cache_259_gb300 as pkv
    _bound_call(s, lambda: pkv.bind_norm_rotary_and_cache(
        s["q_out"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["k_pool"], s["v_pool"], s["slots"],
        s["positions"], s["cos_sin"], eps=EPS, sections=s["sections"], interleaved=s["case"]["interleaved"],
        k_scale=s["scales"][0], v_scale=s["scales"][1]))
    return s["q_out"], _as_values(s["k_pool"]), _as_values(s["v_pool"])


def _own_decode(s):
    import paged_kv_cache_259_gb300 as pkv
    c = s["case"]

    def bind():   # the scratch is the program's, like that of the split decode
        n = pkv.weighed_decode_workspace_size(c["seqs"], c["Hq"], c["D"], c["bs"], s["tables"].shape[1])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return pkv.bind_paged_attention_decode_weighed(
            s["out"], s["weights"], s["rows"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["scale"],
            decay=c["decay"], k_scale=s["scales"][0], v_scale=s["scales"][1], workspace=s["workspace"])

    _bound_call(s, bind)
    return s["out"], s["weights"]


def _own_prompt(s):
    import paged_kv_cache_259_gb300 as pkv
    c = s["case"]

    def bind():
        n = pkv.weigh_prefill_workspace_size(c["seqs"], c["Hq"], s["max_chunk"], c["window"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return pkv.bind_weigh_prefill_tokens(
            s["weights"], s["rows"], s["q"], s["k_pool"], s["tables"], s["lens"], s["start"], s["scale"],
            s["max_chunk"], window=c["window"], decay=c["decay"], workspace=s["workspace"])

    _bound_call(s, bind)
    return s["weights"]


def _own_select(s):
    import paged_kv_cache_259_gb300 as pkv
    _bound_call(s, lambda: pkv.bind_select_tokens(s["kept"], s["weights"], s["rows"], s["lens"],
                                                  first_tokens=s["case"]["first"], last_tokens=s["case"]["last"]))
    return s["kept"]


def _own_keep(s):
    import paged_kv_cache_259_gb300 as pkv
    _bound_call(s, lambda: pkv.bind_keep_tokens(s["kept"], s["weights"], s["rows"], s["k_pool"], s["v_pool"],
                                                s["tables"], s["fresh"], s["lens"]))
    return _as_values(s["k_pool"]), _as_values(s["v_pool"]), s["weights"]


# ---------------------------------------------------------------- plain forms
def _codes(x, scale):
    """E4M3 bytes of x / scale, saturating."""
    return (x / torch.full((), scale, device=x.device)).clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def _normed(x, weight):
    """float32 heads ``[T, H, D]`` over their root mean square, times the weights."""
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _rotated(x, c, s, R, interleaved):
    """Heads ``[T, H, D]`` with the first R dims rotated, cos and sin ``[T, 1, R/2]``."""
    r, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _plain_norm(s):
    c, slots = s["case"], s["slots"]
    kp, vp, D, bs, Hkv = s["k_pool"], s["v_pool"], c["D"], c["bs"], c["Hkv"]
    X, T = kp.shape[-1], slots.shape[0]
    positions = s["positions"].long().reshape(-1, T)
    axis = torch.repeat_interleave(torch.arange(positions.shape[0], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"))
    pair = torch.arange(c["R"] // 2, device="cuda")
    p = positions[axis].t()                                        # [T, R/2]
    cos, sin = s["cos_sin"][p, 0, pair][:, None], s["cos_sin"][p, 1, pair][:, None]
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["R"], c["interleaved"]))
    k, v = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c["R"], c["interleaved"]), s["v"].float()
    k, v = (_codes(k, s["scales"][0]), _codes(v, s["scales"][1])) if c["type"] == "e4m3" else \
        (k.to(kp.dtype), v.to(vp.dtype))
    blk, off = slots // bs, slots % bs
    kp[blk, :, off // 8, :, off % 8] = k.reshape(T, Hkv, D // X, X)
    vp[blk, :, off // X, :, :, off % X] = v.reshape(T, Hkv, D // 8, 8)
    return s["q_out"], _as_values(kp), _as_values(vp)


def _cached(s, keys):
    """K (or V) of every sequence as float32 ``[B, Hkv, width * bs, D]``."""
    c, pool = s["case"], s["k_pool"] if keys else s["v_pool"]
    x = _as_values(pool)[s["tables"].clamp(min=0).long()].float()  # [B, n, Hkv, tile, tile, 8, X]
    B, n, Hkv = x.shape[:3]
    x = x.permute(0, 2, 1, 3, 5, 4, 6) if keys else x.permute(0, 2, 1, 3, 6, 4, 5)
    return x.reshape(B, Hkv, n * c["bs"], c["D"])


def _softmax(x):
    """Softmax over the last dim; rows without a finite entry are zero."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _add_weights(s, gained, new):
    """Adds ``gained`` ``[B, Hkv, n]`` to the sequences' token weights; the newest ``new`` are begun."""
    n, rows = gained.shape[-1], s["rows"].long()
    t = torch.arange(n, device="cuda")
    lens = s["lens"].long()[:, None, None]
    before = s["weights"][rows, :, :n]
    after = torch.where(t < lens - new, before * s["case"]["decay"], 0.0) + gained
    s["weights"][rows, :, :n] = torch.where(t < lens, after, before)


def _plain_decode(s):
    c = s["case"]
    B, Hkv, D, G = c["seqs"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    k = _cached(s, True)
    t = torch.arange(k.shape[2], device="cuda")
    hidden = t >= s["lens"].long()[:, None, None, None]            # [B, 1, 1, n]
    q = s["q"].float().reshape(B, Hkv, G, D)
    p = _softmax((q @ k.transpose(-1, -2) * (s["scale"] * s["scales"][0])).masked_fill(hidden, -math.inf))
    o = p @ _cached(s, False).masked_fill(hidden.transpose(-1, -2), 0.0) * s["scales"][1]
    s["out"].copy_(o.reshape(B, c["Hq"], D))
    _add_weights(s, p.sum(2), 1)
    return s["out"], s["weights"]


def _plain_prompt(s):
    c, w = s["case"], s["watched"]
    B, Hkv, D, G = c["seqs"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    end, size = s["start"][1:].long()[:, None], s["start"].diff().long()[:, None]
    back = torch.arange(w - 1, -1, -1, device="cuda")              # how far before the chunk's end
    counts = (back < size) & ((back < c["window"]) | (c["window"] == 0))
    q = s["q"][(end - 1 - back).clamp(min=0)].float()              # [B, w, Hq, D]
    q = q.reshape(B, w, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * w, D)
    k = _cached(s, True)
    x = (q @ k.transpose(-1, -2) * s["scale"]).reshape(B, Hkv, G, w, -1)
    t = torch.arange(k.shape[2], device="cuda")
    seen = (t <= (s["lens"].long()[:, None] - 1 - back)[..., None]) & counts[..., None]    # [B, w, n]
    p = _softmax(x.masked_fill_(~seen[:, None, None], -math.inf))
    _add_weights(s, p.sum((2, 3)), size[:, :, None])
    return s["weights"]


def _plain_select(s):
    c, lens = s["case"], s["lens"].long()[:, None, None]
    K, cap = c["K"], s["weights"].shape[-1]
    w = s["weights"][s["rows"].long()]
    t = torch.arange(cap, device="cuda")
    kind = ((t < c["first"]) | (t >= lens - c["last"])).int().masked_fill(t >= lens, -1).expand_as(w)
    by = w.sort(dim=-1, descending=True, stable=True).indices
    by = by.gather(-1, kind.gather(-1, by).sort(dim=-1, descending=True, stable=True).indices)[..., :K]
    taken = torch.where(torch.arange(by.shape[-1], device="cuda") < lens, by, cap).sort(-1).values
    s["kept"].fill_(-1)
    s["kept"][..., :by.shape[-1]] = torch.where(taken < cap, taken, -1)
    return s["kept"]


def _plain_keep(s):
    c, kept = s["case"], s["kept"].long()
    kp, vp, bs, X = s["k_pool"], s["v_pool"], c["bs"], s["k_pool"].shape[-1]
    b, h, i = (kept >= 0).nonzero(as_tuple=True)
    t = kept[b, h, i]
    src, dst = s["tables"][b, t // bs].long(), s["fresh"][b, i // bs].long()
    off, to = t % bs, i % bs
    kp[dst, h, to // 8, :, to % 8] = kp[src, h, off // 8, :, off % 8]
    vp[dst, h, to // X, :, :, to % X] = vp[src, h, off // X, :, :, off % X]
    row = s["rows"].long()[b]
    s["weights"][row, h, i] = s["weights"][row, h, t]
    return _as_values(kp), _as_values(vp), s["weights"]


# ----------------------------------------------------- the definition in 64 bits
def _element(pool, blk, h, t, keys):
    """Rows ``[n, D]`` in float64 of tokens ``t`` of blocks ``blk``, one kv head."""
    X = pool.shape[-1]
    x = pool[blk, h, t // 8, :, t % 8] if keys else pool[blk, h, t // X, :, :, t % X]
    return _as_values(x).double().flatten(1)


def exact(c, seed):
    s = prepare(c, seed)
    lens = _lens(c)
    if c["op"] == "norm":
        return _exact_norm(s, c)
    if c["op"] == "select":
        return None                                                # whole numbers
    W, rows = s["weights"].double(), s["rows"].tolist()
    bs, D, Hkv = c["bs"], c["D"], c["Hkv"]
    if c["op"] == "keep":
        kp, vp, old = _as_values(s["k_pool"]).double(), _as_values(s["v_pool"]).double(), W.clone()
        X = kp.shape[-1]
        for b in range(c["seqs"]):
            for h in range(Hkv):
                t = s["kept"][b, h].long()
                t = t[t >= 0]
                i = torch.arange(len(t), device="cuda")
                src, dst = s["tables"][b, t // bs].long(), s["fresh"][b, i // bs].long()
                kp[dst, h, i % bs // 8, :, i % 8] = _element(s["k_pool"], src, h, t % bs, True).reshape(-1, D // X, X)
                vp[dst, h, i % bs // X, :, :, i % X] = _element(s["v_pool"], src, h, t % bs, False).reshape(-1, D // 8, 8)
                W[rows[b], h, :len(t)] = old[rows[b], h, t]
        return kp, vp, W
    G = c["Hq"] // Hkv
    scale = float(torch.tensor(s["scales"][0], dtype=torch.float32)) * s["scale"]
    v_scale = float(torch.tensor(s["scales"][1], dtype=torch.float32))
    new = _chunks(c) if c["op"] == "prompt" else [1] * c["seqs"]
    watched = _watched(c) if c["op"] == "prompt" else None
    out = torch.zeros((c["seqs"], c["Hq"], D), dtype=torch.float64, device="cuda") if c["op"] == "decode" else None
    start = s["start"].tolist() if c["op"] == "prompt" else None
    for b, n in enumerate(lens):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        ids = s["tables"][b, t // bs].long()
        for h in range(Hkv):
            k = _element(s["k_pool"], ids, h, t % bs, True)
            if c["op"] == "decode":
                p = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ k.t() * scale, -1)
                out[b, h * G:(h + 1) * G] = p @ _element(s["v_pool"], ids, h, t % bs, False) * v_scale
                gained = p.sum(0)
            else:
                w = watched[b]
                q = s["q"][start[b + 1] - w:start[b + 1], h * G:(h + 1) * G].double()      # [w, G, D]
                last = n - w + torch.arange(w, device="cuda")
                gained = 0.0
                for g in range(G):
                    x = (q[:, g] @ k.t() * scale).masked_fill(t > last[:, None], -math.inf)
                    gained = gained + torch.softmax(x, -1).sum(0)
            before = W[rows[b], h, :n]
            W[rows[b], h, :n] = torch.where(t < n - new[b], before * c["decay"], 0.0) + gained
    return (out, W) if c["op"] == "decode" else W


def _exact_norm(s, c):
    T, R, bs, D, Hkv = s["slots"].shape[0], c["R"], c["bs"], c["D"], c["Hkv"]
    turn = torch.complex(s["cos_sin"][:, 0].double(), s["cos_sin"][:, 1].double())         # [P, R/2]
    parts, at = [], 0
    for axis, n in enumerate(s["sections"]):
        parts.append(turn[s["positions"].reshape(-1, T)[axis].long()][:, at:at + n])
        at += n
    turn = torch.cat(parts, 1)[:, None]

    def rotate(x, weight):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        pairs = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
        z = torch.complex(x[..., pairs[0]].contiguous(), x[..., pairs[1]].contiguous()) * turn
        x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
        return x

    def stored(x, scale):
        return (x / float(torch.tensor(scale, dtype=torch.float32))).clamp(-448, 448) if c["type"] == "e4m3" else x

    kp, vp = _as_values(s["k_pool"]).double(), _as_values(s["v_pool"]).double()
    X = kp.shape[-1]
    blk, off = s["slots"] // bs, s["slots"] % bs
    kp[blk, :, off // 8, :, off % 8] = stored(rotate(s["k"], s["k_weight"]), s["scales"][0]).reshape(T, Hkv, D // X, X)
    vp[blk, :, off // X, :, :, off % X] = stored(s["v"].double(), s["scales"][1]).reshape(T, Hkv, D // 8, 8)
    return rotate(s["q"], s["q_weight"]), kp, vp
