"""Cases of the long-context decode operators: the rotated append, the key bounds
of the cache's blocks, the choice of blocks for a query, and the attention over
the chosen blocks.

``run`` computes one pass either in plain torch (``own`` false) or with the
framework's calls (``own`` true), on the same state. The pools have the
library's layout: K ``[NB, Hkv, bs/8, D/X, 8, X]`` and V ``[NB, Hkv, bs/X, D/8,
8, X]`` with X elements in 16 bytes.
"""
import math

import torch

own = False

TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
         "e4m3": (torch.bfloat16, torch.uint8)}      # (activations, cache)
ELT = {"f32": 4, "bf16": 2, "e4m3": 1}
K_SCALE, V_SCALE = 0.037, 0.041                     # E4M3 caches: value = code * scale
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a 64-sequence batch: q, k, v are views of the fused projection
        {"name": "rotary decode 64", "op": "rotary", "type": "bf16", "seqs": 64, "tokens": 1, "len": 32768,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "R": 128, "axes": 1, "interleaved": False, "fused": True},
        # a prompt with image tokens: (time, height, width) positions, 16 sequences' chunks of 512
        {"name": "rotary chunk 8192 3 axes", "op": "rotary", "type": "bf16", "seqs": 16, "tokens": 512, "len": 4096,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "R": 128, "axes": 3, "interleaved": False, "fused": True},
        # a quantised cache, half of each head rotated, pairs side by side, ragged chunk ends
        {"name": "rotary e4m3 partial", "op": "rotary", "type": "e4m3", "seqs": 3, "tokens": 357, "len": 2011,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 32, "R": 64, "axes": 1, "interleaved": True, "fused": False},
        # one decode step: only the sequences' last blocks changed
        {"name": "bounds decode 64", "op": "bounds", "type": "bf16", "seqs": 64, "new": 1, "len": 2048,
         "Hq": 40, "Hkv": 40, "D": 128, "bs": 16},
        # after a prompt's chunks: every block of the last 2048 tokens
        {"name": "bounds chunk 16384 e4m3", "op": "bounds", "type": "e4m3", "seqs": 8, "new": 2048, "len": 32768,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # one long conversation
        {"name": "select 1 x 131072", "op": "select", "type": "bf16", "seqs": 1, "len": 131072, "K": 128, "first": 1,
         "last": 2, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # a batch of long documents, ragged
        {"name": "select 32 x 32768", "op": "select", "type": "bf16", "seqs": 32, "len": 32768, "K": 64, "first": 1,
         "last": 2, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # short sequences: latency, small heads, many query heads a kv head
        {"name": "select 4 x 2000", "op": "select", "type": "e4m3", "seqs": 4, "len": 2000, "K": 16, "first": 1,
         "last": 1, "Hq": 32, "Hkv": 4, "D": 64, "bs": 32},
        # one long conversation: few rows
        {"name": "sparse 1 x 128 blocks", "op": "sparse", "type": "bf16", "seqs": 1, "len": 131072, "K": 128,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # a batch with a quantised cache
        {"name": "sparse 64 x 128 blocks e4m3", "op": "sparse", "type": "e4m3", "seqs": 64, "len": 32768, "K": 128,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16},
        # multi-head attention, ragged, some sequences shorter than their selection
        {"name": "sparse 32 x 64 blocks mha", "op": "sparse", "type": "bf16", "seqs": 32, "len": 8192, "K": 64,
         "Hq": 40, "Hkv": 40, "D": 128, "bs": 16},
        # float32, small heads, an empty sequence
        {"name": "sparse f32 3 x 5 blocks", "op": "sparse", "type": "f32", "seqs": 3, "len": 500, "K": 5,
         "Hq": 8, "Hkv": 8, "D": 64, "bs": 32},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "bounds", "select", "sparse"])
    kind = rng.choice(["bf16", "bf16", "e4m3", "f32"])
    D, bs = rng.choice([64, 128]), rng.choice([16, 32])
    G, Hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    c = {"op": op, "type": kind, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "bs": bs}
    if op == "rotary":
        tokens = rng.choice([1, _log(rng, 2, 900)])
        seqs = _log(rng, 1, max(1, min(200, 8192 // tokens)))
        R = rng.choice([D, D, D // 2, D // 4])
        c.update(seqs=seqs, tokens=tokens, len=tokens + _log(rng, 1, 16384), R=R,
                 axes=rng.choice([1, 1, 2, 3]) if R >= 32 else 1, interleaved=rng.random() < 0.4,
                 fused=rng.random() < 0.6)
    elif op == "bounds":
        new = rng.choice([1, _log(rng, 2, 2048)])
        c.update(seqs=_log(rng, 1, max(1, min(64, 16384 // new))), new=new, len=new + _log(rng, 1, 16384))
    else:
        c.update(seqs=_log(rng, 1, 32))
        c.update(len=_log(rng, 1 if op == "sparse" else 16 * bs, min(131072, (1 << 20) // c["seqs"])))
        K = _log(rng, 3, 200)
        c.update(K=K)
        if op == "select":
            c.update(first=rng.randint(0, 1), last=rng.randint(0, min(4, K - 1)))
    return c


def _lens(c):
    """The sequences' lengths, from the case alone: the longest first, then spread
    over (0, len]; the last one empty where the attention has three or more."""
    low = c.get("new", c.get("tokens", 1))
    lens = [max(low, int(c["len"] * ((0.6180339887498949 * i) % 1.0 or 1.0))) for i in range(c["seqs"])]
    if c["op"] == "sparse" and c["seqs"] >= 3:
        lens[-1] = 0
    return lens


def work(c):
    Hq, Hkv, D, bs, lens = c["Hq"], c["Hkv"], c["D"], c["bs"], _lens(c)
    act, elt = 2 if c["type"] != "f32" else 4, ELT[c["type"]]
    bound = 4 if c["type"] == "f32" else 2
    G = Hq // Hkv
    blocks = [-(-n // bs) for n in lens]
    if c["op"] == "rotary":
        T = c["seqs"] * c["tokens"]
        rows = len({n - 1 - t for n in lens for t in range(c["tokens"])}) if c["axes"] == 1 else c["len"] // 256 + 33
        return {"bytes": T * D * ((2 * Hq + 2 * Hkv) * act + 2 * Hkv * elt) + T * (8 + 4 * c["axes"]) + rows * c["R"] * 4,
                "flops": 3 * T * (Hq + Hkv) * c["R"]}
    if c["op"] == "bounds":
        tokens = sum(n - (n - c["new"]) // bs * bs for n in lens)
        changed = sum(-(-n // bs) - (n - c["new"]) // bs for n in lens)
        return {"bytes": Hkv * D * (tokens * elt + changed * 2 * bound) + 4 * changed + 8 * c["seqs"],
                "flops": 2 * tokens * Hkv * D}
    if c["op"] == "select":
        scored = sum(max(0, n - c["first"] - c["last"]) for n in blocks if n > c["K"])
        return {"bytes": scored * (Hkv * D * 2 * bound + 4) + c["seqs"] * (Hq * D * act + 4 + Hkv * c["K"] * 4),
                "flops": 2 * scored * Hq * D}
    # the last block is among the selected ones
    tokens = sum(min(n, c["K"]) * bs - ((n * bs - L) if n else 0) for n, L in zip(blocks, lens))
    taken = sum(min(n, c["K"]) for n in blocks)
    return {"bytes": tokens * Hkv * D * 2 * elt + taken * Hkv * 8 + c["seqs"] * (2 * Hq * D * act + 4),
            "flops": 4 * tokens * Hkv * G * D}


# ------------------------------------------------------------- what a program has
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(shape, c, g, spread=False):
    """Activations: N(0, 1); keys (``spread``) with a few strong channels, as trained ones have."""
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:
        gain = torch.ones(shape[-1], device="cuda")
        gain[:: shape[-1] // 4] = 4.0
        x *= gain
    return x.to(TYPES[c["type"]][0])


def _pool(shape, c, g):
    """A filled pool of the library's layout: N(0, 1) values, for E4M3 the codes' bytes."""
    cache = TYPES[c["type"]][1]
    if c["type"] != "e4m3":
        return torch.randn(shape, generator=g, device="cuda", dtype=cache)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(1.0 / K_SCALE).to(F8).view(torch.uint8)


def _pools(c, NB, g, keys_only=False):
    X, D, bs = 16 // ELT[c["type"]], c["D"], c["bs"]
    k = _pool((NB, c["Hkv"], bs // 8, D // X, 8, X), c, g)
    v = None if keys_only else _pool((NB, c["Hkv"], bs // X, D // 8, 8, X), c, g)
    return k, v


def _tables(c, lens, g):
    """Block tables of sequences whose blocks lie anywhere in the pool, and the pool's size."""
    blocks = [-(-n // c["bs"]) for n in lens]
    width, total = max(1, max(blocks)), sum(blocks)
    NB = total + total // 16 + 2
    ids = torch.randperm(NB, generator=g, device="cuda")[:total].to(torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        tables[b, :n] = ids[at:at + n]
        at += n
    return tables, NB


def _scales(c):
    return (K_SCALE, V_SCALE) if c["type"] == "e4m3" else (1.0, 1.0)


def prepare(c, seed):
    g, lens = _gen(seed), _lens(c)
    act, cache = TYPES[c["type"]]
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["bs"]
    s = {"case": c, "scales": _scales(c)}
    tables, NB = _tables(c, lens, g)
    s.update(tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if c["op"] == "rotary":
        n, T = c["tokens"], c["seqs"] * c["tokens"]
        at = (s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")).reshape(-1)
        seq = torch.arange(c["seqs"], device="cuda").repeat_interleave(n)
        s["slots"] = tables[seq, at // bs].long() * bs + at % bs
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
        if c["fused"]:
            qkv = _rows((T, Hq + 2 * Hkv, D), c, g)
            s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        else:
            s["q"], s["k"], s["v"] = (_rows((T, h, D), c, g) for h in (Hq, Hkv, Hkv))
        s["k_pool"], s["v_pool"] = _pools(c, NB, g)
        s["q_out"] = torch.empty((T, Hq, D), dtype=act, device="cuda")
    elif c["op"] == "bounds":
        s["k_pool"], _ = _pools(c, NB, g, keys_only=True)
        s["first"] = s["lens"] - c["new"]
        s["bounds"] = torch.randn((NB, Hkv, 2, D), generator=g, device="cuda").to(act)
    elif c["op"] == "select":
        s["q"] = _rows((c["seqs"], Hq, D), c, g)
        # bounds as blocks of bs keys have them: about +-1.8 for 16 normal keys, some channels stronger
        a, b = _rows((NB, Hkv, D), c, g, True), _rows((NB, Hkv, D), c, g, True)
        mid, wide = 0.25 * a.float(), 1.3 + 0.3 * b.float().abs()
        s["bounds"] = torch.stack([mid - wide, mid + wide], 2).to(act)
        if c["type"] == "e4m3":   # what codes can be
            s["bounds"] = (s["bounds"].float() / K_SCALE).clamp(-448, 448).to(F8).to(act)
        s["selected"] = torch.empty((c["seqs"], Hkv, c["K"]), dtype=torch.int32, device="cuda")
    else:
        s["q"] = _rows((c["seqs"], Hq, D), c, g) * 2.0
        s["k_pool"], s["v_pool"] = _pools(c, NB, g)
        # the last block and a random choice of the others, ascending
        width, n = tables.shape[1], (s["lens"] + bs - 1) // bs
        rank = torch.rand((c["seqs"], Hkv, width), generator=g, device="cuda")
        j = torch.arange(width, device="cuda")
        rank = torch.where(j == n[:, None, None] - 1, 2.0, rank).masked_fill(j >= n[:, None, None], -1.0)
        top = rank.topk(min(c["K"], width), -1)
        chosen = torch.where(top.values >= 0, top.indices, width).sort(-1).values
        s["selected"] = torch.full((c["seqs"], Hkv, c["K"]), -1, dtype=torch.int32, device="cuda")
        s["selected"][..., :chosen.shape[-1]] = torch.where(chosen < width, chosen, -1)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# ------------------------------------------------------------------- one pass
def _bound_call(s, bind):
    """A serving loop checks and binds its buffers once and launches on them many times."""
    if "call" not in s:
        s["call"] = bind()
    s["call"]()


def run(s):
    op = s["case"]["op"]
    if op == "rotary":
        return _own_rotary(s) if own else _plain_rotary(s)
    if op == "bounds":
        return _own_bounds(s) if own else _plain_bounds(s)
    if op == "select":
        return _own_select(s) if own else _plain_select(s)
    return _own_sparse(s) if own else _plain_sparse(s)


def _as_values(pool):
    return pool.view(F8) if pool.dtype == torch.uint8 else pool


def _own_rotary(s):
    import paged_kv_cache_259_gb300 as pkv
    _bound_call(s, lambda: pkv.bind_rotary_and_cache(
        s["q_out"], s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"], s["positions"], s["cos_sin"],
        sections=s["sections"], interleaved=s["case"]["interleaved"], k_scale=s["scales"][0], v_scale=s["scales"][1]))
    return s["q_out"], _as_values(s["k_pool"]), _as_values(s["v_pool"])


def _own_bounds(s):
    import paged_kv_cache_259_gb300 as pkv
    _bound_call(s, lambda: pkv.bind_update_key_bounds(s["k_pool"], s["bounds"], s["tables"], s["lens"], s["first"],
                                                      max_new_tokens=s["case"]["new"]))
    return s["bounds"]


def _own_select(s):
    import paged_kv_cache_259_gb300 as pkv
    c = s["case"]

    def bind():   # the scratch is the program's, like that of the split decode
        n = pkv.select_blocks_workspace_size(c["seqs"], c["Hkv"], s["tables"].shape[1])
        s["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
        return pkv.bind_select_blocks(s["selected"], s["q"], s["bounds"], s["tables"], s["lens"], c["bs"],
                                      first_blocks=c["first"], last_blocks=c["last"], workspace=s["workspace"])

    _bound_call(s, bind)
    return s["selected"]


def _own_sparse(s):
    import paged_kv_cache_259_gb300 as pkv
    _bound_call(s, lambda: pkv.bind_paged_attention_decode_sparse(
        s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["selected"], s["scale"],
        k_scale=s["scales"][0], v_scale=s["scales"][1]))
    return s["out"]


# ---------------------------------------------------------------- plain forms
def _codes(x, scale):
    """E4M3 bytes of x / scale, saturating."""
    return (x / torch.full((), scale, device=x.device)).clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def _rotated(x, c, s, R, interleaved):
    """float32 heads ``[T, H, D]`` with the first R dims rotated, cos and sin ``[T, 1, R/2]``."""
    r, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _plain_rotary(s):
    c, slots = s["case"], s["slots"]
    kp, vp, D, bs, Hkv = s["k_pool"], s["v_pool"], c["D"], c["bs"], c["Hkv"]
    X, T = kp.shape[-1], slots.shape[0]
    positions = s["positions"].long().reshape(-1, T)
    axis = torch.repeat_interleave(torch.arange(positions.shape[0], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"))
    pair = torch.arange(c["R"] // 2, device="cuda")
    p = positions[axis].t()                                        # [T, R/2]
    cos, sin = s["cos_sin"][p, 0, pair][:, None], s["cos_sin"][p, 1, pair][:, None]
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, c["R"], c["interleaved"]))
    k, v = _rotated(s["k"].float(), cos, sin, c["R"], c["interleaved"]), s["v"].float()
    k, v = (_codes(k, s["scales"][0]), _codes(v, s["scales"][1])) if c["type"] == "e4m3" else \
        (k.to(kp.dtype), v.to(vp.dtype))
    blk, off = slots // bs, slots % bs
    kp[blk, :, off // 8, :, off % 8] = k.reshape(T, Hkv, D // X, X)
    vp[blk, :, off // X, :, :, off % X] = v.reshape(T, Hkv, D // 8, 8)
    return s["q_out"], _as_values(kp), _as_values(vp)


def _tokens(pool, bs, D, keys):
    """Blocks of a pool ``[..., 2 tile axes, 8, X]`` as float32 ``[..., bs, D]``."""
    x = _as_values(pool).float()
    n = x.dim()
    lead = list(range(n - 4))
    order = [n - 4, n - 2, n - 3, n - 1] if keys else [n - 4, n - 1, n - 3, n - 2]
    return x.permute(lead + order).reshape(*x.shape[:n - 4], bs, D)


def _plain_bounds(s):
    c, bs, D = s["case"], s["case"]["bs"], s["case"]["D"]
    lens, width = s["lens"].long(), s["tables"].shape[1]
    j = torch.arange(width, device="cuda")
    changed = (j >= s["first"].long()[:, None] // bs) & (j < (lens[:, None] + bs - 1) // bs)
    seq, blk = changed.nonzero(as_tuple=True)
    ids = s["tables"][seq, blk].long()
    k = _tokens(s["k_pool"][ids], bs, D, True)                     # [n, Hkv, bs, D]
    filled = (blk[:, None] * bs + torch.arange(bs, device="cuda") < lens[seq][:, None])[:, None, :, None]
    lo = k.masked_fill(~filled, math.inf).amin(2)
    hi = k.masked_fill(~filled, -math.inf).amax(2)
    s["bounds"][ids] = torch.stack([lo, hi], 2).to(s["bounds"].dtype)
    return s["bounds"]


def _plain_select(s):
    c, lens = s["case"], s["lens"].long()
    B, Hkv, K = s["selected"].shape
    width = s["tables"].shape[1]
    n = ((lens + c["bs"] - 1) // c["bs"])[:, None, None]
    b = s["bounds"][s["tables"].clamp(min=0).long()].double()      # [B, n, Hkv, 2, D]
    lo, hi = b[..., 0, :].permute(0, 2, 3, 1), b[..., 1, :].permute(0, 2, 3, 1)
    q = s["q"].double().reshape(B, Hkv, c["Hq"] // Hkv, c["D"])
    score = (q.clamp(min=0) @ hi + q.clamp(max=0) @ lo).amax(2)    # [B, Hkv, n]
    score = torch.where(score.isfinite(), score, math.inf)
    j = torch.arange(width, device="cuda")
    kind = ((j < c["first"]) | (j >= n - c["last"])).int().expand(B, Hkv, width).masked_fill(j >= n, -1)
    by = score.sort(dim=-1, descending=True, stable=True).indices
    by = by.gather(-1, kind.gather(-1, by).sort(dim=-1, descending=True, stable=True).indices)[..., :K]
    taken = torch.where(torch.arange(by.shape[-1], device="cuda") < n, by, width).sort(-1).values
    s["selected"].fill_(-1)
    s["selected"][..., :by.shape[-1]] = torch.where(taken < width, taken, -1)
    return s["selected"]


def _plain_sparse(s):
    c, sel = s["case"], s["selected"].long()
    B, Hkv, K = sel.shape
    bs, D, G = c["bs"], c["D"], c["Hq"] // Hkv
    ids = s["tables"].long()[:, None].expand(-1, Hkv, -1).gather(-1, sel.clamp(min=0)).clamp(min=0)
    head = torch.arange(Hkv, device="cuda")[:, None]
    k = _tokens(s["k_pool"][ids, head], bs, D, True).reshape(B, Hkv, K * bs, D) * s["scales"][0]
    v = _tokens(s["v_pool"][ids, head], bs, D, False).reshape(B, Hkv, K * bs, D)
    at = sel[..., None] * bs + torch.arange(bs, device="cuda")
    seen = ((sel[..., None] >= 0) & (at < s["lens"].long()[:, None, None, None])).reshape(B, Hkv, 1, K * bs)
    q = s["q"].float().reshape(B, Hkv, G, D)
    x = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen.transpose(-1, -2), 0.0)
    o = torch.where(total > 0, (p @ v) / total.clamp(min=1e-38), 0.0) * s["scales"][1]
    s["out"].copy_(o.reshape(B, c["Hq"], D))
    return s["out"]


# ----------------------------------------------------- the definition in 64 bits
def _element(pool, blk, h, t, keys):
    """Rows ``[n, D]`` in float64 of tokens ``t`` of blocks ``blk``, one kv head."""
    X = pool.shape[-1]
    x = pool[blk, h, t // 8, :, t % 8] if keys else pool[blk, h, t // X, :, :, t % X]
    return _as_values(x).double().flatten(1)


def exact(c, seed):
    s = prepare(c, seed)
    bs, D, Hkv, lens = c["bs"], c["D"], c["Hkv"], _lens(c)
    if c["op"] == "rotary":
        T = s["slots"].shape[0]
        turn = torch.complex(s["cos_sin"][:, 0].double(), s["cos_sin"][:, 1].double())   # [P, R/2]
        parts, at = [], 0
        for axis, n in enumerate(s["sections"]):
            parts.append(turn[s["positions"].reshape(-1, T)[axis].long()][:, at:at + n])
            at += n
        turn = torch.cat(parts, 1)[:, None]

        def rotate(x):
            x = x.double().clone()
            pairs = (slice(0, c["R"], 2), slice(1, c["R"], 2)) if c["interleaved"] else \
                (slice(0, c["R"] // 2), slice(c["R"] // 2, c["R"]))
            z = torch.complex(x[..., pairs[0]].contiguous(), x[..., pairs[1]].contiguous()) * turn
            x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
            return x

        def stored(x, scale):
            return (x / float(torch.tensor(scale, dtype=torch.float32))).clamp(-448, 448) if c["type"] == "e4m3" else x

        kp, vp = _as_values(s["k_pool"]).double(), _as_values(s["v_pool"]).double()
        X = kp.shape[-1]
        blk, off = s["slots"] // bs, s["slots"] % bs
        kp[blk, :, off // 8, :, off % 8] = stored(rotate(s["k"]), s["scales"][0]).reshape(T, Hkv, D // X, X)
        vp[blk, :, off // X, :, :, off % X] = stored(s["v"].double(), s["scales"][1]).reshape(T, Hkv, D // 8, 8)
        return rotate(s["q"]), kp, vp
    if c["op"] == "bounds":
        out = s["bounds"].double()
        for b, n in enumerate(lens):
            first = (n - c["new"]) // bs
            at = torch.arange(first * bs, n, device="cuda")
            ids = s["tables"][b, at // bs].long()
            for h in range(Hkv):
                k = _element(s["k_pool"], ids, h, at % bs, True)
                to = s["tables"][b, first:-(-n // bs)].long()
                where = (at // bs - first)[:, None].expand(-1, D)
                for i, how in ((0, "amin"), (1, "amax")):
                    out[to, h, i] = torch.zeros((len(to), D), dtype=torch.float64, device="cuda").scatter_reduce(
                        0, where, k, how, include_self=False)
        return out
    if c["op"] == "select":
        return None                                                # whole numbers
    out = torch.zeros((c["seqs"], c["Hq"], D), dtype=torch.float64, device="cuda")
    G = c["Hq"] // Hkv
    ks, vs = (float(torch.tensor(x, dtype=torch.float32)) for x in s["scales"])
    for b, n in enumerate(lens):
        for h in range(Hkv):
            j = s["selected"][b, h].long()
            j = j[j >= 0]
            at = (j[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
            at = at[at < n]
            if not len(at):
                continue
            ids = s["tables"][b, at // bs].long()
            k = _element(s["k_pool"], ids, h, at % bs, True)
            v = _element(s["v_pool"], ids, h, at % bs, False)
            p = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ k.t() * (ks * s["scale"]), -1)
            out[b, h * G:(h + 1) * G] = p @ v * vs
    return out
