"""Oracle: the long-context operators -- position rotation, key bounds, block
choice and attention over chosen blocks -- as their definitions.

TEST INFRASTRUCTURE (see ``oracle/__init__``). The pages do not describe these
operators; the definitions are the header's. Arithmetic is float64, except the
rotation that decides stored bits: its products and sums are rounded to float32
one by one, because the operator fixes that precision.
"""
import numpy as np

from .attention import decode_one


def pair_dims(rotary_dim, interleaved):
    """The two dims of every pair: arrays (first, second) of length R / 2."""
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def turns(positions, cos_sin, sections):
    """Cosines and sines ``[T, R / 2]`` of every token's pairs (float32 values of
    the table): pair i takes the position of the axis its section names."""
    positions = np.asarray(positions)
    positions = positions.reshape(-1, positions.shape[-1])
    axis = np.repeat(np.arange(len(sections)), sections)
    p = positions[axis].T                                   # [T, R/2]
    i = np.arange(cos_sin.shape[2])
    return cos_sin[p, 0, i], cos_sin[p, 1, i]


def rotate_f32(x, cos, sin, interleaved):
    """float32 heads ``[T, H, D]`` rotated, each operation rounded to float32."""
    x = np.asarray(x, dtype=np.float32)
    a, b = pair_dims(2 * cos.shape[1], interleaved)
    c, s = (np.asarray(t, dtype=np.float32)[:, None] for t in (cos, sin))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotate_f64(x, cos, sin, interleaved):
    """The same in float64: each pair as a complex number times e^(i angle)."""
    x = np.asarray(x, dtype=np.float64)
    a, b = pair_dims(2 * cos.shape[1], interleaved)
    z = (x[..., a] + 1j * x[..., b]) * (cos.astype(np.float64) + 1j * sin.astype(np.float64))[:, None]
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def key_bounds(k, filled):
    """``[2, D]``: smallest and largest value of each dim over the first ``filled``
    tokens of one (block, kv head) ``[bs, D]``; NaN where a key is."""
    return np.stack([k[:filled].min(0), k[:filled].max(0)])


def block_scores(q, bounds):
    """``[n]`` scores of n blocks ``[n, 2, D]`` under the query heads ``[G, D]`` of
    one kv head; inf where no finite number describes the block."""
    q, b = np.asarray(q, dtype=np.float64), np.asarray(bounds, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        t = np.maximum(q, 0)[:, None] * b[None, :, 1] + np.minimum(q, 0)[:, None] * b[None, :, 0]
        s = t.sum(-1).max(0)
    return np.where(np.isfinite(s), s, np.inf)


def select(scores, k, first, last):
    """The chosen blocks of one row, ascending: all of them if there are at most k,
    else the first, the last, and the best of the others (ties: lower index)."""
    n = len(scores)
    if n <= k:
        return np.arange(n)
    middle = np.arange(first, n - last)
    best = middle[np.argsort(-scores[middle], kind="stable")][:k - first - last]
    return np.sort(np.concatenate([np.arange(first), best, np.arange(n - last, n)]))


def select_blocks(q, bounds, block_tables, seq_lens, block_size, num_kv_heads, k, first, last):
    """``[B, Hkv, k]`` logical blocks, -1 padded. q ``[B, Hq, D]``, bounds ``[NB,
    Hkv, 2, D]`` (numpy)."""
    B, Hq, _ = q.shape
    G = Hq // num_kv_heads
    out = np.full((B, num_kv_heads, k), -1, dtype=np.int32)
    for b in range(B):
        n = -(-int(seq_lens[b]) // block_size)
        ids = np.asarray(block_tables[b][:n], dtype=np.int64)
        for h in range(num_kv_heads):
            chosen = select(block_scores(q[b, h * G:(h + 1) * G], bounds[ids, h]), k, first, last)
            out[b, h, :len(chosen)] = chosen
    return out


def sparse_decode(q, k, v, block_tables, seq_lens, selected, scale, block_size, k_scale=1.0,
                  v_scale=1.0, with_bound=False):
    """``[B, Hq, D]`` attention over the listed blocks' tokens. q ``[B, Hq, D]``; k,
    v float64 ``[NB, Hkv, bs, D]``. ``with_bound``: also, per element, sum_t p_t
    |V_t| (times v_scale) and per row the largest sum_d |q_d K_td| times scale and
    k_scale: what rounding errors of the weights and of the logits scale with."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    q = np.asarray(q, dtype=np.float64)
    out, mag, logit = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        L = int(seq_lens[b])
        for h in range(Hkv):
            t = np.concatenate([np.arange(j * block_size, min(L, (j + 1) * block_size))
                                for j in selected[b][h] if j >= 0] or [np.zeros(0, int)]).astype(np.int64)
            ids = np.asarray(block_tables[b], dtype=np.int64)[t // block_size]
            K, V = k[ids, h, t % block_size], v[ids, h, t % block_size]
            for g in range(h * G, (h + 1) * G):
                out[b, g] = decode_one(q[b, g], K, V, scale, k_scale, v_scale)
                if len(t):
                    mag[b, g] = decode_one(q[b, g], K, np.abs(V), scale, k_scale, v_scale)
                    logit[b, g] = (np.abs(K) @ np.abs(q[b, g])).max() * scale * k_scale
    return (out, mag, logit) if with_bound else out
