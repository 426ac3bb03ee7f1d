"""Oracle: the cache eviction operators -- heads normalised and rotated, the attention
weight that cached tokens draw, the choice of the tokens to keep -- as their definitions.

TEST INFRASTRUCTURE (see ``oracle/__init__``). The pages do not describe these operators;
the definitions are the header's. Arithmetic is float64.
"""
import numpy as np


def normed(x, weight, eps):
    """Heads ``[..., D]`` over their root mean square, times ``weight`` (``[D]`` or ``[H, D]``)."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def softmax(x):
    """Softmax over the last axis; rows that are all -inf are zero, a NaN or +inf entry
    makes its row NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        top = x.max(-1, keepdims=True)
        e = np.exp(x - np.where(top == -np.inf, 0.0, top))
        total = e.sum(-1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def decode_weights(q, k, scale, missing=()):
    """``[G, L]`` softmax weights of the tokens ``k [L, D]`` under the query heads ``q [G,
    D]``; tokens in ``missing`` have none."""
    x = np.asarray(q, dtype=np.float64) @ np.asarray(k, dtype=np.float64).T * scale
    x[:, list(missing)] = -np.inf
    return softmax(x)


def prompt_weights(q, k, scale, missing=()):
    """``[w, G, L]`` causal softmax weights of ``k [L, D]`` under the last w queries ``q [w, G,
    D]``: query i sees the tokens up to L - w + i."""
    w, L = len(q), len(k)
    x = np.einsum("wgd,td->wgt", np.asarray(q, dtype=np.float64), np.asarray(k, dtype=np.float64)) * scale
    t = np.arange(L)
    x = np.where((t[None] > (L - w + np.arange(w))[:, None])[:, None], -np.inf, x)
    x[..., list(missing)] = -np.inf
    return softmax(x)


def updated(before, gained, new, decay):
    """A row's weights of L tokens after a call that ``gained`` and that begins the last ``new``."""
    L = len(gained)
    old = np.where(np.arange(L) < L - new, np.asarray(before, dtype=np.float64)[:L] * decay, 0.0)
    return old + gained


def select(weights, n, num_kept, first, last):
    """The kept tokens (ascending, -1 padded) of a row with n tokens."""
    if n <= num_kept:
        return list(range(n)) + [-1] * (num_kept - n)
    w = [float(x) if np.isfinite(x) else np.inf for x in weights[:n]]
    inner = sorted(range(first, n - last), key=lambda t: (-w[t], t))
    return sorted(list(range(first)) + inner[:num_kept - first - last] + list(range(n - last, n)))
