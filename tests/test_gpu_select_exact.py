"""select_blocks where float64 sums, or 64-bit keys, cannot tell scores apart: the choice
is that of the scores as rational numbers."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from _lib import library, pkv
from test_gpu_long_context import BF, F32, I32, key_like_bounds, normal, rng_of, select_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


def exact_scores(q, bounds):
    """Scores of blocks ``[n, 2, D]`` under heads ``[G, D]`` as Fractions; None where the
    definition's value is not finite."""
    q, bounds = q.double().numpy(), bounds.double().numpy()
    whole, fine = np.isfinite(q).all(), np.isfinite(bounds).all((1, 2))
    heads = [[(int(x > 0), Fraction(x) if math.isfinite(x) else x) for x in row] for row in q.tolist()]
    out = []
    for block, ok in zip(bounds, fine):
        if not ok:                                         # every bound meets a number or 0
            out.append(None)
            continue
        best, top = None, False
        dims = np.flatnonzero(block.any(0)).tolist() if whole else range(block.shape[1])
        sides = block[:, dims].T.tolist()
        for head in heads:
            s, inf = Fraction(0), 0.0
            for d, two in zip(dims, sides):
                side, x = head[d]
                if not isinstance(x, Fraction):
                    inf += x * two[side]                   # 0 x inf is NaN
                elif x and two[side]:
                    s += x * Fraction(two[side])
            if inf != inf or inf == math.inf:
                top = True
            elif inf == 0.0:
                best = s if best is None else max(best, s)
        out.append(None if top or (best is None and not whole) else best)
    return out


def choice(scores, K, first, last):
    n = len(scores)
    mid = range(first, n - last)
    order = sorted(mid, key=lambda j: (scores[j] is not None, -scores[j] if scores[j] is not None else 0, j))
    return sorted(list(range(first)) + order[:K - first - last] + list(range(n - last, n)))


def check(q, bounds, K, first=0, last=0):
    """One kv head, a row of all blocks in the pool's order."""
    n = bounds.shape[0]
    got = select_gpu(q, bounds[:, None].contiguous(), np.arange(n, dtype=np.int32)[None], [n * 16], 16, 1, K, first, last)
    want = choice(exact_scores(q[0], bounds), K, first, last)
    assert got[0, 0].tolist() == want
    assert pkv.get_device_error() == 0


# fused with the scoring (bf16), ranked from a list, by bisection; one row of each selection
SIZES = [(100, 13), (200, 25), (2500, 25), (5000, 700), (9000, 40)]


def steps(n, dt, unit, rng, D=64):
    """Bounds whose scores under q = 1 are 2^12 + j unit, j a random order of 0 .. n-1."""
    j = rng.permutation(n)
    b = torch.zeros(n, 2, D)
    b[:, 1, 0] = 2.0 ** 12
    b[:, 1, 33] = torch.from_numpy((j % 256).astype(np.float32)) * unit
    b[:, 1, 34] = torch.from_numpy((j // 256 * 256).astype(np.float32)) * unit
    return b.to(dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,K", SIZES)
@pytest.mark.parametrize("bits", [26, 36, 48, 60, 100])
def test_scores_that_differ_below_the_keys(dt, n, K, bits):
    """Steps of 2^-bits beside 2^12, and the same times 2^40 and 2^-20."""
    rng = rng_of(11, n, bits)
    b, q = steps(n, dt, 2.0 ** -bits, rng), torch.ones(1, 2, 64, dtype=dt)
    check(q, b, K, 1, 1)
    check(q * 2.0 ** 40, b * 2.0 ** -20, K)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,K", SIZES[1:3])
def test_the_largest_head_decides(dt, n, K):
    """Four heads, each the largest on some blocks by a last step, one of them negative
    (it meets the lower bounds)."""
    rng = rng_of(12, n)
    b = steps(n, dt, 2.0 ** -50, rng)
    b[:, 0] = -b[:, 1]
    q = torch.ones(1, 4, 64, dtype=dt)
    q[0, 1] = -1.0
    q[0, 2, 33] = 2.0
    q[0, 3, 34], q[0, 3, 33] = 0.5, 3.0
    b[:, 1, 33:35] = b[torch.from_numpy(rng.permutation(n)), 1, 33:35]
    check(q, b, K)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,K", SIZES)
def test_equal_scores_below_the_keys_go_by_index(dt, n, K):
    """Seven values, 2^-60 apart, many blocks each."""
    rng = rng_of(13, n)
    b = torch.zeros(n, 2, 64)
    b[:, 1, 0] = 1.0
    b[:, 1, 40] = torch.from_numpy(rng.integers(0, 7, n).astype(np.float32)) * 2.0 ** -60
    check(torch.ones(1, 1, 64, dtype=dt), b.to(dt), K)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,K", SIZES[:3])
def test_sums_that_cancel_to_their_last_bits(dt, D, n, K):
    """Terms of every size that cancel pairwise, but for one of 2^-70 of them."""
    rng = rng_of(14, n, D)
    x = (rng.standard_normal((n, D)) * 2.0 ** rng.integers(-30, 30, (n, D))).astype(np.float32)
    x[:, 1::2] = -x[:, 0::2]
    b = torch.from_numpy(x).to(dt).float()
    b[:, D - 2] = torch.from_numpy(rng.integers(-100, 100, n).astype(np.float32)) * 2.0 ** -70
    b[:, D - 1] = 0
    q = torch.ones(1, 1, D, dtype=dt)
    check(q, torch.stack([b, b], 1).to(dt), K, 1, 2)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,K", SIZES[1:3])
def test_subnormal_and_largest_values(dt, n, K):
    """Bounds and queries at both ends of the type: products from 2^-266 (bf16) or 2^-298 to
    2^255 within one score."""
    rng = rng_of(15, n)
    tiny, big = (2.0 ** -133, 2.0 ** 127) if dt == BF else (2.0 ** -149, 2.0 ** 127)
    b = torch.zeros(n, 2, 64, dtype=torch.float64)
    b[:, :, 3] = torch.from_numpy(rng.integers(1, 100, n).astype(np.float64))[:, None] * tiny
    b[:, 1, 9] = big
    q = torch.zeros(1, 2, 64, dtype=torch.float64)
    q[0, :, 3], q[0, 0, 9], q[0, 1, 9] = tiny, big, 1.0
    check(q.to(dt), b.to(dt), K)
    q[0, :, 9] = 0                                         # the tiny products alone
    check(q.to(dt), b.to(dt), K)
    q[0, :, 3] = 1.0                                       # subnormal scores
    check(q.to(dt), b.to(dt), K)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,K", SIZES[:3])
@pytest.mark.parametrize("what", ["inf block", "nan block", "inf head", "-inf head", "sum past float32"])
def test_rows_with_values_that_are_not_finite_are_as_exact(dt, n, K, what):
    rng = rng_of(16, n)
    b, q = steps(n, dt, 2.0 ** -60, rng), torch.ones(1, 2, 64, dtype=dt)
    b[:, 0] = b[:, 1] - 8192.0
    b[:, 1, 50] = 1.0
    b[:, 0, 50] = -1.0
    if what == "inf block":
        b[n // 2, 0, 7], b[n // 3, 1, 9] = -math.inf, math.inf
    elif what == "nan block":
        b[5, 1, 3] = math.nan
    elif what == "inf head":                               # every block above every finite one
        q[0, 1, 50] = math.inf
    elif what == "-inf head":                              # that head below, but for two blocks
        q[0, 1, 50] = math.inf
        b[:, :, 50] = -1.0
        b[9, 1, 50], b[n - 4, 1, 50] = 0.0, 2.0
    else:
        q = q * 2.0 ** 126                                 # 64 of them pass float32's range
    check(q, b, K)


@pytest.mark.parametrize("dt", [BF, F32])
def test_random_rows_are_as_exact(dt):
    rng = rng_of(17)
    for n, K in SIZES[:2]:
        q, b = normal(rng, (1, 3, 64), dt), key_like_bounds(rng, n, 1, 64, dt)[:, 0]
        check(q, b, K, 1, 1)
        b[n // 2:] = b[:n - n // 2].flip(0)                # every score twice
        check(q, b, K)


def test_bad_ids_beside_scores_that_differ_below_the_keys():
    """Fewer good blocks than places, and exactly as many: bad ids fill up by index."""
    rng = rng_of(18)
    n = 300
    b, q = steps(n, F32, 2.0 ** -60, rng), torch.ones(1, 1, 64, dtype=F32)
    scores = exact_scores(q[0], b)
    for good in (20, 30, 31, 200):
        t = np.full(n, n, dtype=np.int32)
        at = np.sort(rng.permutation(n)[:good])
        t[at] = at
        got = select_gpu(q, b[:, None].contiguous(), t[None], [n * 16], 16, 1, 30, 0, 0)
        assert pkv.get_device_error() == -4
        order = sorted(at.tolist(), key=lambda j: (-scores[j], j)) + [j for j in range(n) if j not in set(at.tolist())]
        assert got[0, 0].tolist() == sorted(order[:30]), good
