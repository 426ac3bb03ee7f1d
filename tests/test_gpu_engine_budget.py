"""The engine with caches of bounded size where its limits are: rows of token weights of any
number of tokens, used to the last one, each step against float64 on the pool's own values."""
import pytest
import torch

from _lib import library, pkv
from test_gpu_engine_eviction import Loop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def on_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    library()
    torch.cuda.set_device(0)
    pkv.get_device_error()


def loop(max_tokens, max_seqs=6, **kw):
    """A serving loop whose rows of token weights hold ``max_tokens``."""
    x = Loop(**kw)
    x.c.token_weights = None
    x.c.enable_token_weights(max_seqs, max_tokens)
    assert x.c.token_weights.shape[2] == -(-max_tokens // 4) * 4
    return x


@pytest.mark.parametrize("max_tokens", [50, 97, 99])
def test_every_token_that_the_rows_hold(max_tokens):
    """Prompts and steps up to max_tokens, which end inside a block, and an eviction from there."""
    x = loop(max_tokens, seed=max_tokens)
    x.prompts([0, 1], [max_tokens, max_tokens - 3], 8)
    for _ in range(3):
        x.decode([1])
    assert x.c.bm.seq_len(0) == x.c.bm.seq_len(1) == max_tokens
    x.evict([0, 1], 20, 2, 5)
    for _ in range(max_tokens - 20):
        x.decode([1, 0])
    assert x.c.bm.seq_len(0) == max_tokens
    x.evict([1], 33, 0, 1)
    assert pkv.get_device_error() == 0
