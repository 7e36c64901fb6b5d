"""Paged attention against the 64-bit result, row by row in the norm (the bound:
tests/paged_norm.py): the cases that a wrong value somewhere would fail."""
import random

import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from paged_norm import check_rows
from paged_util import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    yield


# ---- many sequences a block -------------------------------------------------

def ragged(seed, B):
    """Chunks of one tile half, two halves and several tiles (8, 129 to 256 and
    more rows per KV head at 4 heads a group), with single tokens among them."""
    rng = random.Random(seed)
    new = [rng.choice([1, rng.randint(3, 32), rng.randint(3, 32), rng.randint(33, 64),
                       rng.randint(65, 200)]) for _ in range(B)]
    return [n + rng.choice([0, rng.randint(0, 300)]) for n in new], new


@pytest.mark.parametrize("d,bits,dtype", [(128, 4, F16), (64, 2, BF16)])
def test_alternating_short_prompts(d, bits, dtype):
    """A ragged prefill of 128 prompts: a block's items alternate between those
    with one query tile and those with two."""
    c = Case([40, 20] * 64, [40, 20] * 64, 32, 8, d, bits, 16, dtype)
    cache = c.filled()
    out = cache.attend(c.queries(), c.batch())
    assert cache.device_status() == 0
    check_rows(c, out)


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("hkv", (1, 8))
def test_ragged_prefill(seed, hkv):
    kv, new = ragged(seed, 64 + 8 * seed)
    c = Case(kv, new, 4 * hkv, hkv, (128, 64)[seed & 1], (4, 8, 2)[seed % 3], 32,
             (F16, BF16)[seed >> 1 & 1], seed=seed)
    cache = c.filled()
    out = cache.attend(c.queries(), c.batch())
    assert cache.device_status() == 0
    check_rows(c, out)


@pytest.mark.parametrize("hkv", (1, 8))
def test_ragged_prefill_with_missing_pages(hkv):
    """Some sequences lose a page: the steps that miss it are theirs alone."""
    kv, new = ragged(11, 72)
    c = Case(kv, new, 4 * hkv, hkv, 128, 4, 16, F16, seed=11)
    cache = c.filled()
    gone = {}
    for b in range(0, 72, 3):
        if c.kv[b] > 40:
            c.table[b, 1] = -1
            gone[b] = range(16, 32)
    out = cache.attend(c.queries(), c.batch())
    assert cache.device_status() == kvq.KVQ_EPAGE
    check_rows(c, out, gone=gone)
