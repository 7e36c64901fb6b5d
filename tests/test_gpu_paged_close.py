"""Paged attention against the 64-bit result, row by row in the norm (the bound:
tests/paged_norm.py): the cases that a wrong value somewhere would fail."""
import random

import numpy as np
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


# ---- small weights beside large ones ----------------------------------------

FORMATS = [(128, 4, F16), (64, 2, F16), (128, 8, F16), (128, 2, BF16), (64, 4, BF16)]


def many(c, new):
    """The cache of one sequence under 320 block table rows, so that a warp has a
    long stretch of tokens under one reference; each attends from `new` tokens."""
    cache, B = c.filled(), 320
    c.table, c.kv, c.new = np.repeat(c.table, B, 0), c.kv * B, [new] * B
    c.K, c.V = c.K * B, c.V * B
    c.cu = (new * np.arange(B + 1)).astype(np.int32)
    c.n_tokens = new * B
    c.q = np.tile(c.q, (B, 1, 1))
    out = cache.attend(c.queries(), c.batch())
    assert cache.device_status() == 0
    return out, (0, 1, 77, 160, 318, 319)


@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("new", (1, 4, 60))
@pytest.mark.parametrize("seen", (True, False))
def test_one_saturated_group_among_normal_ones(d, bits, dtype, new, seen):
    """One token has a group of values at the stored form's limit: the other
    groups keep the precision of their own size and, where no query attends to
    that token, so do the other tokens of its group."""
    c = Case([700], [new], 4, 1, d, bits, 32, dtype, seed=bits)
    c.V[0] = c._round(c.V[0] * np.float32(2.0 ** -6))
    c.V[0][7, :, :32] = np.resize(np.array([np.inf, -32768, 5000], np.float32), 32)
    if not seen:  # all queries share a direction, and this key looks away from it
        base = np.where(c.rng.random(d) < 0.5, -1, 1).astype(np.float32)
        c.q = c._round(base + np.float32(0.1) * c.q)
        c.K[0] = c._round(np.float32(0.3) * c.rng.standard_normal(c.K[0].shape).astype(np.float32))
        c.K[0][7] = -6 * base
    out, only = many(c, new)
    check_rows(c, out, by_group=True, only=only, chunks=new > 4)


@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("new", (1, 4, 40))
def test_a_long_tail_of_small_weights(d, bits, dtype, new):
    """One token holds nearly all of the weight and has no value of its own; the
    output is what 6000 others, each 2^-26.5 of it, add up to."""
    c = Case([6000], [new], 4, 1, d, bits, 64, dtype)
    base = np.where(c.rng.random(d) < 0.5, -1, 1).astype(np.float32)
    c.q = np.broadcast_to(base, (new, 4, d)).copy()
    c.K[0] = c._round(np.float32(0.01) * c.K[0])
    c.K[0][0] = c._round(base * np.float32(26.5 * np.log(2) / d ** 0.5))
    c.V[0] = c._round(1 + np.float32(0.3) * c.V[0])
    c.V[0][0] = 0
    out, only = many(c, new)
    check_rows(c, out, only=only, chunks=new > 4)


# ---- status and scratch -----------------------------------------------------

@pytest.mark.parametrize("new", (1, 60))
def test_a_timeout_is_not_hidden_by_an_earlier_error(new):
    """After a wait that ran out the scratch has to be cleared: the status word
    says so, whatever was recorded before."""
    c = Case([700, 300], [new, new], 8, 2, 128, 4, 32, F16)
    cache, batch, q = c.filled(), c.batch(), c.queries()
    bad = c.batch(new=[700, 300])
    bad.block_table[1, 2] = -1
    cache.read(bad)  # records KVQ_EPAGE
    try:
        kvq.debug_stall_waits(1000)
        cache.attend(q, batch)
        torch.cuda.synchronize()
    finally:
        kvq.debug_stall_waits(0)
    assert cache.device_status() == kvq.KVQ_ETIMEOUT
    check_rows(c, cache.attend(q, batch))
    assert cache.device_status() == 0


@pytest.mark.parametrize("new", (1, 60))
def test_a_new_cache_is_ready_on_every_stream(new):
    """The scratch of a cache made on a busy stream is zero before a call on
    another one starts."""
    c = Case([3000, 2500], [new, new], 8, 2, 128, 4, 64, F16)
    old, batch, q = c.filled(), c.batch(), c.queries()
    out = torch.full_like(q, 7.0)
    side = torch.cuda.Stream()
    dirty = torch.full((old.ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirty  # the allocator hands this block out again
    torch.cuda._sleep(50_000_000)
    cache = kvq.PagedKVCache(c.config(), pages=old.pages)
    with torch.cuda.stream(side):
        cache.attend(q, batch, out=out)
    torch.cuda.synchronize()
    check_rows(c, out)
    assert cache.device_status() == 0
