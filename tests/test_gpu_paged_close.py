"""Paged attention against the 64-bit result, row by row in the norm (the bound:
tests/paged_norm.py): the cases that a wrong value somewhere would fail."""
import itertools
import random

import numpy as np
import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from paged_norm import check_rows
from paged_util import Case, pack_row, quantize, random_case

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


# ---- every form: types, heads, lengths --------------------------------------

def go(c, scale=None, **kw):
    """One call on a cache that holds the case's tokens."""
    cache = c.filled()
    out = cache.attend(c.queries(), c.batch(), scale=scale)
    assert cache.device_status() == 0
    check_rows(c, out, scale, **kw)


ALL = list(itertools.product((64, 128), (2, 4, 8), (F16, BF16)))


@pytest.mark.parametrize("d,bits,dtype", ALL)
@pytest.mark.parametrize("rg", (1, 3, 4, 8, 16))
def test_single_tokens(d, bits, dtype, rg):
    go(Case([17, 130, 515, 1200], [1] * 4, 5 * rg, 5, d, bits, 32, dtype, seed=rg), chunks=False)


@pytest.mark.parametrize("d,bits,dtype", ALL)
@pytest.mark.parametrize("rg,new", [(1, 12), (4, 4), (3, 5)])
def test_speculated_tokens(d, bits, dtype, rg, new):
    """Nine to sixteen rows per KV head in every sequence."""
    go(Case([900, 130, 40], [new, new - 1, new], 2 * rg, 2, d, bits, 16, dtype, seed=rg),
       chunks=False)


@pytest.mark.parametrize("d,bits,dtype", ALL)
@pytest.mark.parametrize("rg", (1, 4, 7))
def test_chunks_of_new_tokens(d, bits, dtype, rg):
    go(Case([700, 300, 129, 90], [70, 33, 128, 1], 2 * rg, 2, d, bits, 64, dtype, seed=rg))


@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("kv,new,hkv", [(40000, 1, 1), (30000, 4, 1), (20000, 40, 1),
                                        (9000, 700, 2)])
def test_long_sequences(d, bits, dtype, kv, new, hkv):
    go(Case([kv], [new], 4 * hkv, hkv, d, bits, 64, dtype), chunks=new > 4)


@pytest.mark.parametrize("seed", range(40, 60))
def test_batches_of_any_shape(seed):
    c = random_case(seed)
    cache = c.filled()
    out = torch.full((c.n_tokens, c.hq, c.d), 7.0, dtype=c.dtype, device="cuda")
    cache.attend(c.queries(), c.batch(n_tokens=c.n_tokens), out=out)
    assert cache.device_status() == 0
    check_rows(c, out)
    assert (out[int(c.cu[-1]):] == 7).all()


@pytest.mark.parametrize("scale", (0.0, -0.09, 1.0, -0.5, 3e-6))
@pytest.mark.parametrize("new", (1, 4, 50))
@pytest.mark.parametrize("bits", (2, 8))
def test_scales_of_the_softmax(scale, new, bits):
    go(Case([400, 164], [new, new], 8, 2, 128, bits, 32, F16), scale)


@pytest.mark.parametrize("kmul,vmul,qmul", [(1e-4, 1e-3, 1.0), (60.0, 3000.0, 0.3),
                                            (1e-3, 1e-5, 900.0), (0.0, 1.0, 1.0),
                                            (1.0, 0.0, 1.0)])
@pytest.mark.parametrize("new,dtype", [(1, F16), (1, BF16), (4, F16), (60, F16), (60, BF16)])
def test_sizes_of_the_numbers(kmul, vmul, qmul, new, dtype):
    c = Case([460], [new], 8, 2, 128, 4, 64, dtype)
    c.K[0], c.V[0] = c._round(c.K[0] * np.float32(kmul)), c._round(c.V[0] * np.float32(vmul))
    c.q = c._round(c.q * np.float32(qmul))
    go(c)


@pytest.mark.parametrize("new", (1, 4, 30))
@pytest.mark.parametrize("at", (690, 40))
def test_one_token_passes_all_others(new, at):
    """The running maximum jumps once, late or early."""
    c = Case([731], [new], 4, 1, 128, 4, 16, F16)
    c.K[0] *= np.float32(0.05)
    c.K[0][at] = 4 * np.sign(c.q[new - 1, 0])
    c.K[0] = c._round(c.K[0])
    go(c)


@pytest.mark.parametrize("new", (1, 40))
def test_scores_that_rise_step_by_step(new):
    """Each 16 tokens score 3 (log2 units) above the last: the reference follows."""
    c = Case([900], [new], 4, 1, 128, 8, 16, F16)
    base = np.where(c.rng.random(128) < 0.5, -1, 1).astype(np.float32)
    c.q = np.broadcast_to(base, (new, 4, 128)).copy()
    step = 3 * np.log(2) / 128 ** 0.5
    c.K[0] = c._round(np.float32(0.02) * c.K[0]
                      + (np.arange(900) // 16 * np.float32(step))[:, None, None] * base)
    go(c)


@pytest.mark.parametrize("scale", (3e38, -3e38, 1e30))
@pytest.mark.parametrize("new", (1, 4, 60))
def test_queries_of_zero_at_any_scale(scale, new):
    """Every score is 0, whatever it is multiplied by: the mean of the values."""
    c = Case([200], [new], 8, 2, 128, 4, 32, BF16)
    c.q[:] = 0
    go(c, scale)


@pytest.mark.parametrize("new", (2, 4, 60))
@pytest.mark.parametrize("bad", (float("nan"), float("inf")))
def test_queries_that_are_no_numbers_stay_alone(new, bad):
    """A row and head with a NaN or an infinity has no output; all others do."""
    c = Case([500, 300], [new, new], 8, 2, 128, 4, 32, F16)
    cache, q = c.filled(), c.queries()
    rows, heads = [0, new - 1, new, 2 * new - 1], [0, 5, 3, 7]
    good = cache.attend(q, c.batch())
    q[rows, heads, 17] = bad
    out = cache.attend(q, c.batch())
    assert out[rows, heads].isnan().all()
    out[rows, heads] = good[rows, heads]
    check_rows(c, out)
    assert cache.device_status() == 0


# ---- pages, replays, streams ------------------------------------------------

@pytest.mark.parametrize("new", (2, 50))
@pytest.mark.parametrize("bad", (-1, 1 << 30))
def test_tokens_of_missing_pages_are_left_out(new, bad):
    c = Case([300], [new], 8, 2, 128, 4, 32, F16)
    cache = c.filled()
    c.table[0, 1] = bad
    out = cache.attend(c.queries(), c.batch())
    assert cache.device_status() == kvq.KVQ_EPAGE
    check_rows(c, out, gone={0: range(32, 64)})


@pytest.mark.parametrize("new", (3, 50))
def test_a_length_beyond_the_table(new):
    """The rows of a length 72 beyond the table's 256 tokens see those 256."""
    c = Case([256], [new], 8, 2, 128, 4, 32, F16)
    cache = c.filled()
    out = cache.attend(c.queries(), c.batch(kv=[328]))
    assert cache.device_status() == kvq.KVQ_EPAGE
    for i in range(new):  # one row at a time: all are behind the last token
        one = Case([256], [1], 8, 2, 128, 4, 32, F16)
        one.q = c.q[i:i + 1]
        check_rows(one, out[i:i + 1])


def test_pages_of_a_shared_prefix():
    c = Case([96 + 10, 96 + 21], [3, 6], 8, 2, 128, 4, 32, F16)
    c.table[1, :3] = c.table[0, :3]
    c.K[1][:96], c.V[1][:96] = c.K[0][:96], c.V[0][:96]
    go(c)


@pytest.mark.parametrize("most", (1, 4, 90))
@pytest.mark.parametrize("bits,dtype", [(4, F16), (2, BF16)])
def test_replays_follow_lengths_and_tables(most, bits, dtype):
    c = Case([200, 290, 300], [most, 1, most], 8, 2, 128, bits, 16, dtype)
    cache, batch = c.filled(), c.batch(n_tokens=3 * most, max_tokens=most)
    q = torch.zeros(3 * most, 8, 128, dtype=dtype, device="cuda")
    out = torch.empty_like(q)
    cache.attend(q, batch, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(q, batch, out=out)
    for kv, new in (([200, 290, 300], [most, 1, most]), ([117, 101, 299], [1, 1, most]),
                    ([128, 0, 95], [0, 0, 1])):
        d = Case(c.kv, new, 8, 2, 128, bits, 16, dtype)
        d.K, d.V = ([x[:n] for x, n in zip(y, kv)] for y in (c.K, c.V))
        d.kv, d.table = kv, c.table
        batch.seq_lens.copy_(torch.tensor(kv, dtype=torch.int32))
        batch.cu_tokens.copy_(torch.from_numpy(d.cu))
        q[:len(d.q)].copy_(d.queries())
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check_rows(d, out)
        assert (out[len(d.q):] == 7).all()
    assert cache.device_status() == 0


def test_replays_that_share_scratch():
    """A decode graph and a chunk graph on one cache, replayed in turn; both
    split pairs over blocks."""
    kv = [3000, 2500]
    cases = [Case(kv, new, 8, 2, 128, 4, 64, F16, seed=3) for new in ([1, 1], [40, 70], [4, 3])]
    cache, runs = cases[0].filled(), []
    for c in cases:
        q, batch = c.queries(), c.batch()
        cache.attend(q, batch)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = cache.attend(q, batch)
        runs.append((g, c, out, q, batch))
    for _, _, out, _, _ in runs:
        out.fill_(7.0)
    for g, _, _, _, _ in runs * 3:
        g.replay()
    torch.cuda.synchronize()
    for _, c, out, _, _ in runs:
        check_rows(c, out)
    assert cache.device_status() == 0


@pytest.mark.parametrize("new", (1, 60))
def test_a_call_waits_for_its_stream(new):
    c = Case([400, 330], [new, 1], 8, 2, 128, 4, 32, F16)
    cache, batch = c.filled(), c.batch()
    q = torch.zeros_like(c.queries())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        q.copy_(c.queries())
        out = cache.attend(q, batch)
    s.synchronize()
    check_rows(c, out)


@pytest.mark.parametrize("what", ("read", "attend"))
def test_an_output_on_another_stream_takes_no_memory_still_in_use(what):
    """A freed tensor that the current stream has yet to read keeps its contents
    while a call given another stream makes its own output."""
    c = Case([1500], [1500], 8, 8, 128, 4, 32, F16)
    cache, batch, q = c.filled(), c.batch(), c.queries()
    side = torch.cuda.Stream()
    old = torch.full_like(q, 3.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    copy = old.clone()              # runs after the sleep
    del old
    out = cache.attend(q, batch, stream=side) if what == "attend" else \
        cache.read(batch, stream=side)[0]
    torch.cuda.synchronize()
    assert (copy == 3).all()
    if what == "attend":
        check_rows(c, out)
    else:
        assert torch.equal(out.cpu(), c.expected_rows("k", c.rows))


@pytest.mark.parametrize("new", (1, 40))
def test_pages_beyond_32_bit_offsets(new):
    c = Case([600], [new], 4, 2, 128, 4, 256, F16)
    cfg = c.config()
    cfg.n_pages = (5 << 30) // kvq.paged_cache_bytes(cfg)[1]
    cache = kvq.PagedKVCache(cfg)
    c.table[0, :3] = [cfg.n_pages - 1, cfg.n_pages - 7, 3]
    cache.write(c.packed("k", whole=True), c.packed("v", whole=True), c.batch(new=[600]))
    check_rows(c, cache.attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


# ---- many heads of written rows ---------------------------------------------

@pytest.mark.parametrize("d,bits,dtype", ALL)
@pytest.mark.parametrize("hkv,rows", [(5, 70), (8, 300), (32, 45), (9, 8200)])
def test_stored_bytes_of_many_heads(d, bits, dtype, hkv, rows):
    """More heads than a warp takes at once, in short and in long calls."""
    c = Case([rows + 9, 20], [rows, 3], hkv, hkv, d, bits, 32, dtype, seed=hkv)
    cache = kvq.PagedKVCache(c.config())
    cache.pages.fill_(0xA5)
    cache.write(c.packed("k"), c.packed("v"), c.batch())
    got = c.pool_view(cache.pages)
    touched = np.zeros(got[0].shape[:1] + got[0].shape[2:4], bool)
    for b, n in enumerate(c.new):
        t = np.arange(c.kv[b] - n, c.kv[b])
        page, atom, row = c.table[b, t // 32], t % 32 // 16, t % 16
        touched[page, atom, row] = True
        for which, src, codes, stats in (("k", c.K, got[0], got[2]), ("v", c.V, got[1], got[3])):
            q, s, z = quantize(src[b][t], bits)
            assert np.array_equal(codes[page, :, atom, row], pack_row(which, q, bits))
            assert np.array_equal(stats[page, :, atom, row],
                                  np.concatenate([s, z], -1).view(np.uint8))
    for f in got:
        assert (f.transpose(0, 2, 3, 1, 4)[~touched] == 0xA5).all()
    k, v = cache.read(c.batch())
    assert torch.equal(k.cpu(), c.expected_rows("k", c.rows))
    assert torch.equal(v.cpu(), c.expected_rows("v", c.rows))
    assert cache.device_status() == 0
