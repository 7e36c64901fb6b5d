"""Cross attention over the pages: every row sees all tokens of its sequence.  The
bound is the causal one's (tests/paged_norm.py) of as many sequences of one row."""
import itertools
import random

import numpy as np
import pytest
import torch

import paged_norm
from bit_kv_cache_14_gb300 import build_lib, kvq
from paged_util import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    yield


def check_rows(case, out, **kw):
    """paged_norm.check_rows, a sequence's stored values worked out once for all of its
    rows."""
    plain, memo = paged_norm.held, {}

    def held(case, which, b, device):
        key = which, id((case.K if which == "k" else case.V)[b])
        if key not in memo:
            memo[key] = plain(case, which, b, device)
        return memo[key]

    paged_norm.held = held
    try:
        return paged_norm.check_rows(case, out, **kw)
    finally:
        paged_norm.held = plain


class Cross(Case):
    """A case whose rows are no tokens of the sequences: any number of them."""

    def filled(self, device="cuda"):
        new, self.new = self.new, [max(k, 0) for k in self.kv]
        cache = super().filled(device)
        self.new = new
        return cache

    def single_rows(self):
        """The same attention as causal rows, one a sequence."""
        one = object.__new__(Case)
        one.__dict__.update(self.__dict__)
        at = [b for b, n in enumerate(self.new) for _ in range(n)]
        one.kv, one.new = [self.kv[b] for b in at], [1] * len(at)
        one.K, one.V = [self.K[b] for b in at], [self.V[b] for b in at]
        one.cu = np.arange(len(at) + 1)
        return one

    def check(self, out, **kw):
        return check_rows(self.single_rows(), out, **kw)


FORMATS = list(itertools.product((64, 128), (2, 4, 8), (F16, BF16)))


@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("new", [(1, 1, 1, 1, 1), (4, 3, 2, 1, 4), (16, 0, 9, 12, 5),
                                 (40, 1, 130, 300, 7)])
def test_against_64_bits(d, bits, dtype, new):
    """Empty encoders, one token, pages and tiles that end inside; more rows than
    tokens; few rows, many, and both in one call."""
    c = Cross([150, 1, 0, 129, 300], new, 8, 2, d, bits, 32, dtype, seed=d + bits)
    cache = c.filled()
    out = cache.cross_attend(c.queries(), c.batch())
    assert cache.device_status() == 0
    c.check(out)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = random.Random(seed)
    hkv, rg = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 8, 16, 20])
    B = rng.randint(1, 6)
    kv = [rng.choice([0, 1, 15, 16, 17, 33, 127, 128, 129, 300, 700]) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 2, 5, 33, 90, 400 // rg]) for _ in range(B)]
    c = Cross(kv, new, hkv * rg, hkv, rng.choice([64, 128]), rng.choice([2, 4, 8]),
              rng.choice([16, 32, 64, 128, 256]), rng.choice([F16, BF16]), seed=seed,
              pad=rng.choice([0, 3]))
    cache = c.filled()
    out = torch.full((c.n_tokens, c.hq, c.d), 7.0, dtype=c.dtype, device="cuda")
    cache.cross_attend(c.queries(), c.batch(n_tokens=c.n_tokens), out=out)
    assert cache.device_status() == 0
    c.check(out)
    assert (out[int(c.cu[-1]):] == 7).all()      # padding is left alone


@pytest.mark.parametrize("bits", (2, 4, 8))
@pytest.mark.parametrize("rg", (1, 4))
def test_one_row_is_the_decode_step(bits, rg):
    """The newest token sees everything: with one row the causal call's bits."""
    c = Cross([900, 64, 1, 333], [1] * 4, 2 * rg, 2, 128, bits, 64, BF16)
    cache = c.filled()
    assert torch.equal(cache.cross_attend(c.queries(), c.batch()),
                       cache.attend(c.queries(), c.batch()))


def test_beams_share_the_reads_of_an_encoder():
    """Beams as rows of one sequence, or as sequences over the same pages: both are
    the operator."""
    c = Cross([700, 90], [4, 4], 8, 2, 128, 4, 16, F16)
    cache = c.filled()
    q = c.queries()
    together = cache.cross_attend(q, c.batch())
    t = lambda a: torch.from_numpy(np.repeat(a, 4, 0).astype(np.int32)).cuda()  # noqa: E731
    apart = kvq.PagedBatch(t(c.table), t(np.array(c.kv)),
                           torch.arange(9, dtype=torch.int32, device="cuda"), 8, 1)
    c.check(together)
    c.check(cache.cross_attend(q, apart))


@pytest.mark.parametrize("rows", (3, 70))
def test_missing_pages_and_lengths(rows):
    """A page that is not there is not attended to; a length beyond the table ends
    with it."""
    c = Cross([200, 200, 64], [rows] * 3, 4, 1, 64, 4, 16, F16)
    cache = c.filled()
    c.table[1, 3] = c.n_pages
    out = cache.cross_attend(c.queries(), c.batch())
    assert cache.device_status() == kvq.KVQ_EPAGE
    one = c.single_rows()
    check_rows(one, out, gone={rows + i: range(48, 64) for i in range(rows)})
    c.table[1, 3] = 0
    long = c.batch(kv=[200, 200, 10 ** 6])
    cache.cross_attend(c.queries(), long)
    assert cache.device_status() == kvq.KVQ_EPAGE
    neg = cache.cross_attend(c.queries(), c.batch(kv=[-3, 0, -2 ** 31]))
    assert (neg == 0).all() and cache.device_status() == 0


@pytest.mark.parametrize("rows", (1, 3, 12, 30, 70))
@pytest.mark.parametrize("length", (65, 10 ** 6, 2 ** 31 - 1))
def test_a_length_beyond_the_table_ends_with_it(rows, length):
    """What is attended to is what the table holds: its 64 tokens, and the other
    sequence's as ever."""
    c = Cross([64, 50], [rows] * 2, 4, 1, 64, 4, 16, F16)
    cache = c.filled()
    out = cache.cross_attend(c.queries(), c.batch(kv=[length, 50]))
    assert cache.device_status() == kvq.KVQ_EPAGE
    c.check(out)
    assert torch.equal(out, cache.cross_attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


def test_queries_of_a_wider_tensor_and_any_scale():
    c = Cross([130, 260], [2, 50], 4, 2, 128, 8, 64, BF16)
    cache = c.filled()
    wide = torch.randn(52, 9, 128, device="cuda").to(BF16)
    wide[:, 3:7] = c.queries()
    for scale in (0.0, -0.05, 0.3):
        out = cache.cross_attend(wide[:, 3:7], c.batch(), scale=scale)
        c.check(out, scale=scale)


def test_captured_with_lengths_that_change():
    c = Cross([300, 40], [2, 30], 4, 1, 64, 4, 16, F16)
    cache = c.filled()
    batch, q = c.batch(), c.queries()
    out = cache.cross_attend(q, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.cross_attend(q, batch, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.cross_attend(q, batch, out=out)
    K, V = c.K, c.V
    for lens in ([300, 40], [17, 0], [1, 33]):
        batch.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.kv, c.K, c.V = lens, [K[0][:lens[0]], K[1][:lens[1]]], [V[0][:lens[0]], V[1][:lens[1]]]
        c.check(out)
    assert cache.device_status() == 0


def test_given_stream():
    c = Cross([500], [3], 4, 2, 64, 2, 32, F16)
    cache = c.filled()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = cache.cross_attend(c.queries(), c.batch(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.check(out)


# ---- a few beams or samples: 9 to 32 rows per KV head --------------------------------

@pytest.mark.parametrize("bits,dtype", list(itertools.product((2, 4, 8), (F16, BF16))))
@pytest.mark.parametrize("rg,new", [(1, [9, 1, 16, 3]), (4, [8, 2, 1, 5]), (1, [31, 32, 0, 17]),
                                    (16, [1, 1, 2, 1]), (5, [6, 6, 6, 6])])
def test_rows_of_beams(bits, dtype, rg, new):
    c = Cross([1000, 127, 0, 385], new, 2 * rg, 2, 128, bits, 64, dtype, seed=rg)
    cache = c.filled()
    out = cache.cross_attend(c.queries(), c.batch())
    assert cache.device_status() == 0
    c.check(out)


@pytest.mark.parametrize("bits", (2, 4, 8))
@pytest.mark.parametrize("kv,rows", [([9000], 12), ([30000], 32), ([128] * 60, 10),
                                     ([1] * 40 + [4000], 16), ([129, 5000, 0, 1] * 9, 20),
                                     ([500] * 19, 24)])
def test_beams_shared_by_blocks(bits, kv, rows):
    """One long encoder over all blocks, several pairs a block, both."""
    c = Cross(kv, [rows] * len(kv), 3, 3, 128, bits, 16, F16, seed=len(kv))
    cache = c.filled()
    q = c.queries()
    out = cache.cross_attend(q, c.batch())
    assert cache.device_status() == 0
    c.check(out)
    for _ in range(3):       # joined in an order of its own: the same bits
        assert torch.equal(out, cache.cross_attend(q, c.batch()))


@pytest.mark.parametrize("d,bits", [(128, 4), (64, 2), (128, 8), (64, 4)])
@pytest.mark.parametrize("kv,new,rg", [([3000], [33], 1), ([9000, 100, 0, 1], [40, 128, 64, 20], 1),
                                       ([700] * 60, [5, 30, 9] * 20, 4),
                                       ([129, 128, 127, 2500] * 6, [17, 32, 100, 31] * 6, 4)])
def test_tiles_of_a_few_dozen_rows(d, bits, kv, new, rg):
    """17 to 128 rows per KV head: a tile over all blocks, tiles of one step, whole tiles
    next to each other, tiles of more rows and of few among them."""
    c = Cross(kv, new, rg * 2, 2, d, bits, 64, (F16, BF16)[bits == 4], seed=d)
    cache = c.filled()
    q = c.queries()
    out = cache.cross_attend(q, c.batch())
    assert cache.device_status() == 0
    c.check(out)
    for _ in range(2):
        assert torch.equal(out, cache.cross_attend(q, c.batch()))


def test_many_sequences_of_beams():
    c = Cross([(37 * i) % 300 for i in range(350)], [9 if i % 7 else 2 for i in range(350)], 1, 1,
              128, 4, 32, BF16)
    cache = c.filled()
    c.check(cache.cross_attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


@pytest.mark.parametrize("rows", (12, 30))
@pytest.mark.parametrize("up", (True, False))
def test_references_that_move(rows, up):
    """Scores that grow (or fall) by hundreds along the sequence, in one row and not in
    the others."""
    c = Cross([1500], [rows], 1, 1, 128, 8, 64, F16, seed=3)
    base = np.where(c.rng.random(128) < 0.5, -1, 1).astype(np.float32)
    ramp = np.linspace(-1, 1, 1500).astype(np.float32) * (1 if up else -1)
    c.K[0] = c._round(0.2 * c.rng.standard_normal((1500, 1, 128)).astype(np.float32)
                      + ramp[:, None, None] * base)
    c.q[:, 0] = c._round(0.3 * c.q[:, 0])
    c.q[3, 0] = 30 * base
    c.q[7, 0] = -30 * base
    cache = c.filled()
    out = cache.cross_attend(c.queries(), c.batch())
    assert cache.device_status() == 0
    c.check(out)


def test_rows_that_are_not_numbers_stay_alone():
    c = Cross([700, 40], [14, 10], 2, 1, 128, 4, 32, F16)
    cache = c.filled()
    q = c.queries()
    want = cache.cross_attend(q, c.batch())
    q[5, 1, 7] = float("nan")
    q[15, 0, 100] = float("inf")
    got = cache.cross_attend(q, c.batch())
    keep = torch.ones(24, 2, dtype=torch.bool)
    keep[5, 1] = keep[15, 0] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])
    assert got[5, 1].isnan().all() and got[15, 0].isnan().all()


@pytest.mark.parametrize("rows", (10, 25))
def test_beams_without_some_pages(rows):
    c = Cross([300, 300, 64], [rows] * 3, 1, 1, 128, 4, 16, F16)
    cache = c.filled()
    c.table[1, 3] = -1
    c.table[1, 18] = c.n_pages
    out = cache.cross_attend(c.queries(), c.batch())
    assert cache.device_status() == kvq.KVQ_EPAGE
    lost = list(range(48, 64)) + list(range(288, 300))
    check_rows(c.single_rows(), out, gone={rows + i: lost for i in range(rows)})
    neg = cache.cross_attend(c.queries(), c.batch(kv=[-3, 0, -2 ** 31]))
    assert (neg == 0).all() and cache.device_status() == 0


def test_bad_rows_of_beams():
    """Rows out of order and more rows than max_tokens says are reported."""
    c = Cross([100, 100], [10, 10], 1, 1, 128, 4, 16, F16)
    cache = c.filled()
    batch = c.batch(max_tokens=12)
    batch.cu_tokens.copy_(torch.tensor([0, 13, 20], dtype=torch.int32))
    cache.cross_attend(c.queries(), batch)
    assert cache.device_status() == kvq.KVQ_EINVAL
    batch.cu_tokens.copy_(torch.tensor([0, 10, 20], dtype=torch.int32))
    c.check(cache.cross_attend(c.queries(), batch))
    assert cache.device_status() == 0


def test_a_wait_that_runs_out_ends_the_call():
    """Beams after the stall switch: the status says so, scratch is cleared, and the
    next call is right."""
    c = Cross([2000, 300], [12, 12], 2, 2, 128, 4, 32, F16)
    cache = c.filled()
    kvq.debug_stall_waits(2000)
    try:
        cache.cross_attend(c.queries(), c.batch())
        assert cache.device_status() == kvq.KVQ_ETIMEOUT
    finally:
        kvq.debug_stall_waits(0)
    c.check(cache.cross_attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


def test_captured_beams_beside_the_causal_call():
    """The same scratch serves cross and causal calls one after the other, captured."""
    c = Cross([900, 64], [3, 3], 8, 2, 128, 4, 64, BF16)
    cache = c.filled()
    q, batch = c.queries(), c.batch()
    want = cache.cross_attend(q, batch), cache.attend(q, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.cross_attend(q, batch), cache.attend(q, batch)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [f(q, batch) for f in (cache.cross_attend, cache.attend) * 2]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want * 2):
            assert torch.equal(x, y)
