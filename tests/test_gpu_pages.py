"""Page tables and page copies on the GPU against the lists of tests/pages_util.py:
every table, count and free page after every call."""
import random

import numpy as np
import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from pages_util import both, cu_of, i32, pairs_of
from paged_util import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    yield


def reserve(m, tab, n, fails=False):
    """One call on both; the device's copies and cu_tokens are the model's."""
    want = m.reserve(n)
    assert (want is None) == fails
    copies, cu = tab.reserve(i32(cu_of(n)))
    assert np.array_equal(copies.cpu().numpy(), pairs_of(want or [], len(n)))
    assert np.array_equal(cu.cpu().numpy(), cu_of(n) * (want is not None))
    assert tab.device_status() == (kvq.KVQ_ECAPACITY if fails else kvq.KVQ_OK)
    m.check(tab)
    return want, copies


def test_a_new_table_is_empty():
    m, tab = both(77, 16, 5, 9)
    m.check(tab)
    assert int(tab.free_pages) == 77


SIZES = [(40, 16, 1, 40), (33, 16, 3, 12), (1, 256, 1, 1), (300, 32, 17, 30), (64, 64, 2, 64),
         (5000, 16, 40, 700), (2100, 16, 1023, 6), (4000, 16, 2048, 4), (70000, 16, 1025, 80)]


@pytest.mark.parametrize("n_pages,page,B,width", SIZES)
@pytest.mark.parametrize("seed", range(3))
def test_random_walk(n_pages, page, B, width, seed):
    """Reserve, drop, select and compact in any order; some reservations fail."""
    rng = random.Random(repr((n_pages, page, B, width, seed)))
    m, tab = both(n_pages, page, B, width)
    share = max(1, 2 * n_pages * page // B)  # tokens a sequence may take of the pool
    for step in range(14):
        kind = rng.choice(["reserve", "reserve", "reserve", "drop", "select", "compact"])
        if kind == "reserve":
            most = rng.choice([1, 2, 20, share])
            n = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(B)]
            trial = type(m)(n_pages, page, B, width)
            trial.rows, trial.lens = [list(r) for r in m.rows], list(m.lens)
            reserve(m, tab, n, fails=trial.reserve(n) is None)
        elif kind == "drop":
            t = [rng.choice([0, -5, 1, rng.randint(0, 3 * page), 2 ** 31 - 1]) for _ in range(B)]
            m.drop(t)
            tab.drop(i32(t))
        elif kind == "select":
            p = [rng.choice([b, b, -1, rng.randrange(B)]) for b in range(B)]
            m.select(p)
            tab.select(i32(p))
        else:
            want = m.compact()
            got = tab.compact()
            assert np.array_equal(got.cpu().numpy(), pairs_of(want, max(1, n_pages // 2)))
        m.check(tab)
        assert tab.device_status() == kvq.KVQ_OK


@pytest.mark.parametrize("n", [1, 15, 16, 17, 160])
def test_lengths_at_a_page_border(n):
    m, tab = both(64, 16, 3, 12)
    reserve(m, tab, [n, 0, 1])
    for t in ([0, 0, 1], [1, 0, 0], [n - 1, 9, 0], [1, 1, 1]):
        m.drop(t)
        tab.drop(i32(t))
        m.check(tab)
        reserve(m, tab, t)


def test_beams_share_and_part():
    """Beams that all hold a begun page and all write: the first keeps it.  Where
    one holder does not write, every writer copies."""
    m, tab = both(200, 16, 12, 20)
    reserve(m, tab, [37] + [0] * 11)
    p = [0] * 8 + list(range(8, 12))
    m.select(p)
    tab.select(i32(p))
    m.check(tab)
    want, _ = reserve(m, tab, [1] * 8 + [0] * 4)
    assert len(want) == 7
    p = [3, 3, 3, 3, 5, 5, 6, 6, 3, -1, -1, 7]
    m.select(p)
    tab.select(i32(p))
    want, _ = reserve(m, tab, [1] * 8 + [0] * 4)
    # 3 is held by slot 8 too and 7 by slot 11, which do not write
    assert len(want) == 4 + 1 + 1
    for _ in range(20):
        p = [random.Random(len(m.rows[0])).randrange(8) for _ in range(8)] + [-1] * 4
        m.select(p)
        tab.select(i32(p))
        m.check(tab)
        reserve(m, tab, [1] * 8 + [0] * 4)


def test_a_failed_reservation_of_shared_pages_changes_nothing():
    m, tab = both(9, 16, 4, 8)
    reserve(m, tab, [40, 0, 0, 16])
    p = [0, 0, 0, 3]
    m.select(p)
    tab.select(i32(p))
    before = [x.clone() for x in (tab.block_table, tab.seq_lens, tab.page_refs)]
    reserve(m, tab, [1, 1, 1, 60], fails=True)   # three writers, one keeps: 2 + 4 of 5 pages
    reserve(m, tab, [1, 1, 0, 64], fails=True)   # a holder does not write: both copy
    for x, y in zip(before, (tab.block_table, tab.seq_lens, tab.page_refs)):
        assert torch.equal(x, y)
    reserve(m, tab, [1, 1, 1, 48])
    assert int(tab.free_pages) == 0
    reserve(m, tab, [0, 0, 0, 1], fails=True)
    reserve(m, tab, [1, 1, 1, 0])                # needs none


def test_rows_longer_than_the_table():
    m, tab = both(100, 16, 3, 4)
    reserve(m, tab, [64, 1, 0])
    reserve(m, tab, [1, 1, 1], fails=True)
    reserve(m, tab, [0, 63, 5])
    n = i32([0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1])   # a length no table holds
    tab.reserve(n)
    assert tab.device_status() == kvq.KVQ_ECAPACITY
    m.check(tab)


@pytest.mark.parametrize("width", (20, 3000))
def test_every_sequence_ends(width):
    """The lengths themselves as what is taken back."""
    m, tab = both(5000, 16, 5, width)
    reserve(m, tab, [100, 0, 17, 1, 16 * min(width, 2000)])
    m.drop(m.lens)
    tab.drop(tab.seq_lens)
    m.check(tab)
    assert int(tab.free_pages) == 5000 and tab.device_status() == 0


def test_long_rows_are_shared_by_warps():
    """Rows of 3000 entries (more than one stretch) forked, dropped and freed."""
    m, tab = both(9000, 16, 3, 3000)
    reserve(m, tab, [47990, 0, 33333])
    for p in ([0, 0, 2], [2, 1, 0], [-1, 1, 0], [1, 1, 1]):
        m.select(p)
        tab.select(i32(p))
        m.check(tab)
        t = [7, 20001, 16]
        m.drop(t)
        tab.drop(i32(t))
        m.check(tab)
    m.drop([2 ** 31 - 1] * 3)
    tab.drop(i32([2 ** 31 - 1] * 3))
    m.check(tab)
    assert int(tab.free_pages) == 9000 and tab.device_status() == 0


@pytest.mark.parametrize("cu", [[0, 5, 4, 9], [0, -3, 4, 9], [2, 5, 7, 9], [-1, 0, 3, 4]])
def test_bad_cu_tokens(cu):
    m, tab = both(50, 16, 3, 8)
    reserve(m, tab, [20, 3, 0])
    copies, call = tab.reserve(i32(cu))
    assert tab.device_status() == kvq.KVQ_EINVAL
    assert (copies == -1).all() and (call == 0).all()
    m.check(tab)


@pytest.mark.parametrize("parents", [[0, 3, 2], [-2, 1, 2], [0, 2 ** 31 - 1, 0],
                                     [-2 ** 31, 0, 1]])
def test_bad_parents(parents):
    m, tab = both(50, 16, 3, 8)
    reserve(m, tab, [20, 3, 40])
    m.select([p if -1 <= p < 3 else b for b, p in enumerate(parents)])
    tab.select(i32(parents))
    assert tab.device_status() == kvq.KVQ_EINVAL
    m.check(tab)


def test_entries_that_are_no_pages():
    """A table the caller broke: reported, skipped, and nothing outside is touched."""
    for bad in (-7, 50, 2 ** 31 - 1):
        m, tab = both(50, 16, 3, 8)
        reserve(m, tab, [20, 3, 40])
        tab.block_table[0, 1] = bad
        tab.reserve(i32([0, 1, 1, 1]))
        assert tab.device_status() == kvq.KVQ_EPAGE
        tab.select(i32([0, 0, 2]))
        assert tab.device_status() == kvq.KVQ_EPAGE
        tab.compact()
        assert tab.device_status() == kvq.KVQ_EPAGE
        tab.drop(i32([20, 20, 40]))
        assert tab.device_status() == kvq.KVQ_EPAGE
        tab.recount()
        assert tab.device_status() == kvq.KVQ_OK and int(tab.free_pages) == 50
    # counts that do not agree with the tables
    m, tab = both(50, 16, 3, 8)
    reserve(m, tab, [20, 3, 40])
    tab.page_refs[int(tab.block_table[1, 0])] = 0
    tab.reserve(i32([0, 0, 1, 1]))
    assert tab.device_status() == kvq.KVQ_EINVAL
    tab.drop(i32([0, 3, 0]))
    assert tab.device_status() == kvq.KVQ_EINVAL
    tab.recount()
    tab.seq_lens[0] = -4
    tab.reserve(i32([0, 1, 1, 1]))
    assert tab.device_status() == kvq.KVQ_EINVAL
    tab.recount()
    assert tab.device_status() == kvq.KVQ_EINVAL


@pytest.mark.parametrize("bad", (-1, -4, -2 ** 31, 8 * 16 + 1, 2 ** 31 - 1))
def test_lengths_that_are_none(bad):
    """A negative length, or one beyond the table: every call that meets it says so and
    leaves that sequence as it is; the others get what they were to."""
    code = kvq.KVQ_EINVAL if bad < 0 else kvq.KVQ_EPAGE
    m, tab = both(50, 16, 4, 8)
    reserve(m, tab, [20, 35, 40, 0])
    tab.seq_lens[1] = bad

    def check(status):
        assert tab.device_status() == status
        true, m.lens[1] = m.lens[1], bad
        m.check(tab)
        m.lens[1] = true

    for tokens in ([1, 5, 17, 0], [0, 0, 0, 0], [0, 2 ** 31 - 1, 3, 9]):
        tab.drop(i32(tokens))
        m.drop([0 if b == 1 else n for b, n in enumerate(tokens)])
        check(code)
    for parents, want in (([0, 1, 1, 0], [0, 1, 2, 0]),   # a parent without a length
                          ([0, 0, 2, -1], [0, 1, 2, -1]),  # itself without one
                          ([2, -1, 0, 0], [2, 1, 0, 0])):
        tab.select(i32(parents))
        m.select(want)
        check(code)
    m.drop([99, 0, 99, 99])
    tab.drop(i32([99, 0, 99, 99]))
    check(code)
    moves = m.compact()                      # pages of all rows move, also that one's
    assert moves and any(to in m.rows[1] for _, to in moves)
    got = tab.compact()
    assert np.array_equal(got.cpu().numpy(), pairs_of(moves, 25))
    check(code)
    tab.seq_lens[1] = m.lens[1]              # put right, the tables agree again
    reserve(m, tab, [1, 1, 1, 1])


@pytest.mark.parametrize("B", (6, 1500))
@pytest.mark.parametrize("forks", (False, True))
def test_a_free_count_beyond_the_map(B, forks):
    """The head of the state says that more pages are free than the map holds (it was
    written to from outside): reported, and as with too few pages nothing changes."""
    n_pages = B + 40
    m, tab = both(n_pages, 16, B, 60)
    reserve(m, tab, [20, 0, 0] + [16] * (B - 3))
    if forks:
        p = [0, 0, 0] + list(range(3, B))
        m.select(p)
        tab.select(i32(p))
    free = int(tab.free_pages)
    n = [1 if forks else 0, 2 if forks else 0, 16 * free, 16] + [0] * (B - 4)
    out = torch.full((B, 2), 7, dtype=torch.int32, device="cuda"), i32([9] * (B + 1))
    tab.free_pages.fill_(2 * n_pages)
    tab.reserve(i32(cu_of(n)), out=out)
    assert tab.device_status() == kvq.KVQ_EINVAL
    assert (out[0] == -1).all() and (out[1] == 0).all()
    assert int(tab.free_pages) == 2 * n_pages
    tab.free_pages.fill_(free)
    m.check(tab)
    reserve(m, tab, [1] * 4 + [0] * (B - 4))


@pytest.mark.parametrize("count", (0, 21, 25, 10 ** 6, -1, -2 ** 31, 2 ** 31 - 1))
def test_compacting_with_a_free_count_that_is_none(count):
    """Reported, and nothing moves; a reservation after it stays inside the pool."""
    m, tab = both(60, 16, 3, 8)
    reserve(m, tab, [100, 37, 90])
    m.drop([99, 0, 0])
    tab.drop(i32([99, 0, 0]))
    free = int(tab.free_pages)
    assert free not in (0, 21, 25)
    tab.free_pages.fill_(count)
    got = tab.compact()
    assert tab.device_status() == kvq.KVQ_EINVAL
    assert (got == -1).all()
    tab.free_pages.fill_(free)
    m.check(tab)
    tab.free_pages.fill_(count)
    tab.reserve(i32([0, 800, 1600, 2400]))       # more than there is, by any count
    assert tab.device_status() != 0
    tab.free_pages.fill_(free)
    m.check(tab)
    reserve(m, tab, [5, 5, 5])


@pytest.mark.parametrize("bad", (-1, 16 * 3000 + 1))
def test_long_rows_without_a_length(bad):
    """The same where several warps share a row: all of them leave it alone, and what
    they count among themselves stays at zero for the next call."""
    m, tab = both(9000, 16, 3, 3000)
    reserve(m, tab, [47990, 20000, 33333])
    tab.seq_lens[1] = bad
    for _ in range(2):
        tab.drop(i32([20001, 20001, 17]))
        m.drop([20001, 0, 17])
        tab.select(i32([2, 0, 1]))
        m.select([2, 1, 2])
        assert tab.device_status() == (kvq.KVQ_EINVAL if bad < 0 else kvq.KVQ_EPAGE)
        true, m.lens[1] = m.lens[1], bad
        m.check(tab)
        m.lens[1] = true
    tab.seq_lens[1] = m.lens[1]
    m.drop([5, 19000, 33333])
    tab.drop(i32([5, 19000, 33333]))
    m.check(tab)
    assert tab.device_status() == 0


def test_tables_taken_over():
    """Given tables with garbage behind each sequence's last entry."""
    m, _ = both(60, 32, 4, 6)
    m.reserve([70, 0, 33, 1])
    m.select([0, 0, 2, 3])
    table = m.table()
    table[table < 0] = 12345
    tab = kvq.PageTable(60, 32, block_table=i32(table), seq_lens=i32(m.lens))
    m.check(tab)
    assert tab.device_status() == 0
    reserve(m, tab, [1, 1, 1, 1])
    tab.seq_lens[2] = 10 ** 6
    tab.recount()
    assert tab.device_status() == kvq.KVQ_EPAGE


def test_on_another_stream_and_outputs_given():
    m, tab = both(100, 16, 4, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = [5, 20, 0, 33]
    copies, cu = tab.reserve(i32(cu_of(n)), stream=side)
    m.reserve(n)
    p = i32([0, 1, 1, 3])
    out = torch.full((4, 2), 7, dtype=torch.int32, device="cuda"), i32([9] * 5)
    side.wait_stream(torch.cuda.current_stream())
    tab.select(p, stream=side)
    tab.reserve(i32(cu_of([1, 1, 1, 1])), out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    m.select([0, 1, 1, 3])
    want = m.reserve([1, 1, 1, 1])
    m.check(tab)
    assert np.array_equal(out[0].cpu().numpy(), pairs_of(want, 4)) and out[1].tolist() == [
        0, 1, 2, 3, 4]
    assert tab.device_status(stream=side) == 0


# ---- copies -------------------------------------------------------------------

@pytest.mark.parametrize("d,bits,page,hkv", [(64, 2, 16, 1), (128, 8, 256, 3), (128, 4, 64, 8),
                                             (64, 8, 32, 5)])
@pytest.mark.parametrize("n", (0, 1, 7, 400))
def test_copied_pages(d, bits, page, hkv, n):
    n_pages = 2 * n + 5
    cache = kvq.PagedKVCache(kvq.make_paged_config(hkv, hkv, d, bits, page, n_pages))
    gen = torch.Generator("cuda").manual_seed(n)
    cache.pages.random_(0, 256, generator=gen)
    before = cache.pages.clone().view(n_pages, -1)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    to = ids[:n]
    src = ids[n:][torch.randint(0, n_pages - n, (n,), generator=gen, device="cuda")]
    copies = torch.full((n + 9, 2), -1, dtype=torch.int32, device="cuda")
    copies[:n, 0], copies[:n, 1] = src, to
    copies[n + 2:] = 1      # behind the end
    cache.copy_pages(copies)
    want = before.clone()
    want[to.long()] = before[src.long()]
    assert torch.equal(cache.pages.view(n_pages, -1), want)
    assert cache.device_status() == 0


def test_lists_that_begin_anywhere_in_a_buffer():
    """A list is 8-byte aligned: parts of a longer one, copied on two streams."""
    n = 700
    pools = [kvq.PagedKVCache(kvq.make_paged_config(2, 2, 64, 4, 16, 2 * n)) for _ in range(2)]
    buf = torch.empty(2 * n + 9, 2, dtype=torch.int32, device="cuda")
    want = []
    for i, pool in enumerate(pools):
        gen = torch.Generator("cuda").manual_seed(i)
        pool.pages.random_(0, 256, generator=gen)
        ids = torch.randperm(2 * n, generator=gen, device="cuda").to(torch.int32)
        part = buf[1 + i * (n + 4):][:n]
        part[:, 0], part[:, 1] = ids[:n], ids[n:]
        part[n - 50 - i] = -1
        w = pool.pages.clone().view(2 * n, -1)
        w[ids[n:2 * n - 50 - i].long()] = w[ids[:n - 50 - i].long()]
        want.append(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pools]
    for i, pool in enumerate(pools):
        pool.copy_pages(buf[1 + i * (n + 4):][:n], stream=streams[i])
    torch.cuda.synchronize()
    for pool, w in zip(pools, want):
        assert torch.equal(pool.pages.view(2 * n, -1), w) and pool.device_status() == 0


def test_copies_of_pages_that_are_not_there():
    cache = kvq.PagedKVCache(kvq.make_paged_config(1, 1, 64, 4, 16, 6))
    cache.pages.random_(0, 256)
    want = cache.pages.clone().view(6, -1)
    cache.copy_pages(i32([[0, 6], [7, 1], [0, -1], [3, 3], [2 ** 31 - 1, 2], [0, 4]]))
    want[4] = want[0]
    assert cache.device_status() == kvq.KVQ_EPAGE
    assert torch.equal(cache.pages.view(6, -1), want)


def test_more_pairs_than_pages():
    cache = kvq.PagedKVCache(kvq.make_paged_config(1, 1, 64, 4, 16, 2))
    cache.pages.random_(0, 256)
    copies = torch.full((50, 2), -1, dtype=torch.int32, device="cuda")
    copies[0] = i32([1, 0])
    cache.copy_pages(copies)
    assert torch.equal(cache.pages.view(2, -1)[0], cache.pages.view(2, -1)[1])


@pytest.mark.parametrize("d,bits,page,hkv", [(64, 2, 16, 1), (128, 4, 64, 4)])
@pytest.mark.parametrize("n,gap,behind", [(0, 1, 1), (1, 1, 1), (0, 3, 300), (7, 1, 60),
                                          (300, 40, 1000), (4095, 1, 900), (4096, 1, 900),
                                          (4000, 200, 4000)])
def test_copies_end_at_the_first_negative_pair(d, bits, page, hkv, n, gap, behind):
    """Pairs behind the list's end that would really copy: another list's, as in a
    buffer used again.  All pages named behind it are left alone, wherever the end lies
    and however the list is shared among warps."""
    n_pages = n + behind + 9
    cache = kvq.PagedKVCache(kvq.make_paged_config(hkv, hkv, d, bits, page, n_pages))
    gen = torch.Generator("cuda").manual_seed(n)
    cache.pages.random_(0, 256, generator=gen)
    want = cache.pages.clone().view(n_pages, -1)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    src = ids[torch.randint(0, 9, (n + behind,), generator=gen, device="cuda")]
    pairs = torch.stack([src, ids[9:]], 1)
    ends = torch.full((gap, 2), -1, dtype=torch.int32, device="cuda")
    ends[:, 0] = torch.tensor([-1, -7, -2 ** 31] * gap, dtype=torch.int32)[:gap].cuda()
    ends[:, 1] = ids[-gap:]     # (a negative pair names a page to copy to, too)
    cache.copy_pages(torch.cat([pairs[:n], ends, pairs[n:]]))
    want[pairs[:n, 1].long()] = want[pairs[:n, 0].long()]
    assert torch.equal(cache.pages.view(n_pages, -1), want)
    assert cache.device_status() == 0


# ---- with the cache -------------------------------------------------------------

def test_forks_write_apart_and_compaction_keeps_every_token():
    """Samples of one prompt, extended by tokens of their own through copied pages;
    others end, the pool is made compact, and every sequence still reads as written."""
    page, H, d, B = 16, 2, 64, 6
    m, tab = both(60, page, B, 12)
    cache = kvq.PagedKVCache(kvq.make_paged_config(H, H, d, 8, page, 60))
    cache.pages.fill_(0xFF)
    gen = torch.Generator("cuda").manual_seed(3)
    held = [torch.zeros(0, H, d) for _ in range(B)]

    def step(n):
        copies, cu = tab.reserve(i32(cu_of(n)))
        assert m.reserve(n) is not None
        cache.copy_pages(copies)
        k = torch.randn(sum(n), H, d, generator=gen, device="cuda").half()
        cache.write(k, -k, tab.batch(cu, sum(n), max(n)))
        back, _ = cache.read(tab.batch(cu, sum(n), max(n)))
        for b, part in enumerate(back.cpu().float().split(n)):
            held[b] = torch.cat([held[b], part])
        check()

    def check():
        lens = [len(x) for x in held]
        m.check(tab)
        whole = tab.batch(i32(cu_of(lens)), sum(lens), max(lens + [1]))
        k, v = cache.read(whole)
        assert cache.device_status() == 0 and tab.device_status() == 0
        assert torch.equal(k.cpu().float(), torch.cat(held))
        assert (v.float() + k.float()).abs().max() < 0.1

    step([37, 0, 0, 16, 0, 0])
    for p in ([0, 0, 0, 3, 3, 5], [0, 2, 2, 4, 4, 1]):
        tab.select(i32(p))
        m.select(p)
        held = [held[a].clone() for a in p]
        check()
        step([1, 3, 1, 1, 20, 0])
    for t in ([0, 99, 0, 2, 3, 0], [99, 0, 5, 0, 0, 1]):
        tab.drop(i32(t))
        m.drop(t)
        held = [x[:max(0, len(x) - n)] for x, n in zip(held, t)]
        check()
        copies = tab.compact()
        m.compact()
        cache.copy_pages(copies)
        check()
        step([2, 1, 1, 0, 17, 1])


def test_a_captured_step_follows_the_tables():
    """Reserve, copy, write and read in one graph, replayed while sequences fork and
    end between replays; a replay that finds no pages writes nothing."""
    page, H, d, B = 16, 1, 64, 4
    m, tab = both(14, page, B, 10)
    cache = kvq.PagedKVCache(kvq.make_paged_config(H, H, d, 8, page, 14))
    cache.pages.zero_()
    n = [3, 3, 3, 3]
    cu_in, k = i32(cu_of(n)), torch.zeros(12, H, d, device="cuda").half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        out = tab.reserve(cu_in)
        cache.write(k, k, tab.batch(out[1], 12, 3))
        tab.drop(i32([3] * 4))
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        tab.reserve(cu_in, out=out)
        cache.copy_pages(out[0])
        cache.write(k, k, tab.batch(out[1], 12, 3))
    rng, held = random.Random(5), [[] for _ in range(B)]
    failed = 0
    for step in range(30):
        k.fill_(float(step + 1))
        graph.replay()
        if m.reserve(n) is None:
            failed += 1
            assert tab.device_status() == kvq.KVQ_ECAPACITY
            m.drop([2 ** 31 - 1, 0, 0, 0])
            tab.drop(i32([2 ** 31 - 1, 0, 0, 0]))
            held[0] = []
        else:
            for x in held:
                x += [float(step + 1)] * 3
        if step % 3 == 0:
            p = [rng.choice([b, rng.randrange(B)]) for b in range(B)]
            m.select(p)
            tab.select(i32(p))
            held = [list(held[a]) for a in p]
        m.check(tab)
        lens = [len(x) for x in held]
        got, _ = cache.read(tab.batch(i32(cu_of(lens)), sum(lens)))
        assert got[:, 0, 0].tolist() == sum(held, [])
    assert failed and cache.device_status() == 0


def test_two_tables_on_two_streams():
    """Tables share nothing: their calls may run at the same time."""
    ms, tabs = zip(*(both(4000, 16, 64, 80) for _ in range(2)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    rng = random.Random(1)
    todo = []
    for _ in range(20):
        n = [rng.randint(0, 40) for _ in range(64)]
        t = [rng.randint(0, 35) for _ in range(64)]
        todo.append((n, t, i32(cu_of(n)), i32(t)))
    torch.cuda.synchronize()
    for n, t, cu, drop in todo:
        for m, tab, s in zip(ms, tabs, streams):
            tab.reserve(cu, stream=s)
            tab.drop(drop, stream=s)
    torch.cuda.synchronize()
    for m, tab in zip(ms, tabs):
        for n, t, _, _ in todo:
            assert m.reserve(n) is not None
            m.drop(t)
        m.check(tab)


def test_case_tables_work_with_the_paged_calls():
    """A table's batch is the batch the paged calls know."""
    c = Case([40, 7, 0, 33], [1, 1, 0, 3], 4, 2, 64, 4, 16, torch.float16)
    cache = c.filled()
    lens = c.kv
    table = np.where(np.arange(c.width)[None] < -(-np.array(lens) // 16)[:, None], c.table, -1)
    tab = kvq.PageTable(c.n_pages, 16, block_table=i32(table), seq_lens=i32(lens))
    out = cache.attend(c.queries(), tab.batch(i32(c.cu), c.n_tokens))
    assert torch.equal(out, cache.attend(c.queries(), c.batch()))
    assert tab.device_status() == 0 and cache.device_status() == 0
