"""Paged cache on the GPU: stored bytes, values read back and causal attention
against the plain reference (tests/paged_util.py)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from paged_util import Case, pack_row, quantize, random_case, values

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    yield


FORMATS = list(itertools.product((64, 128), (2, 4, 8), (F16, BF16)))


# ---- write and read ---------------------------------------------------------

@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("page,hkv", [(16, 1), (32, 3), (256, 2)])
def test_stored_bytes_and_values_read_back(d, bits, dtype, page, hkv):
    c = Case([37, 1, 260, 16], [37, 1, 131, 3], hkv, hkv, d, bits, page, dtype, seed=d + bits)
    cache = kvq.PagedKVCache(c.config())
    cache.pages.fill_(0xA5)
    cache.write(c.packed("k"), c.packed("v"), c.batch())
    got = c.pool_view(cache.pages)
    touched = np.zeros(got[0].shape[:1] + got[0].shape[2:4], bool)
    for b, t in c.rows:
        page_id, atom, row = c.table[b, t // page], t % page // 16, t % 16
        touched[page_id, atom, row] = True
        for which, src, codes, stats in (("k", c.K, got[0], got[2]), ("v", c.V, got[1], got[3])):
            q, s, z = quantize(src[b][t], bits)
            assert np.array_equal(codes[page_id, :, atom, row], pack_row(which, q, bits))
            exp = np.concatenate([s, z], -1).view(np.uint8)
            assert np.array_equal(stats[page_id, :, atom, row], exp)
    for f in got:  # every other slot is as it was
        assert (f.transpose(0, 2, 3, 1, 4)[~touched] == 0xA5).all()
    k, v = cache.read(c.batch())
    assert torch.equal(k.cpu(), c.expected_rows("k", c.rows))
    assert torch.equal(v.cpu(), c.expected_rows("v", c.rows))
    assert cache.device_status() == 0


@pytest.mark.parametrize("bits", (2, 4, 8))
@pytest.mark.parametrize("dtype", (F16, BF16))
def test_values_at_the_edges(bits, dtype):
    """Infinities and large values saturate, NaN reads as 0, constant groups,
    signed zeros and the smallest numbers keep the formula."""
    c = Case([16], [16], 2, 2, 64, bits, 16, dtype)
    top = torch.finfo(dtype).max
    edge = [0.0, -0.0, float("nan"), float("inf"), -float("inf"), top, -top, 32768.0, -32767.0,
            5.9e-8, -5.9e-8, 6.1e-5, 1e-4, 1.0, -1.0, 3.0]
    x = np.zeros((16, 2, 64), np.float32)
    for t in range(16):
        x[t, 0] = edge[t]                                   # constant groups
        x[t, 1] = np.resize(np.roll(np.array(edge, np.float32), t), 64)
        x[t, 1, 32 + t:] = 0
    x[8, 0, 5] = np.nan
    c.K[0], c.V[0] = c._round(x), c._round(x[::-1].copy())
    cache = c.filled()
    k, v = cache.read(c.batch())
    for got, which in ((k, "k"), (v, "v")):
        exp = c.expected_rows(which, c.rows)
        assert torch.isfinite(got.float()).all()
        assert torch.equal(got.cpu().view(torch.int16), exp.view(torch.int16))


def test_rows_of_a_fused_projection_and_padding():
    """Rows may be slices of a wider array; rows behind the last sequence are
    neither read nor written, and the pages hold nothing of them."""
    c = Case([20, 50], [4, 50], 4, 2, 128, 4, 32, BF16, pad=5)
    wide = torch.full((c.n_tokens, 8 * 128), float("nan"), dtype=BF16, device="cuda")
    n = int(c.cu[-1])
    wide[:n, 512:768] = c.packed("k").flatten(1)
    wide[:n, 768:] = c.packed("v").flatten(1)
    wide[:n, :512] = c.queries()[:n].flatten(1)
    q, k, v = (t.unflatten(1, (-1, 128)) for t in wide.split([512, 256, 256], 1))
    cache = c.filled()
    before = cache.pages.clone()
    batch = c.batch(n_tokens=c.n_tokens)
    cache.write(k, v, batch)
    assert torch.equal(cache.pages, before)
    k_out, v_out = (torch.full((c.n_tokens, 2, 128), 7.0, dtype=BF16, device="cuda")
                    for _ in range(2))
    cache.read(batch, out=(k_out, v_out))
    assert torch.equal(k_out[:n].cpu(), c.expected_rows("k", c.rows))
    assert torch.equal(v_out[:n].cpu(), c.expected_rows("v", c.rows))
    out = torch.full((c.n_tokens, 4, 128), 7.0, dtype=BF16, device="cuda")
    cache.attend(q, batch, out=out)
    c.check_attention(out)
    for t in (k_out, v_out, out):
        assert (t[n:] == 7).all()
    assert cache.device_status() == 0


# ---- attention --------------------------------------------------------------

@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("rg", (1, 3, 4, 8, 16))
def test_one_row_per_sequence(d, bits, dtype, rg):
    c = Case([1, 2, 16, 17, 130, 515], [1] * 6, 2 * rg, 2, d, bits, 32, dtype, seed=rg)
    cache = c.filled()
    c.check_attention(cache.attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


@pytest.mark.parametrize("d,bits,dtype", FORMATS)
@pytest.mark.parametrize("rg", (1, 4, 7))
def test_chunks(d, bits, dtype, rg):
    c = Case([70, 300, 129, 5], [70, 33, 1, 5], 2 * rg, 2, d, bits, 64, dtype, seed=rg)
    cache = c.filled()
    c.check_attention(cache.attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    c = random_case(seed)
    cache = c.filled()
    batch = c.batch(n_tokens=c.n_tokens)
    out = torch.full((c.n_tokens, c.hq, c.d), 7.0, dtype=c.dtype, device="cuda")
    cache.attend(c.queries(), batch, out=out)
    c.check_attention(out)
    assert (out[int(c.cu[-1]):] == 7).all()
    assert cache.device_status() == 0


@pytest.mark.parametrize("new", (1, 4, 40))
def test_rows_that_see_nothing_are_zero(new):
    """A sequence shorter than its rows: rows at negative positions."""
    c = Case([0, 2, 33], [new, new, new], 8, 2, 128, 4, 16, F16)
    cache = c.filled()
    out = cache.attend(c.queries(), c.batch())
    c.check_attention(out)
    assert (out[:new] == 0).all()
    k, v = cache.read(c.batch())
    for b, n in enumerate(c.kv):
        for i in range(new):
            if n - new + i < 0:
                assert (k[b * new + i] == 0).all() and (v[b * new + i] == 0).all()
    assert cache.device_status() == 0


@pytest.mark.parametrize("scale", (0.0, -0.09, 1.0, 3e-6))
@pytest.mark.parametrize("new", (1, 50))
def test_softmax_scales(scale, new):
    c = Case([200, 64], [new, new], 8, 2, 128, 8, 32, F16)
    c.check_attention(c.filled().attend(c.queries(), c.batch(), scale=scale), scale)


@pytest.mark.parametrize("kmul,vmul,qmul", [(1e-4, 1e-3, 1.0), (60.0, 3000.0, 0.3),
                                            (1e-3, 1e-5, 900.0), (0.0, 1.0, 1.0),
                                            (1.0, 0.0, 1.0)])
@pytest.mark.parametrize("new,dtype", [(1, F16), (1, BF16), (60, F16), (60, BF16)])
def test_magnitudes(kmul, vmul, qmul, new, dtype):
    """Keys, values and queries far from 1: no step may overflow, and small
    values keep their relative precision."""
    c = Case([260], [new], 8, 2, 128, 4, 64, dtype)
    c.K[0], c.V[0] = c._round(c.K[0] * np.float32(kmul)), c._round(c.V[0] * np.float32(vmul))
    c.q = c._round(c.q * np.float32(qmul))
    c.check_attention(c.filled().attend(c.queries(), c.batch()))


def test_one_token_dominates_late():
    """The running maximum jumps at the very last tokens, after many small ones."""
    for new in (1, 30):
        c = Case([700], [new], 4, 1, 128, 4, 16, F16)
        c.K[0] *= np.float32(0.05)
        c.K[0][690] = 4 * np.sign(c.q[new - 1, 0])
        c.K[0] = c._round(c.K[0])
        c.check_attention(c.filled().attend(c.queries(), c.batch()))


def test_shared_prefix_pages():
    """Two sequences read the same pages; only their last pages differ."""
    c = Case([64 + 10, 64 + 21], [3, 6], 4, 2, 128, 4, 32, F16)
    c.table[1, :2] = c.table[0, :2]
    c.K[1][:64], c.V[1][:64] = c.K[0][:64], c.V[0][:64]
    cache = c.filled()
    c.check_attention(cache.attend(c.queries(), c.batch()))


def test_bad_pages_are_reported_and_skipped():
    """An entry outside the pool: its tokens are not written, read as zeros and
    are not attended to; the status word says KVQ_EPAGE, once."""
    for bad in (-1, 1 << 30):
        for new in (2, 50):
            c = Case([100], [new], 4, 2, 128, 4, 32, F16)
            cache = c.filled()
            good, n_pages = c.table.copy(), c.n_pages
            c.table[0, 1] = n_pages if bad > 0 else bad
            before = cache.pages.clone()
            whole = c.batch(new=[100])
            cache.write(c.packed("k", whole=True), c.packed("v", whole=True), whole)
            assert cache.device_status() == kvq.KVQ_EPAGE
            assert cache.device_status() == 0
            assert torch.equal(cache.pages, before)  # the same bytes, nothing elsewhere
            k, v = cache.read(whole)
            exp = c.expected_rows("k", [(0, t) for t in range(100)])
            exp[32:64] = 0
            assert torch.equal(k.cpu(), exp)
            assert cache.device_status() == kvq.KVQ_EPAGE
            out = cache.attend(c.queries(), c.batch())
            assert cache.device_status() == kvq.KVQ_EPAGE
            # the same as a sequence without those tokens
            c.K[0], c.V[0] = (np.delete(x[0], slice(32, 64), 0) for x in (c.K, c.V))
            c.kv, c.table = [68], np.delete(good, 1, 1)
            c.check_attention(out)


def test_sequence_longer_than_its_table():
    """Every slot of the table is written; the length claims 72 tokens more:
    the rows see the 128 that exist."""
    for new in (3, 50):
        c = Case([128], [new], 4, 2, 128, 4, 32, F16)
        cache = c.filled()
        batch = c.batch(kv=[200])
        k, v = cache.read(batch)
        assert (k == 0).all() and (v == 0).all()
        assert cache.device_status() == kvq.KVQ_EPAGE
        out = cache.attend(c.queries(), batch)
        assert cache.device_status() == kvq.KVQ_EPAGE
        # every row at position 127 or later sees all 128: one row at a time
        for i in range(new):
            one = Case([128], [1], 4, 2, 128, 4, 32, F16)
            one.q = c.q[i:i + 1]
            one.check_attention(out[i:i + 1])


@pytest.mark.parametrize("kv,new", [([513, 40, 900], [1, 1, 1]), ([513, 40, 900], [200, 1, 77])])
def test_same_bits_every_time(kv, new):
    c = Case(kv, new, 8, 2, 128, 4, 16, BF16)
    cache = c.filled()
    batch, q = c.batch(), c.queries()
    first = cache.attend(q, batch)
    for _ in range(5):
        assert torch.equal(cache.attend(q, batch), first)


@pytest.mark.parametrize("most", (1, 4, 90))
def test_captured_graph_follows_lengths(most):
    """A captured step replayed with other lengths, tables and rows."""
    c = Case([200, 90, 300], [most, 1, most], 8, 2, 128, 4, 16, F16)
    cache = c.filled()
    batch, q = c.batch(n_tokens=3 * most, max_tokens=most), torch.zeros(3 * most, 8, 128, dtype=F16,
                                                                     device="cuda")
    out = torch.empty_like(q)
    cache.attend(q, batch, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.attend(q, batch, out=out)
    for kv, new in (([200, 90, 300], [most, 1, most]), ([17, 1, 299], [1, 1, most]),
                    ([128, 0, 5], [0, 0, 1])):
        d = Case(c.kv, new, 8, 2, 128, 4, 16, F16)
        d.K, d.V = ([x[:n] for x, n in zip(y, kv)] for y in (c.K, c.V))
        d.kv, d.table = kv, c.table
        batch.seq_lens.copy_(torch.tensor(kv, dtype=torch.int32))
        batch.cu_tokens.copy_(torch.from_numpy(d.cu))
        q[:len(d.q)].copy_(d.queries())
        g.replay()
        torch.cuda.synchronize()
        d.check_attention(out)
    assert cache.device_status() == 0


def test_captured_step_writes_attends_and_reads():
    """A whole serving step in one graph: the new rows of each replay enter the
    pages, are attended to and read back."""
    c = Case([100, 37], [1, 1], 8, 2, 64, 2, 16, BF16)
    cache = c.filled()
    batch = c.batch()
    k, v = c.packed("k"), c.packed("v")
    q = c.queries()
    cache.write(k, v, batch)
    cache.attend(q, batch)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.write(k, v, batch)
        out = cache.attend(q, batch)
        back = cache.read(batch)
    for seed in (1, 2):
        d = Case([100, 37], [1, 1], 8, 2, 64, 2, 16, BF16, seed=seed)
        d.table = c.table
        for b in range(2):  # the tokens before stay
            d.K[b][:-1], d.V[b][:-1] = c.K[b][:-1], c.V[b][:-1]
        k.copy_(d.packed("k")), v.copy_(d.packed("v")), q.copy_(d.queries())
        g.replay()
        torch.cuda.synchronize()
        d.check_attention(out)
        assert torch.equal(back[0].cpu(), d.expected_rows("k", d.rows))
        assert torch.equal(back[1].cpu(), d.expected_rows("v", d.rows))


def test_two_graphs_share_a_cache_and_its_scratch():
    """Replayed one after the other, a decode graph and a chunk graph that both
    split pairs over blocks use the same scratch."""
    kv = [3000, 2500]
    a = Case(kv, [1, 1], 8, 2, 128, 4, 64, F16, seed=3)
    b = Case(kv, [40, 70], 8, 2, 128, 4, 64, F16, seed=3)
    cache = a.filled()
    runs = []
    for c in (a, b):
        q, batch = c.queries(), c.batch()
        cache.attend(q, batch)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = cache.attend(q, batch)
        runs.append((g, c, out, q, batch))
    for g, _, _, _, _ in runs * 3:
        g.replay()
    torch.cuda.synchronize()
    for _, c, out, _, _ in runs:
        c.check_attention(out)
    assert cache.device_status() == 0


@pytest.mark.parametrize("new", (1, 60))
def test_a_wait_that_runs_out_is_reported(new):
    """The debug switch makes a wait run out: KVQ_ETIMEOUT in the status word,
    and the next call, with the scratch cleared, is right again."""
    c = Case([700, 300], [new, new], 8, 2, 128, 4, 32, F16)
    cache, batch, q = c.filled(), c.batch(), c.queries()
    try:
        kvq.debug_stall_waits(1000)
        cache.attend(q, batch)
        torch.cuda.synchronize()
    finally:
        kvq.debug_stall_waits(0)
    assert cache.device_status() == kvq.KVQ_ETIMEOUT
    c.check_attention(cache.attend(q, batch))
    assert cache.device_status() == 0


@pytest.mark.parametrize("new,launches", [(1, 1), (2, 1), (3, 2), (200, 2)])
def test_launch_counts(new, launches):
    """Up to 16 query rows a KV head are the split kernel's alone; a call that may
    hold more launches both kernels."""
    c = Case([300], [new], 8, 1, 128, 4, 32, F16)
    cache = c.filled()
    out = cache.attend(c.queries(), c.batch())
    assert kvq.lib().kvq_last_launch_count() == launches
    c.check_attention(out)
    cache.read(c.batch())
    assert kvq.lib().kvq_last_launch_count() == 1


@pytest.mark.parametrize("rg,heads", [(20, 1), (128, 1), (24, 2)])
def test_many_query_heads_per_kv_head(rg, heads):
    """More query heads per KV head than the split kernel's 16 rows: every
    sequence goes to the chunk kernel, single tokens too."""
    c = Case([200, 1, 33], [1, 1, 3], rg * heads, heads, 64, 4, 32, BF16)
    c.check_attention(c.filled().attend(c.queries(), c.batch()))
    assert kvq.lib().kvq_last_launch_count() == 1


@pytest.mark.parametrize("new", (1, 300))
def test_many_sequences(new):
    """More sequences than a warp, and than a block, has lanes."""
    B = 2047
    c = Case([1 + b % 40 for b in range(B)], [1] * B, 2, 1, 64, 8, 16, F16)
    if new > 1:  # one long chunk among them
        c = Case([400] + [1 + b % 40 for b in range(B)], [new] + [1] * B, 2, 1, 64, 8, 16, F16)
    cache = c.filled()
    c.check_attention(cache.attend(c.queries(), c.batch()))
    k, v = cache.read(c.batch())
    assert torch.equal(k.cpu(), c.expected_rows("k", c.rows))


def test_most_sequences_at_the_largest_shared_memory():
    """2048 sequences on the split kernel's 16-row form, the largest block."""
    c = Case([1 + b % 20 for b in range(2048)], [1] * 2048, 16, 1, 128, 4, 16, BF16)
    cache = c.filled()
    c.check_attention(cache.attend(c.queries(), c.batch()))
    assert cache.device_status() == 0


@pytest.mark.parametrize("kv,new,hkv", [(40000, 1, 1), (20000, 40, 1), (9000, 700, 2)])
def test_long_sequences_are_split_and_joined(kv, new, hkv):
    """Pairs that many blocks share.  The reference is torch in 64 bits on the
    GPU, the bound that of the short cases at this length."""
    c = Case([kv], [0], 4 * hkv, hkv, 128, 4, 64, F16)
    cache = c.filled()
    c.new = [new]
    c.cu = np.array([0, new], np.int32)
    c.n_tokens = new
    c.q = c._round(1.2 * c.rng.standard_normal((new, 4 * hkv, 128)).astype(np.float32))
    out = cache.attend(c.queries(), c.batch()).double()
    K, V = (torch.from_numpy(values(*quantize(x, 4))).cuda().double() for x in (c.K[0], c.V[0]))
    q = c.queries().double()
    u = 2.0 ** -11
    hidden = (torch.arange(kv, device="cuda")[None]
              > (kv - new + torch.arange(new, device="cuda"))[:, None])
    for h in range(4 * hkv):
        s = (q[:, h] @ K[:, h // 4].T) / 128 ** 0.5
        A = (q[:, h].abs() @ K[:, h // 4].abs().T) / 128 ** 0.5
        w = torch.softmax(s.masked_fill(hidden, -float("inf")), -1)
        m = V[:, h // 4].abs().amax(0) * 3
        ds = 2 * 2 * u * 3 * A.masked_fill(w < 1e-12, 0).amax(-1, keepdim=True)
        bound = (w @ (3 * V[:, h // 4].abs())) * (2 * u + torch.expm1(ds) + kv * 2.0 ** -24) \
            + kv * 2.0 ** -24 * m
        exp = w @ V[:, h // 4]
        err = (out[:, h] - exp).abs()
        assert (err <= bound + u * (exp.abs() + bound) + 1e-7).all()
        # and on the whole far closer than the worst case
        assert float(err.norm() / exp.norm()) < 2.0 ** -8
    assert cache.device_status() == 0


def test_runs_on_the_stream_it_is_given():
    c = Case([400, 30], [60, 1], 8, 2, 128, 4, 32, F16)
    cache, batch = c.filled(), c.batch()
    q = torch.zeros_like(c.queries())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        q.copy_(c.queries())
        k, v = c.packed("k"), c.packed("v")
        cache.write(k, v, batch)
        out = cache.attend(q, batch)
        k, v = cache.read(batch)
    s.synchronize()
    c.check_attention(out)
    assert torch.equal(v.cpu(), c.expected_rows("v", c.rows))


@pytest.mark.parametrize("most", (0, 2, 19))
def test_too_many_rows_for_max_tokens_is_reported(most):
    c = Case([100, 50], [20, 1], 4, 2, 128, 4, 32, F16)
    cache = c.filled()
    batch = c.batch(max_tokens=most)
    out = torch.full((21, 4, 128), 7.0, dtype=F16, device="cuda")
    cache.attend(c.queries(), batch, out=out)
    assert cache.device_status() == kvq.KVQ_EINVAL
    assert (out[:20] == 7).all()


@pytest.mark.parametrize("cu", ([0, 20, 19, 21], [0, 20, 2**31 - 1, -2**31], [0, 20, -2**31, -1]))
@pytest.mark.parametrize("most", (1, 20, 2**31 - 1))
def test_decreasing_row_offsets_are_reported(cu, most):
    c = Case([100, 50, 30], [20, 1, 1], 4, 2, 128, 4, 32, F16)
    cache = c.filled()
    batch = c.batch(max_tokens=most)
    batch.cu_tokens.copy_(torch.tensor(cu, dtype=torch.int32))
    out = torch.full((22, 4, 128), 7.0, dtype=F16, device="cuda")
    cache.attend(c.queries(), batch, out=out)
    assert cache.device_status() == kvq.KVQ_EINVAL
    assert (out[21:] == 7).all()


def test_serving_loop():
    """What a server does: two prompts enter in chunks, decode together, a third
    joins, one leaves and its pages serve the next; after every step attention
    and the values read back are those of the tokens held."""
    full = Case([90, 150, 60, 40], [0, 0, 0, 0], 8, 2, 128, 4, 16, BF16, seed=5)
    cache = kvq.PagedKVCache(full.config())
    held = [0, 0, 0, 0]
    rng = np.random.default_rng(1)
    steps = [[48, 0, 0, 0], [20, 70, 0, 0], [1, 64, 0, 0], [1, 1, 33, 0], [1, 1, 1, 0],
             [1, 1, 20, 40], [1, 1, 1, 0]]
    for new in steps:
        held = [h + n for h, n in zip(held, new)]
        c = Case(held, new, 8, 2, 128, 4, 16, BF16, seed=int(rng.integers(1 << 30)))
        c.K, c.V = [k[:h] for k, h in zip(full.K, held)], [v[:h] for v, h in zip(full.V, held)]
        c.table, c.n_pages = full.table, full.n_pages
        batch = c.batch()
        cache.write(c.packed("k"), c.packed("v"), batch)
        c.check_attention(cache.attend(c.queries(), batch))
        whole = c.batch(new=held)
        k, v = cache.read(whole)
        tokens = [(b, t) for b, h in enumerate(held) for t in range(h)]
        assert torch.equal(k.cpu(), c.expected_rows("k", tokens))
        assert torch.equal(v.cpu(), c.expected_rows("v", tokens))
    assert cache.device_status() == 0


def test_pool_beyond_32_bit_offsets():
    """Pages whose byte offset passes 2^32."""
    c = Case([300], [40], 4, 2, 128, 4, 256, F16)
    small = c.filled()
    cfg = c.config()
    pool, page = kvq.paged_cache_bytes(cfg)
    cfg.n_pages = (5 << 30) // page
    cache = kvq.PagedKVCache(cfg)
    c.table = c.table.copy()
    c.table[0, :2] = [cfg.n_pages - 1, cfg.n_pages - 7]
    whole = c.batch(new=[300])
    cache.write(c.packed("k", whole=True), c.packed("v", whole=True), whole)
    c.check_attention(cache.attend(c.queries(), c.batch()))
    one = Case([300], [1], 4, 2, 128, 4, 256, F16)
    one.table = c.table
    one.check_attention(cache.attend(one.queries(), one.batch()))
    assert torch.equal(cache.read(whole)[0].cpu(),
                       c.expected_rows("k", [(0, t) for t in range(300)]))
    assert cache.device_status() == 0
    del small, cache
    torch.cuda.empty_cache()
