"""Host side of the paged cache: sizes, refusals and the binding's checks.  No
compute call is made here."""
import ctypes

import numpy as np
import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from paged_util import pack_row, quantize, slot_of, values


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_lib.build()
    yield


def _cfg(**kw):
    base = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, bits=4, page_size=32, n_pages=10)
    base.update(kw)
    return kvq.make_paged_config(**base)


def _batch(**kw):
    v = kvq._PagedBatch(0x1000, 0x1000, 0x1000, 4, 16, 3, 8)
    for k, x in kw.items():
        setattr(v, k, x)
    return v


def test_sizes():
    pool, page = kvq.paged_cache_bytes(_cfg())
    # per token and head: two rows of 64 bytes, two of 4 (scale, zero) fp16 pairs
    assert page == 32 * 2 * (2 * 64 + 2 * 16) and pool == 10 * page
    _, page = kvq.paged_cache_bytes(_cfg(bits=2, head_dim=64, page_size=256))
    assert page == 256 * 2 * (2 * 16 + 2 * 8)


@pytest.mark.parametrize("which", "kv")
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("bits", (2, 4, 8))
def test_layout_is_a_permutation(which, d, bits):
    assert sorted(slot_of(which, c, d, bits) for c in range(d)) == list(range(d))
    codes = np.random.default_rng(0).integers(0, 2 ** bits, d).astype(np.uint8)
    assert np.unpackbits(pack_row(which, codes, bits)).sum() == np.unpackbits(codes).sum()


def test_worked_group():
    """32 channels 0, 1/2, ..., 15.5 in 4 bits: scale fp16(15.5/15), zero 0."""
    x = np.arange(32, dtype=np.float32) / 2
    c, s, z = quantize(x, 4)
    assert z == 0 and s == np.float16(15.5 / 15)
    assert list(c[:5]) == [0, 0, 1, 1, 2] and c[31] == 15
    assert values(c, s, z)[31] == 15 * np.float32(s[0])


@pytest.mark.parametrize("top", (3, 15, 255))
def test_corrected_quotient_is_the_division(top):
    """The write kernel's x / (2^b - 1): q = x * r, then q + (x - top * q) * r,
    each fma rounded once, equals the IEEE quotient for every mantissa (scaling
    by powers of two changes neither)."""
    x = (np.arange(1 << 23, dtype=np.uint32) | 0x3F800000).view(np.float32)
    r = np.float32(1) / np.float32(top)
    q = x * r
    # both fmas in 64 bits: the remainder is exact there, the last sum off by
    # 2^-53 relative, far from any float32 tie it could cross
    rem = (x.astype(np.float64) - np.float64(top) * q).astype(np.float32)
    got = (rem.astype(np.float64) * np.float64(r) + q.astype(np.float64)).astype(np.float32)
    assert np.array_equal(got, x / np.float32(top))


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), kvq.KVQ_EUNSUPPORTED), (dict(bits=3), kvq.KVQ_EUNSUPPORTED),
    (dict(bits=16), kvq.KVQ_EUNSUPPORTED), (dict(page_size=24), kvq.KVQ_EUNSUPPORTED),
    (dict(page_size=8), kvq.KVQ_EUNSUPPORTED), (dict(page_size=512), kvq.KVQ_EUNSUPPORTED),
    (dict(n_q_heads=9), kvq.KVQ_EINVAL), (dict(n_q_heads=0), kvq.KVQ_EINVAL),
    (dict(n_kv_heads=0), kvq.KVQ_EINVAL), (dict(n_pages=0), kvq.KVQ_EINVAL),
    (dict(n_q_heads=258, n_kv_heads=2), kvq.KVQ_EUNSUPPORTED),
    (dict(n_pages=(1 << 31) + 1), kvq.KVQ_EUNSUPPORTED),
])
def test_config_refusals(kw, code):
    with pytest.raises(kvq.KVQError) as e:
        kvq.paged_cache_bytes(_cfg(**kw))
    assert e.value.code == code


def test_unknown_dtype():
    with pytest.raises(TypeError):
        _cfg(dtype=torch.float32)
    bad = _cfg()
    bad.dtype = 5
    with pytest.raises(kvq.KVQError):
        kvq.paged_cache_bytes(bad)


def _calls(cfg, cache, batch, rows=0x2000, stride=1024, out=0x3000, scale=0.1, ws=0x4000,
           ws_bytes=1 << 40):
    L, r = kvq.lib(), ctypes.byref
    return (L.kvq_paged_write(r(cfg), r(cache), r(batch), rows, stride, rows, stride, None),
            L.kvq_paged_read(r(cfg), r(cache), r(batch), rows, out, None),
            L.kvq_paged_attention(r(cfg), r(cache), r(batch), rows, stride, out, scale, ws,
                                  ws_bytes, None))


def test_calls_refuse_before_touching_the_device():
    cfg, cache = _cfg(), kvq._PagedCache(0x1000, 0x1000)
    for kw in (dict(block_table=None), dict(seq_lens=None), dict(cu_tokens=None), dict(n_seqs=0),
               dict(table_width=0), dict(n_tokens=-1), dict(max_tokens=-1)):
        assert set(_calls(cfg, cache, _batch(**kw))) == {kvq.KVQ_EINVAL}, kw
    for kw in (dict(n_seqs=2049), dict(table_width=1 << 40), dict(n_tokens=1 << 31)):
        assert set(_calls(cfg, cache, _batch(**kw))) == {kvq.KVQ_EUNSUPPORTED}, kw
    for kw in (dict(block_table=0x1002), dict(cu_tokens=0x1001)):
        assert set(_calls(cfg, cache, _batch(**kw))) == {kvq.KVQ_EALIGN}, kw
    ok = _batch()
    assert set(_calls(cfg, kvq._PagedCache(None, 0x1000), ok)) == {kvq.KVQ_EINVAL}
    assert set(_calls(cfg, kvq._PagedCache(0x1000, None), ok)) == {kvq.KVQ_EINVAL}
    assert set(_calls(cfg, kvq._PagedCache(0x1008, 0x1000), ok)) == {kvq.KVQ_EALIGN}
    assert set(_calls(_cfg(bits=5), cache, ok)) == {kvq.KVQ_EUNSUPPORTED}
    assert set(_calls(cfg, cache, ok, rows=None)) == {kvq.KVQ_EINVAL}
    assert set(_calls(cfg, cache, ok, rows=0x2002)) == {kvq.KVQ_EALIGN}
    w, _, a = _calls(cfg, cache, ok, stride=255)      # shorter than a row
    assert (w, a) == (kvq.KVQ_EINVAL, kvq.KVQ_EINVAL)
    w, _, a = _calls(cfg, cache, ok, stride=1028)
    assert (w, a) == (kvq.KVQ_EALIGN, kvq.KVQ_EALIGN)
    for kw, code in ((dict(scale=float("nan")), kvq.KVQ_EINVAL),
                     (dict(scale=float("inf")), kvq.KVQ_EINVAL),
                     (dict(ws=None), kvq.KVQ_EINVAL), (dict(ws=0x4008), kvq.KVQ_EALIGN),
                     (dict(ws_bytes=8), kvq.KVQ_ECAPACITY), (dict(out=None), kvq.KVQ_EINVAL),
                     (dict(out=0x3004), kvq.KVQ_EALIGN)):
        assert _calls(cfg, cache, ok, **kw)[2] == code, kw
    assert _calls(cfg, cache, ok, out=0x3004)[1] == kvq.KVQ_EALIGN
    # outputs apart from the queries, and from each other
    assert _calls(cfg, cache, ok, out=0x2000)[1:] == (kvq.KVQ_EINVAL, kvq.KVQ_EINVAL)
    assert _calls(cfg, cache, ok, out=0x2000 + 16 * 256 * 2 - 16)[1:] == (kvq.KVQ_EINVAL,) * 2
    # nothing to do: no launch, no pointer needed
    assert set(_calls(cfg, cache, _batch(n_tokens=0), rows=None)) == {kvq.KVQ_OK}
    assert kvq.lib().kvq_last_launch_count() == 0
    L, r = kvq.lib(), ctypes.byref
    assert L.kvq_paged_status(None, None) == kvq.KVQ_EINVAL
    assert L.kvq_paged_workspace_bytes(r(cfg), None) == kvq.KVQ_EINVAL
    assert L.kvq_paged_write(None, None, None, None, 0, None, 0, None) == kvq.KVQ_EINVAL


def test_strerror():
    assert "block table" in kvq.strerror(kvq.KVQ_EPAGE)


def test_batch_checks():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = kvq.PagedBatch(i32(3, 4), i32(3), i32(4), 16)
    assert (b.view.n_seqs, b.view.table_width, b.view.max_tokens) == (3, 4, 16)
    with pytest.raises(TypeError):
        kvq.PagedBatch(i32(3, 4).long(), i32(3), i32(4), 16)
    for bad in ((i32(3, 4), i32(3), i32(3)), (i32(2, 4), i32(3), i32(4)),
                (i32(4, 3).t(), i32(3), i32(4)), (i32(3), i32(3), i32(4))):
        with pytest.raises(ValueError):
            kvq.PagedBatch(*bad, 16)


def test_binding_checks_rows():
    cache = kvq.PagedKVCache.__new__(kvq.PagedKVCache)
    cache.cfg, cache.device, cache.dtype = _cfg(), torch.device("cpu"), torch.float16
    cache._index = -1
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    batch = kvq.PagedBatch(i32(1, 4), i32(1), i32(2), 5)
    row = torch.zeros(5, 2, 128, dtype=torch.float16)
    assert cache._rows(row, batch, 2) == 256
    assert cache._rows(torch.zeros(5, 6, 128, dtype=torch.float16)[:, 2:4], batch, 2) == 768
    with pytest.raises(TypeError):
        cache._rows(row.float(), batch, 2)
    for bad in (row[:4], row[:, :1], row.transpose(0, 1), row[..., ::2],
                torch.zeros(5, 2, 256, dtype=torch.float16)[..., ::2],
                torch.zeros(2, 5, 128, dtype=torch.float16).transpose(0, 1)):
        with pytest.raises(ValueError):
            cache._rows(bad, batch, 2)
    with pytest.raises(ValueError):
        kvq.PagedKVCache(_cfg(), "cpu", pages=torch.zeros(16, dtype=torch.uint8))


@pytest.mark.parametrize("stride", (0, 257, 1 << 33))
def test_stride_of_a_single_row_does_not_matter(stride):
    cache = kvq.PagedKVCache(_cfg(), device="cpu")
    i32 = dict(dtype=torch.int32)
    batch = kvq.PagedBatch(torch.zeros(1, 4, **i32), torch.ones(1, **i32),
                           torch.tensor([0, 1], **i32), 1)
    k = torch.empty_strided((1, 2, 128), (stride, 128, 1), dtype=torch.float16)
    assert cache._rows(k, batch, 2) == 2 * 128


@pytest.mark.parametrize("most,held", [(2**31 - 1, 2**31 - 1), (2**31, 2**31 - 1),
                                       (2**32 + 1, 2**31 - 1), (2**40, 2**31 - 1), (-1, -1),
                                       (-2**32 + 5, -1)])
def test_bounds_beyond_32_bits_stay_bounds(most, held):
    """max_tokens is an upper bound: one that the call's 32 bits cannot hold may
    not come out as a smaller one."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    assert kvq.PagedBatch(i32(1, 4), i32(1), i32(2), 5, most).view.max_tokens == held


def test_strides_of_no_rows_do_not_matter():
    cache = kvq.PagedKVCache(_cfg(), device="cpu")
    i32 = dict(dtype=torch.int32)
    batch = kvq.PagedBatch(torch.zeros(1, 4, **i32), torch.ones(1, **i32),
                           torch.zeros(2, **i32), 0)
    none = torch.from_numpy(np.zeros((0, 2, 128), np.float16)).as_strided((0, 2, 128), (0, 0, 0))
    assert cache._rows(none, batch, 2) == 2 * 128
    with pytest.raises(ValueError):
        cache._rows(none[:, :1], batch, 2)
