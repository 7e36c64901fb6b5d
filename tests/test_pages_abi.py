"""Host side of the page tables, the page copies, cross attention and draft
verification: sizes, refusals and the binding's checks.  No compute call is made
here."""
import ctypes
import itertools

import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from pages_util import Model

E = kvq


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_lib.build()
    yield


def _table(**kw):
    t = kvq._PageTable(0x1000, 0x1000, 0x1000, 0x1000, 0x1000, 100, 8, 4, 16)
    for k, x in kw.items():
        setattr(t, k, x)
    return t


def _table_calls(t, cu=0x2000, copies=0x3000, call=0x4000, n_copies=50):
    L, r = kvq.lib(), ctypes.byref(t)
    return (L.kvq_pages_recount(r, None), L.kvq_pages_reserve(r, cu, copies, call, None),
            L.kvq_pages_drop(r, cu, None), L.kvq_pages_select(r, cu, None),
            L.kvq_pages_compact(r, copies, n_copies, None))


def _state_bytes(t):
    n = ctypes.c_size_t()
    return kvq.lib().kvq_pages_state_bytes(ctypes.byref(t), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), E.KVQ_EINVAL), (dict(n_seqs=-1), E.KVQ_EINVAL),
    (dict(n_pages=0), E.KVQ_EINVAL), (dict(table_width=0), E.KVQ_EINVAL),
    (dict(n_seqs=2049), E.KVQ_EUNSUPPORTED), (dict(page_size=8), E.KVQ_EUNSUPPORTED),
    (dict(page_size=48), E.KVQ_EUNSUPPORTED), (dict(page_size=512), E.KVQ_EUNSUPPORTED),
    (dict(n_pages=(1 << 26) + 1), E.KVQ_EUNSUPPORTED),
    (dict(table_width=(1 << 26) + 1), E.KVQ_EUNSUPPORTED),
])
def test_table_sizes_refused(kw, code):
    assert _state_bytes(_table(**kw))[0] == code
    assert set(_table_calls(_table(**kw))) == {code}


def test_state_bytes():
    code, n = _state_bytes(_table())
    # head, map, tickets, three lists, rows to come
    assert code == 0 and n == 16 + 16 + 16 + 48 + 4 * 8 * 4
    # compaction's snapshot is 8 bytes a word of the map
    assert _state_bytes(_table(n_pages=1 << 20))[1] == 16 + (1 << 17) + 16 + 48 + (1 << 18)
    assert kvq.lib().kvq_pages_state_bytes(ctypes.byref(_table()), None) == E.KVQ_EINVAL
    assert kvq.lib().kvq_pages_state_bytes(None, ctypes.byref(ctypes.c_size_t())) == E.KVQ_EINVAL


def test_table_calls_refuse_before_touching_the_device():
    for name in ("block_table", "seq_lens", "page_refs", "state", "dev_status"):
        assert set(_table_calls(_table(**{name: None}))) == {E.KVQ_EINVAL}, name
        assert set(_table_calls(_table(**{name: 0x1002}))) == {E.KVQ_EALIGN}, name
    assert set(_table_calls(_table(state=0x1008))) == {E.KVQ_EALIGN}
    L, r = kvq.lib(), ctypes.byref(_table())
    for cu, copies, call, code in ((None, 0x3000, 0x4000, E.KVQ_EINVAL),
                                   (0x2000, None, 0x4000, E.KVQ_EINVAL),
                                   (0x2000, 0x3000, None, E.KVQ_EINVAL),
                                   (0x2000, 0x3000, 0x2000, E.KVQ_EINVAL),
                                   (0x2001, 0x3000, 0x4000, E.KVQ_EALIGN),
                                   (0x2000, 0x3004, 0x4000, E.KVQ_EALIGN),
                                   (0x2000, 0x3000, 0x4002, E.KVQ_EALIGN)):
        assert L.kvq_pages_reserve(r, cu, copies, call, None) == code
    for fn in (L.kvq_pages_drop, L.kvq_pages_select):
        assert fn(r, None, None) == E.KVQ_EINVAL and fn(r, 0x2002, None) == E.KVQ_EALIGN
        assert fn(None, 0x2000, None) == E.KVQ_EINVAL
    assert L.kvq_pages_compact(r, None, 50, None) == E.KVQ_EINVAL
    assert L.kvq_pages_compact(r, 0x3004, 50, None) == E.KVQ_EALIGN
    assert L.kvq_pages_compact(r, 0x3000, 49, None) == E.KVQ_ECAPACITY
    assert L.kvq_read_status(None, None) == E.KVQ_EINVAL


def test_copy_refusals():
    L, r = kvq.lib(), ctypes.byref
    cfg = kvq.make_paged_config(8, 2, 128, 4, 32, 10)
    cache = kvq._PagedCache(0x1000, 0x1000)
    call = lambda g, c, at, n: L.kvq_paged_copy(r(g), r(c), at, n, None)  # noqa: E731
    assert call(cfg, cache, None, 0) == E.KVQ_OK and L.kvq_last_launch_count() == 0
    assert call(cfg, cache, None, 4) == E.KVQ_EINVAL
    assert call(cfg, cache, 0x2000, -1) == E.KVQ_EINVAL
    assert call(cfg, cache, 0x2004, 4) == E.KVQ_EALIGN
    assert call(cfg, cache, 0x2000, 1 << 40) == E.KVQ_EUNSUPPORTED
    assert call(cfg, kvq._PagedCache(0x1008, 0x1000), 0x2000, 4) == E.KVQ_EALIGN
    assert call(cfg, kvq._PagedCache(None, 0x1000), 0x2000, 4) == E.KVQ_EINVAL
    assert call(cfg, kvq._PagedCache(0x1000, None), 0x2000, 4) == E.KVQ_EINVAL
    cfg.bits = 3
    assert call(cfg, cache, 0x2000, 4) == E.KVQ_EUNSUPPORTED


def test_cross_attention_refuses_what_attention_refuses():
    L, r = kvq.lib(), ctypes.byref
    cfg, cache = kvq.make_paged_config(8, 2, 128, 4, 32, 10), kvq._PagedCache(0x1000, 0x1000)
    batch = kvq._PagedBatch(0x1000, 0x1000, 0x1000, 4, 16, 3, 8)
    base = dict(q=0x2000, stride=1024, out=0x3000000, scale=0.1, ws=0x4000, n=1 << 40)
    for kw in (dict(), dict(q=None), dict(q=0x2002), dict(stride=1000), dict(out=0x2000),
               dict(out=None), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None),
               dict(ws=0x4008), dict(n=8)):
        a = {**base, **kw}
        if not kw:
            continue
        args = (r(cfg), r(cache), r(batch), a["q"], a["stride"], a["out"], a["scale"], a["ws"],
                a["n"], None)
        code = L.kvq_paged_cross_attention(*args)
        assert code != E.KVQ_OK and code == L.kvq_paged_attention(*args), kw


def _drafts(**kw):
    d = kvq._DraftBatch(0x1000, 0x1000, 0x1000, 10, 3, 100, kvq.F32)
    for k, x in kw.items():
        setattr(d, k, x)
    return d


VERIFY = dict(logits=0x2000, stride=100, draft=0x2000, dstride=100, temperature=0x2000,
              uniform=0x2000, noise=0x2000, nstride=100, out=0x3000, accepted=0x3000,
              dropped=0x3000, logprobs=0x3000, ws=0x4000, ws_bytes=1 << 40)


def _verify(d, **kw):
    return kvq.lib().kvq_verify_drafts(ctypes.byref(d), *{**VERIFY, **kw}.values(), None)


def test_verify_refusals():
    for kw in (dict(cu_tokens=None), dict(tokens=None), dict(dev_status=None), dict(n_seqs=0),
               dict(vocab=0), dict(n_tokens=-1), dict(dtype=3)):
        assert _verify(_drafts(**kw)) == E.KVQ_EINVAL, kw
    for kw in (dict(n_seqs=2049), dict(n_tokens=65536), dict(vocab=(1 << 24) + 1)):
        assert _verify(_drafts(**kw)) == E.KVQ_EUNSUPPORTED, kw
    for kw in (dict(cu_tokens=0x1002), dict(tokens=0x1001), dict(dev_status=0x1002)):
        assert _verify(_drafts(**kw)) == E.KVQ_EALIGN, kw
    for name in ("logits", "uniform", "noise", "out", "accepted", "dropped", "logprobs", "ws"):
        assert _verify(_drafts(), **{name: None}) == E.KVQ_EINVAL, name
    for name in ("logits", "draft", "temperature", "uniform", "noise", "out", "accepted",
                 "dropped", "logprobs", "ws"):
        assert _verify(_drafts(), **{name: VERIFY[name] + 2}) == E.KVQ_EALIGN, name
    for name in ("stride", "dstride", "nstride"):
        assert _verify(_drafts(), **{name: 99}) == E.KVQ_EINVAL, name
    for at in (0x1000, 0x1000 + 36, 0x1000 - 36):    # outputs on the drafts
        assert _verify(_drafts(), out=at) == E.KVQ_EINVAL
    assert _verify(_drafts(dtype=kvq.BF16), logits=0x2001) == E.KVQ_EALIGN
    n = ctypes.c_size_t()
    bytes_of = lambda d: kvq.lib().kvq_verify_workspace_bytes(ctypes.byref(d), ctypes.byref(n))  # noqa: E731
    assert bytes_of(_drafts()) == 0
    assert _verify(_drafts(), ws_bytes=n.value - 1) == E.KVQ_ECAPACITY
    for kw, code in ((dict(n_seqs=0), E.KVQ_EINVAL), (dict(dtype=9), E.KVQ_EINVAL),
                     (dict(n_tokens=1 << 20), E.KVQ_EUNSUPPORTED)):
        assert bytes_of(_drafts(**kw)) == code


def test_padded_verify_refuses_what_verify_refuses():
    fn = kvq.lib().kvq_verify_drafts_padded
    for kw in (dict(logits=None), dict(out=0x1000), dict(accepted=None), dict(stride=99),
               dict(noise=0x2002), dict(ws=0x4008), dict(ws_bytes=8), dict(uniform=None)):
        code = fn(ctypes.byref(_drafts()), *{**VERIFY, **kw}.values(), None)
        assert code != E.KVQ_OK and code == _verify(_drafts(), **kw), kw
    assert fn(None, *VERIFY.values(), None) == E.KVQ_EINVAL


def test_workspace_grows_with_each_size():
    """A verifier made for the largest sizes has room for every smaller call."""
    n = ctypes.c_size_t()
    last = {}
    for d, B, T, V in itertools.product((kvq.F16, kvq.F32), (1, 2048), (0, 1, 100),
                                        (1, 8191, 8192, 8193, 100000)):
        assert kvq.lib().kvq_verify_workspace_bytes(
            ctypes.byref(_drafts(n_seqs=B, n_tokens=T, vocab=V, dtype=d)), ctypes.byref(n)) == 0
        last[d, B, T, V] = n.value
    for (d, B, T, V), x in last.items():
        assert all(x <= y for (d2, B2, T2, V2), y in last.items()
                   if d2 == d and B2 >= B and T2 >= T and V2 >= V)


def test_binding_checks_tables():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    t = kvq.PageTable(10, 16, n_seqs=3, width=4, device="cpu")
    assert (t.block_table == -1).all() and t.block_table.shape == (3, 4)
    assert t.free_pages.shape == (1,)
    for bad in (i32(3), i32(5), i32(4, 1)):
        with pytest.raises(ValueError):
            t.reserve(bad)
    with pytest.raises(TypeError):
        t.reserve(i32(4).long())
    for fn in (t.drop, t.select):
        with pytest.raises(ValueError):
            fn(i32(4))
        with pytest.raises(ValueError):
            fn(i32(6)[::2])
        with pytest.raises(TypeError):
            fn(i32(3).float())
    with pytest.raises(ValueError):
        t.reserve(i32(4), out=(i32(2, 2), i32(4)))
    with pytest.raises(ValueError):
        t.compact(out=i32(4, 2))
    for kw in (dict(), dict(n_seqs=3), dict(block_table=i32(3, 4)),
               dict(block_table=i32(3, 4), seq_lens=i32(2)),
               dict(block_table=i32(4, 3).t(), seq_lens=i32(3)),
               dict(block_table=i32(3, 4), seq_lens=i32(3), width=5)):
        with pytest.raises(ValueError):
            kvq.PageTable(10, 16, **kw)
    with pytest.raises(kvq.KVQError):
        kvq.PageTable(10, 24, n_seqs=3, width=4, device="cpu")
    cache = kvq.PagedKVCache(kvq.make_paged_config(2, 2, 64, 4, 16, 10), "cpu")
    for bad in (i32(4), i32(4, 3), i32(2, 4).t()):
        with pytest.raises(ValueError):
            cache.copy_pages(bad)
    with pytest.raises(TypeError):
        cache.copy_pages(i32(4, 2).long())


def test_binding_checks_verifier():
    v = kvq.DraftVerifier(2, 6, 50, torch.float16, "cpu")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f32, f16 = (lambda *s: torch.zeros(*s)), (lambda *s: torch.zeros(*s, dtype=torch.float16))
    good = dict(logits=f16(6, 50), tokens=i32(6), cu_tokens=i32(3), draft_logits=f16(6, 50),
                temperature=f32(2), uniform=f32(6), noise=f32(2, 50))
    for name, bad in (("logits", f16(6, 51)), ("logits", f16(5, 50)), ("logits", f16(50, 6).t()),
                      ("logits", f32(6, 50)), ("tokens", i32(7)), ("tokens", i32(6, 1)),
                      ("cu_tokens", i32(4)), ("cu_tokens", i32(1)), ("draft_logits", f16(6, 49)),
                      ("draft_logits", f32(6, 50)), ("temperature", f32(3)),
                      ("temperature", f16(2)), ("uniform", f32(5)), ("uniform", None),
                      ("noise", f32(2, 49)), ("noise", f16(2, 50)), ("noise", None)):
        with pytest.raises((ValueError, TypeError)):
            v.verify(**{**good, name: bad})
    assert v._rows(f16(6, 90)[:, 3:53], 6, torch.float16) == 90
    assert v._rows(f16(1, 90)[:, 3:53], 1, torch.float16) == 50
    with pytest.raises(TypeError):
        kvq.DraftVerifier(2, 6, 50, torch.float64, "cpu")
    with pytest.raises(kvq.KVQError):
        kvq.DraftVerifier(2, 1 << 20, 50, torch.float16, "cpu")


def test_model_of_a_small_pool():
    """The tests' own model on an example worked by hand: pages of 16."""
    m = Model(6, 16, 3, 4)
    assert m.reserve([20, 0, 0]) == [] and m.rows[0] == [0, 1]
    m.select([0, 0, 0])                       # three sequences share pages 0 and 1
    assert list(m.refs) == [3, 3, 0, 0, 0, 0]
    # all write: the first keeps page 1, the others copy it
    assert m.reserve([1, 1, 1]) == [(1, 2), (1, 3)]
    assert m.rows == [[0, 1], [0, 2], [0, 3]] and m.lens == [21] * 3
    assert m.reserve([12, 40, 0]) is None and m.lens == [21] * 3
    m.drop([100, 5, 6])                       # ends; leaves 16; leaves 15
    assert m.rows == [[], [0], [0]] and m.lens == [0, 16, 15]
    assert m.reserve([0, 1, 1]) == [(0, 2)]   # writes into a page that 1 holds too
    assert m.rows == [[], [0, 1], [2]]
    m.drop([0, 1, 0])
    assert m.compact() == [(2, 1)] and m.rows == [[], [0], [1]]
