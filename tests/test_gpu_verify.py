"""Draft verification on the GPU against 64 bits (tests/verify_util.py)."""
import itertools
import random

import numpy as np
import pytest
import torch

from bit_kv_cache_14_gb300 import build_lib, kvq
from pages_util import both, cu_of, i32
from verify_util import call, check, expected

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
KINDS = ("model", "lookup", "greedy")


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    yield


def inputs(n, V, dtype, kind, seed=0, pad=0, noise=0.4):
    """Logits of n[b] rows per sequence, drafts drawn from the draft's distribution."""
    g = torch.Generator("cuda").manual_seed(seed)
    T, B = sum(n) + pad, len(n)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = 2.0 * r(T, V) + 5.0 * (torch.rand(T, V, generator=g, device="cuda") < 5.0 / V)
    y = (x + noise * r(T, V)).to(dtype)
    x = x.to(dtype)
    e = torch.empty(T, V, device="cuda").exponential_(generator=g)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
    temp = 0.5 + torch.rand(B, generator=g, device="cuda")
    t = torch.ones(T, device="cuda")
    t[:sum(n)] = temp[seq]
    pick = (torch.softmax((y if kind == "model" else x).float() / t[:, None], -1) / e).argmax(-1)
    if kind == "greedy":
        pick = torch.where(torch.rand(T, generator=g, device="cuda") < 0.8, x.argmax(-1), pick)
    tokens = torch.roll(pick, 1).to(torch.int32)
    a = dict(logits=x, tokens=tokens, cu=i32(cu_of(n)))
    if kind != "greedy":
        a.update(temperature=temp, uniform=torch.rand(T, generator=g, device="cuda"),
                 noise=torch.empty(B, V, device="cuda").exponential_(generator=g))
    if kind == "model":
        a["draft"] = y
    return a


def run_and_check(a, **kw):
    B, (T, V) = a["cu"].numel() - 1, a["logits"].shape
    v = kvq.DraftVerifier(B, T, V, a["logits"].dtype)
    got = call(v, **a)
    assert v.device_status() == 0
    check(got, expected(**a), a["cu"].tolist(), a["tokens"].cpu().numpy(), **kw)
    assert not v.ws[:2048 * 12].any()      # what has to be zero is zero again
    return v, got


@pytest.mark.parametrize("dtype", (F16, BF16, F32))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", (1, 2, 7, 100, 2047, 2049, 8191, 8193, 33333))
def test_against_64_bits(dtype, kind, V):
    """Odd vocabularies: rows at every alignment; no drafts, some, many."""
    run_and_check(inputs([5, 1, 0, 9, 2, 3], V, dtype, kind, seed=V), allow_close=0.4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,V", [([1], 50), ([3] * 300, 200), ([40, 1], 1000), ([2] * 2048, 20),
                                 ([0] * 9 + [4], 77), ([300], 64)])
def test_numbers_of_sequences_and_drafts(kind, n, V):
    run_and_check(inputs(n, V, BF16, kind, seed=len(n)), allow_close=0.4)


@pytest.mark.parametrize("kind", ("model", "lookup"))
def test_most_drafts_stay_or_none(kind):
    a = inputs([6] * 40, 500, F32, kind, seed=1, noise=0.02)
    a["uniform"] *= 0.01
    _, got = run_and_check(a)
    assert (got[1] == 5).any()      # (the 64-bit form says which)
    a["uniform"] = 1.0 - 2.0 ** -24 - 0.0 * a["uniform"]
    if kind == "model":
        a["draft"] = torch.roll(a["logits"], 7, 1).contiguous()
    run_and_check(a, allow_close=0.5)


def run_and_check_all(a):
    """No sequence of the case has a decision that is too near to call (the 64-bit form
    says so, for these seeds), so all of the call's outputs are compared."""
    assert not any(close for _, _, close in expected(**a))
    run_and_check(a, allow_close=0)


@pytest.mark.parametrize("dtype", (F16, BF16, F32))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", (1, 2, 7, 100, 2047, 2049, 8191, 8193, 33333))
def test_every_decision_against_64_bits(dtype, kind, V):
    run_and_check_all(inputs([5, 1, 0, 9, 2, 3], V, dtype, kind, seed=V))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,V", [([1], 50), ([3] * 300, 200), ([40, 1], 1000), ([2] * 2048, 20),
                                 ([0] * 9 + [4], 77), ([300], 64)])
def test_every_decision_of_many_sequences(kind, n, V):
    run_and_check_all(inputs(n, V, BF16, kind, seed=len(n)))


@pytest.mark.parametrize("kind", ("model", "lookup"))
def test_every_decision_where_drafts_stay_or_go(kind):
    a = inputs([6] * 40, 500, F32, kind, seed=1, noise=0.02)
    a["uniform"] *= 0.01
    run_and_check_all(a)
    a["uniform"] = 1.0 - 2.0 ** -24 - 0.0 * a["uniform"]
    if kind == "model":
        a["draft"] = torch.roll(a["logits"], 7, 1).contiguous()
    run_and_check_all(a)


def test_the_same_model_twice_keeps_everything():
    """q = p: every draft stays for any u < 1 (both sides are the same sums)."""
    a = inputs([9] * 30, 4097, BF16, "model", seed=2)
    a["draft"] = a["logits"].clone()
    a["uniform"].fill_(1.0 - 2.0 ** -24)
    v = kvq.DraftVerifier(30, 270, 4097, BF16)
    out, accepted, dropped, _ = call(v, **a)
    assert (accepted == 8).all() and (dropped == 0).all() and (out >= 0).all()


@pytest.mark.parametrize("dtype", (F16, BF16, F32))
@pytest.mark.parametrize("off,extra", [(0, 0), (1, 0), (3, 5), (8, 8), (7, 1)])
def test_rows_of_wider_tensors(dtype, off, extra):
    """Views into wider logits, draft logits and noise, each at an offset of its own."""
    a = inputs([4, 2, 7], 1003, dtype, "model", seed=off)
    for name, o in (("logits", off), ("draft", (off + 2) % 9), ("noise", (off * 3) % 5)):
        t = a[name]
        big = torch.full((t.shape[0], t.shape[1] + off + extra + 9), 3e4, dtype=t.dtype,
                         device="cuda")
        big[:, o:o + t.shape[1]] = t
        a[name] = big[:, o:o + t.shape[1]]
    run_and_check(a)


@pytest.mark.parametrize("dtype", (F16, BF16, F32))
@pytest.mark.parametrize("kind", KINDS)
def test_masks(dtype, kind):
    """Masked by -infinity, the type's lowest number and NaN: such tokens are never
    drawn, a draft of one is refused; infinities win; rows with nothing give -1."""
    V = 600
    a = inputs([4] * 24, V, dtype, kind, seed=5)
    x = a["logits"]
    g = torch.Generator("cuda").manual_seed(9)
    for r in range(0, 96, 2):
        keep = torch.rand(V, generator=g, device="cuda") < (0.02, 0.5)[r // 2 % 2]
        keep[r % V] = True
        low = (-float("inf"), torch.finfo(dtype).min, float("nan"))[r // 4 % 3]
        if dtype == F16 and low == torch.finfo(dtype).min:
            low = -float("inf")     # (fp16's lowest is a number like any other)
        x[r, ~keep] = low
    x[9, 17] = float("inf")
    x[40:48] = -float("inf")        # two sequences that see nothing
    x[52] = float("nan")
    x[60, 3] = x[60, 4] = float("inf")
    if kind == "model":
        a["draft"][20:24] = -float("inf")
        a["draft"][24, ::2] = float("nan")
    v, got = run_and_check(a, allow_close=0.4)
    assert (got[0][40] == -1) and (got[0][44] == -1) and int(got[1][10]) == 0


def test_lowest_fp16_number_is_a_logit():
    x = torch.full((2, 40), -65504.0, dtype=F16, device="cuda")
    v = kvq.DraftVerifier(2, 2, 40, F16)
    out, _, _, lp = v.verify(x, i32([0, 0]), i32([0, 1, 2]))
    assert out.tolist() == [0, 0] and (lp + np.log(40)).abs().max() < 1e-5


def test_temperatures():
    """Sequences of their own, greedy ones among them; very high and very low."""
    temps = [0.7, 0.0, 1.0, -1.0, float("nan"), 50.0, 0.01, 1e4, 0.0, 1e-3, 2.0, float("inf")]
    a = inputs([3] * 12, 900, F32, "model", seed=3)
    a["temperature"] = torch.tensor(temps, device="cuda")
    # where 64 bits and the call agree on what the temperature is
    want = dict(a, temperature=torch.tensor(
        [2.0 ** 100 if t == float("inf") else t for t in temps], device="cuda").double())
    v = kvq.DraftVerifier(12, 36, 900, F32)
    got = call(v, **a)
    check(got, expected(**want), a["cu"].tolist(), a["tokens"].cpu().numpy(), allow_close=0.5)
    # greedy sequences need no numbers
    a["uniform"][3:6] = float("nan")
    a["noise"][1] = float("nan")
    again = call(v, **a)
    for x, y in zip(got, again):
        assert torch.equal(x[1], y[1])
    assert torch.equal(got[0][3:6], again[0][3:6])


def test_numbers_at_their_ends():
    """u of 0 keeps every draft with a probability; e of 0 and denormal draws its
    token, NaN and infinity never."""
    a = inputs([3] * 20, 300, F32, "model", seed=8)
    a["uniform"].zero_()
    a["noise"][0, 5] = 0.0
    a["noise"][1, 7] = 1e-42
    a["noise"][2, 9] = float("nan")
    a["noise"][3, :] = float("nan")
    a["noise"][4, :] = float("inf")
    _, got = run_and_check(a)
    assert (got[1] == 2).all()
    assert got[0][2] == 5 and got[0][5] == 7 and got[0][11] == -1 and got[0][14] == -1


def test_what_is_left_may_be_nothing():
    """p - q <= 0 everywhere at a refused draft (u of 1 is outside the numbers that
    are given, and refuses what is equal): p itself is drawn from."""
    a = inputs([2] * 10, 64, F32, "model", seed=4)
    a["draft"] = a["logits"].clone()
    a["uniform"].fill_(1.0)
    v = kvq.DraftVerifier(10, 20, 64, F32)
    out, accepted, _, _ = call(v, **a)
    assert (accepted == 0).all()
    p = torch.softmax(a["logits"].double() / a["temperature"].repeat_interleave(2)[:, None], -1)
    assert torch.equal(out[::2], (p[::2] / a["noise"]).argmax(-1).int())


def test_drafts_that_are_no_tokens():
    for bad in (-1, 50, 2 ** 31 - 1, -2 ** 31):
        for kind in KINDS:
            a = inputs([4, 4], 50, BF16, kind, seed=6)
            a["tokens"][2] = bad
            v = kvq.DraftVerifier(2, 8, 50, BF16)
            got = call(v, **a)
            assert v.device_status() == kvq.KVQ_EINVAL
            check(got, expected(**a), [0, 4, 8], a["tokens"].cpu().numpy(), allow_close=0.5)
            assert int(got[1][0]) <= 1


def test_rows_out_of_order():
    """Rows that overlap or lie outside are nobody's: no sequence is judged."""
    for cu in ([0, 5, 3, 9], [0, -1, 4, 9], [0, 4, 9, 13], [3, 1, 4, 9], [-1, 4, 8, 12]):
        for kind in ("model", "greedy"):
            a = inputs([4, 4, 4], 70, F16, kind, seed=7)
            a["cu"] = i32(cu)
            v = kvq.DraftVerifier(3, 12, 70, F16)
            got = call(v, **a)
            assert v.device_status() == kvq.KVQ_EINVAL
            assert not got[1].any() and not got[2].any()
    # many sequences, one border out of order
    n = [2] * 300
    b = inputs(n, 40, BF16, "greedy", seed=1)
    b["cu"][150] = 10
    many = kvq.DraftVerifier(300, 600, 40, BF16)
    got = call(many, **b)
    assert many.device_status() == kvq.KVQ_EINVAL and not got[1].any()
    # what follows is not disturbed
    a = inputs([4, 4, 4], 70, F16, "model", seed=7)
    a["cu"] = i32([0, 4, 8, 12])
    got = call(v, **a)
    check(got, expected(**a), [0, 4, 8, 12], a["tokens"].cpu().numpy(), allow_close=0.5)


def test_padding_rows_are_left_alone():
    a = inputs([3, 2], 90, BF16, "model", seed=2, pad=4)
    v = kvq.DraftVerifier(2, 9, 90, BF16)
    import ctypes
    view = kvq._DraftBatch(a["cu"].data_ptr(), a["tokens"].data_ptr(), v.status.data_ptr(), 9, 2,
                           90, kvq.BF16)
    out, lp = i32([77] * 9), torch.full((9,), 5.0, device="cuda")
    acc, drop = i32([0, 0]), i32([0, 0])
    code = kvq.lib().kvq_verify_drafts(
        ctypes.byref(view), a["logits"].data_ptr(), 90, a["draft"].data_ptr(), 90,
        a["temperature"].data_ptr(), a["uniform"].data_ptr(), a["noise"].data_ptr(), 90,
        out.data_ptr(), acc.data_ptr(), drop.data_ptr(), lp.data_ptr(), v.ws.data_ptr(),
        v.ws_bytes, torch.cuda.current_stream().cuda_stream)
    assert code == 0 and (out[5:] == 77).all() and (lp[5:] == 5).all()
    check((out, acc, drop, lp), expected(**a), [0, 3, 5], a["tokens"].cpu().numpy(),
          allow_close=0.5)


@pytest.mark.parametrize("kind", ("model", "lookup"))
@pytest.mark.parametrize("V,most", [(50, 60), (5000, 60), (70001, 60), (700, 170)])
def test_stated_arithmetic(kind, V, most):
    """Drafts far below their rows' likeliest tokens, fp32: a number off p / q by the
    stated bounds of p and of q (and its own rounding) is decided as the exact one.

    A weight 2^-t: x - max and the product with log2(e) / T are rounded once each, so
    its exponent is off by t 2^-23, itself by 0.7 of that, and the exponential by 2^-22
    (2 units of 2^-23).  The sum's terms have those errors, 0.7 times their mean t, which
    is below log2 V, and 2; a lane adds 4 * 32 pairs to a running sum whose reference
    moves at most 4 times (16 + 10 units at most: roundings of half a unit, moves of 2 and
    a half), five steps join the lanes (5), and a lane joins 1 / 32 of the at most
    V / 1024 parts (2.5 units each: V / 2^13): 64 units cover the constants."""
    B = 256
    rng = np.random.default_rng(V)
    x, y = (2.0 * rng.standard_normal((B, V)) for _ in range(2))
    T = (0.5 + rng.random(B)).astype(np.float32)
    c = rng.integers(0, V, B)
    rows = np.arange(B)
    x[rows, c] = y[rows, c] = -1e4
    tp = rng.uniform(20, most, B)
    tq = rng.uniform(0, tp - 18)
    unit = T.astype(np.float64) * np.log(2)
    x[rows, c] = x.max(1) - tp * unit
    y[rows, c] = y.max(1) - tq * unit
    x, y = x.astype(np.float32), y.astype(np.float32)

    def exact(z):
        t = (z.astype(np.float64) - z.max(1, keepdims=True)) / T[:, None].astype(np.float64)
        e = np.exp(t)
        return t[rows, c] - np.log(e.sum(1)), -t[rows, c] / np.log(2)

    lp, ep = exact(x)
    lq, eq = exact(y) if kind == "model" else (0.0, -64 - V / 2 ** 13)
    bound = (ep + eq + 2 * (64 + V / 2 ** 13)) * 2.0 ** -23 + 2.0 ** -24
    odds = np.exp(lp - lq)
    # (a number below 2^-126 has fewer bits)
    ok = (odds < 0.9) & (odds > 2.0 ** -120)
    assert ok.sum() > B // 3
    up = lambda a: np.repeat(a, 2, 0)  # noqa: E731
    v = kvq.DraftVerifier(B, 2 * B, V, F32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    noise = torch.ones(1, V, device="cuda").expand(B, V).contiguous()
    for side, stays in ((1 - bound, 1), (1 + bound, 0)):
        u = up((odds * side).astype(np.float32))
        tokens = np.stack([0 * c, c], 1).reshape(-1).astype(np.int32)
        _, accepted, _, _ = v.verify(
            dev(up(x)), dev(tokens), i32(2 * np.arange(B + 1)),
            dev(up(y)) if kind == "model" else None, dev(T), dev(u), noise)
        assert (accepted.cpu().numpy()[ok] == stays).all()
    assert v.device_status() == 0


def used_memory(T):
    """Memory that the next outputs are likely to get, as a step before left it."""
    held = [torch.full((T,), 7, dtype=torch.int32, device="cuda") for _ in range(12)]
    del held


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,pad", [([3, 2], 4), ([1, 0, 4], 3000), ([0, 0], 9)])
def test_rows_that_nobody_has(kind, n, pad):
    """Padding, rows before the first sequence's, all rows where no pages were reserved
    or cu_tokens is out of order: -1 and 0 from the binding."""
    a = inputs(n, 90, BF16, kind, seed=2, pad=pad)
    T, real = sum(n) + pad, cu_of(n)
    v = kvq.DraftVerifier(len(n), T, 90, BF16)
    used_memory(T)
    got = call(v, **a)
    assert v.device_status() == 0
    check(got, expected(**a), real.tolist(), a["tokens"].cpu().numpy(), allow_close=0.5)
    assert (got[0][sum(n):] == -1).all() and (got[3][sum(n):] == 0).all()
    late = dict(a, cu=i32(real + 2))
    used_memory(T)
    got = call(v, **late)
    assert v.device_status() == 0
    assert (got[0][:2] == -1).all() and (got[3][:2] == 0).all()
    assert (got[0][sum(n) + 2:] == -1).all() and (got[3][sum(n) + 2:] == 0).all()
    for cu, status in ((0 * real, 0), (real[::-1].copy(), kvq.KVQ_EINVAL if sum(n) else 0),
                       (real - 1, kvq.KVQ_EINVAL), (real + pad + 1, kvq.KVQ_EINVAL)):
        used_memory(T)
        got = call(v, **dict(a, cu=i32(cu)))
        assert v.device_status() == status
        assert (got[0] == -1).all() and not got[3].any() and not got[1].any() and not got[2].any()


def test_a_captured_step_without_pages():
    """A captured speculative step, replayed until the pool is used up and on: a step
    that gets no pages gives no tokens and takes none back, and once a sequence has
    ended the steps go on."""
    page, H, d, B, V, n = 16, 1, 64, 3, 200, [4, 4, 4]
    T = sum(n)
    g = torch.Generator("cuda").manual_seed(0)
    m, tab = both(7, page, B, 8)
    cache = kvq.PagedKVCache(kvq.make_paged_config(H, H, d, 8, page, 7))
    cache.pages.zero_()
    a = inputs(n, V, F16, "model", seed=3)
    ver = kvq.DraftVerifier(B, T, V, F16)
    k = torch.randn(T, H, d, generator=g, device="cuda").half()
    bufs = torch.empty(B, 2, dtype=torch.int32, device="cuda"), i32([0] * (B + 1))

    def step():
        copies, cu = tab.reserve(a["cu"], out=bufs)
        cache.copy_pages(copies)
        batch = tab.batch(cu, T, 4)
        cache.write(k, k, batch)
        x = cache.attend(k, batch)
        res = ver.verify(a["logits"], a["tokens"], cu, a["draft"], a["temperature"],
                         a["uniform"], a["noise"])
        tab.drop(res[2])
        return (x,) + res

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        tab.drop(i32([99] * B))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, tokens, kept, dropped, logs = step()
    want = expected(**a)
    failed = 0
    for i in range(40):
        graph.replay()
        if m.reserve(n) is None:
            failed += 1
            assert tab.device_status() == kvq.KVQ_ECAPACITY
            assert (tokens == -1).all() and not logs.any()
            assert not kept.any() and not dropped.any()
            m.check(tab)
            if failed % 3 == 0:
                m.drop([0, 99, 0])
                tab.drop(i32([0, 99, 0]))
        else:
            assert tab.device_status() == 0
            check((tokens, kept, dropped, logs), want, cu_of(n).tolist(),
                  a["tokens"].cpu().numpy(), allow_close=0.5)
            m.drop(dropped.tolist())
        m.check(tab)
    assert failed >= 3 and cache.device_status() == ver.device_status() == 0


def test_no_rows_at_all():
    v = kvq.DraftVerifier(3, 4, 50, F16)
    empty = torch.zeros(0, 50, dtype=F16, device="cuda")
    out, accepted, dropped, lp = v.verify(empty, i32([]), i32([0] * 4))
    assert out.numel() == 0 and not accepted.any() and not dropped.any()
    assert v.device_status() == 0


def test_one_verifier_for_many_sizes():
    """Scratch made for the largest sizes serves calls of any smaller ones, and the
    same call gives the same bits."""
    v = kvq.DraftVerifier(64, 300, 5000, BF16)
    rng = random.Random(4)
    for i in range(12):
        n = [rng.randint(0, 5) for _ in range(rng.randint(1, 60))]
        a = inputs(n, 5000, BF16, rng.choice(KINDS), seed=i, pad=1)
        got = call(v, **a)
        check(got, expected(**a), cu_of(n).tolist(), a["tokens"].cpu().numpy())
        for x, y in zip(got, call(v, **a)):
            assert torch.equal(x[:sum(n)], y[:sum(n)])
    assert v.device_status() == 0


def test_captured_and_on_other_streams():
    a = inputs([4] * 6, 3000, F16, "model", seed=1)
    v = kvq.DraftVerifier(6, 24, 3000, F16)
    want = call(v, **a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(v, **a, stream=side)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    with torch.cuda.stream(side):
        call(v, **a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(v, **a)
    for seed in range(5):
        b = inputs([4] * 6, 3000, F16, "model", seed=seed)
        for k in a:
            a[k].copy_(b[k])
        graph.replay()
        check(got, expected(**a), a["cu"].tolist(), a["tokens"].cpu().numpy())


def test_large_vocabulary_and_offsets_beyond_32_bits():
    """Rows that lie more than 2^32 bytes into a wide tensor."""
    V, B = 131071, 3
    a = inputs([3] * B, V, BF16, "model", seed=11)
    big = torch.empty(9, 1 << 28, dtype=BF16, device="cuda")   # 512 MB a row
    big[:, 5:5 + V] = a["logits"]
    a["logits"] = big[:, 5:5 + V]
    run_and_check(a)


def test_a_speculative_step_together():
    """A decoder's step from end to end, captured: pages for the new rows, copies,
    write, causal and cross attention, verification, and the refused rows' pages
    back; then the same without a graph."""
    page, H, rg, d, B, V = 16, 2, 2, 64, 5, 700
    n = [4, 1, 3, 0, 5]
    T = sum(n)
    g = torch.Generator("cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").half()  # noqa: E731
    cfg = kvq.make_paged_config(H * rg, H, d, 8, page, 60)
    enc_cfg = kvq.make_paged_config(H * rg, H, d, 4, page, 12)
    enc = kvq.PagedKVCache(enc_cfg)
    enc_tab = kvq.PageTable(12, page, n_seqs=B, width=4)
    _, ecu = enc_tab.reserve(i32(cu_of([20, 33, 1, 0, 40])))
    enc.write(r(94, H, d), r(94, H, d), enc_tab.batch(ecu, 94))
    ks, vs, qs, hs = r(T, H, d), r(T, H, d), r(T, H * rg, d), r(H * rg * d, V) * 0.2
    a = inputs(n, V, F16, "model", seed=0)
    uniform, noise, temp, draft, tokens = (a[k] for k in ("uniform", "noise", "temperature",
                                                          "draft", "tokens"))
    cu_in = i32(cu_of(n))

    def build():
        tab = kvq.PageTable(60, page, n_seqs=B, width=8)
        cache = kvq.PagedKVCache(cfg)
        cache.pages.zero_()
        _, cu = tab.reserve(i32(cu_of([30, 2, 0, 0, 47])))
        gg = torch.Generator("cuda").manual_seed(1)
        kk = torch.randn(79, H, d, generator=gg, device="cuda").half()
        cache.write(kk, kk, tab.batch(cu, 79))
        tab.select(i32([0, 1, 0, 4, 4]))
        return tab, cache, kvq.DraftVerifier(B, T, V, F16)

    def step(tab, cache, ver, out):
        copies, cu = tab.reserve(cu_in, out=out)
        cache.copy_pages(copies)
        batch = tab.batch(cu, T, 5)
        cache.write(ks, vs, batch)
        x = cache.attend(qs, batch)
        x = x + enc.cross_attend(x, kvq.PagedBatch(enc_tab.block_table, enc_tab.seq_lens, cu, T))
        logits = x.flatten(1) @ hs
        res = ver.verify(logits, tokens, cu, draft, temp, uniform, noise)
        tab.drop(res[2])
        return (logits,) + res

    bufs = lambda: (torch.empty(B, 2, dtype=torch.int32, device="cuda"), i32([0] * (B + 1)))  # noqa: E731
    eager, captured = build(), build()
    out = bufs()
    torch.cuda.synchronize()
    warm = build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*warm, bufs())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*captured, out)
    held = eager[0].seq_lens.tolist()
    for i in range(6):
        want = step(*eager, bufs())
        graph.replay()
        for x, y in zip(want, got):
            assert torch.equal(x, y), i
        assert torch.equal(eager[0].block_table, captured[0].block_table)
        assert torch.equal(eager[0].page_refs, captured[0].page_refs)
        check(want[1:], expected(want[0], tokens, cu_in, draft, temp, uniform, noise),
              cu_of(n).tolist(), tokens.cpu().numpy(), allow_close=0.5)
        held = [h + 1 + int(k) if m else h for h, k, m in zip(held, want[2].tolist(), n)]
        assert eager[0].seq_lens.tolist() == held
    for tab, cache, ver in (eager, captured):
        assert tab.device_status() == cache.device_status() == ver.device_status() == 0
