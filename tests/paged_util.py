"""Plain reference of the paged cache for the tests: the packed layout and the
stored form straight from include/kvq.h, attention in 64 bits, and the
tolerance of the attention output.

Stored bytes and values read back are compared bit for bit: the stored form is
defined operation by operation in fp32 with every rounding to nearest even.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

from bit_kv_cache_14_gb300 import kvq

GROUP, ATOM, LIMIT = 32, 16, 32768.0


def slot_of(which, c, d, b):
    """Slot (in units of b bits) of channel c in a row of codes."""
    G, r = divmod(c, 32)
    if which == "k":
        j, k, e = r // 8, (r % 8) // 2, r % 2
        p = 4 * G + k
        bit = j * (d * b // 4) + (p * b // 16) * 32 + (p * b) % 16 + 16 * e
    else:
        h, e, g, i = G // 2, G % 2, r // 4, r % 4
        p, w = 4 * h + i, 8 if (d == 64 and b == 2) else 16
        bit = g * (d * b // 8) + (p * b // w) * 2 * w + (p * b) % w + w * e
    assert bit % b == 0
    return bit // b


def quantize(x, bits):
    """fp32 numpy [..., d] -> codes uint8 [..., d], scale and zero fp16 [..., d/32]."""
    x = np.where(np.isnan(x), np.float32(0), x.astype(np.float32))
    x = np.clip(x, np.float32(-LIMIT), np.float32(LIMIT))
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    mn, mx = g.min(-1), g.max(-1)
    scale = ((mx - mn) / np.float32(2 ** bits - 1)).astype(np.float16)
    zero = (mn + np.float32(0)).astype(np.float16)
    s, z = scale.astype(np.float32)[..., None], zero.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.rint((g - z) / s), np.float32(0))
    c = np.clip(c, 0, 2 ** bits - 1).astype(np.uint8)
    return c.reshape(x.shape), scale, zero


def values(codes, scale, zero):
    """Stored values in fp32: code * scale + zero."""
    c = codes.astype(np.float32).reshape(codes.shape[:-1] + (codes.shape[-1] // GROUP, GROUP))
    x = c * scale.astype(np.float32)[..., None] + zero.astype(np.float32)[..., None]
    return x.astype(np.float32).reshape(codes.shape)


def pack_row(which, codes, bits):
    """codes [..., d] -> packed bytes [..., d*bits/8]."""
    d = codes.shape[-1]
    per = 8 // bits
    out = np.zeros(codes.shape[:-1] + (d // per,), np.uint8)
    for c in range(d):
        s = slot_of(which, c, d, bits)
        out[..., s // per] |= (codes[..., c] << ((s % per) * bits)).astype(np.uint8)
    return out


class Case:
    """A pool with sequences of given lengths whose last `new` tokens are a
    call's rows; pages in random order, `shared` leading pages common to all."""

    def __init__(self, kv, new, hq, hkv, d, bits, page, dtype, seed=0, pad=0, spare=2):
        self.kv, self.new, self.hq, self.hkv, self.d = list(kv), list(new), hq, hkv, d
        self.bits, self.page, self.dtype, self.seed = bits, page, dtype, seed
        rng = np.random.default_rng(seed)
        need = [-(-max(k, 0) // page) for k in self.kv]
        self.width = max(need + [1])
        self.n_pages = sum(need) + spare
        ids = rng.permutation(self.n_pages)
        # entries behind a sequence's pages are never read: any value
        self.table = rng.integers(-5, 1 << 30, (len(self.kv), self.width)).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.n_tokens = int(self.cu[-1]) + pad
        self.rng = rng
        # raw rows of every token of every sequence, 16-bit values kept as fp32
        self.K, self.V = [], []
        ks = np.exp(0.3 * rng.standard_normal((hkv, d))).astype(np.float32)
        ks[rng.random((hkv, d)) < 0.03] *= 8
        for k in self.kv:
            shape = (max(k, 0), hkv, d)
            self.K.append(self._round(rng.standard_normal(shape).astype(np.float32) * ks))
            self.V.append(self._round(rng.standard_normal(shape).astype(np.float32)))
        self.q = self._round(1.2 * rng.standard_normal((self.n_tokens, hq, d)).astype(np.float32))

    def _round(self, x):
        return torch.from_numpy(x).to(self.dtype).float().numpy()

    @property
    def rows(self):
        """(b, position) of every real row."""
        return [(b, self.kv[b] - n + i) for b, n in enumerate(self.new) for i in range(n)]

    # ---- device side ------------------------------------------------------
    def config(self):
        return kvq.make_paged_config(self.hq, self.hkv, self.d, self.bits, self.page,
                                     self.n_pages, self.dtype)

    def batch(self, new=None, kv=None, n_tokens=None, max_tokens=None, device="cuda"):
        new = self.new if new is None else new
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(cu[-1]) if n_tokens is None else n_tokens
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
        return kvq.PagedBatch(t(self.table),
                              t(np.array(self.kv if kv is None else kv, np.int32)), t(cu), n,
                              max(list(new) + [0]) if max_tokens is None else max_tokens)

    def packed(self, which, device="cuda", whole=False):
        """The call's rows (or all tokens of all sequences) as one tensor."""
        src = self.K if which == "k" else self.V
        parts = [x if whole else x[len(x) - min(n, len(x)):] for x, n in zip(src, self.new)]
        return torch.from_numpy(np.concatenate(parts)).to(device=device, dtype=self.dtype)

    def filled(self, device="cuda"):
        """A cache that holds every token, written in one call."""
        cache = kvq.PagedKVCache(self.config(), device)
        cache.pages.fill_(0xFF)  # never-written slots: statistics are NaN
        cache.write(self.packed("k", device, True), self.packed("v", device, True),
                    self.batch(new=[max(k, 0) for k in self.kv], device=device))
        return cache

    def queries(self, device="cuda"):
        return torch.from_numpy(self.q).to(device=device, dtype=self.dtype)

    # ---- expected ---------------------------------------------------------
    def expected_rows(self, which, tokens):
        """Values read back, in the case's type, as a torch tensor."""
        src = self.K if which == "k" else self.V
        x = np.stack([src[b][t] for b, t in tokens]) if tokens else np.zeros((0, self.hkv, self.d))
        return torch.from_numpy(values(*quantize(x.astype(np.float32), self.bits))).to(self.dtype)

    def pool_view(self, pages):
        """numpy views of a pool: K codes, V codes, K stats, V stats as
        [page][head][atom][16][bytes]."""
        d, b = self.d, self.bits
        rb, sb = d * b // 8, 4 * d // GROUP
        at = pages.cpu().numpy().reshape(self.n_pages, self.hkv, self.page // ATOM, -1)
        cut = np.cumsum([0, ATOM * rb, ATOM * rb, ATOM * sb, ATOM * sb])
        return [at[..., x:y].reshape(at.shape[:3] + (ATOM, -1)) for x, y in zip(cut, cut[1:])]

    def attention(self, scale=None):
        """(out, bound) in 64 bits for every real row: [rows][hq][d].

        The bound counts what a 16-bit tensor-core form rounds, u = 2^-11 (half
        a step of fp16): the key operand (scores move by at most u * sum|q k|
        times the scale, plus as much again for fp32 accumulation and a query
        carried in fp16), the weight and the value operand (u each, relative to
        code * scale or zero, whose magnitudes are at most |v| + 2 |zero|), 2^-24
        per added token for the fp32 sums and for weights below fp16's normal
        range, and the output's own rounding.  A score error e moves the
        weights by at most a factor exp(2 e)."""
        rg = self.hq // self.hkv
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        u = 2.0 ** -11
        half_step = torch.finfo(self.dtype).eps / 2
        outs, bounds = [], []
        at = 0
        for b, n in enumerate(self.new):
            kv = max(self.kv[b], 0)
            kc = quantize(self.K[b], self.bits)
            vc = quantize(self.V[b], self.bits)
            K, V = values(*kc).astype(np.float64), values(*vc).astype(np.float64)
            Z = np.repeat(np.abs(vc[2].astype(np.float64)), GROUP, -1)
            KZ = np.abs(K) + 2 * np.repeat(np.abs(kc[2].astype(np.float64)), GROUP, -1)
            for i in range(n):
                pos = self.kv[b] - n + i
                o = np.zeros((self.hq, self.d))
                e = np.zeros((self.hq, self.d))
                if pos >= 0:
                    for h in range(self.hq):
                        q = self.q[at].astype(np.float64)[h]
                        s = scale * (K[:pos + 1, h // rg] @ q)
                        A = abs(scale) * (KZ[:pos + 1, h // rg] @ np.abs(q))
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        m = np.abs(V[:pos + 1, h // rg]) + 2 * Z[:pos + 1, h // rg]
                        o[h] = w @ V[:pos + 1, h // rg]
                        ds = 2 * (2 * u * A[w > 1e-12].max())
                        e[h] = ((w @ m) * (2 * u + math.expm1(ds) + (pos + 1) * 2.0 ** -24)
                                + (pos + 1) * 2.0 ** -24 * m.max(0))
                outs.append(o)
                bounds.append(e + half_step * (np.abs(o) + e) + 1e-7)
                at += 1
        shape = (0, self.hq, self.d)
        return (np.stack(outs) if outs else np.zeros(shape),
                np.stack(bounds) if bounds else np.zeros(shape))

    def check_attention(self, out, scale=None):
        exp, bound = self.attention(scale)
        got = out[:len(exp)].double().cpu().numpy()
        assert np.isfinite(got).all()
        err = np.abs(got - exp)
        worst = np.unravel_index(np.argmax(err / bound), err.shape) if err.size else None
        assert (err <= bound).all(), "error %g > bound %g at %s" % (err[worst], bound[worst], worst)


def random_case(seed):
    rng = random.Random(seed)
    hkv = rng.choice([1, 2, 3])
    rg = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 20])
    B = rng.randint(1, 5)
    kv = [rng.choice([0, 1, 15, 16, 17, 33, 127, 128, 129, 300]) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 2, min(k, 40), k, min(k, 130)]) for k in kv]
    return Case(kv, new, hkv * rg, hkv, rng.choice([64, 128]), rng.choice([2, 4, 8]),
                rng.choice([16, 32, 64, 128, 256]), rng.choice([torch.float16, torch.bfloat16]),
                seed=seed, pad=rng.choice([0, 3]))
