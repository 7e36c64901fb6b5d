"""Cases of the paged-cache operators: what they are timed on, and their plain forms.

The operators (include/kvq.h, "Paged cache"):
  store   new keys and values are quantised into the pages of a paged cache
          (kvq_paged_write) and read back as the values they now stand for
          (kvq_paged_read);
  read    a stretch of every sequence's tokens is gathered from its pages and
          dequantised into packed 16-bit rows (kvq_paged_read);
  attend  new tokens -- one per sequence, a chunk of them, or a batch that
          mixes both -- attend causally to all tokens their sequence holds in
          the pages (kvq_paged_attention).

The plain forms are elementary torch operations in 32 bits on the same packed
pages.  `exact` states the operators once more in 64 bits.
"""
import math
import random

import torch

own = False  # True: run() calls the library's kernels instead of the plain forms

GROUP = 32   # channels that share a scale and a zero point
ATOM = 16    # tokens stored together inside a page
LIMIT = 32768.0  # stored magnitudes saturate here


# --------------------------------------------------------------------------
# cases

def _case(name, op, batch, ctx, new, hq, hkv, d, bits, page, dtype, ragged=False, decodes=0):
    return dict(name=name, op=op, batch=batch, ctx=ctx, new=new, hq=hq, hkv=hkv, d=d, bits=bits,
                page=page, dtype=dtype, ragged=ragged, decodes=decodes)


def listed():
    return [
        # one decode step's keys and values of a small batch entering the cache
        _case("store_step_b16", "store", 16, 900, 1, 32, 8, 128, 4, 16, "bf16", ragged=True),
        # prompts of uneven lengths entering a 2-bit cache
        _case("store_chunks_2bit", "store", 6, 1500, 700, 32, 32, 128, 2, 32, "fp16", ragged=True),
        # long prompts entering a 4-bit cache
        _case("store_prompts_4bit", "store", 8, 4096, 4096, 32, 8, 128, 4, 64, "bf16"),
        # one short sequence copied out of a 2-bit cache of small heads
        _case("read_short_d64", "read", 1, 777, 777, 8, 8, 64, 2, 16, "fp16"),
        # whole sequences copied out, to be edited or moved elsewhere
        _case("read_long_8bit", "read", 16, 4100, 4100, 32, 8, 128, 8, 64, "bf16", ragged=True),
        # decode step of a few short conversations: latency
        _case("decode_short_b4", "attend", 4, 301, 1, 32, 8, 128, 4, 16, "bf16", ragged=True),
        # decode step of the Llama-2-7B-shaped layer, 2-bit, every head its own keys
        _case("decode_mha_2bit", "attend", 8, 4096, 1, 32, 32, 128, 2, 64, "fp16"),
        # decode step of a large batch of long grouped-query conversations
        _case("decode_gqa_b64", "attend", 64, 16384, 1, 32, 8, 128, 4, 64, "bf16", ragged=True),
        # a short question on top of a cached prefix, small heads
        _case("chunk_small_d64", "attend", 2, 1999, 77, 8, 2, 64, 8, 16, "fp16", ragged=True),
        # chunked prefill of a few sequences
        _case("chunk_b4_512", "attend", 4, 8192, 512, 32, 8, 128, 4, 32, "bf16"),
        # one chunk of a long document
        _case("chunk_long_4096", "attend", 1, 32768, 4096, 32, 8, 128, 4, 64, "bf16"),
        # a serving step that mixes a prefill chunk with decoding sequences
        _case("mixed_step_b16", "attend", 16, 4000, 256, 32, 8, 128, 4, 16, "fp16", ragged=True,
              decodes=15),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    d, bits = rng.choice([64, 128]), rng.choice([2, 4, 8])
    page, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["fp16", "bf16"])
    kind = rng.choice(["store", "read", "decode", "decode", "chunk", "chunk", "mixed"])
    ragged = rng.random() < 0.7
    if kind in ("store", "read"):
        batch = _log(rng, 1, 24)
        new = min(_log(rng, 1, 4096), 32768 // batch)
        ctx = new if kind == "read" else new + rng.randrange(0, 1000)
        return dict(op=kind, batch=batch, ctx=ctx, new=new, hq=hq, hkv=hkv, d=d, bits=bits,
                    page=page, dtype=dtype, ragged=ragged, decodes=0)
    if kind == "decode":
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 1, 16384)
        while batch > 1 and batch * ctx * hkv * d * bits > 4e9:
            batch -= 1
        return dict(op="attend", batch=batch, ctx=ctx, new=1, hq=hq, hkv=hkv, d=d, bits=bits,
                    page=page, dtype=dtype, ragged=ragged, decodes=0)
    new = _log(rng, 2, 2048)
    ctx = new + _log(rng, 1, 12000)
    batch = _log(rng, 1, 6)
    while batch > 1 and batch * hq * new * ctx > 6e8:
        batch -= 1
    return dict(op="attend", batch=batch, ctx=ctx, new=new, hq=hq, hkv=hkv, d=d, bits=bits,
                page=page, dtype=dtype, ragged=ragged,
                decodes=(batch - 1 if kind == "mixed" else 0))


def _lengths(case):
    """(tokens held, new tokens) of each sequence, from the case alone."""
    B, ctx, new = case["batch"], case["ctx"], case["new"]
    kv, n = [ctx] * B, [new] * B
    rng = random.Random("%d %d %d %d" % (B, ctx, new, case["d"]))
    if case["ragged"]:
        n = [new if b == 0 else rng.randint(max(1, new // 4), new) for b in range(B)]
        kv = [ctx if b == 0 else max(n[b], rng.randint(max(1, ctx // 3), ctx)) for b in range(B)]
        if case["op"] == "read":
            n = list(kv)
    for b in range(B - case["decodes"], B):
        n[b] = 1
    return kv, n


def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _row_bytes(case):
    """Bytes one token and head holds: codes and statistics of the key and the value."""
    return 2 * (case["d"] * case["bits"] // 8 + case["d"] // GROUP * 4)


def work(case):
    kv, n = _lengths(case)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    T = sum(n)
    held, rows = _row_bytes(case) * hkv, 2 * 2 * hkv * d  # bytes of a token: in pages, as rows
    if case["op"] == "store":
        return {"bytes": T * (held + 2 * rows), "flops": 8.0 * T * hkv * d}
    if case["op"] == "read":
        return {"bytes": T * (held + rows), "flops": 4.0 * T * hkv * d}
    pairs = sum(m * (k - m) + m * (m + 1) // 2 for k, m in zip(kv, n))
    return {"bytes": sum(kv) * held + 2 * 2 * T * hq * d, "flops": 4.0 * hq * d * pairs}


# --------------------------------------------------------------------------
# the packed layout: code slot s of a row (slots of `bits` bits, little
# endian) holds channel order[s]

def _order(which, d, bits):
    order = [0] * d
    for c in range(d):
        g32, r = divmod(c, GROUP)
        if which == "k":
            j, e, pair = r // 8, r % 2, g32 * 4 + r % 8 // 2
            base, width = j * (d * bits // 4), 16
        else:
            e, pair = g32 % 2, g32 // 2 * 4 + r % 4
            base, width = r // 4 * (d * bits // 8), min(16, d // 16 * bits)
        word, off = divmod(pair * bits, width)
        order[(base + word * 2 * width + off + width * e) // bits] = c
    return order


def _regions(case):
    """Byte offsets inside an atom (16 tokens of one head): key codes, value
    codes, key statistics, value statistics, end."""
    rb, st = case["d"] * case["bits"] // 8, case["d"] // GROUP * 4
    return [0, ATOM * rb, 2 * ATOM * rb, 2 * ATOM * rb + ATOM * st, 2 * ATOM * (rb + st)]


def _quantise(x, bits):
    """fp32 [..., d] -> whole codes, scale and zero (fp16 values) of each group."""
    x = torch.nan_to_num(x, nan=0.0, posinf=LIMIT, neginf=-LIMIT).clamp(-LIMIT, LIMIT)
    x = x.unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    top = float(2 ** bits - 1)
    scale, zero = ((hi - lo) / top).half(), (lo + 0.0).half()
    s = scale.float()
    q = torch.where(s > 0, torch.round((x - zero.float()) / torch.where(s > 0, s, 1.0)), 0.0)
    return q.clamp(0, top).to(torch.uint8).flatten(-2), scale.squeeze(-1), zero.squeeze(-1)


def _pack(codes, order, bits):
    per = 8 // bits
    c = codes[..., order].unflatten(-1, (-1, per))
    shift = torch.arange(per, device=codes.device, dtype=torch.uint8) * bits
    return (c << shift).sum(-1, dtype=torch.uint8)


def _unpack(rows, where, bits):
    per = 8 // bits
    shift = torch.arange(per, device=rows.device, dtype=torch.uint8) * bits
    c = (rows.unsqueeze(-1) >> shift) & (2 ** bits - 1)
    return c.flatten(-2)[..., where]


# --------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    kv, n = _lengths(case)
    B, P, H, Hq, d, bits = (case[k] for k in ("batch", "page", "hkv", "hq", "d", "bits"))
    dt, T = _dtype(case), sum(n)
    pages_of = [-(-k // P) for k in kv]
    n_pages, width = sum(pages_of) + 3, max(pages_of)
    # pages are handed out in any order: a table of a random permutation
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor([sum(pages_of[:b]) for b in range(B)], device=dev)
    at = first[:, None] + torch.arange(width, device=dev)
    held = torch.arange(width, device=dev) < torch.tensor(pages_of, device=dev)[:, None]
    table = torch.where(held, ids[at.clamp(max=n_pages - 1)], 0).to(torch.int32).contiguous()
    cu = [sum(n[:b]) for b in range(B + 1)]
    # channels of different size, some keys with large channels, as a model's are
    kscale = torch.exp(0.3 * torch.randn(H, d, generator=gen, device=dev))
    kscale *= torch.where(torch.rand(H, d, generator=gen, device=dev) < 0.02, 8.0, 1.0)

    def rows(*shape):
        x = torch.randn(*shape, H, d, generator=gen, device=dev)
        return (x * kscale).to(dt), torch.randn(*shape, H, d, generator=gen, device=dev).to(dt)

    off = _regions(case)
    korder = torch.tensor(_order("k", d, bits), device=dev)
    vorder = torch.tensor(_order("v", d, bits), device=dev)
    pages = torch.empty(n_pages, H, P // ATOM, off[4], dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (P * H * d))
    for p0 in range(0, n_pages, step):
        part = pages[p0:p0 + step]
        fields = _fields(part, case)
        for x, order, codes, stats in zip(rows(part.shape[0], P // ATOM, ATOM), (korder, vorder),
                                          fields[:2], fields[2:]):
            q, s, z = _quantise(x.float(), bits)
            codes.copy_(_pack(q, order, bits).permute(0, 3, 1, 2, 4))
            stats.copy_(torch.cat([s, z], -1).view(torch.uint8).permute(0, 3, 1, 2, 4))
    state = {
        "op": case["op"], "case": dict(case), "pages": pages, "table": table,
        "lens": torch.tensor(kv, dtype=torch.int32, device=dev),
        "cu": torch.tensor(cu, dtype=torch.int32, device=dev), "T": T, "most": max(n),
        "width": max(kv), "scale": 1.0 / math.sqrt(d), "korder": korder, "vorder": vorder,
        "kwhere": torch.argsort(korder), "vwhere": torch.argsort(vorder),
    }
    if case["op"] == "store":
        state["k"], state["v"] = rows(T)
    elif case["op"] == "attend":
        # queries aligned to the keys' channels: some tokens stand out, most do not
        state["q"] = (torch.randn(T, Hq, d, generator=gen, device=dev) * 1.2).to(dt)
    if own:
        from bit_kv_cache_14_gb300 import kvq
        cfg = kvq.make_paged_config(Hq, H, d, bits, P, n_pages, dt)
        state["cache"] = kvq.PagedKVCache(cfg, dev, pages=pages)
        state["batch"] = kvq.PagedBatch(table, state["lens"], state["cu"], n_tokens=T,
                                        max_tokens=max(n))
    return state


def _fields(pages, case):
    """Views of the pages: key codes, value codes [page][head][atom][16][bytes],
    key and value statistics (the scales of a token's groups, then their zeros)."""
    off = _regions(case)
    return [pages[..., a:b].unflatten(-1, (ATOM, -1)) for a, b in zip(off, off[1:])]


# --------------------------------------------------------------------------
# one pass

def run(state):
    if own:
        cache, batch = state["cache"], state["batch"]
        if state["op"] == "store":
            cache.write(state["k"], state["v"], batch)
            return cache.read(batch)
        if state["op"] == "read":
            return cache.read(batch)
        return cache.attend(state["q"], batch, scale=state["scale"])
    if state["op"] == "store":
        _plain_write(state)
        return _plain_read(state)
    return _plain_read(state) if state["op"] == "read" else _plain_attend(state)


def _slots(state):
    """(page, atom, row) of each packed token: the last n_b of its sequence."""
    P = state["case"]["page"]
    i = torch.arange(state["T"], device=state["cu"].device)
    b = torch.searchsorted(state["cu"].long(), i, right=True) - 1
    pos = state["lens"][b].long() - state["cu"][b + 1].long() + i
    return state["table"][b, pos // P].long(), pos % P // ATOM, pos % ATOM


def _plain_write(state):
    case = state["case"]
    page, atom, row = _slots(state)
    kc, vc, ks, vs = _fields(state["pages"], case)
    for x, order, codes, stats in ((state["k"], state["korder"], kc, ks),
                                   (state["v"], state["vorder"], vc, vs)):
        q, s, z = _quantise(x.float(), case["bits"])
        codes[page, :, atom, row] = _pack(q, order, case["bits"])
        stats[page, :, atom, row] = torch.cat([s, z], -1).view(torch.uint8)


def _values(codes, stats, where, bits):
    c = _unpack(codes, where, bits).float().unflatten(-1, (-1, GROUP))
    s, z = stats.contiguous().view(torch.float16).float().chunk(2, -1)
    return (c * s.unsqueeze(-1) + z.unsqueeze(-1)).flatten(-2)


def _plain_read(state):
    case = state["case"]
    page, atom, row = _slots(state)
    kc, vc, ks, vs = _fields(state["pages"], case)
    return tuple(_values(c[page, :, atom, row], s[page, :, atom, row], where,
                         case["bits"]).to(_dtype(case))
                 for c, s, where in ((kc, ks, state["kwhere"]), (vc, vs, state["vwhere"])))


def _plain_attend(state):
    case = state["case"]
    H, Hq, d, P = case["hkv"], case["hq"], case["d"], case["page"]
    rg, dev = Hq // H, state["q"].device
    lens, cu = state["lens"].long(), state["cu"].long()
    # every sequence padded to the longest: keys and values [B][H][W][d]
    pos = torch.arange(state["width"], device=dev)
    page = state["table"].long()[:, pos // P]
    kc, vc, ks, vs = _fields(state["pages"], case)
    at = (page, slice(None), (pos % P // ATOM).expand_as(page), (pos % ATOM).expand_as(page))
    K, V = (_values(c[at], s[at], where, case["bits"]).transpose(1, 2)
            for c, s, where in ((kc, ks, state["kwhere"]), (vc, vs, state["vwhere"])))
    # queries padded to the longest chunk: [B][H][rg * n][d]
    i = torch.arange(state["most"], device=dev)
    count = cu[1:] - cu[:-1]
    real = i < count[:, None]
    src = (cu[:-1, None] + i).clamp(max=state["T"] - 1)
    q = state["q"].float()[src].unflatten(2, (H, rg)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, K.transpose(2, 3)).mul_(state["scale"])
    last = (lens - count)[:, None] + i                              # newest token a query sees
    seen = pos <= torch.where(real, last, -1)[..., None]            # [B][n][W]
    x = x.unflatten(2, (rg, -1)).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    w = x.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.flatten(2, 3), V).unflatten(2, (rg, -1)) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                      # [B][n][Hq][d]
    return o[real].to(_dtype(case))


# --------------------------------------------------------------------------
# the operators in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kv, n = _lengths(case)
    d, bits, P, H = case["d"], case["bits"], case["page"], case["hkv"]
    if case["op"] == "store":
        return tuple(_exact_stored(s[x].double(), bits) for x in "kv")
    if case["op"] == "read":
        both = [_exact_rows(s, case, b, kv[b] - n[b], kv[b]) for b in range(case["batch"])]
        return torch.cat([k for k, _ in both]), torch.cat([v for _, v in both])
    outs, at = [], 0
    for b in range(case["batch"]):
        K, V = _exact_rows(s, case, b, 0, kv[b])
        out = torch.empty(n[b], case["hq"], d, dtype=torch.float64, device=K.device)
        sees = torch.arange(n[b], device=K.device)[:, None] + (kv[b] - n[b])
        hidden = torch.arange(kv[b], device=K.device)[None] > sees
        for h in range(case["hq"]):
            x = s["q"][at:at + n[b], h].double() @ K[:, h // (case["hq"] // H)].T * s["scale"]
            x[hidden] = -math.inf
            out[:, h] = torch.softmax(x, -1) @ V[:, h // (case["hq"] // H)]
        outs.append(out)
        at += n[b]
    return torch.cat(outs)


def _exact_stored(x, bits):
    """Each group of 32 channels on the grid zero + scale * (0 .. 2^bits - 1)."""
    T, H, d = x.shape
    out = torch.empty_like(x)
    for c in range(0, d, GROUP):
        part = x[..., c:c + GROUP]
        lo, hi = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        step = ((hi - lo) / (2 ** bits - 1)).half().double()
        base = lo.half().double()
        k = torch.round((part - base) / step.clamp(min=1e-30)).clamp(0, 2 ** bits - 1)
        out[..., c:c + GROUP] = torch.where(step > 0, base + k * step, base)
    return out


def _exact_rows(s, case, b, t0, t1):
    """Keys and values of tokens [t0, t1) of sequence b, bit by bit."""
    d, bits, P, H = case["d"], case["bits"], case["page"], case["hkv"]
    t = torch.arange(t0, t1, device=s["pages"].device)
    atoms = s["pages"][s["table"][b, t // P].long(), :, t % P // ATOM]     # [t][H][bytes]
    rb, ng = d * bits // 8, d // GROUP
    outs = []
    for which, code0, stat0 in (("k", 0, 2 * ATOM * rb),
                                ("v", ATOM * rb, 2 * ATOM * rb + ATOM * ng * 4)):
        out = torch.empty(t1 - t0, H, d, dtype=torch.float64, device=t.device)
        r = (t % ATOM)[:, None, None]
        idx = stat0 + r * ng * 4 + torch.arange(ng * 4, device=t.device)
        st = atoms.gather(2, idx.expand(-1, H, -1)).contiguous().view(torch.float16).double()
        row = atoms.gather(2, (code0 + r * rb + torch.arange(rb, device=t.device)).expand(-1, H, -1))
        for slot, c in enumerate(_order(which, d, bits)):
            byte, bit = divmod(slot * bits, 8)
            code = (row[..., byte] >> bit) & (2 ** bits - 1)
            out[..., c] = code.double() * st[..., c // GROUP] + st[..., ng + c // GROUP]
        outs.append(out)
    return outs
