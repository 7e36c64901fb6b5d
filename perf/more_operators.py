"""Cases of the serving operators around the paged cache, and their plain forms.

The operators (include/kvq.h):
  pages   bookkeeping of block tables on the device: pages for new tokens with
          copies of shared ones (kvq_pages_reserve), tokens taken back and pages
          freed (kvq_pages_drop), sequences forked, reordered or ended
          (kvq_pages_select), holders counted (kvq_pages_recount), live pages
          moved to the front of the pool (kvq_pages_compact), and the copies
          themselves (kvq_paged_copy);
  cross   packed query rows attend to everything their sequence holds, an
          encoder's states (kvq_paged_cross_attention);
  verify  drafted tokens are accepted or refused by the target's probabilities
          and given random numbers, the next token is drawn, and the tokens'
          log probabilities are given (kvq_verify_drafts).

The plain forms are elementary torch operations.  `exact` states the operators
once more: computed numbers in 64 bits, tables by lists.
"""
import math
import random

import torch

own = False  # True: run() calls the library's kernels instead of the plain forms

GROUP = 32   # channels that share a scale and a zero point
ATOM = 16    # tokens stored together inside a page
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases

def _step(name, seqs, ctx, new, page, spare):
    return dict(name=name, op="step", seqs=seqs, ctx=ctx, new=new, page=page, spare=spare)


def _fork(name, prompts, samples, ctx, page, hkv, d, bits, dtype):
    return dict(name=name, op="fork", prompts=prompts, samples=samples, ctx=ctx, page=page,
                hkv=hkv, d=d, bits=bits, dtype=dtype)


def _compact(name, seqs, ctx, page, spare, hkv, d, bits, dtype):
    return dict(name=name, op="compact", seqs=seqs, ctx=ctx, page=page, spare=spare, hkv=hkv, d=d,
                bits=bits, dtype=dtype)


def _cross(name, batch, ctx, rows, hq, hkv, d, bits, page, dtype, ragged=False):
    return dict(name=name, op="cross", batch=batch, ctx=ctx, rows=rows, hq=hq, hkv=hkv, d=d,
                bits=bits, page=page, dtype=dtype, ragged=ragged)


def _verify(name, batch, drafts, vocab, dtype, draft, ragged=False):
    return dict(name=name, op="verify", batch=batch, drafts=drafts, vocab=vocab, dtype=dtype,
                draft=draft, ragged=ragged)


def listed():
    return [
        # tables of a small speculating batch, step after step: latency
        _step("tables_step_b16", 16, 2000, 5, 16, 200),
        # the most sequences a call takes, over a pool of very many pages
        _step("tables_step_b2048", 2048, 1500, 8, 16, 300000),
        # a few prompts, each sampled several times: shared pages, copied on write
        _fork("fork_samples_4x15", 4, 15, 4000, 64, 8, 128, 4, "fp16"),
        # a pool left half empty by ended sequences, brought to its front
        _compact("compact_b64", 64, 8192, 64, 8192, 8, 128, 4, "bf16"),
        # decode step of a few sequences against short encoders: latency
        _cross("cross_step_b4", 4, 377, 1, 8, 8, 64, 8, 16, "fp16", ragged=True),
        # decode step of a batch of beam groups, four beams to an encoder
        _cross("cross_beams_b32", 32, 4096, 4, 32, 8, 128, 4, 64, "bf16", ragged=True),
        # decoder prompts of uneven sizes against encoders of uneven lengths
        _cross("cross_prompts_b6", 6, 1999, 333, 32, 32, 128, 2, 32, "fp16", ragged=True),
        # many decoder positions at once against long encoders
        _cross("cross_long_2048", 2, 16384, 2048, 32, 8, 128, 4, 64, "bf16"),
        # one conversation's drafts, small vocabulary: latency
        _verify("verify_b1_v32000", 1, 4, 32000, "fp16", "model"),
        # tokens found by lookup, an odd vocabulary, none to eight drafts each
        _verify("verify_lookup_b24", 24, 8, 50001, "bf16", "lookup", ragged=True),
        # a serving batch with a large vocabulary
        _verify("verify_b64_v131072", 64, 4, 131072, "bf16", "model"),
        # greedy decoding of fp32 logits
        _verify("verify_greedy_b128", 128, 3, 65537, "fp32", "greedy"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page, hkv = rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    d, bits, dtype = rng.choice([64, 128]), rng.choice([2, 4, 8]), rng.choice(["fp16", "bf16"])
    kind = rng.choice(["step", "fork", "compact", "cross", "cross", "cross", "verify", "verify",
                       "verify"])
    if kind == "step":
        seqs = _log(rng, 1, 2048)
        ctx = _log(rng, 1, min(20000, 3000000 // seqs))
        return _named(_step, seqs, ctx, _log(rng, 1, 600 if seqs < 100 else 20), page,
                      _log(rng, 10, 300000) + 2 * seqs * (600 // page + 2))
    if kind == "fork":
        prompts, samples = _log(rng, 1, 12), _log(rng, 1, 24)
        return _named(_fork, prompts, samples, _log(rng, 1, 6000), page, hkv, d, bits, dtype)
    if kind == "compact":
        seqs = _log(rng, 1, 200)
        ctx = _log(rng, 1, min(16384, 500000 // seqs))
        pages = seqs * (ctx // page + 1)
        return _named(_compact, seqs, ctx, page, _log(rng, 1, max(2, pages)), hkv, d, bits, dtype)
    if kind == "cross":
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        rows, ctx, batch = _log(rng, 1, 1500), _log(rng, 1, 16000), _log(rng, 1, 48)
        while batch > 1 and (batch * hq * rows * ctx > 6e8 or batch * ctx * hkv * d > 2.5e8):
            batch -= 1
        return _named(_cross, batch, ctx, rows, hq, hkv, d, bits, page, dtype, rng.random() < 0.7)
    vocab, drafts, batch = _log(rng, 100, 140000), rng.randint(0, 9), _log(rng, 1, 96)
    while batch > 1 and batch * (drafts + 1) * vocab > 2.2e7:
        batch -= 1
    return _named(_verify, batch, drafts, vocab, rng.choice(["fp16", "bf16", "fp32"]),
                  rng.choice(["model", "model", "lookup", "greedy"]), rng.random() < 0.7)


def _named(make, *args):
    case = make("", *args)
    del case["name"]
    return case


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _spread(case, n, top, low):
    """n whole numbers from low to top, the first of them top."""
    rng = _rng(case)
    return [top if i == 0 else rng.randint(min(low, top), top) for i in range(n)]


def _lengths(case):
    """Tokens that each sequence holds."""
    op = case["op"]
    if op == "cross":
        low = max(1, case["ctx"] // 3) if case["ragged"] else case["ctx"]
        return _spread(case, case["batch"], case["ctx"], low)
    if op == "fork":
        return (_spread(case, case["prompts"], case["ctx"], max(1, case["ctx"] // 2))
                + [0] * (case["prompts"] * case["samples"]))
    return _spread(case, case["seqs"], case["ctx"], max(1, case["ctx"] // 3))


def _rows(case):
    """The call's rows of each sequence."""
    op, rng = case["op"], _rng(case)
    if op == "cross":
        low = max(1, case["rows"] // 4) if case["ragged"] else case["rows"]
        return [rng.randint(low, case["rows"]) for _ in range(case["batch"])]
    if op == "verify":
        low = 0 if case["ragged"] else case["drafts"]
        return [1 + rng.randint(low, case["drafts"]) for _ in range(case["batch"])]
    if op == "fork":
        return [0] * case["prompts"] + [1] * (case["prompts"] * case["samples"])
    return [rng.randint(1, case["new"]) for _ in range(case["seqs"])]


def _row_bytes(case):
    """Bytes one token and head holds: codes and statistics of the key and the value."""
    return 2 * (case["d"] * case["bits"] // 8 + case["d"] // GROUP * 4)


def _page_bytes(case):
    return case["page"] * case["hkv"] * _row_bytes(case)


def work(case):
    op = case["op"]
    if op == "verify":
        n, V = _rows(case), case["vocab"]
        size = 4 if case["dtype"] == "fp32" else 2
        drafts = sum(n) - len(n)
        nbytes = sum(n) * V * size + 20 * sum(n)
        if case["draft"] == "model":
            nbytes += drafts * V * size
        if case["draft"] != "greedy":
            nbytes += len(n) * V * 4
        return {"bytes": nbytes, "flops": 4.0 * nbytes / size}
    if op == "cross":
        kv, n = _lengths(case), _rows(case)
        d, hq = case["d"], case["hq"]
        pairs = sum(k * m for k, m in zip(kv, n))
        return {"bytes": sum(kv) * case["hkv"] * _row_bytes(case) + 2 * 2 * sum(n) * hq * d,
                "flops": 4.0 * hq * d * pairs}
    lens, page = _lengths(case), case["page"]
    if op == "step":
        # pages of the new tokens: table entries and holder counts, twice
        new = sum(-(-k // page) - -(-(k - n) // page) for k, n in zip(_step_lengths(case),
                                                                       _rows(case)))
        return {"bytes": 2 * 16 * new + 16 * len(lens), "flops": 2.0 * len(lens)}
    held = [-(-k // page) for k in lens]
    if op == "fork":
        # tables and holder counts of the forks, and their partly filled pages
        entries = case["samples"] * sum(held)
        copied = case["samples"] * sum(k % page != 0 for k in lens[:case["prompts"]])
        return {"bytes": 16 * entries + 2 * copied * _page_bytes(case), "flops": float(entries)}
    live = sum(held)
    moved = int(live * case["spare"] / (live + case["spare"]))
    return {"bytes": 8 * live + 8 * (live + case["spare"]) + 2 * moved * _page_bytes(case),
            "flops": float(live)}


def _step_lengths(case):
    return [k + n for k, n in zip(_lengths(case), _rows(case))]


# --------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    make = {"cross": _prepare_cross, "verify": _prepare_verify}.get(case["op"], _prepare_tables)
    state = make(case, gen, dev)
    state["case"] = dict(case)
    return state


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _cu(n, dev):
    return _i32([sum(n[:b]) for b in range(len(n) + 1)], dev) if len(n) < 64 else torch.cat(
        [_i32([0], dev), torch.cumsum(_i32(n, dev), 0).to(torch.int32)])


def _tables(lens, page, width, spare, gen, dev):
    """Block tables that hand out pages in any order, -1 behind each sequence's last."""
    held = _i32([-(-k // page) for k in lens], dev)
    n_pages = int(held.sum()) + spare
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    at = (torch.cumsum(held, 0) - held)[:, None] + torch.arange(width, device=dev)
    used = torch.arange(width, device=dev) < held[:, None]
    table = torch.where(used, ids[at.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    return table, n_pages


def _prepare_tables(case, gen, dev):
    op, page = case["op"], case["page"]
    lens = _step_lengths(case) if op == "step" else _lengths(case)
    n = [] if op == "compact" else _rows(case)
    width = -(-max(lens) // page) + 2
    spare = case["spare"] if op != "fork" else len(lens) + 5
    table, n_pages = _tables(lens, page, width, spare, gen, dev)
    state = {"table": table, "lens": _i32(lens, dev), "n_pages": n_pages, "cu": _cu(n, dev)}
    state["refs"] = _holders(table, state["lens"], page, n_pages)
    if op == "step":
        # a step's rows are taken back before the next step's get their pages
        state["drop"] = _i32(n, dev)
    else:
        shape = (n_pages, case["hkv"], page // ATOM, ATOM * _row_bytes(case))
        state["pool"] = torch.randint(0, 256, shape, dtype=torch.uint8, generator=gen, device=dev)
    if op == "fork":
        P, S = case["prompts"], case["samples"]
        order = torch.randperm(P * S, generator=gen, device=dev) % P
        state["parents"] = torch.cat([torch.arange(P, device=dev), order]).to(torch.int32)
    if op == "compact":
        state["saved"] = table.clone()
    if own:
        from bit_kv_cache_14_gb300 import kvq
        state["tab"] = kvq.PageTable(n_pages, page, block_table=table, seq_lens=state["lens"])
        if op != "step":
            cfg = kvq.make_paged_config(case["hkv"], case["hkv"], case["d"], case["bits"], page,
                                        n_pages, DTYPES[case["dtype"]])
            state["cache"] = kvq.PagedKVCache(cfg, dev, pages=state["pool"])
    return state


def _holders(table, lens, page, n_pages):
    used = _used(table, lens, page)
    ids = torch.where(used, table, n_pages).flatten().long()
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device=table.device)
    return refs.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))[:n_pages].contiguous()


def _used(table, lens, page):
    held = (lens + page - 1) // page
    return torch.arange(table.shape[1], device=table.device) < held[:, None]


def _prepare_cross(case, gen, dev):
    kv, n = _lengths(case), _rows(case)
    B, P, H, Hq, d, bits = (case[k] for k in ("batch", "page", "hkv", "hq", "d", "bits"))
    dt, T, top = DTYPES[case["dtype"]], sum(n), 2 ** bits - 1
    table, n_pages = _tables(kv, P, -(-max(kv) // P), 3, gen, dev)
    # the pages' statistics are those of states of deviation 1, some channel groups larger
    pages = torch.empty(n_pages, H, P // ATOM, ATOM * _row_bytes(case), dtype=torch.uint8,
                        device=dev)
    big = torch.where(torch.rand(H, d // GROUP, generator=gen, device=dev) < 0.15, 3.0, 1.0)
    step = max(1, (1 << 27) // (P * H * d))
    for p0 in range(0, n_pages, step):
        part = pages[p0:p0 + step]
        fields = _fields(part, case)
        for i in range(2):
            fields[i].copy_(torch.randint(0, 256, fields[i].shape, dtype=torch.uint8,
                                          generator=gen, device=dev))
            shape = fields[2 + i].shape[:-1] + (d // GROUP,)
            size = 4.0 / top * (0.8 + 0.4 * torch.rand(shape, generator=gen, device=dev))
            low = -2.0 + 0.3 * torch.randn(shape, generator=gen, device=dev)
            if i == 0:
                size, low = size * big[:, None, None], low * big[:, None, None]
            fields[2 + i].copy_(torch.cat([size, low], -1).half().view(torch.uint8))
    state = {
        "pages": pages, "table": table.clamp(min=0), "lens": _i32(kv, dev), "cu": _cu(n, dev),
        "T": T, "most": max(n), "width": max(kv), "scale": 1.0 / math.sqrt(d),
        "kwhere": torch.argsort(torch.tensor(_order("k", d, bits), device=dev)),
        "vwhere": torch.argsort(torch.tensor(_order("v", d, bits), device=dev)),
        "q": torch.randn(T, Hq, d, generator=gen, device=dev).to(dt),
    }
    if own:
        from bit_kv_cache_14_gb300 import kvq
        cfg = kvq.make_paged_config(Hq, H, d, bits, P, n_pages, dt)
        state["cache"] = kvq.PagedKVCache(cfg, dev, pages=pages)
        state["batch"] = kvq.PagedBatch(state["table"], state["lens"], state["cu"], n_tokens=T,
                                        max_tokens=max(n))
    return state


def _prepare_verify(case, gen, dev):
    n, V, dt = _rows(case), case["vocab"], DTYPES[case["dtype"]]
    B, T = len(n), sum(n)
    cu = _cu(n, dev)
    logits = torch.empty(T, V, dtype=dt, device=dev)
    draft = torch.empty(T, V, dtype=dt, device=dev) if case["draft"] == "model" else None
    tokens = torch.randint(0, V, (T,), generator=gen, device=dev)
    temperature = 0.6 + 0.6 * torch.rand(B, generator=gen, device=dev)
    seq = torch.repeat_interleave(torch.arange(B, device=dev), _i32(n, dev))
    step = max(1, (1 << 26) // V)
    for r0 in range(0, T, step):
        m = min(step, T - r0)
        # a model's logits: most tokens far below the few that are likely
        x = 2.0 * torch.randn(m, V, generator=gen, device=dev)
        x += 9.0 * (torch.rand(m, V, generator=gen, device=dev) < 20.0 / V)
        logits[r0:r0 + m] = x.to(dt)
        pick = x
        if draft is not None:
            pick = x + 0.5 * torch.randn(m, V, generator=gen, device=dev)
            draft[r0:r0 + m] = pick.to(dt)
            pick = draft[r0:r0 + m].float() / temperature[seq[r0:r0 + m], None]
            noise = torch.empty(m, V, device=dev).exponential_(generator=gen)
            pick = pick - torch.log(noise.clamp(min=1e-30))
        # the next row's token is what was drafted here, or now and then another
        best = pick.argmax(-1)
        if draft is None:
            other = torch.randint(0, V, (m,), generator=gen, device=dev)
            best = torch.where(torch.rand(m, generator=gen, device=dev) < 0.75, best, other)
        to = torch.arange(r0 + 1, min(r0 + m, T - 1) + 1, device=dev)
        tokens[to] = best[:len(to)]
    state = {"logits": logits, "draft": draft, "tokens": tokens.to(torch.int32), "cu": cu}
    state["temperature"] = state["uniform"] = state["noise"] = None
    if case["draft"] != "greedy":
        state["temperature"] = temperature
        state["uniform"] = torch.rand(T, generator=gen, device=dev)
        state["noise"] = torch.empty(B, V, device=dev).exponential_(generator=gen)
    if own:
        from bit_kv_cache_14_gb300 import kvq
        state["verifier"] = kvq.DraftVerifier(B, T, V, dt, dev)
    return state


# --------------------------------------------------------------------------
# one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if op == "cross":
        if own:
            return state["cache"].cross_attend(state["q"], state["batch"], scale=state["scale"])
        return _plain_cross(state)
    if op == "verify":
        args = [state[k] for k in ("logits", "tokens", "cu", "draft", "temperature", "uniform",
                                   "noise")]
        if own:
            return state["verifier"].verify(*args)
        return _plain_verify(*args)
    if own:
        tab = state["tab"]
        if op == "step":
            tab.drop(state["drop"])
            copies, _ = tab.reserve(state["cu"])
        elif op == "fork":
            tab.select(state["parents"])
            copies, _ = tab.reserve(state["cu"])
            state["cache"].copy_pages(copies)
        else:
            tab.block_table.copy_(state["saved"])
            tab.recount()
            copies = tab.compact()
            state["cache"].copy_pages(copies)
        out = [tab.block_table, tab.seq_lens, tab.page_refs, copies]
    else:
        page = case["page"]
        if op == "step":
            _plain_drop(state, state["drop"], page)
            copies = _plain_reserve(state, state["cu"], page)
        elif op == "fork":
            _plain_select(state, state["parents"], page)
            copies = _plain_reserve(state, state["cu"], page)
            _plain_copy(state, copies)
        else:
            state["table"].copy_(state["saved"])
            state["refs"].copy_(_holders(state["table"], state["lens"], page, state["n_pages"]))
            copies = _plain_compact(state, page)
            _plain_copy(state, copies)
        out = [state["table"], state["lens"], state["refs"], copies]
    if op != "step":
        out.append(state["pool"].view(torch.int64))
    return out


def _pairs(src, dst, rows):
    out = torch.full((rows, 2), -1, dtype=torch.int32, device=src.device)
    out[:len(src), 0] = src.to(torch.int32)
    out[:len(src), 1] = dst.to(torch.int32)
    return out


def _plain_reserve(state, cu, page):
    table, lens, refs = state["table"], state["lens"], state["refs"]
    B, n_pages = len(lens), state["n_pages"]
    b = torch.arange(B, device=cu.device)
    n = cu[1:] - cu[:-1]
    # a partly filled page that others hold too is copied before it is written; of
    # sequences that all write to it now, and are all its holders, the first keeps it
    last = (lens // page).long()
    own_page = table.gather(1, last[:, None])[:, 0].long()
    part = (n > 0) & (lens % page != 0)
    claim = part & (refs[own_page.clamp(min=0)] > 1)
    at = torch.where(claim, own_page, n_pages)
    claims = torch.zeros(n_pages + 1, dtype=torch.int32, device=cu.device)
    claims.index_add_(0, at, torch.ones_like(lens))
    first = torch.full((n_pages + 1,), B, device=cu.device)
    first.scatter_reduce_(0, at, b, "amin")
    keep = claim & (claims[at] == refs[at.clamp(max=n_pages - 1)]) & (first[at] == b)
    copy = claim & ~keep
    refs -= claims[:n_pages]
    refs.index_add_(0, at[keep], torch.ones_like(lens[keep]))
    held = (lens + page - 1) // page
    need = (lens + n + page - 1) // page - held
    need = torch.where(n > 0, need, 0) + copy
    # free pages, the lowest first, sequence by sequence
    total = int(need.sum())
    free = (refs == 0).nonzero()[:total, 0]
    who = torch.repeat_interleave(b, need)
    off = torch.arange(total, device=cu.device) - (torch.cumsum(need, 0) - need)[who]
    entry = torch.where(copy[who] & (off == 0), last[who], held[who] + off - copy[who].long())
    table[who, entry] = free.to(torch.int32)
    refs[free] = 1
    lens += torch.where(n > 0, n, 0)
    return _pairs(own_page[copy], free[off == 0][copy[who[off == 0]]], B)


def _plain_drop(state, drop, page):
    table, lens, refs = state["table"], state["lens"], state["refs"]
    before = _used(table, lens, page)
    lens -= torch.minimum(drop.clamp(min=0), lens)
    gone = before & ~_used(table, lens, page)
    ids = table[gone].long()
    refs.index_add_(0, ids, torch.full_like(table[gone], -1))
    table.masked_fill_(gone, -1)


def _plain_select(state, parents, page):
    table, lens, refs = state["table"], state["lens"], state["refs"]
    n_pages = state["n_pages"]
    change = parents != torch.arange(len(lens), device=parents.device)
    src = parents.clamp(min=0).long()
    new_lens = torch.where(parents >= 0, lens[src], 0)
    new_table = torch.where(_used(table, new_lens, page), table[src], -1)
    old = _used(table, lens, page) & change[:, None]
    new = _used(table, new_lens, page) & change[:, None]
    for mask, t, by in ((new, new_table, 1), (old, table, -1)):
        ids = t[mask].long()
        refs.index_add_(0, ids, torch.full_like(t[mask], by))
    table.copy_(torch.where(change[:, None], new_table, table))
    lens.copy_(torch.where(change, new_lens, lens))


def _plain_compact(state, page):
    table, lens, refs, n_pages = state["table"], state["lens"], state["refs"], state["n_pages"]
    live = refs > 0
    front = int(live.sum())
    src = live[front:].nonzero()[:, 0] + front
    dst = (~live[:front]).nonzero()[:, 0]
    where = torch.arange(n_pages, device=table.device, dtype=torch.int32)
    where[src] = dst.to(torch.int32)
    table.copy_(torch.where(_used(table, lens, page), where[table.clamp(min=0).long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    return _pairs(src, dst, max(1, n_pages // 2))


def _plain_copy(state, copies):
    pairs = copies[copies[:, 0] >= 0].long()
    state["pool"][pairs[:, 1]] = state["pool"][pairs[:, 0]]


def _order(which, d, bits):
    """Channel in code slot s of a row (slots of `bits` bits, little endian)."""
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


def _fields(pages, case):
    """Views of the pages: key codes, value codes [page][head][atom][16][bytes],
    key and value statistics (the scales of a token's groups, then their zeros)."""
    rb, st = case["d"] * case["bits"] // 8, case["d"] // GROUP * 4
    off = [0, ATOM * rb, 2 * ATOM * rb, 2 * ATOM * rb + ATOM * st, 2 * ATOM * (rb + st)]
    return [pages[..., a:b].unflatten(-1, (ATOM, -1)) for a, b in zip(off, off[1:])]


def _values(codes, stats, where, bits):
    per = 8 // bits
    shift = torch.arange(per, device=codes.device, dtype=torch.uint8) * bits
    c = ((codes.unsqueeze(-1) >> shift) & (2 ** bits - 1)).flatten(-2)[..., where]
    s, z = stats.contiguous().view(torch.float16).float().chunk(2, -1)
    c = c.float().unflatten(-1, (-1, GROUP))
    return (c * s.unsqueeze(-1) + z.unsqueeze(-1)).flatten(-2)


def _plain_cross(state):
    case = state["case"]
    H, Hq, P, bits = case["hkv"], case["hq"], case["page"], case["bits"]
    rg, dev = Hq // H, state["q"].device
    lens, cu = state["lens"].long(), state["cu"].long()
    pos = torch.arange(state["width"], device=dev)
    page = state["table"].long()[:, pos // P]
    kc, vc, ks, vs = _fields(state["pages"], case)
    at = (page, slice(None), (pos % P // ATOM).expand_as(page), (pos % ATOM).expand_as(page))
    K, V = (_values(c[at], s[at], where, bits).transpose(1, 2)
            for c, s, where in ((kc, ks, state["kwhere"]), (vc, vs, state["vwhere"])))
    # queries padded to the most rows of a sequence: [B][H][rg * n][d]
    i = torch.arange(state["most"], device=dev)
    real = i < (cu[1:] - cu[:-1])[:, None]
    src = (cu[:-1, None] + i).clamp(max=state["T"] - 1)
    q = state["q"].float()[src].unflatten(2, (H, rg)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, K.transpose(2, 3)).mul_(state["scale"])
    x.masked_fill_((pos >= lens[:, None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    w = x.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, V) / torch.where(total > 0, total, 1.0)
    o = o.unflatten(2, (rg, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return o[real].to(DTYPES[case["dtype"]])


def _plain_verify(logits, tokens, cu, draft, temperature, uniform, noise):
    dev, (T, V), B = logits.device, logits.shape, len(cu) - 1
    first, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    row = torch.arange(T, device=dev)
    seq = torch.repeat_interleave(torch.arange(B, device=dev), n)
    drafted = row < first[seq] + n[seq] - 1            # rows whose next token was drafted
    nxt = tokens.long()[(row + 1).clamp(max=T - 1)]
    ids = torch.arange(V, device=dev)
    greedy = temperature is None
    temp = torch.ones(T, device=dev).double() if greedy else temperature.double()[seq]

    def log_sums(x):
        """Largest value of each row, and the 64-bit logarithm of the sum of its weights."""
        x = x.float()
        top = x.amax(-1, keepdim=True)
        z = ((x - top) / temp[:, None].float()).exp_().sum(-1, dtype=torch.float64)
        return top[:, 0].double(), z.log()

    def log_of(x, sums, chosen):
        mine = x.gather(1, chosen[:, None])[:, 0].double()
        return (mine - sums[0]) / temp - sums[1]

    sums = log_sums(logits)
    if greedy:
        x = logits.float()
        best = torch.where(x == x.amax(-1, keepdim=True), ids, V).amin(-1)
        good = nxt == best
    else:
        odds = log_of(logits, sums, nxt)
        if draft is not None:
            odds = odds - log_of(draft, log_sums(draft), nxt)
        good = uniform.double().log() < odds
    # the first refused draft of each sequence, or its last row
    stop = torch.where(drafted & good, T, row)
    at = torch.full((B,), T, device=dev).scatter_reduce_(0, seq, stop, "amin")
    accepted = at - first
    if greedy:
        token = best[at]
    else:
        refused = (accepted < n - 1)[:, None]

        def weights(x):
            x = (x[at].double() - x[at].amax(-1, keepdim=True).double())
            w = (x / temperature.double()[:, None]).exp_()
            return w / w.sum(-1, keepdim=True)

        p = weights(logits)
        if draft is not None:
            rest = (p - weights(draft)).clamp_(min=0)
        else:
            rest = torch.where(ids == nxt[at][:, None], 0.0, p)
        some = (rest > 0).any(-1, keepdim=True)
        p = torch.where(refused & some, rest, p)
        score = p / noise.double()
        token = torch.where(score == score.amax(-1, keepdim=True), ids, V).amin(-1)
    out = torch.where(row < at[seq], nxt, torch.where(row == at[seq], token[seq], -1))
    logs = torch.where(out >= 0, log_of(logits, sums, out.clamp(min=0)), 0.0).float()
    return tuple(t.to(torch.int32) for t in (out, accepted, n - 1 - accepted)) + (logs,)


# --------------------------------------------------------------------------
# the operators once more

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cross":
        return _exact_cross(s, case)
    if case["op"] == "verify":
        return _exact_verify(s, case)
    return _exact_tables(s, case)


def _exact_cross(s, case):
    outs, at, H, rg = [], 0, case["hkv"], case["hq"] // case["hkv"]
    for b, (kv, n) in enumerate(zip(_lengths(case), _rows(case))):
        K, V = _exact_rows(s, case, b, kv)
        out = torch.empty(n, case["hq"], case["d"], dtype=torch.float64, device=K.device)
        for h in range(case["hq"]):
            x = s["q"][at:at + n, h].double() @ K[:, h // rg].T * s["scale"]
            out[:, h] = torch.softmax(x, -1) @ V[:, h // rg]
        outs.append(out)
        at += n
    return torch.cat(outs)


def _exact_rows(s, case, b, n):
    """Keys and values of the first n tokens of sequence b, slot by slot."""
    d, bits, P, H = case["d"], case["bits"], case["page"], case["hkv"]
    t = torch.arange(n, device=s["pages"].device)
    atoms = s["pages"][s["table"][b, t // P].long(), :, t % P // ATOM]     # [t][H][bytes]
    rb, ng = d * bits // 8, d // GROUP
    outs = []
    for which, code0, stat0 in (("k", 0, 2 * ATOM * rb),
                                ("v", ATOM * rb, 2 * ATOM * rb + ATOM * ng * 4)):
        out = torch.empty(n, H, d, dtype=torch.float64, device=t.device)
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


def _exact_verify(s, case):
    """Sequence by sequence and draft by draft, as the rule is told."""
    n, V, greedy = _rows(case), case["vocab"], case["draft"] == "greedy"
    tokens = s["tokens"].tolist()
    out, logs, accepted, at = [], [], [], 0

    def lowest(x):
        return int((x == x.max()).nonzero()[0])

    for b, m in enumerate(n):
        T = 1.0 if greedy else float(s["temperature"][b])
        emitted = []
        for i in range(m):
            x = s["logits"][at + i].double()
            p = torch.softmax(x / T, -1)
            c, go_on = -1, False
            if i == m - 1:
                c = lowest(x if greedy else p / s["noise"][b].double())
            elif greedy:
                c = lowest(x)
                go_on = c == tokens[at + i + 1]
            else:
                c = tokens[at + i + 1]
                q = torch.zeros_like(p)
                q[c] = 1.0
                if s["draft"] is not None:
                    q = torch.softmax(s["draft"][at + i].double() / T, -1)
                go_on = float(s["uniform"][at + i]) * float(q[c]) < float(p[c])
                if not go_on:
                    rest = (p - q).clamp(min=0)
                    rest = rest if float(rest.max()) > 0 else p
                    c = lowest(rest / s["noise"][b].double())
            emitted.append(c)
            logs.append(torch.log_softmax(x / T, -1)[c])
            if not go_on:
                break
        logs += [torch.zeros_like(logs[0])] * (m - len(emitted))
        accepted.append(len(emitted) - 1)
        out += emitted + [-1] * (m - len(emitted))
        at += m
    dev = s["logits"].device
    return (_i32(out, dev), _i32(accepted, dev),
            _i32([m - 1 - a for m, a in zip(n, accepted)], dev), torch.stack(logs))


def _exact_tables(s, case):
    page, n_pages, op = case["page"], s["n_pages"], case["op"]
    lens = s["lens"].tolist()
    width = s["table"].shape[1]
    rows = [t[:-(-k // page)] for t, k in zip(s["table"].tolist(), lens)]
    refs = [0] * n_pages
    for r in rows:
        for i in r:
            refs[i] += 1
    pairs = []

    def reserve(n):
        free = iter([i for i in range(n_pages) if refs[i] == 0])
        wanted = {}
        for b, m in enumerate(n):
            if m > 0 and lens[b] % page and refs[rows[b][-1]] > 1:
                wanted.setdefault(rows[b][-1], []).append(b)
        copying = set()
        for i, who in wanted.items():
            everyone = len(who) == refs[i]
            copying.update(who[1:] if everyone else who)
            refs[i] = 1 if everyone else refs[i] - len(who)
        for b, m in enumerate(n):
            if b in copying:
                i = next(free)
                pairs.append((rows[b][-1], i))
                rows[b][-1], refs[i] = i, 1
            lens[b] += m
            while len(rows[b]) * page < lens[b]:
                i = next(free)
                rows[b].append(i)
                refs[i] = 1

    if op == "step":
        for b, m in enumerate(s["drop"].tolist()):
            lens[b] = max(0, lens[b] - m)
            while (len(rows[b]) - 1) * page >= lens[b] and rows[b]:
                refs[rows[b].pop()] -= 1
        reserve(_rows(case))
        size = len(lens)
    elif op == "fork":
        before = [(list(r), k) for r, k in zip(rows, lens)]
        for b, a in enumerate(s["parents"].tolist()):
            if a != b:
                for i in rows[b]:
                    refs[i] -= 1
                rows[b], lens[b] = list(before[a][0]), before[a][1]
                for i in rows[b]:
                    refs[i] += 1
        reserve(_rows(case))
        size = len(lens)
    else:
        front = sum(x > 0 for x in refs)
        high = [i for i in range(front, n_pages) if refs[i] > 0]
        holes = [i for i in range(front) if refs[i] == 0]
        pairs = list(zip(high, holes))
        to = dict(pairs)
        rows = [[to.get(i, i) for i in r] for r in rows]
        for a, z in pairs:
            refs[z], refs[a] = refs[a], 0
        size = max(1, n_pages // 2)
    dev = s["table"].device
    out = [_i32([r + [-1] * (width - len(r)) for r in rows], dev), _i32(lens, dev),
           _i32(refs, dev), _i32(pairs + [(-1, -1)] * (size - len(pairs)), dev)]
    if op != "step":
        pool = s["pool"].view(torch.int64).clone()
        for a, z in pairs:
            pool[z] = s["pool"].view(torch.int64)[a]
        out.append(pool)
    return out
