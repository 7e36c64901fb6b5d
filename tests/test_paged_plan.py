"""The chunk kernel's plan and its rings, restated on the host.

Blocks share the (sequence, head, 256-row tile) lists by a cut that every block
computes for itself, and inside a block the roles pass items and steps through
two small rings.  The model here runs the roles in any order until nothing can
move, so a wait that can never end shows as a stall, and reports a step's entry
that is overwritten before its last reader is done.  The constants are read from
the kernel's source.
"""
import os
import random
import re

import pytest

from bit_kv_cache_14_gb300 import build_lib

SOURCE = open(os.path.join(build_lib.CSRC, "kvq_paged_chunk.cu")).read()


def const(name):
    return int(re.search(r"constexpr int [^;]*\b%s = (\d+)" % name, SOURCE).group(1))


ITEMS, STEPS, AHEAD = const("kItems"), const("kSteps"), const("kAhead")
STEP, ROWS, OVER, MIN_UNITS = const("kStep"), const("kTileRows"), const("kOver"), const("kMinUnits")
PIECES = [6, 8, 12]


def ceil(a, b):
    return -(-a // b)


# ---- the cut ----------------------------------------------------------------

def tiles_of(kv, new, rg, H, few=8):
    """(sequence, head, rows of the tile, its steps), in the list's order."""
    out = []
    for b, (length, n) in enumerate(zip(kv, new)):
        rows = n * rg
        if rows <= few:
            continue
        for h in range(H):
            for first in range(0, rows, ROWS):
                last = min(first + ROWS, rows) - 1
                see = min(length - n + last // rg, length - 1) + 1
                out.append((b, h, min(rows - first, ROWS), max(1, ceil(see, STEP))))
    return out


def pieces_of(steps, size):
    return max(1, (steps + size // 2) // size)


def cut(tiles, blocks):
    """Per block its items (tile, first step, end step), as the kernel lists
    them, and per tile the blocks the kernel takes for its first and last."""
    for size in PIECES:
        if sum(pieces_of(t[3], size) for t in tiles) <= blocks:
            break
    else:
        size = 0
    cost = [pieces_of(t[3], size) if size else t[3] + OVER for t in tiles]
    start = [0]
    for c in cost:
        start.append(start[-1] + c)
    total = start[-1]
    U = 1 if size else max(ceil(total, blocks), MIN_UNITS)

    def border(c):
        x = c * U
        if x >= total:
            return total
        t = max(i for i in range(len(tiles)) if start[i] <= x)
        off = x - start[t]
        if size:
            return x
        if off <= OVER + 1:
            return x - off
        return x + cost[t] - off if cost[t] - off <= 1 else x

    plan, shares = [], []
    edges = [border(c) for c in range(blocks + 1)]
    t = 0
    for c in range(blocks):
        x0, x1 = edges[c], edges[c + 1]
        items, x = [], x0
        while x < x1:
            while start[t + 1] <= x:
                t += 1
            off, n = x - start[t], min(start[t + 1], x1) - x
            if size:
                j0, j1 = tiles[t][3] * off // cost[t], tiles[t][3] * (off + 1) // cost[t]
                c0, c1 = start[t], start[t + 1] - 1
            else:
                j0, j1 = max(off - OVER, 0), off + n - OVER
                c0, c1 = start[t] // U, (start[t + 1] - 1) // U
                if (c0 + 1) * U - start[t] <= OVER + 1:
                    c0 += 1
                if start[t + 1] - c1 * U <= 1:
                    c1 -= 1
            items.append((t, j0, j1))
            shares.append((c, t, j0, j1, c0, c1))
            x += n
        plan.append(items)
    return plan, shares


def lengths(rng, most=160):
    """Ragged batches of the sizes that make many items a block."""
    B = rng.choice([3, 20, 64, 128, 200])
    top = rng.choice([8, 40, 60, most, 600])
    new = [rng.choice([1, rng.randint(1, top)]) for _ in range(B)]
    return [n + rng.choice([0, rng.randint(0, 200), rng.randint(0, 3000)]) for n in new], new


@pytest.mark.parametrize("seed", range(60))
def test_every_step_has_one_block(seed):
    rng = random.Random(seed)
    kv, new = lengths(rng)
    tiles = tiles_of(kv, new, rng.choice([1, 4, 8]), rng.choice([1, 2, 8]))
    _, shares = cut(tiles, rng.choice([148, 152]))
    parts = {}
    for c, t, j0, j1, c0, c1 in shares:
        assert j0 < j1
        parts.setdefault(t, []).append((c, j0, j1, c0, c1))
    assert sorted(parts) == list(range(len(tiles)))
    for t, p in parts.items():
        assert p[0][1] == 0 and p[-1][2] == tiles[t][3]
        assert all(a[2] == b[1] and a[0] + 1 == b[0] for a, b in zip(p, p[1:]))
        if len(p) > 1:  # those that join it agree on who they are
            assert {x[3:] for x in p} == {(p[0][0], p[-1][0])}


# ---- the rings --------------------------------------------------------------

class Stall(Exception):
    pass


def run_block(items, rng, skip_ahead=False):
    """One block's roles over `items` = (two query tiles?, steps), each a
    generator that yields what it waits for.  Raises Stall when nothing can move.

    skip_ahead: query tile 1 looks on past items without rows for it before it
    releases the item it has finished."""
    n_items = len(items)
    published, released = [0], {}       # items listed; releases of each
    listed, fetched = [0], [0]          # steps listed; read by the producers
    kfull, kfree, vfull, vfree = [0], [0], [0], [0]
    q, s, p, o = [0, 0], [0, 0], [0, 0], [0, 0]

    def release(n):
        released[n] = released.get(n, 0) + 1

    def taken(n):
        return lambda: published[0] > n

    def list_warp():
        for n in range(n_items + 1):
            if n >= ITEMS:
                yield lambda: released.get(n - ITEMS, 0) == 3
            published[0] += 1
            for _ in range(items[n][1] if n < n_items else 1):
                if listed[0] >= AHEAD:
                    yield lambda: fetched[0] > listed[0] - AHEAD
                listed[0] += 1
                yield None

    def producers():
        total = sum(n for _, n in items)
        yield lambda: listed[0] > 0
        fetched[0] = 1
        for n in range(total):
            yield lambda: n < 2 or kfree[0] > n - 2
            kfull[0] += 1
            yield lambda: listed[0] > n + 1
            yield lambda: n < 2 or vfree[0] > n - 2
            vfull[0] += 1
            if n + 1 < total:
                fetched[0] += 1

    def mma():
        kn, vn, used, pn = 0, 0, [0, 0], [0, 0]
        for n, (two, steps) in enumerate(items):
            yield taken(n)
            release(n)
            for i in range(2 if two else 1):
                used[i] += 1
                yield lambda: q[i] >= used[i]
            yield lambda: kfull[0] > kn
            s[0] += 1
            s[1] += two
            kn += 1
            kfree[0] += 1
            for j in range(steps):
                more = j + 1 < steps
                pn[0] += 1
                yield lambda: vfull[0] > vn and p[0] >= pn[0]
                o[0] += not more
                vfree[0] += not two
                if more:
                    yield lambda: kfull[0] > kn
                    s[0] += 1
                if two:
                    pn[1] += 1
                    yield lambda: p[1] >= pn[1]
                    o[1] += not more
                    vfree[0] += 1
                    s[1] += more
                vn += 1
                if more:
                    kfree[0] += 1
                    kn += 1

    def tile(i):
        item = step = sn = on = 0
        mine = lambda n: i == 0 or items[n][0]  # noqa: E731
        cur = None
        while True:
            if cur is None:
                while True:
                    yield taken(item)
                    if item == n_items or mine(item):
                        break
                    step += items[item][1]
                    release(item)
                    item += 1
                if item == n_items:
                    return
                cur = item
                q[i] += 1
            for _ in range(items[cur][1]):
                sn += 1
                yield lambda: s[i] >= sn
                assert listed[0] - step <= STEPS, "a step's entry was overwritten"
                p[i] += 1
                step += 1
                yield None
            this, nxt = item, None
            item += 1
            yield taken(item)
            while skip_ahead and item < n_items and not mine(item):
                step += items[item][1]
                release(item)
                item += 1
                yield taken(item)
            if item < n_items and mine(item):
                nxt = item
            on += 1
            yield lambda: o[i] >= on
            if nxt is not None:
                q[i] += 1
            yield None
            release(this)
            cur = nxt

    roles = [list_warp(), producers(), mma(), tile(0), tile(1)]
    waits = [None] * len(roles)
    alive = set(range(len(roles)))
    while alive:
        ready = [r for r in alive if waits[r] is None or waits[r]()]
        if not ready:
            raise Stall(alive)
        # one role runs for a while, then another: fast and slow ones by chance
        r = rng.choice(ready)
        for _ in range(rng.choice([1, 1, 4, 30])):
            try:
                waits[r] = next(roles[r])
            except StopIteration:
                alive.discard(r)
                break
            if waits[r] is not None and not waits[r]():
                break


def ring_items(tiles, items):
    return [(tiles[t][2] > 128, j1 - j0) for t, j0, j1 in items]


def test_a_tile_that_skips_ahead_would_stall():
    """Why query tile 1 looks at one item only: holding a finished item, it
    would wait for entries that the ring refills once it has let go."""
    items = [(True, 1)] + [(False, 1)] * 4 + [(True, 1)]
    with pytest.raises(Stall):
        run_block(items, random.Random(0), skip_ahead=True)
    run_block(items, random.Random(0))
    assert "bar_arrive_warp(bar_ie(this_item))" in SOURCE


@pytest.mark.parametrize("seed", range(40))
def test_rings_of_any_items(seed):
    rng = random.Random(seed)
    for _ in range(10):
        items = [(rng.random() < rng.choice([0.1, 0.5, 0.9]), rng.choice([1, 1, 2, 5, 30]))
                 for _ in range(rng.randint(1, 30))]
        run_block(items, rng)


def batches():
    """The start of a ragged prefill: alternating and random short prompts."""
    yield [40, 20] * 64, [40, 20] * 64, 4, 8
    for seed in range(6):
        rng = random.Random(seed)
        kv, new = lengths(rng)
        yield kv, new, rng.choice([1, 2, 4]), rng.choice([1, 2, 8])


@pytest.mark.parametrize("kv,new,rg,H", list(batches()))
def test_rings_of_whole_plans(kv, new, rg, H):
    rng = random.Random(len(kv))
    tiles = tiles_of(kv, new, rg, H)
    for blocks in (148, 152):
        for items in cut(tiles, blocks)[0]:
            run_block(ring_items(tiles, items), rng)
