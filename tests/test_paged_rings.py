"""The chunk kernel's roles as its present source orders them, restated on the host.

A query tile brings the next item's queries in as soon as the last scores of the item
at hand are there, before that item's output is complete.  The model runs the roles in
any order until nothing can move (a wait that can never end shows as a stall), and
checks what the early queries could break: that the tile's scores have all been issued
when its queries are overwritten, that scores are issued with their own item's queries,
and that an output is read before the next item's first sums replace it.
"""
import random

import pytest

from test_paged_plan import (AHEAD, ITEMS, SOURCE, STEPS, Stall, batches, cut, ring_items,
                             tiles_of)


def run_block(items, rng, early=True):
    """One block's roles over items = (two query tiles?, steps).  early: queries come in
    before the wait for the output, as in the kernel."""
    n_items = len(items)
    published, released = 0, [0] * n_items
    listed = fetched = 0                     # steps listed; read by the producers
    kfull = vfull = kfree = vfree = 0
    q, s, p, o = [0, 0], [0, 0], [0, 0], [0, 0]
    holds = [None, None]                     # the item whose queries a tile holds
    open_scores = [0, 0]                     # scores its item has yet to be issued
    unread = [False, False]                  # a complete output that was not read

    def list_warp():
        nonlocal published, listed
        for n in range(n_items + 1):
            if n >= ITEMS:
                yield lambda: released[n - ITEMS] == 3
            published += 1
            for _ in range(items[n][1] if n < n_items else 1):
                if listed >= AHEAD:
                    yield lambda: fetched > listed - AHEAD
                listed += 1
                yield None

    def producers():
        nonlocal kfull, vfull, fetched
        total = sum(n for _, n in items)
        yield lambda: listed > 0
        fetched = 1
        for n in range(total):
            yield lambda: n < 2 or kfree > n - 2
            kfull += 1
            yield lambda: listed > n + 1
            yield lambda: n < 2 or vfree > n - 2
            vfull += 1
            if n + 1 < total:
                fetched += 1

    def scores(i, n):
        assert holds[i] == n, "scores with another item's queries"
        open_scores[i] -= 1
        s[i] += 1

    def outputs(i, first, last):
        assert not (first and unread[i]), "an output was replaced before it was read"
        if last:
            o[i] += 1
            unread[i] = True

    def mma():
        nonlocal kfree, vfree
        kn = vn = 0
        used, pn = [0, 0], [0, 0]
        for n, (two, steps) in enumerate(items):
            yield lambda: published > n
            released[n] += 1
            for i in range(1 + two):
                used[i] += 1
                yield lambda: q[i] >= used[i]
            yield lambda: kfull > kn
            for i in range(1 + two):
                scores(i, n)
            kn += 1
            kfree += 1
            for j in range(steps):
                more = j + 1 < steps
                pn[0] += 1
                yield lambda: vfull > vn and p[0] >= pn[0]
                outputs(0, j == 0, not more)
                if not two:
                    vfree += 1
                if more:
                    yield lambda: kfull > kn
                    scores(0, n)
                if two:
                    pn[1] += 1
                    yield lambda: p[1] >= pn[1]
                    outputs(1, j == 0, not more)
                    vfree += 1
                    if more:
                        scores(1, n)
                vn += 1
                if more:
                    kfree += 1
                    kn += 1

    def tile(i):
        item = step = sn = on = 0
        cur = None

        def mine(n):
            return i == 0 or items[n][0]

        def queries(n):
            assert open_scores[i] == 0, "queries replaced before their last scores"
            holds[i], open_scores[i] = n, items[n][1]
            q[i] += 1

        while True:
            if cur is None:
                while True:
                    yield lambda: published > item
                    if item == n_items or mine(item):
                        break
                    step += items[item][1]
                    released[item] += 1
                    item += 1
                if item == n_items:
                    return
                cur = item
                queries(cur)
            for _ in range(items[cur][1]):
                sn += 1
                yield lambda: s[i] >= sn
                assert listed - step <= STEPS, "a step's entry was overwritten"
                p[i] += 1
                step += 1
                yield None
            this, nxt = item, None
            item += 1
            yield lambda: published > item
            if item < n_items and mine(item):
                nxt = item
            if nxt is not None and early:
                queries(nxt)
                yield None
            on += 1
            yield lambda: o[i] >= on
            if nxt is not None and not early:
                queries(nxt)
            yield None
            unread[i] = False
            released[this] += 1
            cur = nxt

    roles = [list_warp(), producers(), mma(), tile(0), tile(1)]
    waits = [None] * len(roles)
    alive = set(range(len(roles)))
    while alive:
        ready = [r for r in alive if waits[r] is None or waits[r]()]
        if not ready:
            raise Stall(alive)
        r = rng.choice(ready)
        for _ in range(rng.choice([1, 1, 4, 30])):
            try:
                waits[r] = next(roles[r])
            except StopIteration:
                alive.discard(r)
                break
            if waits[r] is not None and not waits[r]():
                break


def test_the_source_has_this_order():
    """Scores of all steps, the next item's queries, the output's wait, the release."""
    at = SOURCE.index("const uint32_t this_item = item++;")
    rest = SOURCE[at:]
    marks = [rest.index(x) for x in ("take_item(item)", "load_queries(next)", "scale_queries()",
                                     "queries_in()", "wait_warp(bar_o(i)",
                                     "bar_arrive_warp(bar_ie(this_item))")]
    assert marks == sorted(marks)
    assert SOURCE.rindex("bar_arrive_warp(bar_p(i))", 0, at) > SOURCE.rindex(
        "wait_warp(bar_s(i)", 0, at)


@pytest.mark.parametrize("early", (True, False))
@pytest.mark.parametrize("seed", range(40))
def test_rings_of_any_items(seed, early):
    rng = random.Random(seed)
    for _ in range(10):
        items = [(rng.random() < rng.choice([0.1, 0.5, 0.9]), rng.choice([1, 1, 2, 5, 30]))
                 for _ in range(rng.randint(1, 30))]
        run_block(items, rng, early)


@pytest.mark.parametrize("kv,new,rg,H", list(batches()))
def test_rings_of_whole_plans(kv, new, rg, H):
    rng = random.Random(len(kv))
    tiles = tiles_of(kv, new, rg, H)
    for blocks in (148, 152):
        for items in cut(tiles, blocks)[0]:
            run_block(ring_items(tiles, items), rng)
