"""The attention kernel's query slots beside an 8-bit cache, as a model whose
schedules are all tried: two slots, a scout that fills them, two softmax
warpgroups that convert the rows, wait for them and give the slots back, and the
MMA issuer. A barrier tells a waiter only the parity of its phase, as the
hardware's does, so a waiter must not fall two phases behind.

A warpgroup is one warp here, a tile's products are done when they are issued,
and the keys are always there: each of these only takes schedules away from a
waiter that the barriers of this model hold back, none from one they do not.
"""
import itertools

import pytest

# units: key tiles and whether they have two row tiles
ONE, TWO_TILES, THREE_TILES, PAIR = (1, False), (2, False), (3, False), (1, True)


def _items(seg, w):
    tiles, pair = seg
    return tiles if pair else (tiles + 1 - w) // 2


def programs(segs, wait_without_items):
    """Each actor's waits (barrier, number of the phase) and arrivals, in order."""
    scout, issuer, groups = [], [], ([], [])
    n = 0
    for seg in segs + [None]:
        for _ in range(2 if seg and seg[1] else 1):
            scout.append(("wait", f"q_empty{n & 1}", (n >> 1) - 1))
            scout.append(("arrive", f"q_full{n & 1}", 0))
            n += 1
    n_q = n_merge = 0
    item, n_seg = [0, 0], [0, 0]
    for seg in segs:
        slots = [n_q, n_q + 1] if seg[1] else [n_q]
        counts = [_items(seg, w) for w in range(2)]
        joined = not seg[1] and counts[1] > 0
        # issuer: scores run two items ahead of the products with the values
        issuer.append(("wait", f"q_full{n_q & 1}", n_q >> 1))
        for s in slots:
            issuer.append(("wait", f"q_ready{s & 1}", s >> 1))
        total = sum(counts)
        for i in range(min(2, total)):
            issuer.append(("arrive", f"s_full{i & 1}", 0))
        for i in range(total):
            w = i & 1
            issuer.append(("wait", f"p_ready{w}", item[w] + i // 2))
            if i + 2 >= total:
                issuer.append(("arrive", f"o_full{w}", 0))
            else:
                issuer.append(("arrive", f"s_full{w}", 0))
        for w, g in enumerate(groups):
            for s in slots:
                g.append(("wait", f"q_full{s & 1}", s >> 1))
            give = [("arrive", f"q_empty{s & 1}", 0) for s in slots]
            if counts[w] == 0:
                g.extend(give)
            mine = n_q + (w if seg[1] else 0)
            if seg[1] or w == 0:
                g.append(("arrive", f"q_ready{mine & 1}", 0))
            if counts[w] > 0 or wait_without_items:
                g.append(("wait", f"q_ready{mine & 1}", mine >> 1))
            for k in range(counts[w]):
                g.append(("wait", f"s_full{w}", item[w] + k))
                if k == counts[w] - 1:
                    g.extend(give)
                g.append(("arrive", f"p_ready{w}", 0))
            if counts[w] > 0:
                g.append(("wait", f"o_full{w}", n_seg[w]))
            if joined:
                if w == 1:
                    g.append(("arrive", "merge1", 0))
                    g.append(("wait", "merge0", n_merge))
                else:
                    g.append(("wait", "merge1", n_merge))
                    g.append(("arrive", "merge0", 0))
                g.append(("arrive", "merged", 0))
                g.append(("wait", "merged", n_merge))
        n_merge += joined
        for w in range(2):
            item[w] += counts[w]
            n_seg[w] += counts[w] > 0
        n_q += len(slots)
    return [scout, issuer, *groups]


def faults(segs, wait_without_items):
    """Over all schedules: a state in which nobody can go on, or a wait that let
    its actor pass in another phase than the one it waits for."""
    progs = programs(list(segs), wait_without_items)
    bars = sorted({op[1] for p in progs for op in p})
    at = {b: i for i, b in enumerate(bars)}
    count = [2 if b.startswith("q_empty") or b == "merged" else 1 for b in bars]
    start = (tuple([0] * len(progs)), tuple([0] * len(bars)), tuple(count))
    seen, todo, found = {start}, [start], set()
    while todo:
        pcs, phase, pending = todo.pop()
        moved = False
        for a, prog in enumerate(progs):
            if pcs[a] == len(prog):
                continue
            kind, bar, number = prog[pcs[a]]
            i = at[bar]
            ph, pe = phase, pending
            if kind == "wait":
                if (phase[i] & 1) == (number & 1):  # its parity has not passed
                    continue
                if phase[i] != number + 1:
                    found.add("a wait passed in another phase")
            else:
                left = pending[i] - 1
                if left == 0:
                    ph = phase[:i] + (phase[i] + 1,) + phase[i + 1:]
                    left = count[i]
                pe = pending[:i] + (left,) + pending[i + 1:]
            moved = True
            nxt = (pcs[:a] + (pcs[a] + 1,) + pcs[a + 1:], ph, pe)
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
        if not moved and any(pc < len(p) for pc, p in zip(pcs, progs)):
            found.add("a wait that never ends")
    return found


@pytest.mark.parametrize("segs", list(itertools.product((ONE, TWO_TILES, PAIR), repeat=4))
                         + [(ONE,) * 7, (THREE_TILES, ONE, ONE, ONE, THREE_TILES, ONE)])
def test_every_schedule_of_the_query_slots_ends(segs):
    assert faults(segs, wait_without_items=False) == set()


def test_the_model_sees_a_wait_behind_a_slot_that_was_given_back():
    """The second warpgroup of units of one tile, waiting for rows of a slot that
    it has given back: the slot can be filled and converted again before it looks."""
    assert "a wait that never ends" in faults((ONE,) * 4, wait_without_items=True)
