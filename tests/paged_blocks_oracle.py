"""Plain statements of forking, freeing and compacting: loops over lists, which the
calls change. A cache's tables are a dict: table (rows), held, cached, stack (from
the bottom), shares (or None), N."""


def fork(t, src, dst, page, max_copies=1 << 30):
    """The pairs to copy and the codes a device may report."""
    codes, copies, named, wanted = set(), [], [], 0
    have, S, M = len(t["stack"]), len(t["table"]), len(t["table"][0])
    for s, d in zip(src, dst):
        if s < 0 or d < 0:
            continue
        before, named = d in named, named + [d]
        if s >= S or d >= S or before or s in [y for x, y in zip(src, dst) if x >= 0]:
            codes.add(-5)
            continue
        n = t["cached"][s]
        need = -(-n // page)
        if n < 0 or not need <= t["held"][s] <= M or t["held"][d]:
            codes.add(-5)
            continue
        keep = n // page if t["shares"] is not None else 0
        wanted += need - keep
        if need > keep and wanted > have:
            codes.add(-9)
            continue
        if need > keep and wanted > max_copies:
            codes.add(-5)
            continue
        for j in range(need):
            block = t["table"][s][j]
            if j < keep:
                t["shares"][block] += 1
            else:
                copies.append((block, t["stack"].pop()))
                block = copies[-1][1]
            t["table"][d][j] = block
        t["held"][d], t["cached"][d] = need, n
    return copies, codes


def free(t, slots):
    codes, goes, seen = set(), [], set()
    for s in slots:
        if s < 0:
            continue
        if s >= len(t["table"]) or s in seen or not 0 <= t["held"][s] <= len(t["table"][0]):
            codes.add(-5)
            continue
        seen.add(s)
        goes.append((s, t["table"][s][:t["held"][s]]))
    holders = {}
    for _, row in goes:
        for block in row:
            holders[block] = holders.get(block, 0) + 1
    gone = {b for b, n in holders.items() if t["shares"] is None or t["shares"][b] + 1 == n}
    for s, row in reversed(goes):
        for block in reversed(row):
            if block in gone:
                gone.discard(block)
                t["stack"].append(block)
                if t["shares"] is not None:
                    t["shares"][block] = 0
            elif t["shares"] is not None and t["shares"][block] > 0 and holders[block] <= t["shares"][block]:
                t["shares"][block] -= 1
                holders[block] -= 1
        for j in range(t["held"][s]):
            t["table"][s][j] = -1
        t["held"][s] = t["cached"][s] = 0
    return codes


def compact(t):
    loose = set(t["stack"])
    used = t["N"] - len(loose)
    movers = [b for b in range(used, t["N"]) if b not in loose]
    holes = [b for b in range(used) if b in loose]
    to = dict(zip(movers, holes))
    for row, n in zip(t["table"], t["held"]):
        row[:n] = [to.get(b, b) for b in row[:n]]
    if t["shares"] is not None:
        for a, b in to.items():
            t["shares"][b], t["shares"][a] = t["shares"][a], 0
    t["stack"] = list(range(t["N"] - 1, used - 1, -1))
    return list(zip(movers, holes))


def check(t):
    """What always holds: a block is on the stack or in one row more than it has shares."""
    rows = {}
    for row, n in zip(t["table"], t["held"]):
        assert len(set(row[:n])) == n and all(0 <= b < t["N"] for b in row[:n])
        assert all(b == -1 for b in row[n:])
        for b in row[:n]:
            rows[b] = rows.get(b, 0) + 1
    assert len(set(t["stack"])) == len(t["stack"]) and not set(t["stack"]) & set(rows)
    for b in range(t["N"]):
        shares = 0 if t["shares"] is None else t["shares"][b]
        assert shares == max(0, rows.get(b, 0) - 1), (b, shares, rows.get(b))
