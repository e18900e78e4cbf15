"""Forking, freeing, compacting and copying on the GPU, against the plain statement."""
import random

import pytest
import torch

import paged_blocks_oracle as bo
import paged_oracle as po

pytestmark = pytest.mark.gpu


class Tables:
    """A cache's tables on the GPU and as lists, and the calls on both."""

    def __init__(self, S, M, N, page, sharing, rng, lens):
        self.S, self.M, self.N, self.page = S, M, N, page
        stack = list(range(N))
        rng.shuffle(stack)
        t = {"table": [[-1] * M for _ in range(S)], "held": [0] * S, "cached": [0] * S, "stack": stack,
             "shares": [0] * N if sharing else None, "N": N}
        for s, n in lens.items():
            for j in range(-(-n // page)):
                t["table"][s][j] = stack.pop()
            t["held"][s], t["cached"][s] = -(-n // page), n
        self.t = t
        self.upload()

    def upload(self):
        def ints(x):
            return torch.tensor(x, dtype=torch.int32, device="cuda")
        t = self.t
        self.table, self.held, self.cached = ints(t["table"]), ints(t["held"]), ints(t["cached"])
        self.free = ints(t["stack"] + [-7] * (self.N - len(t["stack"])))
        self.pool = ints([len(t["stack"]), 0])
        self.shares = None if t["shares"] is None else ints(t["shares"])
        self.copies = torch.full((self.N, 2), -3, dtype=torch.int32, device="cuda")
        self.count, self.status = ints([0]), ints([0])

    def compare(self, codes=(), copies=None):
        torch.cuda.synchronize()
        t = self.t
        got = self.status.item()
        assert got in codes if codes else got == 0, (got, codes)
        self.status.zero_()
        assert self.pool.tolist() == [len(t["stack"]), 0]
        assert self.free[:len(t["stack"])].tolist() == t["stack"]
        assert self.held.tolist() == t["held"] and self.cached.tolist() == t["cached"]
        assert self.table.tolist() == t["table"]
        if self.shares is not None:
            assert self.shares.tolist() == t["shares"]
        if copies is not None:
            assert self.count.item() == len(copies)
            assert [tuple(p) for p in self.copies[:len(copies)].tolist()] == copies

    def _common(self):
        return self.table, self.held, self.free, self.pool

    def fork(self, src, dst, max_copies=None):
        from verify_dspark_markov_step_gb300 import paged_fork
        ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst)]
        C = self.N if max_copies is None else max_copies
        table, held, free, pool = self._common()
        paged_fork(*ints, self.cached, table, held, free, pool, self.copies[:C], self.count, self.page,
                   shares=self.shares, status=self.status)
        copies, codes = bo.fork(self.t, src, dst, self.page, C)
        self.compare(codes, copies)
        return copies

    def give_up(self, slots):
        from verify_dspark_markov_step_gb300 import paged_free
        table, held, free, pool = self._common()
        paged_free(torch.tensor(slots, dtype=torch.int32, device="cuda"), self.cached, table, held, free, pool,
                   shares=self.shares, status=self.status)
        self.compare(bo.free(self.t, slots))

    def compact(self):
        from verify_dspark_markov_step_gb300 import paged_compact
        table, held, free, pool = self._common()
        paged_compact(table, held, free, pool, self.copies, self.count, shares=self.shares, status=self.status)
        copies = bo.compact(self.t)
        self.compare(copies=copies)
        return copies


@pytest.mark.parametrize("sharing", [False, True])
@pytest.mark.parametrize("S,M,N,page,most", [(6, 4, 40, 16, 4), (40, 130, 3000, 32, 12), (1030, 9, 9000, 16, 1024),
                                             (9, 1500, 9001, 64, 6), (3, 1, 2, 16, 3)])
def test_random_calls(S, M, N, page, most, sharing):
    """Many calls one after the other: padding, slots out of range or named twice, forks of
    forks, a stack that runs out."""
    for seed in range(3):
        rng = random.Random(seed * 100 + S)
        left, lens = N - 1, {}
        for s in rng.sample(range(S), S // 2):
            n = rng.choice((0, rng.randint(1, M * page), rng.randint(1, M) * page))
            if -(-n // page) <= left // 2:
                lens[s] = n
                left -= -(-n // page)
        x = Tables(S, M, N, page, sharing, rng, lens)
        x.compare()
        for _ in range(12):
            k = rng.choice((0, 1, rng.randint(1, most), most))
            what = rng.random()
            if what < 0.45:
                src, dst = ([rng.randint(-1, S) if rng.random() < 0.2 else rng.randrange(S) for _ in range(k)] for _ in range(2))
                if rng.random() < 0.6:  # forks that can be made, of few slots
                    empty = [s for s in range(S) if x.t["held"][s] == 0]
                    rng.shuffle(empty)
                    full = [s for s in range(S) if x.t["held"][s]] or [0]
                    dst = empty[:k]
                    src = [rng.choice(full[:3]) for _ in dst]
                x.fork(src, dst, rng.choice((None, None, max(0, N // 8))))
            elif what < 0.8:
                x.give_up([rng.randint(-1, S) for _ in range(k)] if rng.random() < 0.5 else rng.sample(range(S), min(k, S)))
            else:
                x.compact()
            bo.check(x.t)


@pytest.mark.parametrize("sharing", [False, True])
def test_forks_freed_in_their_order_leave_the_stack(sharing):
    rng = random.Random(4)
    x = Tables(20, 30, 700, 16, sharing, rng, {0: 477, 1: 16, 2: 300, 3: 0})
    stack = list(x.t["stack"])
    src, dst = [0, 1, 0, 2, 3, 0], [9, 5, 6, 12, 8, 15]
    x.fork(src, dst)
    x.give_up(dst)
    assert x.t["stack"] == stack


def test_sources_freed_before_their_forks():
    rng = random.Random(5)
    x = Tables(8, 40, 100, 16, True, rng, {0: 500, 1: 100})
    x.fork([0, 0, 1], [2, 3, 4])
    x.give_up([0])              # the prompt's blocks stay with the samples
    x.compact()
    x.fork([2], [0])
    x.give_up([2, 3, 0, 1, 4])  # shared blocks go once
    assert len(x.t["stack"]) == 100 and not any(x.t["shares"])


def test_tables_leave_shared_blocks():
    """A request whose length was lowered into its shared blocks is refused; one that grows
    past them, and shrinks back to them, is served."""
    from verify_dspark_markov_step_gb300 import paged_tables
    rng = random.Random(6)
    x = Tables(4, 20, 60, 16, True, rng, {0: 100})
    x.fork([0], [1])

    def plan(slot, new):
        out = [torch.zeros(n, dtype=d, device="cuda") for n, d in ((2, torch.int32), (1, torch.int32), (64, torch.int64), (64, torch.int64))]
        paged_tables(*(torch.tensor([v], dtype=torch.int32, device="cuda") for v in (slot, new)), x.cached, x.table, x.held,
                     x.free, x.pool, *out, 16, status=x.status, shares=x.shares)
        t = x.t
        want = po.tables([slot], [new], t["cached"], None, t["table"], t["held"], t["stack"] + [-7] * (60 - len(t["stack"])),
                         len(t["stack"]), 64, 16)
        return out, want

    def taken(want):
        x.t.update(table=want["block_table"], held=want["held_blocks"], cached=want["cached_lens"], stack=want["stack"])
    for slot, new in ((1, 40), (0, 7), (1, 0), (0, 0)):
        out, want = plan(slot, new)
        taken(want)
        x.compare()
        assert out[3].tolist() == want["slot_map"]
    x.cached[1] = x.t["cached"][1] = 90  # the fork's own last block goes back, six shared ones would stay
    _, want = plan(1, 0)
    taken(want)
    x.compare()
    x.cached[1] = x.t["cached"][1] = 30
    out, _ = plan(1, 0)
    assert x.status.item() == -5 and out[1].item() == 0
    x.status.zero_()
    x.compare()
    bo.check(x.t)
    # nor do new tokens come to lie in one, whether blocks go back or not
    for n, new in ((90, 1), (90, 60), (95, 1), (80, 16), (16, 64), (0, 64)):
        x.cached[1] = x.t["cached"][1] = n
        out, _ = plan(1, new)
        assert x.status.item() == -5 and out[1].item() == 0 and (out[3] == -1).all()
        x.status.zero_()
        x.compare()
    x.cached[1] = x.t["cached"][1] = 96
    _, want = plan(1, 20)
    taken(want)
    x.compare()
    bo.check(x.t)


def test_corrupt_tables_stay_in_bounds():
    """Entries, counts and lengths out of range are reported; nothing else changes hands."""
    x = Tables(6, 8, 50, 16, True, random.Random(7), {0: 100, 1: 50, 2: 20})
    from verify_dspark_markov_step_gb300 import paged_compact, paged_fork, paged_free
    x.table[0, 2], x.table[1, 0] = 77, -2
    src, dst = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1], [3, 4]))
    paged_fork(src, dst, x.cached, x.table, x.held, x.free, x.pool, x.copies, x.count, 16, shares=x.shares, status=x.status)
    assert x.status.item() == -5 and x.table[3, 2].item() == 77
    x.status.zero_()
    paged_free(dst, x.cached, x.table, x.held, x.free, x.pool, shares=x.shares, status=x.status)
    assert x.status.item() == -5 and x.held[3].item() == 0 and (x.table[3:5] == -1).all()
    x.status.zero_()
    x.free[0], x.held[5] = 1000, 99
    paged_compact(x.table, x.held, x.free, x.pool, x.copies, x.count, shares=x.shares, status=x.status)
    assert x.status.item() == -5 and x.table[0, 2].item() == 77
    x.status.zero_()
    x.pool[0] = 51
    x.held[5] = -1
    paged_compact(x.table, x.held, x.free, x.pool, x.copies, x.count, shares=x.shares, status=x.status)
    assert x.status.item() == -5 and 0 <= x.pool[0].item() <= 50


@pytest.mark.parametrize("layout", ["heads", "tokens", "pairs"])
@pytest.mark.parametrize("dtype,H,P,D,layers,N,n", [
    ("bf16", 8, 16, 128, 3, 60, 25), ("e4m3", 1, 16, 64, 1, 40, 20), ("fp16", 3, 32, 64, 2, 30, 1),
    ("e4m3", 5, 256, 128, 2, 12, 6), ("bf16", 2, 64, 128, 70, 10, 4), ("bf16", 8, 64, 128, 1, 400, 200)])
def test_copy(dtype, H, P, D, layers, N, n, layout):
    from verify_dspark_markov_step_gb300 import PagedCaches, paged_copy
    e = 1 if dtype == "e4m3" else 2
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}[dtype]
    g = torch.Generator("cuda").manual_seed(n)
    raw = torch.uint8 if e == 1 else torch.int16

    def some(*shape):
        return torch.randint(-100 if e == 2 else 0, 100, shape, device="cuda", generator=g, dtype=raw)
    made = []
    for _ in range(layers):
        if layout == "heads":
            made.append((some(N, H, P, D), some(N, H, P, D)))
        elif layout == "tokens":
            made.append(tuple(some(N, P, H, D).transpose(1, 2) for _ in range(2)))
        else:
            both = some(N, 2, H, P, D)
            made.append((both[:, 0], both[:, 1]))
    order = torch.randperm(N, device="cuda", generator=g)
    source, to = order[:n], order[n:2 * n]
    copies = torch.full((n + 3, 2), 10 ** 6, dtype=torch.int32, device="cuda")
    copies[:n, 0], copies[:n, 1] = source, to
    want = []
    for pair in made:
        want.append([])
        for c in pair:
            w = c.clone()
            w[to] = w[source]
            want[-1].append(w)
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    views = [tuple(c.view(dt) for c in pair) for pair in made]
    paged_copy(PagedCaches(views) if layers > 2 else views, copies, count, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for pair, expect in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(pair, expect))


def test_copy_of_bad_blocks():
    from verify_dspark_markov_step_gb300 import paged_copy
    k = torch.arange(6 * 16 * 64, device="cuda").to(torch.int16).view(6, 1, 16, 64).view(torch.float16)
    v = k.clone()
    before = k.clone()
    copies = torch.tensor([[0, 6], [-1, 2], [3, 4], [2 ** 31 - 1, 1]], dtype=torch.int32, device="cuda")
    for n, moved in ((4, True), (9, True), (-2, False), (0, False)):
        k.copy_(before), v.copy_(before)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        paged_copy([(k, v)], copies, torch.tensor([n], dtype=torch.int32, device="cuda"), status=status)
        assert status.item() == (0 if n == 0 else -5)
        want = before.view(torch.int16).clone()
        if moved:
            want[4] = want[3]
        assert torch.equal(k.view(torch.int16), want) and torch.equal(v.view(torch.int16), want)


def test_captured():
    """Fork, copies, free and compaction in one graph, replayed: each replay does the same
    to the state it finds."""
    from verify_dspark_markov_step_gb300 import paged_compact, paged_copy, paged_fork, paged_free
    x = Tables(6, 20, 90, 16, False, random.Random(8), {0: 250, 4: 77})
    k, v = (torch.randn(90, 2, 16, 64, device="cuda").half() for _ in range(2))
    src, dst = (torch.tensor([s], dtype=torch.int32, device="cuda") for s in (0, 1))
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")

    def step():
        for a, b in ((src, dst), (dst, src)):
            paged_fork(a, b, x.cached, x.table, x.held, x.free, x.pool, x.copies, x.count, 16, status=x.status)
            paged_copy([(k, v)], x.copies, x.count, status=x.status)
            paged_free(a, x.cached, x.table, x.held, x.free, x.pool, status=x.status)
            paged_compact(x.table, x.held, x.free, x.pool, x.copies, x.count, workspace_buf=ws, status=x.status)
            paged_copy([(k, v)], x.copies, x.count, status=x.status)

    def contents(s):
        n = x.t["held"][s]
        return k[x.table[s, :n].long()].clone(), v[x.table[s, :n].long()].clone()
    want = contents(0), contents(4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        for a, b in ((0, 1), (1, 0)):
            bo.fork(x.t, [a], [b], 16)
            bo.free(x.t, [a])
            bo.compact(x.t)
        x.compare()
        got = contents(0), contents(4)
        assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))
