"""A step's tables of a cache with shared blocks: several requests, some of them lowered
into blocks that other rows hold, against the plain statement."""
import random

import pytest
import torch

import paged_oracle as po

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _made(B, S, M, page, rng, most):
    """Rows of blocks of which some runs are held by a second row too, with lengths lowered
    by more or less: lists, and what the step is to do with them."""
    held = [rng.randint(1, M) for _ in range(S)]
    N = sum(held) + S * 4
    stack = list(range(N))
    rng.shuffle(stack)
    table = [[stack.pop() for _ in range(h)] + [-1] * (M - h) for h in held]
    shares = [0] * N
    for row, h in zip(table, held):
        kind = rng.random()
        if kind < 0.3:  # a fork's: the first blocks
            for j in range(rng.randint(1, h)):
                shares[row[j]] = rng.randint(1, 3)
        elif kind < 0.6:  # one anywhere
            shares[row[rng.randrange(h)]] = 1
    slots = rng.sample(range(S), B)
    for i in range(B // 9):
        slots[rng.randrange(B)] = -1
    accepted = [rng.randint(-1, 5) for _ in range(B)]
    new = [rng.choice((0, 1, rng.randint(0, most))) for _ in range(B)]
    cached = [0] * S
    for b, s in enumerate(slots):
        if s >= 0:  # room for what is accepted and new
            top = max(0, min(held[s], M) * page - accepted[b] - 1 - new[b])
            cached[s] = rng.choice((top, max(0, top - rng.randint(0, 3 * page)), rng.randint(0, top)))
    return table, held, cached, stack, shares, slots, new, accepted, N


def _lies_in_shared(table, held, shares, first):
    return any(shares[i] > 0 for i in table[first:held])


@pytest.mark.parametrize("B,S,M,page,most", [(1, 3, 700, 16, 40), (5, 9, 300, 32, 60), (40, 60, 33, 16, 130),
                                             (300, 400, 9, 16, 20), (1024, 1100, 5, 64, 9), (8, 8, 5000, 16, 700)])
@pytest.mark.parametrize("accepts", [False, True])
def test_several_requests_over_several_ctas(B, S, M, page, most, accepts):
    from verify_dspark_markov_step_gb300 import paged_tables
    for seed in range(4):
        rng = random.Random(seed * 1000 + B)
        table, held, cached, stack, shares, slots, new, accepted, N = _made(B, S, M, page, rng, most)
        if not accepts:
            accepted = None
        T = sum(new) + 5000  # three CTAs and more
        refused = [False] * B
        for b, s in enumerate(slots):
            if s >= 0:
                c = cached[s] + (accepted[b] + 1 if accepts else 0)
                need = -(-(c + new[b]) // page)
                refused[b] = need <= M and _lies_in_shared(table[s], held[s], shares, c // page if new[b] else need)
        want = po.tables([-1 if r else s for s, r in zip(slots, refused)], new, cached, accepted, table, held,
                         stack + [-7] * (N - len(stack)), len(stack), T, page)
        dev = [_ints(x) for x in (cached, table, held, stack + [-7] * (N - len(stack)), [len(stack), 0])]
        out = [torch.full((n,), -9, dtype=d, device="cuda") for n, d in ((B + 1, torch.int32), (B, torch.int32), (T, torch.int64),
                                                                         (T, torch.int64))]
        status, counts = _ints([0]), _ints(shares)
        paged_tables(_ints(slots), _ints(new), *dev, *out, page, num_accepted=_ints(accepted) if accepts else None,
                     status=status, shares=counts)
        torch.cuda.synchronize()
        codes = want["status"] | ({-5} if any(refused) else set())
        assert status.item() in codes if codes else status.item() == 0
        assert B < 40 or any(refused) and not all(refused)
        assert out[0].tolist() == want["query_start"] and out[1].tolist() == want["seq_lens"]
        assert out[2].tolist() == want["positions"] and out[3].tolist() == want["slot_map"]
        assert dev[0].tolist() == want["cached_lens"] and dev[1].tolist() == want["block_table"]
        assert dev[2].tolist() == want["held_blocks"] and dev[4].tolist() == [len(want["stack"]), 0]
        assert dev[3][:len(want["stack"])].tolist() == want["stack"] and counts.tolist() == shares


@pytest.mark.parametrize("requests", [1, 40])
def test_a_long_row_lowered_to_its_start(requests):
    """65536 blocks to look at, the last one shared: refused, nothing changes, and soon (a
    block after the other takes milliseconds, by warps a fraction of one)."""
    from verify_dspark_markov_step_gb300 import paged_tables
    M = 65536
    N = M + requests
    held = [M] + [1] * (requests - 1)
    table = torch.full((requests, M), -1, dtype=torch.int32)
    table[0] = torch.arange(M)
    for s in range(1, requests):
        table[s, 0] = M + s
    shares = torch.zeros(N, dtype=torch.int32)
    shares[M - 1] = 1
    dev = [_ints([0] + [5] * (requests - 1)), table.cuda(), _ints(held), torch.full((N,), -7, dtype=torch.int32, device="cuda"),
           _ints([0, 0])]
    out = [torch.empty(n, dtype=d, device="cuda") for n, d in ((requests + 1, torch.int32), (requests, torch.int32),
                                                               (3 * requests, torch.int64), (3 * requests, torch.int64))]
    slots, new, status, shares = _ints(list(range(requests))), _ints([3] * requests), _ints([0]), shares.cuda()
    times = []
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        paged_tables(slots, new, *dev, *out, 16, status=status, shares=shares)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    assert status.item() == -5
    assert out[1].tolist() == [0] + [8] * (requests - 1)
    assert torch.equal(dev[1].cpu(), table) and dev[2].tolist() == held and dev[4].tolist() == [0, 0]
    assert min(times) < 2.0, times  # milliseconds
