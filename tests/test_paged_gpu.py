"""The paged-cache operators on the GPU against their plain statements.

Tolerances (fixed before the first run). A rounding to a type t is off by at
most u_t = eps_t / 2, relative. An attention output rounds three things: the
probabilities (to fp16 for fp16 rows or an 8-bit cache, to bf16 otherwise),
which moves out by at most u_p * sum_j p_j |v_j|; the scores in fp32 (D products
and sums, scale and exponent), which move every p_j relatively by at most
e_x = 2 (D + 8) 2^-24 * max_j sum_d |scale q_d k_d| + 2^-18; and the output, by
u_out |out|. All sums are fp32 over at most a few thousand terms of one sign
for the mass: 2^-18 covers them. lse moves by e_x and its own fp32 rounding.
"""
import math
import random

import numpy as np
import pytest

import paged_oracle as po
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _half_eps(torch, dtype):
    return torch.finfo(dtype).eps / 2


# ---- block tables ---------------------------------------------------------------------


class Tables:
    """Device buffers of the tables and one call, checked against the oracle."""

    def __init__(self, torch, B, S, M, N, T, page, seed):
        self.torch, self.page, self.T = torch, page, T
        self.r = random.Random(seed)
        free = list(range(N))
        self.r.shuffle(free)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.i32 = i32
        self.table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
        self.held, self.cached = i32([0] * S), i32([0] * S)
        self.free, self.pool = i32(free), i32([N, 0])
        self.start, self.seq = i32([-7] * (B + 1)), i32([-7] * B)
        self.pos = torch.full((T,), -7, dtype=torch.int64, device="cuda")
        self.slot = torch.full((T,), -7, dtype=torch.int64, device="cuda")
        self.status = i32([0])

    def step(self, rsi, new, num_accepted=None, stream=None):
        from verify_dspark_markov_step_gb300 import paged_tables
        before = [t.tolist() for t in (self.cached, self.table, self.held, self.free, self.pool)]
        self.status.zero_()
        acc = None if num_accepted is None else self.i32(num_accepted)
        paged_tables(self.i32(rsi), self.i32(new), self.cached, self.table, self.held, self.free,
                     self.pool, self.start, self.seq, self.pos, self.slot, self.page,
                     num_accepted=acc, status=self.status, stream=stream)
        self.torch.cuda.synchronize()
        want = po.tables(rsi, new, before[0], num_accepted, before[1], before[2], before[3],
                         before[4][0], self.T, self.page)
        assert self.start.tolist() == want["query_start"]
        assert self.seq.tolist() == want["seq_lens"]
        assert self.held.tolist() == want["held_blocks"]
        if num_accepted is None:
            assert self.cached.tolist() == before[0]
        else:
            assert self.cached.tolist() == want["cached_lens"]
        assert self.table.tolist() == want["block_table"]
        assert self.pool.tolist() == [len(want["stack"]), 0]
        assert self.free.tolist()[:len(want["stack"])] == want["stack"]
        assert self.pos.tolist() == want["positions"]
        assert self.slot.tolist() == want["slot_map"]
        got = self.status.item()
        assert got in want["status"] if want["status"] else got == 0
        return want


@pytest.mark.parametrize("B,S,M,page,big", [(1, 1, 40, 16, 300), (5, 9, 12, 16, 40),
                                            (32, 40, 30, 32, 200), (257, 300, 20, 128, 2000),
                                            (1024, 1024, 6, 256, 900)])
def test_tables_follow_the_statement_over_steps(B, S, M, page, big):
    """Random steps: growth, accepted drafts, shrinking, padding, more requests
    than blocks, more tokens than the maps hold, lengths past the table."""
    torch = require_gpu()
    N = max(4, S * M * 2 // 5)
    T = max(20, B * big // 3)
    d = Tables(torch, B, S, M, N, T, page, seed=B)
    r = d.r
    for step in range(12):
        rsi = r.sample(range(S), B)
        for _ in range(B // 8):
            rsi[r.randrange(B)] = -1
        new = [r.choice((0, 1, 8, r.randint(0, big))) for _ in rsi]
        acc = None
        if step % 3 == 1:
            acc = [r.choice((-1, -1, 0, 7)) for _ in rsi]
        if step % 4 == 3:
            d.cached.copy_(torch.tensor([r.choice((0, c // 2, c)) for c in d.cached.tolist()]))
        want = d.step(rsi, new, acc)
        if acc is None:
            cached = want["cached_lens"]
            for b, s in enumerate(rsi):
                if s >= 0 and want["seq_lens"][b]:
                    cached[s] = r.randint(cached[s], want["seq_lens"][b])
            d.cached.copy_(torch.tensor(cached))


def test_tables_bad_values_leave_the_request_alone():
    torch = require_gpu()
    d = Tables(torch, 6, 6, 8, 30, 64, 16, seed=3)
    d.step([0, 1, 2, 3, 4, 5], [5, 17, 0, 33, 1, 16])
    d.cached.copy_(torch.tensor([5, 17, 0, 33, 1, 16]))
    d.step([0, 99, 2, 3, 4, 5], [1] * 6)              # slot out of range
    d.step([0, 1, 2, 3, 4, 5], [1, -4, 1, 1, 1, 1])   # negative length
    d.step([0, 1, 2, 3, 4, 5], [1, 1, 1, 100, 1, 1])  # past the table
    d.step([0, 1, 2, 3, 4, 5], [1, 1, 1, 1, 1, 1], [-1, -5, -1, 0, 0, 0])
    d.cached[2] = -3
    d.step([0, 1, 2, 3, 4, 5], [1] * 6)
    d.cached[2] = 0
    d.held[4] = 9
    d.step([0, 1, 2, 3, 4, 5], [2] * 6)


def test_tables_of_an_empty_batch_and_of_no_tokens():
    torch = require_gpu()
    d = Tables(torch, 0, 3, 4, 9, 5, 16, seed=1)
    d.step([], [])
    d = Tables(torch, 2, 3, 4, 9, 0, 16, seed=1)
    d.step([1, -1], [0, 0])


def test_tables_step_and_its_taking_back_replay_in_a_graph():
    torch = require_gpu()
    from verify_dspark_markov_step_gb300 import paged_tables
    B, page, T = 40, 16, 40 * 300
    d = Tables(torch, B, B, 64, 2000, T, page, seed=9)
    d.step(list(range(B)), [13 + 7 * b for b in range(B)])
    d.cached.copy_(d.seq)
    rsi, new, zero = d.i32(list(range(B))), d.i32([290] * B), d.i32([0] * B)
    before = [t.clone() for t in (d.table, d.held, d.free, d.pool)]
    two = torch.full((2, T), -9, dtype=torch.int64, device="cuda")

    def both(stream):
        paged_tables(rsi, new, d.cached, d.table, d.held, d.free, d.pool, d.start, d.seq, two[0],
                     d.slot, page, status=d.status, stream=stream)
        paged_tables(rsi, zero, d.cached, d.table, d.held, d.free, d.pool, d.start, d.seq, d.pos,
                     two[1], page, status=d.status, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    want = d.slot.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both(s)
    for _ in range(3):
        d.slot.fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d.slot, want)
        for a, b in zip(before, (d.table, d.held, d.free, d.pool)):
            assert torch.equal(a, b)
    assert d.status.item() == 0 and (two[1] == -1).all()


# ---- append ----------------------------------------------------------------------------


def _pages(torch, N, H, P, D, dtype, layout, fill=None):
    """k_cache and v_cache [N, H, P, D] of a memory layout."""
    if layout == "heads":
        out = [torch.empty(N, H, P, D, dtype=torch.float32, device="cuda") for _ in range(2)]
    elif layout == "tokens":
        out = [torch.empty(N, P, H, D, dtype=torch.float32, device="cuda").transpose(1, 2)
               for _ in range(2)]
    else:  # keys and values of a block side by side, token-major
        kv = torch.empty(N, 2, P, H, D, dtype=torch.float32, device="cuda")
        out = [kv[:, i].transpose(1, 2) for i in range(2)]
    if fill is not None:
        for t in out:
            t.fill_(fill)
    if layout == "both":
        kv = kv.to(dtype)
        return [kv[:, i].transpose(1, 2) for i in range(2)]
    return [t.to(dtype, memory_format=torch.preserve_format) for t in out]


@pytest.mark.parametrize("T,H,D,page,dtype,cache,layout,fused", [
    (1, 1, 64, 16, "bfloat16", "bfloat16", "heads", False),
    (37, 3, 64, 32, "float16", "float16", "tokens", True),
    (130, 8, 128, 128, "bfloat16", "bfloat16", "both", True),
    (61, 5, 128, 256, "float16", "float8_e4m3fn", "both", False),
    (517, 4, 64, 64, "bfloat16", "float8_e4m3fn", "heads", True)])
def test_append_writes_the_rows_and_nothing_else(T, H, D, page, dtype, cache, layout, fused):
    torch = require_gpu()
    from verify_dspark_markov_step_gb300 import kv_append
    dt, cdt = getattr(torch, dtype), getattr(torch, cache)
    g = torch.Generator(device="cuda").manual_seed(T)
    N = -(-T // page) + 2
    kc, vc = _pages(torch, N, H, page, D, cdt, layout, fill=1.5)
    qkv = torch.randn(T, 3 * H * D, device="cuda", generator=g).to(dt)
    k, v = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (1, 2))
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    k[0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, -0.0])
    slots = torch.randperm(N * page, device="cuda", generator=g)[:T]
    slots[T // 2] = -1
    ks = vs = None
    if cache == "float8_e4m3fn":
        ks = 0.005 + 0.01 * torch.rand(H, device="cuda", generator=g)
        vs = None if T == 61 else 0.005 + 0.01 * torch.rand(H, device="cuda", generator=g)
    wants = [po.append(x, c, slots, s) for x, c, s in ((k, kc, ks), (v, vc, vs))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_append(k, v, kc, vc, slots, k_scale=ks, v_scale=vs, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for got, want in zip((kc, vc), wants):
        got = got.double()
        assert torch.equal(got.isnan(), want.isnan())
        if cache == dtype:
            assert torch.equal(got.nan_to_num(), want.nan_to_num())
        else:  # half a step of e4m3 (2^-4, below 2^-6: 2^-10), the division in fp32
            off = (got - want).nan_to_num().abs()
            assert (off <= (want.abs() * (2 ** -4 + 2 ** -23)).clamp(min=2 ** -10)
                    .nan_to_num()).all()


def test_append_past_the_cache_is_refused_on_the_device():
    torch = require_gpu()
    from verify_dspark_markov_step_gb300 import kv_append
    kc = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([5, 48, 1 << 40, -9], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_append(x, x, kc, vc, slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == -5
    for c in (kc, vc):
        assert (c[0, :, 5] == 1).all() and c.float().sum() == 2 * 64


# ---- attention --------------------------------------------------------------------------


class Attend:
    """A ragged batch with its cache; what no request holds is NaN."""

    def __init__(self, torch, lens, news, Hq, H, D, page, dtype="bfloat16", cache=None,
                 layout="heads", fused=False, pad_slots=(), seed=0, peak=2.0, extra_blocks=3):
        self.torch = torch
        dt = getattr(torch, dtype)
        cdt = getattr(torch, cache or dtype)
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        r = np.random.RandomState(seed)
        B = len(lens)
        self.B, self.lens, self.news = B, lens, news
        S = B + 2
        self.slots = [int(x) for x in r.permutation(S)[:B]]
        for b in pad_slots:
            self.slots[b] = -1
        M = max(1, max(-(-n // page) for n in lens))
        owns = [-(-n // page) for n in lens]
        N = sum(owns) + extra_blocks
        ids = r.permutation(N)
        self.table = np.full((S, M), -1)
        self.kc, self.vc = _pages(torch, N, H, page, D, cdt, layout, fill=math.nan)
        at = 0
        for b, s in enumerate(self.slots):
            row = ids[at:at + owns[b]]
            at += owns[b]
            if s < 0:
                continue
            self.table[s, :owns[b]] = row
            for j, i in enumerate(row):
                n = min(page, lens[b] - j * page)
                for c in (self.kc, self.vc):
                    x = torch.randn(H, n, D, device="cuda", generator=g)
                    c[int(i), :, :n] = (x * 96).clamp(-448, 448).to(cdt) \
                        if cdt == torch.float8_e4m3fn else x.to(cdt)
        self.ks = self.vs = None
        if cdt == torch.float8_e4m3fn:
            self.ks = 0.008 + 0.004 * torch.rand(H, device="cuda", generator=g)
            self.vs = 0.008 + 0.004 * torch.rand(H, device="cuda", generator=g)
        self.starts = [0] + [int(x) for x in np.cumsum(news)]
        T = self.starts[-1] + 3  # rows of no request at the end
        q = torch.randn(T, (Hq + 2 * H) * D, device="cuda", generator=g).mul_(peak).to(dt)
        self.q = q[:, :Hq * D].unflatten(1, (Hq, D))
        if not fused:
            self.q = self.q.contiguous()
        self.out = torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((T, Hq), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5
        self.dev = [torch.tensor(x, dtype=torch.int32, device="cuda")
                    for x in (self.table, self.slots, self.starts, lens)]

    def call(self, causal=True, window=0, stream=None, lse=True, ws=None):
        from verify_dspark_markov_step_gb300 import paged_attention
        paged_attention(self.q, self.kc, self.vc, *self.dev, self.out, scale=self.scale,
                        causal=causal, window=window, k_scale=self.ks, v_scale=self.vs,
                        lse=self.lse if lse else None, status=self.status, stream=stream,
                        workspace_buf=ws)

    def check(self, causal=True, window=0):
        torch = self.torch
        self.call(causal, window)
        torch.cuda.synchronize()
        assert self.status.item() == 0
        self.compare(causal, window)

    def compare(self, causal=True, window=0):
        torch = self.torch
        D = self.q.shape[2]
        out, lse, mass, slack = po.attention(
            self.q, self.kc, self.vc, self.table.tolist(), self.slots, self.starts, self.lens,
            self.scale, causal, window, self.ks, self.vs)
        n = self.starts[-1]
        assert (self.out[n:] == 7).all() and (self.lse[n:] == 7).all()
        e_x = (2 * (D + 8) * 2.0 ** -24 * slack[:n] + 2.0 ** -18)[..., None]
        f16 = self.q.dtype == torch.float16 or self.kc.dtype == torch.float8_e4m3fn
        u_p = _half_eps(torch, torch.float16 if f16 else torch.bfloat16)
        u_out = _half_eps(torch, self.q.dtype)
        got, want = self.out[:n].double(), out[:n]
        assert torch.equal(got.isnan(), want.isnan())
        room = (u_p + 2 * e_x) * mass[:n] * (1 + u_out) + u_out * want.abs() + 2.0 ** -24
        self.room = room
        off = (got - want).abs()
        worst = torch.where(want.isfinite(), off / room, 0.0).max().item() if n else 0.0
        assert worst <= 1.0, worst
        empty = lse[:n] == -math.inf
        assert torch.equal(empty, self.lse[:n] == -math.inf)
        assert (got[empty] == 0).all()
        dl = torch.where(lse[:n].isfinite(), (self.lse[:n].double() - lse[:n]).abs(), 0.0)
        assert (dl <= e_x[..., 0] + lse[:n].abs().nan_to_num(posinf=0, neginf=0) * 2.0 ** -22).all()
        return worst


CASES = [
    # single tokens: one head, grouped, many splits, lengths around the tiles
    dict(lens=[1], news=[1], Hq=1, H=1, D=64, page=16),
    dict(lens=[1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257], news=[1] * 11, Hq=8, H=2, D=128,
         page=16),
    dict(lens=[5000, 3, 0, 911], news=[1, 1, 0, 1], Hq=32, H=8, D=128, page=64, fused=True),
    dict(lens=[20011], news=[1], Hq=8, H=1, D=64, page=32, dtype="float16"),
    # verification steps, odd groups, a group of one, a group of 128
    dict(lens=[700, 64, 8, 1300], news=[8] * 4, Hq=28, H=4, D=128, page=16, dtype="float16"),
    dict(lens=[300, 333], news=[4, 3], Hq=15, H=3, D=64, page=128, layout="tokens"),
    dict(lens=[260, 7, 513], news=[5, 7, 2], Hq=3, H=3, D=128, page=256, layout="both"),
    dict(lens=[150, 90], news=[2, 1], Hq=128, H=1, D=128, page=32, fused=True),
    dict(lens=[150, 90], news=[3, 9], Hq=240, H=2, D=64, page=16, dtype="float16"),
    # prompts: whole, continued, ragged, mixed with single tokens
    dict(lens=[128], news=[128], Hq=2, H=2, D=64, page=16),
    dict(lens=[1000, 333, 1, 129], news=[1000, 200, 1, 129], Hq=4, H=2, D=128, page=16),
    dict(lens=[2048 + 77], news=[517], Hq=7, H=1, D=128, page=64, dtype="float16", fused=True),
    dict(lens=[400, 900, 80, 1500], news=[1, 300, 80, 2], Hq=12, H=2, D=64, page=32,
         layout="both"),
    # an 8-bit cache under both row types
    dict(lens=[600, 31, 1025], news=[4, 4, 1], Hq=16, H=2, D=128, page=32, cache="float8_e4m3fn"),
    dict(lens=[600, 450], news=[300, 1], Hq=8, H=2, D=64, page=16, dtype="float16",
         cache="float8_e4m3fn", layout="tokens"),
    dict(lens=[1500], news=[700], Hq=4, H=1, D=128, page=128, cache="float8_e4m3fn", fused=True),
    # padding, no tokens, fewer keys than tokens (rows that see nothing)
    dict(lens=[50, 60, 70], news=[2, 3, 4], Hq=4, H=2, D=128, page=16, pad_slots=(1,)),
    dict(lens=[3, 0, 40], news=[9, 5, 300], Hq=4, H=2, D=64, page=16),
]


def _ragged(B, lo, hi, new, seed):
    r = np.random.RandomState(seed)
    news = [int(x) for x in r.randint(1, new + 1, B)]
    return dict(lens=[n + int(x) for n, x in zip(news, r.randint(lo, hi + 1, B))], news=news)


# more requests than CTAs, more than threads of a CTA, units that end anywhere in a
# CTA's run, units of single and of two row tiles beside each other
MANY = [
    dict(**_ragged(40, 100, 3000, 9, 1), Hq=16, H=4, D=128, page=32),
    dict(**_ragged(40, 100, 3000, 9, 2), Hq=24, H=4, D=64, page=16, cache="float8_e4m3fn"),
    dict(**_ragged(60, 0, 2500, 3, 3), Hq=8, H=2, D=128, page=64, dtype="float16",
         cache="float8_e4m3fn", fused=True),
    dict(**_ragged(12, 0, 900, 700, 4), Hq=12, H=2, D=128, page=16, layout="tokens"),
    dict(**_ragged(9, 0, 500, 600, 5), Hq=5, H=1, D=64, page=128, cache="float8_e4m3fn"),
    dict(**_ragged(300, 0, 300, 2, 6), Hq=4, H=2, D=64, page=16),
    dict(**_ragged(1024, 0, 60, 1, 7), Hq=2, H=1, D=64, page=16),
    dict(**_ragged(500, 0, 1700, 1, 8), Hq=3, H=1, D=128, page=16, dtype="float16"),
]


@pytest.mark.parametrize("window", [0, 333])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_of_many_requests(case, window):
    torch = require_gpu()
    Attend(torch, seed=100 + case, **MANY[case]).check(True, window)


# many short requests of several key heads, an odd number of heads, heads that end a
# CTA's run, tables that can hold long requests (units may be cut) or cannot
HEADS = [
    dict(**_ragged(200, 0, 700, 1, 9), Hq=8, H=8, D=64, page=16, dtype="float16"),
    dict(**_ragged(200, 0, 700, 1, 10), Hq=8, H=8, D=64, page=64, dtype="float16",
         cache="float8_e4m3fn", fused=True),
    dict(**_ragged(150, 0, 500, 8, 11), Hq=20, H=5, D=128, page=32),
    dict(**_ragged(150, 0, 500, 8, 12), Hq=12, H=3, D=128, page=16, cache="float8_e4m3fn"),
    dict(**_ragged(90, 300, 2600, 4, 13), Hq=35, H=7, D=128, page=16, dtype="float16"),
    dict(**_ragged(90, 300, 2600, 4, 14), Hq=14, H=7, D=64, page=128, cache="float8_e4m3fn"),
    # one token tile, two of them and prompts beside each other
    dict(**_ragged(60, 0, 900, 90, 15), Hq=32, H=8, D=64, page=16),
]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 150)])
@pytest.mark.parametrize("case", range(len(HEADS)))
def test_attention_of_short_requests_and_many_heads(case, causal, window):
    torch = require_gpu()
    Attend(torch, seed=200 + case, **HEADS[case]).check(causal, window)


@pytest.mark.parametrize("table", [40, 4000])
@pytest.mark.parametrize("B,ctx,new,H", [(28, 900, 32, 4), (28, 1900, 16, 4), (3, 500, 300, 2),
                                         (1, 2, 700, 2), (150, 1500, 4, 4), (14, 2500, 8, 4)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 205)])
def test_attention_whether_units_are_split_or_not(B, ctx, new, H, causal, window, table):
    """Equal requests, for which units are kept whole or cut by how they fill the
    SMs, under tables that can hold short or long requests."""
    torch = require_gpu()
    a = Attend(torch, [ctx + new] * B, [new] * B, Hq=2 * H, H=H, D=64, page=64, seed=B)
    if table * 64 > ctx + new:
        a.dev[0] = torch.nn.functional.pad(a.dev[0], (0, table - a.dev[0].shape[1]), value=-1)
    a.check(causal, window)


@pytest.mark.parametrize("cache", [None, "float8_e4m3fn"])
def test_a_value_that_one_head_does_not_see_stays_out_of_all(cache):
    """A NaN in one key head's values, at the last token of every third request:
    earlier rows of that head and all rows of the others keep their results."""
    torch = require_gpu()
    a = Attend(torch, seed=31, cache=cache, **_ragged(120, 0, 400, 6, 16), Hq=12, H=6, D=64,
               page=16)
    a.check()
    clean = a.out.clone()
    for b in range(0, a.B, 3):
        last = a.lens[b] - 1
        a.vc[int(a.table[a.slots[b], last // 16]), b % 6, last % 16, 11] = math.nan
    a.call()
    torch.cuda.synchronize()
    for b in range(a.B):
        rows, h = slice(a.starts[b], a.starts[b + 1]), b % 6
        got, was = a.out[rows].clone(), clean[rows].clone()
        if b % 3 == 0:
            assert got[-1, 2 * h:2 * h + 2, 11].isnan().all()
            got[-1, 2 * h:2 * h + 2, 11] = was[-1, 2 * h:2 * h + 2, 11]
            # (that head's products may be summed in another order: compared below)
            got[:, 2 * h:2 * h + 2] = was[:, 2 * h:2 * h + 2]
        assert torch.equal(got, was)
    a.compare()


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 37), (False, 130)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_follows_the_definition(case, causal, window):
    torch = require_gpu()
    Attend(torch, seed=case, **CASES[case]).check(causal, window)


@pytest.mark.parametrize("peak", [0.0, 60.0, 3000.0])
@pytest.mark.parametrize("dtype,cache", [("bfloat16", None), ("float16", None),
                                         ("bfloat16", "float8_e4m3fn")])
def test_attention_of_flat_and_of_peaked_scores(peak, dtype, cache):
    """All keys equal, and scores far apart (one key takes everything): the
    running maximum moves by much between tiles."""
    torch = require_gpu()
    Attend(torch, [900, 300], [3, 290], Hq=8, H=2, D=128, page=16, dtype=dtype, cache=cache,
           peak=peak, seed=4).check()


@pytest.mark.parametrize("dtype,scale", [("bfloat16", 1e30), ("bfloat16", 1e-30),
                                         ("float16", 30000.0)])
def test_attention_rows_of_extreme_size(dtype, scale):
    """Query rows near the end of their type's range over an 8-bit or 16-bit
    cache, brought back by the softmax scale."""
    torch = require_gpu()
    for cache in (None, "float8_e4m3fn"):
        a = Attend(torch, [400], [5], Hq=4, H=2, D=128, page=16, dtype=dtype, cache=cache, seed=8)
        a.q.copy_((a.q.float() * (scale / 16)).to(a.q.dtype))
        a.scale = a.scale * 16 / scale
        a.check()


def test_attention_negative_and_zero_scale():
    torch = require_gpu()
    for scale in (-0.3, 0.0):
        a = Attend(torch, [400, 260], [5, 200], Hq=4, H=2, D=64, page=16, seed=8)
        a.scale = scale
        a.call()
        torch.cuda.synchronize()
        out, lse, mass, slack = po.attention(a.q, a.kc, a.vc, a.table.tolist(), a.slots, a.starts,
                                             a.lens, scale)
        n = a.starts[-1]
        e_x = 2 * (64 + 8) * 2.0 ** -24 * 64 * 8 * abs(scale) * 4 + 2.0 ** -18
        room = (2.0 ** -8 + 2 * e_x) * mass[:n] + 2.0 ** -8 * out[:n].abs() + 2.0 ** -24
        assert ((a.out[:n].double() - out[:n]).abs() <= room).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("cache", [None, "float8_e4m3fn"])
def test_what_a_row_does_not_see_does_not_reach_it(bad, cache):
    """Keys and values of later tokens, and of tokens before the window, hold
    NaN or infinities: only the rows that see them change."""
    torch = require_gpu()
    if cache and math.isinf(bad):
        pytest.skip("an 8-bit cache holds no infinities")
    for news, lens in (([8], [300]), ([150], [150]), ([260], [700])):
        a = Attend(torch, lens, news, Hq=8, H=2, D=128, page=16, cache=cache, seed=2)
        a.check(True, 100)
        clean, clean_lse, room = a.out.clone(), a.lse.clone(), a.room
        n = news[0]
        spot = lens[0] - 3  # the position of row n - 3
        page = int(a.table[a.slots[0], spot // 16])
        a.kc[page, 1, spot % 16, 5] = bad
        a.vc[page, 1, spot % 16, 9] = bad
        early = max(0, lens[0] - n - 140)
        page = int(a.table[a.slots[0], early // 16])
        if early < lens[0] - n - 100:
            a.vc[page, 0, early % 16, 3] = bad
            a.kc[page, 0, early % 16, 3] = bad
        a.call(True, 100)
        torch.cuda.synchronize()
        # (how the products of these rows are summed may depend on what is there)
        off = (a.out[:n - 3].double() - clean[:n - 3].double()).abs()
        assert (off <= 2 * room[:n - 3]).all()
        assert torch.equal(a.lse[:n - 3], clean_lse[:n - 3])
        assert torch.equal(a.out[n - 3:n, :4], clean[n - 3:n, :4])  # the other head
        if math.isnan(bad):
            assert a.out[n - 3:n, 4:].isnan().all() and a.lse[n - 3:n, 4:].isnan().all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_an_unseen_value_alone_does_not_reach_a_row(bad):
    """As above with the values alone: the rows that see the value get it where
    it is (their other columns stay), the others nothing."""
    torch = require_gpu()
    for news, lens in (([8], [300]), ([200], [420])):
        a = Attend(torch, lens, news, Hq=8, H=2, D=64, page=16, dtype="float16", seed=3)
        a.check()
        clean = a.out.clone()
        n = news[0]
        spot = lens[0] - 2
        page = int(a.table[a.slots[0], spot // 16])
        a.vc[page, 0, spot % 16, 7] = bad
        a.call()
        torch.cuda.synchronize()
        assert torch.equal(a.out[:n, 4:], clean[:n, 4:])  # the other head
        assert not a.out[n - 2:n, :4, 7].isfinite().any()
        a.compare()


def test_attention_reports_bad_pages_slots_and_lengths():
    """Values out of range never fault: the status says so, other requests are
    as they were."""
    torch = require_gpu()
    a = Attend(torch, [100, 200, 300], [2, 2, 2], Hq=4, H=2, D=64, page=16, seed=6)
    a.check()
    clean = a.out.clone()

    def broken(which, at, value):
        kept = a.dev[which].clone()
        a.dev[which].view(-1)[at] = value
        a.status.zero_()
        a.call()
        torch.cuda.synchronize()
        a.dev[which].copy_(kept)
        return a.status.item()
    M = a.table.shape[1]
    for value in (-1, a.kc.shape[0], 1 << 30, -(1 << 31)):
        assert broken(0, a.slots[1] * M + 2, value) == -5
        assert torch.equal(a.out[[0, 1, 4, 5]], clean[[0, 1, 4, 5]])
    assert broken(1, 1, a.table.shape[0]) == -5
    assert (a.out[2:4] == 0).all() and (a.lse[2:4] == -math.inf).all()
    assert torch.equal(a.out[[0, 1, 4, 5]], clean[[0, 1, 4, 5]])
    for value in (-1, M * 16 + 1, (1 << 31) - 1):
        assert broken(3, 1, value) == -5
        assert (a.out[2:4] == 0).all()
        assert torch.equal(a.out[[0, 1, 4, 5]], clean[[0, 1, 4, 5]])
    a.out.fill_(7)
    for value in (-2, a.q.shape[0] + 1, 1 << 30):
        assert broken(2, 3, value) == -5
        assert torch.equal(a.out[:4], clean[:4]) and (a.out[4:] == 7).all()
    a.status.zero_()
    a.check()


def test_attention_is_the_same_every_time_in_graphs_and_on_streams():
    torch = require_gpu()
    a = Attend(torch, [3000, 10, 1700], [4, 4, 200], Hq=8, H=2, D=128, page=32, seed=1)
    from verify_dspark_markov_step_gb300 import _lib
    ws = _lib.workspace(_lib.paged_attention_workspace_bytes(3, 8, 2, 128))
    ws.fill_(255)
    a.call(ws=ws)
    torch.cuda.synchronize()
    want, want_lse = a.out.clone(), a.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.out.fill_(7)
    torch.cuda.synchronize()
    a.call(stream=s)
    s.synchronize()
    assert torch.equal(a.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a.call(stream=s, ws=ws)
    for _ in range(3):
        a.out.fill_(7)
        a.lse.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want) and torch.equal(a.lse, want_lse)
    a.lse.fill_(5)
    a.call(lse=False)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want) and (a.lse == 5).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: appended to and read at its end."""
    torch = require_gpu()
    from verify_dspark_markov_step_gb300 import kv_append, paged_attention
    H, P, D = 8, 64, 128
    N = (1 << 32) // (H * P * D) + 40
    kc, vc = (torch.empty(N, H, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L = 5 * P - 3
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(L, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    ids = [N - 1, 0, N - 7, 3, N - 30]
    slots = torch.tensor([ids[t // P] * P + t % P for t in range(L)], device="cuda")
    kv_append(k, v, kc, vc, slots)
    torch.cuda.synchronize()
    for t in (0, 1, P, 2 * P + 5, L - 1):
        assert torch.equal(kc[ids[t // P], :, t % P], k[t])
        assert torch.equal(vc[ids[t // P], :, t % P], v[t])
    q = torch.randn(2, H, D, device="cuda", generator=g).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty_like(q)
    status = i32([0])
    paged_attention(q, kc, vc, i32([ids]), i32([0]), i32([0, 2]), i32([L]), out, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, _, mass, _ = po.attention(q, kc, vc, [ids], [0], [0, 2], [L], D ** -0.5)
    room = 2.0 ** -7 * mass + 2.0 ** -8 * want.abs()
    assert ((out.double() - want).abs() <= room).all()
