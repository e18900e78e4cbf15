"""Paged attention with a window and first tokens that stay visible, against its
definition in 64 bits, and what lies between them."""
import math
import random
from unittest import mock

import pytest

import paged_oracle as po
import paged_sinks_oracle as so
from gpu_util import require_gpu
from test_paged_gpu import Attend

pytestmark = pytest.mark.gpu


class Sinks(Attend):
    """A batch whose calls have `sinks`."""

    def __init__(self, *args, sinks, **kw):
        super().__init__(*args, **kw)
        self.sinks = sinks

    def call(self, causal=True, window=0, stream=None, lse=True, ws=None):
        from verify_dspark_markov_step_gb300 import paged_attention
        paged_attention(self.q, self.kc, self.vc, *self.dev, self.out, scale=self.scale, causal=causal, window=window,
                        sinks=self.sinks, k_scale=self.ks, v_scale=self.vs, lse=self.lse if lse else None,
                        status=self.status, stream=stream, workspace_buf=ws)

    def compare(self, causal=True, window=0):
        def attention(*a):
            return so.attention(*a, sinks=self.sinks)
        with mock.patch.object(po, "attention", attention):
            super().compare(causal, window)

    def poison(self, window, causal, drop):
        """NaN wherever no row of a request looks; with `drop` the tables lose pages that none looks at."""
        P = self.kc.shape[2]
        for b, s in enumerate(self.slots):
            L, n = self.lens[b], self.news[b]
            if s < 0 or not L or not n:
                continue
            seen = so.visible(n, L, causal, window, self.sinks, "cpu").any(0)
            for j in range(-(-L // P)):
                page = seen[j * P:(j + 1) * P]
                i = int(self.table[s, j])
                gone = (~page).nonzero().flatten().cuda()
                for c in (self.kc, self.vc):
                    eight = c.element_size() == 1
                    raw = c.view(self.torch.uint8) if eight else c
                    raw[i].index_fill_(1, gone, 127 if eight else math.nan)
                if drop and not page.any():
                    self.table[s, j] = -1
        self.dev[0] = self.torch.tensor(self.table, dtype=self.torch.int32, device="cuda")


CASES = [  # lens, news, Hq, H, D, page, dtype, cache, layout
    ([1, 700, 0, 2000, 35], [1, 1, 2, 1, 1], 8, 2, 128, 16, "bfloat16", None, "heads"),
    ([1500, 129, 4000, 128], [8, 8, 5, 8], 16, 2, 128, 64, "bfloat16", None, "tokens"),
    ([900, 2, 3000], [300, 5, 77], 7, 1, 64, 32, "float16", None, "both"),
    ([2100, 640], [1, 4], 32, 4, 128, 32, "bfloat16", "float8_e4m3fn", "heads"),
    ([777, 3333, 12], [13, 1, 12], 12, 3, 64, 256, "float16", "float8_e4m3fn", "tokens"),
    ([1290], [700], 28, 4, 128, 128, "float16", None, "heads"),
    ([5000, 300, 300, 301] + [260] * 20, [1] * 24, 8, 8, 64, 16, "bfloat16", None, "heads"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window,sinks", [(1, 1), (37, 4), (130, 100), (333, 128), (256, 129), (1000, 300), (100, 5000)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_follows_the_definition(case, window, sinks, causal):
    torch = require_gpu()
    lens, news, Hq, H, D, page, dtype, cache, layout = CASES[case]
    a = Sinks(torch, lens, news, Hq, H, D, page, dtype, cache, layout, fused=bool(case & 1), seed=case, sinks=sinks,
              pad_slots=(1,) if case == 4 else ())
    a.poison(window, causal, drop=True)
    a.check(causal, window)


@pytest.mark.parametrize("table", [0, 4000])
@pytest.mark.parametrize("B,ctx,new,H,window,sinks", [(28, 1900, 16, 4, 700, 40), (3, 2500, 300, 2, 500, 300), (64, 3000, 4, 8, 1024, 4),
                                                      (1, 9000, 1, 8, 4096, 4), (177, 800, 1, 4, 128, 16)])
def test_whether_units_are_split_or_not(B, ctx, new, H, window, sinks, table):
    torch = require_gpu()
    rng = random.Random(B)
    news = [rng.randint(1, new) for _ in range(B)]
    lens = [rng.randint(ctx // 2, ctx) + n for n in news]
    a = Sinks(torch, lens, news, 8, H, 64, 16, sinks=sinks, seed=B)
    if table:  # rows of the table so long that the units might be
        wide = torch.full((a.dev[0].shape[0], table), -1, dtype=torch.int32, device="cuda")
        wide[:, :a.dev[0].shape[1]] = a.dev[0]
        a.dev[0] = wide
    a.check(True, window)


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(seed):
    torch = require_gpu()
    rng = random.Random(seed)
    for _ in range(4):
        H = rng.choice((1, 2, 3, 8))
        G = rng.choice((1, 2, 5, 7, 16))
        D = rng.choice((64, 128))
        dtype = rng.choice(("bfloat16", "float16"))
        cache = rng.choice((None, None, "float8_e4m3fn"))
        news = [rng.choice((0, 1, 1, rng.randint(2, 20), rng.randint(30, 200))) for _ in range(rng.randint(1, 6))]
        lens = [max(0, n + rng.choice((-1, 0, 0, rng.randint(0, 100), rng.randint(0, 3000)))) for n in news]
        a = Sinks(torch, lens, news, H * G, H, D, rng.choice((16, 32, 64, 128, 256)), dtype, cache,
                  rng.choice(("heads", "tokens", "both")), seed=seed, sinks=rng.choice((1, 4, rng.randint(1, 600))))
        causal, window = rng.random() < 0.7, rng.choice((1, rng.randint(2, 300), rng.randint(100, 3000)))
        a.poison(window, causal, drop=rng.random() < 0.5)
        a.check(causal, window)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("cache", [None, "float8_e4m3fn"])
@pytest.mark.parametrize("window,sinks,where", [(300, 20, (20, 21, 127)), (40, 200, (255, 130)), (150, 128, (128, 200)), (64, 3, (5, 300))])
def test_a_value_that_some_rows_see_reaches_them_alone(window, sinks, where, cache, bad):
    """The window moves over it, the sinks end before it, in one tile with keys that all see."""
    torch = require_gpu()
    if cache and math.isinf(bad):
        pytest.skip("e4m3 has no infinities")
    a = Sinks(torch, [420, 200], [260, 50], 4, 2, 64, 16, "float16", cache, sinks=sinks)
    for b, s in enumerate(a.slots):
        for p in where:
            if p < a.lens[b]:
                a.vc[int(a.table[s, p // 16]), :, p % 16, 3] = bad
    a.call(True, window)
    torch.cuda.synchronize()
    for b in range(2):
        sees = so.visible(a.news[b], a.lens[b], True, window, sinks, "cuda")
        hit = torch.zeros(a.news[b], dtype=torch.bool, device="cuda")
        for p in where:
            if p < a.lens[b]:
                hit |= sees[:, p]
        out = a.out[a.starts[b]:a.starts[b + 1]].float()
        assert not out[hit][..., 3].isfinite().any()
        assert out[~hit].isfinite().all()
        keep = [d for d in range(64) if d != 3]
        assert out[..., keep].isfinite().all()


def test_without_a_window_and_without_sinks():
    """No window: sinks say nothing; no sinks: the same bits as before; sinks over all: the
    whole context."""
    torch = require_gpu()
    a = Sinks(torch, [1000, 40, 600], [3, 40, 1], 8, 2, 128, 16, sinks=7)
    made = []
    for sinks, window in ((7, 0), (0, 0), (0, 200), (10 ** 9, 200), (2 ** 31 - 1, 2 ** 31 - 1)):
        a.sinks = sinks
        a.call(True, window)
        torch.cuda.synchronize()
        a.compare(True, window)
        made.append((a.out.clone(), a.lse.clone()))
    assert torch.equal(made[0][0], made[1][0]) and torch.equal(made[0][1], made[1][1])
    assert torch.equal(made[4][0], made[1][0])
    plain = Attend.call
    a.sinks = 0
    plain(a, True, 200)
    torch.cuda.synchronize()
    assert torch.equal(a.out, made[2][0]) and torch.equal(a.lse, made[2][1])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_key_scales_of_a_16_bit_cache(dtype):
    torch = require_gpu()
    a = Sinks(torch, [900, 1300], [4, 30], 9, 3, 64, 32, dtype, sinks=33)
    a.ks = torch.tensor([0.5, -1.25, 0.0], device="cuda")
    a.vs = torch.tensor([2.0, -0.5, 1.0], device="cuda")
    a.check(True, 250)


def test_missing_page_among_the_sinks_is_reported():
    torch = require_gpu()
    a = Sinks(torch, [2000], [2], 4, 2, 64, 16, sinks=20)
    a.dev[0][a.slots[0], 50] = -1          # between sinks and window: nobody looks
    a.check(True, 100)
    a.dev[0][a.slots[0], 1] = 10 ** 6      # tokens 16 .. 31
    a.call(True, 100)
    torch.cuda.synchronize()
    assert a.status.item() == -5


def test_the_same_every_time_in_graphs_and_on_streams():
    torch = require_gpu()
    a = Sinks(torch, [9000, 500, 3000], [2, 9, 1], 32, 8, 128, 16, sinks=100)
    from verify_dspark_markov_step_gb300 import _lib
    ws = _lib.workspace(_lib.paged_attention_workspace_bytes(3, 32, 8, 128))
    a.call(True, 2000, ws=ws)
    torch.cuda.synchronize()
    want = a.out.clone(), a.lse.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.call(True, 2000, stream=side, ws=ws)
    for _ in range(3):
        a.out.fill_(3), a.lse.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        n = a.starts[-1]
        assert torch.equal(a.out[:n], want[0][:n]) and torch.equal(a.lse[:n], want[1][:n])
