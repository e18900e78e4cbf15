"""Edges of the paged attention and append on the GPU. Bounds are those of
test_paged_gpu.py, whose ragged batches (``Attend``) these tests use."""
import math

import pytest

import paged_oracle as po
from gpu_util import require_gpu
from test_paged_gpu import Attend, _half_eps, _ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
def test_requests_of_one_key_tile_over_an_8_bit_cache(D, dtype):
    """Units of one key tile, several to a CTA (of one key head: each alone), of
    which a warpgroup has nothing to do, and longer ones between them: every call
    of many in a row gives the definition's result, the same bits each time."""
    torch = require_gpu()
    for seed, case in enumerate((_ragged(1000, 0, 120, 1, 21), _ragged(700, 0, 300, 3, 22))):
        a = Attend(torch, seed=seed, **case, Hq=4, H=1, D=D, page=16, dtype=dtype,
                   cache="float8_e4m3fn")
        a.check()
        want, want_lse = a.out.clone(), a.lse.clone()
        for _ in range(60):
            a.call()
        torch.cuda.synchronize()
        assert a.status.item() == 0
        assert torch.equal(a.out, want) and torch.equal(a.lse, want_lse)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 70), (False, 0)])
@pytest.mark.parametrize("small", [2.0 ** -10, 2.0 ** -40])
def test_a_zero_softmax_scale_over_an_8_bit_cache(small, causal, window):
    """Every visible key weighs the same, whatever the size of the query rows,
    the scales of the cache's heads and what is masked."""
    torch = require_gpu()
    a = Attend(torch, [400, 260, 0, 7], [5, 200, 0, 2], Hq=4, H=2, D=64, page=16, seed=8,
               cache="float8_e4m3fn")
    a.q.copy_((a.q.float() * small).to(a.q.dtype))
    a.scale = 0.0
    a.check(causal, window)


@pytest.mark.parametrize("cache", [None, "float8_e4m3fn"])
@pytest.mark.parametrize("H,D,news,lens", [
    (5, 64, [1] * 40, list(range(90, 490, 10))),       # heads side by side
    (5, 128, [3, 40, 1], [300, 90, 1300]),             # one row tile, cut units
    (5, 128, [200, 333], [200, 700])])                 # two row tiles
def test_scales_of_zero_and_below(cache, H, D, news, lens):
    """A head's scale multiplies what the cache stores, of either sign or zero."""
    torch = require_gpu()
    a = Attend(torch, lens, news, Hq=2 * H, H=H, D=D, page=32, cache=cache, seed=11)
    size = 0.01 if cache else 1.0
    a.ks = size * torch.tensor([1.25, -1.5, 0.0, -0.75, 1.0], device="cuda")
    a.vs = size * torch.tensor([-1.0, 1.5, 0.5, 0.0, -2.0], device="cuda")
    a.check()
    a.check(True, 100)


@pytest.mark.parametrize("dtype,cache", [("float16", None), ("float16", "float8_e4m3fn"),
                                         ("bfloat16", "float8_e4m3fn"), ("bfloat16", None)])
@pytest.mark.parametrize("lens,news", [([400, 700], [2, 5]), ([9000], [1]), ([300], [260])])
def test_scores_whose_fp32_steps_are_large(dtype, cache, lens, news):
    """Large queries and large keys, scores past 2^29: a key that fits a row takes
    all of it, every row is an average of its values, nothing overflows."""
    torch = require_gpu()
    H, G, D, page = 2, 2, 128, 16
    a = Attend(torch, lens, news, Hq=G * H, H=H, D=D, page=page, dtype=dtype, cache=cache, seed=12)
    g = torch.Generator(device="cuda").manual_seed(3)
    a.q.copy_(torch.randn(a.q.shape, device="cuda", generator=g) * 8000)
    if cache:
        a.ks = torch.full((H,), 50.0, device="cuda")
        fit = lambda row: 448.0 * row.sign()  # noqa: E731
    else:
        a.kc.copy_(torch.randn(a.kc.shape, device="cuda", generator=g) * 8000)
        fit = lambda row: row  # noqa: E731
    spots = {}  # (row, key head): the position of the key that fits the head's first query head
    for b in range(a.B):
        n, L, s = a.news[b], a.lens[b], a.slots[b]
        for i in range(min(n, 40)):
            for h in range(H):
                at = (37 * i + 211 * h + 5) % (L - n)
                t = a.starts[b] + i
                spots[t, h] = (int(a.table[s, at // page]), at % page)
    assert len(set((h, *p) for (t, h), p in spots.items())) == len(spots)
    for (t, h), (block, off) in spots.items():
        a.kc[block, h, off] = fit(a.q[t, h * G].float()).to(a.kc.dtype)
    a.call()
    torch.cuda.synchronize()
    assert a.status.item() == 0
    n = a.starts[-1]
    out, lse, mass, slack = po.attention(a.q, a.kc, a.vc, a.table.tolist(), a.slots, a.starts,
                                         a.lens, a.scale, True, 0, a.ks, a.vs)
    assert slack[:n].max() > 2.0 ** 29
    got = a.out[:n].double()
    assert got.isfinite().all() and a.lse[:n].isfinite().all()
    u_p = 2.0 ** -11 if dtype == "float16" or cache else 2.0 ** -8
    u = _half_eps(torch, a.q.dtype)
    top = max(a.vc[int(i), :, :min(page, a.lens[b] - j * page)].double().abs().max().item()
              for b in range(a.B) for j, i in enumerate(a.table[a.slots[b]]) if j * page < a.lens[b])
    top *= 1.0 if a.vs is None else a.vs.max().item()
    assert (got.abs() <= top * (1 + u_p + 2 * u)).all()
    for (t, h), (block, off) in spots.items():
        v = a.vc[block, h, off].double() * (1.0 if a.vs is None else a.vs[h].double())
        assert ((got[t, h * G] - v).abs() <= (u_p + u + 2.0 ** -20) * v.abs() + 2.0 ** -24).all()
    e_x = 2 * (D + 8) * 2.0 ** -24 * slack[:n] + 2.0 ** -18
    assert ((a.lse[:n].double() - lse[:n]).abs() <= e_x + lse[:n].abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("both", [True, False])
def test_append_divides_by_the_scales_of_a_16_bit_cache(dtype, both):
    """round(x / scale) to the cache's type, and attention over such a cache sees
    the rows that were appended."""
    torch = require_gpu()
    from verify_dspark_markov_step_gb300 import kv_append, paged_attention
    dt = getattr(torch, dtype)
    T, H, D, page = 300, 3, 64, 32
    g = torch.Generator(device="cuda").manual_seed(6)
    N = -(-T // page) + 1
    k, v, q = (torch.randn(T, H, D, device="cuda", generator=g).to(dt) for _ in range(3))
    kc, vc = (torch.full((N, H, page, D), 3.0, dtype=dt, device="cuda") for _ in range(2))
    ks = torch.tensor([0.3, 7.0, -1.7], device="cuda")
    vs = torch.tensor([1.9, 0.011, -3.0], device="cuda") if both else None
    edge = torch.tensor([math.nan, math.inf, -math.inf, -0.0], device="cuda").to(dt)
    last = k[T - 1, 1, :4].clone()
    k[T - 1, 1, :4] = edge
    slots = torch.arange(T, device="cuda") + page
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append():
        kv_append(k, v, kc, vc, slots, k_scale=ks, v_scale=vs, status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
    want = [po.append(x, c, slots, s) for x, c, s in ((k, kc, ks), (v, vc, vs))]
    append()
    u = _half_eps(torch, dt)
    for got, w in zip((kc, vc), want):
        got = got.double()
        assert torch.equal(got.isnan(), w.isnan())
        fin = w.isfinite()
        assert torch.equal(got[~fin].nan_to_num(), w[~fin].nan_to_num())
        # the quotient to fp32, then to 16 bits (fp16 below 2^-14: steps of 2^-24)
        off = (got - w)[fin].abs()
        assert (off <= w[fin].abs() * (u + 2.0 ** -23) + 2.0 ** -25).all()
    if not both:
        assert torch.equal(vc[1:].transpose(1, 2).reshape(-1, H, D)[:T], v)
    k[T - 1, 1, :4] = last
    append()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty_like(q)
    paged_attention(q, kc, vc, i32([list(range(1, N))]), i32([0]), i32([0, T]), i32([T]), out,
                    k_scale=ks, v_scale=vs, status=status)
    torch.cuda.synchronize()
    pages = [x.new_zeros(N, H, page, D) for x in (k, v)]
    for c, x in zip(pages, (k, v)):  # the rows as they were given
        c[1:] = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, (N - 1) * page - T)) \
            .view(N - 1, page, H, D).transpose(1, 2)
    want, _, mass, slack = po.attention(q, *pages, [list(range(1, N))], [0], [0, T], [T], D ** -0.5)
    # roundings of the keys move a score by u * slack, those of values, of
    # probabilities and of the output what they are
    e_x = (u + 2 * (D + 8) * 2.0 ** -24) * slack[..., None] + 2.0 ** -18
    room = (2 * e_x * (1 + e_x) + 2 * u) * mass * (1 + u) + u * want.abs() + 2.0 ** -24
    assert ((out.double() - want).abs() <= room).all()
