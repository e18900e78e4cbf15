"""Norm and rotation of query and key rows, alone and with keys and values written into
their pages, against a statement in 64 bits."""
import random

import pytest
import torch

import qk_rope_oracle as qo
from verify_dspark_markov_step_gb300.rotary import Rotary

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _rows(T, heads, D, dt, g, spread=1.0):
    """A view of a fused projection: tokens further apart than their values."""
    x = torch.randn(T, (sum(heads) + 1) * D, device="cuda", generator=g).mul_(spread).to(dt)
    return [t.unflatten(1, (-1, D)) for t in x[:, D:].split([h * D for h in heads], 1)]


def _check(got, want, size, dtype, normed, live):
    got, ok = got.cpu().double(), live[:, None, None].expand(got.shape)
    off = (got - want).abs()
    bound = qo.room(want, size, dtype, normed)
    assert (off <= bound)[ok].all(), ((off / bound)[ok].max(), off[ok].max())


def _positions(T, far, rng, gone=()):
    p = [rng.randrange(far) for _ in range(T)]
    for i in gone:
        p[i % T] = -1 - rng.randrange(3)
    return torch.tensor(p, dtype=torch.int64)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,R,norm", [
    (1, 32, 8, 128, 128, "qk"), (1, 1, 0, 64, 64, ""), (2, 3, 1, 128, 64, "q"), (5, 7, 7, 64, 32, "k"),
    (37, 64, 8, 128, 64, "qk"), (300, 28, 4, 128, 128, ""), (19, 5, 2, 96, 48, "qk"), (3, 4, 2, 96, 96, ""),
    (11, 6, 3, 192, 64, "qk"), (9, 2, 1, 256, 256, "qk"), (7, 9, 2, 256, 16, ""), (13, 3, 5, 16, 16, "qk"),
    (4, 3, 2, 32, 16, "q"), (6, 10, 1, 48, 32, "qk"), (4100, 3, 1, 64, 64, "qk"), (21, 4, 4, 128, 0, "qk"),
    # several tokens a warp and a round
    (8192, 5, 1, 64, 64, "qk"), (8215, 1, 0, 128, 32, "q"), (8193, 9, 2, 96, 48, "k"), (8200, 2, 3, 256, 64, ""),
    (9001, 1, 1, 16, 16, "qk"), (8211, 17, 4, 128, 128, "qk"),
])
def test_rows(T, Hq, H, D, R, norm, interleaved, dtype):
    from verify_dspark_markov_step_gb300 import qk_rope
    dt = DT[dtype]
    rng = random.Random(T * 1000 + D + R)
    g = torch.Generator("cuda").manual_seed(T + D)
    q, k = _rows(T, (Hq, H), D, dt, g, 3.0)
    qw, kw = ((1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dt) if c in norm else None for c in "qk")
    positions = _positions(T, 200000, rng, gone=(T // 2, T - 1, T - 2) if T > 99 else (T // 2,) if T > 2 else ())
    rot = Rotary(R, 1e6, interleaved=interleaved) if R else None
    args = rot.args() if rot else {"interleaved": interleaved}
    q_out = torch.full_like(q.contiguous(), 7.0)
    k_out = torch.full((T, 2 * H, D), 7.0, device="cuda", dtype=dt)[:, H:]  # strided, too
    qk_rope(q, k if H else None, positions.cuda(), q_weight=qw, k_weight=kw, eps=1e-5, q_out=q_out,
            k_out=k_out if H else None, **args)
    torch.cuda.synchronize()
    live = positions >= 0
    for x, out, w in ((q, q_out, qw), (k, k_out, kw)):
        want, size = qo.rows(x.cpu(), positions.clamp(min=0), rot.turns.cpu() if rot else None, 1.0, interleaved,
                             None if w is None else w.cpu(), 1e-5)
        if x.shape[1]:
            _check(out, want, size, dt, w is not None, live)
            assert (out.cpu()[~live] == 7.0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles keep their fraction of a turn where 32 (and 53) bits have lost it."""
    from verify_dspark_markov_step_gb300 import qk_rope
    g = torch.Generator("cuda").manual_seed(5)
    positions = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31 + 5, 2 ** 40 + 12345, 2 ** 62 + 1], dtype=torch.int64)
    T = positions.numel()
    rot = Rotary(128, 1e4, {"type": "yarn", "factor": 4, "original_max_position": 4096}, interleaved=interleaved)
    q, k = _rows(T, (4, 2), 128, torch.float16, g)
    want = [qo.rows(x.cpu(), positions, rot.turns.cpu(), rot.factor, interleaved) for x in (q, k)]
    qk_rope(q, k, positions.cuda(), **rot.args())  # in place
    for x, (w, size) in zip((q, k), want):
        _check(x, w, size, torch.float16, False, positions >= 0)


def test_rotation_by_radians_and_relative_positions():
    """What the frequencies say in radians; and products of rotated rows depend on the
    positions' difference alone."""
    from verify_dspark_markov_step_gb300 import qk_rope
    g = torch.Generator("cuda").manual_seed(6)
    rot = Rotary(64, 5e5)
    x = torch.randn(1, 1, 64, device="cuda", generator=g).half()
    y = torch.randn(1, 1, 64, device="cuda", generator=g).half()
    p = torch.tensor([3, 1003, 50003], dtype=torch.int64)
    q, k = x.repeat(3, 1, 1), y.repeat(3, 1, 1)
    qk_rope(q, k, p.cuda(), **rot.args())
    t = p.double()[:, None] * torch.tensor(rot.radians, dtype=torch.float64)
    a, b = x.cpu().double()[..., :32], x.cpu().double()[..., 32:]
    want = torch.cat([a * t.cos()[:, None] - b * t.sin()[:, None], b * t.cos()[:, None] + a * t.sin()[:, None]], -1)
    assert ((q.cpu().double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -20 * 8).all()
    k2 = y.repeat(3, 1, 1)
    qk_rope(k2, None, (p + 17).cuda(), **rot.args())
    dots = (q.double() * k2.double()).sum(-1).flatten().cpu()
    # each of the 128 rounded factors is off by 2^-11 at most
    room = 2 * 2.0 ** -11 * (q.double() * k2.double()).abs().sum(-1).flatten().cpu().max() + 1e-3
    assert (dots - dots[0]).abs().max() <= 2 * room


def test_infinities_and_nan_stay_in_their_pairs():
    from verify_dspark_markov_step_gb300 import qk_rope
    rot = Rotary(32)
    q = torch.ones(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    q[0, 0, 3], q[0, 1, 40], q[1, 0, 63] = float("inf"), float("nan"), float("-inf")
    qk_rope(q, None, torch.tensor([5, 6], device="cuda"), **rot.args())
    bad = ~q.isfinite()
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 19]
    assert bad[0, 1].nonzero().flatten().tolist() == [40]
    assert bad[1, 0].nonzero().flatten().tolist() == [63]


def _cache(layout, N, H, P, D, dt, g):
    """k and v caches [N, H, P, D] in a layout, filled with something."""
    def some(*shape):
        x = torch.randn(shape, device="cuda", generator=g).to(torch.float16)
        return x.to(dt)
    if layout == "heads":
        return some(N, H, P, D), some(N, H, P, D)
    if layout == "tokens":
        return some(N, P, H, D).transpose(1, 2), some(N, P, H, D).transpose(1, 2)
    both = some(N, 2, H, P, D)
    return both[:, 0], both[:, 1]


@pytest.mark.parametrize("layout", ["heads", "tokens", "pairs"])
@pytest.mark.parametrize("dtype,cache,scaled", [("bf16", "bf16", False), ("fp16", "fp16", False), ("bf16", "e4m3", True),
                                                ("fp16", "e4m3", True), ("fp16", "e4m3", False), ("bf16", "bf16", True)])
@pytest.mark.parametrize("T,Hq,H,D,R,P,norm,interleaved", [
    (1, 32, 8, 128, 128, 16, True, False), (45, 5, 1, 64, 32, 32, True, True), (130, 16, 8, 128, 64, 64, False, False),
    (700, 4, 2, 64, 64, 256, True, False), (8197, 3, 1, 128, 64, 32, True, False), (8321, 9, 3, 64, 48, 64, False, True)])
def test_append(T, Hq, H, D, R, P, norm, interleaved, dtype, cache, scaled, layout):
    from verify_dspark_markov_step_gb300 import qk_rope_append
    dt = DT[dtype]
    ct = torch.float8_e4m3fn if cache == "e4m3" else dt
    rng = random.Random(T + P)
    g = torch.Generator("cuda").manual_seed(T)
    q, k, v = _rows(T, (Hq, H, H), D, dt, g, 2.0)
    N = -(-T // P) + 4
    kc, vc = _cache(layout, N, H, P, D, ct, g)
    before = kc.clone(), vc.clone()
    ks = vs = None
    if scaled:
        ks, vs = (0.01 + 0.01 * torch.rand(H, device="cuda", generator=g) for _ in range(2))
    w = [(1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dt) if norm else None for _ in range(2)]
    positions = _positions(T, 30000, rng, gone=(3, T // 3, T - 1) if T > 99 else (3,) if T > 9 else ())
    slots = torch.randperm(N * P, generator=torch.Generator().manual_seed(T))[:T]
    if T > 9:
        slots[5] = -1
    if T > 99:
        slots[T // 2:T // 2 + 9] = -1
    rot = Rotary(R, 1e5, interleaved=interleaved)
    q_out = torch.zeros(T, Hq, D, device="cuda", dtype=dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qk_rope_append(q, k, v, kc, vc, positions.cuda(), slots.cuda(), q_weight=w[0], k_weight=w[1], q_out=q_out, k_scale=ks,
                   v_scale=vs, status=status, **rot.args())
    assert status.item() == 0
    live = positions >= 0
    cpu = [None if x is None else x.cpu() for x in w]
    pos = positions.clamp(min=0)
    want, size = qo.rows(q.cpu(), pos, rot.turns.cpu(), 1.0, interleaved, cpu[0])
    _check(q_out, want, size, dt, norm, live)
    assert (q_out.cpu()[~live] == 0).all()
    stored = live & (slots >= 0)
    for x, got, old, s, weight, turn in ((k, kc, before[0], ks, cpu[1], rot), (v, vc, before[1], vs, None, None)):
        want, size = qo.rows(x.cpu(), pos, None if turn is None else turn.turns.cpu(), 1.0, interleaved, weight)
        if s is not None:
            want, size = (y / s.cpu().double()[None, :, None] for y in (want, size))
        flat = got.float().cpu().transpose(1, 2).reshape(N * P, H, D)
        was = old.float().cpu().transpose(1, 2).reshape(N * P, H, D)
        if cache == "e4m3":
            want = want.clamp(-448, 448)
        _check(flat[slots.clamp(min=0)].double(), want, size, ct, norm, stored)
        untouched = torch.ones(N * P, dtype=torch.bool)
        untouched[slots[stored]] = False
        assert torch.equal(flat[untouched], was[untouched])


@pytest.mark.parametrize("cache,scaled", [("bf16", False), ("bf16", True), ("e4m3", True), ("e4m3", False)])
def test_append_without_norm_and_rotation_is_kv_append(cache, scaled):
    """Bit for bit, infinities, NaN, saturating and tiny values and odd scales among them."""
    from verify_dspark_markov_step_gb300 import kv_append, qk_rope_append
    g = torch.Generator("cuda").manual_seed(9)
    T, H, D, P = 67, 4, 128, 16
    q, k, v = _rows(T, (4, H, H), D, torch.bfloat16, g)
    k *= 10.0 ** torch.randint(-6, 6, (T, 1, D), device="cuda", generator=g)
    k[1, 0, 5], k[2, 1, 6], v[3, 2, 7], v[4, 3, 8] = float("inf"), float("nan"), float("-inf"), 1e38
    ct = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    scale = torch.tensor([0.02, 1e-12, -3.0, 1e30], device="cuda") if scaled else None
    slots = torch.randperm(6 * P, device="cuda", generator=g)[:T]
    made = []
    for call in (0, 1):
        kc, vc = (torch.zeros(6, H, P, D, device="cuda", dtype=torch.bfloat16).to(ct) for _ in range(2))
        if call:
            kv_append(k, v, kc, vc, slots, k_scale=scale, v_scale=scale)
        else:
            q_out = torch.empty_like(q.contiguous())
            qk_rope_append(q, k, v, kc, vc, torch.zeros_like(slots), slots, k_scale=scale, v_scale=scale, q_out=q_out)
            assert torch.equal(q_out, q)
        made.append([c.view(torch.uint8 if cache == "e4m3" else torch.int16) for c in (kc, vc)])
    nan = [c.view(ct).float().isnan() for c in made[0]]
    for a, b, n in zip(*made, nan):
        assert torch.equal(n, b.view(ct).float().isnan())
        assert torch.equal(a[~n], b[~n])


def test_slot_past_the_cache():
    from verify_dspark_markov_step_gb300 import qk_rope_append
    kc, vc = (torch.zeros(2, 1, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.ones(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.ones(3, 1, 64, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([32, 4, 2 ** 40], device="cuda")
    q_out = torch.zeros_like(q)
    qk_rope_append(q, k, k, kc, vc, torch.zeros(3, dtype=torch.int64, device="cuda"), slots, q_out=q_out, status=status)
    assert status.item() == -5
    assert (q_out == 1).all()
    assert kc.sum().item() == 64 and (kc[0, 0, 4] == 1).all() and vc.sum().item() == 64


def test_captured_and_on_another_stream():
    from verify_dspark_markov_step_gb300 import qk_rope_append
    g = torch.Generator("cuda").manual_seed(12)
    rot = Rotary(64)
    q, k, v = _rows(33, (8, 2, 2), 128, torch.bfloat16, g)
    kc, vc = (torch.zeros(4, 2, 16, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pos = torch.arange(33, device="cuda")
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros(33, 8, 128, device="cuda", dtype=torch.bfloat16)

    def call(stream=None):
        qk_rope_append(q, k, v, kc, vc, pos, pos, q_weight=w, k_weight=w, q_out=out, stream=stream, **rot.args())
    call()
    want = out.clone(), kc.clone(), vc.clone()
    for x in (out, kc, vc):
        x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, kc, vc), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    q.mul_(2)  # the norm takes it back, exactly in 16 bits: eps is far below the squares
    pos.add_(0)
    for x in (out, kc, vc):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    off = (out.float() - want[0].float()).abs().max().item()
    # eps / mean square changes by a factor of 4 from 1e-6: 2^-20 of a value, one step of bf16 at most
    assert off <= 2.0 ** -7 * want[0].float().abs().max().item()
    assert torch.equal(vc, want[2])


def test_binding_refusals():
    from verify_dspark_markov_step_gb300 import _lib, qk_rope, qk_rope_append
    q = torch.zeros(4, 8, 128, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    rot = Rotary(64)
    for kw, what in (({"positions": pos.int()}, TypeError), ({"positions": pos[:3]}, ValueError),
                     ({"k": k[:3]}, ValueError), ({"k": k.half()}, ValueError), ({"q": q.float()}, TypeError),
                     ({"q": q[..., ::2]}, ValueError), ({"q": q.transpose(0, 1)}, ValueError), ({"q": q[0]}, ValueError),
                     ({"q_out": k}, ValueError), ({"k": None, "k_out": k}, ValueError),
                     ({"q_weight": q[0, 0, :64].contiguous()}, ValueError), ({"k_weight": torch.ones(128, device="cuda")}, TypeError),
                     ({"turns": rot.turns[:, None]}, ValueError), ({"turns": rot.turns.double()}, TypeError),
                     ({"turns": torch.zeros(72, dtype=torch.int64, device="cuda")}, _lib.DsparkError),
                     ({"turns": rot.turns[:12]}, _lib.DsparkError), ({"turns": rot.turns, "factor": float("inf")}, _lib.DsparkError),
                     ({"q_weight": q[0, 0], "eps": -1.0}, _lib.DsparkError), ({"q": q.expand(4, 8, 128)[:, :, :].as_strided((4, 8, 128), (0, 128, 1))}, _lib.DsparkError)):
        with pytest.raises(what):
            qk_rope(**{"q": q, "k": k, "positions": pos, **kw})
    cache = torch.zeros(2, 2, 16, 128, device="cuda", dtype=torch.bfloat16)
    for kw, what in (({"v": k[:3]}, ValueError), ({"k": q}, ValueError), ({"slot_map": pos[:3]}, ValueError),
                     ({"q": q[..., :64]}, ValueError), ({"v": k.half()}, ValueError), ({"k_cache": cache.half()}, ValueError)):
        with pytest.raises(what):
            qk_rope_append(**{"q": q, "k": k, "v": k.clone(), "k_cache": cache, "v_cache": cache, "positions": pos, "slot_map": pos, **kw})
    qk_rope(q[:0], k[:0], pos[:0], **rot.args())
    assert (q == 0).all()


def test_pages_past_32_bits_of_offset():
    """Blocks whose values lie more than 2^32 elements into the cache: written, and copied."""
    from verify_dspark_markov_step_gb300 import paged_copy, qk_rope_append
    N, H, P, D = 40000, 8, 256, 64  # 5.2e9 values
    k = torch.zeros(N, H, P, D, device="cuda", dtype=torch.float8_e4m3fn)
    v = torch.zeros(N, H, P, D, device="cuda", dtype=torch.float8_e4m3fn)
    q, kk, vv = (torch.ones(2, h, D, device="cuda", dtype=torch.bfloat16) for h in (3, H, H))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([(N - 1) * P + 255, 35000 * P + 3], device="cuda")
    qk_rope_append(q, kk, vv, k, v, torch.zeros(2, dtype=torch.int64, device="cuda"), slots, status=status)
    paged_copy([(k, v)], torch.tensor([[N - 1, 17], [35000, N - 2]], dtype=torch.int32, device="cuda"),
               torch.tensor([2], dtype=torch.int32, device="cuda"), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for c in (k, v):
        for block, at in ((N - 1, 255), (35000, 3), (17, 255), (N - 2, 3)):
            x = c[block].float()
            assert (x[:, at] == 1).all() and x.sum().item() == H * D
        assert c[0].float().sum().item() == 0 and c[N - 3].float().sum().item() == 0
