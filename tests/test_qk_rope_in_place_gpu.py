"""Rows normalised and rotated where they lie, in batches of every path: the same bits as
into other rows, and nothing beside them."""
import random

import pytest
import torch

from test_qk_rope_gpu import DT, _cache, _positions
from verify_dspark_markov_step_gb300.rotary import Rotary

pytestmark = pytest.mark.gpu


def _fused(T, heads, D, dt, g):
    """A fused projection with something before, between and after its rows; views of them."""
    x = torch.randn(T, (sum(heads) + len(heads) + 1) * D, device="cuda", generator=g).to(dt)
    at, views = D, []
    for h in heads:
        views.append(x[:, at:at + h * D].unflatten(1, (-1, D)))
        at += (h + 1) * D
    return x, views


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,R,norm", [
    (3000, 9, 2, 128, 128, "qk"), (8191, 1, 1, 64, 64, "qk"), (8192, 1, 1, 64, 64, "qk"), (8193, 64, 8, 128, 128, "qk"),
    (8200, 5, 3, 96, 48, "q"), (8217, 1, 0, 16, 16, ""), (9000, 17, 4, 128, 64, ""), (16384, 2, 2, 128, 128, "k"),
    (20011, 3, 1, 256, 32, "qk"), (40000, 1, 1, 32, 32, ""), (33000, 8, 1, 128, 128, "qk"),
])
def test_long_batches(T, Hq, H, D, R, norm, interleaved, dtype):
    from verify_dspark_markov_step_gb300 import qk_rope
    dt = DT[dtype]
    g = torch.Generator("cuda").manual_seed(T + D)
    x, views = _fused(T, (Hq, H) if H else (Hq,), D, dt, g)
    q, k = views if H else (*views, None)
    qw, kw = ((1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dt) if c in norm else None for c in "qk")
    positions = _positions(T, 200000, random.Random(T), gone=(0, T // 2, T // 2 + 1, T - 1)).cuda()
    rot = Rotary(R, 1e6, interleaved=interleaved)
    outs = [None if t is None else t.contiguous() for t in (q, k)]
    call = dict(positions=positions, q_weight=qw, k_weight=kw, **rot.args())
    qk_rope(q, k, q_out=outs[0], k_out=outs[1], **call)
    want = x.clone()
    at = D
    for out in outs:
        if out is not None:
            want[:, at:at + out[0].numel()] = out.flatten(1)
            at += out[0].numel() + D
    qk_rope(q, k, **call)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


@pytest.mark.parametrize("cache,scaled", [("bf16", False), ("e4m3", True), ("bf16", True)])
@pytest.mark.parametrize("T,Hq,H,D,P", [(8192, 1, 1, 64, 16), (8205, 8, 1, 128, 32), (12000, 64, 8, 128, 64), (5000, 4, 2, 64, 16)])
def test_queries_beside_the_pages(T, Hq, H, D, P, cache, scaled):
    from verify_dspark_markov_step_gb300 import qk_rope_append
    ct = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    g = torch.Generator("cuda").manual_seed(T)
    x, (q, k, v) = _fused(T, (Hq, H, H), D, torch.bfloat16, g)
    before = x.clone()
    N = -(-T // P) + 2
    w = [(1 + 0.3 * torch.randn(D, device="cuda", generator=g)).bfloat16() for _ in range(2)]
    ks, vs = ((0.01 + 0.01 * torch.rand(H, device="cuda", generator=g)) if scaled else None for _ in range(2))
    positions = _positions(T, 30000, random.Random(T), gone=(3, T // 3, T - 1)).cuda()
    slots = torch.randperm(N * P, device="cuda", generator=g)[:T]
    slots[T // 2:T // 2 + 9] = -1
    rot = Rotary(64, 1e5)
    q_out = q.contiguous()
    made = []
    for out in (q_out, None):
        kc, vc = _cache("heads", N, H, P, D, ct, torch.Generator("cuda").manual_seed(1))
        qk_rope_append(q, k, v, kc, vc, positions, slots, q_weight=w[0], k_weight=w[1], q_out=out, k_scale=ks, v_scale=vs,
                       **rot.args())
        made.append([c.view(torch.uint8 if cache == "e4m3" else torch.int16) for c in (kc, vc)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*made))
    before[:, D:D + Hq * D] = q_out.flatten(1)
    assert torch.equal(x, before)


def test_rows_interleaved_with_those_that_are_read():
    """Rows of a wider buffer into others of it: apart, though the memory ranges meet."""
    from verify_dspark_markov_step_gb300 import _lib, qk_rope
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(50, 6, 64, device="cuda", generator=g).half()
    before, pos, rot = x.clone(), torch.arange(50, device="cuda"), Rotary(64)
    want = x[:, :3].contiguous()
    qk_rope(want, None, pos, **rot.args())
    qk_rope(x[:, :3], None, pos, q_out=x[:, 3:], **rot.args())
    torch.cuda.synchronize()
    assert torch.equal(x[:, 3:], want) and torch.equal(x[:, :3], before[:, :3])
    for q, out in ((x[:, :3], x[:, 2:5]), (x[:, 1:4], x[:, :3]), (x[:25, :3], x.view(25, 12, 64)[:, 5:8]),
                   (x[:, :3], x.as_strided((50, 3, 64), (128, 64, 1)))):
        with pytest.raises(_lib.DsparkError):
            qk_rope(q, None, pos[:q.shape[0]], q_out=out, **rot.args())
    assert torch.equal(x[:, :3], before[:, :3])
