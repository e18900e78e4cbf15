"""Rotation at far positions against angles worked out from the frequencies in radians, as
whole fractions, without the library's own table of turns."""
from fractions import Fraction

import pytest
import torch

import qk_rope_oracle as qo
from test_rotary_bounds_cpu import angle
from verify_dspark_markov_step_gb300.rotary import Rotary

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,scaling", [(1e4, None), (5e5, {"type": "linear", "factor": 8}),
                                          (1e4, {"type": "yarn", "factor": 4, "original_max_position": 4096})])
def test_far_positions_in_radians(base, scaling, interleaved):
    from verify_dspark_markov_step_gb300 import qk_rope
    positions = [1, 130000, 2 ** 24 + 1, 2 ** 31 + 5, 2 ** 36 + 11, 2 ** 40 + 12345, 2 ** 44 + 1]
    rot = Rotary(64, base, scaling, interleaved=interleaved)
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(len(positions), 3, 128, device="cuda", generator=g).half()
    t = torch.tensor([[angle(p, Fraction(w)) for w in rot.radians] for p in positions], dtype=torch.float64)
    c, s = t.cos()[:, None] * rot.factor, t.sin()[:, None] * rot.factor
    rows = x.cpu().double()
    a, b = (rows[..., 0:64:2], rows[..., 1:64:2]) if interleaved else (rows[..., :32], rows[..., 32:64])
    want, size = rows.clone(), rows.abs()
    for at, value in ((0, a * c - b * s), (1, b * c + a * s)):
        part = slice(at, 64, 2) if interleaved else slice(32 * at, 32 * at + 32)
        want[..., part] = value
        size[..., part] = (a.abs() + b.abs()) * rot.factor
    qk_rope(x, None, torch.tensor(positions, device="cuda"), **rot.args())
    # the turns are rounded to 2^-64: the angle is off by 2 pi p 2^-65 more
    room = qo.room(want, size, torch.float16, False)
    room += size * (6.2832 * 2.0 ** -65 * torch.tensor(positions, dtype=torch.float64))[:, None, None]
    off = (x.cpu().double() - want).abs()
    assert (off <= room).all(), (off / room).max()
