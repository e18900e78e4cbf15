"""Plain statement in 64 bits of the rotating calls, and the bound they are held to."""
import torch


def angles(positions, turns):
    """[T, R/2] angles in radians, from whole numbers modulo 2^64."""
    at = [[(p * (t % 2 ** 64)) % 2 ** 64 for t in turns.tolist()] for p in positions.tolist()]
    signed = [[a - 2 ** 64 if a >= 2 ** 63 else a for a in row] for row in at]
    return torch.tensor(signed, dtype=torch.float64).view(len(signed), -1) * (torch.pi / 2.0 ** 63)


def rows(x, positions, turns=None, factor=1.0, interleaved=False, weight=None, eps=1e-6):
    """x [T, H, D] (CPU) normalised and rotated, in 64 bits; and the size that roundings
    in 32 bits are relative to."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
    size = x.abs()
    if turns is None:
        return x, size
    t = angles(positions, turns)
    R = 2 * t.shape[1]
    c, s = t.cos()[:, None] * factor, t.sin()[:, None] * factor
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    out, big = x.clone(), size.clone()
    p, q, m = a * c - b * s, b * c + a * s, (a.abs() + b.abs()) * abs(factor)
    if interleaved:
        out[..., 0:R:2], out[..., 1:R:2] = p, q
        big[..., 0:R:2], big[..., 1:R:2] = m, m
    else:
        out[..., :R // 2], out[..., R // 2:R] = p, q
        big[..., :R // 2], big[..., R // 2:R] = m, m
    return out, big


def room(want, size, dtype, normed):
    """Half a step of the stored type (of its smallest normal below that), and fp32
    roundings in units of 2^-24 of the operands' size. Without a norm: cosine and sine are
    off by 2 (the rest of a quarter turn rounded: pi/4; the series: 1/2; its last steps),
    the factor, products and the sum add 4: 8 covers them. With one: the sum of squares
    (16 in a row, then a tree of up to 4) is off by at most 20, half of it in the root, the
    root's reciprocal by 4, three products by 3: 32 covers both."""
    info = torch.finfo(dtype)
    least = info.smallest_normal * info.eps / 2
    return want.abs() * (info.eps / 2 * (1 + 2.0 ** -10)) + least + size * ((32 if normed else 8) * 2.0 ** -24)
