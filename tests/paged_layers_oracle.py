"""ToyTarget with head norms, rotated positions and a window beside which the first
tokens stay visible: its logits in 64 bits, with the roundings of its 16-bit forward or
a mistake put in, and the bound that its forward is held to."""
import math

import torch

import paged_sinks_oracle as so


def sharp(target):
    """Attention that depends on what the cache holds: query weights three times as large,
    an output head of its own."""
    for i, (q, k) in enumerate(target.norms):
        target.norms[i] = (q * 3, k)
    g = torch.Generator(device=target.embed.device).manual_seed(1)
    target.head = (torch.randn(target.embed.shape, device=target.embed.device, generator=g)
                   * target.embed.shape[1] ** -0.5).to(target.embed.dtype)
    return target


def logits(target, tokens, rounded=lambda t, what: t, mistake=None):
    """[n, V] for every position of a token list. mistake: None, or what is done wrong."""
    Hq, H, D = target.heads
    dev = target.embed.device
    x = target.embed[torch.as_tensor(tokens, device=dev)].double()
    n = len(tokens)
    rot = target.rotary
    sinks = 0 if mistake == "no sinks" else target.sinks
    window = 0 if mistake == "no window" else target.window
    sees = so.visible(n, n, True, window, sinks, dev)
    at = torch.arange(n, device=dev, dtype=torch.float64)
    angle = at[:, None] * torch.tensor(rot.radians, dtype=torch.float64, device=dev)

    def turned(t, angle):
        R = rot.rotary_dim
        a, b = (t[..., 0:R:2], t[..., 1:R:2]) if rot.interleaved != (mistake == "other pairs") else (t[..., :R // 2], t[..., R // 2:R])
        c, s = (f(angle)[:, None] * rot.factor for f in (torch.cos, torch.sin))
        p, q = a * c - b * s, b * c + a * s
        both = torch.stack([p, q], -1).flatten(-2) if rot.interleaved != (mistake == "other pairs") else torch.cat([p, q], -1)
        return torch.cat([both, t[..., R:]], -1)

    def normed(t, w):
        return t / torch.sqrt(t.square().mean(-1, keepdim=True) + target.eps) * w.double()
    for (wqkv, wo), (qw, kw) in zip(zip(target.qkv, target.proj), target.norms):
        q, k, v = rounded(x @ wqkv.double(), "rows").split((Hq * D, H * D, H * D), 1)
        q, k, v = (t.reshape(n, -1, D) for t in (q, k, v))
        if mistake != "no norm of queries":
            q = normed(q, qw)
        if mistake != "no norm of keys":
            k = normed(k, kw)
        if mistake != "no rotation":
            q = turned(q, angle + (rot_step(rot, dev) if mistake == "queries one further" else 0))
            k = turned(k, angle)
        q, k, v = rounded(q, "rows").view(n, H, Hq // H, D), rounded(k, "cache"), rounded(v, "cache")
        s = torch.einsum("nhgd,mhd->hgnm", q, k) * D ** -0.5
        p = rounded(s.masked_fill(~sees, -math.inf).softmax(-1), "rows")
        out = rounded(torch.einsum("hgnm,mhd->nhgd", p, v).reshape(n, Hq * D), "rows")
        x = rounded(x + rounded(out @ wo.double(), "rows"), "rows")
    return rounded(x @ target.head.double().T, "rows")


def rot_step(rot, dev):
    return torch.tensor(rot.radians, dtype=torch.float64, device=dev)


MISTAKES = ("no sinks", "no window", "no rotation", "queries one further", "other pairs", "no norm of queries", "no norm of keys")


def room(want, cache_is_8_bit):
    """How far a logit may be off: the 16-bit forward's roundings, restated on the CPU, move
    none of them by a third of it, and every mistake above moves one by more."""
    return want.std() * (1.0 if cache_is_8_bit else 0.2)
