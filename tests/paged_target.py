"""A target for tests of the whole cached forward: ToyTarget with sharp attention and
an output head of its own, so that its logits depend on what the cache holds (under
the tied head a token's own embedding outweighs everything else), its logits in 64
bits, and the bound its 16-bit forward is held to."""
import math

import torch


def sensitive(target, seed=1):
    """Queries three times as large, a random head."""
    Hq, H, D = target.heads
    for w in target.qkv:
        w[:, :Hq * D] *= 3
    g = torch.Generator(device=target.embed.device).manual_seed(seed)
    target.head = (torch.randn(target.embed.shape, device=target.embed.device, generator=g)
                   * target.embed.shape[1] ** -0.5).to(target.embed.dtype)
    return target


def attend(p, v):
    return torch.einsum("hgnm,mhd->nhgd", p, v)


def logits(target, tokens, attend=attend, rounded=lambda t, what: t):
    """[n, V] for every position of a token list, in 64 bits; ``rounded(t, what)`` is
    applied to what a 16-bit forward rounds."""
    Hq, H, D = target.heads
    x = target.embed[torch.as_tensor(tokens, device=target.embed.device)].double()
    n = len(tokens)
    hidden = torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1)
    for wqkv, wo in zip(target.qkv, target.proj):
        q, k, v = rounded(x @ wqkv.double(), "rows").split((Hq * D, H * D, H * D), 1)
        q = q.reshape(n, H, Hq // H, D)
        k, v = (rounded(t.reshape(n, H, D), "cache") for t in (k, v))
        s = torch.einsum("nhgd,mhd->hgnm", q, k) * D ** -0.5
        p = rounded(s.masked_fill(hidden, -math.inf).softmax(-1), "rows")
        out = rounded(attend(p, v).reshape(n, Hq * D), "rows")
        x = rounded(x + rounded(out @ wo.double(), "rows"), "rows")
    return rounded(x @ target.head.double().T, "rows")


def room(want, cache_is_8_bit):
    """How far a logit may be off: the same roundings, restated on the CPU, move one of
    a few hundred positions by up to 0.051 of the logits' spread (0.51 with an e4m3
    cache); attention that is zero, negated, of other values, heads or weights by 2 or
    more in any four positions."""
    return want.std() * (1.5 if cache_is_8_bit else 0.2)
