"""Attention over pages with a window and first tokens that stay visible, in 64 bits."""
import math

import torch


def visible(n, L, causal, window, sinks, device):
    """[n, L] truth values: what each of the last n of L tokens sees."""
    at = torch.arange(L, device=device).expand(n, L)
    pos = torch.arange(L - n, L, device=device)[:, None]
    sees = torch.ones(n, L, dtype=torch.bool, device=device)
    if window:
        sees = (at > pos - window) | (at < sinks)
    return sees & (at <= pos) if causal else sees


def attention(q, k_cache, v_cache, table, rsi, starts, lens, scale, causal=True, window=0,
              k_scale=None, v_scale=None, sinks=0):
    """(out, lse, mass, slack) as in paged_oracle.attention. Pages that the table does not
    have (-1) hold NaN."""
    T, Hq, D = q.shape
    H, P = k_cache.shape[1], k_cache.shape[2]
    G = Hq // H
    f64 = dict(dtype=torch.float64, device=q.device)
    out, lse = torch.full((T, Hq, D), math.nan, **f64), torch.full((T, Hq), math.nan, **f64)
    mass, slack = torch.zeros(T, Hq, D, **f64), torch.zeros(T, Hq, **f64)
    nothing = torch.full((P, D), math.nan, **f64)
    for b, s in enumerate(rsi):
        a, e = starts[b], starts[b + 1]
        n, L = e - a, lens[b] if s >= 0 else 0
        if n == 0:
            continue
        out[a:e], lse[a:e] = 0, -math.inf
        if L == 0:
            continue
        sees = visible(n, L, causal, window, sinks, q.device)
        some = sees.any(0)[:, None]
        for h in range(H):
            k, v = (torch.cat([nothing if i < 0 else c[i, h].double() for i in table[s][:-(-L // P)]])[:L]
                    for c in (k_cache, v_cache))
            k = k * (1.0 if k_scale is None else k_scale[h].double())
            v = v * (1.0 if v_scale is None else v_scale[h].double())
            rows = q[a:e, h * G:(h + 1) * G].double()
            k, vis = torch.where(some, k, 0.0), torch.where(some, v, 0.0)
            x = (torch.einsum("ngd,jd->ngj", rows, k) * scale).masked_fill(~sees[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
            if torch.isfinite(vis).all():
                o = torch.einsum("ngj,jd->ngd", p, vis)
            else:
                o = torch.stack([torch.where(sees[i][None, :, None], p[i][..., None] * v, 0.0).sum(1) for i in range(n)])
            out[a:e, h * G:(h + 1) * G], lse[a:e, h * G:(h + 1) * G] = o, z
            mass[a:e, h * G:(h + 1) * G] = torch.einsum("ngj,jd->ngd", p.nan_to_num(), vis.nan_to_num(posinf=0, neginf=0).abs())
            big = torch.einsum("ngd,jd->ngj", rows.abs(), k.abs().nan_to_num()) * abs(scale)
            slack[a:e, h * G:(h + 1) * G] = torch.where(sees[:, None], big, 0.0).amax(-1)
    return out, lse, mass, slack
