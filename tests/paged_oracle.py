"""Plain statements of the paged-cache operators for their tests: the tables as
a loop over a real stack, the attention per request and head in 64 bits."""
from __future__ import annotations

import math

import torch


def tables(rsi, new, cached, num_accepted, table, held, free, count, T, page):
    """Lists in, lists out (the inputs are not changed): a dict of every output
    of dspark_paged_tables, and "status", the codes a device may report."""
    table, held, cached = [list(r) for r in table], list(held), list(cached)
    S, M = len(table), len(table[0])
    stack = list(free[:count])
    codes = set()
    todo = []
    spent = 0
    for b, s in enumerate(rsi):
        if s < 0:
            continue
        acc = -1 if num_accepted is None else num_accepted[b]
        if s >= S:
            codes.add(-5)
            continue
        c = cached[s] + acc + 1
        need = -(-(c + new[b]) // page)
        if acc < -1 or cached[s] < 0 or new[b] < 0 or not 0 <= held[s] <= M or need > M:
            codes.add(-5)
            continue
        spent += new[b]
        if new[b] and spent > T:
            codes.add(-5)
            continue
        todo.append((b, s, c, need))
    for b, s, c, need in reversed(todo):
        for j in range(held[s] - 1, need - 1, -1):
            stack.append(table[s][j])
    have, wanted = len(stack), 0
    for b, s, c, need in reversed(todo):
        for j in range(need, held[s]):
            table[s][j] = -1
    seq, starts, positions, slots = [0] * len(rsi), [], [], []
    served = {b: (s, c, need) for b, s, c, need in todo}
    for b in range(len(rsi)):
        starts.append(len(positions))
        if b not in served:
            continue
        s, c, need = served[b]
        take = max(0, need - held[s])
        wanted += take
        if take and wanted > have:
            codes.add(-9)
            continue
        for j in range(held[s], need):
            table[s][j] = stack.pop()
        held[s], cached[s], seq[b] = need, c, c + new[b]
        for p in range(c, c + new[b]):
            positions.append(p)
            slots.append(table[s][p // page] * page + p % page)
    starts.append(len(positions))
    pad = [-1] * (T - len(positions))
    return {"block_table": table, "held_blocks": held, "cached_lens": cached, "stack": stack,
            "query_start": starts, "seq_lens": seq, "positions": positions + pad,
            "slot_map": slots + pad, "status": codes}


def append(x, cache, slot_map, scale):
    """New contents of a cache (64 bits, before any rounding of an 8-bit cache)."""
    out = cache.double().clone()
    P = cache.shape[2]
    x = x.double()
    if scale is not None:
        x = x / scale.double()[:, None]
    if cache.dtype == torch.float8_e4m3fn:
        x = torch.where(x.isnan(), x, x.clamp(-448, 448))
    for t, at in enumerate(slot_map.tolist()):
        if at >= 0:
            out[at // P, :, at % P] = x[t]
    return out


def attention(q, k_cache, v_cache, table, rsi, starts, lens, scale, causal=True, window=0,
              k_scale=None, v_scale=None):
    """(out, lse, mass, slack) in 64 bits on q's device: mass is
    sum_j p_j |v_j| (what relative errors of the probabilities scale with),
    slack the sum of |scale q_d k_d| of the row's largest key (what rounding
    errors of the scores scale with). Rows of no request are NaN."""
    T, Hq, D = q.shape
    H, P = k_cache.shape[1], k_cache.shape[2]
    G = Hq // H
    f64 = dict(dtype=torch.float64, device=q.device)
    out, lse = torch.full((T, Hq, D), math.nan, **f64), torch.full((T, Hq), math.nan, **f64)
    mass, slack = torch.zeros(T, Hq, D, **f64), torch.zeros(T, Hq, **f64)
    for b, s in enumerate(rsi):
        a, e = starts[b], starts[b + 1]
        n, L = e - a, lens[b] if s >= 0 else 0
        if n == 0:
            continue
        out[a:e], lse[a:e] = 0, -math.inf
        if L == 0:
            continue
        ids = table[s][:-(-L // P)]
        at = torch.arange(L, device=q.device)[None]
        pos = torch.arange(L - n, L, device=q.device)[:, None]
        sees = (at <= pos) if causal else torch.ones(n, L, dtype=torch.bool, device=q.device)
        if window:
            sees = sees & (at > pos - window)
        for h in range(H):
            k = torch.cat([k_cache[i, h].double() for i in ids])[:L]
            v = torch.cat([v_cache[i, h].double() for i in ids])[:L]
            if k_scale is not None:
                k = k * k_scale[h].double()
            if v_scale is not None:
                v = v * v_scale[h].double()
            rows = q[a:e, h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,jd->ngj", rows, k) * scale
            x = torch.where(sees[:, None], x, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
            p = torch.where(sees[:, None], p, 0.0)
            # a value that no row sees stays out of the sums, NaN or not
            vis = torch.where(sees.any(0)[:, None], v, 0.0)
            if torch.isfinite(vis).all():
                o = torch.einsum("ngj,jd->ngd", p, vis)
            else:
                o = torch.stack([torch.where(sees[i][None, :, None], p[i][..., None] * v, 0.0).sum(1)
                                 for i in range(n)])
            out[a:e, h * G:(h + 1) * G] = o
            lse[a:e, h * G:(h + 1) * G] = z
            mass[a:e, h * G:(h + 1) * G] = torch.einsum("ngj,jd->ngd", p.nan_to_num(),
                                                        vis.nan_to_num(posinf=0, neginf=0).abs())
            big = torch.einsum("ngd,jd->ngj", rows.abs(), k.abs().nan_to_num()) * scale
            slack[a:e, h * G:(h + 1) * G] = torch.where(sees[:, None], big, 0.0).amax(-1)
    return out, lse, mass, slack
