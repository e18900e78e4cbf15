"""The operators around the paged key/value cache, as measured cases.

Three operators of the target model's verification pass, which is what surrounds the Markov drafting step and
the rejection sampler: the block tables and slot map of a step, built on the GPU from the request lengths; the
step's new keys and values written into their pages; and the attention of the step's new tokens over the paged
cache. ``run`` computes each of them either in plain torch operations (``own`` false) or by the calls a user
makes of this package (``own`` true).

Lengths of a ragged batch are spread evenly over the case's ranges and dealt to the requests in an order that
the seed decides, so that the work of a case does not depend on the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}


def listed():
    return [
        # one verification step of 32 requests with 7 drafts each, prompts of about 22k tokens
        {"name": "tables_verify_32", "op": "tables", "B": 32, "ctx_lo": 22000, "ctx_hi": 23147, "new_lo": 8, "new_hi": 8, "page": 16},
        # a mixed batch of prompts and continuations, the most tokens one step plans
        {"name": "tables_prompts_256", "op": "tables", "B": 256, "ctx_lo": 0, "ctx_hi": 8192, "new_lo": 1, "new_hi": 1023, "page": 16},
        # the verification step's keys and values, out of the fused projection
        {"name": "append_verify_32", "op": "append", "T": 256, "pad": 0, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "bf16", "cache": "bf16"},
        # a long prompt into an 8-bit cache, some padding tokens at the end
        {"name": "append_prompt_e4m3", "op": "append", "T": 16384, "pad": 37, "kv_heads": 8, "dim": 128, "page": 32, "dtype": "bf16", "cache": "e4m3"},
        # one request, one token: latency
        {"name": "attend_one_token", "op": "attend", "B": 1, "ctx_lo": 22000, "ctx_hi": 22000, "new_lo": 1, "new_hi": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "dtype": "bf16", "cache": "bf16", "causal": True, "window": 0, "fused": False},
        # verification of 7 drafts at low concurrency
        {"name": "attend_verify_4", "op": "attend", "B": 4, "ctx_lo": 22000, "ctx_hi": 22111, "new_lo": 8, "new_hi": 8, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 16, "dtype": "bf16", "cache": "bf16", "causal": True, "window": 0, "fused": True},
        # the same at the benchmark's batch of 32
        {"name": "attend_verify_32", "op": "attend", "B": 32, "ctx_lo": 22000, "ctx_hi": 23147, "new_lo": 8, "new_hi": 8, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16", "cache": "bf16", "causal": True, "window": 0, "fused": True},
        # verification of 3 drafts at batch 256 over an 8-bit cache
        {"name": "attend_verify_256_e4m3", "op": "attend", "B": 256, "ctx_lo": 1900, "ctx_hi": 6100, "new_lo": 4, "new_hi": 4, "heads": 32, "kv_heads": 4,
         "dim": 128, "page": 32, "dtype": "bf16", "cache": "e4m3", "causal": True, "window": 0, "fused": True},
        # a sliding-window layer, 7 query heads to a key head
        {"name": "attend_window_16", "op": "attend", "B": 16, "ctx_lo": 21000, "ctx_hi": 23000, "new_lo": 6, "new_hi": 8, "heads": 28, "kv_heads": 4,
         "dim": 64, "page": 16, "dtype": "fp16", "cache": "fp16", "causal": True, "window": 1024, "fused": False},
        # the drafter's block of parallel queries, which all see each other
        {"name": "attend_draft_block_32", "op": "attend", "B": 32, "ctx_lo": 3900, "ctx_hi": 4300, "new_lo": 7, "new_hi": 7, "heads": 16, "kv_heads": 16,
         "dim": 64, "page": 32, "dtype": "bf16", "cache": "bf16", "causal": False, "window": 0, "fused": False},
        # prompts of different lengths, some of them continued
        {"name": "attend_prompts_6", "op": "attend", "B": 6, "ctx_lo": 0, "ctx_hi": 1503, "new_lo": 101, "new_hi": 2999, "heads": 28, "kv_heads": 4,
         "dim": 128, "page": 16, "dtype": "fp16", "cache": "fp16", "causal": True, "window": 0, "fused": False},
        # a chunk of a long prompt: the largest
        {"name": "attend_prompt_chunk", "op": "attend", "B": 1, "ctx_lo": 12288, "ctx_hi": 12288, "new_lo": 4096, "new_hi": 4096, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16", "cache": "bf16", "causal": True, "window": 0, "fused": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "append", "attend", "attend", "attend"))
    page = rng.choice((16, 32, 64, 128))
    if op == "tables":
        B = _log_int(rng, 1, 256)
        ctx = _log_int(rng, 1, 23000)
        new = _log_int(rng, 1, min(1023, 131072 // B))
        return {"op": op, "B": B, "ctx_lo": ctx // 2, "ctx_hi": ctx, "new_lo": rng.choice((1, new)), "new_hi": new, "page": page}
    kv_heads = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128, 128))
    dtype = rng.choice(("bf16", "fp16"))
    cache = rng.choice((dtype, dtype, "e4m3"))
    if op == "append":
        T = _log_int(rng, 1, 16384)
        return {"op": op, "T": T, "pad": rng.choice((0, T // 9)), "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "cache": cache}
    heads = kv_heads * rng.choice((1, 2, 4, 5, 7, 8, 12, 16))
    causal = rng.random() < 0.8
    if rng.random() < 0.6:  # single tokens and verification steps
        B = _log_int(rng, 1, 256)
        new = rng.choice((1, 1, rng.randint(2, 17)))
        ctx = _log_int(rng, 16, max(17, min(23000, 700000 // B)))
        new_lo = rng.choice((1, new))
    else:  # prompts, chunked or whole
        B = _log_int(rng, 1, 8)
        heads = min(heads, 32)
        heads -= heads % kv_heads
        new = _log_int(rng, 33, 4096 // B)
        ctx = _log_int(rng, 1, 12000 // B)
        new_lo = rng.choice((new // 3, new))
    window = rng.choice((0, 0, 0, _log_int(rng, 100, 4096)))
    return {"op": op, "B": B, "ctx_lo": rng.choice((ctx // 3, ctx)), "ctx_hi": ctx, "new_lo": max(1, new_lo), "new_hi": new, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "cache": cache, "causal": causal, "window": window, "fused": rng.random() < 0.5}


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _lengths(case, seed):
    """(tokens cached before the step, new tokens) of each request."""
    B = case["B"]
    r = np.random.RandomState(seed % (1 << 31))
    return (r.permutation(np.array(_spread(case["ctx_lo"], case["ctx_hi"], B), np.int64)),
            r.permutation(np.array(_spread(case["new_lo"], case["new_hi"], B), np.int64)))


def _int(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": case["op"], "page": case["page"]}
    P = case["page"]
    if case["op"] == "append":
        H, D, n = case["kv_heads"], case["dim"], case["T"] + case["pad"]
        blocks = -(-case["T"] // P) + 3
        dt = DTYPES[case["dtype"]]
        qkv = torch.randn(n, 4 * H * D, device="cuda", generator=g).to(dt)  # two query heads to a key head, then keys, values
        s["k"] = qkv[:, 2 * H * D:3 * H * D].unflatten(1, (H, D))
        s["v"] = qkv[:, 3 * H * D:].unflatten(1, (H, D))
        for name in ("k_cache", "v_cache"):
            s[name] = torch.randn(blocks, H, P, D, device="cuda", generator=g).to(DTYPES[case["cache"]])
        page_of = torch.randperm(blocks, device="cuda", generator=g)[:-(-case["T"] // P)]
        t = torch.arange(case["T"], device="cuda")
        s["slot_map"] = torch.cat([page_of[t // P] * P + t % P, torch.full((case["pad"],), -1, device="cuda")])
        if case["cache"] == "e4m3":  # scales that leave some room below 448 and let a few values saturate
            s["k_scale"] = 0.008 + 0.004 * torch.rand(H, device="cuda", generator=g)
            s["v_scale"] = 0.008 + 0.004 * torch.rand(H, device="cuda", generator=g)
        else:
            s["k_scale"] = s["v_scale"] = None
        return s
    B = case["B"]
    ctx, new = _lengths(case, seed)
    S = B + 3
    rsi = np.random.RandomState((seed + 1) % (1 << 31)).permutation(S)[:B]
    s["req_state_idx"] = _int(rsi)
    if case["op"] == "tables":
        M = -(-(case["ctx_hi"] + case["new_hi"]) // P) + 1
        cached = np.zeros(S, np.int64)
        cached[rsi] = ctx
        held = -(-cached // P)
        blocks = int(held.sum() + (-(-new // P)).sum()) + 5
        ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
        table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
        held_t = _int(held, torch.int64)
        j = torch.arange(M, device="cuda")
        mask = j[None] < held_t[:, None]
        start = torch.cumsum(held_t, 0) - held_t
        used = int(held.sum())
        s["block_table"] = torch.where(mask, ids[(start[:, None] + j[None]).clamp(max=blocks - 1)], table)
        s["held_blocks"] = held_t.to(torch.int32)
        s["free_blocks"] = torch.cat([ids[used:], torch.full((used,), -1, dtype=torch.int32, device="cuda")])
        s["pool"] = _int([blocks - used, 0])
        s["cached_lens"] = _int(cached)
        s["new_lens"] = _int(new)
        s["no_lens"] = torch.zeros_like(s["new_lens"])
        T = B * case["new_hi"]
        s["made"] = [{"query_start": torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                      "seq_lens": torch.empty(B, dtype=torch.int32, device="cuda"),
                      "positions": torch.empty(T, dtype=torch.int64, device="cuda"),
                      "slot_map": torch.empty(T, dtype=torch.int64, device="cuda")} for _ in range(2)]
        return s
    Hq, H, D = case["heads"], case["kv_heads"], case["dim"]
    seq = ctx + new
    T = int(new.sum())
    dt = DTYPES[case["dtype"]]
    if case["fused"]:
        s["q"] = torch.randn(T, (Hq + 2 * H) * D, device="cuda", generator=g).mul_(2).to(dt)[:, :Hq * D].unflatten(1, (Hq, D))
    else:
        s["q"] = torch.randn(T, Hq, D, device="cuda", generator=g).mul_(2).to(dt)
    need = -(-seq // P)
    blocks = int(need.sum()) + 2
    for name in ("k_cache", "v_cache"):
        if case["cache"] == "e4m3":
            s[name] = torch.randn(blocks, H, P, D, device="cuda", generator=g, dtype=torch.bfloat16).mul_(96).clamp_(-448, 448).to(torch.float8_e4m3fn)
            s[name[0] + "_scale"] = 0.008 + 0.004 * torch.rand(H, device="cuda", generator=g)
        else:
            s[name] = torch.randn(blocks, H, P, D, device="cuda", generator=g, dtype=dt)
            s[name[0] + "_scale"] = None
    M = -(-(case["ctx_hi"] + case["new_hi"]) // P)
    ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    need_s = np.zeros(S, np.int64)
    need_s[rsi] = need
    need_t = _int(need_s, torch.int64)
    j = torch.arange(M, device="cuda")
    start = torch.cumsum(need_t, 0) - need_t
    s["block_table"] = torch.where(j[None] < need_t[:, None], ids[(start[:, None] + j[None]).clamp(max=blocks - 1)], -1)
    s["query_start"] = _int(np.concatenate([[0], np.cumsum(new)]))
    s["seq_lens"] = _int(seq)
    s["out"] = torch.empty(T, Hq, D, device="cuda", dtype=dt)
    s["lse"] = torch.empty(T, Hq, device="cuda")
    s["scale"] = D ** -0.5
    s["causal"], s["window"] = case["causal"], case["window"]
    s["max_new"], s["max_seq"] = case["new_hi"], case["ctx_hi"] + case["new_hi"]
    return s


def run(state):
    if state["op"] == "tables":
        return _tables(state)
    if state["op"] == "append":
        return _append(state)
    return _attend(state)


# -- block tables and slot map ---------------------------------------------------------------------------------
def _tables(s):
    """A step is planned (the requests grow by their new tokens) and taken back (they shrink to what they had, as
    when its drafts are rejected): the second call returns the blocks, so that the state is as it was."""
    first, second = s["made"]
    if own:
        from verify_dspark_markov_step_gb300 import paged_tables
        for new, made in ((s["new_lens"], first), (s["no_lens"], second)):
            paged_tables(s["req_state_idx"], new, s["cached_lens"], s["block_table"], s["held_blocks"], s["free_blocks"], s["pool"],
                         made["query_start"], made["seq_lens"], made["positions"], made["slot_map"], s["page"])
    else:
        _plain_tables(s, s["new_lens"], first)
        _plain_tables(s, s["no_lens"], second)
    return {"planned": first, "taken_back": second, "block_table": s["block_table"], "held_blocks": s["held_blocks"],
            "free_blocks": s["free_blocks"], "free_count": s["pool"][:1]}


def _plain_tables(s, new_lens, made):
    P, table, free = s["page"], s["block_table"], s["free_blocks"]
    S, M = table.shape
    N, T = free.numel(), made["slot_map"].numel()
    dev = table.device
    rsi = s["req_state_idx"].long()
    slot = rsi.clamp(min=0)
    new, cached, held, count = new_lens.long(), s["cached_lens"].long()[slot], s["held_blocks"].long()[slot], s["pool"][0].long()
    need = (cached + new + P - 1) // P
    ok = (rsi >= 0) & (new >= 0) & (need <= M)
    ok = ok & ((new == 0) | (torch.cumsum(torch.where(ok, new, 0), 0) <= T))
    release = torch.where(ok, (held - need).clamp(min=0), 0)
    take = torch.where(ok, (need - held).clamp(min=0), 0)
    top = count + release.sum()
    taken = torch.cumsum(take, 0)
    ok = ok & ((take == 0) | (taken <= top))
    take = torch.where(ok, take, 0)
    new = torch.where(ok, new, 0)
    j = torch.arange(M, device=dev)[None]
    rows = table[slot].long()
    # released blocks go on the free list last request first, last column first
    leaves = ok[:, None] & (j >= need[:, None]) & (j < held[:, None])
    at = count + (release.sum() - torch.cumsum(release, 0) + held - 1)[:, None] - j
    grown = torch.cat([free, free.new_empty(1)])
    grown[torch.where(leaves, at, N).reshape(-1)] = rows.reshape(-1).to(torch.int32)
    free.copy_(grown[:N])
    # new blocks come off it in the order of the requests and their columns
    comes = ok[:, None] & (j >= held[:, None]) & (j < need[:, None])
    source = (top - 1 - ((torch.cumsum(take, 0) - take - held)[:, None] + j)).clamp(0, N - 1)
    rows = torch.where(comes, free[source].long(), torch.where(leaves, -1, rows))
    to = torch.where(ok, slot, S)
    wide = torch.cat([table, table.new_empty(1, M)])
    wide[to] = rows.to(torch.int32)
    table.copy_(wide[:S])
    many = torch.cat([s["held_blocks"], s["held_blocks"].new_empty(1)])
    many[to] = need.to(torch.int32)
    s["held_blocks"].copy_(many[:S])
    s["pool"][0] = top - take.sum()
    start = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    t = torch.arange(T, device=dev)
    b = (torch.searchsorted(start, t, right=True) - 1).clamp(max=new.numel() - 1)
    position = cached[b] + t - start[b]
    block = rows[b, (position // P).clamp(max=M - 1)]
    live = t < start[-1]
    made["query_start"].copy_(start)
    made["seq_lens"].copy_(torch.where(ok, cached + new, 0))
    made["positions"].copy_(torch.where(live, position, -1))
    made["slot_map"].copy_(torch.where(live, block * P + position % P, -1))


# -- keys and values into their pages --------------------------------------------------------------------------
def _append(s):
    if own:
        from verify_dspark_markov_step_gb300 import kv_append
        kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_map"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        _plain_append(s["k"], s["k_cache"], s["slot_map"], s["k_scale"], s["page"])
        _plain_append(s["v"], s["v_cache"], s["slot_map"], s["v_scale"], s["page"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_append(x, cache, slot_map, scale, P):
    live = slot_map >= 0
    at = slot_map[live]
    x = x[live]
    if scale is not None:
        x = (x.float() / scale[:, None]).clamp(-448, 448)
    x = x.to(cache.dtype)
    if cache.dtype == torch.float8_e4m3fn:
        cache, x = cache.view(torch.uint8), x.view(torch.uint8)
    cache[at // P, :, at % P] = x


# -- attention of the new tokens over the pages ----------------------------------------------------------------
def _attend(s):
    if own:
        from verify_dspark_markov_step_gb300 import _lib, paged_attention
        if "workspace" not in s:
            s["workspace"] = _lib.workspace(_lib.paged_attention_workspace_bytes(s["seq_lens"].numel(), s["q"].shape[1], s["k_cache"].shape[1], s["q"].shape[2]))
        paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["req_state_idx"], s["query_start"], s["seq_lens"], s["out"],
                        scale=s["scale"], causal=s["causal"], window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=s["lse"],
                        workspace_buf=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    out, lse = _plain_attend(s)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_attend(s):
    q, P = s["q"].float(), s["page"]
    T, Hq, D = q.shape
    B, H = s["seq_lens"].numel(), s["k_cache"].shape[1]
    dev = q.device
    pages = -(-s["max_seq"] // P)
    ids = s["block_table"][s["req_state_idx"].long(), :pages].long().clamp(min=0)
    seq, start = s["seq_lens"].long(), s["query_start"].long()
    n = start[1:] - start[:-1]
    col = torch.arange(pages * P, device=dev)

    def all_of(cache, scale):
        x = cache.view(torch.uint8)[ids].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[ids]
        x = x.float().transpose(1, 2).reshape(B, H, pages * P, D)
        x = torch.where((col[None] < seq[:, None])[:, None, :, None], x, 0)
        return x if scale is None else x * scale[None, :, None, None]

    i = torch.arange(s["max_new"], device=dev)
    rows = q[(start[:-1, None] + i[None]).clamp(max=T - 1)].reshape(B, i.numel(), H, Hq // H, D)
    rows = rows.permute(0, 2, 1, 3, 4).reshape(B, H, i.numel() * (Hq // H), D)
    x = (rows @ all_of(s["k_cache"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    at = (seq - n)[:, None] + i[None]  # the position of each new token
    sees = (col[None, None] < seq[:, None, None]) & (i[None, :, None] < n[:, None, None])
    if s["causal"]:
        sees = sees & (col[None, None] <= at[:, :, None])
    if s["window"]:
        sees = sees & (col[None, None] > at[:, :, None] - s["window"])
    x = x.view(B, H, i.numel(), Hq // H, col.numel()).masked_fill_(~sees[:, None, :, None], -torch.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, -1, col.numel()) @ all_of(s["v_cache"], s["v_scale"])).view(B, H, i.numel(), Hq // H, D)
    out = torch.where(total > 0, out / total, 0)
    lse = (top + total.log())[..., 0]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(start, t, right=True) - 1
    return (out.permute(0, 2, 1, 3, 4)[b, t - start[b]].reshape(T, Hq, D),
            lse.permute(0, 2, 1, 3)[b, t - start[b]].reshape(T, Hq))


# -- what a pass cannot do without -----------------------------------------------------------------------------
def work(case):
    P = case["page"]
    if case["op"] == "append":
        values = 2 * case["T"] * case["kv_heads"] * case["dim"]
        return {"bytes": values * (BYTES[case["dtype"]] + BYTES[case["cache"]]) + 8 * (case["T"] + case["pad"]), "flops": values}
    ctx, new = _lengths(case, 0)
    if case["op"] == "tables":
        grown = int((-(-(ctx + new) // P) - -(-ctx // P)).sum())
        T, B = int(new.sum()), case["B"]
        per_call = B * (4 * 5 + 8) + 16 * B * case["new_hi"]
        return {"bytes": 2 * per_call + 16 * grown + 4 * (T // P), "flops": 4 * T}
    heads, H, D, W = case["heads"], case["kv_heads"], case["dim"], case["window"]
    keys = pairs = 0
    for c, n in zip(ctx.tolist(), new.tolist()):
        first = max(0, c - W + 1) if W else 0
        keys += c + n - first
        at = c + np.arange(n)
        seen = (at + 1 if case["causal"] else np.full(n, c + n)) - (np.maximum(0, at - W + 1) if W else 0)
        pairs += int(seen.sum())
    T = int(new.sum())
    return {"bytes": 2 * keys * H * D * BYTES[case["cache"]] + T * heads * (2 * D * BYTES[case["dtype"]] + 4), "flops": 4 * pairs * heads * D}


# -- the same by definition, in 64 bits ------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    P = case["page"]
    if case["op"] == "append":
        out = {}
        places = s["slot_map"].tolist()
        live = [t for t, at in enumerate(places) if at >= 0]
        at = torch.tensor([places[t] for t in live], device="cuda")
        for name in ("k", "v"):
            cache = s[name + "_cache"].double()
            x = s[name][torch.tensor(live, device="cuda")].double()
            if s[name + "_scale"] is not None:
                x = torch.clamp(x / s[name + "_scale"].double().view(1, -1, 1), -448.0, 448.0)
            flat = cache.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])  # a row for each token of each page
            flat[at] = x
            out[name + "_cache"] = flat.view(cache.shape[0], P, cache.shape[1], cache.shape[3]).transpose(1, 2)
        return out
    T, Hq, D = s["q"].shape
    H = case["kv_heads"]
    G = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    starts, lens, slots = s["query_start"].tolist(), s["seq_lens"].tolist(), s["req_state_idx"].tolist()
    for b in range(case["B"]):
        n, L = starts[b + 1] - starts[b], lens[b]
        ids = s["block_table"][slots[b], :-(-L // P)].long()
        key = torch.arange(L, device="cuda").view(1, L)
        pos = torch.arange(L - n, L, device="cuda").view(n, 1)
        hidden = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= key > pos
        if case["window"]:
            hidden |= key <= pos - case["window"]
        for h in range(H):
            k = s["k_cache"][:, h].view(torch.uint8)[ids].view(s["k_cache"].dtype).double().reshape(-1, D)[:L]
            v = s["v_cache"][:, h].view(torch.uint8)[ids].view(s["v_cache"].dtype).double().reshape(-1, D)[:L]
            ks = 1.0 if s["k_scale"] is None else float(s["k_scale"][h])
            vs = 1.0 if s["v_scale"] is None else float(s["v_scale"][h])
            q = s["q"][starts[b]:starts[b + 1], h * G:(h + 1) * G].double()
            score = torch.einsum("ngd,ld->gnl", q, k) * (s["scale"] * ks)
            score.masked_fill_(hidden, -math.inf)
            total = torch.logsumexp(score, -1)
            prob = torch.exp(score - torch.where(total == -math.inf, 0.0, total)[..., None])
            out[starts[b]:starts[b + 1], h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", prob, v) * vs
            lse[starts[b]:starts[b + 1], h * G:(h + 1) * G] = total.transpose(0, 1)
            del score, prob
    return {"out": out, "lse": lse}
