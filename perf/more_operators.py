"""Four more operators of the target model's verification pass, as measured cases.

They stand around the same paged key/value cache as the operators of ``operators.py``: the position rotation of
query and key rows; the norm of each head, the rotation and the writing of keys and values into their pages in
one pass; attention with a sliding window beside which the first tokens stay visible; and the upkeep of the
pages themselves (a prompt forked into several samples with or without sharing its pages, the pages copied, the
slots freed, the cache compacted). ``run`` computes each of them either in plain torch operations (``own``
false) or by the calls a user makes of this package (``own`` true).

Lengths of a ragged batch are spread evenly over the case's ranges and dealt to the requests in an order that
the seed decides, so that the work of a case does not depend on the seed.
"""
import math
from fractions import Fraction

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889")


def listed():
    return [
        # a verification step's queries and keys, half of each head rotated
        {"name": "rotary_verify_32", "op": "rotary", "T": 256, "pad": 0, "heads": 64, "kv_heads": 8, "dim": 128, "rotary": 64, "interleaved": False,
         "base": 5e6, "scaling": "none", "ctx": 22000, "dtype": "bf16"},
        # a long prompt past the trained length: neighbouring values paired, frequencies scaled
        {"name": "rotary_prompt_yarn", "op": "rotary", "T": 16384, "pad": 37, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": True,
         "base": 1e4, "scaling": "yarn", "ctx": 100000, "dtype": "fp16"},
        # one request, one token: latency
        {"name": "qk_append_one_token", "op": "qk_append", "T": 1, "pad": 0, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False,
         "base": 1e6, "scaling": "none", "ctx": 22000, "dtype": "bf16", "cache": "bf16", "page": 16, "norm": True},
        # the verification step at the benchmark's batch of 32, some padding tokens at the end
        {"name": "qk_append_verify_32", "op": "qk_append", "T": 256, "pad": 8, "heads": 64, "kv_heads": 8, "dim": 128, "rotary": 64, "interleaved": False,
         "base": 5e6, "scaling": "none", "ctx": 22000, "dtype": "bf16", "cache": "bf16", "page": 64, "norm": True},
        # a long prompt into an 8-bit cache
        {"name": "qk_append_prompt_e4m3", "op": "qk_append", "T": 16384, "pad": 37, "heads": 64, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "base": 1e6, "scaling": "linear", "ctx": 0, "dtype": "bf16", "cache": "e4m3", "page": 32, "norm": True},
        # one token of a long conversation that sees its last 4096 and its first 4 tokens
        {"name": "sinks_one_token", "op": "sinks", "B": 1, "ctx_lo": 22000, "ctx_hi": 22000, "new_lo": 1, "new_hi": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "dtype": "bf16", "cache": "bf16", "causal": True, "window": 4096, "sinks": 4, "fused": False},
        # verification of 7 drafts at the benchmark's batch of 32, a system prompt that stays visible
        {"name": "sinks_verify_32", "op": "sinks", "B": 32, "ctx_lo": 22000, "ctx_hi": 23147, "new_lo": 8, "new_hi": 8, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16", "cache": "bf16", "causal": True, "window": 4096, "sinks": 300, "fused": True},
        # a chunk of a long prompt
        {"name": "sinks_prompt_chunk", "op": "sinks", "B": 1, "ctx_lo": 12288, "ctx_hi": 12288, "new_lo": 4096, "new_hi": 4096, "heads": 28, "kv_heads": 4,
         "dim": 128, "page": 16, "dtype": "fp16", "cache": "fp16", "causal": True, "window": 2048, "sinks": 16, "fused": False},
        # eight samples of one prompt, which share its pages, taken and given up: latency
        {"name": "branch_one_prompt", "op": "pages", "kind": "branch", "prompts": 1, "samples": 8, "len_lo": 500, "len_hi": 500, "others": 3, "page": 16,
         "layers": 2, "kv_heads": 2, "dim": 128, "dtype": "bf16"},
        # sixteen long prompts in eight samples each
        {"name": "branch_16_prompts", "op": "pages", "kind": "branch", "prompts": 16, "samples": 8, "len_lo": 20001, "len_hi": 22999, "others": 2, "page": 64,
         "layers": 2, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # a few requests copied whole, the old ones freed and the cache compacted: twice, there and back
        {"name": "move_4", "op": "pages", "kind": "move", "prompts": 4, "samples": 1, "len_lo": 300, "len_hi": 2100, "others": 5, "page": 32,
         "layers": 2, "kv_heads": 4, "dim": 64, "dtype": "e4m3"},
        # the same with long requests: the largest
        {"name": "move_8_long", "op": "pages", "kind": "move", "prompts": 8, "samples": 1, "len_lo": 20000, "len_hi": 23000, "others": 4, "page": 16,
         "layers": 2, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "qk_append", "sinks", "sinks", "pages"))
    page = rng.choice((16, 32, 64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128, 128))
    dtype = rng.choice(("bf16", "fp16"))
    cache = rng.choice((dtype, dtype, "e4m3"))
    heads = kv_heads * rng.choice((1, 2, 4, 5, 7, 8))
    if op in ("rotary", "qk_append"):
        T = _log_int(rng, 1, 16384)
        case = {"op": op, "T": T, "pad": rng.choice((0, T // 9)), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rotary": rng.choice((dim, dim, dim // 2, dim // 4, 48)), "interleaved": rng.random() < 0.4, "base": rng.choice((1e4, 5e5, 1e6)),
                "scaling": rng.choice(("none", "none", "linear", "yarn")), "ctx": _log_int(rng, 1, 130000), "dtype": dtype}
        if op == "rotary":
            return {**case, "dim": rng.choice((dim, 96, 192, 256))} if case["rotary"] <= 64 else case
        return {**case, "cache": cache, "page": page, "norm": rng.random() < 0.7}
    if op == "pages":
        kind = rng.choice(("branch", "move"))
        n = _log_int(rng, 1, 32)
        most = _log_int(rng, 40, 180000 // n if kind == "move" else 23000)
        return {"op": op, "kind": kind, "prompts": n, "samples": 1 if kind == "move" else rng.randint(1, 8), "len_lo": max(1, rng.choice((most // 3, most - 9))),
                "len_hi": most, "others": rng.randint(0, 8), "page": page, "layers": rng.randint(1, 2), "kv_heads": kv_heads, "dim": dim, "dtype": cache}
    causal = rng.random() < 0.8
    if rng.random() < 0.6:  # single tokens and verification steps
        B = _log_int(rng, 1, 256)
        new = rng.choice((1, 1, rng.randint(2, 17)))
        ctx = _log_int(rng, 16, max(17, min(23000, 700000 // B)))
        new_lo = rng.choice((1, new))
    else:  # prompts, chunked or whole
        B = _log_int(rng, 1, 8)
        new = _log_int(rng, 33, 4096 // B)
        ctx = _log_int(rng, 1, 12000 // B)
        new_lo = rng.choice((new // 3, new))
        heads = min(heads, 28 // kv_heads * kv_heads)
    window = _log_int(rng, 100, 4096)
    return {"op": op, "B": B, "ctx_lo": rng.choice((ctx // 3, ctx)), "ctx_hi": ctx, "new_lo": max(1, new_lo), "new_hi": new, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "cache": cache, "causal": causal, "window": window,
            "sinks": rng.choice((1, 4, _log_int(rng, 2, 1000))), "fused": rng.random() < 0.5}


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _dealt(lo, hi, n, seed):
    return np.random.RandomState(seed % (1 << 31)).permutation(np.array(_spread(lo, hi, n), np.int64))


def _int(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, seed, g)
    if case["op"] == "sinks":
        return _prepare_sinks(case, seed, g)
    return _prepare_rows(case, g)


def run(state):
    if state["op"] == "pages":
        return _branch(state) if state["kind"] == "branch" else _move(state)
    if state["op"] == "sinks":
        return _attend(state)
    return _rotate(state) if state["op"] == "rotary" else _qk_append(state)


# -- rows of queries and keys: norm, rotation, pages -----------------------------------------------------------
def _frequencies(case):
    """Radians a position of each pair, and what cosines and sines are multiplied by."""
    R, base, how = case["rotary"], case["base"], case["scaling"]
    inv = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if how == "none":
        return inv, 1.0
    if how == "linear":
        return inv / 8.0, 1.0
    # "yarn": pairs that turn often within the trained 8192 positions keep their frequency, slow ones are
    # interpolated, with a ramp between 32 turns and 1
    trained, factor = 8192.0, 16.0

    def pair_of(turns):
        return R * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
    lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), R - 1)
    ramp = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return inv / factor * ramp + inv * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


def _prepare_rows(case, g):
    Hq, H, D, n = case["heads"], case["kv_heads"], case["dim"], case["T"] + case["pad"]
    dt = DTYPES[case["dtype"]]
    s = {"op": case["op"], "interleaved": case["interleaved"]}
    qkv = torch.randn(n, (Hq + 2 * H) * D, device="cuda", generator=g).mul_(2).to(dt)  # the fused projection
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split((Hq * D, H * D, H * D), 1))
    s["q_out"] = torch.randn(n, Hq, D, device="cuda", generator=g).to(dt)
    inv, s["factor"] = _frequencies(case)
    s["inv_freq"] = torch.from_numpy(inv).cuda()
    # the same as the library's table: 2^-64 turns a position, modulo a whole turn
    turns = [round(Fraction(float(f)) * 2 ** 64 / TWO_PI) % 2 ** 64 for f in inv]
    s["turns"] = torch.from_numpy(np.array(turns, np.uint64).view(np.int64)).cuda()
    t = torch.arange(case["T"], device="cuda")
    first = torch.randint(case["ctx"] + 1, (1,), device="cuda", generator=g) if case["ctx"] else torch.zeros(1, dtype=torch.int64, device="cuda")
    gone = torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda")
    s["positions"] = torch.cat([t + first, gone])
    if case["op"] == "rotary":
        s["k_out"] = torch.randn(n, H, D, device="cuda", generator=g).to(dt)
        return s
    P, c = case["page"], DTYPES[case["cache"]]
    s["page"] = P
    blocks = -(-case["T"] // P) + 3
    for name in ("k_cache", "v_cache"):
        s[name] = torch.randn(blocks, H, P, D, device="cuda", generator=g).to(c)
    page_of = torch.randperm(blocks, device="cuda", generator=g)[:-(-case["T"] // P)]
    s["slot_map"] = torch.cat([page_of[t // P] * P + t % P, gone])
    s["k_scale"] = s["v_scale"] = s["q_weight"] = s["k_weight"] = None
    if case["cache"] == "e4m3":  # scales that leave some room below 448 and let a few values saturate
        s["k_scale"], s["v_scale"] = (0.008 + 0.004 * torch.rand(H, device="cuda", generator=g) for _ in range(2))
    if case["norm"]:
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt) for _ in range(2))
    s["eps"] = 1e-6
    return s


def _rotate(s):
    if own:
        from verify_dspark_markov_step_gb300 import qk_rope
        qk_rope(s["q"], s["k"], s["positions"], turns=s["turns"], factor=s["factor"], interleaved=s["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    else:
        live = s["positions"] >= 0
        s["q_out"][live] = _plain_rotated(s, s["q"].float())[live].to(s["q_out"].dtype)
        s["k_out"][live] = _plain_rotated(s, s["k"].float())[live].to(s["k_out"].dtype)
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_rotated(s, x):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    R = 2 * cos.shape[-1]
    rows, rest = x[..., :R], x[..., R:]
    if s["interleaved"]:
        a, b = rows[..., 0::2], rows[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rows[..., :R // 2], rows[..., R // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _qk_append(s):
    if own:
        from verify_dspark_markov_step_gb300 import qk_rope_append
        qk_rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["positions"], s["slot_map"], turns=s["turns"], factor=s["factor"],
                       interleaved=s["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], q_out=s["q_out"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        live = s["positions"] >= 0
        s["q_out"][live] = _plain_rotated(s, _plain_normed(s["q"], s["q_weight"], s["eps"]))[live].to(s["q_out"].dtype)
        _plain_append(_plain_rotated(s, _plain_normed(s["k"], s["k_weight"], s["eps"])), s["k_cache"], s["slot_map"], s["k_scale"], s["page"])
        _plain_append(s["v"].float(), s["v_cache"], s["slot_map"], s["v_scale"], s["page"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_normed(x, weight, eps):
    x = x.float()
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()


def _plain_append(x, cache, slot_map, scale, P):
    live = slot_map >= 0
    at = slot_map[live]
    x = x[live]
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448, 448)
    x = x.to(cache.dtype)
    if cache.dtype == torch.float8_e4m3fn:
        cache, x = cache.view(torch.uint8), x.view(torch.uint8)
    cache[at // P, :, at % P] = x


# -- attention over the pages: a window, and first tokens that stay visible -------------------------------------
def _lengths(case, seed):
    """(tokens cached before the step, new tokens) of each request."""
    return _dealt(case["ctx_lo"], case["ctx_hi"], case["B"], seed), _dealt(case["new_lo"], case["new_hi"], case["B"], seed + 1)


def _prepare_sinks(case, seed, g):
    B, P, Hq, H, D = case["B"], case["page"], case["heads"], case["kv_heads"], case["dim"]
    s = {"op": "sinks", "page": P}
    ctx, new = _lengths(case, seed)
    seq, T, dt = ctx + new, int(new.sum()), DTYPES[case["dtype"]]
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
    S = B + 3
    rsi = np.random.RandomState((seed + 2) % (1 << 31)).permutation(S)[:B]
    s["req_state_idx"] = _int(rsi)
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
    s["causal"], s["window"], s["sinks"] = case["causal"], case["window"], case["sinks"]
    s["max_new"], s["max_seq"] = case["new_hi"], case["ctx_hi"] + case["new_hi"]
    return s


def _attend(s):
    if own:
        from verify_dspark_markov_step_gb300 import _lib, paged_attention
        if "workspace" not in s:
            s["workspace"] = _lib.workspace(_lib.paged_attention_workspace_bytes(s["seq_lens"].numel(), s["q"].shape[1], s["k_cache"].shape[1], s["q"].shape[2]))
        paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["req_state_idx"], s["query_start"], s["seq_lens"], s["out"],
                        scale=s["scale"], causal=s["causal"], window=s["window"], sinks=s["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                        lse=s["lse"], workspace_buf=s["workspace"])
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
    sees = (col[None, None] > at[:, :, None] - s["window"]) | (col < s["sinks"])
    sees = sees & (col[None, None] < seq[:, None, None]) & (i[None, :, None] < n[:, None, None])
    if s["causal"]:
        sees = sees & (col[None, None] <= at[:, :, None])
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


# -- the pages: forking, copying, freeing, compacting ------------------------------------------------------------
def _prepare_pages(case, seed, g):
    P, n, F, others = case["page"], case["prompts"], case["samples"], case["others"]
    lens = _dealt(case["len_lo"], case["len_hi"], n, seed)
    rest = _dealt(case["len_lo"], case["len_hi"], others, seed + 1) if others else np.zeros(0, np.int64)
    share = case["kind"] == "branch"
    S = n + others + n * F + 2
    slots = np.random.RandomState((seed + 2) % (1 << 31)).permutation(S)
    src, bystanders, dst = slots[:n], slots[n:n + others], slots[n + others:n + others + n * F]
    s = {"op": "pages", "kind": case["kind"], "page": P, "layers": case["layers"]}
    s["src"], s["dst"] = _int(np.repeat(src, F)), _int(dst)
    cached = np.zeros(S, np.int64)
    cached[src], cached[bystanders] = lens, rest
    held = -(-cached // P)
    used = int(held.sum())
    blocks = used + (n * F if share else int((-(-lens // P)).sum())) + 7
    M = -(-case["len_hi"] // P) + 1
    # the first `used` blocks are held, in no order; the others are free
    ids = torch.cat([torch.randperm(used, device="cuda", generator=g), used + torch.randperm(blocks - used, device="cuda", generator=g)]).to(torch.int32)
    held_t = _int(held, torch.int64)
    j = torch.arange(M, device="cuda")
    start = torch.cumsum(held_t, 0) - held_t
    s["block_table"] = torch.where(j[None] < held_t[:, None], ids[(start[:, None] + j[None]).clamp(max=blocks - 1)], -1)
    s["held_blocks"], s["cached_lens"] = held_t.to(torch.int32), _int(cached)
    s["free_blocks"] = torch.cat([ids[used:], torch.full((used,), -1, dtype=torch.int32, device="cuda")])
    s["pool"] = _int([blocks - used, 0])
    s["shares"] = torch.zeros(blocks, dtype=torch.int32, device="cuda") if share else None
    shape = (case["layers"], 2, blocks, case["kv_heads"], P, case["dim"])
    c = DTYPES[case["dtype"]]
    if case["dtype"] == "e4m3":  # any bytes but the two that are no numbers
        u = torch.randint(127, shape, device="cuda", generator=g, dtype=torch.uint8)
        s["caches"] = u.bitwise_or_(torch.randint(2, (1, 1, blocks, 1, P, 1), device="cuda", generator=g, dtype=torch.uint8) << 7).view(c)
    else:
        s["caches"] = torch.randn(shape, device="cuda", generator=g, dtype=c)
    s["copies"] = torch.empty(blocks, 2, dtype=torch.int32, device="cuda")
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _branch(s):
    """Every prompt is forked into its samples, which share its full pages and have a copy of the last one, and the samples are freed."""
    if own:
        from verify_dspark_markov_step_gb300 import paged_copy, paged_fork, paged_free
        paged_fork(s["src"], s["dst"], s["cached_lens"], s["block_table"], s["held_blocks"], s["free_blocks"], s["pool"], s["copies"], s["count"],
                   s["page"], shares=s["shares"])
        paged_copy([tuple(layer) for layer in s["caches"]], s["copies"], s["count"])
        forked = s["block_table"].index_select(0, s["dst"]), s["shares"].clone()
        paged_free(s["dst"], s["cached_lens"], s["block_table"], s["held_blocks"], s["free_blocks"], s["pool"], shares=s["shares"])
    else:
        _plain_copy(s, *_plain_fork(s, s["src"], s["dst"]))
        forked = s["block_table"].index_select(0, s["dst"]), s["shares"].clone()
        _plain_free(s, s["dst"])
    return {"forked": forked, **_pages(s)}


def _move(s):
    """The requests are copied into other slots, the first ones freed and the cache compacted, and the same back."""
    _moved(s, s["src"], s["dst"])
    _moved(s, s["dst"], s["src"])
    return _pages(s)


def _moved(s, src, dst):
    if own:
        from verify_dspark_markov_step_gb300 import _lib, paged_compact, paged_copy, paged_fork, paged_free
        if "workspace" not in s:
            s["workspace"] = _lib.workspace(_lib.paged_compact_workspace_bytes(s["free_blocks"].numel()))
        layers = [tuple(layer) for layer in s["caches"]]
        paged_fork(src, dst, s["cached_lens"], s["block_table"], s["held_blocks"], s["free_blocks"], s["pool"], s["copies"], s["count"], s["page"])
        paged_copy(layers, s["copies"], s["count"])
        paged_free(src, s["cached_lens"], s["block_table"], s["held_blocks"], s["free_blocks"], s["pool"])
        paged_compact(s["block_table"], s["held_blocks"], s["free_blocks"], s["pool"], s["copies"], s["count"], workspace_buf=s["workspace"])
        paged_copy(layers, s["copies"], s["count"])
    else:
        _plain_copy(s, *_plain_fork(s, src, dst))
        _plain_free(s, src)
        _plain_copy(s, *_plain_compact(s))


def _pages(s):
    return {name: s[name] for name in ("block_table", "held_blocks", "cached_lens", "free_blocks", "caches")} | {"free_count": s["pool"][:1]}


def _plain_copy(s, source, to):
    cache = s["caches"]
    if cache.dtype == torch.float8_e4m3fn:
        cache = cache.view(torch.uint8)
    cache[:, :, to] = cache[:, :, source]


def _plain_fork(s, src, dst):
    """The blocks to copy, and where to."""
    P, table, free = s["page"], s["block_table"], s["free_blocks"]
    src, dst = src.long(), dst.long()
    n, M, top = s["cached_lens"][src].long(), table.shape[1], s["pool"][0].long()
    need = (n + P - 1) // P
    keep = n // P if s["shares"] is not None else torch.zeros_like(n)
    take = need - keep
    j = torch.arange(M, device=table.device)[None]
    rows = table[src]
    first = torch.cumsum(take, 0) - take
    comes = (j >= keep[:, None]) & (j < need[:, None])
    place = (top - 1 - (first[:, None] + j - keep[:, None])).clamp(0, free.numel() - 1)
    ids = torch.where(comes, free[place], torch.where(j < need[:, None], rows, -1))
    if s["shares"] is not None:
        kept = rows[j < keep[:, None]].long()
        s["shares"].index_add_(0, kept, torch.ones_like(kept, dtype=torch.int32))
    table[dst] = ids
    s["held_blocks"][dst] = need.to(torch.int32)
    s["cached_lens"][dst] = n.to(torch.int32)
    s["pool"][0] -= take.sum()
    return rows[comes].long(), ids[comes].long()


def _plain_free(s, slots):
    """A block that no other row holds goes on the stack: of the call's slots last request first, last column first."""
    table, free, slots = s["block_table"], s["free_blocks"], slots.long()
    rows, top = table[slots], s["pool"][0].long()
    goes = torch.arange(table.shape[1], device=table.device)[None] < s["held_blocks"][slots][:, None]
    if s["shares"] is not None:
        ids, of = rows[goes].long(), torch.arange(slots.numel(), device=table.device)[:, None].expand_as(rows)
        left = s["shares"].index_add(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
        last = torch.full_like(left, -1, dtype=torch.int64).scatter_reduce(0, ids, of[goes], "amax")
        s["shares"].copy_(left.clamp(min=0))
        at = rows.long().clamp(min=0)
        goes = goes & (left[at] < 0) & (last[at] == of)
    back = rows[goes].flip(0)
    free[top + torch.arange(back.numel(), device=table.device)] = back
    s["pool"][0] += back.numel()
    table[slots] = -1
    s["held_blocks"][slots] = 0
    s["cached_lens"][slots] = 0


def _plain_compact(s):
    """The held blocks become the first ones: the blocks to copy, and where to."""
    table, free, N = s["block_table"], s["free_blocks"], s["free_blocks"].numel()
    ids = torch.arange(N, device=table.device)
    count = s["pool"][0].long()
    is_free = torch.zeros(N, dtype=torch.bool, device=table.device)
    is_free[free[ids < count].long()] = True
    movers, holes = ids[~is_free & (ids >= N - count)], ids[is_free & (ids < N - count)]
    to = ids.clone()
    to[movers] = holes
    holds = torch.arange(table.shape[1], device=table.device)[None] < s["held_blocks"][:, None]
    table.copy_(torch.where(holds, to[table.long().clamp(min=0)].to(torch.int32), table))
    free.copy_(torch.where(ids < count, N - 1 - ids, free))
    return movers, holes


# -- what a pass cannot do without -----------------------------------------------------------------------------
def work(case):
    if case["op"] in ("rotary", "qk_append"):
        T, Hq, H, D, e = case["T"], case["heads"], case["kv_heads"], case["dim"], BYTES[case["dtype"]]
        if case["op"] == "rotary":
            return {"bytes": T * (2 * (Hq + H) * D * e + 8), "flops": 3 * T * (Hq + H) * case["rotary"]}
        norm = 4 * D if case["norm"] else 0
        return {"bytes": T * (2 * Hq * D * e + 2 * H * D * (e + BYTES[case["cache"]]) + 16), "flops": T * (Hq + H) * (3 * case["rotary"] + norm)}
    if case["op"] == "pages":
        P = case["page"]
        lens = _dealt(case["len_lo"], case["len_hi"], case["prompts"], 0)
        page = 2 * case["layers"] * case["kv_heads"] * P * case["dim"] * BYTES[case["dtype"]]
        entries = int((-(-lens // P)).sum()) * case["samples"]
        if case["kind"] == "branch":  # a row's entries read, written and taken back, a share more and less of each
            return {"bytes": 2 * page * int((lens % P > 0).sum()) * case["samples"] + entries * (4 + 4 + 4 + 4 * 4), "flops": entries}
        return {"bytes": 2 * (2 * 2 * page * entries + entries * 5 * 8), "flops": 4 * entries}
    ctx, new = _lengths(case, 0)
    heads, H, D, W, sinks = case["heads"], case["kv_heads"], case["dim"], case["window"], case["sinks"]
    keys = pairs = 0
    for c, n in zip(ctx.tolist(), new.tolist()):
        first = max(0, c - W + 1)
        keys += c + n - first + min(first, sinks)
        at = c + np.arange(n)
        low = np.maximum(0, at - W + 1)
        pairs += int(((at + 1 if case["causal"] else np.full(n, c + n)) - low + np.minimum(low, sinks)).sum())
    T = int(new.sum())
    return {"bytes": 2 * keys * H * D * BYTES[case["cache"]] + T * heads * (2 * D * BYTES[case["dtype"]] + 4), "flops": 4 * pairs * heads * D}


# -- the same by definition, in 64 bits ------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers, and values that are only moved
    s = prepare(case, seed)
    if case["op"] == "sinks":
        return _exact_attend(case, s)
    inv, factor = _frequencies(case)
    pos = s["positions"].cpu().numpy().astype(np.float64)
    unit = torch.polar(torch.full((pos.size, inv.size), factor, dtype=torch.float64), torch.from_numpy(np.outer(pos, inv))).cuda()[:, None]
    R = case["rotary"]

    def turned(x, weight=None):
        x = x.double()
        if weight is not None:
            x = weight.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dim"] + s["eps"])
        pairs = x[..., :R].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :R].unflatten(-1, (2, -1)).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        pairs = pairs.flatten(-2) if case["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
        return torch.cat([pairs, x[..., R:]], -1)

    def kept(out, x):
        out = out.double()
        out[:case["T"]] = x[:case["T"]]
        return out

    if case["op"] == "rotary":
        return {"q": kept(s["q_out"], turned(s["q"])), "k": kept(s["k_out"], turned(s["k"]))}
    out = {"q": kept(s["q_out"], turned(s["q"], s["q_weight"]))}
    at = s["slot_map"][:case["T"]]
    for name, x in (("k", turned(s["k"], s["k_weight"])), ("v", s["v"].double())):
        cache, x = s[name + "_cache"].double(), x[:case["T"]]
        if s[name + "_scale"] is not None:
            x = torch.clamp(x / s[name + "_scale"].double().view(1, -1, 1), -448.0, 448.0)
        flat = cache.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])  # a row for each token of each page
        flat[at] = x
        out[name + "_cache"] = flat.view(cache.shape[0], case["page"], cache.shape[1], cache.shape[3]).transpose(1, 2)
    return out


def _exact_attend(case, s):
    P, H = case["page"], case["kv_heads"]
    T, Hq, D = s["q"].shape
    G = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    starts, lens, slots = s["query_start"].tolist(), s["seq_lens"].tolist(), s["req_state_idx"].tolist()
    for b in range(case["B"]):
        n, L = starts[b + 1] - starts[b], lens[b]
        ids = s["block_table"][slots[b], :-(-L // P)].long()
        key = torch.arange(L, device="cuda").view(1, L)
        pos = torch.arange(L - n, L, device="cuda").view(n, 1)
        hidden = (key <= pos - case["window"]) & (key >= case["sinks"])
        if case["causal"]:
            hidden |= key > pos
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
