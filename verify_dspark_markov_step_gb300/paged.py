"""The paged key/value cache of the target model's verification pass, and a
speculative decoding loop that runs on it.

``PagedCache`` holds the buffers (the caches of every layer, the block tables, the
free blocks, a step's offsets and slots) and makes the library calls: a step's tables,
keys and values (with the norm of each head and the rotation by position, or as they
are), attention; and between steps slots forked and freed and the blocks compacted.
Every length stays on the device, so a step follows from the last one's accept counts
without the host. ``main`` runs whole steps of a small random model: the drafter's
Markov loop, the target's forward over anchor and drafts (projections in torch, cache
and attention in the library), the rejection sampler.
"""
from __future__ import annotations

import torch

from . import _lib


class PagedCache:
    """Caches of ``layers`` layers for ``slots`` request slots of up to ``max_len``
    tokens, ``num_blocks`` blocks of ``page_size`` tokens shared by all slots (the same
    tables serve every layer). ``cache_dtype`` is the rows' dtype or float8_e4m3fn;
    ``k_scale``/``v_scale`` [layers, kv_heads] are what its values stand for multiples of.
    With ``sharing`` a fork's full blocks are its parent's own, counted in ``shares``.

    The calls run on ``stream``, or on torch's current stream. A step's plan, appends and
    attentions share the tables and the plan's results, forks, frees and compactions the
    tables and the list of copies: on several streams the caller orders them. Each stream
    has an attention workspace of its own, so attentions of one plan may run on different
    streams side by side."""

    def __init__(self, *, layers, slots, max_len, num_blocks, page_size, q_heads, kv_heads,
                 head_dim, dtype=torch.bfloat16, cache_dtype=None, k_scale=None, v_scale=None,
                 device="cuda", sharing=False):
        self.page_size, self.q_heads = page_size, q_heads
        shape = (num_blocks, kv_heads, page_size, head_dim)
        cache_dtype = cache_dtype or dtype
        self.k, self.v = ([torch.zeros(shape, dtype=cache_dtype, device=device)
                           for _ in range(layers)] for _ in range(2))
        self.k_scale, self.v_scale = k_scale, v_scale

        def ints(shape, value=0):
            return torch.full(shape, value, dtype=torch.int32, device=device)
        self.block_table = ints((slots, -(-max_len // page_size)), -1)
        self.held_blocks, self.cached_lens = ints((slots,)), ints((slots,))
        self.free_blocks = torch.arange(num_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        self.pool = torch.tensor([num_blocks, 0], dtype=torch.int32, device=device)
        self.status = ints((1,))
        self.shares = ints((num_blocks,)) if sharing else None
        self.copies, self.copied = ints((num_blocks, 2)), ints((1,))
        self._caches, self._compacting = _lib.PagedCaches(()), None
        self._dims = (q_heads, kv_heads, head_dim)
        self._made = {}  # buffers of plans, by the power of two that holds their tokens
        self._last = None, None
        self._workspaces = {}  # by stream

    def plan(self, req_state_idx, new_lens, max_tokens, num_accepted=None, stream=None):
        """Block tables and slots of a step in which request b brings new_lens[b] tokens
        (at most max_tokens in all); with num_accepted the slots' lengths first grow by
        what the last step's verification kept. Returns (query_start, seq_lens,
        positions, slot_map), which later plans may overwrite."""
        self.req_state_idx = req_state_idx
        self.step = self._buffers(req_state_idx.shape[0], max_tokens, stream)
        _lib.paged_tables(req_state_idx, new_lens, self.cached_lens, self.block_table,
                          self.held_blocks, self.free_blocks, self.pool, *self.step,
                          self.page_size, num_accepted=num_accepted, status=self.status,
                          stream=stream, **self._sharing())
        return self.step

    def _sharing(self):
        return {} if self.shares is None else {"shares": self.shares}

    def _buffers(self, B, T, stream):
        """Views of a plan's buffers. Sizes that vary share them, and none is given back:
        a captured plan goes on writing where it did."""
        if self._last[0] == (B, T):
            return self._last[1]
        size = max(1024, 1 << max(0, T - 1).bit_length())
        with torch.cuda.stream(stream):  # memory of the stream that uses it

            def made(key, count, dtype):
                if key not in self._made:
                    self._made[key] = torch.empty(count, dtype=dtype, device=self.pool.device)
                return self._made[key]
            requests = made("requests", 2 * _lib.MAX_PAGED_BATCH + 1, torch.int32)
            tokens = made(size, 2 * size, torch.int64)
        most = _lib.MAX_PAGED_BATCH
        views = (requests[:B + 1], requests[most + 1:most + 1 + B], tokens[:T],
                 tokens[size:size + T])
        self._last = (B, T), views
        return views

    def _scales(self, layer):
        return {"k_scale": None if self.k_scale is None else self.k_scale[layer],
                "v_scale": None if self.v_scale is None else self.v_scale[layer]}

    def append(self, layer, k, v, stream=None):
        """The planned step's keys and values [max_tokens, kv_heads, head_dim] into the
        pages of a layer."""
        _lib.kv_append(k, v, self.k[layer], self.v[layer], self.step[3], status=self.status,
                       stream=stream, **self._scales(layer))

    def append_qk(self, layer, q, k, v, rotary=None, q_weight=None, k_weight=None, eps=1e-6,
                  q_out=None, stream=None):
        """The norm of each head of q and k (with weights [head_dim]) and the rotation by
        the planned step's positions (with a rotary.Rotary): q [max_tokens, q_heads,
        head_dim] in place or into q_out, the keys, and the values as they are, into the
        pages of a layer."""
        _lib.qk_rope_append(q, k, v, self.k[layer], self.v[layer], self.step[2], self.step[3],
                            q_weight=q_weight, k_weight=k_weight, eps=eps, q_out=q_out,
                            status=self.status, stream=stream, **self._scales(layer),
                            **({} if rotary is None else rotary.args()))

    def attend(self, layer, q, out, causal=True, window=0, scale=None, lse=None, stream=None,
               sinks=0):
        """The planned step's attention of q [max_tokens, q_heads, head_dim] over a
        layer's pages, into out; the first ``sinks`` tokens stay visible beside a window."""
        key = _lib._raw_stream(stream, self.pool)
        if key not in self._workspaces:
            need = _lib.paged_attention_workspace_bytes(_lib.MAX_PAGED_BATCH, *self._dims)
            with torch.cuda.stream(stream):
                self._workspaces[key] = _lib.workspace(need, self.pool.device)
        _lib.paged_attention(q, self.k[layer], self.v[layer], self.block_table,
                             self.req_state_idx, self.step[0], self.step[1], out, scale=scale,
                             causal=causal, window=window, lse=lse,
                             workspace_buf=self._workspaces[key], status=self.status, stream=stream,
                             **({"sinks": sinks} if sinks else {}), **self._scales(layer))

    def fork(self, src, dst, stream=None):
        """The tokens of slots src [n] (as cached_lens counts them: a plan without new
        tokens adds the last accept counts) into the empty slots dst [n], in all layers."""
        _lib.paged_fork(src, dst, self.cached_lens, self.block_table, self.held_blocks,
                        self.free_blocks, self.pool, self.copies, self.copied, self.page_size,
                        shares=self.shares, status=self.status, stream=stream)
        self._copy(stream)

    def free(self, slots, stream=None):
        """Gives up all tokens and blocks of slots [n]."""
        _lib.paged_free(slots, self.cached_lens, self.block_table, self.held_blocks,
                        self.free_blocks, self.pool, shares=self.shares, status=self.status,
                        stream=stream)

    def compact(self, stream=None):
        """Moves the held blocks to the lowest numbers, in all layers: then the blocks from
        num_blocks - pool[0] on hold nothing. Plans made before it hold for no more calls."""
        if self._compacting is None:
            need = _lib.paged_compact_workspace_bytes(self.free_blocks.shape[0])
            with torch.cuda.stream(stream):
                self._compacting = _lib.workspace(need, self.pool.device)
        _lib.paged_compact(self.block_table, self.held_blocks, self.free_blocks, self.pool,
                           self.copies, self.copied, shares=self.shares,
                           workspace_buf=self._compacting, status=self.status, stream=stream)
        self._copy(stream)

    def _copy(self, stream):
        kept = self._caches
        kept.tensors = list(zip(self.k, self.v))
        try:
            _lib.paged_copy(kept, self.copies, self.copied, status=self.status, stream=stream)
        finally:
            kept.tensors = []  # (caches that are replaced are not kept alive)

    def status_code(self) -> int:
        return int(self.status.item())


class ToyTarget:
    """A random transformer without feed-forward blocks: embedding, ``layers`` of
    attention with a residual, and an output head ([V, width], the embedding again unless
    another is set). With a ``rotary`` (rotary.Rotary) queries and keys are rotated by their
    positions, with ``qk_norm`` each head of them is normalised before; ``window`` and
    ``sinks`` are the attention's."""

    def __init__(self, V, layers, q_heads, kv_heads, head_dim, dtype=torch.bfloat16, seed=0,
                 device="cuda", rotary=None, qk_norm=False, window=0, sinks=0):
        g = torch.Generator(device=device).manual_seed(seed)
        width = q_heads * head_dim

        def w(*shape):
            return (torch.randn(*shape, device=device, generator=g) * shape[0] ** -0.5).to(dtype)
        self.heads = (q_heads, kv_heads, head_dim)
        self.embed = self.head = torch.randn(V, width, device=device, generator=g).to(dtype)
        self.qkv = [w(width, (q_heads + 2 * kv_heads) * head_dim) for _ in range(layers)]
        self.proj = [w(width, width) for _ in range(layers)]
        self.rotary, self.window, self.sinks, self.eps = rotary, window, sinks, 1e-6
        self.norms = [tuple((1 + 0.2 * torch.randn(head_dim, device=device, generator=g)).to(dtype)
                            if qk_norm else None for _ in range(2)) for _ in range(layers)]

    def forward(self, tokens, cache: PagedCache, stream=None):
        """Logits [T, V] (fp32) of the planned step's tokens [T], all on ``stream`` (or the
        current one), which has to come after whatever made the tokens."""
        Hq, H, D = self.heads
        with torch.cuda.stream(stream):
            x = self.embed[tokens]
            for layer, (wqkv, wo) in enumerate(zip(self.qkv, self.proj)):
                qkv = x @ wqkv
                q, k, v = qkv.split((Hq * D, H * D, H * D), 1)
                q, k, v = (t.unflatten(1, (-1, D)) for t in (q, k, v))
                q_norm, k_norm = self.norms[layer]
                if self.rotary is None and q_norm is None:
                    cache.append(layer, k, v, stream=stream)
                else:
                    cache.append_qk(layer, q, k, v, self.rotary, q_norm, k_norm, self.eps,
                                    stream=stream)
                out = torch.zeros(x.shape[0], Hq, D, dtype=x.dtype, device=x.device)
                cache.attend(layer, q, out, window=self.window, stream=stream,
                             **({"sinks": self.sinks} if self.sinks else {}))
                x = x + out.flatten(1) @ wo
            return (x @ self.head.T).float()


def _laid_out(rows, used, query_start, max_tokens):
    """The entries of rows [B, n] that are used (truth values [B, n]) at their requests'
    places among the planned step's tokens [max_tokens]; 0 where no token is."""
    i = torch.arange(rows.shape[1], device=rows.device)
    at = torch.where(used, query_start[:-1, None].long() + i, max_tokens)
    out = rows.new_zeros(max_tokens + 1)
    out[at] = rows
    return out[:-1]


def speculative_loop(step, target: ToyTarget, cache: PagedCache, prompts, steps, draft_logits,
                     parents=None):
    """``steps`` speculative steps after the prompts (a list of token lists, one for each
    request of the DecodeStep ``step``). draft_logits(tokens) gives the drafter's base
    logits [B, K, V] from the anchors [B]. Returns the emitted tokens (prompt excluded)
    of each request.

    With ``parents`` (for each request itself, or the request whose prompt it continues
    too; its own is not looked at) a prompt runs once and its slot is forked into its other
    samples' slots, which are empty before.

    Padding requests (slot < 0) emit nothing, and neither does a request whose prompt the
    tables refuse. A request that they refuse later (the status says so) emits nothing in
    that step and is planned again in the next, as it was."""
    w = step.w
    B, K, V = w.B, w.K, w.V
    dev = step.device
    parents = list(range(B)) if parents is None else [int(p) for p in parents]
    if len(parents) != B or any(not 0 <= p < B or parents[p] != p for p in parents):
        raise ValueError("parents must be requests that have none themselves")
    slots = w.req_state_idx.tolist()
    prompts = [list(p) if s >= 0 and a == b else []
               for b, (p, s, a) in enumerate(zip(prompts, slots, parents))]
    if any(s >= 0 and a == b and not p for b, (p, s, a) in enumerate(zip(prompts, slots, parents))):
        raise ValueError("a prompt must have a token at least")
    longest = max(1, *(len(p) for p in prompts))
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
    rows = torch.tensor([p + [0] * (longest - len(p)) for p in prompts], dtype=torch.int64,
                        device=dev)
    total = max(1, sum(len(p) for p in prompts))
    query_start, seq_lens, *_ = cache.plan(step.rsi, lens, total)
    served = seq_lens > 0
    used = served[:, None] & (torch.arange(longest, device=dev) < lens[:, None])
    logits = target.forward(_laid_out(rows, used, query_start, total), cache)
    # the prompts are in the cache; their last logits choose the first anchors
    cache.cached_lens.index_add_(0, step.rsi.clamp(min=0), torch.where(served, lens, 0))
    last = (query_start[1:].long() - 1).clamp(min=0)
    samples = [b for b in range(B) if parents[b] != b]
    if samples:  # a fork that was refused (the status says so) is a request that is not served
        of, own = (torch.tensor(x, device=dev) for x in (parents, samples))
        slot = step.rsi.clamp(min=0).long()
        empty = (step.rsi >= 0) & (cache.held_blocks[slot] == 0)
        cache.fork(torch.where(served, step.rsi, -1)[of[own]], step.rsi[own])
        forked = served[of] & empty & (cache.held_blocks[slot] > 0)
        served = served.index_copy(0, own, forked[own])
        last = last[of]
    rsi = torch.where(served, step.rsi, -1)
    anchor = torch.where(served, logits[last].argmax(1), 0)
    emitted = [torch.where(served, anchor, -1)[:, None]]
    new = torch.full((B,), K + 1, dtype=torch.int32, device=dev)
    accepted = torch.full((B,), -1, dtype=torch.int32, device=dev)  # not yet in cached_lens
    i = torch.arange(K + 1, device=dev)
    for _ in range(steps):
        step.base.copy_(draft_logits(anchor))
        step.anchor.copy_(anchor)
        query_start, seq_lens, *_ = cache.plan(rsi, new, B * (K + 1), accepted)
        served = seq_lens > 0
        step.pos.copy_((seq_lens - K).clamp(min=0))  # of the first draft
        step.markov()
        tokens = torch.cat([anchor[:, None], step.draft.long()], 1)
        tokens = _laid_out(tokens, served[:, None].expand(-1, K + 1), query_start, B * (K + 1))
        at = (query_start[:-1, None].long() + i).clamp(max=B * (K + 1) - 1)
        step.target.copy_(target.forward(tokens, cache)[at])
        step.verify()
        accepted = torch.where(served, step.num_accepted, accepted)
        out = step.out.long()
        anchor = torch.where(served, out.gather(1, accepted.long().clamp(min=0)[:, None])[:, 0],
                             anchor)
        emitted.append(torch.where(served[:, None], out, -1))
    out = torch.cat(emitted, 1).tolist()
    return [[t for t in row if t >= 0] for row in out]


def main(argv=None):
    """Speculative decoding of a small random model on the paged cache:
    python -m verify_dspark_markov_step_gb300.paged --batch 8 --steps 20"""
    import argparse

    from . import build, workloads
    from .rotary import Rotary
    from .step import DecodeStep

    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=7)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--e4m3", action="store_true", help="8-bit cache")
    ap.add_argument("--samples", type=int, default=1, help="samples of each prompt (of a batch)")
    ap.add_argument("--rope", action="store_true", help="rotary positions and head norms")
    ap.add_argument("--window", type=int, default=0, help="attention window")
    ap.add_argument("--sinks", type=int, default=0, help="first tokens visible beside the window")
    args = ap.parse_args(argv)
    if args.samples < 1:
        ap.error("--samples must be 1 at least")
    build.build()
    V, layers, heads = 4096, 2, (8, 2, 128)
    w = workloads.custom(args.batch, args.drafts, V, 64, w_std=0.0)
    step = DecodeStep(w)
    target = ToyTarget(V, layers, *heads, rotary=Rotary(heads[2]) if args.rope else None,
                       qk_norm=args.rope, window=args.window, sinks=args.sinks)
    max_len = args.prompt + (args.steps + 1) * (args.drafts + 1)
    ones = torch.full((layers, heads[1]), 0.02, device="cuda") if args.e4m3 else None
    cache = PagedCache(layers=layers, slots=w.S, max_len=max_len,
                       num_blocks=w.S * -(-max_len // args.page), page_size=args.page,
                       q_heads=heads[0], kv_heads=heads[1], head_dim=heads[2],
                       cache_dtype=torch.float8_e4m3fn if args.e4m3 else None, k_scale=ones,
                       v_scale=ones, sharing=args.samples > 1)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(V, (args.prompt - 3 * b,), generator=g).tolist()
               for b in range(args.batch)]
    scores = (target.embed @ target.embed.T).float()

    def draft_logits(anchor):  # a drafter that expects the anchor's neighbours
        return scores[anchor][:, None].expand(-1, args.drafts, -1)
    parents = [b - b % args.samples for b in range(args.batch)]
    out = speculative_loop(step, target, cache, prompts, args.steps, draft_logits, parents)
    torch.cuda.synchronize()
    made = sum(len(o) - 1 for o in out)
    left = int(cache.pool[0])
    cache.free(step.rsi[::2].contiguous())  # half of the requests end
    cache.compact()
    torch.cuda.synchronize()
    print(f"{args.batch} requests, {args.steps} steps: status {cache.status_code()} / "
          f"{step.status_code()}, {made / args.steps / args.batch:.2f} tokens a step and request, "
          f"{left} blocks free, {int(cache.pool[0])} without every second request")


if __name__ == "__main__":
    main()
