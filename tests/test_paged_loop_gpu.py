"""The speculative loop on the GPU with padding requests, a cache that is full for
a while, and a target whose tokens depend on what the cache holds."""
import pytest

from gpu_util import require_gpu
from verify_dspark_markov_step_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

HEADS, V, K, PAGE = (4, 2, 64), 512, 3, 16


def _loop(torch, rsi, prompts, steps, blocks=None, before_step=None):
    """speculative_loop at temperature 0: (emitted tokens, cache, step)."""
    from verify_dspark_markov_step_gb300.paged import PagedCache, ToyTarget, speculative_loop
    from verify_dspark_markov_step_gb300.step import DecodeStep
    step = DecodeStep(wl.custom(len(rsi), K, V, 64, w_std=0.0, temperature=0.0, S=9, rsi=rsi))
    target = ToyTarget(V, 2, *HEADS, seed=3)
    cache = PagedCache(layers=2, slots=9, max_len=400, num_blocks=blocks or 9 * 25,
                       page_size=PAGE, q_heads=HEADS[0], kv_heads=HEADS[1], head_dim=HEADS[2])
    near = (target.embed @ target.embed.T).float()
    calls = []

    def draft_logits(anchor):
        if before_step:
            before_step(len(calls), cache)
        calls.append(0)
        return near[anchor][:, None].repeat(1, K, 1)
    out = speculative_loop(step, target, cache, prompts, steps, draft_logits)
    torch.cuda.synchronize()
    return out, cache, step


def _prompts(torch, lens):
    g = torch.Generator().manual_seed(7)
    return [torch.randint(V, (n,), generator=g).tolist() for n in lens]


def test_padding_requests_in_the_loop():
    torch = require_gpu()
    prompts = _prompts(torch, (1, 60, 200, 33))
    want, _, _ = _loop(torch, [7, 0, 3, 8], prompts, 6)
    out, cache, step = _loop(torch, [-1, 7, 0, -1, 3, 8, -1],
                             [[1, 2], *prompts[:2], [], *prompts[2:], [9]], 6)
    assert cache.status_code() == 0 and step.status_code() == 0
    assert out[0] == out[3] == out[6] == []
    assert [out[b] for b in (1, 2, 4, 5)] == want


@pytest.mark.parametrize("spare", [1, 3])
def test_a_full_cache_in_the_loop(spare):
    """The pool is short of blocks until the fifth step: a request that is refused
    emits nothing, then goes on where it was; the others' tokens stay."""
    torch = require_gpu()
    prompts = _prompts(torch, (40, 60, 90, 30))
    rsi, steps = [7, 0, 3, 8], 9
    want, _, _ = _loop(torch, rsi, prompts, steps)
    blocks = 40
    held_back, refused = [], []

    def before_step(n, cache):
        count = int(cache.pool[0])
        if n == 0:  # the prompts are in
            held_back.extend(cache.free_blocks[spare:count].tolist())
            cache.pool[0] = spare
        else:
            refused.append([b for b, x in enumerate(cache.step[1].tolist()) if x == 0])
        if n == 5:
            cache.free_blocks[count:count + len(held_back)] = torch.tensor(
                held_back, dtype=torch.int32, device="cuda")
            cache.pool[0] = count + len(held_back)
    out, cache, step = _loop(torch, rsi, prompts, steps, blocks, before_step)
    assert cache.status_code() == -9 and step.status_code() == 0
    assert any(refused[:5]) and not any(refused[5:])
    late = {b for r in refused for b in r}
    for b in range(4):
        n = len(out[b])
        assert out[b] == want[b][:n]
        assert n == len(want[b]) if b not in late else n >= 1 + steps - 5
    held = cache.held_blocks.tolist()
    owned = [int(cache.block_table[s, j]) for s in range(9) for j in range(held[s])]
    free = cache.free_blocks[:int(cache.pool[0])].tolist()
    assert sorted(owned + free) == list(range(blocks))


@pytest.mark.parametrize("cache_dtype,page,K", [(None, 16, 3), ("float8_e4m3fn", 32, 5)])
def test_every_logit_of_the_cached_forward(cache_dtype, page, K):
    """A target whose logits depend on what was cached, drafts that are its own
    greedy tokens for every other request: all logits of the prompts and of every step
    against the target's over the whole token list, in 64 bits."""
    torch = require_gpu()
    import paged_target as pt
    from verify_dspark_markov_step_gb300.paged import PagedCache, ToyTarget, speculative_loop
    from verify_dspark_markov_step_gb300.step import DecodeStep
    rsi = [7, -1, 0, 3, 8, 2]
    lens, steps = [1, 4, 17, 64, 200, 333], 7
    step = DecodeStep(wl.custom(len(rsi), K, V, 64, w_std=0.0, temperature=0.0, S=9, rsi=rsi))
    target = pt.sensitive(ToyTarget(V, 2, *HEADS, seed=3))
    scale = torch.full((2, 2), 0.02, device="cuda") if cache_dtype else None
    cache = PagedCache(layers=2, slots=9, max_len=400, num_blocks=9 * 25, page_size=page,
                       q_heads=4, kv_heads=2, head_dim=64,
                       cache_dtype=getattr(torch, cache_dtype) if cache_dtype else None,
                       k_scale=scale, v_scale=scale)
    prompts = _prompts(torch, lens)
    past, forward, worst, accepted = {}, target.forward, [], []

    def checked(tokens, cache):
        got = forward(tokens, cache)
        start, seq, positions, _ = (t.tolist() for t in cache.step)
        all_tokens = tokens.tolist()
        for b, s in enumerate(cache.req_state_idx.tolist()):
            n = start[b + 1] - start[b]
            if s < 0:
                assert n == 0
                continue
            kept = seq[b] - n
            assert positions[start[b]:start[b + 1]] == list(range(kept, seq[b]))
            past[s] = past.get(s, [])[:kept] + all_tokens[start[b]:start[b + 1]]
            assert len(past[s]) == seq[b]
            want = pt.logits(target, past[s])
            off = (got[start[b]:start[b + 1]].double() - want[-n:]).abs().max()
            worst.append((off / pt.room(want, cache_dtype is not None)).item())
        return got
    target.forward = checked

    def draft_logits(anchor):
        out = torch.zeros(len(rsi), K, V, device="cuda")
        for b, s in enumerate(rsi):
            if s < 0 or b % 2:
                continue
            kept = len(past[s]) - (K + 1) + int(step.num_accepted[b]) + 1 if accepted else lens[b]
            seen = past[s][:kept] + [int(anchor[b])]
            for i in range(K):
                seen.append(int(pt.logits(target, seen)[-1].argmax()))
                out[b, i, seen[-1]] = 9.0
        accepted.append(step.num_accepted.clone())
        return out
    out = speculative_loop(step, target, cache, prompts, steps, draft_logits)
    torch.cuda.synchronize()
    assert cache.status_code() == 0 and step.status_code() == 0
    assert len(worst) == 5 * (steps + 1) and max(worst) <= 1.0, max(worst)
    assert out[1] == [] and all(len(out[b]) >= steps + 1 for b in (0, 2, 3, 4, 5))
    if not cache_dtype:  # (an e4m3 cache may choose other tokens than 64 bits)
        assert sum(len(out[b]) for b in (0, 2, 4)) > 3 * (steps + 1) + 2 * K
