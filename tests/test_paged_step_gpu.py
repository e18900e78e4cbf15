"""The paged cache in a speculative decoding loop: Markov drafts, the target's
forward on the paged cache, rejection sampling, and the next step's tables from
the accept counts, all on the device."""
import math

import pytest

from gpu_util import require_gpu
from verify_dspark_markov_step_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def _plain_logits(torch, target, tokens):
    """The toy target's logits for every position of a token list, in 64 bits."""
    Hq, H, D = target.heads
    x = target.embed[torch.tensor(tokens, device="cuda")].double()
    n = len(tokens)
    hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    for wqkv, wo in zip(target.qkv, target.proj):
        q, k, v = (x @ wqkv.double()).split((Hq * D, H * D, H * D), 1)
        q = q.view(n, H, Hq // H, D)
        s = torch.einsum("nhgd,mhd->hgnm", q, k.view(n, H, D)) * D ** -0.5
        p = s.masked_fill(hidden, -math.inf).softmax(-1)
        out = torch.einsum("hgnm,mhd->nhgd", p, v.view(n, H, D)).reshape(n, Hq * D)
        x = x + out @ wo.double()
    return x @ target.embed.double().T


@pytest.mark.parametrize("cache_dtype,page,K", [(None, 16, 3), ("float8_e4m3fn", 32, 5)])
def test_greedy_speculation_emits_the_targets_own_tokens(cache_dtype, page, K):
    """At temperature 0 the loop's tokens are what the target would choose one by
    one, whatever the drafter proposes: the logit of every emitted token is the
    largest, within the rounding of the 16-bit forward (8-bit: of the cache)."""
    torch = require_gpu()
    from verify_dspark_markov_step_gb300.paged import PagedCache, ToyTarget, speculative_loop
    from verify_dspark_markov_step_gb300.step import DecodeStep
    B, V, heads, steps = 5, 512, (4, 2, 64), 9
    w = wl.custom(B, K, V, 64, w_std=0.0, temperature=0.0, S=9, rsi=[7, 0, 3, 8, 2])
    step = DecodeStep(w)
    target = ToyTarget(V, 2, *heads, seed=3)
    scale = torch.full((2, 2), 0.02, device="cuda") if cache_dtype else None
    cache = PagedCache(layers=2, slots=9, max_len=400, num_blocks=9 * 25, page_size=page,
                       q_heads=4, kv_heads=2, head_dim=64,
                       cache_dtype=getattr(torch, cache_dtype) if cache_dtype else None,
                       k_scale=scale, v_scale=scale)
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(V, (n,), generator=g).tolist() for n in (1, 17, 64, 200, 333)]
    table = torch.randn(V, V, device="cuda", generator=torch.Generator("cuda").manual_seed(9))

    def draft_logits(anchor):
        # half of the drafts follow the target's favourite, so that some are accepted
        near = (target.embed @ target.embed.T).float()[anchor][:, None].repeat(1, K, 1)
        near[::2] = table[anchor[::2]][:, None]
        return near
    out = speculative_loop(step, target, cache, prompts, steps, draft_logits)
    torch.cuda.synchronize()
    assert cache.status_code() == 0 and step.status_code() == 0
    for b in range(B):
        assert len(out[b]) >= steps + 1
        tokens = prompts[b] + out[b]
        logits = _plain_logits(torch, target, tokens)[len(prompts[b]) - 1:-1]
        chosen = logits.gather(1, torch.tensor(out[b], device="cuda")[:, None])[:, 0]
        # a bf16 forward: about ten roundings of 2^-8 on sums of `width` terms of
        # logits' scale; the 8-bit cache adds roundings of 2^-4 to keys and values
        spread = logits.std(1)
        room = spread * (0.5 if cache_dtype else 0.1)
        assert (logits.amax(1) - chosen <= room).all()
        # slots and lengths: what was kept is the prompt and all but the last token
        kept = int(cache.cached_lens[w.req_state_idx[b]]) + int(step.num_accepted[b]) + 1
        assert kept == len(tokens) - 1
    # no block was lost: held and free ones make up the pool
    held = cache.held_blocks.tolist()
    owned = [int(cache.block_table[s, j]) for s in range(9) for j in range(held[s])]
    free = cache.free_blocks[:int(cache.pool[0])].tolist()
    assert sorted(owned + free) == list(range(9 * 25))


def test_the_command_runs():
    require_gpu()
    from verify_dspark_markov_step_gb300 import paged
    paged.main(["--batch", "3", "--drafts", "3", "--prompt", "40", "--steps", "3"])
    paged.main(["--batch", "2", "--drafts", "2", "--prompt", "70", "--steps", "2", "--e4m3"])
