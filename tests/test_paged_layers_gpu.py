"""Norms, rotation, pages, window with sinks, forks, frees and compaction together, as a
server uses them: every logit against 64 bits."""
import pytest
import torch

import paged_layers_oracle as lo
from gpu_util import require_gpu
from test_paged_layers_cpu import made
from verify_dspark_markov_step_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def _cache(eight, sharing, slots=6, blocks=80):
    from verify_dspark_markov_step_gb300.paged import PagedCache
    scale = torch.full((2, 2), 0.02, device="cuda") if eight else None
    return PagedCache(layers=2, slots=slots, max_len=320, num_blocks=blocks, page_size=16, q_heads=4, kv_heads=2,
                      head_dim=64, cache_dtype=torch.float8_e4m3fn if eight else None, k_scale=scale, v_scale=scale,
                      sharing=sharing)


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("sharing", [False, True])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_conversation_forked_freed_and_compacted(interleaved, eight, sharing):
    require_gpu()
    target = made(interleaved, "cuda")
    cache = _cache(eight, sharing)
    g = torch.Generator().manual_seed(4)
    said = {}  # tokens of each slot

    def run(news):
        """Appends tokens to slots; every logit of theirs against 64 bits."""
        slots = list(news)
        flat = [t for s in slots for t in news[s]]
        pad = 5
        query_start, seq_lens, *_ = cache.plan(_ints(*slots, -1), _ints(*(len(news[s]) for s in slots), 0), len(flat) + pad)
        got = target.forward(torch.tensor(flat + [0] * pad, device="cuda"), cache)
        cache.cached_lens[torch.tensor(slots, device="cuda")] = seq_lens[:-1]
        starts = query_start.tolist()
        for i, s in enumerate(slots):
            said[s] = said.get(s, []) + news[s]
            assert int(seq_lens[i]) == len(said[s])
            want = lo.logits(target, said[s])
            off = (got[starts[i]:starts[i + 1]].double() - want[-len(news[s]):]).abs().max()
            assert off <= lo.room(want, eight), (s, off / want.std())

    def some(n):
        return torch.randint(300, (n,), generator=g).tolist()
    run({3: some(150), 0: some(16), 5: some(1)})
    run({3: some(7), 5: some(60), 0: some(32)})
    # the first prompt in two samples, one whose length fills its pages in another
    cache.fork(_ints(3, 0, 3), _ints(1, 2, 4))
    said[1], said[2], said[4] = list(said[3]), list(said[0]), list(said[3])
    run({1: some(9), 3: some(9), 4: some(1), 2: some(20)})
    # the parents leave, their samples stay
    cache.free(_ints(3, 0))
    del said[3], said[0]
    run({2: some(3), 1: some(40)})
    cache.compact()
    torch.cuda.synchronize()
    used = 80 - int(cache.pool[0])
    rows = [cache.block_table[s, :int(cache.held_blocks[s])] for s in (1, 2, 4, 5)]
    assert all((r < used).all() and (r >= 0).all() for r in rows)
    run({1: some(5), 2: some(5), 4: some(33), 5: some(5)})
    # freed slots are used again
    cache.fork(_ints(1), _ints(3))
    said[3] = list(said[1])
    run({3: some(2), 0: some(20)})
    cache.free(_ints(0, 1, 2, 3, 4, 5))
    torch.cuda.synchronize()
    assert cache.status_code() == 0 and int(cache.pool[0]) == 80
    assert sorted(cache.free_blocks.tolist()) == list(range(80))
    assert not sharing or not cache.shares.any()


@pytest.mark.parametrize("sharing", [False, True])
def test_greedy_speculation_of_samples_emits_the_targets_own_tokens(sharing):
    """Samples of a prompt run once and forked: at temperature 0 they emit what their parent
    does, which is what the target would choose."""
    require_gpu()
    from verify_dspark_markov_step_gb300.paged import speculative_loop
    from verify_dspark_markov_step_gb300.step import DecodeStep
    B, K, steps = 5, 3, 6
    target = made(False, "cuda")
    w = wl.custom(B, K, 300, 64, w_std=0.0, temperature=0.0, S=6, rsi=[4, 0, -1, 3, 2])
    step = DecodeStep(w)
    cache = _cache(False, sharing, blocks=120)
    prompts = [torch.randint(300, (n,), generator=torch.Generator().manual_seed(n)).tolist() for n in (77, 1, 3, 1, 64)]

    def draft_logits(anchor):
        return (target.embed @ target.embed.T).float()[anchor][:, None].repeat(1, K, 1)
    out = speculative_loop(step, target, cache, prompts, steps, draft_logits, parents=[0, 0, 0, 0, 4])
    torch.cuda.synchronize()
    assert cache.status_code() == 0 and step.status_code() == 0
    assert out[1] == out[0] == out[3] and out[2] == [] and len(out[0]) >= steps + 1 and len(out[4]) >= steps + 1
    for b in (0, 4):
        want = lo.logits(target, prompts[b] + out[b])[len(prompts[b]) - 1:-1]
        chosen = want.gather(1, torch.tensor(out[b], device="cuda")[:, None])[:, 0]
        assert (want.amax(1) - chosen <= lo.room(want, False)).all()


def test_a_fork_that_does_not_fit_is_not_served():
    require_gpu()
    from verify_dspark_markov_step_gb300.paged import speculative_loop
    from verify_dspark_markov_step_gb300.step import DecodeStep
    target = made(False, "cuda")
    w = wl.custom(3, 2, 300, 64, w_std=0.0, temperature=0.0, S=4, rsi=[0, 1, 2])
    step = DecodeStep(w)
    cache = _cache(False, False, slots=4, blocks=12)  # a prompt of 5 blocks, one sample, room to go on
    prompt = torch.randint(300, (70,), generator=torch.Generator().manual_seed(1)).tolist()

    def draft_logits(anchor):
        return torch.zeros(3, 2, 300, device="cuda")
    out = speculative_loop(step, target, cache, [prompt, [], []], 2, draft_logits, parents=[0, 0, 0])
    torch.cuda.synchronize()
    assert cache.status_code() == -9
    assert out[0] == out[1] and len(out[0]) >= 3 and out[2] == []


def test_a_sample_whose_slot_is_taken_is_not_served():
    require_gpu()
    from verify_dspark_markov_step_gb300.paged import speculative_loop
    from verify_dspark_markov_step_gb300.step import DecodeStep
    target = made(False, "cuda")
    w = wl.custom(3, 2, 300, 64, w_std=0.0, temperature=0.0, S=4, rsi=[0, 1, 2])
    step = DecodeStep(w)
    cache = _cache(False, True, slots=4, blocks=40)
    prompt = torch.randint(300, (70,), generator=torch.Generator().manual_seed(1)).tolist()
    cache.plan(_ints(1), _ints(70), 70)  # slot 1 holds something of another's
    cache.cached_lens[1] = 70

    def draft_logits(anchor):
        return torch.zeros(3, 2, 300, device="cuda")
    out = speculative_loop(step, target, cache, [prompt, [], []], 2, draft_logits, parents=[0, 0, 0])
    torch.cuda.synchronize()
    assert cache.status_code() == -5
    assert out[1] == [] and out[2] == out[0] and len(out[0]) >= 3
    assert int(cache.cached_lens[1]) == 70 and int(cache.held_blocks[1]) == 5


def test_caches_that_were_replaced_are_the_ones_copied():
    require_gpu()
    cache = _cache(False, False, slots=3, blocks=12)
    cache.plan(_ints(0), _ints(20), 20)
    cache.cached_lens[0] = 20
    cache.fork(_ints(0), _ints(1))
    cache.k[1] = torch.randn_like(cache.k[1])
    cache.k.append(torch.randn_like(cache.k[0])), cache.v.append(torch.randn_like(cache.v[0]))
    cache.fork(_ints(0), _ints(2))
    torch.cuda.synchronize()
    a, b = cache.block_table[0, :2].long(), cache.block_table[2, :2].long()
    assert cache.status_code() == 0
    for c in cache.k + cache.v:
        assert torch.equal(c[a], c[b])


def test_the_command_runs_with_samples_rotation_and_sinks():
    require_gpu()
    from verify_dspark_markov_step_gb300 import paged
    paged.main(["--batch", "4", "--drafts", "3", "--prompt", "90", "--steps", "3", "--samples", "2", "--rope",
                "--window", "48", "--sinks", "4"])
    paged.main(["--batch", "3", "--drafts", "2", "--prompt", "40", "--steps", "2", "--rope", "--e4m3"])
