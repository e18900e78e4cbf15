"""The speculative loop's bookkeeping without a GPU: the cache's tables by their
plain statement, a target that reads every token back from the slots the tables
give, a drafter that is right half of the time. What the loop emits has to be what
the target says one token at a time, for every request that is served."""
import types

import numpy as np
import pytest

import paged_oracle as po

torch = pytest.importorskip("torch")
V = 97


def _next(history):
    """The target's greedy choice after a list of tokens."""
    likely = (3 * history[-1] + 1) % V  # what the drafter expects
    return likely if sum(history) % 4 else (likely + sum(history) // 4 + 1) % V


def _generate(prompt, n):
    out = list(prompt)
    for _ in range(n):
        out.append(_next(out))
    return out[len(prompt):]


class Cache:
    """PagedCache's plan on lists."""

    def __init__(self, slots, max_len, num_blocks, page):
        self.page, self.codes = page, set()
        self.table = [[-1] * -(-max_len // page) for _ in range(slots)]
        self.held, self.stack = [0] * slots, list(range(num_blocks))[::-1]
        self.cached_lens = torch.zeros(slots, dtype=torch.int32)

    def plan(self, rsi, new, max_tokens, num_accepted=None, stream=None):
        o = po.tables(rsi.tolist(), new.tolist(), self.cached_lens.tolist(),
                      None if num_accepted is None else num_accepted.tolist(), self.table,
                      self.held, self.stack, len(self.stack), max_tokens, self.page)
        self.table, self.held, self.stack = o["block_table"], o["held_blocks"], o["stack"]
        self.codes |= o["status"]
        if num_accepted is not None:
            self.cached_lens.copy_(torch.tensor(o["cached_lens"]))
        self.rsi = rsi.tolist()
        self.step = (torch.tensor(o["query_start"], dtype=torch.int32),
                     torch.tensor(o["seq_lens"], dtype=torch.int32),
                     torch.tensor(o["positions"]), torch.tensor(o["slot_map"]))
        return self.step


class Target:
    def __init__(self):
        self.store = {}

    def forward(self, tokens, cache):
        start, seq, positions, slots = (t.tolist() for t in cache.step)
        assert tokens.shape[0] == len(slots)
        for t, s in zip(tokens.tolist(), slots):
            if s >= 0:
                self.store[s] = t
        logits = torch.zeros(len(slots), V)
        for b, r in enumerate(cache.rsi):
            for t in range(start[b], start[b + 1]):
                past = [self.store[cache.table[r][p // cache.page] * cache.page + p % cache.page]
                        for p in range(positions[t] + 1)]
                logits[t, _next(past)] = 1.0
        return logits


class Step:
    """DecodeStep at temperature 0."""

    def __init__(self, rsi, K):
        B = len(rsi)
        self.w = types.SimpleNamespace(B=B, K=K, V=V, req_state_idx=np.array(rsi, np.int32))
        self.device = "cpu"
        self.rsi = torch.tensor(rsi, dtype=torch.int32)
        self.base, self.target = torch.zeros(B, K, V), torch.zeros(B, K + 1, V)
        self.anchor = torch.zeros(B, dtype=torch.int32)
        self.pos = torch.zeros(B, dtype=torch.int64)
        self.draft = torch.full((B, K), -1, dtype=torch.int32)
        self.out = torch.full((B, K + 1), -1, dtype=torch.int32)
        self.num_accepted = torch.zeros(B, dtype=torch.int32)
        self.first_drafts = []

    def markov(self):
        self.draft.copy_(torch.where(self.rsi[:, None] >= 0, self.base.argmax(2), -1))
        self.first_drafts.append(self.pos.clone())

    def verify(self):
        for b, s in enumerate(self.rsi.tolist()):
            self.out[b], self.num_accepted[b] = -1, -1 if s < 0 else 0
            for i in range(self.w.K + 1 if s >= 0 else 0):
                best = int(self.target[b, i].argmax())
                self.out[b, i] = best
                if i == self.w.K or best != int(self.draft[b, i]):
                    break
                self.num_accepted[b] += 1


def _run(rsi, lens, K=3, steps=9, blocks=200, page=16, slots=8, before_step=None):
    from verify_dspark_markov_step_gb300.paged import speculative_loop
    r = np.random.RandomState(3)
    prompts = [[int(x) for x in r.randint(V, size=n)] for n in lens]
    step, cache = Step(rsi, K), Cache(slots, 300, blocks, page)
    calls = []

    def draft_logits(anchor):
        """The chain 3 t + 1 from the anchor."""
        if before_step:
            before_step(len(calls), cache)
        calls.append(anchor.clone())
        out = torch.zeros(len(rsi), K, V)
        for b, t in enumerate(anchor.tolist()):
            for i in range(K):
                t = (3 * t + 1) % V
                out[b, i, t] = 1.0
        return out
    out = speculative_loop(step, Target(), cache, prompts, steps, draft_logits)
    return prompts, out, cache, step


def test_requests_follow_the_target():
    prompts, out, cache, step = _run([3, 0, 7, 2], [1, 40, 17, 100])
    assert not cache.codes
    accepted = 0
    for p, o in zip(prompts, out):
        assert len(o) >= 10 and o == _generate(p, len(o))
        accepted += len(o) - 10
    assert accepted > 20
    assert step.first_drafts[0].tolist() == [2, 41, 18, 101]  # the anchor's position is before


@pytest.mark.parametrize("rsi", [[-1, 4, 1], [4, -1, 1], [4, 1, -1], [-1, -1, 5]])
def test_padding_requests_emit_nothing_and_change_nothing(rsi):
    prompts, out, cache, _ = _run(rsi, [23, 31, 9])
    assert not cache.codes
    for s, p, o in zip(rsi, prompts, out):
        assert o == (_generate(p, len(o)) if s >= 0 else []) and (s < 0 or len(o) >= 10)


def test_a_refused_request_waits_and_goes_on():
    """The pool is short for one request at a time; blocks come back at the sixth
    step. A request that is refused emits nothing, keeps its accept count, and
    the others are as ever."""
    refused = []

    def give_back(step, cache):
        if step:
            refused.append([r for r, n in zip(cache.rsi, cache.step[1].tolist()) if n == 0])
        if step == 6:
            cache.stack += list(range(100, 160))
    prompts, out, cache, _ = _run([2, 5, 0, 6], [30, 30, 45, 14], steps=14, blocks=9,
                                  before_step=give_back)
    assert cache.codes == {-9}
    assert any(refused[:6]) and not any(refused[6:])
    late = {r for step in refused for r in step}
    assert 0 < len(late) < 4
    for r, p, o in zip([2, 5, 0, 6], prompts, out):
        assert o == _generate(p, len(o))
        assert len(o) >= (15 if r not in late else 9)


def test_a_request_whose_prompt_is_refused_is_padding_from_then_on():
    """(and with it, as the tables have it, those after it that need blocks)"""
    prompts, out, cache, _ = _run([2, 5, 0], [30, 90, 12], blocks=6, steps=4)
    assert cache.codes == {-9} and out[1] == out[2] == []
    assert cache.held[5] == cache.held[0] == 0
    assert len(out[0]) >= 5 and out[0] == _generate(prompts[0], len(out[0]))


def test_a_batch_of_padding_emits_nothing():
    assert _run([-1, -1], [4, 5])[1] == [[], []]


def test_an_empty_prompt_is_refused():
    with pytest.raises(ValueError, match="prompt"):
        _run([2, 5], [3, 0])
