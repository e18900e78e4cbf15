"""The bound of the whole cached forward with norms, rotation, window and sinks tells
its roundings from mistakes; the loop's refusals of parents."""
import pytest
import torch

import paged_layers_oracle as lo
from verify_dspark_markov_step_gb300.paged import ToyTarget
from verify_dspark_markov_step_gb300.rotary import Rotary


def made(interleaved, device="cpu"):
    return lo.sharp(ToyTarget(300, 2, 4, 2, 64, seed=3, device=device, qk_norm=True, window=40, sinks=5,
                              rotary=Rotary(32, 1e4, interleaved=interleaved, device=device)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eight", [False, True])
def test_the_bound_tells_roundings_from_mistakes(interleaved, eight):
    target = made(interleaved)
    tokens = torch.randint(300, (150,), generator=torch.Generator().manual_seed(2)).tolist()
    want = lo.logits(target, tokens)

    def rounded(t, what):
        if what == "cache" and eight:
            return (t / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).double() * 0.02
        return t.to(torch.bfloat16).double()
    off = (lo.logits(target, tokens, rounded) - want).abs()
    assert off.max() < lo.room(want, eight) / 3, off.max() / want.std()
    for mistake in lo.MISTAKES:
        off = (lo.logits(target, tokens, mistake=mistake) - want).abs()
        assert off.max() > 1.2 * lo.room(want, eight), (mistake, off.max() / want.std())


def test_parents_have_none_themselves():
    import types
    from verify_dspark_markov_step_gb300.paged import speculative_loop
    step = types.SimpleNamespace(device="cpu", w=types.SimpleNamespace(B=3, K=2, V=10, req_state_idx=torch.tensor([0, 1, 2])))
    for parents in ([0, 0], [0, 0, 1], [0, 1, 3], [0, -1, 2]):
        with pytest.raises(ValueError, match="parents"):
            speculative_loop(step, None, None, [[1]] * 3, 1, None, parents)
    with pytest.raises(ValueError, match="token"):
        speculative_loop(step, None, None, [[], [1], [1]], 1, None, [0, 0, 2])
