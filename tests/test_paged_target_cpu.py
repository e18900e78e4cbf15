"""That the bound of the cached forward's logits (paged_target) tells roundings from
mistakes, on the CPU."""
import pytest

torch = pytest.importorskip("torch")
import paged_target as pt  # noqa: E402

SCALE = 0.02  # of the e4m3 cache


def _bf16(x, what):
    return x.bfloat16().double()


def _e4m3(x, what):
    if what != "cache":
        return _bf16(x, what)
    return (x / SCALE).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * SCALE


def _plain(n):
    from verify_dspark_markov_step_gb300.paged import ToyTarget
    target = pt.sensitive(ToyTarget(512, 2, 4, 2, 64, device="cpu", seed=3))
    g = torch.Generator().manual_seed(n)
    tokens = torch.randint(512, (n,), generator=g).tolist()
    return target, tokens, pt.logits(target, tokens)


@pytest.mark.parametrize("n", [1, 17, 64, 200, 333])
def test_roundings_stay_within_the_bound(n):
    target, tokens, want = _plain(n)
    for eight, rounded in ((False, _bf16), (True, _e4m3)):
        off = (pt.logits(target, tokens, rounded=rounded) - want).abs().max()
        assert off <= pt.room(want, eight) / 2


@pytest.mark.parametrize("n", [17, 64, 200, 333])
@pytest.mark.parametrize("mistake", [
    lambda p, v: pt.attend(p, v) * 0, lambda p, v: -pt.attend(p, v),
    lambda p, v: pt.attend(p, v.roll(1, 0)),       # every value one position on
    lambda p, v: pt.attend(p, v.flip(0)),          # in another order
    lambda p, v: pt.attend(p, v.flip(1)),          # another head's
    lambda p, v: pt.attend((p > 0) / (p > 0).sum(-1, keepdim=True).double(), v)],
    ids=["zero", "negated", "shifted", "reversed", "heads", "no scores"])
def test_mistakes_do_not(n, mistake):
    """Planted in the plain target: beyond the bound in its last four positions."""
    target, tokens, want = _plain(n)
    off = (pt.logits(target, tokens, attend=mistake) - want)[-4:].abs().max()
    assert off > pt.room(want, True)
