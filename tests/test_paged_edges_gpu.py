"""Edges of the paged attention and append on the GPU. Bounds are those of
test_paged_gpu.py, whose ragged batches (``Attend``) these tests use."""
import math

import pytest

import paged_oracle as po
from gpu_util import require_gpu
from test_paged_gpu import Attend, _half_eps, _ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
def test_requests_of_one_key_tile_over_an_8_bit_cache(D, dtype):
    """Units of one key tile, several to a CTA (of one key head: each alone), of
    which a warpgroup has nothing to do, and longer ones between them: every call
    of many in a row gives the definition's result, the same bits each time."""
    torch = require_gpu()
    for seed, case in enumerate((_ragged(1000, 0, 120, 1, 21), _ragged(700, 0, 300, 3, 22))):
        a = Attend(torch, seed=seed, **case, Hq=4, H=1, D=D, page=16, dtype=dtype,
                   cache="float8_e4m3fn")
        a.check()
        want, want_lse = a.out.clone(), a.lse.clone()
        for _ in range(60):
            a.call()
        torch.cuda.synchronize()
        assert a.status.item() == 0
        assert torch.equal(a.out, want) and torch.equal(a.lse, want_lse)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 70), (False, 0)])
@pytest.mark.parametrize("small", [2.0 ** -10, 2.0 ** -40])
def test_a_zero_softmax_scale_over_an_8_bit_cache(small, causal, window):
    """Every visible key weighs the same, whatever the size of the query rows,
    the scales of the cache's heads and what is masked."""
    torch = require_gpu()
    a = Attend(torch, [400, 260, 0, 7], [5, 200, 0, 2], Hq=4, H=2, D=64, page=16, seed=8,
               cache="float8_e4m3fn")
    a.q.copy_((a.q.float() * small).to(a.q.dtype))
    a.scale = 0.0
    a.check(causal, window)


@pytest.mark.parametrize("cache", [None, "float8_e4m3fn"])
@pytest.mark.parametrize("H,D,news,lens", [
    (5, 64, [1] * 40, list(range(90, 490, 10))),       # heads side by side
    (5, 128, [3, 40, 1], [300, 90, 1300]),             # one row tile, cut units
    (5, 128, [200, 333], [200, 700])])                 # two row tiles
def test_scales_of_zero_and_below(cache, H, D, news, lens):
    """A head's scale multiplies what the cache stores, of either sign or zero."""
    torch = require_gpu()
    a = Attend(torch, lens, news, Hq=2 * H, H=H, D=D, page=32, cache=cache, seed=11)
    size = 0.01 if cache else 1.0
    a.ks = size * torch.tensor([1.25, -1.5, 0.0, -0.75, 1.0], device="cuda")
    a.vs = size * torch.tensor([-1.0, 1.5, 0.5, 0.0, -2.0], device="cuda")
    a.check()
    a.check(True, 100)
