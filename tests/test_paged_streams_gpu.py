"""The paged cache on streams other than the current one."""
import pytest

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _cache(torch, layers, heads, max_len, slots):
    from verify_dspark_markov_step_gb300.paged import PagedCache
    return PagedCache(layers=layers, slots=slots, max_len=max_len,
                      num_blocks=slots * -(-max_len // 16), page_size=16, q_heads=heads[0],
                      kv_heads=heads[1], head_dim=heads[2])


def test_a_forward_on_a_side_stream():
    """While the current stream is busy: the same logits, bit for bit."""
    torch = require_gpu()
    from verify_dspark_markov_step_gb300.paged import ToyTarget
    heads, lens = (8, 2, 64), [300, 7, 90]
    target = ToyTarget(512, 2, *heads, seed=2)
    tokens = torch.randint(512, (sum(lens),), device="cuda")
    rsi = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    new = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def forward(stream, busy):
        cache = _cache(torch, 2, heads, 400, 3)
        torch.cuda.synchronize()
        if busy:
            for _ in range(20):
                busy[0].copy_(busy[0] @ busy[1])
        cache.plan(rsi, new, sum(lens), stream=stream)
        out = target.forward(tokens, cache, stream=stream)
        torch.cuda.synchronize()
        assert cache.status_code() == 0
        return out
    want = forward(None, None)
    big = [torch.randn(8192, 8192, device="cuda").bfloat16() for _ in range(2)]
    for _ in range(3):
        assert torch.equal(forward(torch.cuda.Stream(), big), want)


def test_attentions_of_one_plan_on_two_streams():
    """Two layers side by side, their units split over CTAs and joined: each has its
    own place for the parts."""
    torch = require_gpu()
    heads, L = (8, 2, 128), 9000
    cache = _cache(torch, 2, heads, L, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (*cache.k, *cache.v):
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))
    rsi = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.plan(rsi, rsi + L, L)  # the table's blocks
    cache.cached_lens.fill_(L - 8)
    cache.plan(rsi, rsi + 8, 8)
    q = [torch.randn(8, 8, 128, device="cuda", generator=g).bfloat16() for _ in range(2)]
    want = [torch.empty_like(x) for x in q]
    for i in range(2):
        cache.attend(i, q[i], want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [torch.zeros_like(x) for x in q]
        torch.cuda.synchronize()
        for i in range(2):
            cache.attend(i, q[i], got[i], stream=streams[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cache.status_code() == 0
