"""Copies of blocks of more chunks than a launch has CTAs for, in the caches of many layers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H,P,D,layers,N,n", [
    ("bf16", 8, 256, 128, 64, 4, 2),    # 16 chunks a block, ten CTAs in x
    ("bf16", 8, 256, 128, 70, 4, 2),    # and six layers in a second launch
    ("bf16", 5, 256, 128, 64, 7, 3),    # ten chunks: as many as CTAs
    ("e4m3", 11, 256, 128, 64, 7, 3),   # eleven
    ("fp16", 40, 256, 64, 33, 5, 2),    # 40 chunks, 19 CTAs
    ("bf16", 97, 256, 128, 3, 5, 2),    # 194 chunks, 203 CTAs
])
def test_blocks_of_many_chunks(dtype, H, P, D, layers, N, n):
    from verify_dspark_markov_step_gb300 import PagedCaches, paged_copy
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}[dtype]
    raw = torch.uint8 if dtype == "e4m3" else torch.int16
    g = torch.Generator("cuda").manual_seed(H + layers)
    caches = [tuple(torch.randint(0, 100, (N, H, P, D), device="cuda", generator=g, dtype=raw) for _ in range(2))
              for _ in range(layers)]
    order = torch.randperm(N, device="cuda", generator=g)
    source, to = order[:n], order[n:2 * n]
    want = [tuple(c.clone() for c in pair) for pair in caches]
    for pair in want:
        for c in pair:
            c[to] = c[source]
    copies = torch.stack([source, to], 1).to(torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged_copy(PagedCaches([tuple(c.view(dt) for c in pair) for pair in caches]), copies,
               torch.tensor([n], dtype=torch.int32, device="cuda"), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for pair, expect in zip(caches, want):
        assert all(torch.equal(a, b) for a, b in zip(pair, expect))
