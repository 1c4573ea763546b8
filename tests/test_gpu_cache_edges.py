"""The cache at the ends of its memory and of its positions.

Tolerances as in test_gpu_decoder.
"""
import random

import pytest
import torch

from tests import test_gpu_decoder as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

DEV, F16, BF16, I32 = "cuda", torch.float16, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("N,G", [(1, 4), (6, 8), (12, 8), (9, 32)])
def test_whole_tiles_up_to_the_last_row(ctx, D, N, G):
    """Tiles that lie wholly in the cache and end with its last row, in a cache that ends its allocation
    but for a guard of NaN; the new nodes' rows likewise."""
    HK, page, n, guard = 2, 64, 512, 256
    g = torch.Generator().manual_seed(D + N)
    size = n // page * page * HK * D
    bufs = [torch.full((size + guard,), float("nan"), dtype=BF16, device=DEV) for _ in range(2)]
    pages = [torch.randn(n // page, page, HK, D, generator=g).to(BF16) for _ in range(2)]
    k, v = (b[:size].view(n // page, page, HK, D).copy_(p.to(DEV)) for b, p in zip(bufs, pages))
    table = torch.randperm(n // page, generator=g).to(I32).view(1, -1)
    q = (2 * torch.randn(1, N, HK * G, D, generator=g)).to(BF16)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(BF16) for _ in range(2))
    sees = base.sees_of(base.trees(random.Random(5), 1, N, 3))
    attn = pi.Attn(ctx, pi.KvCache(ctx, k, v), HK * G, 1, N)
    out = torch.full(q.shape, float("nan"), dtype=BF16, device=DEV)
    pi.tree_attention(ctx, attn, q.to(DEV), kn.to(DEV), vn.to(DEV), base.words_of(sees), table.to(DEV),
                      torch.tensor([n], dtype=I32, device=DEV), out)
    torch.cuda.synchronize()
    base.check_attention(out, q, *pages, kn, vn, sees, table, [n], D ** -0.5)
    assert all(b[size:].isnan().all() for b in bufs)
