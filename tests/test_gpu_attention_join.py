"""The join of a long sequence's chunks: every count of chunks, and infinities that nodes see.

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


# On 256 CUs one sequence of these sizes has `chunks` chunks of one tile: 128 positions up to 32 rows
# (nodes x query heads of a key head), 64 above.
MANY = ([(1, 64, 8, 128, c, F16) for c in (33, 35, 63, 64)] +
        [(1, 64, 8, 64, 33, BF16), (4, 64, 8, 128, 63, BF16)] +                     # 8 and 32 rows
        [(6, 64, 8, 64, c, F16) for c in (33, 63)] +                                # 48 rows
        [(16, 64, 8, 128, 35, BF16), (16, 64, 8, 64, 64, F16)] +                    # 128 rows
        [(1, 16, 4, 80, c, F16) for c in (33, 64, 65, 97)] + [(8, 64, 4, 64, 65, BF16), (10, 64, 4, 128, 33, F16)] +
        [(1, 1, 1, 128, c, F16) for c in (33, 65, 97)] + [(2, 64, 1, 64, 97, BF16), (1, 40, 1, 128, 127, F16)])


@pytest.mark.parametrize("N,H,HK,D,chunks,dtype", MANY, ids=lambda v: str(v))
def test_every_chunk_counts(ctx, N, H, HK, D, chunks, dtype):
    """Half the weight or more lies on the last chunk: a few cached positions and the tree."""
    g = torch.Generator().manual_seed(chunks)
    tile = 128 if N * H // HK <= 32 else 64
    n = (chunks - 1) * tile + 5
    k, v, table = base.make_cache(ctx, [n], n + N, HK, D, 16, dtype, chunks)
    q = torch.randn(1, N, H, D, generator=g).abs().to(dtype)
    kn, vn = (torch.randn(1, N, HK, D, generator=g) for _ in range(2))
    lift = 9 / (0.8 * D ** 0.5)  # keys along the queries' mean: scores of about 9
    kn = (0.1 * kn + lift).to(dtype)
    vn = (vn + 1).to(dtype)
    for p in range(n - 5, n):
        at = int(table[0, p // 16]), p % 16
        k[at] = (0.1 * torch.randn(HK, D, generator=g) + lift).to(dtype)
        v[at] = (v[at].float() + 1).to(dtype)
    sees = base.sees_of(base.trees(random.Random(3), 1, N, 3))
    out = base.run_attention(ctx, q, k, v, kn, vn, base.words_of(sees), table, [n], D ** -0.5)
    base.check_attention(out, q, k, v, kn, vn, sees, table, [n], D ** -0.5)


def test_long_decode_of_a_grouped_head_model(ctx):
    """One token, 64 heads of 8, 4400 positions: 35 chunks."""
    g = torch.Generator().manual_seed(1)
    n, H, HK, D = 4400, 64, 8, 128
    k, v, table = base.make_cache(ctx, [n], n + 1, HK, D, 16, BF16, 2)
    q = (2 * torch.randn(1, 1, H, D, generator=g)).to(BF16)
    kn, vn = (torch.randn(1, 1, HK, D, generator=g).to(BF16) for _ in range(2))
    kn = (q.view(1, 1, HK, H // HK, D).float().mean(3)).to(BF16)  # the newest token answers its queries
    out = base.run_attention(ctx, q, k, v, kn, vn, None, table, [n], D ** -0.5)
    base.check_attention(out, q, k, v, kn, vn, base.sees_of([[-1]]), table, [n], D ** -0.5)


@pytest.mark.parametrize("score", [0.0, -200.0])
@pytest.mark.parametrize("n", [20, 700, 768, 4400])
@pytest.mark.parametrize("HK,D,dtype", [(1, 64, F16), (8, 128, BF16), (2, 256, F16)])
def test_infinities_that_a_node_sees(ctx, HK, D, dtype, n, score):
    """One chunk or many, a number of them that is no multiple of 8, and a last one that weighs nothing
    beside the others: an infinite value is the output of the node that sees it, and of no other."""
    N = 3
    g = torch.Generator().manual_seed(n)
    k, v, table = base.make_cache(ctx, [n], n + N, HK, D, 16, dtype, 4)
    k.zero_()
    q = torch.ones(1, N, HK, D, dtype=dtype)
    kn = torch.full((1, N, HK, D), score / D, dtype=dtype)
    vn = torch.randn(1, N, HK, D, generator=g).to(dtype)
    clean = vn.clone()
    vn[0, 1, :, 5], vn[0, 1, :, 6], vn[0, 1, :, 7] = float("inf"), float("-inf"), float("nan")
    clean[0, 1, :, 5:8] = 0
    sees = torch.eye(N, dtype=torch.bool)[None]
    out = base.run_attention(ctx, q, k, v, kn, vn, base.words_of(sees), table, [n], 1.0).cpu()
    assert (out[0, 1, :, 5] == float("inf")).all() and (out[0, 1, :, 6] == float("-inf")).all()
    assert out[0, 1, :, 7].isnan().all()
    want = base.ref.tree_attention(q, k, v, kn, clean, sees, table, [n], 1.0)[0]
    out[0, 1, :, 5:8] = want[0, 1, :, 5:8].to(dtype)
    base.check_attention(out, q, k, v, kn, clean, sees, table, [n], 1.0)
