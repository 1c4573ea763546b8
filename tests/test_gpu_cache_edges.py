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


# ---------------------------------------------------------------- the last positions

PAGE, WIDTH = 243, 8837381
CAP = PAGE * WIDTH  # 2^31 - 65, the most positions that a table may have


def last_positions_case(H, HK, D, N, seed):
    """A table of one page again and again, with small keys, and another one last, with keys that weigh
    as much as the new nodes'."""
    g = torch.Generator().manual_seed(seed)
    k = 0.02 * torch.randn(2, PAGE, HK, D, generator=g)
    v = torch.randn(2, PAGE, HK, D, generator=g)
    k[1] += 26 / D
    kn = 0.02 * torch.randn(1, N, HK, D, generator=g) + 31 / D
    vn = torch.randn(1, N, HK, D, generator=g)
    q = 1 + 0.1 * torch.randn(1, N, H, D, generator=g)
    table = torch.zeros(1, WIDTH, dtype=I32)
    table[0, -1] = 1
    return [t.to(F16) for t in (q, k, v, kn, vn)], table


@pytest.mark.parametrize("n", [CAP, CAP - 1, CAP - 86, CAP - 130])
@pytest.mark.parametrize("H,N,D", [(1, 3, 64), (8, 8, 64), (8, 16, 128), (32, 9, 64)])
def test_attention_at_the_last_positions(ctx, H, N, D, n):
    """Tiles that end beyond 2^31 keep the last cached positions and the nodes. The same page's rows
    repeat, so the sum over them is their weights' times how often they come."""
    (q, k, v, kn, vn), table = last_positions_case(H, 1, D, N, n % 97)
    sees = base.sees_of(base.trees(random.Random(2), 1, N, 3))
    out = base.run_attention(ctx, q, k, v, kn, vn, base.words_of(sees), table, [n], 1.0).cpu().double()
    times = torch.zeros(2, PAGE, dtype=torch.float64)
    times[0] = WIDTH - 1
    times[1, :n - PAGE * (WIDTH - 1)] = 1
    rows, val = k.double().flatten(0, 1)[:, 0], v.double().flatten(0, 1)[:, 0]
    f, u = 2.0 ** -24, torch.finfo(F16).eps / 2
    for h in range(H):
        x = q[0, :, h].double()
        s = torch.cat([x @ rows.t(), torch.where(sees[0], x @ kn[0, :, 0].double().t(), -torch.inf)], 1)
        w = torch.exp(s - s.amax(1, keepdim=True)) * torch.cat([times.flatten(), torch.ones(N, dtype=torch.float64)])
        far = w[:, :PAGE].sum(1, keepdim=True) / w.sum(1, keepdim=True)  # the repeated page's share, some 1e-4
        assert float(far.max()) < 1e-3
        w = w / w.sum(1, keepdim=True)
        vals = torch.cat([val, vn[0, :, 0].double()])
        score = x.abs() @ torch.cat([rows, kn[0, :, 0].double()]).abs().t()
        # as elsewhere, and of the share that is summed in 2^20 steps at most: any of it
        rel = 2 * u + 2 * (D + 4) * f * score.amax(1, keepdim=True) + 2.0 ** -16
        tol = rel * (w @ vals.abs()) + 2 * far * vals.abs().max()
        assert ((out[0, :, h] - w @ vals).abs() <= tol).all(), h


@pytest.mark.parametrize("listed", [False, True])
def test_append_at_the_last_positions(ctx, listed):
    """Tokens beyond the table are dropped, also those whose position would pass 2^31."""
    N, left = 200, 100
    table = torch.zeros(2, WIDTH, dtype=I32, device=DEV)
    table[0, -1] = table[1, 0] = 1
    k = torch.zeros(2, PAGE, 1, 8, dtype=F16, device=DEV)
    v = torch.zeros_like(k)
    kn = torch.arange(1, 2 * N + 1, device=DEV).view(2, N, 1, 1).expand(2, N, 1, 8).to(F16).contiguous()
    lens = torch.tensor([CAP - left, 7], dtype=I32, device=DEV)
    grown = torch.zeros_like(lens)
    nodes = torch.arange(N, dtype=I32, device=DEV).flip(0).expand(2, N).contiguous() if listed else None
    n = torch.tensor([N, 3], dtype=I32, device=DEV)
    pi.kv_append(ctx, pi.KvCache(ctx, k, v), kn, -kn, table, lens, grown, nodes, n)
    torch.cuda.synchronize()
    rows = torch.arange(N, 0, -1) if listed else torch.arange(1, N + 1)
    want = torch.zeros(PAGE, dtype=torch.int64)
    want[PAGE - left:] = rows[:left]
    want[7:10] = N + rows[:3]
    assert k[1, :, 0, 0].tolist() == want.tolist() and (k[0] == 0).all() and torch.equal(v, -k)
    assert grown.tolist() == [CAP, 10]
