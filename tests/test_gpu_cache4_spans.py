"""Attention over the 4-bit cache where a workgroup takes a span of several tiles that ends in one sequence and goes on in
the next, and the forms of 17 to 32 query rows. Tolerances as in the operator's other tests; references in 64 bits on the GPU.
"""
import pytest
import torch

from tests import prompt_ref as ref
from tests.test_gpu_prompts import BF16, DEV, F16, I32, NAN, f, half_step, ints

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


def filled(g, lens, room, HK, D, page, by_head):
    """Random codes and scales of 8 significant bits ([codes, scales] of keys, then of values) and a table; scales beyond a
    sequence's length are NaN."""
    B = len(lens)
    if page == 0:
        page, width, table = room, 1, None
    else:
        width = -(-room // page)
        table = torch.randperm(B * width, generator=g, device=DEV).to(I32).view(B, width)
    slot = torch.arange(width * page, device=DEV)
    out = []
    for _ in range(2):
        c = torch.randint(0, 256, (B * width, page, HK, D // 2), generator=g, device=DEV, dtype=torch.uint8)
        s = (0.2 * torch.randn(B * width, page, HK, D // 32, generator=g, device=DEV)).to(BF16).to(F16)
        for b, n in enumerate(lens):
            pg = torch.full_like(slot, b) if table is None else table[b].long()[slot // page]
            s[pg[n:], slot[n:] % page] = NAN
        out += [t.transpose(1, 2).contiguous().transpose(1, 2) if by_head else t for t in (c, s)]
    return out, table


def held(parts, table, b, n):
    """Keys and values of a sequence's n positions as float64 [n][HK][D]."""
    at, page = torch.arange(n, device=DEV), parts[0].shape[1]
    pg = torch.full_like(at, b) if table is None else table[b].long()[at // page]
    return [ref.values(c[pg, at % page], s[pg, at % page]) for c, s in (parts[:2], parts[2:])]


def words(sees):
    return (sees.to(torch.int64) << torch.arange(sees.shape[2], device=DEV)).sum(2)


def check(out, q, parts, kn, vn, sees, table, lens, scale):
    B, N, H, D = q.shape
    HK = kn.shape[2]
    G, u = H // HK, half_step(q.dtype)
    for b in range(B):
        kc, vc = held(parts, table, b, lens[b])
        k, v = torch.cat([kc, kn[b].double()]), torch.cat([vc, vn[b].double()])
        seen = torch.cat([torch.ones(N, lens[b], dtype=torch.bool, device=DEV), sees[b]], 1).repeat_interleave(G, 0)
        for h in range(HK):
            x = q[b, :, h * G:(h + 1) * G].reshape(N * G, D).double()
            ks, vs = k[:, h].contiguous(), v[:, h].contiguous()
            s = (x @ ks.t().contiguous() * scale).masked_fill(~seen, -torch.inf)
            w = torch.softmax(s, 1).nan_to_num(0)  # a row that sees nothing: zeros
            want, spread = w @ vs, w @ vs.abs()
            score = (x.abs() @ ks.abs().t().contiguous() * scale).masked_fill(~seen, 0).amax(1, keepdim=True)
            bound = (2 * u + 2 * (D + 4) * f * score + 2.0 ** -16) * spread + 1e-30
            err = (out[b, :, h * G:(h + 1) * G].reshape(N * G, D).double() - want).abs()
            assert (err <= bound).all(), f"sequence {b}, kv head {h}: off by {float((err / bound).max()):.2f} of the bound"


def attend(ctx, parts, dtype, q, kn, vn, sees, table, lens, scale, max_batch=None):
    cache = pi.KvCache4(ctx, parts[0], parts[2], parts[1], parts[3], dtype)
    attn = pi.Attn(ctx, cache, q.shape[2], max_batch or q.shape[0], q.shape[1], scale)
    out = torch.full(q.shape, NAN, dtype=dtype, device=DEV)
    pi.tree_attention(ctx, attn, q, kn, vn, words(sees), table, ints(lens), out)
    torch.cuda.synchronize()
    return out


LENS = [1500, 0, 3, 2300, 127, 128, 129, 700, 0, 64, 1025]


# A call has 1 to 3 times 256 / HK workgroups for a head, here 4 to 16, and some 50 tiles of 128 positions, or 100 of 64.
@pytest.mark.parametrize("N,G,HK,D,page,dtype", [
    (1, 4, 64, 128, 16, F16), (1, 8, 64, 128, 64, BF16),  # up to 16 rows: one tile ahead
    (3, 1, 96, 64, 5, BF16),                              # pages that end inside 16 keys
    (2, 2, 64, 96, 16, F16), (5, 3, 64, 32, 7, F16), (1, 1, 64, 64, 0, BF16),
    (1, 2, 64, 256, 16, F16), (4, 4, 64, 160, 6, BF16),   # two tiles ahead
    (10, 2, 64, 64, 16, F16), (32, 1, 64, 96, 16, BF16), (4, 8, 64, 128, 64, F16), (17, 1, 48, 128, 11, BF16),  # 17 to 32 rows
    (9, 2, 64, 32, 0, BF16), (4, 8, 32, 256, 16, BF16), (21, 1, 32, 192, 3, F16),
    (20, 2, 64, 128, 16, F16), (33, 1, 64, 64, 48, BF16), (26, 4, 32, 96, 5, F16),  # four waves
    (64, 4, 32, 128, 16, BF16), (40, 4, 32, 64, 16, F16), (64, 8, 16, 128, 64, F16), (12, 3, 32, 256, 16, F16),
    (64, 5, 16, 224, 7, BF16),                            # eight
])
def test_spans_of_several_tiles_and_sequences(ctx, N, G, HK, D, page, dtype):
    B = len(LENS)
    g = torch.Generator(DEV).manual_seed(51)
    parts, table = filled(g, LENS, max(LENS) + N, HK, D, page, by_head=G % 2 == 0)
    q = torch.randn(B, N, HK * G, D, generator=g, device=DEV).to(dtype)
    kn, vn = (torch.randn(B, N, HK, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    sees = torch.rand(B, N, N, generator=g, device=DEV) < 0.4
    sees[:, 0] = False  # over an empty sequence these rows see nothing
    out = attend(ctx, parts, dtype, q, kn, vn, sees, table, LENS, D ** -0.5)
    check(out, q, parts, kn, vn, sees, table, LENS, D ** -0.5)
    assert (out[1, 0] == 0).all()
    assert torch.equal(out, attend(ctx, parts, dtype, q, kn, vn, sees, table, LENS, D ** -0.5, max_batch=B + 5))
    # infinite values of a node that only some rows of one sequence see stay with them
    vn[4, N - 1, 1, 5], vn[6, N - 1, 0, 7] = float("inf"), NAN
    odd = attend(ctx, parts, dtype, q, kn, vn, sees, table, LENS, D ** -0.5)
    for b, h, c in ((4, 1, 5), (6, 0, 7)):
        see = sees[b, :, N - 1]
        assert not odd[b, see, h * G:(h + 1) * G, c].isfinite().any()
        odd[b, see, h * G:(h + 1) * G, c] = out[b, see, h * G:(h + 1) * G, c]
    assert torch.equal(odd, out)


@pytest.mark.parametrize("N,G,HK,D,page,dtype", [(1, 8, 8, 128, 64, F16), (1, 1, 64, 128, 5, BF16), (26, 2, 4, 64, 16, BF16),
                                                  (5, 4, 2, 256, 16, F16)])
def test_one_long_sequence(ctx, N, G, HK, D, page, dtype):
    """A single sequence, whose spans are of several tiles."""
    n = 30001
    g = torch.Generator(DEV).manual_seed(52)
    parts, table = filled(g, [n], n + N, HK, D, page, by_head=True)
    q = torch.randn(1, N, HK * G, D, generator=g, device=DEV).to(dtype)
    kn, vn = (torch.randn(1, N, HK, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    sees = torch.ones(1, N, N, dtype=torch.bool, device=DEV).tril()
    out = attend(ctx, parts, dtype, q, kn, vn, sees, table, [n], D ** -0.5)
    check(out, q, parts, kn, vn, sees, table, [n], D ** -0.5)
