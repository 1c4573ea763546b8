"""The decoder operators around the sparse FFN against plain 64-bit statements.

Tolerances follow from the roundings: u is half a step of the output's type relative to the
value (torch.finfo(t).eps / 2), f = 2^-24 the same of fp32, whose sums of n terms are off by at
most n f times the sum of the terms' magnitudes.
"""
import random

import pytest
import torch

from tests import decoder_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
f = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


def trees(r, B, N, width):
    """Parents [B][N] (a chain for width 0)."""
    rows = []
    for _ in range(B):
        par, kids = [-1], [0] * N
        for i in range(1, N):
            p = i - 1 if width == 0 else r.choice([j for j in range(max(0, i - 2 * width), i) if kids[j] < width])
            kids[p] += 1
            par.append(p)
        rows.append(par)
    return rows


def sees_of(parents):
    """Truth values [B][N][N]: node i sees itself and what is above it."""
    B, N = len(parents), len(parents[0])
    s = torch.zeros(B, N, N, dtype=torch.bool)
    for b, par in enumerate(parents):
        for i, p in enumerate(par):
            if p >= 0:
                s[b, i] |= s[b, p]
            s[b, i, i] = True
    return s


def words_of(sees):
    B, N, _ = sees.shape
    out = torch.zeros(B, N, dtype=torch.int64)
    for b in range(B):
        for i in range(N):
            w = sum(1 << j for j in range(N) if sees[b, i, j])
            out[b, i] = w - (1 << 64) if w >= 1 << 63 else w
    return out.to(DEV)


def make_cache(ctx, lens, room, HK, D, page, dtype, seed, fill=0.0):
    """A paged cache with shuffled pages; what lies beyond a sequence's length holds ``fill``."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    if page == 0:
        page, width, table = room, 1, None
    else:
        width = -(-room // page)
        table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width)
    k = torch.randn(B * width, page, HK, D, generator=g).to(dtype)
    v = torch.randn(B * width, page, HK, D, generator=g).to(dtype)
    for b in range(B):
        for p in range(lens[b], width * page):
            pg = b if table is None else int(table[b, p // page])
            k[pg, p % page] = fill
            v[pg, p % page] = fill
    return k, v, table


def run_attention(ctx, q, k, v, kn, vn, words, table, lens, scale, out=None, max_batch=None):
    cache = pi.KvCache(ctx, k.to(DEV), v.to(DEV))
    attn = pi.Attn(ctx, cache, q.shape[2], max_batch or q.shape[0], q.shape[1], scale)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV) if out is None else out
    dev = lambda t: t if t.device.type == "cuda" else t.to(DEV)  # noqa: E731
    pi.tree_attention(ctx, attn, dev(q), dev(kn), dev(vn), words, None if table is None else table.to(DEV),
                      torch.tensor(lens, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    return out


def check_attention(out, q, k, v, kn, vn, sees, table, lens, scale):
    want, spread, score = ref.tree_attention(q.cpu(), k, v, kn.cpu(), vn.cpu(), sees, table, lens, scale)
    u, D = half_step(q.dtype), q.shape[3]
    # the weights' rounding and the output's (u each); a score's error enters a weight and the
    # sum; the exponentials and sums of weights in fp32
    rel = 2 * u + 2 * (D + 4) * f * score + 2.0 ** -16
    err = (out.cpu().double() - want).abs()
    bad = err > rel * spread + 1e-30
    assert not bad.any(), f"off by {float((err / (rel * spread + 1e-30)).max()):.2f} of the bound at {bad.nonzero()[0].tolist()}"
    return want


ATTN = [
    # B, N, H, HK, D, lens, page, dtype, tree width
    (1, 1, 4, 4, 64, [1], 16, F16, 0),
    (1, 1, 8, 8, 128, [513], 16, F16, 0),
    (1, 1, 8, 1, 128, [0], 0, BF16, 0),
    (2, 3, 8, 2, 80, [130, 7], 48, F16, 3),
    (3, 5, 6, 2, 40, [65, 0, 200], 64, BF16, 3),
    (1, 26, 16, 4, 64, [300], 48, BF16, 3),
    (2, 8, 16, 2, 128, [257, 1000], 16, F16, 3),
    (1, 64, 8, 2, 128, [129], 64, F16, 0),
    (1, 33, 40, 8, 128, [700], 256, BF16, 3),
    (2, 13, 5, 1, 256, [31, 33], 1, F16, 3),
    (1, 1, 2, 2, 256, [400], 16, BF16, 0),
    (1, 7, 96, 8, 96, [63], 7, F16, 3),
    (1, 40, 16, 2, 256, [95], 16, BF16, 3),
    (5, 2, 4, 2, 8, [9, 1, 0, 100, 64], 5, F16, 0),
    (70, 1, 2, 1, 64, [3 * i for i in range(70)], 16, F16, 0),
]


@pytest.mark.parametrize("B,N,H,HK,D,lens,page,dtype,width", ATTN, ids=lambda v: str(v)[:24])
def test_tree_attention(ctx, B, N, H, HK, D, lens, page, dtype, width):
    g = torch.Generator().manual_seed(7)
    # what a sequence does not hold is NaN: it must not enter the result
    k, v, table = make_cache(ctx, lens, max(lens) + N, HK, D, page, dtype, 3, fill=float("nan"))
    q = (2 * torch.randn(B, N, H, D, generator=g)).to(dtype)
    kn, vn = (torch.randn(B, N, HK, D, generator=g).to(dtype) for _ in range(2))
    sees = sees_of(trees(random.Random(5), B, N, width))
    words = None if width == 0 else words_of(sees)
    out = run_attention(ctx, q, k, v, kn, vn, words, table, lens, D ** -0.5)
    check_attention(out, q, k, v, kn, vn, sees, table, lens, D ** -0.5)


def test_tree_attention_long_split_and_uneven(ctx):
    """Many chunks of unlike sequences, joined; the largest weights far apart."""
    g = torch.Generator().manual_seed(11)
    lens, H, HK, D, N = [5000, 1, 777], 4, 1, 64, 4
    k, v, table = make_cache(ctx, lens, 5000 + N, HK, D, 16, F16, 4)
    q = (6 * torch.randn(3, N, H, D, generator=g)).to(F16)
    kn, vn = (torch.randn(3, N, HK, D, generator=g).to(F16) for _ in range(2))
    sees = sees_of(trees(random.Random(2), 3, N, 3))
    out = run_attention(ctx, q, k, v, kn, vn, words_of(sees), table, lens, D ** -0.5)
    check_attention(out, q, k, v, kn, vn, sees, table, lens, D ** -0.5)


@pytest.mark.parametrize("G,N", [(1, 3), (8, 5), (8, 12), (8, 40)])
@pytest.mark.parametrize("n", [0, 40])
def test_rows_that_see_nothing_and_unseen_values(ctx, G, N, n):
    """A word of 0 over an empty cache gives zeros; nodes that nobody sees may hold NaN and
    infinities; bits past the last node mean nothing."""
    g = torch.Generator().manual_seed(1)
    HK, D = 2, 64
    k, v, table = make_cache(ctx, [n], n + N, HK, D, 16, F16, 9, fill=float("inf"))
    q = torch.randn(1, N, HK * G, D, generator=g).to(F16)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(F16) for _ in range(2))
    kn[0, 1], vn[0, 1] = float("nan"), float("inf")
    sees = torch.zeros(1, N, N, dtype=torch.bool)
    for i in range(2, N):
        sees[0, i, i] = True
        sees[0, i, 0] = True
    words = words_of(sees)
    if N < 64:
        words |= 1 << N
    out = run_attention(ctx, q, k, v, kn, vn, words, table, [n], D ** -0.5)
    kz, vz = kn.clone(), vn.clone()
    kz[0, 1], vz[0, 1] = 0, 0
    check_attention(out, q, k, v, kz, vz, sees, table, [n], D ** -0.5)
    if n == 0:
        assert (out[0, :2] == 0).all()


def test_attention_seen_nan_stays(ctx):
    """A NaN value that a node sees is its output, and only its own."""
    HK, D, N = 1, 64, 3
    q, kn = torch.ones(1, N, HK, D, dtype=F16), torch.ones(1, N, HK, D, dtype=F16)
    vn = torch.ones(1, N, HK, D, dtype=F16)
    vn[0, 1, 0, 5] = float("nan")
    vn[0, 1, 0, 6] = float("inf")
    k, v, table = make_cache(ctx, [4], 16, HK, D, 16, F16, 2)
    sees = torch.eye(N, dtype=torch.bool)[None]
    out = run_attention(ctx, q, k, v, kn, vn, words_of(sees), table, [4], 1.0).cpu()
    assert out[0, 1, 0, 5].isnan() and out[0, 1, 0, 6] == float("inf")
    assert out[0, 0].isfinite().all() and out[0, 2].isfinite().all() and out[0, 1, 0, 7].isfinite()


def test_attention_bad_pages_and_lengths(ctx):
    """Page numbers outside the cache read as zeros, lengths are taken into range; nothing else
    is read (the kernels check both)."""
    g = torch.Generator().manual_seed(3)
    HK, D, N, page = 2, 64, 2, 16
    k, v, _ = make_cache(ctx, [64, 64], 64, HK, D, page, F16, 8)
    table = torch.tensor([[0, -1, 2, 1 << 30], [4, 5, 8, 7]], dtype=torch.int32)
    q = torch.randn(2, N, 4, D, generator=g).to(F16)
    kn, vn = (torch.randn(2, N, HK, D, generator=g).to(F16) for _ in range(2))
    sees = sees_of(trees(random.Random(1), 2, N, 0))
    out = run_attention(ctx, q, k, v, kn, vn, None, table, [1 << 30, -5], D ** -0.5)
    check_attention(out, q, k, v, kn, vn, sees, table, [64, 0], D ** -0.5)


def test_attention_strided_views(ctx):
    """q, k and v as views of one projection, the cache's halves of one allocation, the output
    a slice of something wider."""
    g = torch.Generator().manual_seed(21)
    B, N, H, HK, D, n, page = 2, 6, 8, 2, 64, 50, 16
    qkv = torch.randn(B, N, H + 2 * HK, D, generator=g).to(BF16).to(DEV)
    q, kn, vn = qkv[:, :, :H], qkv[:, :, H:H + HK], qkv[:, :, H + HK:]
    kv = torch.randn(2 * 4, 2, page, HK, D, generator=g).to(BF16).to(DEV)
    table = torch.randperm(8, generator=g).to(torch.int32).view(2, 4)
    wide = torch.zeros(B, N, H, 2 * D, dtype=BF16, device=DEV)
    cache = pi.KvCache(ctx, kv[:, 0], kv[:, 1])
    attn = pi.Attn(ctx, cache, H, B, N)
    big = torch.full((B, 7), -1, dtype=torch.int32, device=DEV)
    big[:, :4] = table.to(DEV)
    lens = torch.tensor([n, 3], dtype=torch.int32, device=DEV)
    sees = sees_of(trees(random.Random(4), B, N, 3))
    pi.tree_attention(ctx, attn, q, kn, vn, words_of(sees), big[:, :4], lens, wide[..., D:])
    torch.cuda.synchronize()
    assert (wide[..., :D] == 0).all()
    check_attention(wide[..., D:], q.contiguous(), kv[:, 0].cpu(), kv[:, 1].cpu(), kn.contiguous(), vn.contiguous(), sees,
                    table, [n, 3], D ** -0.5)


def test_attention_repeats_and_smaller_batches(ctx):
    """The same call gives the same bits, and a handle made for more takes less."""
    g = torch.Generator().manual_seed(5)
    k, v, table = make_cache(ctx, [900], 910, 2, 128, 16, F16, 6)
    q = torch.randn(1, 3, 4, 128, generator=g).to(F16)
    kn, vn = (torch.randn(1, 3, 2, 128, generator=g).to(F16) for _ in range(2))
    a = run_attention(ctx, q, k, v, kn, vn, None, table, [900], 0.1)
    b = run_attention(ctx, q, k, v, kn, vn, None, table, [900], 0.1)
    assert torch.equal(a, b)
    c = run_attention(ctx, q, k, v, kn, vn, None, table, [900], 0.1, max_batch=9)
    check_attention(c, q, k, v, kn, vn, sees_of(trees(random.Random(0), 1, 3, 0)), table, [900], 0.1)


# ------------------------------------------------------------------------------- append

@pytest.mark.parametrize("page,dtype,D", [(0, F16, 64), (1, F16, 8), (16, BF16, 80), (48, F16, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_append(ctx, page, dtype, D, in_place):
    g = torch.Generator().manual_seed(2)
    B, N, HK = 3, 7, 2
    lens, room = [0, 17, 95], 98
    k, v, table = make_cache(ctx, lens, room, HK, D, page, dtype, 1)
    kn, vn = (torch.randn(B, N, HK, D, generator=g).to(dtype) for _ in range(2))
    nodes = torch.tensor([[0, 2, 5, -1, -1, -1, -1], [6, 5, 4, 3, 2, 1, 0], [1, 9, 3, 4, 5, -1, -1]], dtype=torch.int32)
    n = torch.tensor([3, 7, 5], dtype=torch.int32)
    kd, vd = k.to(DEV), v.to(DEV)
    cache = pi.KvCache(ctx, kd, vd)
    ctx_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    len_out = ctx_len if in_place else torch.empty_like(ctx_len)
    pi.kv_append(ctx, cache, kn.to(DEV), vn.to(DEV), None if table is None else table.to(DEV), ctx_len, len_out,
                 nodes.to(DEV), n.to(DEV))
    torch.cuda.synchronize()
    size = k.shape[1]
    cap = size * (1 if table is None else table.shape[1])
    for b in range(B):
        for j in range(int(n[b])):
            p, src = lens[b] + j, int(nodes[b, j])
            if p < cap and 0 <= src < N:
                pg = b if table is None else int(table[b, p // size])
                k[pg, p % size], v[pg, p % size] = kn[b, src], vn[b, src]
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)
    assert len_out.tolist() == [min(l + int(m), cap) for l, m in zip(lens, n)]


def test_append_all_tokens_and_bad_pages(ctx):
    """Without nodes every token goes in; a page number outside the cache loses its tokens and
    nothing else changes."""
    k = torch.zeros(3, 4, 1, 8, dtype=F16, device=DEV)
    v = torch.zeros_like(k)
    cache = pi.KvCache(ctx, k, v)
    table = torch.tensor([[2, 77, 1]], dtype=torch.int32, device=DEV)
    kn = torch.arange(1, 11, device=DEV).view(1, 10, 1, 1).expand(1, 10, 1, 8).to(F16).contiguous()
    n_out = torch.zeros(1, dtype=torch.int32, device=DEV)
    pi.kv_append(ctx, cache, kn, -kn, table, torch.tensor([1], dtype=torch.int32, device=DEV), n_out)
    torch.cuda.synchronize()
    assert k[2, :, 0, 0].tolist() == [0, 1, 2, 3] and k[1, :, 0, 0].tolist() == [8, 9, 10, 0]
    assert (k[0] == 0).all() and torch.equal(v, -k) and n_out.tolist() == [11]


# ------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("T,d", [(1, 8), (3, 512), (2, 520), (5, 4096), (1, 5000), (2, 16384), (1, 32768)])
@pytest.mark.parametrize("xt,rt", [(F32, F16), (F16, F16), (BF16, F32), (F16, BF16), (F32, None)])
def test_add_rmsnorm(ctx, T, d, xt, rt):
    g = torch.Generator().manual_seed(d)
    x = torch.randn(T, d, generator=g).to(xt).to(DEV)
    res = None if rt is None else (3 * torch.randn(T, d, generator=g)).to(rt).to(DEV)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    ro = torch.empty(T, d, dtype=rt or xt, device=DEV)
    q, scale = torch.empty(T, d, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    y = torch.empty(T, d, dtype=F16, device=DEV)
    pi.add_rmsnorm(ctx, x, res, w, 1e-5, ro, q=q, scale=scale, y=y)
    torch.cuda.synchronize()
    total = x.double() + (0 if res is None else res.double())
    u = half_step(ro.dtype)
    assert ((ro.double() - total).abs() <= (u + 2 * f) * total.abs() + torch.finfo(ro.dtype).tiny * u * 2).all()
    h = ro.double()
    want = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    # fp32: the sum of squares (each thread's up to 32, 6 + 4 steps of the tree), half of it in the
    # root; division, root, reciprocal and two products
    rel = (21 + 6) * f
    assert ((y.double() - want).abs() <= (rel + half_step(F16)) * want.abs() + 2.0 ** -25).all()
    top = want.abs().amax(1)
    assert ((scale.double() * 127 - top).abs() <= (rel + 2 * f) * top).all()
    steps = want / scale.double()[:, None]
    assert ((q.double() - steps).abs() <= 0.5 + 127 * (2 * rel + 4 * f)).all()
    assert (q.abs().amax(1) == 127).all()


def test_add_rmsnorm_in_place_views_and_special_rows(ctx):
    """Rows of wider tensors, the residual updated in place; a row of zeros has scale 0 and
    zeros, a row with an infinity or a NaN the scale NaN and zeros."""
    T, d = 4, 64
    g = torch.Generator().manual_seed(0)
    wide = torch.randn(T, 3 * d, generator=g).to(F16).to(DEV)
    x, res = wide[:, :d], wide[:, d:2 * d]
    wide[1, :2 * d] = 0
    wide[2, 5] = float("inf")
    wide[3, d + 7] = float("nan")
    keep = wide.clone()
    w = torch.ones(d, device=DEV)
    qw = torch.full((T, 2 * d), 9, dtype=torch.int8, device=DEV)
    scale = torch.empty(T, device=DEV)
    pi.add_rmsnorm(ctx, x, res, w, 0.0, res, q=qw[:, :d], scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(wide[:2, d:2 * d], (keep[:2, :d].float() + keep[:2, d:2 * d].float()).half())
    assert torch.equal(wide[:, :d].nan_to_num(), keep[:, :d].nan_to_num()) and torch.equal(wide[:, 2 * d:], keep[:, 2 * d:])
    assert (qw[:, d:] == 9).all() and (qw[1:, :d] == 0).all() and scale[1] == 0 and scale[2:].isnan().all()
    assert qw[0, :d].abs().max() == 127


# ------------------------------------------------------------------------------- product

@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 100, 528), (2, 33, 1024), (17, 64, 272), (33, 130, 4096),
                                   (48, 129, 2064), (64, 128, 512), (65, 257, 1040), (129, 96, 256), (257, 131, 144),
                                   (300, 260, 1104), (513, 1000, 528)])
@pytest.mark.parametrize("dtype,bias", [(F16, True), (F32, False), (BF16, True)])
def test_linear_q8(ctx, M, N, K, dtype, bias):
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randint(-128, 128, (M, K), generator=g).to(torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    xs, ws = torch.rand(M, generator=g) / 100, torch.rand(N, generator=g) / 1000
    b = torch.randn(N, generator=g) if bias else None
    lin = pi.Linear(ctx, w.to(DEV), ws.to(DEV), None if b is None else b.to(DEV), max_tokens=M)
    y = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    pi.linear_q8(ctx, lin, x.to(DEV), xs.to(DEV), y)
    torch.cuda.synchronize()
    prod = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    want = prod if b is None else prod + b.double()
    # the sum to fp32, two products, the bias; then the output's type
    tol = 3 * f * prod.abs() + f * want.abs() + half_step(dtype) * want.abs() * (1 + 2.0 ** -8) + torch.finfo(dtype).tiny * 2
    assert ((y.cpu().double() - want).abs() <= tol).all()


def test_linear_q8_largest_sums_and_views(ctx):
    """-128 x -128 over the whole of K stays exact; rows of wider tensors; rows of y that start
    off a vector's boundary."""
    K, M, N = 131056, 2, 3
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    x = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(N, device=DEV)
    lin = pi.Linear(ctx, w, one, max_tokens=M)
    y = torch.empty(M, N, device=DEV)
    pi.linear_q8(ctx, lin, x, one[:M].contiguous(), y)
    assert (y == float(128 * 128 * K)).all()
    g = torch.Generator().manual_seed(1)
    for M in (5, 260):
        big = torch.randint(-9, 9, (M, 192), generator=g).to(torch.int8).to(DEV)
        wb = torch.randint(-9, 9, (37, 128), generator=g).to(torch.int8).to(DEV)
        lin = pi.Linear(ctx, wb[:, 32:96], torch.ones(37, device=DEV), max_tokens=M)
        out = torch.full((M, 41), 7.0, dtype=F16, device=DEV)
        pi.linear_q8(ctx, lin, big[:, 64:128], torch.ones(M, device=DEV), out[:, 1:38])
        torch.cuda.synchronize()
        want = (big[:, 64:128].double() @ wb[:, 32:96].double().t())
        assert (out[:, 1:38].double() == want.half().double()).all() and (out[:, 0] == 7).all() and (out[:, 38:] == 7).all()


# ------------------------------------------------------------------------------- verification

def verify_case(B, N, V, dtype, width, with_q, temp, seed):
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    par = trees(r, B, N, width)
    base = 2 * torch.randn(B, N, V, generator=g) + 7.0 * (torch.rand(B, N, V, generator=g) < 8.0 / V)
    logits = base.to(dtype)
    near = torch.softmax((base + 0.7 * torch.randn(B, N, V, generator=g)) / (temp or 1.0), 2)
    tok = torch.zeros(B, N, dtype=torch.int32)
    for b in range(B):
        for i in range(1, N):
            p = near[b, par[b][i]]
            tok[b, i] = int(torch.multinomial(p, 1, generator=g)) if with_q or r.random() < 0.5 else int(p.argmax())
    return dict(logits=logits, tokens=tok, parents=torch.tensor(par, dtype=torch.int32),
                u=torch.rand(B, N, generator=g), u_next=torch.rand(B, generator=g), q=near if with_q else None,
                temp=torch.full((B,), temp))


def run_verify(ctx, c, max_batch=None):
    B, N, V = c["logits"].shape
    ver = pi.Verifier(ctx, V, max_batch or B, N)
    nodes, out = (torch.full((B, N), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    n = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    d = {k: None if t is None else t.to(DEV) for k, t in c.items()}
    for _ in range(2):  # twice: the scratch is ready for the next call
        pi.verify(ctx, ver, d["logits"], d["tokens"], d["parents"], d["u"], d["u_next"], nodes, out, n, q=d["q"],
                  temperature=d["temp"])
    torch.cuda.synchronize()
    return nodes.cpu(), out.cpu(), n.cpu()


def check_verify(got, c):
    nodes, out, n = got
    for b in range(nodes.shape[0]):
        path, toks = ref.verify(c["logits"][b], c["tokens"][b], c["parents"][b], c["u"][b], c["u_next"][b],
                                None if c["q"] is None else c["q"][b], 1.0 if c["temp"] is None else float(c["temp"][b]))
        pad = [-1] * (nodes.shape[1] - len(path))
        assert nodes[b].tolist() == path + pad, (b, nodes[b].tolist(), path)
        assert out[b].tolist() == toks + pad, (b, out[b].tolist(), toks)
        assert int(n[b]) == len(path)


@pytest.mark.parametrize("B,N,V,dtype,width", [(1, 1, 1, F32, 0), (1, 5, 3, F16, 0), (2, 6, 500, F16, 3),
                                                (3, 64, 4097, BF16, 4), (1, 70, 33, F32, 2), (2, 16, 12289, F16, 8),
                                                (1, 12, 9001, F32, 0)])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("temp", [0.0, 0.6, 1.3])
def test_verify(ctx, B, N, V, dtype, width, with_q, temp):
    for seed in range(3):
        c = verify_case(B, N, V, dtype, width, with_q, temp, seed)
        check_verify(run_verify(ctx, c), c)


def test_verify_many_rejections(ctx):
    """A family of 40 that the target hardly likes: every residual in turn, past the launches
    that share one."""
    N, V = 41, 6000
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(1, N, V, generator=g)
    q = torch.softmax(torch.randn(1, N, V, generator=g), 2)
    tok = torch.randint(0, V, (1, N), generator=g, dtype=torch.int32)
    par = torch.zeros(1, N, dtype=torch.int32)
    par[0, 0] = -1
    for u in (0.999, 0.2):
        c = dict(logits=logits, tokens=tok, parents=par, u=torch.full((1, N), u), u_next=torch.tensor([0.37]), q=q, temp=None)
        check_verify(run_verify(ctx, c, max_batch=3), c)


def test_verify_special_rows_and_trees(ctx):
    """NaN, infinities and rows of nothing; tokens and parents out of range; repeated tokens; a
    draft equal to the target; draws at the ends."""
    V, N, B = 40, 4, 7
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(B, N, V, generator=g)
    q = torch.softmax(torch.randn(B, N, V, generator=g), 2)
    tok = torch.tensor([[0, 3, 3, 4]] * B, dtype=torch.int32)
    par = torch.tensor([[-1, 0, 0, 1]] * B, dtype=torch.int32)
    logits[0, 0, 5], logits[0, 0, 3] = float("nan"), float("-inf")
    logits[1, 0] = float("-inf")
    logits[2, 0, 7] = float("inf")
    logits[2, 0, 9] = float("inf")
    tok[3] = torch.tensor([0, -1, V, 2])
    par[4] = torch.tensor([-1, 0, 2, 7])
    q[5] = torch.softmax(logits[5].double(), 1).float()
    u = torch.tensor([[0.9, 0.9, 0.9, 0.9]] * B)
    u_next = torch.tensor([0.5, 0.5, 0.99, 0.0, 1.0, 0.3, 0.9999999])
    for quse in (q, None):
        for temp in (None, torch.zeros(B)):
            c = dict(logits=logits, tokens=tok, parents=par, u=u, u_next=u_next, q=quse, temp=temp)
            check_verify(run_verify(ctx, c), c)


def test_verify_strided_rows(ctx):
    """Rows of wider tensors: logits of a padded vocabulary, one model's of two."""
    c = verify_case(2, 6, 501, F16, 3, True, 1.0, 4)
    wide = torch.zeros(2, 6, 513, dtype=F16, device=DEV)
    wide[..., 5:506] = c["logits"].to(DEV)
    qq = torch.zeros(2, 2, 6, 501, device=DEV)
    qq[:, 1] = c["q"].to(DEV)
    d = dict(c, logits=wide[..., 5:506], q=qq[:, 1])
    check_verify(run_verify(ctx, d), c)


# ------------------------------------------------------------------------------- refusals

def test_refusals_name_the_reason(ctx):
    k = torch.zeros(4, 16, 2, 64, dtype=F16, device=DEV)
    cache = pi.KvCache(ctx, k, k.clone())
    for bad in (lambda: pi.KvCache(ctx, k.float(), k.float()), lambda: pi.KvCache(ctx, k, k[:, :8]),
                lambda: pi.KvCache(ctx, k[..., 4:12], k[..., 4:12]), lambda: pi.KvCache(ctx, k[..., :60], k[..., :60]),
                lambda: pi.Attn(ctx, cache, 3, 1, 1), lambda: pi.Attn(ctx, cache, 4, 0, 1),
                lambda: pi.Attn(ctx, cache, 4, 1, 65), lambda: pi.Attn(ctx, cache, 4, 1, 1, scale=0.0),
                lambda: pi.Attn(ctx, cache, 4, 1, 1, scale=float("nan")), lambda: pi.Verifier(ctx, 0, 1, 1),
                lambda: pi.Verifier(ctx, 10, 1, 257),
                lambda: pi.Linear(ctx, torch.zeros(4, 24, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV)),
                lambda: pi.Linear(ctx, torch.zeros(4, 131072, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV))):
        with pytest.raises(pi.PiError):
            bad()
    attn = pi.Attn(ctx, cache, 4, 2, 8)
    q, kn = torch.zeros(2, 8, 4, 64, dtype=F16, device=DEV), torch.zeros(2, 8, 2, 64, dtype=F16, device=DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    table = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    run = lambda **o: pi.tree_attention(ctx, attn, *[dict(q=q, k=kn, v=kn, w=None, t=table, l=lens, o=out, **{})[n] if n not in o  # noqa: E731
                                                    else o[n] for n in "qkvwtlo"])
    run()
    three = lambda t: torch.cat([t, t[:1]])  # noqa: E731
    for o in (dict(q=q.float()), dict(q=q[:, :, :2]), dict(k=kn[:1]), dict(l=lens.long()), dict(t=table.long()),
              dict(t=table[:1]), dict(w=torch.zeros(2, 7, dtype=torch.int64, device=DEV)), dict(q=q.cpu()),
              dict(q=three(q), k=three(kn), v=three(kn), t=three(table), l=three(lens), o=three(out))):
        with pytest.raises(pi.PiError):
            run(**o)
    x = torch.zeros(2, 64, dtype=F16, device=DEV)
    w = torch.ones(64, device=DEV)
    with pytest.raises(pi.PiError, match="together"):
        pi.add_rmsnorm(ctx, x, None, w, 1e-5, x.clone(), scale=torch.empty(2, device=DEV))
    with pytest.raises(pi.PiError):
        pi.add_rmsnorm(ctx, x, None, w, -1.0, x.clone())
    with pytest.raises(pi.PiError):
        pi.add_rmsnorm(ctx, x[:, :60], None, w[:60].contiguous(), 1e-5, x[:, :60].clone())
    lin = pi.Linear(ctx, torch.zeros(4, 64, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV), max_tokens=1)
    with pytest.raises(pi.PiError, match="out of range"):
        pi.linear_q8(ctx, lin, torch.zeros(2, 64, dtype=torch.int8, device=DEV), torch.ones(2, device=DEV),
                     torch.empty(2, 4, device=DEV))
    other = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)
    with pytest.raises(pi.PiError, match="another context"):
        pi.linear_q8(other, lin, torch.zeros(1, 64, dtype=torch.int8, device=DEV), torch.ones(1, device=DEV),
                     torch.empty(1, 4, device=DEV))
    torch.cuda.synchronize()
