"""Norm and rotary positions of heads, attention of packed prompts, and the 4-bit cache, against plain 64-bit
statements.

Tolerances follow from the roundings: u is half a step of the output's type relative to the value
(torch.finfo(t).eps / 2), f = 2^-24 the same of fp32, whose sums of n terms are off by at most n f times the sum of
the terms' magnitudes.
"""
import random

import pytest
import torch

from tests import decoder_ref, prompt_ref as ref
from tests.test_gpu_decoder import sees_of, trees, words_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

DEV = "cuda"
F16, BF16, F32, I32 = torch.float16, torch.bfloat16, torch.float32, torch.int32
f = 2.0 ** -24
NAN = float("nan")


def half_step(t):
    return torch.finfo(t).eps / 2


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


# ---------------------------------------------------------------- norm and rotary positions

def check_rope(out, x, w, pos, freq, eps, pairs):
    want, size = ref.rope(x, w, pos, freq, eps, pairs)
    D, yt = x.shape[-1], out.dtype
    angle = 0 if freq is None else (pos.double().abs()[:, None, None] * freq.double().max())
    # The turn is rounded to fp32 at half a turn (2^-25 of a turn: 3.2 f), its sine and cosine are off by 2 f each,
    # products and their sum by f each; angles in 64 bits by 4 steps of theirs; the norm by its sum over D.
    rel = (12 + (D + 8 if w is not None else 0)) * f + 4 * 2.0 ** -53 * angle
    tiny = torch.finfo(yt).tiny * torch.finfo(yt).eps / 2  # half the smallest step
    err = (out.cpu().double() - want).abs()
    bound = half_step(yt) * want.abs() + rel * size * (1 + half_step(yt)) + tiny
    assert (err <= bound).all(), f"off by {float((err / bound).max()):.2f} of the bound"


ROPE = [
    # T, H, HK, D, rot, x, y, norm, pairs
    (1, 1, 1, 8, 8, F16, F16, False, False),
    (3, 4, 2, 128, 128, BF16, BF16, True, False),
    (5, 5, 1, 80, 40, F16, F16, True, False),
    (2, 3, 3, 64, 20, F32, F16, True, True),
    (7, 32, 8, 128, 64, F16, F32, True, True),
    (4, 2, 1, 256, 252, BF16, F32, False, False),
    (4, 2, 1, 256, 256, BF16, BF16, False, True),
    (3, 9, 0, 96, 96, F32, BF16, True, False),
    (3, 0, 7, 512, 512, F16, F16, True, False),
    (3, 2, 2, 504, 8, F16, F16, True, True),
    (2, 3, 1, 40, 0, BF16, F16, True, False),
    (300, 8, 2, 64, 64, F16, BF16, False, True),
]


@pytest.mark.parametrize("T,H,HK,D,rot,xt,yt,norm,pairs", ROPE, ids=lambda v: str(v)[-8:])
def test_qk_norm_rope(ctx, T, H, HK, D, rot, xt, yt, norm, pairs):
    g = torch.Generator().manual_seed(1)
    qkv = (3 * torch.randn(T, H + 2 * HK, D, generator=g)).to(xt)
    pos = torch.randint(0, 200000, (T,), generator=g).to(I32)
    pos[0] = 0
    freq = (10000.0 ** (-torch.arange(rot // 2).double() / max(1, rot // 2))).float() if rot else None
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)) if norm else None for _ in range(2))
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    x = qkv.to(DEV)
    q, k = (x[:, :H] if H else None), (x[:, H:H + HK] if HK else None)
    qo, ko = (torch.full((T, n, D), NAN, dtype=yt, device=DEV) if n else None for n in (H, HK))
    pi.qk_norm_rope(ctx, q, k, dev(pos), dev(freq), qo, ko, q_norm=dev(wq), k_norm=dev(wk), interleaved=pairs)
    torch.cuda.synchronize()
    assert torch.equal(x.cpu(), qkv)
    if H:
        check_rope(qo, qkv[:, :H], wq, pos, freq, 1e-6, pairs)
    if HK:
        check_rope(ko, qkv[:, H:H + HK], wk, pos, freq, 1e-6, pairs)


def test_rope_in_place_one_side_normalised_far_positions(ctx):
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(6, 12, 128, generator=g).to(BF16)
    pos = torch.tensor([0, 1, 1 << 20, -5, (1 << 31) - 1, 12345678], dtype=I32)
    freq = (1000000.0 ** (-torch.arange(64).double() / 64)).float()
    w = 1 + 0.3 * torch.randn(128, generator=g)
    x = qkv.to(DEV)
    q, k = x[:, :8], x[:, 8:10]
    pi.qk_norm_rope(ctx, q, k, pos.to(DEV), freq.to(DEV), q, k, k_norm=w.to(DEV), eps=1e-5)
    torch.cuda.synchronize()
    check_rope(q, qkv[:, :8], None, pos, freq, 1e-5, False)
    check_rope(k, qkv[:, 8:10], w, pos, freq, 1e-5, False)
    assert torch.equal(x[:, 10:].cpu(), qkv[:, 10:])


def test_rope_of_extreme_heads(ctx):
    """Squares beyond fp32's range or lost below it, zeros, and heads with an infinity or a NaN beside others."""
    D = 64
    x = torch.randn(1, 7, D, generator=torch.Generator().manual_seed(3))
    x[0, 1] *= 1e30
    x[0, 2] *= 1e-30
    x[0, 3] = 0
    x[0, 4, 5] = float("inf")
    x[0, 5, 6] = NAN
    x[0, 6] = 3e38
    w, pos, freq = torch.ones(D), torch.zeros(1, dtype=I32), torch.ones(D // 2)
    out = torch.empty(1, 7, D, device=DEV)
    pi.qk_norm_rope(ctx, x.to(DEV), None, pos.to(DEV), freq.to(DEV), out, None, q_norm=w.to(DEV), eps=0.0)
    torch.cuda.synchronize()
    o = out.cpu()
    for h in (0, 1, 2, 3, 6):
        check_rope(out[:, h:h + 1], x[:, h:h + 1], w, pos, freq, 0.0, False)
    assert o[0, 4].isnan().sum() >= 1 and o[0, 5].isnan().all()


# ---------------------------------------------------------------- the 4-bit cache

def make_cache4(lens, room, HK, D, page, seed, by_head=False, dtype=F16, junk=True):
    """Codes, scales, table and values [pages][page][HK][D] of a filled cache. What lies beyond a sequence's length
    has NaN scales."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    if page == 0:
        page, width, table = room, 1, None
    else:
        width = -(-room // page)
        table = torch.randperm(B * width, generator=g).to(I32).view(B, width)
    out = []
    for _ in range(2):
        c, s = ref.quantize(torch.randn(B * width, page, HK, D, generator=g).to(dtype))
        if junk:
            for b in range(B):
                for p in range(lens[b], width * page):
                    s[b if table is None else int(table[b, p // page]), p % page] = NAN
        out += [c, s]
    if by_head:  # a head's tokens next to each other
        out = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in out]
    return out, table


def cache_on_gpu(ctx, parts, dtype):
    k, ks, v, vs = (t.to(DEV) for t in parts)
    return pi.KvCache4(ctx, k, v, ks, vs, dtype)


def special_blocks(dtype, D):
    """Rows with ties, zeros, tiny and huge values, infinities and NaN: [n][D]."""
    x = torch.zeros(9, 32)
    x[0] = torch.arange(32) / 4 - 4                     # ties at a scale of 0.5 (and 0.484375: -m/8 rounded)
    x[1] = 0
    x[2, 3], x[2, 4] = 5, -5                            # two alike: the positive one
    x[3, 7], x[3, 8] = -5, 4.9
    x[4] = torch.finfo(dtype).tiny * torch.arange(32)
    x[5] = torch.finfo(dtype).max * torch.linspace(-1, 1, 32)
    x[6] = 1
    x[6, 31] = float("inf")
    x[7, 0] = NAN
    x[8] = torch.arange(32) - 15.5
    return x.repeat(1, D // 32).to(dtype)


@pytest.mark.parametrize("page,dtype,D,by_head,in_place", [(16, F16, 128, True, False), (5, BF16, 96, False, True),
                                                          (0, F16, 32, True, True), (64, BF16, 256, True, False),
                                                          (7, F16, 64, False, False)])
def test_append_and_read_4_bits(ctx, page, dtype, D, by_head, in_place):
    B, N, HK, lens = 4, 12, 3, [0, 9, 30, 17]
    g = torch.Generator().manual_seed(4)
    parts, table = make_cache4(lens, 50, HK, D, page, 5, by_head, dtype)
    want = [t.clone() for t in parts]
    kn, vn = (torch.randn(B, N, HK, D, generator=g).to(dtype) for _ in range(2))
    kn[1, :9, 1] = special_blocks(dtype, D)
    nodes = torch.tensor([[3, 1, 11, 0] + [-1] * 8, list(range(12)), [5] + [-1] * 11, [2, 40, 7] + [-1] * 9], dtype=I32)
    n = torch.tensor([4, 12, 1, 3], dtype=I32)
    cache = cache_on_gpu(ctx, parts, dtype)
    ln = ints(lens)
    out_len = ln if in_place else torch.empty_like(ln)
    tab = None if table is None else table.to(DEV)
    pi.kv_append(ctx, cache, kn.to(DEV), vn.to(DEV), tab, ln, out_len, nodes.to(DEV), n.to(DEV))
    torch.cuda.synchronize()
    size = parts[0].shape[1]
    for b in range(B):
        for j in range(int(n[b])):
            src, p = int(nodes[b, j]), lens[b] + j
            if not 0 <= src < N:
                continue
            pg = b if table is None else int(table[b, p // size])
            want[0][pg, p % size], want[1][pg, p % size] = ref.quantize(kn[b, src])
            want[2][pg, p % size], want[3][pg, p % size] = ref.quantize(vn[b, src])
    got = [cache.k, cache.k_scale, cache.v, cache.v_scale]
    for w, o in zip(want, got):
        assert torch.equal(w.view(torch.int16) if w.dtype is F16 else w, o.cpu().view(torch.int16) if w.dtype is F16 else o.cpu()) \
            or torch.equal(w.nan_to_num(nan=1e9), o.cpu().nan_to_num(nan=1e9))
    total = [a + int(m) for a, m in zip(lens, n)]
    assert out_len.tolist() == total

    # read it back: from the start, from somewhere, beyond the length, and nothing
    start, ask = [0, 4, 31, 3], [4, 19, 5, 0]
    cu = [2]  # two rows of no sequence in front
    for m in ask:
        cu.append(cu[-1] + m)
    ko, vo = (torch.full((cu[-1] + 3, HK, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    pi.kv_read(ctx, cache, tab, out_len, ints(cu), ko, vo, start=ints(start))
    torch.cuda.synchronize()
    for o, (c, s) in ((ko, want[:2]), (vo, want[2:])):
        exp = torch.full(o.shape, 7.0, dtype=dtype)
        val = ref.values(c, s)
        for b in range(B):
            for i in range(ask[b]):
                p = start[b] + i
                if p < total[b]:
                    exp[cu[b] + i] = val[b if table is None else int(table[b, p // size]), p % size].to(dtype)
        assert torch.equal(exp.nan_to_num(nan=1e4), o.cpu().nan_to_num(nan=1e4))
    if dtype is F16:  # every value is an fp16 number
        v64 = ref.values(*[t.cpu() for t in (cache.k, cache.k_scale)])
        fin = v64.isfinite()
        assert torch.equal(v64[fin].half().double(), v64[fin])


@pytest.mark.parametrize("kind", ["plain", "4 bits"])
def test_read_bad_pages_many_sequences_and_odd_offsets(ctx, kind):
    B, HK, D, page = 70, 2, 64, 8
    lens = [(5 * b) % 23 for b in range(B)]
    g = torch.Generator().manual_seed(6)
    table = torch.randperm(B * 3, generator=g).to(I32).view(B, 3)
    if kind == "plain":
        k, v = (torch.randn(B * 3, page, HK, D, generator=g).to(BF16) for _ in range(2))
        cache, vals = pi.KvCache(ctx, k.to(DEV), v.to(DEV)), (k, v)
    else:
        c = [ref.quantize(torch.randn(B * 3, page, HK, D, generator=g)) for _ in range(2)]
        cache = pi.KvCache4(ctx, c[0][0].to(DEV), c[1][0].to(DEV), c[0][1].to(DEV), c[1][1].to(DEV), BF16)
        vals = [ref.values(*x).to(BF16) for x in c]
    table[3, 1], table[10, 0] = -1, B * 3  # outside the cache: zeros
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    wide = [torch.full((cu[-1] + 40, HK, 2 * D), 3.0, dtype=BF16, device=DEV) for _ in range(2)]
    ko, vo = (w[..., :D] for w in wide)
    pi.kv_read(ctx, cache, table.to(DEV), ints(lens), ints(cu), ko, vo)
    torch.cuda.synchronize()
    for o, x in ((ko, vals[0]), (vo, vals[1])):
        exp = torch.full(o.shape, 3.0, dtype=BF16)
        for b in range(B):
            for p in range(lens[b]):
                pg = int(table[b, p // page])
                exp[cu[b] + p] = x[pg, p % page] if 0 <= pg < B * 3 else 0
        assert torch.equal(exp, o.cpu())
    assert all((w[..., D:] == 3).all() for w in wide)
    # offsets that descend or lie outside the rows write inside the outputs or nothing
    for bad in ([5, 2, 900000, -7] + [0] * (B - 3), [1 << 30] * (B + 1), [-(1 << 31)] + [(1 << 31) - 1] * B):
        pi.kv_read(ctx, cache, table.to(DEV), ints(lens), ints(bad), ko, vo)
    torch.cuda.synchronize()
    assert all((w[..., D:] == 3).all() for w in wide)


ATTN4 = [
    # B, N, H, HK, D, lens, page, dtype, tree width
    (1, 1, 4, 4, 64, [1], 16, F16, 0),
    (1, 1, 8, 8, 128, [513], 16, F16, 0),
    (1, 1, 8, 1, 128, [0], 0, BF16, 0),
    (2, 3, 8, 2, 32, [130, 7], 48, F16, 3),
    (3, 5, 6, 2, 96, [65, 0, 200], 64, BF16, 3),
    (1, 26, 16, 4, 64, [300], 48, BF16, 3),
    (2, 8, 16, 2, 128, [257, 1000], 16, F16, 3),
    (1, 64, 8, 2, 128, [128], 64, F16, 0),
    (1, 33, 40, 8, 128, [700], 256, BF16, 3),
    (2, 13, 5, 1, 256, [31, 33], 1, F16, 3),
    (1, 1, 2, 2, 256, [400], 16, BF16, 0),
    (1, 7, 96, 8, 96, [63], 7, F16, 3),
    (1, 40, 16, 2, 256, [95], 16, BF16, 3),
    (1, 6, 16, 2, 160, [64], 16, F16, 3),
    (5, 2, 4, 2, 32, [9, 1, 0, 100, 64], 5, F16, 0),
    (70, 1, 2, 1, 64, [3 * i for i in range(70)], 16, F16, 0),
    (1, 64, 16, 2, 128, [5000], 16, BF16, 3),
    (3, 1, 32, 4, 128, [3000, 1, 777], 16, BF16, 0),
]


def run_attention4(ctx, q, parts, kn, vn, words, table, lens, scale, max_batch=None):
    cache = cache_on_gpu(ctx, parts, q.dtype)
    attn = pi.Attn(ctx, cache, q.shape[2], max_batch or q.shape[0], q.shape[1], scale)
    out = torch.full(q.shape, NAN, dtype=q.dtype, device=DEV)
    pi.tree_attention(ctx, attn, q.to(DEV), kn.to(DEV), vn.to(DEV), words, None if table is None else table.to(DEV), ints(lens), out)
    torch.cuda.synchronize()
    return out


def check_attention4(out, q, parts, kn, vn, sees, table, lens, scale):
    k, v = ref.values(*parts[:2]), ref.values(*parts[2:])
    want, spread, score = decoder_ref.tree_attention(q, k, v, kn, vn, sees, table, lens, scale)
    u, D = half_step(q.dtype), q.shape[3]
    # as over a plain cache: the weights' rounding and the output's, scores, exponentials and sums in fp32
    rel = 2 * u + 2 * (D + 4) * f * score + 2.0 ** -16
    err = (out.cpu().double() - want).abs()
    bad = err > rel * spread + 1e-30
    assert not bad.any(), f"off by {float((err / (rel * spread + 1e-30)).max()):.2f} of the bound at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("B,N,H,HK,D,lens,page,dtype,width", ATTN4, ids=lambda v: str(v)[:24])
def test_tree_attention_4_bits(ctx, B, N, H, HK, D, lens, page, dtype, width):
    g = torch.Generator().manual_seed(7)
    parts, table = make_cache4(lens, max(lens) + N, HK, D, page, 3, by_head=B % 2 == 1)
    q = (2 * torch.randn(B, N, H, D, generator=g)).to(dtype)
    kn, vn = (torch.randn(B, N, HK, D, generator=g).to(dtype) for _ in range(2))
    sees = sees_of(trees(random.Random(5), B, N, width))
    out = run_attention4(ctx, q, parts, kn, vn, None if width == 0 else words_of(sees), table, lens, D ** -0.5)
    check_attention4(out, q, parts, kn, vn, sees, table, lens, D ** -0.5)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("G,N,n", [(1, 3, 0), (8, 20, 0), (2, 64, 70), (1, 1, 5)])
def test_attention4_nothing_seen_and_odd_values(ctx, G, N, n, dtype):
    """Nodes that see nothing, infinities and NaN of nodes that are not seen, and of nodes that are."""
    HK, D = 2, 64
    g = torch.Generator().manual_seed(8)
    parts, table = make_cache4([n], n + N, HK, D, 16, 9)
    q = torch.randn(1, N, HK * G, D, generator=g).to(dtype)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(dtype) for _ in range(2))
    sees = torch.eye(N, dtype=torch.bool)[None].clone()
    sees[0, 0] = False
    if N > 2:
        vn[0, 1, 0, 5], vn[0, 2, 1, 6], kn[0, 0, :, 3], vn[0, 0] = float("inf"), NAN, NAN, float("-inf")
    out = run_attention4(ctx, q, parts, kn, vn, words_of(sees), table, [n], D ** -0.5).cpu()
    clean_k, clean_v = kn.clone(), vn.clone()
    clean_k[0, 0], clean_v[~vn.isfinite()] = 0, 0
    if n == 0:
        assert (out[0, 0] == 0).all()
    check = [i for i in range(N) if i not in (1, 2)]
    want = run_attention4(ctx, q, parts, clean_k, clean_v, words_of(sees), table, [n], D ** -0.5).cpu()
    assert torch.equal(out[0, check], want[0, check])
    if N > 2:
        assert (out[0, 1, :G, 5] == float("inf")).all() and out[0, 2, G:, 6].isnan().all()
        assert out[0, 1, G:].isfinite().all() and out[0, 2, :G].isfinite().all()


def test_attention4_bad_pages_lengths_and_repeats(ctx):
    B, N, HK, D = 3, 2, 2, 128
    g = torch.Generator().manual_seed(10)
    parts, table = make_cache4([40, 64, 90], 96, HK, D, 16, 11, junk=False)
    table[0, 1], table[2, 3] = -3, 1 << 20
    q = torch.randn(B, N, 8, D, generator=g).to(F16)
    kn, vn = (torch.randn(B, N, HK, D, generator=g).to(F16) for _ in range(2))
    out = run_attention4(ctx, q, parts, kn, vn, None, table, [40, -7, 1 << 30], D ** -0.5, max_batch=9)
    lens = [40, 0, 96]
    check_attention4(out, q, parts, kn, vn, torch.ones(B, N, N, dtype=torch.bool).tril(), table, lens, D ** -0.5)
    for _ in range(3):
        assert torch.equal(out, run_attention4(ctx, q, parts, kn, vn, None, table, [40, -7, 1 << 30], D ** -0.5, max_batch=9))


@pytest.mark.parametrize("scale", [2.0 ** -30, 1.0, 2.0 ** 60])
def test_attention4_query_range(ctx, scale):
    """bf16 queries beyond fp16's range on both sides: their size is taken off before the products."""
    B, N, HK, D, n = 1, 3, 1, 64, 100
    g = torch.Generator().manual_seed(12)
    parts, table = make_cache4([n], n, HK, D, 0, 13)
    q = (torch.randn(B, N, 2, D, generator=g) * scale).to(BF16)
    kn = torch.zeros(B, N, HK, D, dtype=BF16)
    vn = torch.randn(B, N, HK, D, generator=g).to(BF16)
    sees = torch.ones(B, N, N, dtype=torch.bool).tril()
    out = run_attention4(ctx, q, parts, kn, vn, None, table, [n], 0.1 / scale)
    check_attention4(out, q, parts, kn, vn, sees, table, [n], 0.1 / scale)


# ---------------------------------------------------------------- attention of packed prompts

def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def run_prompt(ctx, q, k, v, cu_q, cu_k, scale, out=None):
    p = pi.PromptAttn(ctx, q.shape[1], k.shape[1], q.shape[2], q.dtype, q.shape[0], len(cu_q) - 1, scale)
    out = torch.full(q.shape, NAN, dtype=q.dtype, device=DEV) if out is None else out
    dev = lambda t: t if t.device.type == "cuda" else t.to(DEV)  # noqa: E731
    pi.prompt_attention(ctx, p, dev(q), dev(k), dev(v), ints(cu_q), None if cu_k is None else ints(cu_k), out)
    torch.cuda.synchronize()
    return out


def check_prompt(out, q, k, v, cu_q, cu_k, scale):
    want, spread, score = ref.prompt(q, k, v, cu_q, cu_k, scale)
    u, D = half_step(q.dtype), q.shape[2]
    rel = 2 * u + 2 * (D + 4) * f * score + 2.0 ** -16  # as for trees
    o = out.cpu().double()
    outside = want.isnan()
    assert o[outside].isnan().all(), "rows of no sequence were written"
    err = torch.where(outside, 0.0, (o - want).abs())
    bad = ~(err <= rel * spread + 1e-30)
    assert not bad.any(), f"off by {float((err / (rel * spread + 1e-30)).max()):.2f} of the bound at {bad.nonzero()[0].tolist()}"


PROMPT = [
    # H, HK, D, dtype, [(queries, held before)]
    (1, 1, 8, F16, [(1, 0)]),
    (4, 4, 64, F16, [(5, 0), (0, 0), (1, 0), (64, 0), (65, 0)]),
    (8, 1, 128, BF16, [(33, 0), (7, 90), (1, 200)]),
    (8, 2, 80, F16, [(40, 3), (2, 0), (0, 9), (31, 64)]),
    (12, 4, 96, BF16, [(100, 27)]),
    (5, 1, 256, F16, [(70, 0), (3, 61)]),
    (2, 2, 256, BF16, [(130, 5)]),
    (6, 2, 40, BF16, [(20, 0)] * 5),
    (2, 1, 64, F16, [(1, i) for i in range(70)]),
    (2, 2, 128, F16, [(300, 0)]),
    (1, 1, 128, BF16, [(257, 130), (1, 1)]),
    (16, 2, 64, F16, [(1, 700), (2, 1000)]),
]


@pytest.mark.parametrize("H,HK,D,dtype,seqs", PROMPT, ids=lambda v: str(v)[:20])
def test_prompt_attention(ctx, H, HK, D, dtype, seqs):
    g = torch.Generator().manual_seed(14)
    cu_q, cu_k = offsets([n for n, _ in seqs]), offsets([n + h for n, h in seqs])
    # rows behind the last sequence: NaN, which may not enter, and outputs that stay as they are
    q = (2 * torch.randn(cu_q[-1] + 3, H, D, generator=g)).to(dtype)
    k, v = (torch.randn(cu_k[-1] + 2, HK, D, generator=g).to(dtype) for _ in range(2))
    k[cu_k[-1]:], v[cu_k[-1]:] = NAN, NAN
    out = run_prompt(ctx, q, k, v, cu_q, cu_k if any(h for _, h in seqs) else None, D ** -0.5)
    check_prompt(out, q, k, v, cu_q, cu_k, D ** -0.5)


def test_prompt_more_queries_than_keys(ctx):
    """The first queries of a sequence with fewer keys see nothing; one without keys is all zeros."""
    g = torch.Generator().manual_seed(15)
    cu_q, cu_k = offsets([90, 4, 10]), offsets([20, 0, 10])
    q = torch.randn(104, 4, 64, generator=g).to(F16)
    k, v = (torch.randn(30, 2, 64, generator=g).to(F16) for _ in range(2))
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, 0.125)
    check_prompt(out, q, k, v, cu_q, cu_k, 0.125)
    assert (out[:70] == 0).all() and (out[90:94] == 0).all()
    none = torch.empty(0, 2, 64, dtype=F16)
    assert (run_prompt(ctx, q, none, none, cu_q, [0, 0, 0, 0], 0.125) == 0).all()


@pytest.mark.parametrize("dtype,H,HK", [(F16, 4, 4), (BF16, 16, 2)])
def test_prompt_unseen_values_do_not_enter(ctx, dtype, H, HK):
    """Infinities and NaN of later keys, of other sequences' keys, and of seen ones."""
    g = torch.Generator().manual_seed(16)
    lens, D = [70, 130], 64
    cu = offsets(lens)
    q = torch.randn(200, H, D, generator=g).to(dtype)
    k, v = (torch.randn(200, HK, D, generator=g).to(dtype) for _ in range(2))
    want = run_prompt(ctx, q, k, v, cu, None, 0.125).cpu()
    v[40, 0, 7], v[41, 0, 8], k[50, 0, 3], v[170, HK - 1, 9] = float("inf"), NAN, NAN, float("-inf")
    out = run_prompt(ctx, q, k, v, cu, None, 0.125).cpu()
    G = H // HK
    assert torch.equal(out[:40], want[:40])
    assert (out[40:50, :G, 7] == float("inf")).all() and out[41:50, :G, 8].isnan().all()
    assert torch.equal(out[40:50, :G, :7], want[40:50, :G, :7])
    assert out[50:70, :G].isnan().all()  # a score that is NaN
    assert torch.equal(out[:70, G:H], want[:70, G:H])
    assert torch.equal(out[70:170], want[70:170])
    assert (out[170:, H - G:, 9] == float("-inf")).all()
    assert torch.equal(out[170:, H - G:, :9], want[170:, H - G:, :9])


def test_prompt_views_odd_offsets_and_repeats(ctx):
    g = torch.Generator().manual_seed(17)
    H, HK, D, T = 6, 2, 64, 150
    qkv = torch.randn(T, H + 2 * HK, D, generator=g).to(F16).to(DEV)
    q, k, v = qkv.split([H, HK, HK], 1)
    wide = torch.full((T, 2 * H, D), NAN, dtype=F16, device=DEV)
    cu = [3, 60, 60, 141]  # rows in front of the first sequence stay too
    out = run_prompt(ctx, q, k, v, cu, None, 0.125, out=wide[:, ::2])
    x = qkv.cpu()
    check_prompt(out, x[:, :H], x[:, H:H + HK], x[:, H + HK:], cu, cu, 0.125)
    assert wide[:, 1::2].isnan().all()
    for _ in range(3):
        assert torch.equal(out.nan_to_num(), run_prompt(ctx, q, k, v, cu, None, 0.125).nan_to_num())
    # offsets that descend or lie outside the rows stay inside the tensors
    for bad in ([-5, 100000, 20, 7], [140, 30, 160, 10], [-(1 << 31), (1 << 31) - 1, 0, 150]):
        run_prompt(ctx, q, k, v, bad, None, 0.125, out=wide[:, ::2])
    assert wide[:, 1::2].isnan().all()


# ---------------------------------------------------------------- together

def serve(ctx, dtype=F16, graph=False):
    """A prompt, a drafted step and the prompt's continuation of two sequences over a 4-bit cache. Returns what
    each attention gave and was given."""
    g = torch.Generator().manual_seed(18)
    H, HK, D, page, L, N = 8, 2, 64, 16, [37, 20], 3
    freq = (10000.0 ** (-torch.arange(D // 2).double() / (D // 2))).float().to(DEV)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DEV)
    table = torch.randperm(2 * 8, generator=g).to(I32).view(2, 8).to(DEV)
    codes = [torch.zeros(16, page, HK, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros(16, page, HK, D // 32, dtype=F16, device=DEV) for _ in range(2)]
    cache = pi.KvCache4(ctx, *codes, *scales, dtype)
    attn = pi.Attn(ctx, cache, H, 2, N)
    prompt = pi.PromptAttn(ctx, H, HK, D, dtype, 100, 2)
    held = ints([0, 0])
    out = []

    def heads(T, pos):
        qkv = torch.randn(T, H + 2 * HK, D, generator=g).to(dtype).to(DEV)
        q, k, v = qkv.split([H, HK, HK], 1)
        pi.qk_norm_rope(ctx, q, k, ints(pos), freq, q, k, q_norm=w, k_norm=w)
        return q, k, v

    # the prompts, packed; each enters the cache from its rows
    cu = offsets(L)
    q, k, v = heads(cu[-1], [*range(L[0]), *range(L[1])])
    o = torch.empty(q.shape, dtype=dtype, device=DEV)
    pi.prompt_attention(ctx, prompt, q, k, v, ints(cu), None, o)
    out.append((o, q, k, v, cu, cu))
    most = max(L)
    kn, vn = (torch.zeros(2, most, HK, D, dtype=dtype, device=DEV) for _ in range(2))
    for b in range(2):
        kn[b, :L[b]], vn[b, :L[b]] = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
    pi.kv_append(ctx, cache, kn, vn, table, held, held, n=ints(L))
    # a chain of drafted tokens, all kept
    q, k, v = (t.unflatten(0, (2, N)) for t in heads(2 * N, [L[b] + i for b in range(2) for i in range(N)]))
    o = torch.empty(2, N, H, D, dtype=dtype, device=DEV)
    pi.tree_attention(ctx, attn, q, k, v, None, table, held, o)
    out.append((o, q, k, v, held.tolist()))
    pi.kv_append(ctx, cache, k, v, table, held, held)
    # the continuation: what is held is read back, the new rows follow it
    more, now = [11, 5], [a + N for a in L]
    cu_q, cu_k = offsets(more), offsets([a + m for a, m in zip(now, more)])
    q, k, v = heads(cu_q[-1], [now[b] + i for b in range(2) for i in range(more[b])])
    ka, va = (torch.full((cu_k[-1], HK, D), NAN, dtype=dtype, device=DEV) for _ in range(2))
    pi.kv_read(ctx, cache, table, held, ints(cu_k), ka, va)
    for b in range(2):
        ka[cu_k[b] + now[b]:cu_k[b + 1]], va[cu_k[b] + now[b]:cu_k[b + 1]] = k[cu_q[b]:cu_q[b + 1]], v[cu_q[b]:cu_q[b + 1]]
    o = torch.empty(q.shape, dtype=dtype, device=DEV)
    pi.prompt_attention(ctx, prompt, q, ka, va, ints(cu_q), ints(cu_k), o)
    out.append((o, q, ka, va, cu_q, cu_k))
    torch.cuda.synchronize()
    return out, cache, table


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_draft_and_continuation(ctx, dtype):
    (first, step, more), cache, table = serve(ctx, dtype)
    o, q, k, v, cu, _ = first
    check_prompt(o, q.cpu(), k.cpu(), v.cpu(), cu, cu, 0.125)
    parts = [t.cpu() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    # the cache holds the prompt's keys, quantised
    for b in range(2):
        for p in range(cu[b + 1] - cu[b]):
            c, s = ref.quantize(k[cu[b] + p].cpu())
            pg = int(table[b, p // 16])
            assert torch.equal(parts[0][pg, p % 16], c) and torch.equal(parts[1][pg, p % 16], s)
    o, q, k, v, held = step
    sees = torch.ones(2, 3, 3, dtype=torch.bool).tril()
    check_attention4(o, q.cpu(), parts, k.cpu(), v.cpu(), sees, table.cpu(), held, 0.125)
    o, q, k, v, cu_q, cu_k = more
    val = ref.values(*parts[:2]).to(dtype)
    for b in range(2):
        for p in range(held[b] + 3):
            assert torch.equal(k[cu_k[b] + p].cpu(), val[int(table[b, p // 16]), p % 16])
    check_prompt(o, q.cpu(), k.cpu(), v.cpu(), cu_q, cu_k, 0.125)


def test_prompts_in_a_graph_and_on_a_stream():
    """All operators captured into one graph on a stream of their own, replayed with other inputs and lengths."""
    st = torch.cuda.Stream()
    c = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0, stream=st)
    g = torch.Generator().manual_seed(19)
    H, HK, D, T, N = 4, 2, 128, 40, 2
    freq = torch.linspace(1, 0.01, D // 2).to(DEV)
    qkv = torch.empty(T, H + 2 * HK, D, dtype=F16, device=DEV)
    q, k = (torch.empty(T, n, D, dtype=F16, device=DEV) for n in (H, HK))
    v = torch.empty(T, HK, D, dtype=F16, device=DEV)
    pos, cu = torch.arange(T, dtype=I32, device=DEV), ints([0, 25, 40])
    codes = [torch.zeros(8, 16, HK, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros(8, 16, HK, D // 32, dtype=F16, device=DEV) for _ in range(2)]
    cache = pi.KvCache4(c, *codes, *scales, F16)
    attn, prompt = pi.Attn(c, cache, H, 1, N), pi.PromptAttn(c, H, HK, D, F16, T, 2)
    held, now, rows = ints([0]), ints([0]), ints([0, T])
    o, o4 = torch.empty(T, H, D, dtype=F16, device=DEV), torch.empty(1, N, H, D, dtype=F16, device=DEV)
    kr, vr = (torch.empty(T, HK, D, dtype=F16, device=DEV) for _ in range(2))
    table = ints([[3, 1, 7, 0, 2, 6, 5, 4]])

    def work():
        pi.qk_norm_rope(c, qkv[:, :H], qkv[:, H:H + HK], pos, freq, q, k)
        pi.prompt_attention(c, prompt, q, k, qkv[:, H + HK:], cu, None, o)
        pi.kv_append(c, cache, k[None], v[None], table, held, now)
        pi.tree_attention(c, attn, q[None, :N], k[None, :N], v[None, :N], None, table, now, o4)
        pi.kv_read(c, cache, table, now, rows, kr, vr, start=held)

    def fresh(i):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        v.copy_(qkv[:, H + HK:])
        held.fill_(7 * i)
        cu.copy_(torch.tensor([0, 10 + i, 40 - i]))
        for t in (o, o4, kr, vr):
            t.zero_()
        torch.cuda.synchronize()

    fresh(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        work()
    for i in range(4):
        fresh(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, o4, kr, vr, now)]
        for t in (o, o4, kr, vr):
            t.zero_()
        torch.cuda.synchronize()
        work()
        torch.cuda.synchronize()
        for a, b in zip(got, (o, o4, kr, vr, now)):
            assert torch.equal(a, b)
        assert int(now) == 7 * i + T and o4.abs().sum() > 0


def test_refusals_of_prompt_operators(ctx):
    def refused(match, call, *a, **kw):
        with pytest.raises(pi.PiError, match=match):
            call(*a, **kw)

    e = lambda *s, dtype=F16: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    k, s = e(4, 16, 2, 32, dtype=torch.uint8), e(4, 16, 2, 2)
    cache = pi.KvCache4(ctx, k, k, s, s, F16)
    refused("multiples of 16 bytes", pi.KvCache4, ctx, e(4, 16, 2, 40, dtype=torch.uint8)[..., :32], e(4, 16, 2, 40, dtype=torch.uint8)[..., :32], s, s, F16)
    refused("above 256", pi.KvCache4, ctx, *[e(4, 16, 2, 144, dtype=torch.uint8)] * 2, *[e(4, 16, 2, 9)] * 2, F16)
    refused("must be even", pi.KvCache4, ctx, k, k, *[e(4, 16, 2, 3)[..., :2]] * 2, F16)
    refused("has shape", pi.KvCache4, ctx, k, k, s, e(4, 16, 2, 3), F16)
    refused("no multiple", pi.Attn, ctx, cache, 3, 1, 1)
    refused("without a page table", pi.kv_read, ctx, cache, None, ints([1] * 5), ints([0] * 6), e(1, 2, 64), e(1, 2, 64))
    refused("multiples of 8", pi.kv_read, ctx, cache, None, ints([1]), ints([0, 1]), e(2, 2, 68)[..., :64], e(2, 2, 68)[..., :64])
    refused("no multiple", pi.PromptAttn, ctx, 4, 3, 64, F16, 8, 1)
    refused("multiple of 8", pi.PromptAttn, ctx, 4, 2, 60, F16, 8, 1)
    refused("above 256", pi.PromptAttn, ctx, 4, 2, 264, F16, 8, 1)
    refused("too many", pi.PromptAttn, ctx, 1024, 2, 64, F16, 1 << 20, 1)
    refused("scale", pi.PromptAttn, ctx, 4, 2, 64, F16, 8, 1, 0.0)
    p = pi.PromptAttn(ctx, 4, 2, 64, F16, 8, 1)
    q, kv = e(9, 4, 64), e(9, 2, 64)
    refused("above the handle's", pi.prompt_attention, ctx, p, q, kv, kv, ints([0, 9]), None, q)
    refused("above the handle's", pi.prompt_attention, ctx, p, q[:8], kv, kv, ints([0, 4, 8]), None, q[:8])
    refused("has type", pi.prompt_attention, ctx, p, q.to(BF16), kv, kv, ints([0, 9]), None, q)
    other = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)
    refused("another context", pi.prompt_attention, other, p, q[:8], kv, kv, ints([0, 8]), None, q[:8])
    refused("another context", pi.kv_read, other, cache, None, ints([1]), ints([0, 1]), e(1, 2, 64), e(1, 2, 64))
    fr = e(32, dtype=F32)
    refused("multiple of 4", pi.qk_norm_rope, ctx, q, None, ints([0] * 9), e(31, dtype=F32), q, None)
    refused("heads of 64", pi.qk_norm_rope, ctx, q, None, ints([0] * 9), e(33, dtype=F32), q, None)
    refused("16-byte aligned", pi.qk_norm_rope, ctx, e(9, 4, 68)[..., :64], None, ints([0] * 9), fr, q, None)
    refused("in place", pi.qk_norm_rope, ctx, q, None, ints([0] * 9), fr, q.view(BF16), None)
    refused("eps", pi.qk_norm_rope, ctx, q, None, ints([0] * 9), fr, q, None, eps=-1.0)
