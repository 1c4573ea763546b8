"""Every kernel variant of the decoder operators at its borders, calls captured into a graph, on
another stream, over strides past 32 bits, and all operators together in one serving step.

Tolerances as in test_gpu_decoder: u is half a step of the output's type, f = 2^-24.
"""
import importlib.util
import os
import random

import pytest
import torch

from tests import decoder_ref as ref
from tests import test_gpu_decoder as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

DEV, F16, BF16, F32, I32 = "cuda", torch.float16, torch.bfloat16, torch.float32, torch.int32
f = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


# ------------------------------------------------------------------------------- product

@pytest.mark.parametrize("M,N,K", [(1, 33, 131056), (2, 48, 32768), (15, 40, 4096), (16, 40, 4096), (16, 300, 4080),
                                   (17, 300, 272), (130, 260, 2064), (129, 129, 16), (300, 2000, 528), (4100, 4097, 144),
                                   (8200, 2049, 16)])
def test_product_sums_are_exact(ctx, M, N, K):
    """Unit scales and fp32 output: the whole-number sums themselves, below 2^24 where they are not
    multiples of a power of two that keeps them exact."""
    g = torch.Generator(DEV).manual_seed(K + M)
    top = 127 if K < 1040 else 11  # 11^2 K below 2^24
    x = torch.randint(-top, top + 1, (M, K), generator=g, device=DEV).to(torch.int8)
    w = torch.randint(-top, top + 1, (N, K), generator=g, device=DEV).to(torch.int8)
    lin = pi.Linear(ctx, w, torch.ones(N, device=DEV), max_tokens=M)
    y = torch.full((M, N), float("nan"), device=DEV)
    pi.linear_q8(ctx, lin, x, torch.ones(M, device=DEV), y)
    # fp32 products of such values are exact whatever their order
    assert torch.equal(y, x.float() @ w.float().t())


@pytest.mark.parametrize("M,N", [(5, 300), (40, 300), (200, 129)])
def test_product_views_of_split_tiles(ctx, M, N):
    """Rows of wider tensors with their neighbours untouched, outputs off a vector's boundary."""
    K = 2064
    g = torch.Generator(DEV).manual_seed(M)
    xb = torch.randint(-9, 10, (M, K + 64), generator=g, device=DEV).to(torch.int8)
    wb = torch.randint(-9, 10, (N, K + 32), generator=g, device=DEV).to(torch.int8)
    out = torch.full((M, N + 9), 7.0, device=DEV)
    bias = torch.randint(-5, 6, (N,), generator=g, device=DEV).float()
    lin = pi.Linear(ctx, wb[:, 16:16 + K], torch.ones(N, device=DEV), bias, max_tokens=M)
    pi.linear_q8(ctx, lin, xb[:, 32:32 + K], torch.ones(M, device=DEV), out[:, 3:3 + N])
    assert torch.equal(out[:, 3:3 + N], xb[:, 32:32 + K].float() @ wb[:, 16:16 + K].float().t() + bias)
    assert (out[:, :3] == 7).all() and (out[:, 3 + N:] == 7).all()


def test_product_refuses_far_rows(ctx):
    w = torch.empty_strided((2, 64), (1 << 22, 1), dtype=torch.int8, device=DEV)
    with pytest.raises(pi.PiError, match="2\\^22"):
        pi.Linear(ctx, w, torch.ones(2, device=DEV))
    lin = pi.Linear(ctx, torch.zeros(2, 64, dtype=torch.int8, device=DEV), torch.ones(2, device=DEV), max_tokens=2)
    with pytest.raises(pi.PiError, match="2\\^22"):
        pi.linear_q8(ctx, lin, w, torch.ones(2, device=DEV), torch.empty(2, 2, device=DEV))


# ------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("step", [0.5, 3.0, 9.0, -3.0])
@pytest.mark.parametrize("G,dtype", [(1, F16), (40, F16), (40, BF16), (8, BF16)])
def test_attention_scores_that_climb(ctx, step, G, dtype):
    """Scores that rise (or fall) along the cache by less and by more than the kernel lets the
    maximum run ahead of its base."""
    g = torch.Generator().manual_seed(3)
    n, N, HK, D, page = 700, 5, 1, 64, 16
    k, v, table = base.make_cache(ctx, [n], n + N, HK, D, page, dtype, 3)
    rise = torch.arange(n) / 64 * step  # per 64 keys, in units of the score
    for p in range(n):
        k[int(table[0, p // page]), p % page] = (rise[p] / D + 0.02 * torch.randn(D, generator=g)).to(dtype)
    q = torch.ones(1, N, G, D).to(dtype)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(dtype) for _ in range(2))
    sees = base.sees_of(base.trees(random.Random(5), 1, N, 3))
    out = base.run_attention(ctx, q, k, v, kn, vn, base.words_of(sees), table, [n], 1.0)
    base.check_attention(out, q, k, v, kn, vn, sees, table, [n], 1.0)


@pytest.mark.parametrize("D,H,HK,N,page", [(128, 32, 1, 64, 1), (128, 16, 2, 40, 0), (64, 64, 1, 5, 3), (96, 24, 1, 11, 100),
                                           (256, 12, 1, 30, 33), (40, 9, 3, 64, 17)])
def test_attention_many_rows(ctx, D, H, HK, N, page):
    """Several row tiles, pages that end inside tiles, head sizes that are not the tile's."""
    g = torch.Generator().manual_seed(D)
    lens = [191, 0, 64]
    k, v, table = base.make_cache(ctx, lens, 191 + N, HK, D, page, F16, 3, fill=float("nan"))
    q = (2 * torch.randn(3, N, H, D, generator=g)).to(F16)
    kn, vn = (torch.randn(3, N, HK, D, generator=g).to(F16) for _ in range(2))
    sees = base.sees_of(base.trees(random.Random(7), 3, N, 3))
    out = base.run_attention(ctx, q, k, v, kn, vn, base.words_of(sees), table, lens, D ** -0.5)
    base.check_attention(out, q, k, v, kn, vn, sees, table, lens, D ** -0.5)


def test_cache_past_32_bits(ctx):
    """Pages 2^30 elements apart: element offsets up to 3 * 2^30."""
    page, HK, D, n, N = 16, 1, 64, 50, 3
    buf = [torch.empty(3 * (1 << 30) + page * D, dtype=F16, device=DEV) for _ in range(2)]
    kv = [b.as_strided((4, page, HK, D), (1 << 30, D, D, 1)) for b in buf]
    for t in kv:
        t.zero_()
    g = torch.Generator().manual_seed(5)
    table = torch.tensor([[3, 0, 2, 1]], dtype=I32)
    old_k, old_v = (torch.randn(1, n, HK, D, generator=g).to(F16) for _ in range(2))
    cache = pi.KvCache(ctx, *kv)
    lens = torch.zeros(1, dtype=I32, device=DEV)
    pi.kv_append(ctx, cache, old_k.to(DEV), old_v.to(DEV), table.to(DEV), lens, lens)
    q = torch.randn(1, N, 2, D, generator=g).to(F16)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(F16) for _ in range(2))
    attn = pi.Attn(ctx, cache, 2, 1, N)
    out = torch.empty(1, N, 2, D, dtype=F16, device=DEV)
    pi.tree_attention(ctx, attn, q.to(DEV), kn.to(DEV), vn.to(DEV), None, table.to(DEV), lens, out)
    torch.cuda.synchronize()
    k, v = (t.cpu() for t in kv)
    assert lens.tolist() == [n]
    for p in range(n):
        assert torch.equal(k[int(table[0, p // page]), p % page], old_k[0, p])
    base.check_attention(out, q, k, v, kn, vn, base.sees_of([[-1, 0, 1]]), table, [n], D ** -0.5)


# ------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("d", [64, 4096, 20000])
def test_norm_of_extreme_rows(ctx, d):
    """Rows whose squares leave fp32's range, rows of zeros, rows with what has no norm."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn(6, d, generator=g)
    x[1] *= 1e25
    x[2] *= 1e-25
    x[3] = 0
    x[4, 7] = float("nan")
    x[5, d - 1] = float("-inf")
    x = x.to(DEV)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    ro, y = torch.empty_like(x), torch.empty_like(x)
    q, scale = torch.empty(6, d, dtype=torch.int8, device=DEV), torch.empty(6, device=DEV)
    pi.add_rmsnorm(ctx, x, None, w, 0.0, ro, q=q, scale=scale, y=y)
    torch.cuda.synchronize()
    h = x[:3].double()
    want = h / h.square().mean(1, keepdim=True).sqrt() * w.double()
    # as for ordinary rows (each thread's up to 32 squares, 10 steps of the tree, half of it in the
    # root; division, root, reciprocal, products), and the scaling's two exact steps
    rel = (21 + 6) * f
    assert ((y[:3].double() - want).abs() <= rel * want.abs()).all()
    assert ((scale[:3].double() * 127 - want.abs().amax(1)).abs() <= (rel + 2 * f) * want.abs().amax(1)).all()
    assert (q[:3].abs().amax(1) == 127).all()
    assert (y[3] == 0).all() and scale[3] == 0 and (q[3:] == 0).all() and scale[4:].isnan().all()


# ------------------------------------------------------------------------------- verification

@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("V", [700, 40001])
def test_verify_draws_at_the_border(ctx, with_q, V):
    """A first child whose number lies as near to its border as fp32 goes, on either side."""
    for seed in range(8):
        c = base.verify_case(2, 6, V, F16, 3, with_q, 1.0, seed)
        for b in range(2):
            kid = int((c["parents"][b] == 0).nonzero()[0, 0])
            t = int(c["tokens"][b, kid])
            p = torch.softmax(c["logits"][b, 0].double(), 0)[t]
            c["u"][b, kid] = p if c["q"] is None else (p / c["q"][b, 0, t].double()).clamp(max=1.0)
        base.check_verify(base.run_verify(ctx, c), c)


@pytest.mark.parametrize("V,N,u", [(70001, 9, 0.999), (70001, 3, 0.999), (131072, 2, 0.5), (66000, 1, 0.5)])
def test_verify_rejections_of_large_vocabularies(ctx, V, N, u):
    """More and fewer rejections in one family than there are passes."""
    g = torch.Generator().manual_seed(V + N)
    logits = 3 * torch.randn(2, N, V, generator=g)
    q = torch.softmax(3 * torch.randn(2, N, V, generator=g), 2)
    tok = torch.stack([torch.multinomial(q[b, 0], N, generator=g) for b in range(2)]).to(I32)
    par = torch.zeros(2, N, dtype=I32)
    par[:, 0] = -1
    c = dict(logits=logits, tokens=tok, parents=par, u=torch.full((2, N), u), u_next=torch.tensor([0.37, 0.9999]), q=q,
             temp=torch.tensor([1.0, 0.7]))
    base.check_verify(base.run_verify(ctx, c), c)
    base.check_verify(base.run_verify(ctx, dict(c, q=None)), dict(c, q=None))


def test_verify_many_sequences_of_a_large_vocabulary(ctx):
    """A batch that takes the longer run of passes, its sequences done after unlike numbers of them."""
    c = base.verify_case(17, 9, 66001, F16, 3, True, 1.0, 5)
    c["u"] = (c["u"] * torch.linspace(0.2, 1.0, 17)[:, None] + 0.3).clamp(max=0.999)
    base.check_verify(base.run_verify(ctx, c), c)


def test_verify_very_cold_and_very_hot(ctx):
    for temp in (1e-3, 1e-30, 1e6):
        c = base.verify_case(2, 5, 3000, F32, 2, False, 1.0, 3)
        c["temp"] = torch.full((2,), temp)
        base.check_verify(base.run_verify(ctx, c), c)


# ------------------------------------------------------------------------------- together

def _example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("draft_step", os.path.join(root, "examples", "draft_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _inputs(dec, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    tokens = torch.randint(0, dec.vocab, (dec.batch, dec.nodes), generator=g, device=DEV).to(I32)
    u = torch.rand(dec.batch, dec.nodes, generator=g, device=DEV)
    return tokens, u, u[:, 0].contiguous()


def test_serving_step(ctx):
    """Steps of the example: what is kept follows from the step's logits, the caches hold the kept
    nodes' keys and values in order, and a step repeated gives the same bits."""
    ex = _example()
    dec = ex.Decoder(layers=2, d=512, heads=8, kv_heads=2, vocab=1000, batch=2, nodes=6, page=8, pages=32)
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2], [-1, 0, 1, 2, 3, 4]], dtype=I32, device=DEV)
    tree = ex.ancestors(parents)
    held = [[], []]
    for s in range(3):
        tokens, u, un = _inputs(dec, s)
        logits = dec.forward(tokens, tree).clone()
        assert logits.isfinite().all()
        for b in range(2):  # drafts that the target likes: some are kept
            for i in range(1, 6):
                tokens[b, i] = logits[b, int(parents[b, i])].argmax() if i % 2 else tokens[b, i]
        before = dec.len.tolist()
        path, out, n = dec.step(tokens, parents, tree, u, un)
        first = [t.clone() for t in (path, out, n)]
        torch.cuda.synchronize()
        for b in range(2):
            want, toks = ref.verify(dec.logits[b].cpu(), tokens[b].cpu(), parents[b].cpu(), u[b].cpu(), un[b].cpu(), None, 1.0)
            assert path[b, :len(want)].tolist() == want and out[b, :len(want)].tolist() == toks and int(n[b]) == len(want)
            new = dec.layers[1]["new"][b, want, dec.heads:dec.heads + dec.kv_heads].clone()
            held[b].append(new)
            assert dec.len.tolist()[b] == before[b] + len(want)
            rows = torch.cat(held[b])
            k = dec.layers[1]["cache"].k[dec.table[b].long()].flatten(0, 1)[:len(rows)]
            assert torch.equal(k, rows)
    dec.len.copy_(torch.tensor(before, dtype=I32))
    again = dec.step(tokens, parents, tree, u, un)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_operators_in_a_graph_and_on_a_stream():
    """All operators captured once and replayed on new inputs, with eager work of the same handles
    in between; every replay equals the eager result."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ctx = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)
        g = torch.Generator(DEV).manual_seed(0)
        randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        B, N, H, HK, D, V = 2, 20, 16, 2, 64, 70000
        d = H * D
        w = torch.randint(-127, 128, ((H + 2 * HK) * D, d), generator=g, device=DEV).to(torch.int8)
        lin = pi.Linear(ctx, w, torch.full((w.shape[0],), 1e-3, device=DEV), max_tokens=B * N)
        cache = pi.KvCache(ctx, *(randn(64, 16, HK, D).to(F16) for _ in range(2)))
        attn = pi.Attn(ctx, cache, H, B, N)
        ver = pi.Verifier(ctx, V, B, N)
        x, res, nw = randn(B * N, d).to(F16), randn(B * N, d).to(F16), torch.ones(d, device=DEV)
        h, q8, sc = torch.empty_like(x), torch.empty(B * N, d, dtype=torch.int8, device=DEV), torch.empty(B * N, device=DEV)
        qkv = torch.empty(B, N, H + 2 * HK, D, dtype=F16, device=DEV)
        att = torch.empty(B, N, H, D, dtype=F16, device=DEV)
        table = torch.randperm(64, generator=g, device=DEV).to(I32).view(2, 32)
        lens = torch.tensor([300, 17], dtype=I32, device=DEV)
        grown = torch.empty_like(lens)
        logits, tok = randn(B, N, V).to(F16), torch.randint(0, V, (B, N), generator=g, device=DEV).to(I32)
        qd = torch.softmax(logits.float() + randn(B, N, V), 2)
        par = torch.tensor(base.trees(random.Random(1), B, N, 3), dtype=I32, device=DEV)
        u, un = torch.rand(B, N, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
        path, out = (torch.empty(B, N, dtype=I32, device=DEV) for _ in range(2))
        n = torch.empty(B, dtype=I32, device=DEV)

        def work():
            pi.add_rmsnorm(ctx, x, res, nw, 1e-5, h, q=q8, scale=sc)
            pi.linear_q8(ctx, lin, q8, sc, qkv.view(B * N, -1))
            q, k, v = qkv.split([H, HK, HK], 2)
            pi.tree_attention(ctx, attn, q, k, v, None, table, lens, att)
            pi.verify(ctx, ver, logits, tok, par, u, un, path, out, n, q=qd)
            pi.kv_append(ctx, cache, k, v, table, lens, grown, path, n)
            return [t.clone() for t in (h, q8, sc, qkv, att, path, out, n, cache.k, cache.v, grown)]

        work()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = work()
        for i in range(4):
            x.copy_(randn(B * N, d))
            logits.copy_(randn(B, N, V))
            u.copy_(torch.rand(B, N, generator=g, device=DEV))
            start = cache.k.clone(), cache.v.clone()
            graph.replay()
            stream.synchronize()
            got = [t.clone() for t in captured]
            cache.k.copy_(start[0])
            cache.v.copy_(start[1])
            want = work()
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_other_stream_than_the_tensors():
    """A context of one stream with tensors made and freed on another: their memory is not given
    away before the context's stream is done with it."""
    side = torch.cuda.Stream()
    ctx = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0, stream=side)
    M, N, K = 64, 4096, 4096
    w = torch.randint(-9, 10, (N, K), device=DEV).to(torch.int8)
    lin = pi.Linear(ctx, w, torch.ones(N, device=DEV), max_tokens=M)
    y = torch.empty(M, N, device=DEV)
    for i in range(10):
        x = torch.full((M, K), i - 5, dtype=torch.int8, device=DEV)
        xs = torch.ones(M, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        pi.linear_q8(ctx, lin, x, xs, y)
        del x, xs
        junk = [torch.full((M, K), 77, dtype=torch.int8, device=DEV) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y[0], (i - 5) * w.float().sum(1)), i
        del junk
