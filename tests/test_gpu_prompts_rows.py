"""Norm and rotation, the append to the 4-bit cache and the reading of both caches at sizes where a workgroup takes several
rows; and memory borrowed by a stream that is still busy."""
import pytest
import torch

from tests import prompt_ref as ref
from tests.test_gpu_prompts import BF16, DEV, F16, F32, I32, check_rope, ints

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


# T / 1024 tokens a workgroup at 256 compute units, up to 8, where a token has few heads
@pytest.mark.parametrize("T,H,HK,D,rot,xt,yt,norm,pairs", [
    (2051, 8, 2, 128, 128, F16, F16, True, False), (2051, 8, 2, 128, 64, BF16, BF16, True, True),
    (5003, 4, 1, 80, 40, BF16, F32, True, True), (9001, 3, 2, 64, 64, F32, F32, False, False),
    (9005, 12, 2, 96, 20, F16, BF16, True, False), (8203, 2, 0, 256, 252, BF16, F16, False, True),
    (4099, 0, 3, 512, 512, F16, F16, True, True), (10007, 2, 1, 8, 8, F32, F16, True, False),
    (3001, 70, 5, 64, 48, F16, F16, True, True), (9007, 4, 4, 48, 0, BF16, BF16, True, False),
])
def test_rope_of_many_tokens(ctx, T, H, HK, D, rot, xt, yt, norm, pairs):
    g = torch.Generator().manual_seed(61)
    qkv = (3 * torch.randn(T, H + 2 * HK, D, generator=g)).to(xt)
    pos = torch.randint(0, 200000, (T,), generator=g).to(I32)
    freq = (10000.0 ** (-torch.arange(rot // 2).double() / max(1, rot // 2))).float() if rot else None
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)) if norm else None for _ in range(2))
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    x = qkv.to(DEV)
    q, k = (x[:, :H] if H else None), (x[:, H:H + HK] if HK else None)
    qo, ko = (torch.full((T, n, D), float("nan"), dtype=yt, device=DEV) if n else None for n in (H, HK))
    pi.qk_norm_rope(ctx, q, k, dev(pos), dev(freq), qo, ko, q_norm=dev(wq), k_norm=dev(wk), interleaved=pairs)
    torch.cuda.synchronize()
    assert torch.equal(x.cpu(), qkv)
    if H:
        check_rope(qo, qkv[:, :H], wq, pos, freq, 1e-6, pairs)
    if HK:
        check_rope(ko, qkv[:, H:H + HK], wk, pos, freq, 1e-6, pairs)
    if xt is yt:  # in place
        pi.qk_norm_rope(ctx, q, k, dev(pos), dev(freq), q, k, q_norm=dev(wq), k_norm=dev(wk), interleaved=pairs)
        torch.cuda.synchronize()
        assert (not H or torch.equal(q, qo)) and (not HK or torch.equal(k, ko)) and torch.equal(x[:, H + HK:].cpu(), qkv[:, H + HK:])


def same(a, b):
    a, b = a.cpu(), b.cpu()
    if a.dtype is F16:  # scales: NaN are alike, zeros by their sign too
        nan = a.isnan()
        return torch.equal(nan, b.isnan()) and torch.equal(a.view(torch.int16)[~nan], b.view(torch.int16)[~nan])
    return torch.equal(a, b)


# B * N / 2048 tokens a workgroup, up to 16
@pytest.mark.parametrize("B,N,HK,D,page,dtype", [(3, 2001, 2, 64, 16, F16), (5, 7003, 1, 96, 48, BF16), (2, 20011, 2, 32, 5, F16),
                                                  (40, 130, 3, 256, 64, BF16)])
def test_append_of_many_tokens(ctx, B, N, HK, D, page, dtype):
    g = torch.Generator().manual_seed(62)
    lens = [(37 * b) % 101 for b in range(B)]
    width = -(-(N + 60) // page)  # some sequences reach past it
    pages = B * width
    table = torch.randperm(pages, generator=g).to(I32).view(B, width)
    table[0, 2], table[1, width // 2] = -1, pages  # outside the cache: dropped
    kn, vn = (torch.randn(B, N, HK, D, generator=g).to(dtype) for _ in range(2))
    kn[0, 100, 0, :32], vn[1, 3, 0, 1], kn[1, 50, 0, 2] = 0, float("inf"), float("nan")
    n = torch.tensor([(N, N - 1, N // 2, 0, N + 5)[b % 5] for b in range(B)], dtype=I32)
    nodes = torch.stack([torch.randperm(N, generator=g) for _ in range(B)]).to(I32)
    nodes[0, 7], nodes[1, 8], nodes[0, 9] = -1, N, nodes[0, 8]  # dropped, dropped, the same one twice
    parts = []
    for _ in range(2):
        parts += [torch.randint(0, 256, (pages, page, HK, D // 2), generator=g, dtype=torch.uint8),
                  torch.randn(pages, page, HK, D // 32, generator=g).to(F16)]
    want = [t.clone() for t in parts]
    for b in range(B):
        j = torch.arange(min(int(n[b]), N))
        at, src = lens[b] + j, nodes[b, j].long()
        ok = (at < width * page) & (src >= 0) & (src < N)
        at, src = at[ok], src[ok]
        pg = table[b].long()[at // page]
        ok = (pg >= 0) & (pg < pages)
        at, src, pg = at[ok], src[ok], pg[ok]
        for i, x in ((0, kn), (2, vn)):
            want[i][pg, at % page], want[i + 1][pg, at % page] = ref.quantize(x[b, src])
    k, ks, v, vs = (t.to(DEV) for t in parts)
    cache = pi.KvCache4(ctx, k, v, ks, vs, dtype)
    out_len = ints([-1] * B)
    pi.kv_append(ctx, cache, kn.to(DEV), vn.to(DEV), table.to(DEV), ints(lens), out_len, nodes.to(DEV), n.to(DEV))
    torch.cuda.synchronize()
    for w, o in zip(want, (k, ks, v, vs)):
        assert same(w, o)
    assert out_len.tolist() == [min(a + min(int(m), N), width * page) for a, m in zip(lens, n)]


# rows / 1024 a workgroup, up to 16
@pytest.mark.parametrize("kind", ["plain", "4 bits"])
@pytest.mark.parametrize("B,most,HK,D", [(3001, 12, 2, 64), (700, 9, 1, 256), (9, 900, 3, 96), (1, 20003, 1, 32)])
def test_read_of_many_rows(ctx, kind, B, most, HK, D):
    """Sequences of fewer rows than a workgroup takes, empty ones, and long ones; positions beyond the length stay."""
    page, g = 8, torch.Generator().manual_seed(63)
    ask = torch.randint(0, most + 1, (B,), generator=g)
    ask[torch.rand(B, generator=g) < 0.2] = 0
    if B == 1:
        ask[0] = most
    start = torch.randint(-2, 4, (B,), generator=g)
    lens = (start.clamp(min=0) + ask - torch.randint(0, 3, (B,), generator=g)).clamp(min=0)
    width = (most + 10) // page + 1
    pages = B * width
    table = torch.randperm(pages, generator=g).to(I32).view(B, width)
    table[B // 2, 0] = pages + 3  # zeros
    if kind == "plain":
        k, v = (torch.randn(pages, page, HK, D, generator=g).to(BF16) for _ in range(2))
        cache, vals = pi.KvCache(ctx, k.to(DEV), v.to(DEV)), (k, v)
    else:
        c = [ref.quantize(torch.randn(pages, page, HK, D, generator=g)) for _ in range(2)]
        cache = pi.KvCache4(ctx, c[0][0].to(DEV), c[1][0].to(DEV), c[0][1].to(DEV), c[1][1].to(DEV), BF16)
        vals = [ref.values(*x).to(BF16) for x in c]
    cu = torch.cat([torch.tensor([3]), 3 + ask.cumsum(0)])  # rows of no sequence in front and behind
    rows = int(cu[-1]) + 5
    b = torch.repeat_interleave(torch.arange(B), ask)
    row = torch.arange(3, int(cu[-1]))
    at = start.clamp(min=0)[b] + row - cu[b]
    row, b, at = (t[at < lens[b]] for t in (row, b, at))
    pg = table.long()[b, at // page]
    bad = pg >= pages
    ko, vo = (torch.full((rows, HK, D), 5.0, dtype=BF16, device=DEV) for _ in range(2))
    pi.kv_read(ctx, cache, table.to(DEV), lens.to(I32).to(DEV), cu.to(I32).to(DEV), ko, vo, start=start.to(I32).to(DEV))
    torch.cuda.synchronize()
    for o, x in ((ko, vals[0]), (vo, vals[1])):
        want = torch.full((rows, HK, D), 5.0, dtype=BF16)
        want[row] = torch.where(bad[:, None, None], 0, x[pg.clamp(max=pages - 1), at % page])
        assert torch.equal(want, o.cpu())


def test_memory_of_a_busy_stream_is_not_reused():
    """Inputs freed while the context's stream has not come to the call yet: new tensors lie elsewhere, and the results are
    those of an idle stream."""
    st = torch.cuda.Stream()
    c = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0, stream=st)
    g = torch.Generator().manual_seed(64)
    H, HK, D, T, N, page = 8, 4, 64, 1500, 4, 16
    host = dict(q=torch.randn(T, H, D, generator=g).to(F16), k=torch.randn(T, HK, D, generator=g).to(F16),
                v=torch.randn(T, HK, D, generator=g).to(F16), cu=torch.tensor([0, 700, T], dtype=I32),
                pos=torch.arange(T, dtype=I32), freq=torch.linspace(1, 0.01, D // 2), w=torch.randn(D, generator=g),
                held=torch.tensor([0], dtype=I32), full=torch.tensor([T], dtype=I32), rows=torch.tensor([0, T], dtype=I32),
                table=torch.randperm(100, generator=g).to(I32).view(1, 100))
    prompt = pi.PromptAttn(c, H, HK, D, F16, T, 2)
    a = torch.randn(4096, 4096, device=DEV)
    b = torch.empty_like(a)
    done = torch.cuda.Event()

    def work(busy):
        """Everything once; what came out, and the addresses of what went in and is free again."""
        t = {n: x.to(DEV) for n, x in host.items()}
        codes = [torch.zeros(100, page, HK, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros(100, page, HK, D // 32, dtype=F16, device=DEV) for _ in range(2)]
        cache = pi.KvCache4(c, *codes, *scales, F16)
        attn = pi.Attn(c, cache, H, 1, N)
        o, qr, kr, kb, vb = (torch.zeros(T, n, D, dtype=F16, device=DEV) for n in (H, H, HK, HK, HK))
        o4 = torch.zeros(1, N, H, D, dtype=F16, device=DEV)
        torch.cuda.synchronize()
        if busy:
            with torch.cuda.stream(st):
                for _ in range(200):
                    torch.mm(a, a, out=b)
        pi.qk_norm_rope(c, t["q"], t["k"], t["pos"], t["freq"], qr, kr, q_norm=t["w"])
        pi.prompt_attention(c, prompt, t["q"], t["k"], t["v"], t["cu"], None, o)
        pi.kv_append(c, cache, t["k"][None], t["v"][None], t["table"], t["held"])
        pi.tree_attention(c, attn, t["q"][None, :N], t["k"][None, :N], t["v"][None, :N], None, t["table"], t["full"], o4)
        pi.kv_read(c, cache, t["table"], t["full"], t["rows"], kb, vb)
        done.record(st)
        lent = [*t.values(), *codes, *scales]
        return (o, qr, kr, o4, kb, vb), {x.data_ptr() for x in lent}, [(x.shape, x.dtype) for x in lent], attn

    want, *_ = work(False)
    torch.cuda.synchronize()
    got, lent, shapes, attn = work(True)
    new = [torch.full(s, 1, dtype=d, device=DEV) for s, d in shapes]
    still = not done.query()
    attn.cache = None  # the handle held the cache's tensors until here
    new += [torch.full(s, 1, dtype=d, device=DEV) for s, d in shapes]
    still = still and not done.query()
    assert still, "the stream was done before the memory could be reused"
    assert lent.isdisjoint(x.data_ptr() for x in new)
    st.synchronize()
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert torch.equal(w, o)
