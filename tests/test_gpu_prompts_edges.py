"""Edges of the prompt and 4-bit cache operators: strides past 32 bits, split keys with infinities, handles that outlive
their context's other users, a stream that is not the tensors'."""
import pytest
import torch

from tests import prompt_ref as ref
from tests.test_gpu_decoder import words_of
from tests.test_gpu_prompts import BF16, DEV, F16, I32, NAN, check_prompt, ints, make_cache4, offsets, run_attention4, run_prompt

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


@pytest.mark.parametrize("page,N,G", [(16, 1, 2), (5, 2, 1), (16, 20, 4)])
def test_cache4_past_32_bits(ctx, page, N, G):
    """Pages whose codes lie 2^32 bytes apart and scales 2^31 elements: the same results as pages side by side."""
    HK, D, n = 1, 64, 2 * page - 1
    g = torch.Generator().manual_seed(21)
    parts, table = make_cache4([n], 4 * page, HK, D, page, 22, junk=False)
    table = torch.tensor([[1, 3, 0, 2]], dtype=I32)
    far = []
    for i, t in enumerate(parts):
        stride = (1 << 32) // 2 if i % 2 == 0 else 1 << 30  # page 3 starts beyond 2^32 bytes and 2^31 elements
        buf = torch.zeros(3 * stride + t[0].numel(), dtype=t.dtype, device=DEV)
        v = buf.as_strided(t.shape, (stride, HK * t.shape[3], t.shape[3], 1))
        v.copy_(t)
        far.append(v)
    q = torch.randn(1, N, HK * G, D, generator=g).to(F16)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(F16) for _ in range(2))
    want = run_attention4(ctx, q, parts, kn, vn, None, table, [n], 0.125)
    cache = pi.KvCache4(ctx, far[0], far[2], far[1], far[3], F16)
    attn = pi.Attn(ctx, cache, HK * G, 1, N, 0.125)
    out = torch.full(q.shape, NAN, dtype=F16, device=DEV)
    tab, held = table.to(DEV), ints([n])
    pi.tree_attention(ctx, attn, q.to(DEV), kn.to(DEV), vn.to(DEV), None, tab, held, out)
    now = torch.empty_like(held)
    pi.kv_append(ctx, cache, kn.to(DEV), vn.to(DEV), tab, held, now)
    ko, vo = (torch.empty(n + N, HK, D, dtype=F16, device=DEV) for _ in range(2))
    pi.kv_read(ctx, cache, tab, now, ints([0, n + N]), ko, vo)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for o, (c, s), new in ((ko, parts[:2], kn), (vo, parts[2:], vn)):
        rows = [ref.values(c, s)[int(table[0, p // page]), p % page] for p in range(n)]
        rows += list(ref.values(*ref.quantize(new[0])))
        assert torch.equal(torch.stack(rows).to(F16), o.cpu())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_split_keys_and_odd_values(ctx, dtype):
    """Few queries over many keys, whose keys are cut: unseen infinities stay out, seen ones stay."""
    g = torch.Generator().manual_seed(23)
    cu_q, cu_k = offsets([6, 3]), offsets([2300, 1700])
    q = torch.randn(9, 4, 64, generator=g).to(dtype)
    k, v = (torch.randn(4000, 2, 64, generator=g).to(dtype) for _ in range(2))
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, 0.125)
    check_prompt(out, q, k, v, cu_q, cu_k, 0.125)
    v[2298, 0, 5], k[2299, :, 1], v[100, 1, 9], v[3000, 1, 2] = float("inf"), NAN, float("-inf"), NAN
    odd = run_prompt(ctx, q, k, v, cu_q, cu_k, 0.125).cpu()
    out = out.cpu()
    assert torch.equal(odd[:4, :2], out[:4, :2])                       # before position 2298
    assert (odd[4, :2, 5] == float("inf")).all() and torch.equal(odd[4, :2, :5], out[4, :2, :5])
    assert odd[5].isnan().all()                                        # a score that is NaN
    assert not odd[:5, 2:, 9].isfinite().any() and torch.equal(odd[:5, 2:, :9], out[:5, 2:, :9])
    assert odd[6:, 2:, 2].isnan().all() and torch.equal(odd[6:, :2], out[6:, :2])


def test_prompts_on_another_stream():
    """The context's stream is not the one that the tensors are made on: their memory is kept until it is done."""
    st = torch.cuda.Stream()
    c = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0, stream=st)
    g = torch.Generator().manual_seed(24)
    q, k, v = (torch.randn(50, n, 64, generator=g).to(F16) for n in (4, 2, 2))
    p = pi.PromptAttn(c, 4, 2, 64, F16, 50, 1)
    for _ in range(3):
        dq, dk, dv, cu = q.to(DEV), k.to(DEV), v.to(DEV), ints([0, 50])
        out = torch.empty_like(dq)
        torch.cuda.synchronize()
        pi.prompt_attention(c, p, dq, dk, dv, cu, None, out)
        del dq, dk, dv, cu
        torch.full((50, 8, 64), NAN, dtype=F16, device=DEV)  # may take the freed memory only once the stream is done
    st.synchronize()
    torch.cuda.synchronize()
    check_prompt(out, q, k, v, [0, 50], [0, 50], 0.125)


def test_handles_outlive_the_context():
    c = pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)
    k, s = torch.zeros(1, 16, 1, 32, dtype=torch.uint8, device=DEV), torch.zeros(1, 16, 1, 2, dtype=F16, device=DEV)
    cache = pi.KvCache4(c, k, k, s, s, F16)
    attn, prompt = pi.Attn(c, cache, 2, 1, 4), pi.PromptAttn(c, 2, 1, 64, F16, 100, 1)
    c.close()
    for h in (cache, attn, prompt):
        h.close()


def test_tree_words_over_4_bits_see_only_their_nodes(ctx):
    """All 64 nodes, each seeing itself alone over an empty cache: the weights are 1."""
    N, D = 64, 64
    g = torch.Generator().manual_seed(25)
    parts, table = make_cache4([0], N, 1, D, 16, 26)
    q, kn, vn = (torch.randn(1, N, n, D, generator=g).to(F16) for n in (2, 1, 1))
    out = run_attention4(ctx, q, parts, kn, vn, words_of(torch.eye(N, dtype=torch.bool)[None]), table, [0], 0.125)
    assert torch.equal(out.cpu(), vn.expand(1, N, 2, D))
