"""Prompt attention by the kernels of large calls: eight waves a workgroup with rows of two tiles on their way, and keys
cut into parts at every padded head size. Tolerances as in the operator's other tests; references in 64 bits on the GPU.
"""
import pytest
import torch

from tests.test_gpu_prompts import BF16, DEV, F16, NAN, f, half_step, offsets, run_prompt

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


def inputs(seed, H, HK, D, dtype, seqs):
    g = torch.Generator(DEV).manual_seed(seed)
    cu_q, cu_k = offsets([n for n, _ in seqs]), offsets([n + h for n, h in seqs])
    q = (2 * torch.randn(cu_q[-1], H, D, generator=g, device=DEV)).to(dtype)
    k, v = (torch.randn(cu_k[-1], HK, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    return q, k, v, cu_q, cu_k


def check(out, q, k, v, cu_q, cu_k, scale):
    """Every row against the formula: the weights' rounding and the output's, scores, exponentials and sums in fp32."""
    H, D = q.shape[1:]
    G, u = H // k.shape[1], half_step(q.dtype)
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, m = rows.stop - rows.start, keys.stop - keys.start
        hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).triu(1 + m - n)
        for h in range(H):
            x, ks, vs = q[rows, h].double(), k[keys, h // G].double(), v[keys, h // G].double()
            s = (x @ ks.t().contiguous() * scale).masked_fill(hidden, -torch.inf)
            w = torch.softmax(s, 1)
            want, spread = w @ vs, w @ vs.abs()
            score = (x.abs() @ ks.abs().t().contiguous() * scale).masked_fill(hidden, 0).amax(1, keepdim=True)
            bound = (2 * u + 2 * (D + 4) * f * score + 2.0 ** -16) * spread + 1e-30
            err = (out[rows, h].double() - want).abs()
            assert (err <= bound).all(), f"sequence {b}, head {h}: off by {float((err / bound).max()):.2f} of the bound"


LARGE = [(1500, 600), (3, 0), (0, 70), (800, 0)]


# 2303 tokens: rows / 256 * kv heads fill 256 compute units, which takes the kernel of eight waves
@pytest.mark.parametrize("H,HK,D,dtype", [(32, 8, 64, F16), (32, 32, 64, BF16), (32, 8, 80, BF16), (64, 8, 96, F16), (32, 8, 128, F16),
                                          (40, 8, 128, BF16), (16, 16, 256, F16)])
def test_many_rows(ctx, H, HK, D, dtype):
    q, k, v, cu_q, cu_k = inputs(41, H, HK, D, dtype, LARGE)
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, D ** -0.5)
    check(out, q, k, v, cu_q, cu_k, D ** -0.5)
    # values and keys that only later queries see: an infinity, a NaN, a score that is NaN
    G = H // HK
    v[1000, 0, 5], v[1001, 0, 6], k[1900, 0, 3] = float("inf"), NAN, NAN
    odd = run_prompt(ctx, q, k, v, cu_q, cu_k, D ** -0.5)
    assert torch.equal(odd[:400], out[:400]) and torch.equal(odd[:, G:], out[:, G:]) and torch.equal(odd[1500:], out[1500:])
    assert (odd[400:1300, :G, 5] == float("inf")).all() and odd[401:1300, :G, 6].isnan().all()
    assert torch.equal(odd[400:1300, :G, :5], out[400:1300, :G, :5]) and torch.equal(odd[400:1300, :G, 7:], out[400:1300, :G, 7:])
    assert odd[1300:1500, :G].isnan().all()


@pytest.mark.parametrize("dtype,D", [(F16, 64), (BF16, 128)])
def test_many_rows_of_one_key_tile(ctx, dtype, D):
    """Workgroups whose keys are a single tile, with a later query's infinite value among them."""
    q, k, v, cu_q, cu_k = inputs(42, 64, 1, D, dtype, [(5, 0), (7, 20), (4, 60)] * 70)
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, 0.1)
    check(out[:16], q[:16], k, v, cu_q[:4], cu_k[:4], 0.1)
    check(out[-16:], q[-16:], k[-96:], v[-96:], cu_q[:4], cu_k[:4], 0.1)
    v[4, 0, 9] = float("-inf")  # the first sequence's last key
    odd = run_prompt(ctx, q, k, v, cu_q, cu_k, 0.1)
    assert (odd[4, :, 9] == float("-inf")).all()
    odd[4, :, 9] = out[4, :, 9]
    assert torch.equal(odd, out)


@pytest.mark.parametrize("D,dtype", [(8, F16), (40, BF16), (80, F16), (96, BF16), (128, F16), (128, BF16), (136, BF16), (256, F16)])
def test_keys_in_parts(ctx, D, dtype):
    """Few queries over many keys."""
    seqs = [(6, 2300), (33, 1700), (1, 4000), (0, 300)]
    q, k, v, cu_q, cu_k = inputs(43, 4, 2, D, dtype, seqs)
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, D ** -0.5)
    check(out, q, k, v, cu_q, cu_k, D ** -0.5)
    for _ in range(2):
        assert torch.equal(out, run_prompt(ctx, q, k, v, cu_q, cu_k, D ** -0.5))
    v[700, 1, 2] = float("inf")
    odd = run_prompt(ctx, q, k, v, cu_q, cu_k, D ** -0.5)
    assert not odd[:6, 2:, 2].isfinite().any()
    odd[:6, 2:, 2] = out[:6, 2:, 2]
    assert torch.equal(odd, out)


def test_one_query_among_many_empty_sequences(ctx):
    """Few rows of many sequences: each part of the keys is launched for every sequence's row tile, which may not pass
    the threads of a launch (35000 * 16 heads * 32 parts * 256). All rows of keys are one, repeated."""
    B, HK, D = 35000, 16, 8
    g = torch.Generator(DEV).manual_seed(44)
    q = torch.randn(1, HK, D, generator=g, device=DEV).to(F16)
    k, v = (torch.randn(1, HK, D, generator=g, device=DEV).to(F16).expand(B << 13, HK, D) for _ in range(2))
    prompt = pi.PromptAttn(ctx, HK, HK, D, F16, 1, B, 0.5)
    cu_q, cu_k = (torch.zeros(B + 1, dtype=torch.int32, device=DEV) for _ in range(2))
    cu_q[-1], cu_k[-1] = 1, 3000
    out = torch.full_like(q, NAN)
    pi.prompt_attention(ctx, prompt, q, k, v, cu_q, cu_k, out)
    torch.cuda.synchronize()
    # equal weights (fp16's largest power of two below 2^15 is exact) of equal values
    assert ((out.double() - v[:1].double()).abs() <= 2.0 ** -11 * v[:1].double().abs() + 3000 * f * v[:1].double().abs()).all()
