"""Attention of values near the end of bf16's range: a mean of values is no larger than the largest of them, so that its
parts may not leave fp32 on the way. Tolerances are those of the operators' other tests, relative to the values."""
import math
import random

import pytest
import torch

from tests.test_gpu_decoder import make_cache, run_attention, sees_of, trees, words_of
from tests.test_gpu_prompts import BF16, check_attention4, check_prompt, make_cache4, offsets, run_attention4, run_prompt

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

MAX = torch.finfo(BF16).max


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


def far_values(g, *shape):
    """bf16 values of either sign up to the largest one, a quarter of them the largest itself."""
    x = (2 * torch.rand(*shape, generator=g) - 1) * MAX
    return torch.where(torch.rand(*shape, generator=g) < 0.25, MAX, x).to(BF16)


@pytest.mark.parametrize("B,N,G,D,lens", [
    (1, 1, 1, 64, [0]),
    (2, 3, 2, 96, [40, 0]),             # rows of a few waves
    (1, 28, 1, 128, [300]),
    (1, 30, 2, 128, [0]),               # a row tile of four waves
    (2, 64, 4, 64, [5, 200]),           # of eight
    (1, 64, 1, 256, [130]),
])
def test_new_values_over_4_bits(ctx, B, N, G, D, lens):
    HK = 2
    g = torch.Generator().manual_seed(31)
    parts, table = make_cache4(lens, max(lens) + N, HK, D, 16, 32, dtype=BF16)
    q = torch.randn(B, N, HK * G, D, generator=g).to(BF16)
    kn = torch.randn(B, N, HK, D, generator=g).to(BF16)
    vn = far_values(g, B, N, HK, D)
    sees = sees_of(trees(random.Random(5), B, N, 3))
    out = run_attention4(ctx, q, parts, kn, vn, words_of(sees), table, lens, D ** -0.5)
    check_attention4(out, q, parts, kn, vn, sees, table, lens, D ** -0.5)


@pytest.mark.parametrize("N,G", [(32, 1), (64, 1), (64, 8)])
def test_the_largest_value_of_every_new_node_over_4_bits(ctx, N, G):
    """Equal weights and equal values: the value itself."""
    D = 64
    parts, table = make_cache4([0], N, 1, D, 16, 33)
    q = torch.zeros(1, N, G, D, dtype=BF16)
    vn = torch.full((1, N, 1, D), MAX, dtype=BF16)
    out = run_attention4(ctx, q, parts, vn, vn, None, table, [0], 1.0)
    assert (out == MAX).all()


@pytest.mark.parametrize("H,HK,D,seqs", [
    (4, 2, 64, [(70, 0), (1, 100)]),
    (2, 2, 256, [(65, 30)]),
    (8, 2, 128, [(9, 2500)]),           # keys cut into parts
    (1, 1, 40, [(3, 0), (200, 7)]),
])
def test_prompt_values(ctx, H, HK, D, seqs):
    g = torch.Generator().manual_seed(34)
    cu_q, cu_k = offsets([n for n, _ in seqs]), offsets([n + h for n, h in seqs])
    q = torch.randn(cu_q[-1], H, D, generator=g).to(BF16)
    k, v = torch.randn(cu_k[-1], HK, D, generator=g).to(BF16), far_values(g, cu_k[-1], HK, D)
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, D ** -0.5)
    check_prompt(out, q, k, v, cu_q, cu_k, D ** -0.5)


@pytest.mark.parametrize("n,held", [(130, 0), (2, 4000)])
def test_the_largest_value_of_every_key_of_a_prompt(ctx, n, held):
    """Equal weights and equal values: the value itself."""
    q = torch.zeros(n, 2, 64, dtype=BF16)
    v = torch.full((n + held, 1, 64), MAX, dtype=BF16)
    assert (run_prompt(ctx, q, v, v, [0, n], [0, n + held], 1.0) == MAX).all()


def test_scales_whose_logarithm_leaves_the_range(ctx):
    """The kernels use scale times log2(e): up to 2^127 it is a number, and keys of zeros weigh alike."""
    parts, table = make_cache4([20], 22, 1, 64, 16, 35)
    plain = pi.KvCache(ctx, *[torch.zeros(2, 16, 1, 64, dtype=BF16, device="cuda")] * 2)
    codes, scales = (torch.zeros(2, 16, 1, n, dtype=t, device="cuda") for n, t in ((32, torch.uint8), (2, torch.float16)))
    for scale in (2.9e38, 1.71e38):
        with pytest.raises(pi.PiError, match="scale"):
            pi.PromptAttn(ctx, 2, 1, 64, BF16, 8, 1, scale)
        for cache in (plain, pi.KvCache4(ctx, codes, codes, scales, scales, BF16)):
            with pytest.raises(pi.PiError, match="scale"):
                pi.Attn(ctx, cache, 2, 1, 1, scale)
    g = torch.Generator().manual_seed(36)
    q, v = torch.randn(9, 2, 64, generator=g).to(BF16), torch.randn(9, 1, 64, generator=g).to(BF16)
    k = torch.zeros_like(v)
    check_prompt(run_prompt(ctx, q, k, v, [0, 9], None, 2.0 ** 127), q, k, v, [0, 9], [0, 9], 2.0 ** 127)
    parts[1].zero_()  # keys: their scales
    kn, vn, sees = (t[None, :2] for t in (k, v, torch.ones(2, 2, dtype=torch.bool).tril()))
    out = run_attention4(ctx, q[None, :2], parts, kn, vn, None, table, [20], 2.0 ** 127)
    check_attention4(out, q[None, :2], parts, kn, vn, sees, table, [20], 2.0 ** 127)


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
@pytest.mark.parametrize("n,held", [(300, 0), (40, 3000)])
def test_unlike_weights_of_the_largest_value(ctx, dtype, n, held):
    """Values that are all the largest one have it as their mean: the weights' rounding may take half a step off it, not
    past it."""
    top = torch.finfo(dtype).max
    g = torch.Generator().manual_seed(37)
    q, k = torch.randn(n, 4, 64, generator=g).to(dtype), torch.randn(n + held, 2, 64, generator=g).to(dtype)
    v = torch.full_like(k, top)
    v[:, 1] = -top
    cu_q, cu_k = [0, n], [0, n + held]
    out = run_prompt(ctx, q, k, v, cu_q, cu_k, 0.3)
    assert out.isfinite().all()
    check_prompt(out, q, k, v, cu_q, cu_k, 0.3)


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
@pytest.mark.parametrize("N,G,lens", [(20, 1, [0, 0]), (64, 2, [0, 0]), (64, 8, [0, 0])])
def test_unlike_weights_of_the_largest_new_value_over_4_bits(ctx, dtype, N, G, lens):
    D, B = 64, len(lens)
    g = torch.Generator().manual_seed(38)
    parts, table = make_cache4(lens, N, 2, D, 16, 39, dtype=dtype)
    q, kn = torch.randn(B, N, 2 * G, D, generator=g).to(dtype), torch.randn(B, N, 2, D, generator=g).to(dtype)
    vn = torch.full_like(kn, torch.finfo(dtype).max)
    vn[:, :, 1] *= -1
    sees = sees_of(trees(random.Random(5), B, N, 0))
    out = run_attention4(ctx, q, parts, kn, vn, None, table, lens, 0.3)
    assert out.isfinite().all()
    check_attention4(out, q, parts, kn, vn, sees, table, lens, 0.3)


def rounded_up(dtype):
    """A scale at which a score of -1 weighs a little over half of a step above 0.5, so that the type rounds it up: by
    nearly a relative 2^-11 in fp16 and 2^-8 in bf16. The largest number is half of that away from an infinity."""
    step = torch.finfo(dtype).eps  # of numbers from 1 to 2
    return -math.log(0.5 * (1 + 0.55 * step))


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
@pytest.mark.parametrize("held", [199, 3999])
def test_weights_rounded_up_of_the_largest_value(ctx, dtype, held):
    """One key of weight 1 and many of a weight that is rounded up, all of the largest value."""
    k = torch.zeros(1 + held, 1, 64, dtype=dtype)
    k[1:, :, 0] = -1
    q, v = torch.zeros(1, 2, 64, dtype=dtype), torch.full_like(k, torch.finfo(dtype).max)
    q[:, :, 0] = 1
    out = run_prompt(ctx, q, k, v, [0, 1], [0, 1 + held], rounded_up(dtype))
    assert (out == torch.finfo(dtype).max).all()


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
@pytest.mark.parametrize("N,G", [(32, 1), (64, 2), (64, 8)])
def test_weights_rounded_up_of_the_largest_new_value_over_4_bits(ctx, dtype, N, G):
    parts, table = make_cache4([0], N, 1, 64, 16, 40, dtype=dtype)
    kn, q = torch.zeros(1, N, 1, 64, dtype=dtype), torch.zeros(1, N, G, 64, dtype=dtype)
    kn[:, 1:, :, 0], q[..., 0] = -1, 1
    vn = torch.full_like(kn, -torch.finfo(dtype).max)
    out = run_attention4(ctx, q, parts, kn, vn, None, table, [0], rounded_up(dtype))
    assert (out == -torch.finfo(dtype).max).all()


@pytest.mark.parametrize("N,G,n", [(32, 1, 0), (64, 2, 0), (64, 8, 0), (1, 1, 2000)])
def test_weights_rounded_up_of_the_largest_value_over_a_plain_cache(ctx, N, G, n):
    dtype = torch.float16
    k, v, table = make_cache(ctx, [n], n + N, 1, 64, 16, dtype, 41)
    k.zero_()
    k[..., 0] = -1
    kn, q = torch.zeros(1, N, 1, 64, dtype=dtype), torch.zeros(1, N, G, 64, dtype=dtype)
    kn[:, 1:, :, 0], q[..., 0] = -1, 1
    v, vn = (torch.full_like(t, torch.finfo(dtype).max) for t in (v, kn))
    out = run_attention(ctx, q, k, v, kn, vn, None, table, [n], rounded_up(dtype))
    assert (out == torch.finfo(dtype).max).all()
