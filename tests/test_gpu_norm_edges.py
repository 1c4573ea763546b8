"""The norm's rows at the ends of fp32's range, and its 8-bit values next to a tie.

f = 2^-24 is half a step of fp32; values below its normal range are off by at most 2^-150 more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

DEV, F16, BF16, F32 = "cuda", torch.float16, torch.bfloat16, torch.float32
f = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


def run(ctx, x, w, eps):
    T, d = x.shape
    ro, y = torch.empty_like(x), torch.full((T, d), float("nan"), device=DEV)
    q, scale = torch.full((T, d), 99, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    pi.add_rmsnorm(ctx, x, None, w, eps, ro, q=q, scale=scale, y=y)
    torch.cuda.synchronize()
    return y, q, scale


def definition(x, w, eps):
    h = x.double()
    return h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def rounded(y, scale):
    """round(y / scale) of the fp32 values that the call gave, with fp32's rounding of the quotient."""
    return torch.round((y.double() / scale.double()[:, None]).float())


@pytest.mark.parametrize("eps", [0.0, 1e-31, 1e-36, 1e-42])
@pytest.mark.parametrize("d", [64, 4096, 20000])
def test_tiny_rows(ctx, d, eps):
    g = torch.Generator().manual_seed(d)
    x = torch.randn(7, d, generator=g)
    x[0] *= 1e-37
    x[1] *= 1e-38
    x[2] *= 1e-40  # below fp32's normal range
    x[3] = 0
    x[3, 3] = 1e-37  # one element
    x[4] = 0
    x[4, d - 1] = -(2.0 ** -149)
    x[5] *= 1e-15
    x[6] *= 1e-17
    x = x.to(DEV)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    y, q, scale = run(ctx, x, w, eps)
    want = definition(x, w, float(torch.tensor(eps, dtype=F32)))
    # as for ordinary rows (the sum of squares, half of it in the root, root, reciprocal and products)
    rel = (21 + 6) * f
    assert ((y.double() - want).abs() <= rel * want.abs() + 2.0 ** -150).all()
    top = want.abs().amax(1)
    assert ((scale.double() * 127 - top).abs() <= (rel + 2 * f) * top + 127 * 2.0 ** -150).all()
    keep = scale > 0
    assert (q[keep].float() == rounded(y, scale)[keep].clamp(-127, 127)).all() and (q[~keep] == 0).all()


@pytest.mark.parametrize("tiny", [1e-36, 1e-38, 1e-40])
def test_scales_below_the_normal_range(ctx, tiny):
    """Weights that leave the largest value's scale with few bits, or none: whole numbers within 127."""
    d = 512
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, d, generator=g).to(DEV)
    w = (tiny * (1 + torch.rand(d, generator=g))).to(DEV)
    y, q, scale = run(ctx, x, w, 1e-5)
    top = y.double().abs().amax(1)
    assert ((scale.double() - top / 127).abs() <= f * top / 127 + 2.0 ** -150).all()
    assert (q.float() == rounded(y, scale).clamp(-127, 127)).all()


def test_values_next_to_a_tie(ctx):
    """The quotient by the scale itself, not a product with its rounded reciprocal."""
    g = torch.Generator(DEV).manual_seed(6)
    x = torch.randn(1024, 4096, generator=g, device=DEV)
    y, q, scale = run(ctx, x, torch.ones(4096, device=DEV), 1e-5)
    assert torch.equal(q.float(), rounded(y, scale))
