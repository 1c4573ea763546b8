"""Verification at the ends of its arguments: temperatures without bound, numbers of 1, drafts that
all but equal the target."""
import pytest
import torch

from tests import test_gpu_decoder as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi

DEV, F16, BF16, F32, I32 = "cuda", torch.float16, torch.bfloat16, torch.float32, torch.int32
BIG = torch.finfo(F32).max


@pytest.fixture(scope="module")
def ctx():
    return pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)


@pytest.mark.parametrize("V,dtype", [(40, F16), (9001, F32), (70001, BF16)])
def test_infinite_temperature_is_uniform(ctx, V, dtype):
    """Every logit that is not -inf has the same weight; NaN counts as -inf, +inf as finite."""
    g = torch.Generator().manual_seed(V)
    B, N = 4, 3
    logits = (20 * torch.randn(B, N, V, generator=g)).to(dtype)
    logits[torch.rand(B, N, V, generator=g) < 0.3] = float("-inf")
    logits[:, :, 5] = float("nan")
    logits[:, :, 7] = float("inf")
    if dtype is not F16:
        logits[:, :, 8], logits[:, :, 9] = BIG / 1.01, -BIG / 1.01
    live = (logits > float("-inf")).double()
    tok = torch.full((B, N), 7, dtype=I32)
    tok[2, 1] = 5  # has no weight
    par = torch.tensor([[-1, 0, 1]] * B, dtype=I32)
    u = torch.zeros(B, N)
    for b in range(B):
        count = live[b].sum(1)
        u[b, 1], u[b, 2] = 0.99 / count[0], (1.01 if b % 2 else 0.99) / count[1]
    u[3, 1] = 1.01 / live[3, 0].sum()
    u_next = torch.tensor([0.0, 0.3, 0.71, 0.9999])
    nodes, out, n = base.run_verify(ctx, dict(logits=logits, tokens=tok, parents=par, u=u, u_next=u_next, q=None,
                                              temp=torch.full((B,), float("inf"))))
    assert n.tolist() == [3, 2, 1, 1]
    for b in range(B):
        p = live[b, int(n[b]) - 1].clone()
        if b in (1, 3):  # a child with weight was refused
            p[7] = 0
        p[5] = 0
        cum = p.cumsum(0)
        assert int(out[b, int(n[b]) - 1]) == int((cum <= float(u_next[b]) * cum[-1]).sum()), b


@pytest.mark.parametrize("with_q", [True, False])
def test_hot_rows_of_the_largest_logits(ctx, with_q):
    """Logits at both ends of fp32's range: their difference is beyond it, their weights are not."""
    B, N, V = 8, 4, 6000
    g = torch.Generator().manual_seed(2)
    logits = torch.where(torch.rand(B, N, V, generator=g) < 0.5, BIG, -BIG)
    logits[:, :, :4] = BIG
    q = torch.softmax(torch.randn(B, N, V, generator=g), 2) if with_q else None
    tok = torch.tensor([[0, 1, 2, 3]] * B, dtype=I32)
    par = torch.tensor([[-1, 0, 0, 1]] * B, dtype=I32)
    temp = torch.full((B,), 3e38)
    u = torch.rand(B, N, generator=g) * 2e-4
    for b in range(B):  # next to the first child's border, by 4%
        p = torch.softmax((logits[b, 0].double() - BIG) / float(temp[b]), 0)[1]
        u[b, 1] = (p if q is None else p / q[b, 0, 1]) * (0.96 if b % 2 else 1.04)
    c = dict(logits=logits, tokens=tok, parents=par, u=u, u_next=torch.rand(B, generator=g), q=q, temp=temp)
    base.check_verify(base.run_verify(ctx, c), c)


def test_numbers_of_one_take_nothing(ctx):
    """Without a q: no probability is above 1, and what is left of 1 after all refusals is nothing."""
    B, N, V = 256, 5, 50
    g = torch.Generator().manual_seed(4)
    logits = torch.full((B, N, V), float("-inf"))
    logits[:, :, :3] = torch.randn(B, N, 3, generator=g)
    tok = torch.tensor([[0, 0, 1, 2, 9]] * B, dtype=I32)  # the fourth child's token has no weight
    par = torch.tensor([[-1, 0, 0, 0, 0]] * B, dtype=I32)
    c = dict(logits=logits, tokens=tok, parents=par, u=torch.ones(B, N), u_next=torch.rand(B, generator=g), q=None, temp=None)
    nodes, out, n = base.run_verify(ctx, c)
    assert n.tolist() == [1] * B and (nodes[:, 1:] == -1).all()
    assert ((out[:, 0] >= 0) & (out[:, 0] < 3)).all()


@pytest.mark.parametrize("V,N", [(3000, 2), (5000, 12), (66001, 3)])
def test_draft_that_all_but_equals_the_target(ctx, V, N):
    """q is p rounded to fp32, but for the first child's token: what is left after its refusal are the
    roundings, which only a sum in 64 bits tells apart."""
    B = 16
    g = torch.Generator().manual_seed(V)
    logits = torch.randn(B, N, V, generator=g)
    q = torch.softmax(logits.double(), 2).float()
    tok = torch.randint(0, V, (B, N), generator=g, dtype=I32)
    par = torch.zeros(B, N, dtype=I32)
    par[:, 0] = -1
    for b in range(B):
        q[b, 0, int(tok[b, 1])] *= 1.05
        tok[b, 2:] = tok[b, 1]
    c = dict(logits=logits, tokens=tok, parents=par, u=torch.full((B, N), 0.999), u_next=torch.rand(B, generator=g), q=q,
             temp=None)
    base.check_verify(base.run_verify(ctx, c), c)
