"""Contexts and handles destroyed in any order."""
import pytest
import torch

from tests import test_gpu_decoder as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import activation_sparse_ffn_layer_amd as pi
    from synth import CONFIGS, make_layer

DEV, F16, I8, I32 = "cuda", torch.float16, torch.int8, torch.int32


def context():
    return pi.Context(max_batch=1, max_d=256, max_ffn=512, max_rank=64)


def handles(ctx):
    import dataclasses

    k = torch.zeros(4, 16, 2, 64, dtype=F16, device=DEV)
    cache = pi.KvCache(ctx, k, k.clone())
    cfg = dataclasses.replace(CONFIGS["opt6.7b"], d=256, ffn=512, rank=64)
    return dict(cache=cache, attn=pi.Attn(ctx, cache, 4, 2, 8), ver=pi.Verifier(ctx, 100, 2, 4),
                lin=pi.Linear(ctx, torch.zeros(4, 64, dtype=I8, device=DEV), torch.ones(4, device=DEV), max_tokens=4),
                ffn=pi.Ffn(ctx, make_layer(cfg, 0, device=DEV)))


@pytest.mark.parametrize("order", [["ctx", "cache", "attn", "ver", "lin", "ffn"], ["cache", "ctx", "ffn", "lin", "ver", "attn"],
                                   ["attn", "ver", "ctx", "cache", "ffn", "lin"]])
def test_any_order(order):
    for _ in range(3):
        ctx = context()
        h = dict(handles(ctx), ctx=ctx)
        for name in order:
            h[name].close()
        fresh = context()  # in the memory that was given back
        for name in order:
            h[name].close()
        fresh.close()


def test_attention_outlives_the_cache_handle():
    """The handle of the cache is gone and its memory another cache's; the tensors are still there."""
    ctx = context()
    g = torch.Generator().manual_seed(1)
    n, N, HK, H, D = 70, 3, 2, 4, 64
    k, v, table = base.make_cache(ctx, [n], n + N, HK, D, 16, F16, 2)
    q = torch.randn(1, N, H, D, generator=g).to(F16)
    kn, vn = (torch.randn(1, N, HK, D, generator=g).to(F16) for _ in range(2))
    cache = pi.KvCache(ctx, k.to(DEV), v.to(DEV))
    attn = pi.Attn(ctx, cache, H, 1, N)
    cache.close()
    small = torch.zeros(1, 1, 1, 8, dtype=F16, device=DEV)
    others = [pi.KvCache(ctx, small, small) for _ in range(8)]
    out = torch.full(q.shape, float("nan"), dtype=F16, device=DEV)
    pi.tree_attention(ctx, attn, q.to(DEV), kn.to(DEV), vn.to(DEV), None, table.to(DEV),
                      torch.tensor([n], dtype=I32, device=DEV), out)
    torch.cuda.synchronize()
    base.check_attention(out, q, k, v, kn, vn, base.sees_of([[-1, 0, 1]]), table, [n], D ** -0.5)
    assert len(others) == 8


def test_a_later_context_is_another_one():
    """Handles of a context that is gone are refused by every later one, at whatever address it lies."""
    ctx = context()
    h = handles(ctx)
    ctx.close()
    x, y = torch.zeros(2, 64, dtype=I8, device=DEV), torch.empty(2, 4, device=DEV)
    for _ in range(20):
        later = context()
        with pytest.raises(pi.PiError, match="another context"):
            pi.linear_q8(later, h["lin"], x, torch.ones(2, device=DEV), y)
        with pytest.raises(pi.PiError, match="another context"):
            pi.Attn(later, h["cache"], 4, 1, 1)
        later.close()
    with pytest.raises(pi.PiError):  # and by the closed one
        pi.linear_q8(ctx, h["lin"], x, torch.ones(2, device=DEV), y)
