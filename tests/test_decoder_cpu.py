"""The decoder operators' refusals that need no GPU: entry points without a context, and the
binding's checks of types, shapes and devices before anything reaches the library."""
import ctypes

import pytest
import torch

import activation_sparse_ffn_layer_amd as pi
from activation_sparse_ffn_layer_amd import _lib

F16, I32, I8 = torch.float16, torch.int32, torch.int8


class Ctx:
    """Stands in for a context of GPU 0: what gets past the binding's checks fails the test."""
    device, handle = 0, None
    stream = None

    def check(self, status):
        raise AssertionError("the library was called")


def made(cls, **fields):
    o = cls.__new__(cls)
    o.__dict__.update(ctx=Ctx(), handle=None, **fields)
    return o


@pytest.fixture
def cache():
    return made(pi.KvCache, k=None, v=None, dtype=F16, pages=4, page_tokens=16, heads=2, head_dim=64)


def test_entry_points_without_a_context():
    L, out = _lib.lib(), ctypes.c_void_p()
    bad = _lib.PI_ERR_INVALID
    assert L.pi_kv_create(None, None, ctypes.byref(out)) == bad
    assert L.pi_attn_create(None, None, 1, 1, 1, 1.0, ctypes.byref(out)) == bad
    assert L.pi_verifier_create(None, 1, 1, 1, ctypes.byref(out)) == bad
    assert L.pi_linear_create(None, None, ctypes.byref(out)) == bad
    assert L.pi_kv_append(None, None, None) == bad
    assert L.pi_tree_attention(None, None, None) == bad
    assert L.pi_verify(None, None, None) == bad
    assert L.pi_add_rmsnorm(None, None) == bad
    assert L.pi_linear_q8(None, None, None, 0, None, 1, None, 0, 0) == bad
    for destroy in (L.pi_kv_destroy, L.pi_attn_destroy, L.pi_verifier_destroy, L.pi_linear_destroy):
        destroy(None)


def refused(match, call, *args, **kw):
    with pytest.raises(pi.PiError, match=match):
        call(*args, **kw)


def test_cache_and_weight_tensors():
    k = torch.zeros(4, 16, 2, 64, dtype=F16)
    refused("fp16 or bf16", pi.KvCache, Ctx(), k.float(), k.float())
    refused("fp16 or bf16", pi.KvCache, Ctx(), k[0], k[0])
    refused("on cpu", pi.KvCache, Ctx(), k, k)
    refused("w must be", pi.Linear, Ctx(), torch.zeros(4, dtype=I8), torch.ones(4))
    refused("has type", pi.Linear, Ctx(), torch.zeros(4, 16), torch.ones(4))


def test_attention_and_append_arguments(cache):
    attn = made(pi.Attn, cache=cache, heads=4)
    q, kn = torch.zeros(2, 3, 4, 64, dtype=F16), torch.zeros(2, 3, 2, 64, dtype=F16)
    lens = torch.zeros(2, dtype=I32)
    run = lambda **o: pi.tree_attention(attn.ctx, attn, *[o.get(n, d) for n, d in  # noqa: E731
                                                          dict(q=q, k=kn, v=kn, tree=None, table=None, lens=lens, out=q).items()])
    refused("q must be", run, q=q[0])
    refused("q has type", run, q=q.float())
    refused("q has shape", run, q=q[:, :, :3])
    refused("q is on cpu", run)
    app = lambda **o: pi.kv_append(cache.ctx, cache, *[o.get(n, d) for n, d in dict(k=kn, v=kn, table=None, lens=lens).items()])  # noqa: E731
    refused("k_new must be", app, k=kn[0])
    refused("k_new has shape", app, k=kn[..., :32])
    refused("k_new is on cpu", app)


def test_verify_norm_and_product_arguments():
    ver = made(pi.Verifier, vocab=10)
    z, i, b = torch.zeros(2, 3, 10), torch.zeros(2, 3, dtype=I32), torch.zeros(2)
    args = [i, i, z[..., 0], b, i, i, torch.zeros(2, dtype=I32)]
    refused("logits must be", pi.verify, ver.ctx, ver, z[0], *args)
    refused("logits must be", pi.verify, ver.ctx, ver, z.double(), *args)
    refused("logits has shape", pi.verify, ver.ctx, ver, z[..., :9], *args)
    x, w = torch.zeros(2, 64, dtype=F16), torch.ones(64)
    refused("x must be", pi.add_rmsnorm, Ctx(), x[0], None, w, 1e-5, x)
    refused("x is on cpu", pi.add_rmsnorm, Ctx(), x, None, w, 1e-5, x)
    lin = made(pi.Linear, w=None, w_scale=None, bias=None, N=4, K=64)
    refused("x must be", pi.linear_q8, lin.ctx, lin, x[0], w, x)
    refused("x has type", pi.linear_q8, lin.ctx, lin, x, torch.ones(2), torch.zeros(2, 4))
    refused("x is on cpu", pi.linear_q8, lin.ctx, lin, x.to(I8), torch.ones(2), torch.zeros(2, 4))


def test_example_masks():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("draft_step", os.path.join(root, "examples", "draft_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert ex.ancestors(torch.tensor([[-1, 0, 0, 1]], dtype=I32)).tolist() == [[1, 3, 5, 11]]
    chain = ex.ancestors(torch.arange(-1, 63, dtype=I32)[None])
    assert chain[0, 63] == -1 and chain[0, 62] == (1 << 63) - 1
    q, s = ex.quantize_rows(torch.tensor([[1.0, -2.0], [0.0, 0.0]]))
    assert q.tolist() == [[64, -127], [0, 0]] and float(s[0]) == pytest.approx(2 / 127)


def test_strides_along_one_element_mean_nothing(cache):
    """A transposed and a plain view of one token: only their strides along the length-1 axis differ."""
    from activation_sparse_ffn_layer_amd import decoder

    plain, turned = torch.zeros(3, 1, 2, 64, dtype=F16), torch.zeros(3, 2, 1, 64, dtype=F16).transpose(1, 2)
    assert plain.shape == turned.shape and plain.stride() != turned.stride()
    for a, b in ((plain, turned), (turned, plain)):
        assert decoder._new_kv(cache, a, b, 3, 1, -1) == (a.data_ptr(), b.data_ptr(), a.stride())
    wide = torch.zeros(3, 1, 2, 128, dtype=F16)[..., :64]
    refused("equal strides", decoder._new_kv, cache, plain, wide, 3, 1, -1)


def test_sizes_past_32_bits_are_refused(cache):
    """Views of one row again and again, 2^32 and a few of them: the library would be told of a few."""
    many = (1 << 32) + 2
    here = Ctx()
    here.device = -1  # the CPU's tensors pass for those of the context's device
    x = torch.zeros(1, 64, dtype=F16).expand(many, 64)
    refused("below 2\\^31", pi.add_rmsnorm, here, x, None, torch.ones(64), 1e-5, x)
    lin = made(pi.Linear, w=None, w_scale=None, bias=None, N=4, K=64)
    x8, y = torch.zeros(1, 64, dtype=I8).expand(many, 64), torch.zeros(1, 4).expand(many, 4)
    refused("below 2\\^31", pi.linear_q8, here, lin, x8, torch.ones(1).expand(many), y)
    refused("below 2\\^31", pi.Linear, here, x8, torch.ones(1).expand(many))
    k = torch.zeros(1, 1, 2, 64, dtype=F16)
    refused("below 2\\^31", pi.KvCache, here, k.expand(many, 1, 2, 64), k.expand(many, 1, 2, 64))
    refused("below 2\\^31", pi.kv_append, here, cache, k.expand(1, many, 2, 64), k.expand(1, many, 2, 64), None,
            torch.zeros(1, dtype=I32))
    attn, q = made(pi.Attn, cache=cache, heads=2), k.expand(many, 1, 2, 64)
    refused("below 2\\^31", pi.tree_attention, here, attn, q, q, q, None, None, torch.zeros(1, dtype=I32).expand(many), q)
    ver, z, i = made(pi.Verifier, vocab=1), torch.zeros(1, 1, 1).expand(many, 1, 1), torch.zeros(1, 1, dtype=I32).expand(many, 1)
    refused("below 2\\^31", pi.verify, here, ver, z, i, i, z[..., 0], z[:, 0, 0], i, i, i[:, 0])
