"""Refusals of the prompt and 4-bit cache operators that need no GPU, and the plain statements they are tested against."""
import ctypes

import torch

import activation_sparse_ffn_layer_amd as pi
from activation_sparse_ffn_layer_amd import _lib
from tests import prompt_ref as ref
from tests.test_decoder_cpu import F16, I32, Ctx, made, refused

U8, BF16 = torch.uint8, torch.bfloat16


def test_entry_points_without_a_context():
    L, out, bad = _lib.lib(), ctypes.c_void_p(), _lib.PI_ERR_INVALID
    assert L.pi_kv4_create(None, None, ctypes.byref(out)) == bad
    assert L.pi_kv_read(None, None, None) == bad
    assert L.pi_prompt_create(None, 1, 1, 1, 64, 1, 1, 1.0, ctypes.byref(out)) == bad
    assert L.pi_prompt_attention(None, None, None) == bad
    assert L.pi_qk_norm_rope(None, None) == bad
    L.pi_prompt_destroy(None)


def test_cache_tensors_of_4_bits():
    k, s = torch.zeros(2, 16, 2, 32, dtype=U8), torch.zeros(2, 16, 2, 2, dtype=F16)
    refused("need fp16 or bf16", pi.KvCache4, Ctx(), k, k, s, s, torch.float32)
    refused("k must be", pi.KvCache4, Ctx(), k[0], k, s, s)
    refused("k must be", pi.KvCache4, Ctx(), k[..., :24], k, s, s)
    refused("k must be", pi.KvCache4, Ctx(), k.to(F16), k, s, s)
    refused("on cpu", pi.KvCache4, Ctx(), k, k, s, s)


def test_read_prompt_and_rope_arguments():
    cache = made(pi.KvCache4, k=None, v=None, dtype=F16, pages=4, page_tokens=16, heads=2, head_dim=64)
    o, lens, cu = torch.zeros(3, 2, 64, dtype=F16), torch.zeros(1, dtype=I32), torch.zeros(2, dtype=I32)
    refused("k_out must be", pi.kv_read, cache.ctx, cache, None, lens, cu, o[0], o)
    refused("k_out has shape", pi.kv_read, cache.ctx, cache, None, lens, cu, o[..., :32], o)
    refused("k_out has type", pi.kv_read, cache.ctx, cache, None, lens, cu, o.float(), o)
    refused("k_out is on cpu", pi.kv_read, cache.ctx, cache, None, lens, cu, o, o)
    refused("need fp16 or bf16", pi.PromptAttn, Ctx(), 4, 2, 64, torch.float32, 8, 1)
    pr = made(pi.PromptAttn, heads=4, kv_heads=2, head_dim=64, dtype=F16)
    q = torch.zeros(3, 4, 64, dtype=F16)
    refused("q and k must be", pi.prompt_attention, pr.ctx, pr, q[0], o, o, cu, None, q)
    refused("q has shape", pi.prompt_attention, pr.ctx, pr, q[:, :2], o, o, cu, None, q)
    refused("q is on cpu", pi.prompt_attention, pr.ctx, pr, q, o, o, cu, None, q)
    pos, freq = torch.zeros(3, dtype=I32), torch.zeros(32)
    refused("q and k must be", pi.qk_norm_rope, Ctx(), None, None, pos, freq, None, None)
    refused("q and k must be", pi.qk_norm_rope, Ctx(), q.long(), None, pos, freq, q, None)
    refused("q is on cpu", pi.qk_norm_rope, Ctx(), q, None, pos, freq, q, None)


def test_plain_quantiser_by_hand():
    x = torch.zeros(1, 64)
    x[0, :3] = torch.tensor([4.0, -4.0, 1.0])  # two alike: m = 4, scale -0.5
    x[0, 32:35] = torch.tensor([-8.0, 7.0, 0.5])  # m = -8, scale 1; 0.5 ties to 0
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[-0.5, 1.0]]
    v = ref.values(codes, scales)[0]
    assert v[:3].tolist() == [4.0, -3.5, 1.0] and v[32:35].tolist() == [-8.0, 7.0, 0.0]
    assert int(codes[0, 0]) == 0 + 16 * 8 and int(codes[0, 1]) == 15 + 16 * 8
    x[0, 5], x[0, 40] = float("nan"), float("inf")
    assert ref.values(*ref.quantize(x)).isnan().all()


def test_plain_rotation_by_hand():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0]]])
    quarter = torch.tensor([torch.pi / 2, 0.0])
    out, _ = ref.rope(x, None, torch.ones(1, dtype=I32), quarter, 0.0, False)
    assert torch.allclose(out[0, 0], torch.tensor([-3.0, 2.0, 1.0, 4.0], dtype=torch.float64), atol=1e-6)
    out, _ = ref.rope(x, None, torch.ones(1, dtype=I32), quarter, 0.0, True)
    assert torch.allclose(out[0, 0], torch.tensor([-2.0, 1.0, 3.0, 4.0], dtype=torch.float64), atol=1e-6)
