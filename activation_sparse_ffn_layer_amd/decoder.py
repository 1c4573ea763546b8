"""The decoder operators around the sparse FFN, over the C ABI of include/pi.h.

:class:`KvCache`, :class:`Attn`, :class:`Verifier` and :class:`Linear` wrap the handles;
:func:`kv_append`, :func:`tree_attention`, :func:`verify`, :func:`add_rmsnorm` and
:func:`linear_q8` enqueue the operators on the context's stream. Tensors may be views as long
as their last axis is contiguous. Shapes, types and devices are checked here (:class:`PiError`
with the status of an invalid argument), everything else in the library.
"""
from __future__ import annotations

import ctypes
from ctypes import c_void_p
from typing import Optional

import torch

from ._lib import (DTYPE, PI_ERR_INVALID, AppendArgs, AttnArgs, KvDesc, LinearDesc, NormArgs, PiError, VerifyArgs,
                   lib)

I8, I32, I64, F32 = torch.int8, torch.int32, torch.int64, torch.float32


def _bad(msg: str):
    raise PiError(PI_ERR_INVALID, msg)


def _refuse(t, name: str, dtype, shape, device: int):
    """Say what is wrong with a tensor that did not pass."""
    if not isinstance(t, torch.Tensor):
        _bad(f"{name} is no tensor")
    if t.dtype is not dtype:
        _bad(f"{name} has type {t.dtype}, need {dtype}")
    if t.shape != shape:
        _bad(f"{name} has shape {tuple(t.shape)}, need {tuple(shape)}")
    if t.get_device() != device:
        _bad(f"{name} is on {t.device}, need GPU {device}")
    _bad(f"{name} must be contiguous")


# The calls are short next to their checks' cost on the host: the checks that pass are one expression.

def _dense(t, name: str, dtype, shape, device: int) -> int:
    """Device pointer of a contiguous tensor of this type and shape."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, device)


def _opt(t, name: str, dtype, shape, device: int) -> Optional[int]:
    return None if t is None else _dense(t, name, dtype, shape, device)


def _view(t, name: str, dtype, shape, device: int):
    """Device pointer and strides of a tensor whose last axis is contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device:
        s = t.stride()
        if s[-1] != 1 and shape[-1] != 1:
            _bad(f"{name}: the last axis must be contiguous")
        return t.data_ptr(), s
    _refuse(t, name, dtype, shape, device)


def _sizes(t, name: str):
    """The library takes sizes in 32 bits, to which ctypes would cut larger ones without a word."""
    if max(t.shape) > 0x7FFFFFFF:
        _bad(f"{name}: sizes are below 2^31, got {tuple(t.shape)}")
    return t.shape


def _common(sa, sb, shape, names: str):
    """Strides that two tensors of this shape share: a stride along one element means nothing."""
    if sa != sb and any(a != b and n != 1 for a, b, n in zip(sa, sb, shape)):
        _bad(f"{names} need equal strides")
    return sa


def _borrow(ctx, *tensors):
    """Keep the tensors' memory from reuse until the context's stream is done with them, where
    that is not the stream they are used on otherwise."""
    s = ctx.stream
    if torch._C._cuda_getCurrentRawStream(ctx.device) != s.cuda_stream:
        for t in tensors:
            if t is not None:
                t.record_stream(s)


class _Handle:
    _destroy = ""

    def close(self):
        if getattr(self, "handle", None):
            getattr(lib(), self._destroy)(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KvCache(_Handle):
    """A pi_kv: a layer's key/value cache over borrowed tensors ``k`` and ``v``
    [pages][page_tokens][heads][head_dim] (fp16 or bf16, equal strides)."""

    _destroy = "pi_kv_destroy"

    def __init__(self, ctx, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4 or k.dtype not in (torch.float16, torch.bfloat16):
            _bad("k must be an fp16 or bf16 tensor [pages][page_tokens][heads][head_dim]")
        pk, sk = _view(k, "k", k.dtype, _sizes(k, "k"), ctx.device)
        pv, sv = _view(v, "v", k.dtype, k.shape, ctx.device)
        sk = _common(sk, sv, k.shape, "k and v")
        self.ctx, self.k, self.v, self.dtype = ctx, k, v, k.dtype
        self.pages, self.page_tokens, self.heads, self.head_dim = k.shape
        desc = KvDesc(DTYPE[k.dtype], self.heads, self.head_dim, self.pages, self.page_tokens, pk, pv, sk[0], sk[1], sk[2])
        h = c_void_p()
        ctx.check(lib().pi_kv_create(ctx.handle, ctypes.byref(desc), ctypes.byref(h)))
        self.handle = h


def _table(table, B: int, device: int):
    if table is None:
        return None, 0, 0
    if table.dim() != 2 or table.shape[0] != B:
        _bad(f"table has shape {tuple(table.shape)}, need [{B}][pages of a sequence]")
    p, s = _view(table, "table", I32, _sizes(table, "table"), device)
    return p, s[0], table.shape[1]


def _new_kv(cache: KvCache, k_new, v_new, B: int, N: int, device: int):
    shape = (B, N, cache.heads, cache.head_dim)
    pk, sk = _view(k_new, "k_new", cache.dtype, shape, device)
    pv, sv = _view(v_new, "v_new", cache.dtype, shape, device)
    return pk, pv, _common(sk, sv, shape, "k_new and v_new")


def kv_append(ctx, cache: KvCache, k_new: torch.Tensor, v_new: torch.Tensor, table: Optional[torch.Tensor],
              ctx_len: torch.Tensor, len_out: Optional[torch.Tensor] = None, nodes: Optional[torch.Tensor] = None,
              n: Optional[torch.Tensor] = None):
    """pi_kv_append: tokens ``nodes[b][:n[b]]`` of ``k_new``/``v_new`` [B][N][heads][head_dim] (all N
    without them) to the positions from ``ctx_len[b]`` on; ``len_out`` gets the new lengths."""
    if k_new.dim() != 4:
        _bad("k_new must be [B][N][heads][head_dim]")
    dev, (B, N) = ctx.device, _sizes(k_new, "k_new")[:2]
    pk, pv, s = _new_kv(cache, k_new, v_new, B, N, dev)
    pt, ts, tw = _table(table, B, dev)
    a = AppendArgs(pk, pv, s[0], s[1], s[2], pt, ts, tw, _dense(ctx_len, "ctx_len", I32, (B,), dev),
                   _opt(nodes, "nodes", I32, (B, N), dev), _opt(n, "n", I32, (B,), dev),
                   _opt(len_out, "len_out", I32, (B,), dev), B, N)
    _borrow(ctx, k_new, v_new, table, ctx_len, len_out, nodes, n, cache.k, cache.v)
    ctx.check(lib().pi_kv_append(ctx.handle, cache.handle, ctypes.byref(a)))


class Attn(_Handle):
    """A pi_attn: tree attention of ``heads`` query heads over a cache, with its scratch for up to
    ``max_batch`` sequences of ``max_nodes`` new nodes. ``scale`` defaults to head_dim ** -0.5."""

    _destroy = "pi_attn_destroy"

    def __init__(self, ctx, cache: KvCache, heads: int, max_batch: int, max_nodes: int, scale: Optional[float] = None):
        self.ctx, self.cache, self.heads = ctx, cache, heads
        scale = cache.head_dim ** -0.5 if scale is None else scale
        h = c_void_p()
        ctx.check(lib().pi_attn_create(ctx.handle, cache.handle, heads, max_batch, max_nodes, scale, ctypes.byref(h)))
        self.handle = h


def tree_attention(ctx, attn: Attn, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   tree: Optional[torch.Tensor], table: Optional[torch.Tensor], ctx_len: torch.Tensor,
                   out: torch.Tensor):
    """pi_tree_attention: ``out`` [B][N][heads][head_dim] from ``q`` over the cached positions below
    ``ctx_len`` and the new nodes that ``tree`` (int64 words [B][N], None: a chain) lets a node see."""
    cache = attn.cache
    if q.dim() != 4:
        _bad("q must be [B][N][heads][head_dim]")
    dev, (B, N) = ctx.device, _sizes(q, "q")[:2]
    shape = (B, N, attn.heads, cache.head_dim)
    pq, sq = _view(q, "q", cache.dtype, shape, dev)
    po, so = _view(out, "out", cache.dtype, shape, dev)
    pk, pv, s = _new_kv(cache, k_new, v_new, B, N, dev)
    pt, ts, tw = _table(table, B, dev)
    a = AttnArgs(pq, sq[0], sq[1], sq[2], pk, pv, s[0], s[1], s[2], _opt(tree, "tree", I64, (B, N), dev), pt, ts, tw,
                 _dense(ctx_len, "ctx_len", I32, (B,), dev), po, so[0], so[1], so[2], B, N)
    _borrow(ctx, q, k_new, v_new, tree, table, ctx_len, out, cache.k, cache.v)
    ctx.check(lib().pi_tree_attention(ctx.handle, attn.handle, ctypes.byref(a)))


class Verifier(_Handle):
    """A pi_verifier: scratch to check drafted tokens over ``vocab`` logits."""

    _destroy = "pi_verifier_destroy"

    def __init__(self, ctx, vocab: int, max_batch: int, max_nodes: int):
        self.ctx, self.vocab = ctx, vocab
        h = c_void_p()
        ctx.check(lib().pi_verifier_create(ctx.handle, vocab, max_batch, max_nodes, ctypes.byref(h)))
        self.handle = h


def verify(ctx, ver: Verifier, logits: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, u: torch.Tensor,
           u_next: torch.Tensor, nodes: torch.Tensor, out: torch.Tensor, n: torch.Tensor,
           q: Optional[torch.Tensor] = None, temperature: Optional[torch.Tensor] = None):
    """pi_verify: the accepted path of every tree (``nodes``), its tokens with the next one
    (``out``) and its length (``n``), from the target's ``logits`` [B][N][vocab] and, optionally,
    the draft's probabilities ``q`` (fp32, alike)."""
    if logits.dim() != 3 or logits.dtype not in DTYPE:
        _bad("logits must be a floating-point tensor [B][N][vocab]")
    dev, (B, N) = ctx.device, _sizes(logits, "logits")[:2]
    shape = (B, N, ver.vocab)
    pl, sl = _view(logits, "logits", logits.dtype, shape, dev)
    pq, sq = (None, (0, 0)) if q is None else _view(q, "q", F32, shape, dev)
    bn, b = (B, N), (B,)
    a = VerifyArgs(pl, DTYPE[logits.dtype], sl[0], sl[1], pq, sq[0], sq[1], _dense(tokens, "tokens", I32, bn, dev),
                   _dense(parents, "parents", I32, bn, dev), _dense(u, "u", F32, bn, dev),
                   _dense(u_next, "u_next", F32, b, dev), _opt(temperature, "temperature", F32, b, dev),
                   _dense(nodes, "nodes", I32, bn, dev), _dense(out, "out", I32, bn, dev), _dense(n, "n", I32, b, dev),
                   B, N)
    _borrow(ctx, logits, tokens, parents, u, u_next, nodes, out, n, q, temperature)
    ctx.check(lib().pi_verify(ctx.handle, ver.handle, ctypes.byref(a)))


def add_rmsnorm(ctx, x: torch.Tensor, res: Optional[torch.Tensor], w: torch.Tensor, eps: float,
                res_out: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None):
    """pi_add_rmsnorm: ``res_out`` = x + res (x alone without ``res``), and its RMS norm times ``w`` as
    int8 ``q`` [T][d] with one ``scale`` per row, as ``y``, or both."""
    if x.dim() != 2 or x.dtype not in DTYPE:
        _bad("x must be a floating-point tensor [T][d]")
    dev, shape = ctx.device, _sizes(x, "x")
    px, sx = _view(x, "x", x.dtype, shape, dev)
    rt = x.dtype if res is None else res.dtype
    if rt not in DTYPE:
        _bad(f"res has type {rt}")
    pr, sr = (None, (0,)) if res is None else _view(res, "res", rt, shape, dev)
    po, so = _view(res_out, "res_out", rt, shape, dev)
    pq, sq = (None, (0,)) if q is None else _view(q, "q", I8, shape, dev)
    if y is not None and y.dtype not in DTYPE:
        _bad(f"y has type {y.dtype}")
    py, sy = (None, (0,)) if y is None else _view(y, "y", y.dtype, shape, dev)
    a = NormArgs(px, pr, po, DTYPE[x.dtype], DTYPE[rt], sx[0], sr[0], so[0], _dense(w, "w", F32, (shape[1],), dev), eps,
                 pq, sq[0], _opt(scale, "scale", F32, (shape[0],), dev), py, 0 if y is None else DTYPE[y.dtype], sy[0],
                 shape[0], shape[1])
    _borrow(ctx, x, res, w, res_out, q, scale, y)
    ctx.check(lib().pi_add_rmsnorm(ctx.handle, ctypes.byref(a)))


class Linear(_Handle):
    """A pi_linear: an 8-bit weight ``w`` [N][K] (int8, borrowed) with a scale per output channel and
    an optional fp32 bias, for up to ``max_tokens`` tokens. The products of a context share its scratch:
    graphs that hold some of them are replayed one after another."""

    _destroy = "pi_linear_destroy"

    def __init__(self, ctx, w: torch.Tensor, w_scale: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 max_tokens: int = 1):
        if w.dim() != 2:
            _bad("w must be [N][K]")
        pw, sw = _view(w, "w", I8, _sizes(w, "w"), ctx.device)
        self.ctx, self.w, self.w_scale, self.bias = ctx, w, w_scale, bias
        self.N, self.K = w.shape
        desc = LinearDesc(self.N, self.K, pw, max(sw[0], self.K) if self.N == 1 else sw[0],
                          _dense(w_scale, "w_scale", F32, (self.N,), ctx.device),
                          _opt(bias, "bias", F32, (self.N,), ctx.device), max_tokens)
        h = c_void_p()
        ctx.check(lib().pi_linear_create(ctx.handle, ctypes.byref(desc), ctypes.byref(h)))
        self.handle = h


def linear_q8(ctx, lin: Linear, x: torch.Tensor, x_scale: torch.Tensor, y: torch.Tensor):
    """pi_linear_q8: ``y`` [M][N] = x_scale * w_scale * (x w^T) + bias for int8 ``x`` [M][K]."""
    if x.dim() != 2 or y.dtype not in DTYPE:
        _bad("x must be [M][K] and y a floating-point tensor [M][N]")
    dev, M = ctx.device, _sizes(x, "x")[0]
    px, sx = _view(x, "x", I8, (M, lin.K), dev)
    py, sy = _view(y, "y", y.dtype, (M, lin.N), dev)
    ps = _dense(x_scale, "x_scale", F32, (M,), dev)
    _borrow(ctx, x, x_scale, y, lin.w, lin.w_scale, lin.bias)
    ctx.check(lib().pi_linear_q8(ctx.handle, lin.handle, px, sx[0], ps, M, py, DTYPE[y.dtype], sy[0]))
