// The key/value cache: its handle and the append of new tokens (pi_kv_append).
#include <new>

#include "pi_kv.hpp"

using namespace pi;

namespace {

struct AppendDev {
  KvDev c;
  const uint8_t *kn, *vn;
  long long kv_batch, kv_node, kv_head;
  const int32_t *ctx_len, *nodes, *n;
  int32_t* len_out;
  int B, N, HK, pieces;  // pieces: 16-byte pieces of one head's row
};

// One workgroup per new token: its key and value rows, 16 bytes a lane, k and v in flight
// together. Bound by memory (each byte is read and written once): 4096 tokens of 32 heads of 128,
// 134 MB, 20 us, 6.7 TB/s; 16 tokens 2.4 us, the latency of a launch and three dependent loads.
__global__ __launch_bounds__(BLOCK) void k_kv_append(AppendDev p) {
  const int b = blockIdx.y, j = blockIdx.x;
  const int len = kv_len(p.c, p.ctx_len, b);
  const int n = p.n == nullptr ? p.N : min(max(p.n[b], 0), p.N);
  if (p.len_out != nullptr && j == 0 && threadIdx.x == 0) p.len_out[b] = (int)min((long long)len + n, (long long)p.c.capacity);
  if (j >= n || (uint32_t)len + (uint32_t)j >= (uint32_t)p.c.capacity) return;  // their sum may pass 2^31
  const int src = p.nodes == nullptr ? j : p.nodes[(long long)b * p.N + j];
  if ((unsigned)src >= (unsigned)p.N) return;
  uint32_t off;
  const int page = kv_page(p.c, b, page_of(p.c.div, (uint32_t)(len + j), &off));
  if (page < 0) return;
  const long long from = (long long)b * p.kv_batch + (long long)src * p.kv_node;
  const long long to = (long long)page * p.c.page_stride + (long long)off * p.c.token_stride;
  for (int i = threadIdx.x; i < p.HK * p.pieces; i += BLOCK) {
    const int h = i / p.pieces, e = 8 * (i % p.pieces);
    const long long f = 2 * (from + h * p.kv_head + e), t = 2 * (to + h * p.c.head_stride + e);
    const u32x4 k = ld16(p.kn + f), v = ld16(p.vn + f);
    *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p.c.k) + t) = k;
    *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p.c.v) + t) = v;
  }
}

// len_out where it is ctx_len itself: after the copy, whose workgroups all read ctx_len.
__global__ __launch_bounds__(BLOCK) void k_kv_len(AppendDev p) {
  const int b = blockIdx.x * BLOCK + threadIdx.x;
  if (b >= p.B) return;
  const int n = p.n == nullptr ? p.N : min(max(p.n[b], 0), p.N);
  p.len_out[b] = (int)min((long long)kv_len(p.c, p.ctx_len, b) + n, (long long)p.c.capacity);
}

}  // namespace

extern "C" {

pi_status pi_kv_create(pi_ctx* ctx, const pi_kv_desc* desc, pi_kv** out) {
  if (ctx == nullptr || out == nullptr) return PI_ERR_INVALID;
  *out = nullptr;
  if (desc == nullptr) return fail(ctx, PI_ERR_INVALID, "desc is NULL");
  const pi_kv_desc& d = *desc;
  if (d.dtype != PI_T_F16 && d.dtype != PI_T_BF16) return fail(ctx, PI_ERR_INVALID, "cache dtype %d: need fp16 or bf16", d.dtype);
  if (d.heads < 1 || d.pages < 1 || d.page_tokens < 1 || d.page_tokens >= (1ll << 31) - 64)
    return fail(ctx, PI_ERR_INVALID, "bad cache shape: %d pages of %d tokens, %d heads", d.pages, d.page_tokens, d.heads);
  if (d.head_dim < 8 || d.head_dim % 8) return fail(ctx, PI_ERR_INVALID, "head_dim must be a multiple of 8 (got %d)", d.head_dim);
  if (d.head_dim > 256) return fail(ctx, PI_ERR_UNSUPPORTED, "head_dim %d above 256", d.head_dim);
  if (d.page_stride < 0 || d.token_stride < 0 || d.head_stride < 0 || ((d.page_stride | d.token_stride | d.head_stride) & 7))
    return fail(ctx, PI_ERR_INVALID, "cache strides must be multiples of 8 elements");
  if (d.page_stride >= (1ll << 35) || d.token_stride >= (1ll << 35))
    return fail(ctx, PI_ERR_UNSUPPORTED, "page and token strides are below 2^35");
  PI_TRY(check_dev_ptr(ctx, d.k, "k"));
  PI_TRY(check_dev_ptr(ctx, d.v, "v"));
  pi_kv* kv = new (std::nothrow) pi_kv{d, ctx};
  if (kv == nullptr) return fail(ctx, PI_ERR_OOM, "host allocation failed");
  ctx_retain(ctx);
  *out = kv;
  return PI_OK;
}

void pi_kv_destroy(pi_kv* kv) {
  if (kv == nullptr) return;
  ctx_release(kv->ctx);
  delete kv;
}

pi_status pi_kv_append(pi_ctx* ctx, const pi_kv* kv, const pi_append_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_append_args& a = *args;
  PI_TRY(check_paging(ctx, kv, a.table, a.table_stride, a.table_width, a.ctx_len, a.B, a.N));
  if (a.B > 65535) return fail(ctx, PI_ERR_UNSUPPORTED, "B %d above 65535", a.B);
  PI_TRY(check_bnh(ctx, "k_new", a.k_new, a.kv_batch, a.kv_node, a.kv_head));
  PI_TRY(check_bnh(ctx, "v_new", a.v_new, a.kv_batch, a.kv_node, a.kv_head));
  PI_HIP(ctx, hipSetDevice(ctx->device));
  // in place as soon as the two ranges meet, not only where they start alike
  const bool in_place = a.len_out != nullptr && a.len_out < a.ctx_len + a.B && a.ctx_len < a.len_out + a.B;
  if (in_place && a.len_out != a.ctx_len) return fail(ctx, PI_ERR_INVALID, "len_out overlaps ctx_len in part");
  AppendDev p{kv_dev(kv, a.table, a.table_stride, a.table_width), static_cast<const uint8_t*>(a.k_new),
              static_cast<const uint8_t*>(a.v_new), a.kv_batch, a.kv_node, a.kv_head, a.ctx_len, a.nodes, a.n,
              in_place ? nullptr : a.len_out, a.B, a.N, kv->desc.heads, kv->desc.head_dim / 8};
  PI_HIP(ctx, launch_k(ctx, 0, k_kv_append, dim3(a.N, a.B), 0, p));
  if (in_place) {
    p.len_out = a.len_out;
    PI_HIP(ctx, launch_k(ctx, 0, k_kv_len, dim3((a.B + BLOCK - 1) / BLOCK), 0, p));
  }
  return PI_OK;
}

}  // extern "C"
