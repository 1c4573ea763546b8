// The key/value cache: its handles, the append of new tokens (pi_kv_append) and the reading of held ones
// (pi_kv_read).
#include <algorithm>
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

// The append to a 4-bit cache. A block of 32 elements is four lanes of 8: its largest element by
// magnitude is an exchange among them away, and so are the halves of its code bytes (elements j and
// j + 16 are two lanes apart). scale = -m/8 rounded to 8 significant bits: times a code it is an fp16
// number exactly. The quotient by the scale: its product with the rounded reciprocal lands off a tie;
// corrected by that product's remainder, which is exact, it is the rounded quotient (Markstein).
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_kv4_append(AppendDev p, Kv4Dev sc) {
  const int b = blockIdx.y, j = blockIdx.x;
  const int len = kv_len(p.c, p.ctx_len, b);
  const int n = p.n == nullptr ? p.N : min(max(p.n[b], 0), p.N);
  if (p.len_out != nullptr && j == 0 && threadIdx.x == 0) p.len_out[b] = (int)min((long long)len + n, (long long)p.c.capacity);
  if (j >= n || (uint32_t)len + (uint32_t)j >= (uint32_t)p.c.capacity) return;
  const int src = p.nodes == nullptr ? j : p.nodes[(long long)b * p.N + j];
  if ((unsigned)src >= (unsigned)p.N) return;
  uint32_t off;
  const int page = kv_page(p.c, b, page_of(p.c.div, (uint32_t)(len + j), &off));
  if (page < 0) return;
  const long long from = (long long)b * p.kv_batch + (long long)src * p.kv_node;
  const long long to = (long long)page * p.c.page_stride + (long long)off * p.c.token_stride;
  const long long sto = (long long)page * sc.page + (long long)off * sc.token;
  const int each = p.HK * p.pieces;  // a multiple of 4: the lanes of a block go together
  for (int i = threadIdx.x; i < 2 * each; i += BLOCK) {
    const bool val = i >= each;
    const int r = val ? i - each : i, h = r / p.pieces, e = r % p.pieces;
    float x[8];
    load8(reinterpret_cast<const T*>(val ? p.vn : p.kn) + from + h * p.kv_head + 8 * e, x);
    float hi = x[0], lo = x[0], sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      hi = fmaxf(hi, x[k]);
      lo = fminf(lo, x[k]);
      sum += 0.f * x[k];  // NaN where an element is infinite or NaN
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      hi = fmaxf(hi, __shfl_xor(hi, o, WAVE));
      lo = fminf(lo, __shfl_xor(lo, o, WAVE));
      sum += __shfl_xor(sum, o, WAVE);
    }
    const float m = hi >= -lo ? hi : lo;
    const float s8 = (float)(bf16_t)(m * -0.125f);
    half_t scale = (half_t)fminf(fmaxf(s8, -8160.f), 8160.f);
    const bool bad = sum != sum;
    if (bad) scale = (half_t)__builtin_nanf("");
    const float f = (float)scale;
    const bool none = bad || f == 0.f;
    const float inv = none ? 0.f : 1.0f / f;
    uint32_t lo4[2] = {0, 0};  // 8 codes, one a byte
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float q = x[k] * inv;
      float v = none ? 0.f : rintf(__builtin_fmaf(__builtin_fmaf(-q, f, x[k]), inv, q));
      v = fminf(fmaxf(v, -8.f), 7.f);
      lo4[k >> 2] |= (uint32_t)((int)v + 8) << (8 * (k & 3));
    }
    // lanes 0 and 2 share bytes 0..7, lanes 1 and 3 bytes 8..15: the lower lane writes the first four
    const uint32_t o0 = __shfl_xor(lo4[0], 2, WAVE), o1 = __shfl_xor(lo4[1], 2, WAVE);
    const bool upper = e & 2;
    const uint32_t word = upper ? o1 | lo4[1] << 4 : lo4[0] | o0 << 4;
    uint8_t* codes = static_cast<uint8_t*>(val ? p.c.v : p.c.k) + to + h * p.c.head_stride + 16 * (e >> 2) + 8 * (e & 1) + (upper ? 4 : 0);
    *reinterpret_cast<uint32_t*>(codes) = word;
    if ((e & 3) == 0) (val ? sc.vs : sc.ks)[sto + h * sc.head + (e >> 2)] = __builtin_bit_cast(uint16_t, scale);
  }
}

struct ReadDev {
  KvDev c;
  Kv4Dev sc;
  const int32_t *ctx_len, *start, *cu;
  uint8_t *ko, *vo;
  long long row, head;
  int B, rows, HK, pieces, per;  // pieces: work items of one head's row; per: rows of a workgroup
};
constexpr int READ_ROWS = 16;

// Rows from the cache, `per` consecutive ones a workgroup: it counts the sequences that start at or before
// its first row, and each row steps on from there. Bound by memory. A 4-bit row's item is 8 code
// bytes, which are 8 elements and the 8 that lie 16 further on; a plain row's is 16 bytes.
template <typename T, bool Q4>
__global__ __launch_bounds__(BLOCK) void k_kv_read(ReadDev p) {
  __shared__ long long s_page[READ_ROWS];  // page number, or -1: zeros, -2: the row stays
  __shared__ int s_off[READ_ROWS], s_count[NWAVES];
  const int r0 = blockIdx.x * p.per;
  int n = 0;
  for (int i = threadIdx.x; i <= p.B; i += BLOCK) n += p.cu[i] <= r0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, WAVE);
  if (threadIdx.x % WAVE == 0) s_count[threadIdx.x / WAVE] = n;
  __syncthreads();
  const int rows = min(p.per, p.rows - r0);
  if ((int)threadIdx.x < rows) {
    n = 0;
#pragma unroll
    for (int w = 0; w < NWAVES; ++w) n += s_count[w];
    const int row = r0 + threadIdx.x;
    int b = n - 1;
    while (b + 1 < p.B && p.cu[b + 1] <= row) ++b;
    long long page = -2;
    if (b >= 0 && b < p.B && row >= p.cu[b] && row < p.cu[b + 1]) {
      const long long at = (long long)(p.start == nullptr ? 0 : max(p.start[b], 0)) + ((long long)row - p.cu[b]);
      if (at < kv_len(p.c, p.ctx_len, b)) {
        uint32_t off;
        page = kv_page(p.c, b, page_of(p.c.div, (uint32_t)at, &off));
        s_off[threadIdx.x] = (int)off;
      }
    }
    s_page[threadIdx.x] = page;
  }
  __syncthreads();
  const int each = p.HK * p.pieces, all = rows * 2 * each;
  for (int i = threadIdx.x; i < all; i += BLOCK) {
    const int r = i / (2 * each), j = i % (2 * each);
    const long long page = s_page[r];
    if (page == -2) continue;
    const bool val = j >= each;
    const int k = val ? j - each : j, h = k / p.pieces, e = k % p.pieces;
    T* o = reinterpret_cast<T*>(val ? p.vo : p.ko) + (long long)(r0 + r) * p.row + h * p.head;
    const long long off = page < 0 ? 0 : s_off[r], pg = page < 0 ? 0 : page;
    if constexpr (Q4) {
      const uint8_t* c = static_cast<const uint8_t*>(val ? p.c.v : p.c.k) + pg * p.c.page_stride + off * p.c.token_stride +
                         h * p.c.head_stride + 8 * e;
      const uint2 w = *reinterpret_cast<const uint2*>(c);
      const uint16_t s16 = (val ? p.sc.vs : p.sc.ks)[pg * p.sc.page + off * p.sc.token + h * p.sc.head + (e >> 1)];
      const float s = page < 0 ? 0.f : half_bits_to_float(s16);
      float lo[8], hi[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t byte = ((x < 4 ? w.x : w.y) >> (8 * (x & 3))) & 0xFFu;
        lo[x] = ((float)(byte & 15u) - 8.f) * s;
        hi[x] = ((float)(byte >> 4) - 8.f) * s;
      }
      o += 32 * (e >> 1) + 8 * (e & 1);
      store8(o, lo);
      store8(o + 16, hi);
    } else {
      const T* c = static_cast<const T*>(val ? p.c.v : p.c.k) + pg * p.c.page_stride + off * p.c.token_stride + h * p.c.head_stride + 8 * e;
      const u32x4 w = ld16(c);
      *reinterpret_cast<u32x4*>(o + 8 * e) = page < 0 ? (u32x4){0, 0, 0, 0} : w;
    }
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

pi_status pi_kv4_create(pi_ctx* ctx, const pi_kv4_desc* desc, pi_kv** out) {
  if (ctx == nullptr || out == nullptr) return PI_ERR_INVALID;
  *out = nullptr;
  if (desc == nullptr) return fail(ctx, PI_ERR_INVALID, "desc is NULL");
  const pi_kv4_desc& d = *desc;
  if (d.dtype != PI_T_F16 && d.dtype != PI_T_BF16) return fail(ctx, PI_ERR_INVALID, "cache dtype %d: need fp16 or bf16", d.dtype);
  if (d.heads < 1 || d.pages < 1 || d.page_tokens < 1 || d.page_tokens >= (1ll << 31) - 64)
    return fail(ctx, PI_ERR_INVALID, "bad cache shape: %d pages of %d tokens, %d heads", d.pages, d.page_tokens, d.heads);
  if (d.head_dim < 32 || d.head_dim % 32) return fail(ctx, PI_ERR_INVALID, "head_dim must be a multiple of 32 (got %d)", d.head_dim);
  if (d.head_dim > 256) return fail(ctx, PI_ERR_UNSUPPORTED, "head_dim %d above 256", d.head_dim);
  if (d.page_stride < 0 || d.token_stride < 0 || d.head_stride < 0 || ((d.page_stride | d.token_stride | d.head_stride) & 15))
    return fail(ctx, PI_ERR_INVALID, "strides of the codes must be multiples of 16 bytes");
  if (d.scale_page_stride < 0 || d.scale_token_stride < 0 || d.scale_head_stride < 0 ||
      (d.head_dim % 64 == 0 && ((d.scale_page_stride | d.scale_token_stride | d.scale_head_stride) & 1)))
    return fail(ctx, PI_ERR_INVALID, "strides of the scales must be even");
  if (d.page_stride >= 1ll << 35 || d.token_stride >= 1ll << 35 || d.head_stride >= 1ll << 35)
    return fail(ctx, PI_ERR_UNSUPPORTED, "strides of the codes are below 2^35");
  if (d.scale_page_stride >= 1ll << 32 || d.scale_token_stride >= 1ll << 32 || d.scale_head_stride >= 1ll << 32)
    return fail(ctx, PI_ERR_UNSUPPORTED, "strides of the scales are below 2^32");
  PI_TRY(check_dev_ptr(ctx, d.k, "k"));
  PI_TRY(check_dev_ptr(ctx, d.v, "v"));
  PI_TRY(check_dev_ptr(ctx, d.k_scale, "k_scale"));
  PI_TRY(check_dev_ptr(ctx, d.v_scale, "v_scale"));
  const pi_kv_desc codes{d.dtype, d.heads, d.head_dim, d.pages, d.page_tokens, d.k, d.v, d.page_stride, d.token_stride, d.head_stride};
  pi_kv* kv = new (std::nothrow) pi_kv{codes, ctx, true, d.k_scale, d.v_scale, d.scale_page_stride, d.scale_token_stride, d.scale_head_stride};
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
  if (!kv->q4) PI_HIP(ctx, launch_k(ctx, 0, k_kv_append, dim3(a.N, a.B), 0, p));
  else if (kv->desc.dtype == PI_T_F16) PI_HIP(ctx, launch_k(ctx, 0, k_kv4_append<half_t>, dim3(a.N, a.B), 0, p, kv4_dev(kv)));
  else PI_HIP(ctx, launch_k(ctx, 0, k_kv4_append<bf16_t>, dim3(a.N, a.B), 0, p, kv4_dev(kv)));
  if (in_place) {
    p.len_out = a.len_out;
    PI_HIP(ctx, launch_k(ctx, 0, k_kv_len, dim3((a.B + BLOCK - 1) / BLOCK), 0, p));
  }
  return PI_OK;
}

pi_status pi_kv_read(pi_ctx* ctx, const pi_kv* kv, const pi_read_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_read_args& a = *args;
  PI_TRY(check_paging(ctx, kv, a.table, a.table_stride, a.table_width, a.ctx_len, a.B, 1));
  if (a.cu == nullptr) return fail(ctx, PI_ERR_INVALID, "cu is NULL");
  if (a.rows < 0) return fail(ctx, PI_ERR_INVALID, "%d rows", a.rows);
  if (a.rows > 1 << 27) return fail(ctx, PI_ERR_UNSUPPORTED, "%d rows: at most 2^27", a.rows);
  if (a.rows == 0) return PI_OK;
  PI_TRY(check_bnh(ctx, "k_out", a.k_out, 0, a.out_row, a.out_head));
  PI_TRY(check_bnh(ctx, "v_out", a.v_out, 0, a.out_row, a.out_head));
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const int pieces = kv->desc.head_dim / (kv->q4 ? 16 : 8);
  // rows of a workgroup: one while the chip is not full of them
  const int per = std::min(READ_ROWS, std::max({1, a.rows / (8 * ctx->cus), (a.rows - 1) / (1 << 23) + 1}));
  const ReadDev p{kv_dev(kv, a.table, a.table_stride, a.table_width), kv4_dev(kv), a.ctx_len, a.start, a.cu,
                  static_cast<uint8_t*>(a.k_out), static_cast<uint8_t*>(a.v_out), a.out_row, a.out_head, a.B, a.rows,
                  kv->desc.heads, pieces, per};
  const dim3 grid((a.rows - 1) / per + 1);
  const bool f16 = kv->desc.dtype == PI_T_F16;
  if (kv->q4) PI_HIP(ctx, f16 ? launch_k(ctx, 0, k_kv_read<half_t, true>, grid, 0, p) : launch_k(ctx, 0, k_kv_read<bf16_t, true>, grid, 0, p));
  else PI_HIP(ctx, f16 ? launch_k(ctx, 0, k_kv_read<half_t, false>, grid, 0, p) : launch_k(ctx, 0, k_kv_read<bf16_t, false>, grid, 0, p));
  return PI_OK;
}

}  // extern "C"
