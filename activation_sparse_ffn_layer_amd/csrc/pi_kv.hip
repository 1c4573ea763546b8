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

// The append to a 4-bit cache: `per` consecutive new tokens of a sequence a workgroup, whose places it finds first, side by
// side. A block of 32 elements is four lanes of 8: its largest element by magnitude is an exchange among them away, and
// so are the halves of its code bytes (elements j and j + 16 are two lanes apart). scale = -m/8 rounded to 8
// significant bits: times a code it is an fp16 number exactly. The quotient by the scale: its product with the rounded
// reciprocal lands off a tie; corrected by that product's remainder, which is exact, it is the rounded quotient
// (Markstein). 16 x 1024 tokens of 8 heads of 128 (86 MB) 26 us, 3.3 TB/s: the quantiser's arithmetic, about 130
// instructions for 8 elements, is 14 of them, next to dependent loads (a token's place, then a row for each of a lane's
// items, waited for where it is converted). 16 short paths 3.8 us, latency.
constexpr int KV_ROWS = 16;  // rows of a workgroup, at most
// The value of a lane of the same four: 0xB1 the neighbour's, 0x4E that two on.
template <int CTRL, typename V>
__device__ __forceinline__ V quad(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_kv4_append(AppendDev p, Kv4Dev sc, PageDiv by_row, PageDiv by_head, int per) {
  __shared__ long long s_from[KV_ROWS], s_to[KV_ROWS], s_scale[KV_ROWS];
  const int b = blockIdx.y, j0 = blockIdx.x * per;
  const int n = p.n == nullptr ? p.N : min(max(p.n[b], 0), p.N);
  const int rows = min(per, p.N - j0);
  if ((int)threadIdx.x < rows) {
    const int j = j0 + threadIdx.x, len = kv_len(p.c, p.ctx_len, b);
    if (p.len_out != nullptr && j == 0) p.len_out[b] = (int)min((long long)len + n, (long long)p.c.capacity);
    long long to = -1;
    if (j < n && (uint32_t)len + (uint32_t)j < (uint32_t)p.c.capacity) {
      const int src = p.nodes == nullptr ? j : p.nodes[(long long)b * p.N + j];
      uint32_t off;
      const int page = kv_page(p.c, b, page_of(p.c.div, (uint32_t)(len + j), &off));
      if (page >= 0 && (unsigned)src < (unsigned)p.N) {
        to = (long long)page * p.c.page_stride + (long long)off * p.c.token_stride;
        s_from[threadIdx.x] = (long long)b * p.kv_batch + (long long)src * p.kv_node;
        s_scale[threadIdx.x] = (long long)page * sc.page + (long long)off * sc.token;
      }
    }
    s_to[threadIdx.x] = to;
  }
  __syncthreads();
  const int each = p.HK * p.pieces;  // a multiple of 4: the lanes of a block go together
  constexpr int U = 2;               // items of a lane a step
  for (int i0 = threadIdx.x; i0 < rows * 2 * each; i0 += U * BLOCK) {
    float x[U][8];
    int row[U], h[U];
    uint32_t e[U], r[U];
    bool val[U], in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * BLOCK;
      in[u] = i < rows * 2 * each;
      row[u] = in[u] ? (int)page_of(by_row, (uint32_t)i, &r[u]) : 0;
      in[u] = in[u] && s_to[row[u]] >= 0;
      val[u] = in[u] && (int)r[u] >= each;
      h[u] = in[u] ? (int)page_of(by_head, r[u] - (val[u] ? each : 0), &e[u]) : 0;
      if (in[u]) {
        load8(reinterpret_cast<const T*>(val[u] ? p.vn : p.kn) + s_from[row[u]] + h[u] * p.kv_head + 8 * e[u], x[u]);
      } else {
        e[u] = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][k] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float hi = x[u][0], lo = x[u][0], sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        hi = fmaxf(hi, x[u][k]);
        lo = fminf(lo, x[u][k]);
        sum = __builtin_fmaf(0.f, x[u][k], sum);  // NaN where an element is infinite or NaN
      }
      hi = fmaxf(hi, quad<0xB1>(hi));
      lo = fminf(lo, quad<0xB1>(lo));
      sum += quad<0xB1>(sum);
      hi = fmaxf(hi, quad<0x4E>(hi));
      lo = fminf(lo, quad<0x4E>(lo));
      sum += quad<0x4E>(sum);
      const float m = hi >= -lo ? hi : lo;
      const float s8 = (float)(bf16_t)(m * -0.125f);
      const bool bad = sum != sum;
      const half_t scale = bad ? (half_t)__builtin_nanf("") : (half_t)fminf(fmaxf(s8, -8160.f), 8160.f);
      const float f = bad ? 0.f : (float)scale, inv = f == 0.f ? 0.f : 1.0f / f;
      uint32_t q[8];  // a code in the low byte: 1.5 2^23 leaves whole numbers in a float's last bits, ties to even
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float y = x[u][k] * inv;
        const float v = __builtin_fmaf(__builtin_fmaf(-y, f, x[u][k]), inv, y);
        q[k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(v, -8.f, 7.f) + 12582920.f);
      }
      uint32_t q4[2];  // 8 codes, one a byte
#pragma unroll
      for (int k = 0; k < 2; ++k)
        q4[k] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[4 * k + 3], q[4 * k + 2], 0x0C0C0400u),
                                      __builtin_amdgcn_perm(q[4 * k + 1], q[4 * k], 0x0C0C0400u), 0x05040100u);
      // lanes 0 and 2 share bytes 0..7, lanes 1 and 3 bytes 8..15: the lower lane writes the first four
      const uint32_t o0 = quad<0x4E>(q4[0]), o1 = quad<0x4E>(q4[1]);
      if (!in[u]) continue;
      const bool upper = e[u] & 2;
      const uint32_t word = bad ? 0x88888888u : upper ? o1 | q4[1] << 4 : q4[0] | o0 << 4;
      uint8_t* codes = static_cast<uint8_t*>(val[u] ? p.c.v : p.c.k) + s_to[row[u]] + h[u] * p.c.head_stride + 16 * (e[u] >> 2) +
                       8 * (e[u] & 1) + (upper ? 4 : 0);
      *reinterpret_cast<uint32_t*>(codes) = word;
      if ((e[u] & 3) == 0) (val[u] ? sc.vs : sc.ks)[s_scale[row[u]] + h[u] * sc.head + (e[u] >> 2)] = __builtin_bit_cast(uint16_t, scale);
    }
  }
}

struct ReadDev {
  KvDev c;
  Kv4Dev sc;
  const int32_t *ctx_len, *start, *cu;
  uint8_t *ko, *vo;
  long long row, head;
  PageDiv by_row, by_head;        // items of a row, keys and values, and of one head's row
  int B, rows, each, per;         // each: items of a row's keys; per: rows of a workgroup
};

// Rows from the cache, `per` consecutive ones a workgroup: it counts the sequences that start at or before
// its first row, and each row steps on from there. Bound by memory:
// 94745 rows (8 sequences of up to 16384) of 8 heads of 128 from 4 bits, 497 MB, 98 to 106 us, 4.7 to 5.1 TB/s; from a plain
// cache, 776 MB, 155 us, 5.0 TB/s. An item is 16 bytes put out, so that a wave's stores are whole lines; of a 4-bit row it is
// one half of 8 code bytes (written as both halves, 32 bytes each of a line in two stores, the same rows took 141 us).
template <typename T, bool Q4>
__global__ __launch_bounds__(BLOCK) void k_kv_read(ReadDev p) {
  __shared__ long long s_page[KV_ROWS];  // page number, or -1: zeros, -2: the row stays
  __shared__ int s_off[KV_ROWS], s_count[NWAVES];
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
  constexpr int U = 4;  // items of a lane in flight
  const int all = rows * 2 * p.each;
  for (int i0 = threadIdx.x; i0 < all; i0 += U * BLOCK) {
    T* o[U];
    uint2 w2[U];
    u32x4 w4[U];
    bool high[U];
    uint16_t s16[U];
    bool put[U], held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * BLOCK, all - 1);
      uint32_t j, e;
      const int r = (int)page_of(p.by_row, (uint32_t)i, &j);
      const long long page = s_page[r];
      put[u] = i0 + u * BLOCK < all && page != -2;
      held[u] = page >= 0;
      const bool val = (int)j >= p.each;
      const int h = (int)page_of(p.by_head, j - (val ? p.each : 0), &e);
      o[u] = reinterpret_cast<T*>(val ? p.vo : p.ko) + (long long)(r0 + r) * p.row + h * p.head;
      const long long pg = held[u] ? page : 0, off = held[u] ? s_off[r] : 0;  // page 0 is there in any case
      const long long at = pg * p.c.page_stride + off * p.c.token_stride + h * p.c.head_stride;
      if constexpr (Q4) {
        w2[u] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(val ? p.c.v : p.c.k) + at + 16 * (e >> 2) + 8 * (e & 1));
        s16[u] = (val ? p.sc.vs : p.sc.ks)[pg * p.sc.page + off * p.sc.token + h * p.sc.head + (e >> 2)];
        high[u] = e & 2;
      } else {
        w4[u] = ld16(static_cast<const T*>(val ? p.c.v : p.c.k) + at + 8 * e);
      }
      o[u] += 8 * e;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!put[u]) continue;
      if constexpr (Q4) {
        const float s = held[u] ? half_bits_to_float(s16[u]) : 0.f;
        const uint32_t c[2] = {(high[u] ? w2[u].x >> 4 : w2[u].x) & 0x0F0F0F0Fu, (high[u] ? w2[u].y >> 4 : w2[u].y) & 0x0F0F0F0Fu};
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = ((float)((c[x >> 2] >> (8 * (x & 3))) & 0xFFu) - 8.f) * s;
        __attribute__((aligned(16))) T r[8];
        store8(r, v);
        __builtin_memcpy(&w4[u], r, 16);
      } else if (!held[u]) {
        w4[u] = (u32x4){0, 0, 0, 0};
      }
      // past the caches' usual order: 127 -> 103 us for 94745 rows of 8 heads of 128
      __builtin_nontemporal_store(w4[u], reinterpret_cast<u32x4*>(o[u]));
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
  if (d.heads > 1 << 16) return fail(ctx, PI_ERR_UNSUPPORTED, "%d heads: at most 65536", d.heads);
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
  else {
    // tokens of a workgroup: one while the chip is not full of them
    const int per = (int)std::min<int64_t>(KV_ROWS, std::max<int64_t>(1, (int64_t)a.N * a.B / (8 * ctx->cus)));
    const dim3 grid((a.N - 1) / per + 1, a.B);
    const PageDiv by_row = page_div(2 * p.HK * p.pieces), by_head = page_div(p.pieces);
    PI_HIP(ctx, kv->desc.dtype == PI_T_F16 ? launch_k(ctx, 0, k_kv4_append<half_t>, grid, 0, p, kv4_dev(kv), by_row, by_head, per)
                                           : launch_k(ctx, 0, k_kv4_append<bf16_t>, grid, 0, p, kv4_dev(kv), by_row, by_head, per));
  }
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
  if (kv->desc.heads > 1 << 16) return fail(ctx, PI_ERR_UNSUPPORTED, "%d heads: at most 65536", kv->desc.heads);
  if (a.rows > 1 << 27) return fail(ctx, PI_ERR_UNSUPPORTED, "%d rows: at most 2^27", a.rows);
  if (a.rows == 0) return PI_OK;
  PI_TRY(check_bnh(ctx, "k_out", a.k_out, 0, a.out_row, a.out_head));
  PI_TRY(check_bnh(ctx, "v_out", a.v_out, 0, a.out_row, a.out_head));
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const int pieces = kv->desc.head_dim / 8;
  // rows of a workgroup: one while the chip is not full of them
  const int per = std::min(KV_ROWS, std::max({1, a.rows / (4 * ctx->cus), (a.rows - 1) / (1 << 23) + 1}));
  const ReadDev p{kv_dev(kv, a.table, a.table_stride, a.table_width), kv4_dev(kv), a.ctx_len, a.start, a.cu,
                  static_cast<uint8_t*>(a.k_out), static_cast<uint8_t*>(a.v_out), a.out_row, a.out_head,
                  page_div(2 * kv->desc.heads * pieces), page_div(pieces), a.B, a.rows, kv->desc.heads * pieces, per};
  const dim3 grid((a.rows - 1) / per + 1);
  const bool f16 = kv->desc.dtype == PI_T_F16;
  if (kv->q4) PI_HIP(ctx, f16 ? launch_k(ctx, 0, k_kv_read<half_t, true>, grid, 0, p) : launch_k(ctx, 0, k_kv_read<bf16_t, true>, grid, 0, p));
  else PI_HIP(ctx, f16 ? launch_k(ctx, 0, k_kv_read<half_t, false>, grid, 0, p) : launch_k(ctx, 0, k_kv_read<bf16_t, false>, grid, 0, p));
  return PI_OK;
}

}  // extern "C"
