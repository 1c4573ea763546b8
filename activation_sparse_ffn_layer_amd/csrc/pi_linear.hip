// The 8-bit matrix product (pi_linear_q8): y[m][n] = xs[m] ws[n] sum_k x[m][k] w[n][k] + b[n].
//
// The sums are whole numbers below 2^31 (K < 131072), exact in the matrix cores' 32-bit
// accumulators whatever their order; the scales are applied once to the sum in fp32. Weight rows
// are the products' A operand, so a lane ends with 4 consecutive output channels of one token.
#include <algorithm>
#include <new>

#include "pi_host.hpp"
#include "pi_types.hpp"

using namespace pi;

struct pi_linear {
  pi_ctx* ctx;
  pi_linear_desc desc;
};

namespace {

struct LinDev {
  const int8_t *x, *w;
  const float *xs, *ws, *bias;
  void* y;
  long long x_stride, w_stride, y_stride;
  int M, N, K;
};

template <typename T> struct Vec4 { typedef T type __attribute__((ext_vector_type(4))); };

// y[m][n0..n0+3] from 4 whole-number sums and their channels' scales and biases
template <typename T>
__device__ __forceinline__ void put4(const LinDev& p, int m, int n0, const float (&ws)[4], const float (&bias)[4], i32x4 s,
                                     bool wide) {
  if (m >= p.M || n0 >= p.N) return;
  const float xs = p.xs[m];
  T* y = static_cast<T*>(p.y) + (long long)m * p.y_stride + n0;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)s[i] * xs * ws[i] + bias[i];
  if (wide && n0 + 3 < p.N) {
    typedef typename Vec4<T>::type V;
    V o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (T)v[i];
    *reinterpret_cast<V*>(y) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < p.N) y[i] = (T)v[i];
  }
}
template <typename T>
__device__ __forceinline__ void put4(const LinDev& p, int m, int n0, i32x4 s, bool wide) {
  float ws[4], bias[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, p.N - 1);
    ws[i] = p.ws[n];
    bias[i] = p.bias != nullptr ? p.bias[n] : 0.f;
  }
  put4<T>(p, m, n0, ws, bias, s, wide);
}

// ---------------------------------------------------------------------------------------
// Few tokens: bound by the weights' bytes. A workgroup owns 16 RB weight rows and 16 MB
// tokens; its waves deal the K axis in pieces of 256 among themselves, each lane reading 16
// bytes of a row straight into the operand's layout (no LDS), and add their sums in LDS.
// ---------------------------------------------------------------------------------------
constexpr int LR_WAVES = 8;

template <typename T, int MB, int RB>
__global__ __launch_bounds__(64 * LR_WAVES) void k_q8_rows(LinDev p, bool wide) {
  constexpr int U = 4;  // 64-wide steps per piece
  __shared__ i32x4 red[LR_WAVES][RB * MB][WAVE];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, l16 = lane & 15;
  const int n0 = blockIdx.x * 16 * RB, m0 = blockIdx.y * 16 * MB;
  const int ko = 16 * (lane >> 4);
  const int8_t *wp[RB], *xp[MB];
  bool xin[MB];
#pragma unroll
  for (int i = 0; i < RB; ++i) wp[i] = p.w + (long long)min(n0 + 16 * i + l16, p.N - 1) * p.w_stride;
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int m = m0 + 16 * j + l16;
    xin[j] = m < p.M;
    xp[j] = p.x + (long long)min(m, p.M - 1) * p.x_stride;
  }
  i32x4 acc[RB][MB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  for (int k0 = wave * 64 * U; k0 < p.K; k0 += LR_WAVES * 64 * U) {
    u32x4 a[U][RB], b[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 64 * u + ko;
      const bool in = k < p.K;
      const int kk = in ? k : 0;
#pragma unroll
      for (int i = 0; i < RB; ++i) a[u][i] = ld_stream_or0(wp[i] + kk, in);
#pragma unroll
      for (int j = 0; j < MB; ++j) b[u][j] = ld16_or0(xp[j] + kk, in && xin[j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a[u][i]),
                                                            __builtin_bit_cast(i32x4, b[u][j]), acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) red[wave][i * MB + j][lane] = acc[i][j];
  __syncthreads();
  for (int t = wave; t < RB * MB; t += LR_WAVES) {
    i32x4 s = red[0][t][lane];
#pragma unroll
    for (int w = 1; w < LR_WAVES; ++w) s += red[w][t][lane];
    put4<T>(p, m0 + 16 * (t % MB) + l16, n0 + 16 * (t / MB) + 4 * (lane >> 4), s, wide);
  }
}

// ---------------------------------------------------------------------------------------
// Many tokens: bound by the matrix cores. Four waves own a square tile of 64 FB weight rows and
// tokens, staged in LDS 128 bytes of K at a time in two stages: during the products of one, the
// other is written from registers and the registers are loaded anew, spread over the steps.
// A wave's quarter of the tile is FB x FB blocks of 32 x 32, so LDS is read 2 FB rows for FB^2
// products: with FB = 4 half as often per product as with 2, which LDS bandwidth bounds.
// ---------------------------------------------------------------------------------------
constexpr int LT_K = 128, LT_P = LT_K + 16;  // K bytes per stage; LDS row pitch (bytes)
constexpr uint32_t LT_OOB = 0xC0000000u;     // past any tile's records: reads as zero
template <int FB> constexpr size_t tile_lds() { return (size_t)2 * 2 * 64 * FB * LT_P; }

// The tile of workgroup id: the XCDs (id % 8) take equal runs of tiles, in an order that
// walks 8 tiles of tokens, then the weight rows, so that an XCD's tiles in flight share rows.
__device__ __forceinline__ void tile_of(int id, int tn, int tm, int* n, int* m) {
  const int total = tn * tm, x = id & 7, each = total >> 3, more = total & 7;
  const int t = x * each + min(x, more) + (id >> 3);
  const int group = t / (8 * tn), r = t - group * 8 * tn, high = min(8, tm - group * 8);
  *m = group * 8 + r % high;
  *n = r / high;
}

template <typename T, int FB>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, FB == 4 ? 1 : 2)))
void k_q8_tile(LinDev p, int tn, int tm, bool wide) {
  constexpr int TL = 64 * FB, R = 4 * FB, STAGE = 2 * TL * LT_P;  // R loads of 32 rows for both operands
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, half = lane >> 5, l32 = lane & 31;
  int nt, mt;
  tile_of(blockIdx.x, tn, tm, &nt, &mt);
  const int n0 = nt * TL, m0 = mt * TL;
  const int lr = threadIdx.x >> 3, lk = 16 * (threadIdx.x & 7);  // row of a pass of 32, byte in the row
  const int wrows = min(TL, p.N - n0), xrows = min(TL, p.M - m0);
  const auto wb = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p.w) + (long long)n0 * p.w_stride, (short)0,
                                                    (int)((wrows - 1) * p.w_stride + p.K), 0x00020000);
  const auto xb = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p.x) + (long long)m0 * p.x_stride, (short)0,
                                                    (int)((xrows - 1) * p.x_stride + p.K), 0x00020000);
  uint32_t at[R];  // rows past the last read it again
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    at[i] = (uint32_t)(min(lr + 32 * i, wrows - 1) * (int)p.w_stride + lk);
    at[R / 2 + i] = (uint32_t)(min(lr + 32 * i, xrows - 1) * (int)p.x_stride + lk);
  }
  u32x4 r[R];
  auto load = [&](int i, int k0) {
    const uint32_t o = k0 + lk < p.K ? at[i] + k0 : LT_OOB;
    r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(i < R / 2 ? wb : xb, o, 0, 0));
  };
  auto store = [&](int i, int s) { *reinterpret_cast<u32x4*>(lds + s * STAGE + (lr + 32 * i) * LT_P + lk) = r[i]; };
  i32x16 acc[FB][FB];
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = (i32x16){};
  const int wn = 32 * FB * (wave & 1), wm = 32 * FB * (wave >> 1);
  const int steps = (p.K + LT_K - 1) / LT_K;
#pragma unroll
  for (int i = 0; i < R; ++i) load(i, 0);
#pragma unroll
  for (int i = 0; i < R; ++i) store(i, 0);
#pragma unroll
  for (int i = 0; i < R; ++i) load(i, LT_K);  // zeros past K
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const uint8_t* base = lds + (s & 1) * STAGE + l32 * LT_P + 16 * half;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      i32x4 a[FB], b[FB];
#pragma unroll
      for (int i = 0; i < FB; ++i) {
        a[i] = *reinterpret_cast<const i32x4*>(base + (wn + 32 * i) * LT_P + 32 * k);
        b[i] = *reinterpret_cast<const i32x4*>(base + (TL + wm + 32 * i) * LT_P + 32 * k);
      }
#pragma unroll
      for (int i = 0; i < R / 4; ++i) {
        store(k * (R / 4) + i, (s + 1) & 1);
        load(k * (R / 4) + i, (s + 2) * LT_K);
      }
#pragma unroll
      for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = n0 + wn + 32 * i + 8 * q + 4 * half;
      float ws[4], bias[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = min(n + e, p.N - 1);
        ws[e] = p.ws[c];
        bias[e] = p.bias != nullptr ? p.bias[c] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < FB; ++j)
        put4<T>(p, m0 + wm + 32 * j + l32, n, ws, bias,
                (i32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]}, wide);
    }
}

template <typename T, int FB>
pi_status launch_tile(pi_ctx* c, const LinDev& p, bool wide) {
  const int tn = (p.N + 64 * FB - 1) / (64 * FB), tm = (p.M + 64 * FB - 1) / (64 * FB);
  PI_HIP(c, allow_lds(k_q8_tile<T, FB>, tile_lds<FB>()));
  PI_HIP(c, launch_kb(c, 0, k_q8_tile<T, FB>, dim3((unsigned)(tn * tm)), 256, tile_lds<FB>(), p, tn, tm, wide));
  return PI_OK;
}

template <typename T>
pi_status launch_linear(pi_ctx* c, const LinDev& p) {
  // 4 outputs in one store where every row starts at such a boundary
  const bool wide = p.y_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(T) - 1)) == 0;
  // a tile's rows are addressed by 32-bit offsets
  if (p.M > 256 && p.x_stride < (1 << 22) && p.w_stride < (1 << 22)) {
    const long long big = (long long)((p.N + 255) / 256) * ((p.M + 255) / 256);
    return big >= c->cus ? launch_tile<T, 4>(c, p, wide) : launch_tile<T, 2>(c, p, wide);
  }
  const int mb = std::min(4, (p.M + 15) / 16);
  const dim3 g((p.N + 31) / 32, (p.M + 16 * mb - 1) / (16 * mb));
  switch (mb) {
    case 1: PI_HIP(c, launch_kb(c, 0, k_q8_rows<T, 1, 2>, g, 64 * LR_WAVES, 0, p, wide)); break;
    case 2: PI_HIP(c, launch_kb(c, 0, k_q8_rows<T, 2, 2>, g, 64 * LR_WAVES, 0, p, wide)); break;
    case 3: PI_HIP(c, launch_kb(c, 0, k_q8_rows<T, 3, 2>, g, 64 * LR_WAVES, 0, p, wide)); break;
    default: PI_HIP(c, launch_kb(c, 0, k_q8_rows<T, 4, 2>, g, 64 * LR_WAVES, 0, p, wide));
  }
  return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_linear_create(pi_ctx* ctx, const pi_linear_desc* desc, pi_linear** out) {
  if (ctx == nullptr || out == nullptr) return PI_ERR_INVALID;
  *out = nullptr;
  if (desc == nullptr) return fail(ctx, PI_ERR_INVALID, "desc is NULL");
  const pi_linear_desc& d = *desc;
  if (d.N < 1 || d.K < 16 || d.K % 16) return fail(ctx, PI_ERR_INVALID, "bad shape N=%d K=%d: K is a multiple of 16", d.N, d.K);
  if (d.K >= 131072) return fail(ctx, PI_ERR_UNSUPPORTED, "K %d: sums are exact below 131072", d.K);
  if (d.max_tokens < 1) return fail(ctx, PI_ERR_INVALID, "max_tokens %d", d.max_tokens);
  if (d.w_stride < d.K || d.w_stride % 16)
    return fail(ctx, PI_ERR_INVALID, "w_stride %lld must be a multiple of 16 and at least K", (long long)d.w_stride);
  PI_TRY(check_dev_ptr(ctx, d.w, "w"));
  PI_TRY(check_dev_ptr(ctx, d.w_scale, "w_scale"));
  PI_TRY(check_dev_ptr(ctx, d.bias, "bias", true));
  pi_linear* l = new (std::nothrow) pi_linear{ctx, d};
  if (l == nullptr) return fail(ctx, PI_ERR_OOM, "host allocation failed");
  *out = l;
  return PI_OK;
}

void pi_linear_destroy(pi_linear* lin) { delete lin; }

pi_status pi_linear_q8(pi_ctx* ctx, pi_linear* lin, const int8_t* x, int64_t x_stride, const float* x_scale, int32_t M,
                       void* y, int32_t y_dtype, int64_t y_stride) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (lin == nullptr) return fail(ctx, PI_ERR_INVALID, "lin is NULL");
  if (lin->ctx != ctx) return fail(ctx, PI_ERR_INVALID, "lin belongs to another context");
  const pi_linear_desc& d = lin->desc;
  if (M < 0 || M > d.max_tokens) return fail(ctx, PI_ERR_INVALID, "M %d out of range 0..%d", M, d.max_tokens);
  if (y_dtype != PI_T_F32 && y_dtype != PI_T_F16 && y_dtype != PI_T_BF16)
    return fail(ctx, PI_ERR_INVALID, "y: unknown dtype %d", y_dtype);
  if (M > 1 && (x_stride < d.K || x_stride % 16))
    return fail(ctx, PI_ERR_INVALID, "x_stride %lld must be a multiple of 16 and at least K", (long long)x_stride);
  if (M > 1 && y_stride < d.N) return fail(ctx, PI_ERR_INVALID, "y_stride %lld below N %d", (long long)y_stride, d.N);
  if (M == 0) return PI_OK;
  PI_TRY(check_dev_ptr(ctx, x, "x"));
  if (x_scale == nullptr || y == nullptr) return fail(ctx, PI_ERR_INVALID, "NULL pointer");
  if ((reinterpret_cast<uintptr_t>(x_scale) & 3u) || (reinterpret_cast<uintptr_t>(y) & (y_dtype == PI_T_F32 ? 3u : 1u)))
    return fail(ctx, PI_ERR_INVALID, "x_scale or y is not aligned to its elements");
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const LinDev p{x, d.w, x_scale, d.w_scale, d.bias, y, x_stride, d.w_stride, y_stride, M, d.N, d.K};
  switch (y_dtype) {
    case PI_T_F32: return launch_linear<float>(ctx, p);
    case PI_T_F16: return launch_linear<half_t>(ctx, p);
    default: return launch_linear<bf16_t>(ctx, p);
  }
}

}  // extern "C"
