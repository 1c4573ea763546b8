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

// y[m][n0..n0+3] from 4 whole-number sums
template <typename T>
__device__ __forceinline__ void put4(const LinDev& p, int m, int n0, i32x4 s, bool wide) {
  if (m >= p.M || n0 >= p.N) return;
  const float xs = p.xs[m];
  T* y = static_cast<T*>(p.y) + (long long)m * p.y_stride + n0;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, p.N - 1);
    v[i] = (float)s[i] * xs * p.ws[n] + (p.bias != nullptr ? p.bias[n] : 0.f);
  }
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
// Many tokens: bound by the matrix cores. A workgroup owns a tile of TN weight rows x TM
// tokens, staged in LDS 128 bytes of K at a time (two stages: the next one's loads are in
// flight during the products).
// ---------------------------------------------------------------------------------------
constexpr int LT_K = 128, LT_P = LT_K + 16;  // K bytes per stage; LDS row pitch (bytes)

template <typename T>
__global__ __launch_bounds__(256) void k_q8_tile(LinDev p, bool wide) {
  constexpr int TN = 128, TM = 128;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][(TN + TM) * LT_P];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, half = lane >> 5, l32 = lane & 31;
  const int n0 = blockIdx.x * TN, m0 = blockIdx.y * TM;
  const int lr = threadIdx.x >> 3, lk = 16 * (threadIdx.x & 7);  // row of a pass of 32, byte in the row
  const int8_t* src[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    src[i] = p.w + (long long)min(n0 + lr + 32 * i, p.N - 1) * p.w_stride;
    src[4 + i] = p.x + (long long)min(m0 + lr + 32 * i, p.M - 1) * p.x_stride;
  }
  u32x4 r[8];
  auto load = [&](int k0) {
    const bool in = k0 + lk < p.K;
    const int k = in ? k0 + lk : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = ld16_or0(src[i] + k, in);
  };
  auto store = [&](int s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<u32x4*>(&lds[s][(lr + 32 * i) * LT_P + lk]) = r[i];
  };
  i32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (i32x16){};
  const int wn = 64 * (wave & 1), wm = 64 * (wave >> 1);
  const int steps = (p.K + LT_K - 1) / LT_K;
  load(0);
  store(0);
  if (steps > 1) load(LT_K);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const uint8_t* base = lds[s & 1] + l32 * LT_P + 16 * half;
#pragma unroll
    for (int k = 0; k < LT_K; k += 32) {
      i32x4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const i32x4*>(base + (wn + 32 * i) * LT_P + k);
        b[i] = *reinterpret_cast<const i32x4*>(base + (TN + wm + 32 * i) * LT_P + k);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < steps) store((s + 1) & 1);
    if (s + 2 < steps) load((s + 2) * LT_K);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        put4<T>(p, m0 + wm + 32 * j + l32, n0 + wn + 32 * i + 8 * q + 4 * half,
                (i32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]}, wide);
}

template <typename T>
pi_status launch_linear(pi_ctx* c, const LinDev& p) {
  // 4 outputs in one store where every row starts at such a boundary
  const bool wide = p.y_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(T) - 1)) == 0;
  if (p.M > 256) {
    PI_HIP(c, launch_k(c, 0, k_q8_tile<T>, dim3((p.N + 127) / 128, (p.M + 127) / 128), 0, p, wide));
    return PI_OK;
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
