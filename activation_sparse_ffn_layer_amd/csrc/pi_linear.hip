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

constexpr long long LIN_STRIDE = 1 << 22;  // a tile's rows (256 at most) have 32-bit offsets

struct LinDev {
  const int8_t *x, *w;
  const float *xs, *ws, *bias;
  void* y;
  long long x_stride, w_stride, y_stride;
  int M, N, K;
};

// Rows [r0, r0 + rows) of K bytes each as a bounds-checked buffer.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const int8_t* base, int r0, int rows, long long stride, int K) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base) + (long long)r0 * stride, (short)0,
                                           (int)((rows - 1) * stride + K), 0x00020000);
}
constexpr uint32_t OOB = 0xC0000000u;  // past any buffer's end: reads as zero
template <int AUX>
__device__ __forceinline__ u32x4 buffer16(__amdgpu_buffer_rsrc_t b, uint32_t offset) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, offset, 0, AUX));
}

template <typename T> struct Vec4 { typedef T type __attribute__((ext_vector_type(4))); };

// y[m][n0..n0+3] from 4 whole-number sums and their channels' scales and biases
template <typename T, bool IN = false>
__device__ __forceinline__ void put4(const LinDev& p, int m, int n0, const float (&ws)[4], const float (&bias)[4], i32x4 s,
                                     bool wide) {
  if (!IN && (m >= p.M || n0 >= p.N)) return;
  const float xs = p.xs[m];
  T* y = static_cast<T*>(p.y) + (long long)m * p.y_stride + n0;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)s[i] * xs * ws[i] + bias[i];
  if (IN || (wide && n0 + 3 < p.N)) {
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
// tokens; its waves deal the K axis in pieces of 128 among themselves, each lane reading 16
// bytes of a row straight into the operand's layout (no LDS), with the next piece's loads in
// flight during a piece's products, and add their sums in LDS. Workgroups start at different
// pieces: rows lie a power of two apart more often than not, and all of them at the same
// offset of K would meet in the same few memory channels.
// ---------------------------------------------------------------------------------------
constexpr int LR_WAVES = 8, LR_U = 2, LR_PIECE = 64 * LR_U;

template <typename T, int MB, int RB>
__global__ __launch_bounds__(64 * LR_WAVES) void k_q8_rows(LinDev p, bool wide) {
  __shared__ i32x4 red[LR_WAVES][RB * MB][WAVE];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, l16 = lane & 15;
  const int n0 = blockIdx.x * 16 * RB, m0 = blockIdx.y * 16 * MB;
  const int ko = 16 * (lane >> 4);
  // bounds-checked buffers: what lies past K reads as zero, rows past the last read it again
  const int wrows = min(16 * RB, p.N - n0), xrows = min(16 * MB, p.M - m0);
  const auto wb = row_buffer(p.w, n0, wrows, p.w_stride, p.K), xb = row_buffer(p.x, m0, xrows, p.x_stride, p.K);
  uint32_t wr[RB], xr[MB];
#pragma unroll
  for (int i = 0; i < RB; ++i) wr[i] = (uint32_t)(min(16 * i + l16, wrows - 1) * (int)p.w_stride);
#pragma unroll
  for (int j = 0; j < MB; ++j) xr[j] = (uint32_t)(min(16 * j + l16, xrows - 1) * (int)p.x_stride);
  i32x4 acc[RB][MB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  const int pieces = (p.K + LR_PIECE - 1) / LR_PIECE, turn = (int)(blockIdx.x * 5u % (uint32_t)pieces);
  u32x4 a[2][LR_U][RB], b[2][LR_U][MB];
  auto load = [&](int set, int i) {
    int at = i + turn;
    at -= at >= pieces ? pieces : 0;
#pragma unroll
    for (int u = 0; u < LR_U; ++u) {
      const int k = LR_PIECE * at + 64 * u + ko;
      const bool in = i < pieces && k < p.K;
#pragma unroll
      for (int r = 0; r < RB; ++r) a[set][u][r] = buffer16<2>(wb, in ? wr[r] + k : OOB);  // streamed
#pragma unroll
      for (int j = 0; j < MB; ++j) b[set][u][j] = buffer16<0>(xb, in ? xr[j] + k : OOB);
    }
  };
  auto products = [&](int set) {
#pragma unroll
    for (int u = 0; u < LR_U; ++u)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a[set][u][i]),
                                                            __builtin_bit_cast(i32x4, b[set][u][j]), acc[i][j], 0, 0, 0);
  };
  // the barriers keep the compiler from moving a piece's loads behind the products before it
  load(0, wave);
  for (int i = wave; i < pieces; i += 2 * LR_WAVES) {
    load(1, i + LR_WAVES);
    __builtin_amdgcn_sched_barrier(0);
    products(0);
    __builtin_amdgcn_sched_barrier(0);
    load(0, i + 2 * LR_WAVES);
    __builtin_amdgcn_sched_barrier(0);
    products(1);
    __builtin_amdgcn_sched_barrier(0);
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
// tokens, staged in LDS 64 bytes of K at a time in three stages. In step s the products of
// stage s run, with the operands of the next 32 bytes of K read ahead (also across the step's
// barrier: stage s + 1 is complete), stage s + 2 is written from registers, and those are
// loaded anew, two steps before they are needed. A wave's quarter of the tile is FB x FB blocks
// of 32 x 32, so LDS is read 2 FB rows for FB^2 products.
// ---------------------------------------------------------------------------------------
constexpr int LT_K = 64, LT_P = LT_K + 16;  // K bytes per stage; LDS row pitch (bytes)
template <int FB> constexpr size_t tile_lds() { return (size_t)3 * 2 * 64 * FB * LT_P; }

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
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(FB == 4 ? 1 : 2, FB == 4 ? 1 : 2)))
void k_q8_tile(LinDev p, int tn, int tm, bool wide) {
  constexpr int TL = 64 * FB, R = 2 * FB, STAGE = 2 * TL * LT_P;  // R loads of 64 rows for both operands
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, half = lane >> 5, l32 = lane & 31;
  int nt, mt;
  tile_of(blockIdx.x, tn, tm, &nt, &mt);
  const int n0 = nt * TL, m0 = mt * TL;
  const int lr = threadIdx.x >> 2, lk = 16 * (threadIdx.x & 3);  // row of a pass of 64, byte in the row
  const int wrows = min(TL, p.N - n0), xrows = min(TL, p.M - m0);
  const auto wb = row_buffer(p.w, n0, wrows, p.w_stride, p.K), xb = row_buffer(p.x, m0, xrows, p.x_stride, p.K);
  uint32_t at[R];  // rows past the last read it again
#pragma unroll
  for (int i = 0; i < FB; ++i) {
    at[i] = (uint32_t)(min(lr + 64 * i, wrows - 1) * (int)p.w_stride + lk);
    at[FB + i] = (uint32_t)(min(lr + 64 * i, xrows - 1) * (int)p.x_stride + lk);
  }
  u32x4 r[2][R];
  auto load = [&](int set, int i, int k0) {
    r[set][i] = buffer16<0>(i < FB ? wb : xb, k0 + lk < p.K ? at[i] + k0 : OOB);
  };
  uint8_t* const put = lds + lr * LT_P + lk;
  auto store = [&](int set, int i, int stage) { *reinterpret_cast<u32x4*>(put + stage + 64 * i * LT_P) = r[set][i]; };
  const int wn = 32 * FB * (wave & 1), wm = 32 * FB * (wave >> 1);
  const uint8_t* const ga = lds + (wn + l32) * LT_P + 16 * half;
  const uint8_t* const gb = lds + (TL + wm + l32) * LT_P + 16 * half;
  i32x4 a[2][FB], b[2][FB];
  auto fetch = [&](int set, int at_) {
#pragma unroll
    for (int i = 0; i < FB; ++i) {
      a[set][i] = *reinterpret_cast<const i32x4*>(ga + at_ + 32 * i * LT_P);
      b[set][i] = *reinterpret_cast<const i32x4*>(gb + at_ + 32 * i * LT_P);
    }
  };
  i32x16 acc[FB][FB];
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = (i32x16){};
  auto products = [&](int set) {
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[set][i], b[set][j], acc[i][j], 0, 0, 0);
  };
  const int steps = (p.K + LT_K - 1) / LT_K;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < R; ++i) load(h, i, h * LT_K);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < R; ++i) store(h, i, h * STAGE);
#pragma unroll
    for (int i = 0; i < R; ++i) load(h, i, (h + 2) * LT_K);  // zeros past K
  }
  __syncthreads();
  int s0 = 0, s1 = STAGE, s2 = 2 * STAGE;  // stages s, s + 1, s + 2
  fetch(0, 0);
  // one step; registers h hold stage s + 2
  auto step = [&](int s, int h) {
    fetch(1, s0 + 32);
#pragma unroll
    for (int i = 0; i < R / 2; ++i) store(h, i, s2);
    products(0);
    fetch(0, s1);
#pragma unroll
    for (int i = R / 2; i < R; ++i) store(h, i, s2);
#pragma unroll
    for (int i = 0; i < R; ++i) load(h, i, (s + 4) * LT_K);
    products(1);
    if constexpr (FB == 4) {  // the memory operations between the products, so that neither waits for the other
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // read of LDS
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // product
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // write to LDS
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (g == 1) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);  // load
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
      }
    }
    __syncthreads();
    const int t = s0;
    s0 = s1;
    s1 = s2;
    s2 = t;
  };
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    step(s, 0);
    step(s + 1, 1);
  }
  if (s < steps) step(s, 0);
  const bool whole = wide && n0 + TL <= p.N && m0 + TL <= p.M;
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
      for (int j = 0; j < FB; ++j) {
        const i32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (whole) put4<T, true>(p, m0 + wm + 32 * j + l32, n, ws, bias, v, true);
        else put4<T, false>(p, m0 + wm + 32 * j + l32, n, ws, bias, v, wide);
      }
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
  if (p.M > 256) {
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
  if (d.w_stride >= LIN_STRIDE) return fail(ctx, PI_ERR_UNSUPPORTED, "w_stride %lld: rows are below 2^22 apart", (long long)d.w_stride);
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
  if (M > 1 && x_stride >= LIN_STRIDE)
    return fail(ctx, PI_ERR_UNSUPPORTED, "x_stride %lld: rows are below 2^22 apart", (long long)x_stride);
  if (M > 1 && y_stride < d.N) return fail(ctx, PI_ERR_INVALID, "y_stride %lld below N %d", (long long)y_stride, d.N);
  if (M == 0) return PI_OK;
  PI_TRY(check_dev_ptr(ctx, x, "x"));
  if (x_scale == nullptr || y == nullptr) return fail(ctx, PI_ERR_INVALID, "NULL pointer");
  if ((reinterpret_cast<uintptr_t>(x_scale) & 3u) || (reinterpret_cast<uintptr_t>(y) & (y_dtype == PI_T_F32 ? 3u : 1u)))
    return fail(ctx, PI_ERR_INVALID, "x_scale or y is not aligned to its elements");
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const LinDev p{x, d.w, x_scale, d.w_scale, d.bias, y, M > 1 ? x_stride : 0, d.w_stride, y_stride, M, d.N, d.K};
  switch (y_dtype) {
    case PI_T_F32: return launch_linear<float>(ctx, p);
    case PI_T_F16: return launch_linear<half_t>(ctx, p);
    default: return launch_linear<bf16_t>(ctx, p);
  }
}

}  // extern "C"
