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
  int32_t* part;  // sums of ranges of K
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
__device__ __forceinline__ void scales4(const LinDev& p, int n0, float (&ws)[4], float (&bias)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, p.N - 1);
    ws[i] = p.ws[n];
    bias[i] = p.bias != nullptr ? p.bias[n] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put4(const LinDev& p, int m, int n0, i32x4 s, bool wide) {
  float ws[4], bias[4];
  scales4(p, n0, ws, bias);
  put4<T>(p, m, n0, ws, bias, s, wide);
}

// ---------------------------------------------------------------------------------------
// Few tokens: bound by the weights' bytes. A workgroup owns 16 RB weight rows and 16 MB
// tokens; its waves deal the K axis in pieces of 128 among themselves, each lane reading 16
// bytes of a row straight into the operand's layout (no LDS), with the next piece's loads in
// flight during a piece's products, and add their sums in LDS. Workgroups start at different
// pieces: rows lie a power of two apart more often than not, and all of them at the same
// offset of K would meet in the same few memory channels. 16 rows per workgroup rather than 32, for
// even shares of the CUs: one token of 12288 x 4096 10.5 us (4.8 TB/s) against 12.6.
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
// More tokens: four waves own a square tile of 64 FB weight rows and tokens, staged in LDS 128
// bytes of K at a time in two stages. A step's products take the stage 32 bytes at a time, with
// the operands of the next 32 bytes read ahead. Its one barrier stands before the last of the
// four: by then the stage has been read to its end and the other one is written, whose first
// operands the last products cover; and the stage just read is free for what the registers
// hold. So no wave waits for an LDS read or a load that it has just issued.
//   FB = 4: bound by the matrix cores (a wave's 128 x 128 take 8 reads of LDS for 16 products).
//   4096 tokens of 8192 x 8192: 276 to 310 us, 1.8 to 2.0 POP/s. The clock falls under it, to some
//   1.6 GHz: on zeros as data the same call takes 215 us; all loads from one cached place 307.
//   FB = 2: where tiles of 256 would leave CUs idle. With SPLIT, for few tiles, each is cut in
//   `splits` ranges of K, whose whole-number sums k_q8_join adds: bound by the loads' latency and
//   the weights' bytes. 48 tokens of 10240 x 8192: 18.5 us (4.6 TB/s) and 4.2 us for the sums,
//   against 50 us when each workgroup kept 32 rows and read all of x.
// Row r's piece c of 16 bytes lies at c ^ (r / 2 % 8), so that 16 rows' reads of one piece meet
// all 64 banks.
// ---------------------------------------------------------------------------------------
constexpr int LT_K = 128;  // K bytes per stage, which is a row of LDS
template <int FB> constexpr size_t tile_lds() { return (size_t)2 * 2 * 64 * FB * LT_K; }

// The tile of workgroup id: the XCDs (id % 8) take equal runs of tiles, in an order that
// walks 8 tiles of tokens, then the weight rows, so that an XCD's tiles in flight share rows.
__device__ __forceinline__ void tile_of(int id, int tn, int tm, int* n, int* m) {
  const int total = tn * tm, x = id & 7, each = total >> 3, more = total & 7;
  const int t = x * each + min(x, more) + (id >> 3);
  const int group = t / (8 * tn), r = t - group * 8 * tn, high = min(8, tm - group * 8);
  *m = group * 8 + r % high;
  *n = r / high;
}

template <typename T, int FB, bool SPLIT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(FB == 4 ? 1 : 2, FB == 4 ? 1 : 2)))
void k_q8_tile(LinDev p, int tn, int tm, bool wide) {
  constexpr int TL = 64 * FB, R = 4 * FB, STAGE = 2 * TL * LT_K;  // R loads of 32 rows for both operands
  constexpr int SETS = FB == 4 ? 1 : 2;                           // stages held in registers
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, half = lane >> 5, l32 = lane & 31;
  int nt, mt;
  tile_of(blockIdx.x, tn, tm, &nt, &mt);
  const int n0 = nt * TL, m0 = mt * TL;
  const int lr = threadIdx.x >> 3, lk = 16 * (threadIdx.x & 7);  // row of a pass of 32, byte in the row
  const int wrows = min(TL, p.N - n0), xrows = min(TL, p.M - m0);
  const auto wb = row_buffer(p.w, n0, wrows, p.w_stride, p.K), xb = row_buffer(p.x, m0, xrows, p.x_stride, p.K);
  uint32_t at[R];  // rows past the last read it again
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    at[i] = (uint32_t)(min(lr + 32 * i, wrows - 1) * (int)p.w_stride + lk);
    at[R / 2 + i] = (uint32_t)(min(lr + 32 * i, xrows - 1) * (int)p.x_stride + lk);
  }
  const int all = (p.K + LT_K - 1) / LT_K;
  const int first = SPLIT ? (int)((long long)all * blockIdx.y / gridDim.y) : 0;
  const int steps = (SPLIT ? (int)((long long)all * (blockIdx.y + 1) / gridDim.y) : all) - first;
  u32x4 r[SETS][R];
  auto load = [&](int set, int i, int step) {
    const int k0 = (first + step) * LT_K;
    r[set][i] = buffer16<0>(i < R / 2 ? wb : xb, step < steps && k0 + lk < p.K ? at[i] + k0 : OOB);
  };
  uint8_t* const put = lds + lr * LT_K + (lk ^ (lr >> 1 & 7) * 16);
  auto store = [&](int set, int i, int stage) { *reinterpret_cast<u32x4*>(put + stage * STAGE + 32 * i * LT_K) = r[set][i]; };
  const int wn = 32 * FB * (wave & 1), wm = 32 * FB * (wave >> 1);
  const uint8_t* const ga = lds + (wn + l32) * LT_K;
  const uint8_t* const gb = lds + (TL + wm + l32) * LT_K;
  const int piece = (half ^ (l32 >> 1 & 7)) * 16;  // of the first 32 bytes; of the k-th 32 at ^ 32 k
  i32x4 a[2][FB], b[2][FB];
  auto fetch = [&](int set, int stage, int k) {
    const int o = stage * STAGE + (piece ^ (32 * k));
#pragma unroll
    for (int i = 0; i < FB; ++i) {
      a[set][i] = *reinterpret_cast<const i32x4*>(ga + o + 32 * i * LT_K);
      b[set][i] = *reinterpret_cast<const i32x4*>(gb + o + 32 * i * LT_K);
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
  // a quarter of a stage's writes, and of the loads into their registers
  auto quarter = [&](int q, int stage, int set, int step) {
#pragma unroll
    for (int i = q * (R / 4); i < (q + 1) * (R / 4); ++i) {
      store(set, i, stage);
      load(set, i, step);
    }
  };
  // Order of a quarter: reads of LDS and products in turn, then writes and loads between products.
  auto order = [&]() {
    if constexpr (FB == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // read of LDS
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // product
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // write to LDS
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < R; ++i) load(0, i, 0);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    store(0, i, 0);
    load(0, i, SETS == 1 ? 1 : 2);
  }
  if constexpr (SETS == 2) {
#pragma unroll
    for (int i = 0; i < R; ++i) load(1, i, 1);
  }
  __syncthreads();
  fetch(0, 0, 0);
  // the last quarter of stage 1's writes is where a step before would have put the first
  quarter(0, 1, SETS - 1, SETS == 1 ? 2 : 3);
  // Step s from stage h; the other stage gets step s + 1 in the first three quarters (its first
  // quarter is written already), and this one the first quarter of step s + 2 in the last.
  auto step = [&](int s, int h) {
    constexpr int D = SETS;  // a register is loaded D steps after the one it held
    const int next = SETS == 1 ? 0 : h ^ 1, then = SETS == 1 ? 0 : h;
    fetch(1, h, 1);
    quarter(1, h ^ 1, next, s + 1 + D);
    products(0);
    order();
    fetch(0, h, 2);
    quarter(2, h ^ 1, next, s + 1 + D);
    products(1);
    order();
    fetch(1, h, 3);
    quarter(3, h ^ 1, next, s + 1 + D);
    products(0);
    order();
    __syncthreads();
    fetch(0, h ^ 1, 0);
    quarter(0, h, then, s + 2 + D);
    products(1);
    order();
  };
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    step(s, 0);
    step(s + 1, 1);
  }
  if (s < steps) step(s, 0);
  if constexpr (SPLIT) {
    const int Np = (p.N + 3) & ~3;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int m = m0 + wm + 32 * j + l32;
      if (m < p.M) {
        int32_t* o = p.part + ((long long)blockIdx.y * p.M + m) * Np;
#pragma unroll
        for (int i = 0; i < FB; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = n0 + wn + 32 * i + 8 * q + 4 * half;
            if (n < p.N)
              *reinterpret_cast<i32x4*>(o + n) = (i32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          }
      }
    }
    return;
  }
  const bool whole = wide && n0 + TL <= p.N && m0 + TL <= p.M;
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = n0 + wn + 32 * i + 8 * q + 4 * half;
      float ws[4], bias[4];
      scales4(p, n, ws, bias);
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        const i32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (whole) put4<T, true>(p, m0 + wm + 32 * j + l32, n, ws, bias, v, true);
        else put4<T, false>(p, m0 + wm + 32 * j + l32, n, ws, bias, v, wide);
      }
    }
}

// The sums of a tile's ranges of K, 4 channels of a token per thread.
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_q8_join(LinDev p, int splits, bool wide) {
  const int n = 4 * (blockIdx.x * BLOCK + threadIdx.x), m = blockIdx.y;
  if (n >= p.N) return;
  const int Np = (p.N + 3) & ~3;
  const int32_t* o = p.part + (long long)m * Np + n;
  const long long next = (long long)p.M * Np;
  i32x4 s = {0, 0, 0, 0};
  for (int i0 = 0; i0 < splits; i0 += 8) {
    i32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const i32x4*>(o + min(i0 + i, splits - 1) * next);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < splits) s += v[i];
  }
  put4<T>(p, m, n, s, wide);
}

template <typename T, int FB, bool SPLIT>
pi_status launch_tile(pi_ctx* c, const LinDev& p, bool wide, int splits) {
  const int tn = (p.N + 64 * FB - 1) / (64 * FB), tm = (p.M + 64 * FB - 1) / (64 * FB);
  PI_HIP(c, allow_lds(k_q8_tile<T, FB, SPLIT>, tile_lds<FB>()));
  PI_HIP(c, launch_kb(c, 0, k_q8_tile<T, FB, SPLIT>, dim3((unsigned)(tn * tm), splits), 256, tile_lds<FB>(), p, tn, tm, wide));
  if (SPLIT) PI_HIP(c, launch_k(c, 0, k_q8_join<T>, dim3(((p.N + 3) / 4 + BLOCK - 1) / BLOCK, p.M), 0, p, splits, wide));
  return PI_OK;
}

// Ranges of K that tiles of 128 are cut in: as many workgroups as two per CU take at once, each
// of four steps at least.
int split_count(int cus, int tiles, int K) {
  return std::max(1, std::min(2 * cus / tiles, (K + LT_K - 1) / LT_K / 4));
}

// Up to 16 tokens. Each workgroup of k_q8_rows reads all of x, which costs 4.4 us per 10^9 of M N K (the
// same at all six shapes measured); tiles read it once for 128 rows, but join their ranges' sums, 2 to
// 5 us, most where the weight is below 64 MB and a range is a few steps. Rows against tiles, us: K = 4096,
// N = 12288: 12.1 / 17.1 at one token, 15.4 / 17.8 at 16; K = 8192, N = 4096: 10.8 / 14.5 at 16; N = 10240:
// 20.6 / 21.7 at 2, 22.2 / 22.0 at 6, 23.1 / 22.2 at 8, 26.9 / 22.9 at 16; K = 4096, N = 32000: 29.7 / 30.5
// at 6, 34.2 / 31.2 at 12; K = 8192, N = 28672: 46.5 / 48.0 at 3, 51.9 / 49.0 at 8. Few rows of great length
// leave most CUs without any: K = 16384, N = 1024: 12.8 / 11.4 at 2, 17.2 / 12.2 at 16, but K = 8192: 8.8 /
// 9.3 at 8. One token has no use for tiles, nor their scratch.
bool by_rows(int M, int N, int K) {
  if (M == 1) return true;
  if (M > 16 || K > 8ll * N) return false;
  const long long weights = (long long)N * K;
  return weights < (1 << 26) || (M * K < 65536 && M * weights < 850000000);
}

template <typename T>
pi_status launch_linear(pi_ctx* c, const LinDev& p) {
  // 4 outputs in one store where every row starts at such a boundary
  const bool wide = p.y_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(T) - 1)) == 0;
  if (by_rows(p.M, p.N, p.K)) {
    PI_HIP(c, launch_kb(c, 0, k_q8_rows<T, 1, 1>, dim3((p.N + 15) / 16), 64 * LR_WAVES, 0, p, wide));
    return PI_OK;
  }
  const long long big = (long long)((p.N + 255) / 256) * ((p.M + 255) / 256);
  if (big >= c->cus) return launch_tile<T, 4, false>(c, p, wide, 1);
  const int splits = split_count(c->cus, ((p.N + 127) / 128) * ((p.M + 127) / 128), p.K);
  return splits > 1 ? launch_tile<T, 2, true>(c, p, wide, splits) : launch_tile<T, 2, false>(c, p, wide, 1);
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
  // one buffer per context: its calls run one after another
  if (d.max_tokens > 1 && ctx->lin_part == nullptr) {
    PI_HIP(ctx, hipSetDevice(ctx->device));
    const size_t bytes = (size_t)2 * ctx->cus * 128 * 128 * 4;
    if (hipMalloc(reinterpret_cast<void**>(&ctx->lin_part), bytes) != hipSuccess) {
      (void)hipGetLastError();
      ctx->lin_part = nullptr;
      return fail(ctx, PI_ERR_OOM, "product scratch of %zu bytes", bytes);
    }
  }
  pi_linear* l = new (std::nothrow) pi_linear{ctx, d};
  if (l == nullptr) return fail(ctx, PI_ERR_OOM, "host allocation failed");
  ctx_retain(ctx);
  *out = l;
  return PI_OK;
}

void pi_linear_destroy(pi_linear* lin) {
  if (lin == nullptr) return;
  ctx_release(lin->ctx);
  delete lin;
}

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
  const LinDev p{x, d.w, x_scale, d.w_scale, d.bias, y, ctx->lin_part, M > 1 ? x_stride : 0, d.w_stride, y_stride, M, d.N, d.K};
  switch (y_dtype) {
    case PI_T_F32: return launch_linear<float>(ctx, p);
    case PI_T_F16: return launch_linear<half_t>(ctx, p);
    default: return launch_linear<bf16_t>(ctx, p);
  }
}

}  // extern "C"
