// The residual's addition and RMS norm with an 8-bit output (pi_add_rmsnorm).
//
// r = round(x + res), y = r / sqrt(mean(r^2) + eps) * w, scale = max|y| / 127, q = round(y / scale).
// Bound by memory: a row is read once, kept in registers between its three steps (sum of
// squares, maximum, output) and written once. 4096 rows of 8192 in fp16, 235 MB: 47 to 49 us, 4.9 TB/s,
// the rate of a plain copy; 8 rows of 4096: 4.4 us, the latency of a load, two sums over the
// workgroup and a store. One workgroup per row, 8 columns per thread and
// step; the two sums over the row go through LDS.
#include "pi_host.hpp"
#include "pi_types.hpp"

using namespace pi;

namespace {

struct NormDev {
  const void *x, *res;
  void *res_out, *y;
  const float* w;
  int8_t* q;
  float* scale;
  long long xs, rs, ros, qs, ys;
  float eps;
  int d, y_dtype;
};

// Sum and maximum over the workgroup's NW waves; red holds NW floats and is free on entry.
template <int NW, bool MAX>
__device__ __forceinline__ float block_fold(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float t = __shfl_xor(v, o, WAVE);
    v = MAX ? fmaxf(v, t) : v + t;
  }
  if constexpr (NW == 1) return v;
  if (threadIdx.x % WAVE == 0) red[threadIdx.x / WAVE] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) s = MAX ? fmaxf(s, red[i]) : s + red[i];
  return s;
}

// J steps of 8 columns per thread; d <= 8 * J * NT.
template <typename TX, typename TR, bool RES, int NT, int J>
__global__ __launch_bounds__(NT) void k_add_rmsnorm(NormDev p) {
  constexpr int NW = NT / WAVE;
  __shared__ float red[2][NW];
  const long long row = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + row * p.xs;
  const TR* res = RES ? static_cast<const TR*>(p.res) + row * p.rs : nullptr;
  TR* ro = static_cast<TR*>(p.res_out) + row * p.ros;
  float h[J][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = 8 * (threadIdx.x + j * NT);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
    if (c < p.d) {
      load8(x + c, h[j]);
      if constexpr (RES) {
        float r[8];
        load8(res + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = (float)(TR)h[j][i];  // the norm is of the residual as stored
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = 8 * (threadIdx.x + j * NT);
    if (c < p.d) store8(ro + c, h[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += h[j][i] * h[j][i];
  }
  ss = block_fold<NW, false>(ss, red[0]);
  const float mean = ss / (float)p.d + p.eps;
  float rinv = mean > 0.f ? 1.0f / sqrtf(mean) : 0.f;  // a row of zeros, without eps: zeros
  bool bad = !(ss < __builtin_inff());
  if (bad || mean < 1e-30f) {
    // Squares beyond fp32's range, or lost below it: again with the row times a power of two that
    // brings its largest element, or eps's root where that is larger, near 1. The scaled row is what
    // goes on: the root's reciprocal for the row as it is may lie beyond the range. A NaN makes the
    // sum one; an infinity is its row's largest.
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(h[j][i]));
    big = block_fold<NW, true>(big, red[1]);
    bad = ss != ss || !(big < __builtin_inff());
    if (!bad && big > 0.f) {
      const int e = -ilogbf(fmaxf(big, sqrtf(p.eps)));
      float s2 = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[j][i] = ldexpf(h[j][i], e);
          s2 += h[j][i] * h[j][i];
        }
      __syncthreads();  // red is free again
      s2 = block_fold<NW, false>(s2, red[0]);
      rinv = 1.0f / sqrtf(s2 / (float)p.d + ldexpf(ldexpf(p.eps, e), e));
    }
    __syncthreads();
  }
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = 8 * (threadIdx.x + j * NT);
    if (c < p.d) {
      float w[8];
      load8(p.w + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[j][i] = h[j][i] * rinv * w[i];
        top = fmaxf(top, fabsf(h[j][i]));
      }
      if (p.y != nullptr) {
        if (p.y_dtype == PI_T_F16) store8(static_cast<half_t*>(p.y) + row * p.ys + c, h[j]);
        else if (p.y_dtype == PI_T_BF16) store8(static_cast<bf16_t*>(p.y) + row * p.ys + c, h[j]);
        else store8(static_cast<float*>(p.y) + row * p.ys + c, h[j]);
      }
    }
  }
  if (p.q == nullptr) return;
  top = block_fold<NW, true>(top, red[1]);
  // a row with an infinity or a NaN has no scale: NaN, and zeros beside it
  const float scale = top / 127.0f;
  // Each value is divided by the scale. Its product with the scale's rounded reciprocal alone lands a step
  // off next to a tie; corrected by that product's remainder, which is exact, it is the rounded quotient
  // (Markstein): 36 us, where a division took 39 (4096 rows of 8192 again and again). Where the scale is
  // so small that the remainder loses bits or the reciprocal is infinite, both are raised first, exactly;
  // values beyond 127 of a scale that has lost its own bits stay at 127.
  float by = scale > 0.f ? scale : 1.f;
  if (by < 0x1p-100f) {
    by *= 0x1p100f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = fminf(fmaxf(h[j][i] * 0x1p100f, -127.f * by), 127.f * by);
  }
  const float inv = 1.0f / by;
  if (threadIdx.x == 0) p.scale[row] = bad ? __builtin_nanf("") : scale;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = 8 * (threadIdx.x + j * NT);
    if (c < p.d) {
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // |q| is at most 127 (1 + 2^-22), which rounds to 127; a scale that became 0 has zeros beside it
        const float q = h[j][i] * inv;
        const int v = bad ? 0 : (int)rintf(__builtin_fmaf(__builtin_fmaf(-q, by, h[j][i]), inv, q));
        o[i >> 2] |= (uint32_t)(v & 0xFF) << (8 * (i & 3));
      }
      *reinterpret_cast<uint2*>(p.q + row * p.qs + c) = make_uint2(o[0], o[1]);
    }
  }
}

template <typename TX, typename TR, bool RES>
pi_status launch_norm(pi_ctx* c, const NormDev& p, int T) {
  const int steps = (p.d + 7) / 8;
  const dim3 g(T);
  if (steps <= 64) PI_HIP(c, launch_kb(c, 0, k_add_rmsnorm<TX, TR, RES, 64, 1>, g, 64, 0, p));
  else if (steps <= 256) PI_HIP(c, launch_kb(c, 0, k_add_rmsnorm<TX, TR, RES, 256, 1>, g, 256, 0, p));
  else if (steps <= 512) PI_HIP(c, launch_kb(c, 0, k_add_rmsnorm<TX, TR, RES, 256, 2>, g, 256, 0, p));
  else if (steps <= 1024) PI_HIP(c, launch_kb(c, 0, k_add_rmsnorm<TX, TR, RES, 256, 4>, g, 256, 0, p));
  else if (steps <= 2048) PI_HIP(c, launch_kb(c, 0, k_add_rmsnorm<TX, TR, RES, 512, 4>, g, 512, 0, p));
  else PI_HIP(c, launch_kb(c, 0, k_add_rmsnorm<TX, TR, RES, 1024, 4>, g, 1024, 0, p));
  return PI_OK;
}

template <typename TX>
pi_status launch_norm_x(pi_ctx* c, const NormDev& p, int T, int res_dtype) {
  if (p.res == nullptr) return launch_norm<TX, TX, false>(c, p, T);
  switch (res_dtype) {
    case PI_T_F32: return launch_norm<TX, float, true>(c, p, T);
    case PI_T_F16: return launch_norm<TX, half_t, true>(c, p, T);
    default: return launch_norm<TX, bf16_t, true>(c, p, T);
  }
}

bool dtype_ok(int t) { return t == PI_T_F32 || t == PI_T_F16 || t == PI_T_BF16; }

// A row stride of d columns of a type whose rows stay 16-byte aligned.
pi_status check_rows(pi_ctx* c, const char* name, int dtype, int64_t stride, int d, int T) {
  if (!dtype_ok(dtype)) return fail(c, PI_ERR_INVALID, "%s: unknown dtype %d", name, dtype);
  if (T > 1 && (stride < d || stride % (dtype == PI_T_F32 ? 4 : 8)))
    return fail(c, PI_ERR_INVALID, "%s: row stride %lld must be at least %d and keep rows 16-byte aligned", name,
                (long long)stride, d);
  return PI_OK;
}

}  // namespace

extern "C" pi_status pi_add_rmsnorm(pi_ctx* ctx, const pi_norm_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_norm_args& a = *args;
  if (a.T < 0 || a.d < 8 || a.d % 8) return fail(ctx, PI_ERR_INVALID, "bad shape T=%d d=%d", a.T, a.d);
  if (a.d > 32768) return fail(ctx, PI_ERR_UNSUPPORTED, "d %d above 32768", a.d);
  if (!(a.eps >= 0.f) || a.eps > 3e38f) return fail(ctx, PI_ERR_INVALID, "eps must be finite and not negative");
  if ((a.q == nullptr) != (a.scale == nullptr)) return fail(ctx, PI_ERR_INVALID, "q and scale go together");
  const int rt = a.res != nullptr ? a.res_dtype : a.x_dtype;
  PI_TRY(check_rows(ctx, "x", a.x_dtype, a.x_stride, a.d, a.T));
  PI_TRY(check_rows(ctx, "res_out", rt, a.res_out_stride, a.d, a.T));
  if (a.res != nullptr) PI_TRY(check_rows(ctx, "res", rt, a.res_stride, a.d, a.T));
  if (a.y != nullptr) PI_TRY(check_rows(ctx, "y", a.y_dtype, a.y_stride, a.d, a.T));
  if (a.T == 0) return PI_OK;
  PI_TRY(check_dev_ptr(ctx, a.x, "x"));
  PI_TRY(check_dev_ptr(ctx, a.res, "res", true));
  PI_TRY(check_dev_ptr(ctx, a.res_out, "res_out"));
  PI_TRY(check_dev_ptr(ctx, a.w, "w"));
  PI_TRY(check_dev_ptr(ctx, a.y, "y", true));
  if (a.q != nullptr) {
    if ((reinterpret_cast<uintptr_t>(a.q) & 7u) || (a.T > 1 && (a.q_stride < a.d || a.q_stride % 8)))
      return fail(ctx, PI_ERR_INVALID, "q: rows must be 8-byte aligned and at least d apart");
    if (reinterpret_cast<uintptr_t>(a.scale) & 3u) return fail(ctx, PI_ERR_INVALID, "scale is not 4-byte aligned");
  }
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const NormDev p{a.x, a.res, a.res_out, a.y, a.w, a.q, a.scale, a.x_stride, a.res_stride, a.res_out_stride,
                  a.q_stride, a.y_stride, a.eps, a.d, a.y_dtype};
  switch (a.x_dtype) {
    case PI_T_F32: return launch_norm_x<float>(ctx, p, a.T, rt);
    case PI_T_F16: return launch_norm_x<half_t>(ctx, p, a.T, rt);
    default: return launch_norm_x<bf16_t>(ctx, p, a.T, rt);
  }
}
