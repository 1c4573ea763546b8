// RMS norm of query and key heads with rotary positions (pi_qk_norm_rope).
//
// y = x / sqrt(mean(x^2) + eps) * w per head, then each pair (a, b) of the first rot elements turns by
// pos * inv_freq: (a cos - b sin, b cos + a sin). Bound by memory: a head is read once, kept in
// registers and written once. A lane has the same 2U elements of every head it takes (U pairs: two
// pieces of U elements each, U * i and rot/2 + U * i, or 2U in a row where pairs are interleaved), so
// a token's sines and cosines are worked out once per wave and serve all its heads.
//
// The angle is a whole number times an fp32 number, exact in 64 bits up to 2^29 and off by 2^-53 of
// itself beyond; as turns, reduced by its nearest whole number, it goes on in fp32 (2^-25 of a turn).
#include "pi_host.hpp"
#include "pi_types.hpp"

using namespace pi;

namespace {

struct RopeSide {
  const void* x;
  void* y;
  const float* w;
  long long row, head, out_row, out_head;
};

struct RopeDev {
  RopeSide q, k;
  const int32_t* pos;
  const float* inv_freq;
  float eps;
  int heads, kv_heads, D, rot, per_wave;  // per_wave: heads that one wave takes, one group of lanes after another
};

template <typename T, int U> struct Piece { typedef T type __attribute__((ext_vector_type(U))); };

template <int U, typename T>
__device__ __forceinline__ void load_piece(const T* p, float (&o)[U]) {
  if constexpr (U == 8) {
    load8(p, o);
  } else {
    const auto v = *reinterpret_cast<const typename Piece<T, U>::type*>(p);
#pragma unroll
    for (int i = 0; i < U; ++i) o[i] = (float)v[i];
  }
}
template <int U, typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&o)[U]) {
  if constexpr (U == 8) {
    store8(p, o);
  } else {
    typename Piece<T, U>::type v;
#pragma unroll
    for (int i = 0; i < U; ++i) v[i] = (T)o[i];
    *reinterpret_cast<typename Piece<T, U>::type*>(p) = v;
  }
}

// LPH lanes per head, a power of two. Heads are numbered queries first, then keys.
template <typename TX, typename TY, int U, bool PAIRS, int LPH>
__global__ __launch_bounds__(BLOCK) void k_qk_norm_rope(RopeDev p) {
  constexpr int HPW = WAVE / LPH;  // heads of a wave at once
  const long long t = blockIdx.x;
  const int lane = threadIdx.x % WAVE, slot = lane % LPH;
  const int half = p.rot >> 1, turning = half / U;
  const bool turns = slot < turning, live = slot < p.D / (2 * U);
  int a0, b0;  // first elements of this lane's two pieces
  if (PAIRS || !turns) {
    a0 = 2 * U * slot;
    b0 = a0 + U;
  } else {
    a0 = U * slot;
    b0 = half + a0;
  }
  if (!live) a0 = b0 = 0;
  const int first = (blockIdx.y * NWAVES + threadIdx.x / WAVE) * p.per_wave + lane / LPH;
  const int total = p.heads + p.kv_heads;
  if (first - lane / LPH >= total) return;

  float c[U], s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (turns) {
    float f[U];
    const double at = (double)p.pos[t];
    load_piece<U>(p.inv_freq + U * slot, f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const double turn = at * (double)f[i] * 0.15915494309189533577;  // 1 / (2 pi)
      sincospif(2.f * (float)(turn - rint(turn)), &s[i], &c[i]);
    }
  }
  for (int j = 0; j < p.per_wave; j += HPW) {
    const int h = first + j;
    if (first - lane / LPH + j >= total) return;  // the wave's last heads
    const bool in = live && h < total;
    const bool key = h >= p.heads;
    const RopeSide& side = key ? p.k : p.q;
    const int hh = in ? (key ? h - p.heads : h) : 0;
    float a[U], b[U];
    if (in) {
      const TX* x = static_cast<const TX*>(side.x) + t * side.row + hh * side.head;
      load_piece<U>(x + a0, a);
      load_piece<U>(x + b0, b);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) a[i] = b[i] = 0.f;
    }
    if (p.q.w != nullptr || p.k.w != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor(ss, o, WAVE);
      const float mean = ss / (float)p.D + p.eps;
      float rinv = mean == 0.f ? 0.f : 1.0f / sqrtf(mean);  // a head of zeros, without eps: zeros
      if (__any(!(ss < __builtin_inff()) || mean < 1e-30f)) {
        // squares beyond fp32's range, or lost below it: again with the head times a power of two that brings
        // its largest element, or eps's root where that is larger, near 1
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) big = fmaxf(big, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) big = fmaxf(big, __shfl_xor(big, o, WAVE));
        const bool again = (!(ss < __builtin_inff()) || mean < 1e-30f) && ss == ss && big > 0.f && big < __builtin_inff();
        const int e = again ? -ilogbf(fmaxf(big, sqrtf(p.eps))) : 0;
        float s2 = 0.f;
        const bool wanted = (key ? p.k.w : p.q.w) != nullptr;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float x = ldexpf(a[i], e), y = ldexpf(b[i], e);
          s2 += x * x + y * y;
          if (wanted && again) {
            a[i] = x;
            b[i] = y;
          }
        }
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) s2 += __shfl_xor(s2, o, WAVE);
        if (again) rinv = 1.0f / sqrtf(s2 / (float)p.D + ldexpf(ldexpf(p.eps, e), e));
      }
      if (side.w != nullptr) {
        float wa[U], wb[U];
        load_piece<U>(side.w + a0, wa);
        load_piece<U>(side.w + b0, wb);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          a[i] = a[i] * rinv * wa[i];
          b[i] = b[i] * rinv * wb[i];
        }
      }
    }
    if (!in) continue;
    TY* y = static_cast<TY*>(side.y) + t * side.out_row + hh * side.out_head;
    if (turns) {
      if constexpr (PAIRS) {  // a and b are 2U elements in a row: pairs (0, 1), (2, 3), ..
#pragma unroll
        for (int i = 0; i < U / 2; ++i) {
          const float a0v = a[2 * i], b0v = b[2 * i];
          a[2 * i] = a0v * c[i] - a[2 * i + 1] * s[i];
          a[2 * i + 1] = a[2 * i + 1] * c[i] + a0v * s[i];
          b[2 * i] = b0v * c[U / 2 + i] - b[2 * i + 1] * s[U / 2 + i];
          b[2 * i + 1] = b[2 * i + 1] * c[U / 2 + i] + b0v * s[U / 2 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float av = a[i];
          a[i] = av * c[i] - b[i] * s[i];
          b[i] = b[i] * c[i] + av * s[i];
        }
      }
    }
    store_piece<U>(y + a0, a);
    store_piece<U>(y + b0, b);
  }
}

template <typename TX, typename TY, int U, bool PAIRS, int LPH>
pi_status launch_rope(pi_ctx* c, RopeDev p, int T) {
  constexpr int HPW = WAVE / LPH;
  const int total = p.heads + p.kv_heads, groups = (total + HPW - 1) / HPW;
  // A wave takes as many heads as leave 8 waves for each SIMD: the sines are worked out once per wave.
  int rounds = 1;
  while (rounds < groups && (long long)T * ((groups + 2 * rounds - 1) / (2 * rounds)) >= 32ll * c->cus) rounds *= 2;
  p.per_wave = rounds * HPW;
  const int waves = (groups + rounds - 1) / rounds;
  PI_HIP(c, launch_k(c, 0, k_qk_norm_rope<TX, TY, U, PAIRS, LPH>, dim3(T, (waves + NWAVES - 1) / NWAVES), 0, p));
  return PI_OK;
}

// Lanes per head: D / (2U), up to the next power of two.
template <typename TX, typename TY, int U, bool PAIRS>
pi_status launch_rope_u(pi_ctx* c, const RopeDev& p, int T) {
  const int slots = p.D / (2 * U);
  if (slots <= 4) return launch_rope<TX, TY, U, PAIRS, 4>(c, p, T);
  if (slots <= 8) return launch_rope<TX, TY, U, PAIRS, 8>(c, p, T);
  if (slots <= 16) return launch_rope<TX, TY, U, PAIRS, 16>(c, p, T);
  if (slots <= 32) return launch_rope<TX, TY, U, PAIRS, 32>(c, p, T);
  return launch_rope<TX, TY, U, PAIRS, 64>(c, p, T);
}

// The widest pieces that the rotated and the other elements divide into.
template <typename TX, typename TY, bool PAIRS>
pi_status launch_rope_p(pi_ctx* c, const RopeDev& p, int T) {
  if (p.rot % 16 == 0 && p.D % 16 == 0) return launch_rope_u<TX, TY, 8, PAIRS>(c, p, T);
  if (p.rot % 8 == 0) return launch_rope_u<TX, TY, 4, PAIRS>(c, p, T);
  return launch_rope_u<TX, TY, 2, PAIRS>(c, p, T);
}

template <typename TX>
pi_status launch_rope_x(pi_ctx* c, const RopeDev& p, int T, int y, bool pairs) {
  switch (y) {
    case PI_T_F32: return pairs ? launch_rope_p<TX, float, true>(c, p, T) : launch_rope_p<TX, float, false>(c, p, T);
    case PI_T_F16: return pairs ? launch_rope_p<TX, half_t, true>(c, p, T) : launch_rope_p<TX, half_t, false>(c, p, T);
    default: return pairs ? launch_rope_p<TX, bf16_t, true>(c, p, T) : launch_rope_p<TX, bf16_t, false>(c, p, T);
  }
}

bool known(int t) { return t == PI_T_F32 || t == PI_T_F16 || t == PI_T_BF16; }

pi_status check_heads(pi_ctx* c, const char* name, const void* p, int64_t row, int64_t head, int dtype) {
  PI_TRY(check_dev_ptr(c, p, name));
  if ((row | head) & (dtype == PI_T_F32 ? 3 : 7)) return fail(c, PI_ERR_INVALID, "%s: strides must keep heads 16-byte aligned", name);
  return PI_OK;
}

}  // namespace

extern "C" pi_status pi_qk_norm_rope(pi_ctx* ctx, const pi_rope_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_rope_args& a = *args;
  if (!known(a.x_dtype) || !known(a.y_dtype)) return fail(ctx, PI_ERR_INVALID, "unknown dtype %d or %d", a.x_dtype, a.y_dtype);
  if (a.T < 0 || a.heads < 0 || a.kv_heads < 0 || a.head_dim < 8 || a.head_dim % 8)
    return fail(ctx, PI_ERR_INVALID, "bad shape T=%d, %d and %d heads of %d", a.T, a.heads, a.kv_heads, a.head_dim);
  if (a.head_dim > 512 || (a.head_dim > 256 && a.rot % 8))
    return fail(ctx, PI_ERR_UNSUPPORTED, "heads of %d with %d rotated elements", a.head_dim, a.rot);
  if ((int64_t)a.heads + a.kv_heads > 65536) return fail(ctx, PI_ERR_UNSUPPORTED, "more than 65536 heads");
  if (a.T > 1 << 23) return fail(ctx, PI_ERR_UNSUPPORTED, "T %d above 2^23", a.T);
  if (a.rot < 0 || a.rot > a.head_dim || a.rot % 4) return fail(ctx, PI_ERR_INVALID, "rot %d: a multiple of 4 up to %d", a.rot, a.head_dim);
  if (!(a.eps >= 0.f) || a.eps > 3e38f) return fail(ctx, PI_ERR_INVALID, "eps must be finite and not negative");
  if (a.T == 0 || a.heads + a.kv_heads == 0) return PI_OK;
  if (a.heads > 0) {
    PI_TRY(check_heads(ctx, "q", a.q, a.q_row, a.q_head, a.x_dtype));
    PI_TRY(check_heads(ctx, "q_out", a.q_out, a.q_out_row, a.q_out_head, a.y_dtype));
    PI_TRY(check_dev_ptr(ctx, a.q_w, "q_w", true));
    if (a.q == a.q_out && (a.x_dtype != a.y_dtype || a.q_row != a.q_out_row || a.q_head != a.q_out_head))
      return fail(ctx, PI_ERR_INVALID, "q in place needs one type and equal strides");
  }
  if (a.kv_heads > 0) {
    PI_TRY(check_heads(ctx, "k", a.k, a.k_row, a.k_head, a.x_dtype));
    PI_TRY(check_heads(ctx, "k_out", a.k_out, a.k_out_row, a.k_out_head, a.y_dtype));
    PI_TRY(check_dev_ptr(ctx, a.k_w, "k_w", true));
    if (a.k == a.k_out && (a.x_dtype != a.y_dtype || a.k_row != a.k_out_row || a.k_head != a.k_out_head))
      return fail(ctx, PI_ERR_INVALID, "k in place needs one type and equal strides");
  }
  if (a.rot > 0) {
    PI_TRY(check_dev_ptr(ctx, a.inv_freq, "inv_freq"));
    if (a.pos == nullptr || (reinterpret_cast<uintptr_t>(a.pos) & 3u)) return fail(ctx, PI_ERR_INVALID, "pos is NULL or not 4-byte aligned");
  }
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const RopeDev p{{a.q, a.q_out, a.heads > 0 ? a.q_w : nullptr, a.q_row, a.q_head, a.q_out_row, a.q_out_head},
                  {a.k, a.k_out, a.kv_heads > 0 ? a.k_w : nullptr, a.k_row, a.k_head, a.k_out_row, a.k_out_head},
                  a.pos, a.inv_freq, a.eps, a.heads, a.kv_heads, a.head_dim, a.rot, 0};
  switch (a.x_dtype) {
    case PI_T_F32: return launch_rope_x<float>(ctx, p, a.T, a.y_dtype, a.interleaved != 0);
    case PI_T_F16: return launch_rope_x<half_t>(ctx, p, a.T, a.y_dtype, a.interleaved != 0);
    default: return launch_rope_x<bf16_t>(ctx, p, a.T, a.y_dtype, a.interleaved != 0);
  }
}
