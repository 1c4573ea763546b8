// RMS norm of query and key heads with rotary positions (pi_qk_norm_rope).
//
// y = x / sqrt(mean(x^2) + eps) * w per head, then each pair (a, b) of the first rot elements turns by
// pos * inv_freq: (a cos - b sin, b cos + a sin). A head is read once and written once. A workgroup takes up to ROPE_TOKENS
// tokens; it works their sines and cosines out first, one angle a thread, into LDS. A lane then has the same 2U elements of
// every head it takes (U pairs: two pieces of U elements each, U * i and rot/2 + U * i, or 2U in a row where pairs are
// interleaved), HEADS_STEP heads a step. As compiled, a head's rows are waited for before the next head's are asked for:
// their conversion to fp32 stands in the branch of the lanes that have a head. But for bf16 in pieces of 8 elements one
// element of each piece also passes through scratch memory (20 to 80 bytes a lane).
// With norms, 302 MB: 8192 tokens of 72 heads of 128 in bf16 62 us, 4.9 TB/s, near a copy's rate (four heads a step 70, one
// 65; with every wave working its sines out itself 89); in fp16 84 us; 4096 such tokens in fp32 126 us. 151 MB in bf16, 40
// heads of 64, of 256, or of 128 half turned: 30 us; of 80: 35. 8 tokens: 4 us, latency.
//
// The angle is a whole number times an fp32 number, exact in 64 bits up to 2^29 and off by 2^-53 of
// itself beyond; as turns, reduced by its nearest whole number, it goes on in fp32 (2^-25 of a turn).
#include <algorithm>

#include "pi_kv.hpp"
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
  PageDiv by_heads;                              // heads of a token
  int T, heads, kv_heads, D, rot, tokens, part;  // tokens of a workgroup, and of their heads (all tokens') it takes
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

// A head's norm and weights; its elements are in LPH lanes.
template <int U, int LPH>
__device__ __forceinline__ void normalise(const RopeDev& p, const RopeSide& side, int a0, int b0, float (&a)[U], float (&b)[U]) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor(ss, o, WAVE);
  const float mean = ss / (float)p.D + p.eps;
  float rinv = mean == 0.f ? 0.f : 1.0f / sqrtf(mean);  // a head of zeros, without eps: zeros
  const bool far = !(ss < __builtin_inff()) || mean < 1e-30f;
  if (__any(far)) {
    // squares beyond fp32's range, or lost below it: again with the head times a power of two that brings its largest
    // element, or eps's root where that is larger, near 1
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) big = fmaxf(big, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) big = fmaxf(big, __shfl_xor(big, o, WAVE));
    const bool again = far && ss == ss && big > 0.f && big < __builtin_inff();
    const int e = again ? -ilogbf(fmaxf(big, sqrtf(p.eps))) : 0;
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float x = ldexpf(a[i], e), y = ldexpf(b[i], e);
      s2 += x * x + y * y;
      if (side.w != nullptr) {
        a[i] = x;
        b[i] = y;
      }
    }
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) s2 += __shfl_xor(s2, o, WAVE);
    if (again) rinv = 1.0f / sqrtf(s2 / (float)p.D + ldexpf(ldexpf(p.eps, e), e));
  }
  if (side.w == nullptr) return;
  float wa[U], wb[U];
  load_piece<U>(side.w + a0, wa);
  load_piece<U>(side.w + b0, wb);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    a[i] = a[i] * rinv * wa[i];
    b[i] = b[i] * rinv * wb[i];
  }
}

constexpr int ROPE_TOKENS = 8, HEADS_STEP = 2;

// LPH lanes per head, a power of two. Heads are numbered token by token, queries first, then keys.
template <typename TX, typename TY, int U, bool PAIRS, int LPH>
__global__ __launch_bounds__(BLOCK) void k_qk_norm_rope(RopeDev p) {
  extern __shared__ float turn[];  // [tokens][2][half]: cosines, sines
  constexpr int HPB = BLOCK / LPH;
  const int t0 = blockIdx.x * p.tokens, tokens = min(p.tokens, p.T - t0);
  const int half = p.rot >> 1, slot = threadIdx.x % LPH;
  const bool turns = slot < half / U, live = slot < p.D / (2 * U);
  int a0, b0;  // first elements of this lane's two pieces
  if (PAIRS || !turns) {
    a0 = 2 * U * slot;
    b0 = a0 + U;
  } else {
    a0 = U * slot;
    b0 = half + a0;
  }
  if (!live) a0 = b0 = 0;
  const int total = p.heads + p.kv_heads;
  const int first = blockIdx.y * p.part + threadIdx.x / LPH, end = min((int)(blockIdx.y + 1) * p.part, tokens * total);
  float a[HEADS_STEP][U], b[HEADS_STEP][U];
  int tok[HEADS_STEP], head[HEADS_STEP];
  bool in[HEADS_STEP], key[HEADS_STEP];
  auto load = [&](int h0) {
#pragma unroll
    for (int n = 0; n < HEADS_STEP; ++n) {
      const int h = h0 + n * HPB;
      in[n] = live && h < end;
      uint32_t hh;
      tok[n] = (int)page_of(p.by_heads, in[n] ? (uint32_t)h : 0u, &hh);
      key[n] = (int)hh >= p.heads;
      head[n] = (int)hh - (key[n] ? p.heads : 0);
      const RopeSide& side = key[n] ? p.k : p.q;
      if (in[n]) {
        const TX* x = static_cast<const TX*>(side.x) + (long long)(t0 + tok[n]) * side.row + head[n] * side.head;
        load_piece<U>(x + a0, a[n]);
        load_piece<U>(x + b0, b[n]);
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i) a[n][i] = b[n][i] = 0.f;
      }
    }
  };
  load(first);  // the rows are converted before the angles' loads
  for (int i = threadIdx.x; i < tokens * half; i += BLOCK) {
    const int t = i / half, k = i - t * half;
    const double turns = (double)p.pos[t0 + t] * (double)p.inv_freq[k] * 0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    turn[2 * t * half + k] = c;
    turn[(2 * t + 1) * half + k] = s;
  }
  __syncthreads();
  for (int h0 = first; h0 - (int)threadIdx.x / LPH < end; h0 += HEADS_STEP * HPB) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int n = 0; n < HEADS_STEP; ++n) {
      const RopeSide& side = key[n] ? p.k : p.q;
      if (p.q.w != nullptr || p.k.w != nullptr) normalise<U, LPH>(p, side, a0, b0, a[n], b[n]);
      if (!in[n]) continue;
      if (turns) {
        float c[U], s[U];
        const float* at = turn + 2 * tok[n] * half + U * slot;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          c[i] = at[i];
          s[i] = at[half + i];
        }
        if constexpr (PAIRS) {  // a and b are 2U elements in a row: pairs (0, 1), (2, 3), ..
#pragma unroll
          for (int i = 0; i < U / 2; ++i) {
            const float av = a[n][2 * i], bv = b[n][2 * i];
            a[n][2 * i] = av * c[i] - a[n][2 * i + 1] * s[i];
            a[n][2 * i + 1] = a[n][2 * i + 1] * c[i] + av * s[i];
            b[n][2 * i] = bv * c[U / 2 + i] - b[n][2 * i + 1] * s[U / 2 + i];
            b[n][2 * i + 1] = b[n][2 * i + 1] * c[U / 2 + i] + bv * s[U / 2 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const float av = a[n][i];
            a[n][i] = av * c[i] - b[n][i] * s[i];
            b[n][i] = b[n][i] * c[i] + av * s[i];
          }
        }
      }
      TY* y = static_cast<TY*>(side.y) + (long long)(t0 + tok[n]) * side.out_row + head[n] * side.out_head;
      store_piece<U>(y + a0, a[n]);
      store_piece<U>(y + b0, b[n]);
    }
  }
}

template <typename TX, typename TY, int U, bool PAIRS, int LPH>
pi_status launch_rope(pi_ctx* c, RopeDev p, int T) {
  constexpr int HPB = BLOCK / LPH;
  const int total = p.heads + p.kv_heads;
  // As many tokens as leave 4 workgroups for each CU, and no more than two steps of heads need; then, where there are few
  // tokens, their heads in parts of as many as a workgroup has lanes for.
  p.tokens = std::max(1, std::min({ROPE_TOKENS, T / (4 * c->cus), (HEADS_STEP * HPB * 2 + total - 1) / total}));
  p.part = p.tokens > 1 ? p.tokens * total : HEADS_STEP * HPB;
  p.by_heads = page_div(total);
  const dim3 grid((T - 1) / p.tokens + 1, (p.tokens * total - 1) / p.part + 1);
  PI_HIP(c, launch_k(c, 0, k_qk_norm_rope<TX, TY, U, PAIRS, LPH>, grid, p.tokens * p.rot * sizeof(float), p));
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
                  a.pos, a.inv_freq, a.eps, PageDiv{}, a.T, a.heads, a.kv_heads, a.head_dim, a.rot, 0, 0};
  switch (a.x_dtype) {
    case PI_T_F32: return launch_rope_x<float>(ctx, p, a.T, a.y_dtype, a.interleaved != 0);
    case PI_T_F16: return launch_rope_x<half_t>(ctx, p, a.T, a.y_dtype, a.interleaved != 0);
    default: return launch_rope_x<bf16_t>(ctx, p, a.T, a.y_dtype, a.interleaved != 0);
  }
}
