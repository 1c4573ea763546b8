// Causal attention of packed prompts (pi_prompt_attention).
//
// A key/value head's query rows (tokens x G heads of the group, token by token) are columns of the matrix
// cores' 32x32x16 products, 32 a wave. For a tile of 64 keys in LDS, S^T = K Q^T leaves each lane 32
// keys of one row, so the softmax's maximum and sum run along in registers; exp(S - max) is, as it lies, the
// B operand of O^T += V^T P^T, V^T by transposing LDS reads. Maximum, sum, S and O are fp32; P is
// rounded to the inputs' type. A workgroup's rows are 256 / G tokens of all heads of a group, so
// that it reads a key once for all of them and little of the diagonal's tiles is masked.
#include <algorithm>
#include <new>

#include "pi_attn.hpp"

using namespace pi;

struct pi_prompt {
  pi_ctx* ctx;
  int dtype, heads, kv_heads, head_dim, max_tokens, max_batch;
  float scale;
};

namespace {

struct PromptDev {
  const uint8_t *q, *k, *v;
  uint8_t* out;
  const int32_t *cu_q, *cu_k;
  long long q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
  int B, q_rows, k_rows, HK, G, D, tiles;  // tiles: row tiles, an upper limit
  float scale2;  // scale * log2(e)
};

constexpr int PKT = 64;  // keys of a tile

// Sequence b's part of `rows` packed rows: from *first on, the number of rows is returned.
__device__ __forceinline__ int packed(const int32_t* cu, int b, int rows, int* first) {
  const int f = min(max(cu[b], 0), rows);
  *first = f;
  return max(min(cu[b + 1], rows), f) - f;
}

template <int DP> constexpr size_t prompt_lds() { return 2 * (size_t)PKT * (k_pitch<DP>() + v_pitch<DP>()); }
constexpr int padded_dim_p(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256; }

template <typename T, int DP, int WQ>
__global__ __launch_bounds__(64 * WQ) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_prompt(PromptDev a) {
  constexpr int KB = 2, KT = PKT, NT = 64 * WQ, KS = DP / 16, DB = DP / 32, R = 32 * WQ;
  constexpr int KP = k_pitch<DP>(), VP = v_pitch<DP>(), STAGE = KT * (KP + VP);
  constexpr int LPR = DP <= 64 ? 8 : DP <= 128 ? 16 : 32, RPP = NT / LPR, PASS = KT / RPP;
  static_assert(PASS >= 1 && KT % RPP == 0, "a tile is whole passes");
  typedef typename Mm<T>::v8 v8;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_odd;  // a value row that not every row sees holds an infinity or a NaN
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, half = lane >> 5, l32 = lane & 31;
  const int hk = blockIdx.x % a.HK;
  // the row tiles from the last one on: those with the most keys start first
  const int slot = a.tiles - 1 - blockIdx.x / a.HK;
  int b = -1, rt = 0, before = 0;
  for (int b0 = 0; b0 < a.B; b0 += WAVE) {
    int first;
    const int n = b0 + lane < a.B ? (packed(a.cu_q, b0 + lane, a.q_rows, &first) * a.G + R - 1) / R : 0;
    int incl = n;
#pragma unroll
    for (int s = 1; s < WAVE; s <<= 1) {
      const int t = __shfl_up(incl, s, WAVE);
      if (lane >= s) incl += t;
    }
    const uint64_t hit = __ballot(before + incl > slot);
    if (hit != 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      b = b0 + l;
      rt = slot - before - __shfl(incl - n, l, WAVE);
      break;
    }
    before += __shfl(incl, WAVE - 1, WAVE);
  }
  if (b < 0) return;
  b = __builtin_amdgcn_readfirstlane(b);
  rt = __builtin_amdgcn_readfirstlane(rt);
  if (threadIdx.x == 0) s_odd = 0;
  int q0, k0;
  const int Lq = packed(a.cu_q, b, a.q_rows, &q0), Lk = packed(a.cu_k, b, a.k_rows, &k0);
  const int rows = Lq * a.G, ahead = Lk - Lq;  // query i sees the keys up to i + ahead
  const int row0 = rt * R, wrow0 = row0 + 32 * wave, row = wrow0 + l32;
  const bool live = row < rows, wave_live = wrow0 < rows;
  const int token = live ? row / a.G : 0, head = hk * a.G + (live ? row % a.G : 0);
  const int lim = live ? token + ahead : -1;
  const int nk = min(max(min(Lq, (row0 + R - 1) / a.G + 1) + ahead, 0), Lk);  // keys that some row sees
  const int all = row0 / a.G + ahead;                                         // the last one that all see
  const int wall = wrow0 / a.G + ahead, wmost = min(Lq - 1, (wrow0 + 31) / a.G) + ahead;
  const int ntiles = (nk + KT - 1) / KT;

  v8 qf[KS];
  {
    const uint8_t* qp = a.q + 2 * ((long long)(q0 + token) * a.q_row + (long long)head * a.q_head);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 16 * s + 8 * half;
      qf[s] = __builtin_bit_cast(v8, ld16_or0(qp + 2 * (d < a.D ? d : 0), live && d < a.D));
    }
  }

  typedef const __attribute__((address_space(1))) uint8_t* gp;  // global by type: a generic load counts as LDS too
  const gp zero = (gp)(const uint8_t*)&attn_zero;
  const int lr = (int)threadIdx.x / LPR, lc = (int)threadIdx.x % LPR;
  const bool piece_in = 8 * lc < a.D;
  const gp kg = (gp)a.k + 2 * ((long long)k0 * a.k_row + (long long)hk * a.k_head + (piece_in ? 8 * lc : 0));
  const gp vg = (gp)a.v + 2 * ((long long)k0 * a.v_row + (long long)hk * a.v_head + (piece_in ? 8 * lc : 0));
  u32x4 kr[2][PASS], vr[2][PASS];
  auto load = [&](int tile, int set) {
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int j = tile * KT + lr + i * RPP;
      const bool in = piece_in && j < nk;
      const gp k = in ? kg + 2 * j * a.k_row : zero, v = in ? vg + 2 * j * a.v_row : zero;
      kr[set][i] = *(const __attribute__((address_space(1))) u32x4*)k;
      vr[set][i] = *(const __attribute__((address_space(1))) u32x4*)v;
    }
  };
  auto store = [&](int tile, int stage, int set) {
    uint8_t* base = smem + stage * STAGE;
    if (tile * KT + KT - 1 > all) {
      // A weight of zero times an infinity or a NaN is a NaN: such elements of keys that not every row sees
      // stay out of the product and are added to the rows that see them at the end.
#pragma unroll
      for (int i = 0; i < PASS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = vr[set][i][e];
          const uint32_t lo = (w & Mm<T>::EXP) == Mm<T>::EXP ? 0xFFFFu : 0u;
          const uint32_t hi = (w & (Mm<T>::EXP << 16)) == Mm<T>::EXP << 16 ? 0xFFFF0000u : 0u;
          if (lo | hi) s_odd = 1;
          vr[set][i][e] = w & ~(lo | hi);
        }
    }
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int r = lr + i * RPP;
      if (DP / 8 == LPR || lc < DP / 8) {
        *reinterpret_cast<u32x4*>(base + r * KP + lc * 16) = kr[set][i];
        *reinterpret_cast<u32x4*>(base + KT * KP + r * VP + lc * 16) = vr[set][i];
      }
    }
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) o[i] = (f32x16){};
  float m = -__builtin_inff(), l = 0.f;  // running maximum (log2 domain); this half's sum

  auto compute = [&](int tile, int stage) {
    const uint8_t* kb0 = smem + stage * STAGE;
    const uint8_t* vb0 = kb0 + KT * KP;
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = (f32x16){};
#pragma unroll
      for (int i = 0; i < KS; ++i)
        s[kb] = Mm<T>::mfma(__builtin_bit_cast(v8, ld16(kb0 + (kb * 32 + l32) * KP + 32 * i + 16 * half)), qf[i], s[kb]);
    }
    if (tile * KT + KT - 1 > wall) {
      const int last = lim - tile * KT;
      const uint64_t seen = last >= 63 ? ~0ull : last < 0 ? 0ull : (2ull << last) - 1;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const uint32_t vis = (uint32_t)(seen >> (32 * kb)) >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[kb][r] = bfi_sel(0u - ((vis >> acc_row(r, 0)) & 1u), s[kb][r], -__builtin_inff());
      }
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
    top = swap_max(top) * a.scale2;
    const float mn = fmaxf(m, top);
    const float base = mn == -__builtin_inff() ? 0.f : mn;  // nothing seen so far: weights 0
    if (__any(mn > m)) {
      const float f = __builtin_amdgcn_exp2f(m - base);
      l *= f;
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= f;
    }
    m = mn;
    v8 pf[KB][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][r], a.scale2, Mm<T>::SHIFT - base));
        l += w;
        pf[kb][r >> 3][r & 7] = (T)w;
      }
    const uint8_t* vl = vb0 + (4 * half + ((lane & 15) >> 2)) * VP + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          typedef __attribute__((address_space(3))) short4_t* lds4;
          const uint8_t* p = vl + (kb * 32 + st * 16) * VP + 64 * i;
          struct { short4_t x, y; } v;
          v.x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p));
          v.y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 8 * VP));
          o[i] = Mm<T>::mfma(__builtin_bit_cast(v8, v), pf[kb][st], o[i]);
        }
  };

  if (ntiles > 0) {
    load(0, 0);
    load(1, 1);
    __syncthreads();  // s_odd is 0
    store(0, 0, 0);
    __syncthreads();
    auto step = [&](int t, int h) {
      load(t + 2, h);
      __builtin_amdgcn_sched_barrier(0);
      if (wave_live && t * KT <= wmost) compute(t, h);
      __builtin_amdgcn_sched_barrier(0);
      store(t + 1, h ^ 1, h ^ 1);
      __syncthreads();
    };
    int t = 0;
    for (; t + 1 < ntiles; t += 2) {
      step(t, 0);
      step(t + 1, 1);
    }
    if (t < ntiles) step(t, 0);
  } else {
    __syncthreads();
  }
  if (!live) return;
  if (s_odd)
    for (int j = max(all, 0) & ~(KT - 1); j <= lim; ++j) {
      const T* x = reinterpret_cast<const T*>(a.v) + (long long)(k0 + j) * a.v_row + (long long)hk * a.v_head;
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int d = 32 * i + acc_row(r, half);
          const float y = d < a.D ? (float)x[d] : 0.f;
          if (!(fabsf(y) < __builtin_inff())) o[i][r] += y;
        }
    }
  l = swap_add(l);
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
  T* const out = reinterpret_cast<T*>(a.out) + (long long)(q0 + token) * a.out_row + (long long)head * a.out_head;
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = 32 * i + 8 * k + 4 * half;
      struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w.e[e] = (T)(l == 0.f ? 0.f : o[i][4 * k + e] * inv);
      if (d < a.D) __builtin_memcpy(__builtin_assume_aligned(out + d, 8), &w, 8);
    }
}

template <typename T, int DP, int WQ>
pi_status launch_prompt_t(pi_ctx* c, PromptDev a) {
  constexpr size_t lds = prompt_lds<DP>();
  auto kern = k_prompt<T, DP, WQ>;
  PI_HIP(c, allow_lds(kern, lds));
  // every sequence's last tile may be a part of one
  a.tiles = (int)(((long long)a.q_rows * a.G + 32 * WQ - 1) / (32 * WQ)) + a.B - 1;
  PI_HIP(c, launch_kb(c, 0, kern, dim3((unsigned)(a.tiles * a.HK)), 64 * WQ, lds, a));
  return PI_OK;
}

// Four waves where sequences are short: a tile of eight would be mostly empty.
template <typename T, int DP>
pi_status launch_prompt_d(pi_ctx* c, const PromptDev& a) {
  if (DP <= 128 && (long long)a.q_rows * a.G <= 128ll * a.B) return launch_prompt_t<T, DP, DP <= 128 ? 4 : 8>(c, a);
  return launch_prompt_t<T, DP, 8>(c, a);
}

template <typename T>
pi_status launch_prompt(pi_ctx* c, const PromptDev& a) {
  switch (padded_dim_p(a.D)) {
    case 64: return launch_prompt_d<T, 64>(c, a);
    case 96: return launch_prompt_d<T, 96>(c, a);
    case 128: return launch_prompt_d<T, 128>(c, a);
    default: return launch_prompt_d<T, 256>(c, a);
  }
}

}  // namespace

extern "C" {

pi_status pi_prompt_create(pi_ctx* ctx, int32_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                           int32_t max_tokens, int32_t max_batch, float scale, pi_prompt** out) {
  if (ctx == nullptr || out == nullptr) return PI_ERR_INVALID;
  *out = nullptr;
  if (dtype != PI_T_F16 && dtype != PI_T_BF16) return fail(ctx, PI_ERR_INVALID, "dtype %d: need fp16 or bf16", dtype);
  if (kv_heads < 1 || heads < 1 || heads % kv_heads)
    return fail(ctx, PI_ERR_INVALID, "%d query heads are no multiple of %d", heads, kv_heads);
  if (head_dim < 8 || head_dim % 8) return fail(ctx, PI_ERR_INVALID, "head_dim must be a multiple of 8 (got %d)", head_dim);
  if (head_dim > 256) return fail(ctx, PI_ERR_UNSUPPORTED, "head_dim %d above 256", head_dim);
  if (max_tokens < 1 || max_batch < 1) return fail(ctx, PI_ERR_INVALID, "bad limits: %d tokens, %d sequences", max_tokens, max_batch);
  if (!(scale > 0.f) || scale > 3e38f) return fail(ctx, PI_ERR_INVALID, "scale must be finite and above 0");
  // row numbers of a head's group, and workgroups, are 32-bit numbers
  if (((int64_t)max_tokens + 256ll * max_batch) * heads >= 1ll << 30)
    return fail(ctx, PI_ERR_UNSUPPORTED, "%d tokens of %d sequences and %d heads are too many", max_tokens, max_batch, heads);
  pi_prompt* p = new (std::nothrow) pi_prompt{ctx, dtype, heads, kv_heads, head_dim, max_tokens, max_batch, scale};
  if (p == nullptr) return fail(ctx, PI_ERR_OOM, "host allocation failed");
  ctx_retain(ctx);
  *out = p;
  return PI_OK;
}

void pi_prompt_destroy(pi_prompt* p) {
  if (p == nullptr) return;
  ctx_release(p->ctx);
  delete p;
}

pi_status pi_prompt_attention(pi_ctx* ctx, pi_prompt* prompt, const pi_prompt_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (prompt == nullptr) return fail(ctx, PI_ERR_INVALID, "prompt is NULL");
  if (prompt->ctx != ctx) return fail(ctx, PI_ERR_INVALID, "prompt belongs to another context");
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_prompt_args& a = *args;
  if (a.B < 1 || a.q_rows < 0 || a.k_rows < 0) return fail(ctx, PI_ERR_INVALID, "bad shape B=%d, %d and %d rows", a.B, a.q_rows, a.k_rows);
  if (a.B > prompt->max_batch || a.q_rows > prompt->max_tokens)
    return fail(ctx, PI_ERR_INVALID, "%d sequences, %d rows above the handle's %d, %d", a.B, a.q_rows, prompt->max_batch, prompt->max_tokens);
  if (a.k_rows > (1 << 30)) return fail(ctx, PI_ERR_UNSUPPORTED, "%d rows of keys: at most 2^30", a.k_rows);
  if (a.cu_q == nullptr) return fail(ctx, PI_ERR_INVALID, "cu_q is NULL");
  if (a.q_rows == 0) return PI_OK;
  PI_TRY(check_bnh(ctx, "q", a.q, 0, a.q_row, a.q_head));
  PI_TRY(check_bnh(ctx, "out", a.out, 0, a.out_row, a.out_head));
  if (a.k_rows > 0) {
    PI_TRY(check_bnh(ctx, "k", a.k, 0, a.k_row, a.k_head));
    PI_TRY(check_bnh(ctx, "v", a.v, 0, a.v_row, a.v_head));
  }
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const PromptDev d{static_cast<const uint8_t*>(a.q), static_cast<const uint8_t*>(a.k), static_cast<const uint8_t*>(a.v),
                    static_cast<uint8_t*>(a.out), a.cu_q, a.cu_k != nullptr ? a.cu_k : a.cu_q, a.q_row, a.q_head, a.k_row,
                    a.k_head, a.v_row, a.v_head, a.out_row, a.out_head, a.B, a.q_rows, a.k_rows, prompt->kv_heads,
                    prompt->heads / prompt->kv_heads, prompt->head_dim, 0, prompt->scale * 1.4426950408889634f};
  return prompt->dtype == PI_T_F16 ? launch_prompt<half_t>(ctx, d) : launch_prompt<bf16_t>(ctx, d);
}

}  // extern "C"
