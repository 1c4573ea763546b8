// Causal attention of packed prompts (pi_prompt_attention).
//
// A key/value head's query rows (tokens x G heads of the group, token by token) are columns of the matrix
// cores' 32x32x16 products, 32 a wave. For a tile of 64 keys in LDS, S^T = K Q^T leaves each lane 32
// keys of one row, so the softmax's maximum and sum run along in registers; exp(S - max) is, as it lies, the
// B operand of O^T += V^T P^T, V^T by transposing LDS reads. Maximum, sum, S and O are fp32; P is
// rounded to the inputs' type. A workgroup's rows are 256 / G tokens of all heads of a group, so
// that it reads a key once for all of them and little of the diagonal's tiles is masked.
//
// Bound by the products and the weights' vector work at a clock that gives way to power: 16384 tokens of 32 heads (8 kv) of
// 128 in bf16, 2199 GFLOP, 2163 to 2249 us, 0.98 to 1.02 PFLOP/s (a large library product: 1.28 to 1.42; the first calls after
// a pause 2320 to 2630 us; with zeros as data 1862). 8192 tokens of 32 heads (8 kv) of 64, 80, 96: 382, 465, 475 us (0.72,
// 0.74, 0.87); of 16 heads (8 kv) of 256, whose registers spill: 1620 (0.34). 16 packed sequences of up to 2047 tokens and
// 1500 held, 64 heads, 1353 to 1403 us: each workgroup starts with some 4 us of dependent loads, with nothing beside it on
// its CU. 500 tokens: 20 to 21 us, up to 8 tiles one after another.
#include <algorithm>
#include <new>

#include "pi_attn.hpp"

using namespace pi;

struct pi_prompt {
  pi_ctx* ctx;
  int dtype, heads, kv_heads, head_dim, max_tokens, max_batch;
  float scale;
  uint8_t* ws;      // partial results of split keys
  size_t ws_rows;   // query rows times splits that it holds
};

namespace {

constexpr int SPLITS = 32;  // at most
// Workgroups that the cutting of keys may launch: the last row tiles of many sequences are each launched for every part,
// and a launch has fewer than 2^32 threads.
constexpr int64_t SPLIT_WGS = 1 << 20;

// How a call is cut. Eight waves a workgroup where their row tiles fill the chip, else four: more workgroups, and tiles that
// fit short sequences (500 tokens of 32 heads: 21 us, with eight 26; with two, whose threads have too many rows to load,
// 30). Where those are still few, the keys are split, four tiles at least a part: 33 tokens after 8192 held ones, 64 heads
// (8 kv), take 40 us, with whole rows 238.
struct PromptPlan {
  int wq, tiles, splits;
};
PromptPlan prompt_plan(int cus, int HK, int G, int DP, int rows, int B, int64_t keys) {
  PromptPlan p;
  const int64_t r = (int64_t)rows * G;
  for (p.wq = 8;; p.wq = 4) {
    // every sequence's last tile may be a part of one
    p.tiles = (int)((r + 32 * p.wq - 1) / (32 * p.wq)) + B - 1;
    if (DP > 128 || p.wq == 4 || (r / (32 * p.wq) * HK >= cus && r > 128ll * B)) break;
  }
  const int64_t full = std::max<int64_t>(1, (r + 32 * p.wq - 1) / (32 * p.wq)) * HK;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({SPLITS, (p.wq == 8 ? 1 : 2) * cus / full, keys / B / (4 * 64),
                                                          SPLIT_WGS / ((int64_t)p.tiles * HK)}));
  return p;
}

struct PromptDev {
  const uint8_t *q, *k, *v;
  uint8_t* out;
  const int32_t *cu_q, *cu_k;
  long long q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
  float *part, *ml;                        // of split keys: partial results [row][head][split][DP], maximum and sum
  int B, q_rows, k_rows, HK, G, D, tiles;  // tiles: row tiles, an upper limit
  int splits;                              // parts that a row tile's keys are cut into, a workgroup each
  float scale2;  // scale * log2(e)
};

constexpr int PKT = 64;  // keys of a tile

// The power of two that weights carry. In bf16 values go up to fp32's end: 2^30 weights of at most 2^-31 keep their sum in
// range, and weights down to 2^-95 of the largest stay normal numbers. fp16: as over a plain cache.
template <typename T> constexpr float PROMPT_SHIFT = __is_same(T, half_t) ? Mm<half_t>::SHIFT : -31.f;

// Sequence b's part of `rows` packed rows: from *first on, the number of rows is returned.
__device__ __forceinline__ int packed(const int32_t* cu, int b, int rows, int* first) {
  const int f = min(max(cu[b], 0), rows);
  *first = f;
  return max(min(cu[b + 1], rows), f) - f;
}

template <int DP> constexpr size_t prompt_lds() { return 2 * (size_t)PKT * (k_pitch<DP>() + v_pitch<DP>()); }

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
  const int hk = blockIdx.x % a.HK, split = blockIdx.x / a.HK % a.splits;
  // the row tiles from the last one on: those with the most keys start first
  const int slot = a.tiles - 1 - blockIdx.x / a.HK / a.splits;
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
  // this workgroup's part of the key tiles
  const int ntiles = (nk + KT - 1) / KT;
  const int t0 = a.splits == 1 ? 0 : (int)((long long)ntiles * split / a.splits);
  const int t1 = a.splits == 1 ? ntiles : (int)((long long)ntiles * (split + 1) / a.splits);

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
  const int lr = (int)threadIdx.x / LPR, lc = (int)threadIdx.x % LPR;
  const bool piece_in = 8 * lc < a.D;
  // Rows of a tile are at a scalar address plus the lane's offset, which is the same for all tiles but the last: rows
  // past the keys that some row sees stand for the last such key there. They weigh nothing.
  const gp kg = (gp)a.k + 2 * ((long long)k0 * a.k_row + (long long)hk * a.k_head);
  const gp vg = (gp)a.v + 2 * ((long long)k0 * a.v_row + (long long)hk * a.v_head);
  const uint32_t kstep = 2 * (uint32_t)a.k_row, vstep = 2 * (uint32_t)a.v_row, lp = piece_in ? 16 * lc : 0;
  uint32_t ko[PASS], vo[PASS];
#pragma unroll
  for (int i = 0; i < PASS; ++i) {
    ko[i] = (uint32_t)(lr + i * RPP) * kstep + lp;
    vo[i] = (uint32_t)(lr + i * RPP) * vstep + lp;
  }
  // rows on their way to LDS: of the next two tiles, of one where a thread has many
  constexpr int SETS = WQ == 8 && DP <= 128 ? 2 : 1;
  u32x4 kr[SETS][PASS], vr[SETS][PASS];
  auto load_rows = [&](gp base, long long row, uint32_t step, const uint32_t (&at)[PASS], int tile, u32x4 (&r)[PASS]) __attribute__((always_inline)) {
    if (tile >= t1) return;
    const gp p = base + 2 * (long long)(tile * KT) * row;
    if (tile * KT + KT <= nk) {
#pragma unroll
      for (int i = 0; i < PASS; ++i) r[i] = *(const __attribute__((address_space(1))) u32x4*)(p + at[i]);
    } else {
#pragma unroll
      for (int i = 0; i < PASS; ++i)
        r[i] = *(const __attribute__((address_space(1))) u32x4*)(p + (uint32_t)min(lr + i * RPP, nk - 1 - tile * KT) * step + lp);
    }
  };
  auto load_k = [&](int tile, int set) __attribute__((always_inline)) { load_rows(kg, a.k_row, kstep, ko, tile, kr[set]); };
  auto load_v = [&](int tile, int set) __attribute__((always_inline)) { load_rows(vg, a.v_row, vstep, vo, tile, vr[set]); };
  auto store_k = [&](uint8_t* to, int set) {
#pragma unroll
    for (int i = 0; i < PASS; ++i)
      if (piece_in) *reinterpret_cast<u32x4*>(to + (lr + i * RPP) * KP + lc * 16) = kr[set][i];
  };
  auto store_v = [&](int tile, uint8_t* to, int set) {
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
    for (int i = 0; i < PASS; ++i)
      if (piece_in) *reinterpret_cast<u32x4*>(to + (lr + i * RPP) * VP + lc * 16) = vr[set][i];
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) o[i] = (f32x16){};
  float m = -__builtin_inff(), l = 0.f;  // running maximum (log2 domain); this half's sum

  f32x16 s[KB];
  v8 pf[KB][2];
  auto scores = [&](const uint8_t* kb0) __attribute__((always_inline)) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = (f32x16){};
#pragma unroll
      for (int i = 0; i < KS; ++i)
        s[kb] = Mm<T>::mfma(__builtin_bit_cast(v8, ld16(kb0 + (kb * 32 + l32) * KP + 32 * i + 16 * half)), qf[i], s[kb]);
    }
  };
  auto weights = [&](int tile) __attribute__((always_inline)) {
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
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][r], a.scale2, PROMPT_SHIFT<T> - base));
        l += w;
        pf[kb][r >> 3][r & 7] = (T)w;
      }
  };
  auto values = [&](const uint8_t* vb0) __attribute__((always_inline)) {
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

  // what lies past the heads' last element in LDS is never stored to: zeros
  if (a.D < DP && t0 < t1)
    for (int i = threadIdx.x; i < 2 * STAGE / 16; i += NT) *reinterpret_cast<u32x4*>(smem + 16 * i) = (u32x4){0, 0, 0, 0};
  if (t0 >= t1) {
    __syncthreads();
  } else {
    auto load = [&](int tile, int set) {
      load_k(tile, set);
      load_v(tile, set);
    };
    auto store = [&](int tile, int stage, int set) {
      store_k(smem + stage * STAGE, set);
      store_v(tile, smem + stage * STAGE + KT * KP, set);
    };
    // Of the two waves of a SIMD one is preferred, so that they fall out of step: one's weights are worked out under the
    // other's products. (Turns kept by barriers, with LDS read four products ahead, were no faster: 2190 us again
    // at 16384 tokens, where the clock gives way to power.)
    if (WQ == 8 && wave < 4) __builtin_amdgcn_s_setprio(1);
    load(t0, 0);
    if (SETS == 2) load(t0 + 1, SETS - 1);
    __syncthreads();  // s_odd is 0
    store(t0, 0, 0);
    __syncthreads();
    auto step = [&](int t, int h) __attribute__((always_inline)) {
      load(t + SETS, SETS == 2 ? h : 0);
      __builtin_amdgcn_sched_barrier(0);
      if (wave_live && t * KT <= wmost) {
        scores(smem + h * STAGE);
        weights(t);
        values(smem + h * STAGE + KT * KP);
      }
      __builtin_amdgcn_sched_barrier(0);
      // Past the last tile the second set may never have been loaded. Above 128 the one set holds the last tile again, whose
      // scan says nothing new; asking there takes 8192 tokens of 16 heads of 256 from 1619 to 1760 us, by registers spilled.
      if (DP > 128 || t + 1 < t1) store(t + 1, h ^ 1, SETS == 2 ? h ^ 1 : 0);
      __syncthreads();
    };
    int t = t0;
    for (; t + 1 < t1; t += 2) {
      step(t, 0);
      step(t + 1, 1);
    }
    if (t < t1) step(t, 0);
  }
  if (!live) return;
  if (s_odd)
    for (int j = max(max(all, 0) & ~(KT - 1), t0 * KT); j <= min(lim, t1 * KT - 1); ++j) {
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
  if (a.splits > 1) {
    const long long at = ((long long)(q0 + token) * a.HK * a.G + head) * a.splits + split;
    if (half == 0) {
      a.ml[2 * at] = m;
      a.ml[2 * at + 1] = l;
    }
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<f32x4*>(a.part + at * DP + 32 * i + 8 * k + 4 * half) =
            (f32x4){o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]};
    return;
  }
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
  T* const out = reinterpret_cast<T*>(a.out) + (long long)(q0 + token) * a.out_row + (long long)head * a.out_head;
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = 32 * i + 8 * k + 4 * half;
      struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w.e[e] = mean_out<T>(l == 0.f ? 0.f : o[i][4 * k + e] * inv, o[i][4 * k + e]);
      if (d < a.D) __builtin_memcpy(__builtin_assume_aligned(out + d, 8), &w, 8);
    }
}

// out = sum_s O_s 2^(m_s - m) / sum_s l_s 2^(m_s - m) over the parts s of a query row's keys: one wave a row, 4 columns a
// lane. Rows of no sequence stay.
template <typename T, int DP>
__global__ __launch_bounds__(BLOCK) void k_prompt_join(PromptDev a) {
  const int lane = threadIdx.x % WAVE, H = a.HK * a.G;
  const long long id = (long long)blockIdx.x * NWAVES + threadIdx.x / WAVE;
  if (id >= (long long)a.q_rows * H) return;
  const int row = (int)(id / H), head = (int)(id % H);
  bool mine = false;
  for (int b = lane; b < a.B; b += WAVE) {
    int first;
    const int n = packed(a.cu_q, b, a.q_rows, &first);
    mine |= row >= first && row < first + n;
  }
  if (!__any(mine)) return;
  float m = -__builtin_inff(), l = 0.f;
  f32x4 v = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.ml[2 * (id * a.splits + s)]);
  const float base = m == -__builtin_inff() ? 0.f : m;
  const int d = 4 * lane;
  for (int s = 0; s < a.splits; ++s) {
    const long long at = id * a.splits + s;
    // not 0: an infinity that a row sees stays one, whatever it weighs
    const float f = fmaxf(__builtin_amdgcn_exp2f(a.ml[2 * at] - base), 1.4e-45f);
    l += a.ml[2 * at + 1] * f;
    const f32x4 x = *reinterpret_cast<const f32x4*>(a.part + at * DP + min(d, DP - 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i] * f;
  }
  if (d >= a.D) return;
  T* out = reinterpret_cast<T*>(a.out) + (long long)row * a.out_row + (long long)head * a.out_head + d;
  struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w.e[i] = mean_out<T>(l == 0.f ? 0.f : v[i] / l, v[i]);
  __builtin_memcpy(__builtin_assume_aligned(out, 8), &w, 8);
}

template <typename T, int DP, int WQ>
pi_status launch_prompt_t(pi_ctx* c, const PromptDev& a) {
  constexpr size_t lds = prompt_lds<DP>();
  auto kern = k_prompt<T, DP, WQ>;
  PI_HIP(c, allow_lds(kern, lds));
  PI_HIP(c, launch_kb(c, 0, kern, dim3((unsigned)(a.tiles * a.HK * a.splits)), 64 * WQ, lds, a));
  if (a.splits > 1) {
    const long long rows = (long long)a.q_rows * a.HK * a.G;
    PI_HIP(c, launch_k(c, 0, k_prompt_join<T, DP>, dim3((unsigned)((rows + NWAVES - 1) / NWAVES)), 0, a));
  }
  return PI_OK;
}

template <typename T, int DP>
pi_status launch_prompt_d(pi_ctx* c, const PromptDev& a, int wq) {
  if constexpr (DP <= 128) {
    if (wq == 4) return launch_prompt_t<T, DP, 4>(c, a);
  }
  return launch_prompt_t<T, DP, 8>(c, a);
}

template <typename T>
pi_status launch_prompt(pi_ctx* c, const PromptDev& a, int wq) {
  switch (padded_dim(a.D)) {
    case 64: return launch_prompt_d<T, 64>(c, a, wq);
    case 96: return launch_prompt_d<T, 96>(c, a, wq);
    case 128: return launch_prompt_d<T, 128>(c, a, wq);
    default: return launch_prompt_d<T, 256>(c, a, wq);
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
  // what the kernels use is its product with log2(e)
  if (!(scale > 0.f) || scale > 0x1p127f) return fail(ctx, PI_ERR_INVALID, "scale must be above 0 and at most 2^127");
  // row numbers of a head's group, and workgroups, are 32-bit numbers
  if (((int64_t)max_tokens + 256ll * max_batch) * heads >= 1ll << 29)
    return fail(ctx, PI_ERR_UNSUPPORTED, "%d tokens of %d sequences and %d heads are too many", max_tokens, max_batch, heads);
  // scratch of the largest call whose keys are split, of however many rows
  const int HK = kv_heads, G = heads / kv_heads, DP = padded_dim(head_dim);
  size_t rows = 0;
  for (int64_t n = 1; n <= max_tokens; n += std::max<int64_t>(1, n / 64)) {
    const int64_t next = std::min<int64_t>(max_tokens, n + std::max<int64_t>(1, n / 64) - 1);
    const PromptPlan q = prompt_plan(ctx->cus, HK, G, DP, (int)n, 1, INT64_MAX);
    if (q.splits > 1) rows = std::max(rows, (size_t)next * heads * q.splits);
  }
  PI_HIP(ctx, hipSetDevice(ctx->device));
  uint8_t* ws = nullptr;
  if (rows > 0 && hipMalloc(reinterpret_cast<void**>(&ws), rows * (DP + 2) * 4) != hipSuccess) {
    (void)hipGetLastError();
    return fail(ctx, PI_ERR_OOM, "prompt attention scratch of %zu bytes", rows * (DP + 2) * 4);
  }
  pi_prompt* p = new (std::nothrow) pi_prompt{ctx, dtype, heads, kv_heads, head_dim, max_tokens, max_batch, scale, ws, rows};
  if (p == nullptr) {
    (void)hipFree(ws);
    return fail(ctx, PI_ERR_OOM, "host allocation failed");
  }
  ctx_retain(ctx);
  *out = p;
  return PI_OK;
}

void pi_prompt_destroy(pi_prompt* p) {
  if (p == nullptr) return;
  (void)hipSetDevice(p->ctx->device);
  (void)hipFree(p->ws);
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
  if (a.k_rows > 1 && (a.k_row < 0 || a.v_row < 0 || a.k_row >= 1 << 24 || a.v_row >= 1 << 24))
    return fail(ctx, PI_ERR_UNSUPPORTED, "rows of k and v are less than 2^24 elements apart");
  if (a.k_rows > 0) {
    PI_TRY(check_bnh(ctx, "k", a.k, 0, a.k_row, a.k_head));
    PI_TRY(check_bnh(ctx, "v", a.v, 0, a.v_row, a.v_head));
  }
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const int HK = prompt->kv_heads, G = prompt->heads / HK, DP = padded_dim(prompt->head_dim);
  PromptPlan p = prompt_plan(ctx->cus, HK, G, DP, a.q_rows, a.B, a.k_rows);
  const int64_t rows = (int64_t)a.q_rows * prompt->heads;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(p.splits, (int64_t)prompt->ws_rows / rows));
  float* part = reinterpret_cast<float*>(prompt->ws);
  const PromptDev d{static_cast<const uint8_t*>(a.q), static_cast<const uint8_t*>(a.k), static_cast<const uint8_t*>(a.v),
                    static_cast<uint8_t*>(a.out), a.cu_q, a.cu_k != nullptr ? a.cu_k : a.cu_q, a.q_row, a.q_head, a.k_row,
                    a.k_head, a.v_row, a.v_head, a.out_row, a.out_head, part, part + prompt->ws_rows * DP, a.B, a.q_rows,
                    a.k_rows, HK, G, prompt->head_dim, p.tiles, p.splits, prompt->scale * 1.4426950408889634f};
  return prompt->dtype == PI_T_F16 ? launch_prompt<half_t>(ctx, d, p.wq) : launch_prompt<bf16_t>(ctx, d, p.wq);
}

}  // extern "C"
