// Attention of drafted trees over a 4-bit cache (pi_tree_attention on a pi_kv4_create cache).
//
// The same products as over a plain cache: for a tile of keys, S^T = K Q^T leaves a lane keys of one query
// row, and exp(S - max) is, as it lies, the B operand of O^T += V^T P^T. The cached tiles come as
// codes and scales; both operands are fp16, which holds (code - 8) * scale exactly, whatever type the
// queries have: bf16 queries are scaled by a power of two to lie below 2^15, where fp16 holds their 8
// bits. The new nodes (64 at most, of the queries' type) are a tile of their own behind the cached ones.
//
// Nibbles turn into fp16 pairs in an order that costs least (q4_pairs): a block's 32 elements lie in
// LDS at positions 8w + e, w the dword of codes, e = 0..7 for elements 4w + {0, 2, 1, 3} and 16 + 4w +
// {0, 2, 1, 3}. Queries are loaded in that order and outputs put back from it.
#include <algorithm>

#include "pi_attn.hpp"

using namespace pi;

namespace {

constexpr int KT4 = 64;  // keys of a tile
constexpr float SHIFT4 = 14.f;  // weights are carried times 2^14, as over a plain fp16 cache

// Elements 4w..4w+3 and 16+4w..+3 of a block in the order of the positions, from a row of 16-bit elements.
__device__ __forceinline__ u32x4 in_order(uint2 a, uint2 b) {
  constexpr uint32_t LO = 0x05040100u, HI = 0x07060302u;  // both low halves, both high halves
  return (u32x4){__builtin_amdgcn_perm(a.y, a.x, LO), __builtin_amdgcn_perm(a.y, a.x, HI),
                 __builtin_amdgcn_perm(b.y, b.x, LO), __builtin_amdgcn_perm(b.y, b.x, HI)};
}

// A block's 16 code bytes as 32 fp16 values at p, 4 x 16 bytes.
__device__ __forceinline__ void put_block(uint8_t* p, u32x4 codes, uint16_t scale) {
  const half_t s = __builtin_bit_cast(half_t, scale);
  const half2_t s2 = (half2_t){s, s};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    half2_t v[4];
    q4_pairs(codes[w], v);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(uint32_t, v[i] * s2);
    *reinterpret_cast<u32x4*>(p + 16 * w) = o;
  }
}

template <int DP> constexpr size_t attn4_lds() { return 2 * (size_t)KT4 * (k_pitch<DP>() + v_pitch<DP>()); }

// WQ waves of 32 query rows each; tiles of 64 keys in LDS, which all waves read.
template <typename T, int DP, int WQ>
__global__ __launch_bounds__(64 * WQ) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_tree_attn4(AttnDev a, Kv4Dev sc) {
  constexpr int KB = 2, KT = KT4, NT = 64 * WQ, KS = DP / 16, DB = DP / 32;
  constexpr int KP = k_pitch<DP>(), VP = v_pitch<DP>(), STAGE = KT * (KP + VP);
  constexpr int ITEMS = 2 * KT * DB, PASS = (ITEMS + NT - 1) / NT;  // blocks of a tile's keys and values
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_odd;  // a new node's value row holds an infinity or a NaN
  const int pair = blockIdx.x % (a.slots * a.HK), rt = blockIdx.x / (a.slots * a.HK);
  const int hk = pair % a.HK, slot = pair / a.HK;
  Chunk ch;
  if (!find_chunk<KT, true>(a, slot, &ch)) return;
  ch = Chunk{__builtin_amdgcn_readfirstlane(ch.b), __builtin_amdgcn_readfirstlane(ch.t0), __builtin_amdgcn_readfirstlane(ch.t1),
             __builtin_amdgcn_readfirstlane(ch.count), __builtin_amdgcn_readfirstlane(ch.first)};
  if (threadIdx.x == 0) s_odd = 0;
  const int b = ch.b;
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, half = lane >> 5, l32 = lane & 31;
  const int len = kv_len(a.c, a.ctx_len, b);
  const int new_tile = key_tiles<KT, true>(a, b) - 1, nblocks = a.D / 32;

  // this lane's query row
  const int row = (rt * WQ + wave) * 32 + l32;
  const bool live = row < a.R, wave_live = (rt * WQ + wave) * 32 < a.R;
  const int node = live ? row / a.G : 0, head = hk * a.G + (live ? row % a.G : 0);
  const uint8_t* const qp = a.q + 2 * ((long long)b * a.q_batch + (long long)node * a.q_node + (long long)head * a.q_head);
  // product i's 8 elements of this half: dword w = 2 (i % 2) + half of block i / 2
  u32x4 qf[KS];
  auto load_q = [&]() {
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const bool in = live && i / 2 < nblocks;
      const uint8_t* p = qp + (in ? 2 * (32 * (i / 2) + 4 * (2 * (i & 1) + half)) : 0);
      const u32x4 v = in_order(*reinterpret_cast<const uint2*>(p), *reinterpret_cast<const uint2*>(p + 32));
      qf[i] = in ? v : (u32x4){0, 0, 0, 0};
    }
  };
  load_q();
  float scale_c = a.scale2;  // of the cached tiles' products
  if constexpr (__is_same(T, bf16_t)) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        big = fmaxf(big, fmaxf(fabsf(u2f(qf[i][e] << 16)), fabsf(u2f(qf[i][e] & 0xFFFF0000u))));
    big = swap_max(big);
    // the power of two that brings the row's largest element into [2^14, 2^15); a product with it may
    // be subnormal in fp16 only where it is 2^28 times smaller
    const int e = big > 0.f && big < __builtin_inff() ? 14 - ilogbf(big) : 0;
    scale_c = ldexpf(scale_c, -e);
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const half2_t h = (half2_t){(half_t)ldexpf(u2f(qf[i][x] << 16), e), (half_t)ldexpf(u2f(qf[i][x] & 0xFFFF0000u), e)};
        qf[i][x] = __builtin_bit_cast(uint32_t, h);
      }
  }

  typedef const __attribute__((address_space(1))) uint8_t* gp;  // global by type: a generic load counts as LDS too
  const gp zero = (gp)(const uint8_t*)&attn_zero;
  const gp kc = (gp)(static_cast<const uint8_t*>(a.c.k) + (long long)hk * a.c.head_stride);
  const gp vc = (gp)(static_cast<const uint8_t*>(a.c.v) + (long long)hk * a.c.head_stride);
  const gp ks = (gp)(reinterpret_cast<const uint8_t*>(sc.ks + (long long)hk * sc.head));
  const gp vs = (gp)(reinterpret_cast<const uint8_t*>(sc.vs + (long long)hk * sc.head));
  const int32_t* const pages = a.c.table + (long long)b * a.c.table_stride;
  const uint32_t last = len > 0 ? (uint32_t)(len - 1) / a.c.div.page : 0;
  // item i of a tile: values after keys, key (i % (KT DB)) / DB, block i % DB
  struct Place {
    uint32_t off;
    int id;
  };
  Place pl[PASS];
  u32x4 cr[2][PASS];
  uint16_t sr[2][PASS];
  auto ids = [&](int tile) {
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int item = (int)threadIdx.x + i * NT;
      const uint32_t n = page_of(a.c.div, (uint32_t)tile * KT + (uint32_t)(item % (KT * DB) / DB), &pl[i].off);
      pl[i].id = pages[min(n, last)];
    }
  };
  auto load = [&](int tile, int set) {
    const int end = tile_from_end<KT>(tile, len);
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int item = (int)threadIdx.x + i * NT, key = item % (KT * DB) / DB, blk = item % DB;
      const bool val = item >= KT * DB;
      const bool in = end + key < 0 && blk < nblocks && (uint32_t)pl[i].id < (uint32_t)a.c.pages && tile < new_tile;
      const long long at = (long long)pl[i].id * a.c.page_stride + (long long)pl[i].off * a.c.token_stride + 16 * blk;
      const long long st = 2 * ((long long)pl[i].id * sc.page + (long long)pl[i].off * sc.token + blk);
      const gp p = in ? (val ? vc : kc) + at : zero, s = in ? (val ? vs : ks) + st : zero;
      cr[set][i] = *(const __attribute__((address_space(1))) u32x4*)p;
      sr[set][i] = *(const __attribute__((address_space(1))) uint16_t*)s;
    }
  };
  auto store = [&](int stage, int set) {
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int item = (int)threadIdx.x + i * NT, key = item % (KT * DB) / DB, blk = item % DB;
      if (ITEMS % NT != 0 && item >= ITEMS) break;
      uint8_t* base = smem + stage * STAGE + (item >= KT * DB ? KT * KP + key * VP : key * KP) + 64 * blk;
      put_block(base, cr[set][i], sr[set][i]);
    }
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) o[i] = (f32x16){};
  float m = -__builtin_inff(), l = 0.f;  // running maximum (log2 domain); this half's sum

  // One tile. `seen` (bit j: key j) counts where `masked`.
  auto compute = [&](auto type, int stage, float scale2, bool masked, uint64_t seen) __attribute__((always_inline)) {
    typedef decltype(type) M;
    typedef typename Mm<M>::v8 v8;
    const uint8_t* kb0 = smem + stage * STAGE;
    const uint8_t* vb0 = kb0 + KT * KP;
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = (f32x16){};
#pragma unroll
      for (int i = 0; i < KS; ++i)
        s[kb] = Mm<M>::mfma(__builtin_bit_cast(v8, ld16(kb0 + (kb * 32 + l32) * KP + 32 * i + 16 * half)),
                            __builtin_bit_cast(v8, qf[i]), s[kb]);
    }
    if (masked) {
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
    top = swap_max(top) * scale2;
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
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][r], scale2, SHIFT4 - base));
        l += w;
        pf[kb][r >> 3][r & 7] = (M)w;
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
          o[i] = Mm<M>::mfma(__builtin_bit_cast(v8, v), pf[kb][st], o[i]);
        }
  };

  const int cend = min(ch.t1, new_tile);  // the chunk's cached tiles
  if (ch.t0 < cend) {
    ids(ch.t0);
    load(ch.t0, 0);
    ids(ch.t0 + 1);
    load(ch.t0 + 1, 1);
    ids(ch.t0 + 2);
    store(0, 0);
    __syncthreads();
    auto step = [&](int t, int h) {
      load(t + 2, h);
      ids(t + 3);
      __builtin_amdgcn_sched_barrier(0);
      const int left = -tile_from_end<KT>(t, len);
      if (wave_live) compute(half_t(), h, scale_c, left < KT, left < KT ? (1ull << left) - 1 : 0);
      __builtin_amdgcn_sched_barrier(0);
      store(h ^ 1, h ^ 1);
      __syncthreads();
    };
    int t = ch.t0;
    for (; t + 1 < cend; t += 2) {
      step(t, 0);
      step(t + 1, 1);
    }
    if (t < cend) step(t, 0);
  }
  if (ch.t1 > new_tile) {
    __syncthreads();  // s_odd is 0
    const long long nhead = (long long)hk * a.kv_head + (long long)b * a.kv_batch;
    for (int i = threadIdx.x; i < 2 * KT * DB * 4; i += NT) {  // 8 positions each
      const int w = i & 3, blk = (i >> 2) % DB, key = (i >> 2) / DB % KT;
      const bool val = i >= KT * DB * 4;
      const bool in = key < a.N && blk < nblocks;
      const uint8_t* p = (val ? a.vn : a.kn) + 2 * (nhead + (in ? (long long)key * a.kv_node + 32 * blk + 4 * w : 0));
      u32x4 v = in_order(*reinterpret_cast<const uint2*>(p), *reinterpret_cast<const uint2*>(p + 32));
      if (!in) v = (u32x4){0, 0, 0, 0};
      if (val) {
        // A weight of zero times an infinity or a NaN is a NaN: such elements stay out of the product and are
        // added to the rows that see them at the end.
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = (v[e] & Mm<T>::EXP) == Mm<T>::EXP ? 0xFFFFu : 0u;
          const uint32_t hi = (v[e] & (Mm<T>::EXP << 16)) == Mm<T>::EXP << 16 ? 0xFFFF0000u : 0u;
          if (lo | hi) s_odd = 1;
          v[e] &= ~(lo | hi);
        }
      }
      *reinterpret_cast<u32x4*>(smem + (val ? KT * KP + key * VP : key * KP) + 64 * blk + 16 * w) = v;
    }
    __syncthreads();
    if constexpr (!__is_same(T, half_t)) load_q();
    uint64_t seen = a.tree != nullptr ? a.tree[(long long)b * a.N + node] : (2ull << node) - 1;
    if (a.N < 64) seen &= (1ull << a.N) - 1;
    if (wave_live) compute(T(), 0, a.scale2, true, seen);
    if (s_odd && live)
      for (int j = 0; j < a.N; ++j)
        if ((seen >> j) & 1) {
          const T* x = reinterpret_cast<const T*>(a.vn) + nhead + (long long)j * a.kv_node + 16 * half;
#pragma unroll
          for (int i = 0; i < DB; ++i)
            if (i < nblocks)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const float y = (float)x[32 * i + 4 * (r >> 2) + ((r & 1) << 1 | (r >> 1 & 1))];
                if (!(fabsf(y) < __builtin_inff())) o[i][r] += y;
              }
        }
  }
  l = swap_add(l);
  if (!live) return;
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
  T* const out = reinterpret_cast<T*>(a.out) + (long long)b * a.out_batch + (long long)node * a.out_node + (long long)head * a.out_head;
  const long long at = ((long long)slot * a.HK + hk) * a.R + row;
  if (ch.count != 1 && half == 0) {
    a.ml[2 * at] = m;
    a.ml[2 * at + 1] = l;
  }
#pragma unroll
  for (int i = 0; i < DB; ++i) {
    if (i >= nblocks) break;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = 32 * i + 16 * half + 4 * k;
      const f32x4 v = (f32x4){o[i][4 * k], o[i][4 * k + 2], o[i][4 * k + 1], o[i][4 * k + 3]};
      if (ch.count == 1) {
        struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w.e[e] = (T)(l == 0.f ? 0.f : v[e] * inv);
        __builtin_memcpy(__builtin_assume_aligned(out + d, 8), &w, 8);
      } else {
        *reinterpret_cast<f32x4*>(a.part + at * DP + d) = v;
      }
    }
  }
}

template <typename T, int DP, int WQ>
pi_status launch_attn4_t(pi_ctx* c, const AttnDev& a, const Kv4Dev& sc) {
  constexpr size_t lds = attn4_lds<DP>();
  auto kern = k_tree_attn4<T, DP, WQ>;
  PI_HIP(c, allow_lds(kern, lds));
  PI_HIP(c, launch_kb(c, 0, kern, dim3((unsigned)(a.slots * a.HK * a.row_tiles)), 64 * WQ, lds, a, sc));
  if (a.slots > a.B) {
    const int rows = a.B * a.HK * a.R;
    PI_HIP(c, launch_k(c, 0, k_attn_join<T, DP, KT4, true>, dim3((rows + NWAVES - 1) / NWAVES), 0, a, rows));
  }
  return PI_OK;
}

template <typename T>
pi_status launch_attn4_d(pi_ctx* c, const AttnDev& a, const Kv4Dev& sc, int wq) {
  switch (padded_dim4(a.D)) {
    case 64: return wq == 4 ? launch_attn4_t<T, 64, 4>(c, a, sc) : launch_attn4_t<T, 64, 8>(c, a, sc);
    case 128: return wq == 4 ? launch_attn4_t<T, 128, 4>(c, a, sc) : launch_attn4_t<T, 128, 8>(c, a, sc);
    default: return launch_attn4_t<T, 256, 8>(c, a, sc);
  }
}

}  // namespace

namespace pi {

AttnPlan attn4_plan(int cus, int HK, int rows, int B, int DP) {
  AttnPlan p;
  p.wq = DP > 128 || rows > 128 ? 8 : 4;
  p.row_tiles = (rows + 32 * p.wq - 1) / (32 * p.wq);
  const int wgs = p.wq == 8 ? cus : 2 * cus;  // workgroups the chip holds at once
  p.slots = std::max(B, wgs / (HK * p.row_tiles));
  return p;
}

pi_status launch_attn4(pi_ctx* c, const AttnDev& a, const Kv4Dev& scales, int wq, bool f16) {
  return f16 ? launch_attn4_d<half_t>(c, a, scales, wq) : launch_attn4_d<bf16_t>(c, a, scales, wq);
}

}  // namespace pi
