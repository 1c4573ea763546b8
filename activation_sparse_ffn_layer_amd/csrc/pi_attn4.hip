// Attention of drafted trees over a 4-bit cache (pi_tree_attention on a pi_kv4_create cache).
//
// The same products as over a plain cache: for a tile of keys, S^T = K Q^T leaves a lane keys of one query
// row, and exp(S - max) is, as it lies, the B operand of O^T += V^T P^T. The cached tiles come as
// codes and scales; both operands are fp16, which holds (code - 8) * scale exactly, whatever type the
// queries have: bf16 queries are scaled by a power of two to lie below 2^15, where fp16 holds their 8
// bits. The new nodes (64 at most, of the queries' type) are a tile of their own behind the cached ones.
//
// A dword of codes has elements 4w..4w+3 and 16+4w..16+4w+3 of its block: so they lie in LDS and in the
// products, at positions 8w..8w+7. Queries are loaded in that order and outputs put back from it.
#include <algorithm>

#include "pi_attn.hpp"

using namespace pi;

namespace {

constexpr int KT4 = 64;  // keys of a tile
constexpr float SHIFT4 = 14.f;  // weights of cached tiles are carried times 2^14, as over a plain fp16 cache
// New nodes in bf16 may hold values up to fp32's end: after the cached tiles the sums go on times 2^-8, so that 64 of them
// with weights up to 1 stay in range. Where nodes are fp16, the 2^14 stays. A factor of 2^-22 loses nothing of the cached
// tiles' sums: a weight that fp16 holds is 2^-38 or more of the largest, a cached value 0 or 2^-24 or more.
template <typename T> constexpr float SHIFT_NEW = __is_same(T, half_t) ? SHIFT4 : -8.f;
template <typename T> constexpr float CACHED_TO_NEW = __is_same(T, half_t) ? 1.f : 0x1p-22f;
static_assert(SHIFT_NEW<bf16_t> - SHIFT4 == -22.f, "the factor between the two");

// Elements 4w..4w+3 and 16+4w..+3 of a block, at p and 32 bytes on.
__device__ __forceinline__ u32x4 two_pieces(const uint8_t* p) {
  const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + 32);
  return (u32x4){a.x, a.y, b.x, b.y};
}

// Four code bytes (byte j: element j | element j + 16 << 4) as 8 fp16 values (code - 8) * scale: elements
// 0..3, then 16..19 of the dword's place. A byte of 0..15 is, as an fp8 number (e4m3), its value times
// 2^-9, below 8 subnormal: the conversion takes pairs to fp16 with that power of two, and the product with the
// scale takes off 8 scale, both exact, in one rounding. 11 instructions, where nibbles put into
// fp16's mantissa by masks take 13 (124 against 117 us at one token of 64 sequences).
__device__ __forceinline__ u32x4 q4_values(uint32_t codes, uint16_t scale) {
  const half_t s = __builtin_bit_cast(half_t, scale), c = s * (half_t)-8.f;
  const half2_t s2 = (half2_t){s, s}, c2 = (half2_t){c, c};
  const uint32_t lo = codes & 0x0F0F0F0Fu, hi = (codes >> 4) & 0x0F0F0F0Fu;
  half2_t v[4];
  v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, false);
  v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, true);
  v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, false);
  v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, true);
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v[i], s2, c2));
  return o;
}
// The first W dwords of a block's codes at p, 16 bytes each.
template <int W>
__device__ __forceinline__ void put_codes(uint8_t* p, u32x4 codes, uint16_t scale) {
#pragma unroll
  for (int w = 0; w < W; ++w) *reinterpret_cast<u32x4*>(p + 16 * w) = q4_values(codes[w], scale);
}

// The exact fp16 form of a query's fragments (the value that scale_c then takes off): bf16 queries times the
// power of two that brings the row's largest element into [2^14, 2^15). Elements more than 2^31 times smaller lose bits in
// fp16, more than 2^39 times smaller ones are zeros: where the largest meets keys of its own size, that is far below the
// score's rounding in fp32; where it meets zeros, it is a limit of the operator.
__device__ __forceinline__ float rows_max(float v);
template <bool QUARTERS, int KS>  // a row's elements are in four lanes, not two
__device__ __forceinline__ float queries_to_half(u32x4 (&qf)[KS]) {
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      big = fmaxf(big, fmaxf(fabsf(u2f(qf[i][e] << 16)), fabsf(u2f(qf[i][e] & 0xFFFF0000u))));
  big = QUARTERS ? rows_max(big) : swap_max(big);
  const int e = big > 0.f && big < __builtin_inff() ? 14 - ilogbf(big) : 0;
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const half2_t h = (half2_t){(half_t)ldexpf(u2f(qf[i][x] << 16), e), (half_t)ldexpf(u2f(qf[i][x] & 0xFFFF0000u), e)};
      qf[i][x] = __builtin_bit_cast(uint32_t, h);
    }
  return ldexpf(1.f, -e);
}

// The tiles of all sequences, one after another (a sequence's cached tiles, then its new nodes as one), are cut into
// equal spans, one per workgroup and head: `per` tiles each, which may begin in one sequence and end in a later one. A
// span's part of sequence b leaves its partial result in slot span + b, so that a sequence's parts follow each other.
// With one span a sequence (`whole`) nothing is left to join.
template <int KT>
__device__ __forceinline__ uint32_t tiles4(const AttnDev& a, int b) {
  return ((uint32_t)kv_len(a.c, a.ctx_len, b) + (uint32_t)(KT - 1)) / (uint32_t)KT + 1;
}
struct Span {
  int b;
  uint32_t t0, left;  // first tile, of sequence b; tiles from it on
};
// The launch sees to it that the tiles of all sequences are fewer than 2^31.
template <int KT>
__device__ __forceinline__ bool find_span(const AttnDev& a, int span, Span* o) {
  const int lane = threadIdx.x % WAVE;
  if (a.B == 1) {
    const uint32_t all = tiles4<KT>(a, 0), per = (all + a.slots - 1) / a.slots, begin = span * per;
    *o = Span{0, begin, min(per, all - begin)};
    return begin < all;
  }
  const uint32_t mine = lane < a.B ? tiles4<KT>(a, lane) : 0;  // the sequence of this lane; more than 64 are read again
  uint32_t all = mine;
  for (int b = lane + WAVE; b < a.B; b += WAVE) all += tiles4<KT>(a, b);
  all = sum_tiles(all);
  const uint32_t per = (all + a.slots - 1) / a.slots, begin = span * per;
  if (begin >= all) return false;
  uint32_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += WAVE) {
    const uint32_t n = b0 == 0 ? mine : b0 + lane < a.B ? tiles4<KT>(a, b0 + lane) : 0;
    uint32_t incl = n;
#pragma unroll
    for (int s = 1; s < WAVE; s <<= 1) {
      const uint32_t t = __shfl_up(incl, s, WAVE);
      if (lane >= s) incl += t;
    }
    const uint64_t hit = __ballot(before + incl > begin);
    if (hit != 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      o->b = __builtin_amdgcn_readfirstlane(b0 + l);
      o->t0 = __builtin_amdgcn_readfirstlane(begin - before - __shfl(incl - n, l, WAVE));
      o->left = min(per, all - begin);
      return true;
    }
    before += __shfl(incl, WAVE - 1, WAVE);
  }
  return false;
}
// out = sum_s O_s 2^(m_s - m) / sum_s l_s 2^(m_s - m) over a sequence's parts s, one wave per query row, as
// k_attn_join for chunks.
template <typename T, int DP, int KT>
__global__ __launch_bounds__(BLOCK) void k_attn4_join(AttnDev a, int rows) {
  const int lane = threadIdx.x % WAVE;
  const int id = blockIdx.x * NWAVES + threadIdx.x / WAVE;  // (b, hk, r)
  if (id >= rows) return;
  const int r = id % a.R, hk = id / a.R % a.HK, b = id / a.R / a.HK;
  uint32_t all, before = 0;
  const uint32_t mine = tiles4<KT>(a, b);
  if (a.B == 1) {
    all = mine;
  } else {
    all = 0;
    for (int i = lane; i < a.B; i += WAVE) {
      const uint32_t n = tiles4<KT>(a, i);
      all += n;
      before += i < b ? n : 0;
    }
    all = sum_tiles(all);
    before = sum_tiles(before);
  }
  const uint32_t per = (all + a.slots - 1) / a.slots;
  const int s0 = (int)(before / per), count = (int)((before + mine - 1) / per) - s0 + 1;
  if (count > 1) join_parts<T, DP>(a, b, hk, r, s0 + b, count);
}

template <int DP> constexpr size_t attn4_lds() { return 2 * (size_t)KT4 * (k_pitch<DP>() + v_pitch<DP>()); }

// WQ waves of 32 query rows each; tiles of 64 keys in LDS, which all waves read: a tile is turned into fp16 once for all of
// them. Bound by products, exponentials and that conversion in turn: 26 nodes of 4 sequences (up to 32768 positions, 64
// heads, 8 kv, of 128, 90 GFLOP; 208 of 256 rows in use) 153 to 173 us, of 64 102; up to 16384 positions, 32 heads (8 kv) of
// 256, whose registers spill, 202 in fp16 and 304 in bf16. Four waves for all: 182; twice as many spans: 190.
template <typename T, int DP, int WQ>
__global__ __launch_bounds__(64 * WQ) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_tree_attn4(AttnDev a, Kv4Dev sc) {
  constexpr int KB = 2, KT = KT4, NT = 64 * WQ, KS = DP / 16, DB = DP / 32;
  constexpr int KP = k_pitch<DP>(), VP = v_pitch<DP>(), STAGE = KT * (KP + VP);
  constexpr int ITEMS = 2 * KT * DB, PASS = (ITEMS + NT - 1) / NT;  // blocks of a tile's keys and values
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_odd;  // a new node's value row holds an infinity or a NaN
  const int pair = blockIdx.x % (a.slots * a.HK), rt = blockIdx.x / (a.slots * a.HK);
  const int hk = pair % a.HK, span = pair / a.HK;
  Span sp;
  if (!find_span<KT>(a, span, &sp)) return;
  const int wave = threadIdx.x / WAVE, nblocks = a.D / 32;
  for (; sp.left > 0; ++sp.b, sp.t0 = 0) {
  int lane = threadIdx.x % WAVE;
  asm("" : "+v"(lane));  // what follows from it is worked out for each part: kept over all, it would fill the registers
  const int half = lane >> 5, l32 = lane & 31;
  const int b = sp.b, len = kv_len(a.c, a.ctx_len, b);
  const int tiles = (int)tiles4<KT>(a, b), new_tile = tiles - 1;
  const int t0 = (int)sp.t0, t1 = t0 + min((int)sp.left, tiles - t0);
  sp.left -= t1 - t0;
  const bool direct = t0 == 0 && t1 == tiles;  // all of a sequence
  __syncthreads();  // LDS is free for this part
  if (threadIdx.x == 0) s_odd = 0;

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
      const u32x4 v = two_pieces(p);
      qf[i] = in ? v : (u32x4){0, 0, 0, 0};
    }
  };
  load_q();
  float scale_c = a.scale2;  // of the cached tiles' products
  if constexpr (__is_same(T, bf16_t)) scale_c *= queries_to_half<false>(qf);

  typedef const __attribute__((address_space(1))) uint8_t* gp;  // global by type: a generic load counts as LDS too
  const gp zero = (gp)(const uint8_t*)&attn_zero;
  const gp kc = (gp)(static_cast<const uint8_t*>(a.c.k) + (long long)hk * a.c.head_stride);
  const gp vc = (gp)(static_cast<const uint8_t*>(a.c.v) + (long long)hk * a.c.head_stride);
  const gp ks = (gp)(reinterpret_cast<const uint8_t*>(sc.ks + (long long)hk * sc.head));
  const gp vs = (gp)(reinterpret_cast<const uint8_t*>(sc.vs + (long long)hk * sc.head));
  const int32_t* const pages = a.c.table + (long long)b * a.c.table_stride;
  const uint32_t last = len > 0 ? (uint32_t)(len - 1) / a.c.div.page : 0, npages = (uint32_t)a.c.pages;
  const uint32_t page_units = (uint32_t)(a.c.page_stride >> 4), token_units = (uint32_t)(a.c.token_stride >> 4);  // 16 bytes
  const uint32_t spage = (uint32_t)sc.page, stoken = (uint32_t)sc.token;
  // item i of a tile: values after keys, key (i % (KT DB)) / DB, block i % DB
  struct Place {
    uint32_t off;
    int id;
  };
  Place pl[2][PASS];  // of two tiles in turn
  u32x4 cr[2][PASS];
  uint16_t sr[2][PASS];
  auto ids = [&](int tile, int p) {
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int item = (int)threadIdx.x + i * NT;
      const uint32_t n = page_of(a.c.div, (uint32_t)tile * KT + (uint32_t)(item % (KT * DB) / DB), &pl[p][i].off);
      pl[p][i].id = pages[min(n, last)];
    }
  };
  auto load = [&](int tile, int set) {
    const int end = tile_from_end<KT>(tile, len);
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int item = (int)threadIdx.x + i * NT, key = item % (KT * DB) / DB, blk = item % DB;
      const bool val = item >= KT * DB;
      const uint32_t pg = (uint32_t)pl[set][i].id, of = pl[set][i].off;
      const bool in = end + key < 0 && blk < nblocks && pg < npages && tile < new_tile;
      const uint64_t at = (((uint64_t)pg * page_units + (uint64_t)of * token_units) << 4) + 16 * blk;
      const uint64_t st = ((uint64_t)pg * spage + (uint64_t)of * stoken + blk) << 1;
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
      put_codes<4>(base, cr[set][i], sr[set][i]);
    }
  };

  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) o[i] = (f32x16){};
  float m = -__builtin_inff(), l = 0.f;  // running maximum (log2 domain); this half's sum

  // One tile. `seen` (bit j: key j) counts where `masked`.
  auto compute = [&](auto type, int stage, float scale2, float shift, bool masked, uint64_t seen) __attribute__((always_inline)) {
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
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][r], scale2, shift - base));
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

  const int cend = min(t1, new_tile);  // the part's cached tiles
  if (t0 < cend) {
    ids(t0, 0);
    ids(t0 + 1, 1);
    load(t0, 0);
    ids(t0 + 2, 0);
    load(t0 + 1, 1);
    store(0, 0);
    __syncthreads();
    auto step = [&](int t, int h) {
      ids(t + 3, h ^ 1);  // before the rows: waiting for the page numbers leaves the rows in flight
      load(t + 2, h);
      __builtin_amdgcn_sched_barrier(0);
      const int left = -tile_from_end<KT>(t, len);
      if (wave_live) compute(half_t(), h, scale_c, SHIFT4, left < KT, left < KT ? (1ull << left) - 1 : 0);
      __builtin_amdgcn_sched_barrier(0);
      store(h ^ 1, h ^ 1);
      __syncthreads();
    };
    int t = t0;
    for (; t + 1 < cend; t += 2) {
      step(t, 0);
      step(t + 1, 1);
    }
    if (t < cend) step(t, 0);
  }
  if constexpr (CACHED_TO_NEW<T> != 1.f) {
    l *= CACHED_TO_NEW<T>;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] *= CACHED_TO_NEW<T>;
  }
  if (t1 > new_tile) {
    __syncthreads();  // s_odd is 0
    const long long nhead = (long long)hk * a.kv_head + (long long)b * a.kv_batch;
    for (int i = threadIdx.x; i < 2 * KT * DB * 4; i += NT) {  // 8 positions each
      const int w = i & 3, blk = (i >> 2) % DB, key = (i >> 2) / DB % KT;
      const bool val = i >= KT * DB * 4;
      const bool in = key < a.N && blk < nblocks;
      const uint8_t* p = (val ? a.vn : a.kn) + 2 * (nhead + (in ? (long long)key * a.kv_node + 32 * blk + 4 * w : 0));
      u32x4 v = two_pieces(p);
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
    if (wave_live) compute(T(), 0, a.scale2, SHIFT_NEW<T>, true, seen);
    if (s_odd && live)
      for (int j = 0; j < a.N; ++j)
        if ((seen >> j) & 1) {
          const T* x = reinterpret_cast<const T*>(a.vn) + nhead + (long long)j * a.kv_node + 16 * half;
#pragma unroll
          for (int i = 0; i < DB; ++i)
            if (i < nblocks)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const float y = (float)x[32 * i + r];
                if (!(fabsf(y) < __builtin_inff())) o[i][r] += y;
              }
        }
  }
  l = swap_add(l);
  if (!live) continue;
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
  T* const out = reinterpret_cast<T*>(a.out) + (long long)b * a.out_batch + (long long)node * a.out_node + (long long)head * a.out_head;
  const long long at = ((long long)(span + b) * a.HK + hk) * a.R + row;
  if (!direct && half == 0) {
    a.ml[2 * at] = m;
    a.ml[2 * at + 1] = l;
  }
#pragma unroll
  for (int i = 0; i < DB; ++i) {
    if (i >= nblocks) break;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = 32 * i + 16 * half + 4 * k;
      const f32x4 v = (f32x4){o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]};
      if (direct) {
        struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w.e[e] = mean_out<T>(l == 0.f ? 0.f : v[e] * inv, v[e]);
        __builtin_memcpy(__builtin_assume_aligned(out + d, 8), &w, 8);
      } else {
        *reinterpret_cast<f32x4*>(a.part + at * DP + d) = v;
      }
    }
  }
  }
}

// Up to 32 query rows: four waves, each with 32 keys of a tile of 128 to itself. The products are the
// 16x16x32 ones: 16 keys by NQ times 16 rows, a lane with one key's block of 32 elements (lanes 16g..16g+15 have
// block 4j + g of 16 keys; of heads of 64, half a block), so that a wave's loads are whole rows. Keys go
// from memory through registers straight into the products; values pass through LDS of the wave's own,
// where they are transposed. No barrier is in the loop. FULL: heads fill the padded size.
// One token of 64 sequences (8191 positions, 64 heads, 8 kv, of 128; 430 MB): 101 to 113 us, of which the loads alone take
// 97 and the rest alone 60; 149 where pages of 5 tokens hold a token's heads side by side. Heads of 32 and of 64: 67 us (of
// 32 half of each wave's lanes hold a block twice), of 96: 96; 32 sequences of heads of 256, whose registers spill: 151. One
// token over 512 positions of 32 heads: 11 us, three dependent loads and the join's launch.
// Workgroups a CU holds (waves per SIMD), and tiles in flight: three with one tile ahead where the registers allow it, 112
// against 118 us with two of two tiles (one token of 64 sequences).
constexpr int few_wgs(int DP, int rows) { return DP > 128 ? (rows > 16 ? 1 : 2) : rows > 16 ? 2 : 3; }
constexpr int FEW_KEYS = 32, FEW_WAVES = 4, FEW_KT = FEW_KEYS * FEW_WAVES;
template <int DP> constexpr int few_pitch() { return 2 * DP + 32; }
template <int DP> constexpr size_t few_lds(int rows) {
  const size_t tiles = (size_t)FEW_WAVES * FEW_KEYS * few_pitch<DP>();
  const size_t merge = (size_t)FEW_WAVES * rows * (DP + 4) * 4 + (size_t)FEW_WAVES * 32 * 2 * 4;
  return tiles > merge ? tiles : merge;
}

template <typename T> struct Mm16;
template <> struct Mm16<half_t> {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  }
};
template <> struct Mm16<bf16_t> {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a), __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
  }
};
// Over the lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float rows_max(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return swap_max(fmaxf(u2f(p[0]), u2f(p[1])));
}
__device__ __forceinline__ float rows_add(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return swap_add(u2f(p[0]) + u2f(p[1]));
}

// UNI: the 16 keys of a product are consecutive rows of one page (pages of a multiple of 16 tokens, or one page a
// sequence), whose address is worked out once for the wave; otherwise each lane finds its key's page.
template <typename T, int DP, int NQ, bool FULL, bool UNI>
__global__ __launch_bounds__(64 * FEW_WAVES) __attribute__((amdgpu_waves_per_eu(few_wgs(DP, 16 * NQ))))
void k_attn4_few(AttnDev a, Kv4Dev sc) {
  constexpr int DEPTH = few_wgs(DP, 16 * NQ) == 3 ? 1 : 2;
  constexpr int KT = FEW_KT, KS = DP / 32, DT = DP / 16, VP = few_pitch<DP>();
  constexpr int NJ = DP >= 128 ? DP / 128 : 1, W = DP >= 128 ? 4 : 2;  // blocks of a lane and their dwords that it has
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  // A span's heads go to one XCD (workgroups are dealt to the 8 in turn): where a token's heads lie next to each other,
  // they share cache lines.
  const int turn = blockIdx.x / 8, hk = turn % a.HK, span = turn / a.HK * 8 + blockIdx.x % 8;
  Span sp;
  if (span >= a.slots || !find_span<KT>(a, span, &sp)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), nblocks = a.D / 32;
  for (; sp.left > 0; ++sp.b, sp.t0 = 0) {
  int lane = threadIdx.x % WAVE;
  asm("" : "+v"(lane));  // what follows from it is worked out for each part: kept over all, it would fill the registers
  const int g = lane >> 4, c16 = lane & 15;
  auto block = [&](int j) { return DP >= 128 ? 4 * j + g : g & 1; };
  const int w0 = DP >= 128 ? 0 : 2 * (g >> 1);  // the first dword of a block that this lane has
  // where an 8-element piece of a block lies in a head of 16-bit elements: dword w of block j
  auto piece = [&](int j, int w) { return 32 * block(j) + 4 * (w0 + w); };

  const int b = sp.b, len = kv_len(a.c, a.ctx_len, b);
  const int tiles = (int)tiles4<KT>(a, b), new_tile = tiles - 1;
  const int t0 = (int)sp.t0, t1 = t0 + min((int)sp.left, tiles - t0);
  sp.left -= t1 - t0;
  const bool direct = t0 == 0 && t1 == tiles;  // all of a sequence

  u32x4 qf[NQ][KS];
  auto load_q = [&]() {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int row = 16 * q + c16;
      const bool live = row < a.R;
      const int node = live ? row / a.G : 0, head = hk * a.G + (live ? row % a.G : 0);
      const uint8_t* qp = a.q + 2 * ((long long)b * a.q_batch + (long long)node * a.q_node + (long long)head * a.q_head);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const bool in = live && block(i / W) < nblocks;
        const uint8_t* p = qp + (in ? 2 * piece(i / W, i % W) : 0);
        const u32x4 v = two_pieces(p);
        qf[q][i] = in ? v : (u32x4){0, 0, 0, 0};
      }
    }
  };
  typedef const __attribute__((address_space(1))) uint8_t* gp;
  typedef const __attribute__((address_space(1))) u32x4* gp16;
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  typedef const __attribute__((address_space(1))) u32x2_t* gp8;
  typedef const __attribute__((address_space(1))) uint16_t* gp2;
  const gp zero = (gp)(const uint8_t*)&attn_zero;
  // An absent block beyond the head's last one: that one again. The queries are zeros there, and its values
  // are not put out.
  const int blk0 = FULL ? block(0) : min(block(0), nblocks - 1), o0 = 16 * blk0 + 4 * w0;
  const gp kc = (gp)(static_cast<const uint8_t*>(a.c.k) + (long long)hk * a.c.head_stride);
  const gp vc = (gp)(static_cast<const uint8_t*>(a.c.v) + (long long)hk * a.c.head_stride);
  const gp ks = (gp)(reinterpret_cast<const uint8_t*>(sc.ks + (long long)hk * sc.head));
  const gp vs = (gp)(reinterpret_cast<const uint8_t*>(sc.vs + (long long)hk * sc.head));
  // Page numbers of two tiles in turn. A tile's are asked for before the rows of the tile in front of it: waiting for
  // them leaves those rows in flight.
  typedef const __attribute__((address_space(4))) int32_t* table_t;
  const table_t pages = (table_t)(a.c.table + (long long)b * a.c.table_stride);
  const uint32_t last = len > 0 ? (uint32_t)(len - 1) / a.c.div.page : 0, npages = (uint32_t)a.c.pages;
  const uint32_t page_units = (uint32_t)(a.c.page_stride >> 4), token_units = (uint32_t)(a.c.token_stride >> 4);  // 16 bytes
  const uint32_t spage = (uint32_t)sc.page, stoken = (uint32_t)sc.token;
  const uint32_t row_at = UNI ? c16 * (token_units << 4) + o0 : o0, srow_at = UNI ? 2 * (c16 * stoken + blk0) : 2 * blk0;
  uint32_t off[2][2];
  int id[2][2];
  auto ids = [&](int tile, int p) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t n = page_of(a.c.div, (uint32_t)tile * KT + (uint32_t)(wave * FEW_KEYS + 16 * t + (UNI ? 0 : c16)), &off[p][t]);
      id[p][t] = pages[min(n, last)];
    }
  };
  u32x4 kr[DEPTH][2][NJ], vr[DEPTH][2][NJ];
  uint16_t ksr[DEPTH][2][NJ], vsr[DEPTH][2][NJ];
  auto load = [&](int tile, int set, int p) {
    const int end = tile_from_end<KT>(tile, len) + wave * FEW_KEYS;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t pg = (uint32_t)id[p][t], at = off[p][t];
      // the page holds this key (UNI: the first of the 16) of a cached tile of the sequence
      const bool in = end + 16 * t + (UNI ? 0 : c16) < 0 && pg < npages && tile < new_tile;
      const uint64_t c = ((uint64_t)pg * page_units + (uint64_t)at * token_units) << 4;
      const uint64_t s = ((uint64_t)pg * spage + (uint64_t)at * stoken) << 1;
      const gp kp = in ? kc + c : zero, vp = in ? vc + c : zero, ksp = in ? ks + s : zero, vsp = in ? vs + s : zero;
      // UNI: keys past the sequence's end stand for the first of the 16, which every row sees; they weigh nothing
      const bool row = UNI ? in && end + 16 * t + c16 < 0 : true;
      const uint32_t ro = row ? row_at : o0, so = row ? srow_at : 2 * blk0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int more = FULL ? 4 * j : min(block(j), nblocks - 1) - blk0;  // blocks past the first
        if constexpr (W == 4) {
          kr[set][t][j] = *(gp16)(kp + ro + 16 * more);
          vr[set][t][j] = *(gp16)(vp + ro + 16 * more);
        } else {
          const auto k = *(gp8)(kp + ro), v = *(gp8)(vp + ro);
          kr[set][t][j] = (u32x4){k.x, k.y, 0, 0};
          vr[set][t][j] = (u32x4){v.x, v.y, 0, 0};
        }
        ksr[set][t][j] = *(gp2)(ksp + so + 2 * more);
        vsr[set][t][j] = *(gp2)(vsp + so + 2 * more);
      }
    }
  };

  // the first tiles' rows are in flight before the queries are waited for
  const int cend = min(t1, new_tile);
  if (t0 < cend) {
    ids(t0, 0);
    ids(t0 + 1, 1);
  }
  load_q();
  if (t0 < cend) {
    load(t0, 0, 0);
    if constexpr (DEPTH == 2) {
      ids(t0 + 2, 0);
      load(t0 + 1, 1, 1);
    }
  }
  float scale_c[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    scale_c[q] = a.scale2;
    if constexpr (__is_same(T, bf16_t)) scale_c[q] *= queries_to_half<true>(qf[q]);
  }

  f32x4 o[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    m[q] = -__builtin_inff();
    l[q] = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[q][i] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }
  uint8_t* const vt = smem + wave * FEW_KEYS * VP;  // this wave's values, a row per key
  const uint8_t* const vl = vt + (4 * g + (c16 >> 2)) * VP + 8 * (c16 & 3);

  // s[q][t]: scores of keys 16t + 4g + 0..3 and row 16q + c16
  auto weigh = [&](auto type, f32x4 (&s)[NQ][2], const float (&scale2)[NQ], float shift) __attribute__((always_inline)) {
    typedef decltype(type) M;
    typedef M m8 __attribute__((ext_vector_type(8)));
    u32x4 pf[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float top = -__builtin_inff();
#pragma unroll
      for (int r = 0; r < 8; ++r) top = fmaxf(top, s[q][r >> 2][r & 3]);
      top = rows_max(top) * scale2[q];
      const float mn = fmaxf(m[q], top);
      const float base = mn == -__builtin_inff() ? 0.f : mn;  // nothing seen so far: weights 0
      if (__any(mn > m[q])) {
        const float f = __builtin_amdgcn_exp2f(m[q] - base);
        l[q] *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[q][i][r] *= f;
      }
      m[q] = mn;
      m8 p;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[q][r >> 2][r & 3], scale2[q], shift - base));
        l[q] += w;
        p[r] = (M)w;
      }
      pf[q] = __builtin_bit_cast(u32x4, p);
    }
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      typedef __attribute__((address_space(3))) short4_t* lds4;
      struct { short4_t x, y; } v;
      v.x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(vl + 32 * i));
      v.y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(vl + 32 * i + 16 * VP));
#pragma unroll
      for (int q = 0; q < NQ; ++q) o[q][i] = Mm16<M>::mfma(__builtin_bit_cast(u32x4, v), pf[q], o[q][i]);
    }
  };
  auto hide = [&](f32x4 (&s)[NQ][2], int q, uint32_t seen) {  // bit k: key k is seen
    const uint32_t vis = seen >> (4 * g);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      s[q][r >> 2][r & 3] = bfi_sel(0u - ((vis >> (16 * (r >> 2) + (r & 3))) & 1u), s[q][r >> 2][r & 3], -__builtin_inff());
  };

  auto step = [&](int t, int p) __attribute__((always_inline)) {  // p: t's parity from the first tile on
    const int set = p % DEPTH;
    f32x4 s[NQ][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) s[q][k] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        put_codes<W>(vt + (16 * k + c16) * VP + 64 * block(j) + 16 * w0, vr[set][k][j], vsr[set][k][j]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const u32x4 kf = q4_values(kr[set][k][j][w], ksr[set][k][j]);
#pragma unroll
          for (int q = 0; q < NQ; ++q) s[q][k] = Mm16<half_t>::mfma(kf, qf[q][W * j + w], s[q][k]);
        }
      }
    }
    ids(t + DEPTH + 1, (p + DEPTH + 1) & 1);
    load(t + DEPTH, set, (p + DEPTH) & 1);
    const int left = -(tile_from_end<KT>(t, len) + wave * FEW_KEYS);  // this wave's keys that are held
    if (left < FEW_KEYS) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) hide(s, q, left <= 0 ? 0u : (1u << left) - 1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    weigh(half_t(), s, scale_c, SHIFT4);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  if (t0 < cend) {
    int t = t0;
    for (; t + 1 < cend; t += 2) {
      step(t, 0);
      step(t + 1, 1);
    }
    if (t < cend) step(t, 0);
  }
  if constexpr (CACHED_TO_NEW<T> != 1.f) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      l[q] *= CACHED_TO_NEW<T>;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[q][i][r] *= CACHED_TO_NEW<T>;
    }
  }
  if (t1 > new_tile && wave == 0) {
    // the new nodes (N <= R <= 32), one a lane and key tile, in the order of the positions
    const long long nhead = (long long)b * a.kv_batch + (long long)hk * a.kv_head;
    if constexpr (!__is_same(T, half_t)) load_q();
    f32x4 s[NQ][2];
    float scale_n[NQ];
    bool odd = false;  // a value row holds an infinity or a NaN
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int n = 16 * k + c16;
#pragma unroll
      for (int q = 0; q < NQ; ++q) s[q][k] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const bool in = n < a.N && block(i / W) < nblocks;
        const long long e = 2 * (nhead + (in ? (long long)n * a.kv_node + piece(i / W, i % W) : 0));
        u32x4 kf = two_pieces(a.kn + e);
        u32x4 v = two_pieces(a.vn + e);
        if (!in) kf = v = (u32x4){0, 0, 0, 0};
        // a weight of zero times an infinity or a NaN is a NaN: left out here, added below to the rows that see it
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t lo = (v[x] & Mm<T>::EXP) == Mm<T>::EXP ? 0xFFFFu : 0u;
          const uint32_t hi = (v[x] & (Mm<T>::EXP << 16)) == Mm<T>::EXP << 16 ? 0xFFFF0000u : 0u;
          odd |= (lo | hi) != 0;
          v[x] &= ~(lo | hi);
        }
        *reinterpret_cast<u32x4*>(vt + n * VP + 64 * block(i / W) + 16 * (w0 + i % W)) = v;
#pragma unroll
        for (int q = 0; q < NQ; ++q) s[q][k] = Mm16<T>::mfma(kf, qf[q][i], s[q][k]);
      }
    }
    uint32_t seen[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int row = 16 * q + c16, node = row < a.R ? row / a.G : 0;
      const uint64_t w = a.tree != nullptr ? a.tree[(long long)b * a.N + node] : (2ull << node) - 1;
      seen[q] = (uint32_t)(w & ((1ull << a.N) - 1));
      hide(s, q, seen[q]);
      scale_n[q] = a.scale2;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    weigh(T(), s, scale_n, SHIFT_NEW<T>);
    if (__any(odd))
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        for (int j = 0; j < a.N; ++j)
          if ((seen[q] >> j) & 1) {
            const T* x = reinterpret_cast<const T*>(a.vn) + nhead + (long long)j * a.kv_node + 16 * (g & 1) + 4 * (g >> 1);
#pragma unroll
            for (int i = 0; i < DT; ++i)
              if (i / 2 < nblocks)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float y = (float)x[32 * (i / 2) + 8 * (i & 1) + r];
                  if (!(fabsf(y) < __builtin_inff())) o[q][i][r] += y;
                }
          }
  }
  // join the four waves through LDS, rows below R only
  constexpr int OP = DP + 4;
  float* const ob = reinterpret_cast<float*>(smem);               // [waves][R][OP]
  float* const ml = ob + FEW_WAVES * a.R * OP;                    // [waves][32][2]
  __syncthreads();  // the tiles are free
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    l[q] = rows_add(l[q]);
    if (g == 0) {
      ml[(wave * 32 + 16 * q + c16) * 2] = m[q];
      ml[(wave * 32 + 16 * q + c16) * 2 + 1] = l[q];
    }
  }
  __syncthreads();
  auto joined = [&](int row, float* base) {  // the maximum of all waves and their sum at it
    float mt = -__builtin_inff(), lt = 0.f;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) mt = fmaxf(mt, ml[(w * 32 + row) * 2]);
    *base = mt;
    const float z = mt == -__builtin_inff() ? 0.f : mt;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) lt += ml[(w * 32 + row) * 2 + 1] * __builtin_amdgcn_exp2f(ml[(w * 32 + row) * 2] - z);
    return lt;
  };
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int row = 16 * q + c16;
    if (row < a.R) {
      float mt;
      joined(row, &mt);
      // not 0: an infinity that a row sees stays one, whatever it weighs
      const float f = fmaxf(__builtin_amdgcn_exp2f(m[q] - (mt == -__builtin_inff() ? 0.f : mt)), 1.4e-45f);
      float* to = ob + (wave * a.R + row) * OP + 16 * (g & 1) + 4 * (g >> 1);
#pragma unroll
      for (int i = 0; i < DT; ++i)
        *reinterpret_cast<f32x4*>(to + 32 * (i / 2) + 8 * (i & 1)) = (f32x4){o[q][i][0] * f, o[q][i][1] * f, o[q][i][2] * f, o[q][i][3] * f};
    }
  }
  __syncthreads();
  constexpr int QP = DP / 4;  // quads of a row
  for (int i = threadIdx.x; i < a.R * QP; i += 64 * FEW_WAVES) {
    const int r = i / QP, d = 4 * (i % QP);
    if (d >= a.D) continue;
    float mt;
    const float lt = joined(r, &mt);
    f32x4 v = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) v += *reinterpret_cast<const f32x4*>(ob + (w * a.R + r) * OP + d);
    if (direct) {
      const float inv = lt > 0.f || lt != lt ? 1.0f / lt : 0.f;
      T* out = reinterpret_cast<T*>(a.out) + (long long)b * a.out_batch + (long long)(r / a.G) * a.out_node +
               (long long)(hk * a.G + r % a.G) * a.out_head + d;
      struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w.e[e] = mean_out<T>(lt == 0.f ? 0.f : v[e] * inv, v[e]);
      __builtin_memcpy(__builtin_assume_aligned(out, 8), &w, 8);
    } else {
      const long long at = ((long long)(span + b) * a.HK + hk) * a.R + r;
      *reinterpret_cast<f32x4*>(a.part + at * DP + d) = v;
      if (d == 0) {
        a.ml[2 * at] = mt;
        a.ml[2 * at + 1] = lt;
      }
    }
  }
  __syncthreads();  // LDS is free for the next part
  }
}

template <typename T, int DP, int KT>
pi_status launch_join4(pi_ctx* c, const AttnDev& a) {
  const int rows = a.B * a.HK * a.R;
  PI_HIP(c, launch_k(c, 0, k_attn4_join<T, DP, KT>, dim3((rows + NWAVES - 1) / NWAVES), 0, a, rows));
  return PI_OK;
}

template <typename T, int DP, int NQ, bool FULL>
pi_status launch_few_t(pi_ctx* c, const AttnDev& a, const Kv4Dev& sc) {
  const bool uni = (a.c.div.page % 16 == 0 || (int)a.c.div.page == a.c.capacity) && a.c.token_stride < 1 << 27 && sc.token < 1 << 26;
  auto kern = uni ? k_attn4_few<T, DP, NQ, FULL, true> : k_attn4_few<T, DP, NQ, FULL, false>;
  PI_HIP(c, allow_lds(kern, few_lds<DP>(16 * NQ)));
  PI_HIP(c, launch_kb(c, 0, kern, dim3((unsigned)((a.slots + 7) / 8 * 8 * a.HK)), 64 * FEW_WAVES, few_lds<DP>(a.R), a, sc));
  return launch_join4<T, DP, FEW_KT>(c, a);
}
template <typename T, int DP>
pi_status launch_few(pi_ctx* c, const AttnDev& a, const Kv4Dev& sc) {
  if (a.D == DP) return a.R <= 16 ? launch_few_t<T, DP, 1, true>(c, a, sc) : launch_few_t<T, DP, 2, true>(c, a, sc);
  return a.R <= 16 ? launch_few_t<T, DP, 1, false>(c, a, sc) : launch_few_t<T, DP, 2, false>(c, a, sc);
}

template <typename T, int DP, int WQ>
pi_status launch_attn4_t(pi_ctx* c, const AttnDev& a, const Kv4Dev& sc) {
  constexpr size_t lds = attn4_lds<DP>();
  auto kern = k_tree_attn4<T, DP, WQ>;
  PI_HIP(c, allow_lds(kern, lds));
  PI_HIP(c, launch_kb(c, 0, kern, dim3((unsigned)(a.slots * a.HK * a.row_tiles)), 64 * WQ, lds, a, sc));
  return launch_join4<T, DP, KT4>(c, a);
}

template <typename T>
pi_status launch_attn4_d(pi_ctx* c, const AttnDev& a, const Kv4Dev& sc, int wq) {
  switch (padded_dim4(a.D)) {
    case 64: return wq == 1 ? launch_few<T, 64>(c, a, sc) : wq == 4 ? launch_attn4_t<T, 64, 4>(c, a, sc) : launch_attn4_t<T, 64, 8>(c, a, sc);
    case 128: return wq == 1 ? launch_few<T, 128>(c, a, sc) : wq == 4 ? launch_attn4_t<T, 128, 4>(c, a, sc) : launch_attn4_t<T, 128, 8>(c, a, sc);
    default: return wq == 1 ? launch_few<T, 256>(c, a, sc) : launch_attn4_t<T, 256, 8>(c, a, sc);
  }
}

}  // namespace

namespace pi {

AttnPlan attn4_plan(int cus, int HK, int rows, int, int DP) {
  AttnPlan p;
  p.wq = rows <= 32 ? 1 : DP > 128 || rows > 128 ? 8 : 4;
  p.row_tiles = (rows + 32 * p.wq - 1) / (32 * p.wq);
  const int wgs = p.wq == 1 ? few_wgs(DP, rows) * cus : p.wq == 8 ? cus : 2 * cus;  // workgroups the chip holds at once
  p.slots = std::max(1, wgs / (HK * p.row_tiles));
  return p;
}

pi_status launch_attn4(pi_ctx* c, const AttnDev& a, const Kv4Dev& scales, int wq, bool f16) {
  if ((int64_t)a.B * ((a.c.capacity + KT4 - 1) / KT4 + 1) >= 1ll << 31)
    return fail(c, PI_ERR_UNSUPPORTED, "%d sequences of %d positions: fewer than 2^37 positions in all", a.B, a.c.capacity);
  return f16 ? launch_attn4_d<half_t>(c, a, scales, wq) : launch_attn4_d<bf16_t>(c, a, scales, wq);
}

}  // namespace pi
