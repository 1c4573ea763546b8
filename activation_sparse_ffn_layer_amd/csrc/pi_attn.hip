// Attention of drafted trees over the paged cache (pi_tree_attention).
//
// A key/value head's query rows (N nodes x G heads of the group) are columns of the matrix
// cores' 32x32x16 products. For a tile of keys, S^T = K Q^T leaves each lane 16 keys of one
// query column, so the softmax's maximum and sum are over a lane's registers and one exchange
// between the wave's halves; exp(S - max) is then, as it lies, the B operand of
// O^T += V^T P^T, where V^T comes from row-major V by transposing LDS reads. The maximum and the
// sum run along (one pass over the cache) and are held in fp32, as are S and O; P is rounded to
// the cache's type for the second product (half a step of that type per weight, as large as the
// rounding of the output itself).
//
// The keys of a sequence are one axis: its cached positions, then its N new nodes. The axis is
// cut in chunks of whole tiles, equally long for all sequences, so that the chunks of all heads
// fill the chip once; partial results (O, max, sum) are joined by k_attn_join.
//
// Many rows are bound by the products and the weights' exponentials, which take the SIMDs nearly in
// turn (47% and 48% of the busy cycles) at a clock that falls to 1.75 GHz: 64 nodes of 64 heads (8
// key heads) over 65536 positions of 128, 137 GFLOP, 160 to 210 us and 10 us for the join. 26 nodes
// of 4 sequences (25 000 positions, 108 MB): 43 us and 10 us. One node of 32 heads over 512
// positions is a chain of latencies: 9.6 us and 4.6 us; joining in the last workgroup to arrive
// instead took 22 us (its release fences). Four waves of 32 rows (two workgroups per CU) were
// slower than eight, 62 against 54 us and 227 against 190; so was working a block's scores out
// under the weights of the one before, 60 and 211.
#include <algorithm>
#include <new>

#include "pi_attn.hpp"

using namespace pi;

namespace {

template <int DP, int WQ, int WK, int KB>
constexpr size_t attn_lds() {
  const size_t kt = 32 * KB * WK;
  const size_t tile = kt * (k_pitch<DP>() + v_pitch<DP>()) * (WQ > 1 ? 2 : 1);
  const size_t merge = WK > 1 ? (size_t)WQ * WK * 32 * (DP + 4) * 4 + (size_t)WQ * WK * 64 * 4 : 0;
  return tile > merge ? tile : merge;
}

// Lanes that load one row, a power of two, and the 16-byte piece that a lane loads: where a row has
// fewer pieces than lanes (heads of 96), the lanes past them load the last one again.
constexpr int row_lanes(int DP) { return DP <= 64 ? 8 : DP <= 128 ? 16 : 32; }
constexpr int row_piece(int DP, int lane) { return lane < DP / 8 ? lane : DP / 8 - 1; }
constexpr bool loads_stay_in_row(int DP) {
  for (int lane = 0; lane < row_lanes(DP); ++lane)
    if (16 * row_piece(DP, lane) + 16 > 2 * DP) return false;
  return row_lanes(DP) * 8 >= DP;
}
static_assert(loads_stay_in_row(64) && loads_stay_in_row(96) && loads_stay_in_row(128) && loads_stay_in_row(256),
              "a tile's loads end with the row, which may be the cache's last");

// WQ waves along the query rows (32 each), WK along a tile's keys (32 KB each). With WQ == 1 a
// wave loads and reads its own keys only and the tile loop has no barrier.
template <typename T, int DP, int WQ, int WK, int KB>
__global__ __launch_bounds__(64 * WQ * WK) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_tree_attn(AttnDev a) {
  constexpr int KW = 32 * KB, KT = KW * WK, NT = 64 * WQ * WK;
  constexpr bool OWN = WQ == 1;                          // tiles private to a wave
  constexpr int LPR = row_lanes(DP);
  constexpr int LROWS = OWN ? KW : KT, LTHR = OWN ? 64 : NT;
  constexpr int RPP = LTHR / LPR, PASS = LROWS / RPP;
  static_assert(PASS >= 1 && LROWS % RPP == 0, "a tile is whole passes");
  constexpr int KS = DP / 16, DB = DP / 32;
  constexpr int KP = k_pitch<DP>(), VP = v_pitch<DP>();
  typedef typename Mm<T>::v8 v8;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_odd;  // a new node's value row holds an infinity or a NaN
  const int pair = blockIdx.x % (a.slots * a.HK), rt = blockIdx.x / (a.slots * a.HK);
  const int hk = pair % a.HK, slot = pair / a.HK;
  Chunk ch;
  if (!find_chunk<KT>(a, slot, &ch)) return;
  // the same on every lane, which the shuffles that found it hide: kept in scalar registers
  ch = Chunk{__builtin_amdgcn_readfirstlane(ch.b), __builtin_amdgcn_readfirstlane(ch.t0), __builtin_amdgcn_readfirstlane(ch.t1),
             __builtin_amdgcn_readfirstlane(ch.count), __builtin_amdgcn_readfirstlane(ch.first)};
  if (threadIdx.x == 0) s_odd = 0;
  __syncthreads();
  const int b = ch.b;
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, half = lane >> 5, l32 = lane & 31;
  const int wq = wave / WK, wk = wave % WK;
  const int len = kv_len(a.c, a.ctx_len, b);

  // this lane's query row
  const int row = (rt * WQ + wq) * 32 + l32;
  const bool live = row < a.R;
  const bool wave_live = (rt * WQ + wq) * 32 < a.R;
  const int node = live ? row / a.G : 0, head = hk * a.G + (live ? row % a.G : 0);
  v8 qf[KS];
  {
    const uint8_t* qp = a.q + 2 * ((long long)b * a.q_batch + (long long)node * a.q_node + (long long)head * a.q_head);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 16 * s + 8 * half;
      qf[s] = __builtin_bit_cast(v8, ld16_or0(qp + 2 * (d < a.D ? d : 0), live && d < a.D));
    }
  }
  uint64_t seen = a.tree != nullptr ? a.tree[(long long)b * a.N + node] : (2ull << node) - 1;
  if (a.N < 64) seen &= (1ull << a.N) - 1;

  // loading: pass i of a thread is row lr + i * RPP of the tile (of the wave's part), piece lc
  const int lt = OWN ? lane : (int)threadIdx.x;
  const int lr = lt / LPR + (OWN ? wk * KW : 0), lc = lt % LPR;
  const int le = 8 * row_piece(DP, lc);
  const bool piece_in = lc * 8 < a.D;
  uint8_t* const ks = smem + (OWN ? wk * KW * (KP + VP) : 0);
  const long long nhead = (long long)hk * a.kv_head + (long long)b * a.kv_batch;
  // A tile's rows are loaded in two steps, their pages' numbers one tile ahead of the rows. What is
  // not there is read from zeros in memory: a select after the load would wait for it. `ready`
  // keeps the compiler from computing an address behind a branch.
  constexpr int SETS = OWN ? 1 : 2;
  u32x4 kr[SETS][PASS], vr[SETS][PASS];
  const int32_t* const pages = a.c.table + (long long)b * a.c.table_stride;
  // global pointers by type: a generic load counts as a read of LDS too, and holds those up
  typedef const __attribute__((address_space(1))) uint8_t* gp;
  const gp zero = (gp)(const uint8_t*)&attn_zero;
  const gp kc = (gp)(static_cast<const uint8_t*>(a.c.k) + 2 * ((long long)hk * a.c.head_stride + le));
  const gp vc = (gp)(static_cast<const uint8_t*>(a.c.v) + 2 * ((long long)hk * a.c.head_stride + le));
  const gp kn = (gp)(a.kn + 2 * (nhead + le)), vn = (gp)(a.vn + 2 * (nhead + le));
  const uint32_t page_units = (uint32_t)(a.c.page_stride >> 3), token_units = (uint32_t)(a.c.token_stride >> 3);  // 16 bytes
  const long long node_bytes = 2 * a.kv_node;
  const uint32_t npages = (uint32_t)a.c.pages;
  auto ready = [](gp p) {
    asm("" : "+v"(p));
    return p;
  };
  // The place of each row of a tile: page of the sequence and offset in it, and the page's number in
  // the cache. Tiles follow each other, so a place moves on by the quotient and rest of KT / page.
  struct Place {
    uint32_t n, off;
    int id;
  };
  const uint32_t page = a.c.div.page, last = len > 0 ? (uint32_t)(len - 1) / page : 0;
  const uint32_t kt_n = KT / page, kt_off = KT % page;
  Place pl[OWN ? 1 : 2][PASS];  // of two tiles in turn
  auto ids = [&](Place (&p)[PASS], const Place (&before)[PASS]) {
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      uint32_t n = before[i].n + kt_n, off = before[i].off + kt_off;
      const bool over = off >= page;
      p[i].n = n + (over ? 1 : 0);
      p[i].off = off - (over ? page : 0);
      p[i].id = pages[min(p[i].n, last)];
    }
  };
  auto load = [&](int tile, int set, const Place (&p)[PASS]) {
    gp kp[PASS], vp[PASS];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const unsigned long long at = (unsigned long long)(uint32_t)p[i].id * page_units + (unsigned long long)p[i].off * token_units;
      kp[i] = kc + (at << 4);
      vp[i] = vc + (at << 4);
      bad |= (uint32_t)p[i].id >= npages;
    }
    const int end = tile_from_end<KT>(tile, len);
    if (end + KT > 0 || a.D != DP || __any(bad)) {  // not all rows are whole rows of the cache
      const bool in = piece_in & (tile < ch.t1);
#pragma unroll
      for (int i = 0; i < PASS; ++i) {
        const int j = end + lr + i * RPP;
        const bool old = in & (j < 0) & ((uint32_t)p[i].id < npages), fresh = in & (j >= 0) & (j < a.N);
        const gp k = ready(kn + j * node_bytes), v = ready(vn + j * node_bytes);
        kp[i] = old ? ready(kp[i]) : zero;
        vp[i] = old ? ready(vp[i]) : zero;
        kp[i] = fresh ? k : kp[i];
        vp[i] = fresh ? v : vp[i];
      }
    }
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      kr[set][i] = *(const __attribute__((address_space(1))) u32x4*)kp[i];
      vr[set][i] = *(const __attribute__((address_space(1))) u32x4*)vp[i];
    }
  };
  // a stage is K rows, then V rows
  constexpr int STAGE = LROWS * (KP + VP);
  auto store = [&](int tile, int stage, int set) {
    uint8_t* base = ks + stage * STAGE;
    const int end = tile_from_end<KT>(tile, len);
    if (end + KT > 0) {
      // A weight of zero times an infinity or a NaN is a NaN: such elements of the new nodes, whom
      // not every row sees, stay out of the product and are added to the rows that see them at
      // the end (every row sees the cached positions, where nothing has to be done).
#pragma unroll
      for (int i = 0; i < PASS; ++i)
        if (end + lr + i * RPP >= 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = vr[set][i][e];
            const uint32_t lo = (w & Mm<T>::EXP) == Mm<T>::EXP ? 0xFFFFu : 0u;
            const uint32_t hi = (w & (Mm<T>::EXP << 16)) == Mm<T>::EXP << 16 ? 0xFFFF0000u : 0u;
            if (lo | hi) s_odd = 1;
            vr[set][i][e] = w & ~(lo | hi);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int r = lt / LPR + i * RPP;
      if (DP / 8 == LPR || lc < DP / 8) {
        *reinterpret_cast<u32x4*>(base + r * KP + lc * 16) = kr[set][i];
        *reinterpret_cast<u32x4*>(base + LROWS * KP + r * VP + lc * 16) = vr[set][i];
      }
    }
  };

  // The two waves of a SIMD would go through products and weights in step: with one preferred, its
  // weights are worked out under the other's products (189 against 196 us at 512 rows, 65536 keys).
  if (WQ == 8 && wave < 4) __builtin_amdgcn_s_setprio(1);
  f32x16 o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) o[i] = (f32x16){};
  float m = -__builtin_inff(), l = 0.f;  // running maximum (log2 domain); this half's sum

  auto compute = [&](int tile, int stage) {
    const uint8_t* kb0 = ks + stage * STAGE + (OWN ? 0 : wk * KW) * KP;
    const uint8_t* vb0 = ks + stage * STAGE + LROWS * KP + (OWN ? 0 : wk * KW) * VP;
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = (f32x16){};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const v8 kf = __builtin_bit_cast(v8, ld16(kb0 + (kb * 32 + l32) * KP + 32 * i + 16 * half));
        s[kb] = Mm<T>::mfma(kf, qf[i], s[kb]);
      }
    }
    // the reads of K four ahead of the products
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int i = 0; i < KB * KS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    const int end = tile_from_end<KT>(tile, len) + wk * KW;
    if (end + KW > 0) {  // the tile reaches the new nodes or the end
      // Masked as bit operations: with a select on `position < len || bit`, the compiler put the
      // -inf of the untaken side over the accumulators of lanes that keep theirs.
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int j0 = end + kb * 32;  // the node of the block's first key
        uint32_t vis = j0 >= 64 ? 0u : (uint32_t)(seen >> (j0 & 63));
        if (j0 < 0) vis = j0 <= -32 ? ~0u : (uint32_t)(seen << -j0) | ((1u << -j0) - 1);
        vis >>= 4 * half;
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
    // The base of the weights is the maximum itself: the largest weight is 1 exactly. (Letting it fall
    // behind by up to 2^8, to scale the sums less often, gained 2% and cost bf16 a quarter of an
    // error of half a step.)
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
    // V^T operand: 4 keys x 16 columns from each group of 16 lanes; a lane's 8 keys of the
    // product are the 8 it holds weights of, 4 half + {0..3} and 8 + 4 half + {0..3}
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
    // a step's weights are worked out under the products of the one before, V read four products ahead
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, 28, 0);
#pragma unroll
    for (int i = 0; i < KB * 2 * DB; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 28 / DB, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };

#pragma unroll
  for (int i = 0; i < PASS; ++i) {
    const uint32_t p = (uint32_t)ch.t0 * KT + (uint32_t)(lr + i * RPP);
    Place& x = pl[0][i];
    x.n = page_of(a.c.div, p, &x.off);
    x.id = pages[min(x.n, last)];
  }
  // the barriers for the compiler keep a tile's loads ahead of the products before it
  if constexpr (OWN) {
    load(ch.t0, 0, pl[0]);
    ids(pl[0], pl[0]);
    for (int t = ch.t0; t < ch.t1; ++t) {
      store(t, 0, 0);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      load(t + 1, 0, pl[0]);
      ids(pl[0], pl[0]);
      __builtin_amdgcn_sched_barrier(0);
      compute(t, 0);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  } else {  // the pages' numbers come before the rows: waiting for them leaves the rows in flight
    ids(pl[1], pl[0]);
    load(ch.t0, 0, pl[0]);
    ids(pl[0], pl[1]);
    load(ch.t0 + 1, 1, pl[1]);
    store(ch.t0, 0, 0);
    __syncthreads();
    // tile t of stage h; registers h are free, the others hold tile t + 1; place h is tile t + 2's
    auto step = [&](int t, int h) {
      ids(pl[h ^ 1], pl[h]);
      load(t + 2, h, pl[h]);
      __builtin_amdgcn_sched_barrier(0);
      if (wave_live) compute(t, h);
      __builtin_amdgcn_sched_barrier(0);
      store(t + 1, h ^ 1, h ^ 1);
      __syncthreads();
    };
    int t = ch.t0;
    for (; t + 1 < ch.t1; t += 2) {
      step(t, 0);
      step(t + 1, 1);
    }
    if (t < ch.t1) step(t, 0);
  }

  l = swap_add(l);
  // the infinities and NaN of the new nodes' values that row r sees, for its columns d..d+3
  auto odd4 = [&](int r, int d, f32x4* v) {
    if (!s_odd || d >= a.D) return;
    const int rn = r / a.G;
    const uint64_t w = a.tree != nullptr ? a.tree[(long long)b * a.N + rn] : (2ull << rn) - 1;
    for (int j = 0; j < a.N; ++j)
      if (((w >> j) & 1) && j >= tile_from_end<KT>(ch.t0, len) && j < tile_from_end<KT>(ch.t1, len)) {
        const T* x = reinterpret_cast<const T*>(a.vn) + nhead + (long long)j * a.kv_node + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = (float)x[i];
          if (!(fabsf(y) < __builtin_inff())) (*v)[i] += y;
        }
      }
  };
  // 4 columns d..d+3 of a query row: the output itself when the sequence is one chunk
  auto put = [&](int r, int d, f32x4 v, float mm, float ll) {
    if (d >= a.D) return;
    if constexpr (WK > 1) odd4(r, d, &v);
    if (ch.count == 1) {
      const float inv = ll > 0.f || ll != ll ? 1.0f / ll : 0.f;
      T* o4 = reinterpret_cast<T*>(a.out) + (long long)b * a.out_batch + (long long)(r / a.G) * a.out_node +
              (long long)(hk * a.G + r % a.G) * a.out_head + d;
      struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w.e[i] = mean_out<T>(ll == 0.f ? 0.f : v[i] * inv, v[i]);
      __builtin_memcpy(__builtin_assume_aligned(o4, 8), &w, 8);
    } else {
      const long long at = ((long long)slot * a.HK + hk) * a.R + r;
      *reinterpret_cast<f32x4*>(a.part + at * DP + d) = v;
      if (d == 0) {
        a.ml[2 * at] = mm;
        a.ml[2 * at + 1] = ll;
      }
    }
  };
  if constexpr (WK == 1) {
    if (!live) return;
    if (s_odd) {
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          f32x4 v = (f32x4){o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]};
          odd4(row, 32 * i + acc_row(r, half), &v);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][r + e] = v[e];
        }
    }
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        put(row, 32 * i + acc_row(r, half), (f32x4){o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]}, m, l);
  } else {
    // join the WK waves of the same rows through LDS
    constexpr int OP = DP + 4;
    float* ob = reinterpret_cast<float*>(smem);              // [WQ][WK][32][OP]
    float* mlb = ob + WQ * WK * 32 * OP;                     // [WQ][WK][32][2]
    __syncthreads();  // the tiles are free
    if (half == 0) {
      mlb[(wave * 32 + l32) * 2] = m;
      mlb[(wave * 32 + l32) * 2 + 1] = l;
    }
    __syncthreads();
    float mt = -__builtin_inff(), ltot = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) mt = fmaxf(mt, mlb[((wq * WK + w) * 32 + l32) * 2]);
    const float mb = mt == -__builtin_inff() ? 0.f : mt;
    const float f = __builtin_amdgcn_exp2f(m - mb);
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<f32x4*>(ob + (wave * 32 + l32) * OP + 32 * i + acc_row(r, half)) =
            (f32x4){o[i][r] * f, o[i][r + 1] * f, o[i][r + 2] * f, o[i][r + 3] * f};
    __syncthreads();
    constexpr int QP = DP / 4;  // quads of a row
    for (int i = wk * WAVE + lane; i < 32 * QP; i += WK * WAVE) {
      const int c = i / QP, d = 4 * (i % QP), r = (rt * WQ + wq) * 32 + c;
      if (r >= a.R) break;
      mt = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < WK; ++w) mt = fmaxf(mt, mlb[((wq * WK + w) * 32 + c) * 2]);
      const float mb2 = mt == -__builtin_inff() ? 0.f : mt;
      ltot = 0.f;
      f32x4 v = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        ltot += mlb[((wq * WK + w) * 32 + c) * 2 + 1] * __builtin_amdgcn_exp2f(mlb[((wq * WK + w) * 32 + c) * 2] - mb2);
        v += *reinterpret_cast<const f32x4*>(ob + ((wq * WK + w) * 32 + c) * OP + d);
      }
      put(r, d, v, mt, ltot);
    }
  }
}

// The plan of a call (pi_attn.hpp). Up to heads of
// 128 as few waves as the rows need. Above, a wave's query and output fill the registers, and only what
// eight waves share of a tile's loads leaves room for them: with one, two and four waves 348, 84 and 89
// registers were spilled, with eight 32, and eight are the fastest also where most of them have no rows.
// 8191 positions, 4 key heads of 256: 4 rows each 32 us (one wave: 67 to 77), 4 sequences of 48 rows 60
// (two: 270), 128 rows 42 (four: 67 to 71), 4 sequences of 104 rows 68 (four: 109).
AttnPlan attn_plan(int cus, int HK, int rows, int B, int DP) {
  AttnPlan p;
  p.wq = DP > 128 ? 8 : rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 ? 4 : 8;
  p.row_tiles = (rows + 32 * p.wq - 1) / (32 * p.wq);
  const int wgs = p.wq == 8 ? cus : 2 * cus;  // workgroups the chip holds at once
  p.slots = std::max(B, wgs / (HK * p.row_tiles));
  return p;
}
template <typename T, int DP, int WQ, int WK, int KB>
pi_status launch_attn_t(pi_ctx* c, const AttnDev& a) {
  constexpr size_t lds = attn_lds<DP, WQ, WK, KB>();
  auto kern = k_tree_attn<T, DP, WQ, WK, KB>;
  PI_HIP(c, allow_lds(kern, lds));
  PI_HIP(c, launch_kb(c, 0, kern, dim3((unsigned)(a.slots * a.HK * a.row_tiles)), 64 * WQ * WK, lds, a));
  if (a.slots > a.B) {
    const int rows = a.B * a.HK * a.R;
    PI_HIP(c, launch_k(c, 0, k_attn_join<T, DP, 32 * KB * WK>, dim3((rows + NWAVES - 1) / NWAVES), 0, a, rows));
  }
  return PI_OK;
}

template <typename T, int DP>
pi_status launch_attn_d(pi_ctx* c, const AttnDev& a, int wq) {
  if constexpr (DP > 128) {
    return launch_attn_t<T, DP, 8, 1, 1>(c, a);
  } else {
    switch (wq) {
      case 1: return launch_attn_t<T, DP, 1, 4, 1>(c, a);
      case 2: return launch_attn_t<T, DP, 2, 2, 1>(c, a);
      case 4: return launch_attn_t<T, DP, 4, 1, 2>(c, a);
      default: return launch_attn_t<T, DP, 8, 1, 2>(c, a);
    }
  }
}

template <typename T>
pi_status launch_attn(pi_ctx* c, const AttnDev& a, int wq) {
  switch (padded_dim(a.D)) {
    case 64: return launch_attn_d<T, 64>(c, a, wq);
    case 96: return launch_attn_d<T, 96>(c, a, wq);
    case 128: return launch_attn_d<T, 128>(c, a, wq);
    default: return launch_attn_d<T, 256>(c, a, wq);
  }
}

}  // namespace

extern "C" {

pi_status pi_attn_create(pi_ctx* ctx, const pi_kv* kv, int32_t heads, int32_t max_batch, int32_t max_nodes, float scale,
                         pi_attn** out) {
  if (ctx == nullptr || out == nullptr) return PI_ERR_INVALID;
  *out = nullptr;
  if (kv == nullptr) return fail(ctx, PI_ERR_INVALID, "kv is NULL");
  if (kv->ctx != ctx) return fail(ctx, PI_ERR_INVALID, "the cache belongs to another context");
  if (heads < 1 || heads % kv->desc.heads)
    return fail(ctx, PI_ERR_INVALID, "%d query heads are no multiple of the cache's %d", heads, kv->desc.heads);
  if (max_batch < 1 || max_nodes < 1) return fail(ctx, PI_ERR_INVALID, "bad limits: %d sequences, %d nodes", max_batch, max_nodes);
  if (max_nodes > 64) return fail(ctx, PI_ERR_UNSUPPORTED, "%d nodes: a tree has at most 64", max_nodes);
  // what the kernels use is its product with log2(e)
  if (!(scale > 0.f) || scale > 0x1p127f) return fail(ctx, PI_ERR_INVALID, "scale must be above 0 and at most 2^127");
  const int HK = kv->desc.heads, G = heads / HK;
  const int DP = kv->q4 ? padded_dim4(kv->desc.head_dim) : padded_dim(kv->desc.head_dim);
  if ((int64_t)max_batch * max_nodes * heads >= (1ll << 31) / 64)
    return fail(ctx, PI_ERR_UNSUPPORTED, "%d sequences of %d nodes and %d heads are too many", max_batch, max_nodes, heads);
  // scratch of the largest call: rows (all heads, all slots) of any number of nodes and sequences
  size_t rows = 0;
  for (int n = 1; n <= max_nodes; ++n) {
    // over a 4-bit cache a sequence's part may end and another begin in each slot
    const AttnPlan p = (kv->q4 ? attn4_plan : attn_plan)(ctx->cus, HK, n * G, max_batch, DP);
    rows = std::max(rows, (size_t)(p.slots + (kv->q4 ? max_batch : 0)) * HK * n * G);
  }
  PI_HIP(ctx, hipSetDevice(ctx->device));
  uint8_t* ws = nullptr;
  const size_t ob = rows * DP * 4, mb = rows * 2 * 4;
  if (hipMalloc(reinterpret_cast<void**>(&ws), ob + mb + (size_t)max_batch * 4) != hipSuccess) {
    (void)hipGetLastError();
    return fail(ctx, PI_ERR_OOM, "attention scratch of %zu bytes", ob + mb);
  }
  int32_t* self = reinterpret_cast<int32_t*>(ws + ob + mb);
  for (int i0 = 0; i0 < max_batch; i0 += 256) {
    int32_t id[256];
    for (int i = 0; i < 256; ++i) id[i] = i0 + i;
    if (hipMemcpy(self + i0, id, (size_t)std::min(256, max_batch - i0) * 4, hipMemcpyHostToDevice) != hipSuccess) {
      (void)hipFree(ws);
      return fail(ctx, PI_ERR_HIP, "filling the attention scratch failed");
    }
  }
  pi_attn* a = new (std::nothrow) pi_attn{ctx, *kv, heads, max_batch, max_nodes, scale, ws, reinterpret_cast<float*>(ws),
                                          reinterpret_cast<float*>(ws + ob), self};
  if (a == nullptr) {
    (void)hipFree(ws);
    return fail(ctx, PI_ERR_OOM, "host allocation failed");
  }
  ctx_retain(ctx);
  *out = a;
  return PI_OK;
}

void pi_attn_destroy(pi_attn* attn) {
  if (attn == nullptr) return;
  (void)hipSetDevice(attn->ctx->device);
  (void)hipFree(attn->ws);
  ctx_release(attn->ctx);
  delete attn;
}

pi_status pi_tree_attention(pi_ctx* ctx, pi_attn* attn, const pi_attn_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (attn == nullptr) return fail(ctx, PI_ERR_INVALID, "attn is NULL");
  if (attn->ctx != ctx) return fail(ctx, PI_ERR_INVALID, "attn belongs to another context");
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_attn_args& a = *args;
  const pi_kv* kv = &attn->kv;
  PI_TRY(check_paging(ctx, kv, a.table, a.table_stride, a.table_width, a.ctx_len, a.B, a.N));
  if (a.B > attn->max_batch || a.N > attn->max_nodes)
    return fail(ctx, PI_ERR_INVALID, "B %d, N %d above the handle's %d, %d", a.B, a.N, attn->max_batch, attn->max_nodes);
  PI_TRY(check_bnh(ctx, "q", a.q, a.q_batch, a.q_node, a.q_head));
  PI_TRY(check_bnh(ctx, "k_new", a.k_new, a.kv_batch, a.kv_node, a.kv_head));
  PI_TRY(check_bnh(ctx, "v_new", a.v_new, a.kv_batch, a.kv_node, a.kv_head));
  PI_TRY(check_bnh(ctx, "out", a.out, a.out_batch, a.out_node, a.out_head));
  if (reinterpret_cast<uintptr_t>(a.tree) & 7u) return fail(ctx, PI_ERR_INVALID, "tree is not 8-byte aligned");
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const int HK = kv->desc.heads, G = attn->heads / HK;
  const int D = kv->desc.head_dim;
  KvDev c = kv_dev(kv, a.table, a.table_stride, a.table_width);
  const AttnPlan p = kv->q4 ? attn4_plan(ctx->cus, HK, a.N * G, a.B, padded_dim4(D)) : attn_plan(ctx->cus, HK, a.N * G, a.B, padded_dim(D));
  if (a.table == nullptr) {
    c.table = attn->self;
    c.table_stride = 1;
  }
  const AttnDev d{c, static_cast<const uint8_t*>(a.q),
                  static_cast<const uint8_t*>(a.k_new), static_cast<const uint8_t*>(a.v_new),
                  static_cast<uint8_t*>(a.out), a.tree, a.ctx_len, attn->part, attn->ml, a.q_batch, a.q_node, a.q_head,
                  a.kv_batch, a.kv_node, a.kv_head, a.out_batch, a.out_node, a.out_head, a.B, a.N, attn->heads, HK, G,
                  kv->desc.head_dim, a.N * G, p.slots, p.row_tiles, attn->scale * 1.4426950408889634f};
  if (kv->q4) return launch_attn4(ctx, d, kv4_dev(kv), p.wq, kv->desc.dtype == PI_T_F16);
  return kv->desc.dtype == PI_T_F16 ? launch_attn<half_t>(ctx, d, p.wq) : launch_attn<bf16_t>(ctx, d, p.wq);
}

}  // extern "C"
