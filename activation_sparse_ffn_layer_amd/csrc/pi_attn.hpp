// What the attention kernels share: matrix core products by type, the cutting of key axes into chunks,
// the join of partial results.
#pragma once
#include "pi_kv.hpp"

struct pi_attn {
  pi_ctx* ctx;
  pi_kv kv;         // a copy: the cache's handle may be destroyed before this one
  int heads, max_batch, max_nodes;
  float scale;
  uint8_t* ws;
  float* part;      // [slots][kv heads][rows][DP]
  float* ml;        // [slots][kv heads][rows][2]: maximum (log2 domain) and sum
  int32_t* self;    // 0, 1, ..: the page table of calls without one
};

namespace pi {

struct AttnDev {
  KvDev c;
  const uint8_t *q, *kn, *vn;
  uint8_t* out;
  const uint64_t* tree;
  const int32_t* ctx_len;
  float *part, *ml;
  long long q_batch, q_node, q_head, kv_batch, kv_node, kv_head, out_batch, out_node, out_head;
  int B, N, H, HK, G, D, R;  // R = N * G query rows of a key/value head
  int slots, row_tiles;
  float scale2;  // scale * log2(e)
};

namespace {

template <typename T> struct Mm;
template <> struct Mm<half_t> {
  typedef half8_t v8;
  // weights are carried times 2^14 (at most 16384), so that fp16 keeps its 11 bits down to 2^-28
  // of the largest; below, a long cache's many small weights would round away together
  static constexpr float SHIFT = 14.f;
  static constexpr uint32_t EXP = 0x7C00u;
  static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mm<bf16_t> {
  typedef bf8_t v8;
  static constexpr float SHIFT = 0.f;
  static constexpr uint32_t EXP = 0x7F80u;
  static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// The mean `x` of values whose weighted sum is `sum`. Values that are numbers have no larger mean, but their weights' rounding
// may bring it past the type's largest number, where the conversion gives an infinity.
template <typename T>
__device__ __forceinline__ T mean_out(float x, float sum) {
  constexpr float TOP = __is_same(T, half_t) ? 65504.f : 0x1.FEp127f;
  if (fabsf(sum) < __builtin_inff()) x = x > TOP ? TOP : x < -TOP ? -TOP : x;
  return (T)x;
}

__device__ __forceinline__ int acc_row(int r, int half) { return 8 * (r >> 2) + 4 * half + (r & 3); }

// The other half's value of v (lane ^ 32).
__device__ __forceinline__ float swap_max(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return fmaxf(u2f(p[0]), u2f(p[1]));
}
__device__ __forceinline__ float swap_add(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return u2f(p[0]) + u2f(p[1]);
}

// Tiles of KT keys that a sequence's positions and nodes take. Positions go up to 2^31 - 65 and a tile
// or its successors may end beyond 2^31: sums of them are unsigned, and the kernels go by a tile's
// place relative to the sequence's end, which is small where it matters.
template <int KT>
__device__ __forceinline__ int key_tiles(const AttnDev& a, int b) {
  return (int)(((uint32_t)kv_len(a.c, a.ctx_len, b) + (uint32_t)(a.N + KT - 1)) / (uint32_t)KT);
}
template <int KT>
__device__ __forceinline__ int tile_from_end(int tile, int len) {
  return (int)((uint32_t)tile * (uint32_t)KT - (uint32_t)len);
}
// A sum over all sequences of what each lane adds up: a lane's stops at 2^25, above any number of slots
// that it is compared with, so that 64 of them stay below 2^32.
__device__ __forceinline__ uint32_t lane_tiles(uint32_t n, uint32_t more) { return min(n + more, 1u << 25); }
__device__ __forceinline__ uint32_t sum_tiles(uint32_t n) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) n += __shfl_xor(n, s, WAVE);
  return n;
}

// Where chunk `slot` lies: sequence b, its tiles [t0, t1), its number of chunks and the first
// one's slot; false past the last chunk. Chunks are `c` tiles long, the least c that needs no
// more than `slots` of them in all (slots >= B). Every wave works it out for itself.
struct Chunk {
  int b, t0, t1, count, first;
};
template <int KT>
__device__ __forceinline__ bool find_chunk(const AttnDev& a, int slot, Chunk* o) {
  const int lane = threadIdx.x % WAVE;
  auto tiles = [&](int b) { return b < a.B ? key_tiles<KT>(a, b) : 0; };
  if (a.B == 1) {
    const int t = tiles(0), c = (t + a.slots - 1) / a.slots;
    *o = Chunk{0, slot * c, min(t, slot * c + c), (t + c - 1) / c, 0};
    return o->t0 < t;
  }
  const int mine = tiles(lane);  // the sequence of this lane; more than 64 are read again
  auto sum = [&](int c) {
    uint32_t n = lane_tiles(lane < a.B ? (mine + c - 1) / c : 0, 0);
    for (int b = lane + WAVE; b < a.B; b += WAVE) n = lane_tiles(n, (tiles(b) + c - 1) / c);
    return sum_tiles(n);
  };
  const uint32_t slots = (uint32_t)a.slots;
  int c = max(1, (int)((sum(1) + slots - 1) / slots));
  while (c > 1 && sum(c) > slots) c += max(1, c >> 5);
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += WAVE) {
    const int tl = b0 == 0 ? mine : tiles(b0 + lane);
    const int n = (tl + c - 1) / c;
    int incl = n;
#pragma unroll
    for (int s = 1; s < WAVE; s <<= 1) {
      const int t = __shfl_up(incl, s, WAVE);
      if (lane >= s) incl += t;
    }
    const uint64_t hit = __ballot(before + incl > slot);
    if (hit != 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int first = before + __shfl(incl - n, l, WAVE);
      const int tb = __shfl(tl, l, WAVE);
      o->b = b0 + l;
      o->first = first;
      o->count = __shfl(n, l, WAVE);
      o->t0 = (slot - first) * c;
      o->t1 = min(tb, o->t0 + c);
      return true;
    }
    before += __shfl(incl, WAVE - 1, WAVE);
  }
  return false;
}

__device__ u32x4 attn_zero[8];  // zeros, never written

// LDS of a workgroup: keys, then values, of one tile (two where tiles are shared by waves). A
// row's pitch spreads what is read at once over the 64 banks: 16 rows of 16 bytes of K, and of V,
// by its transposing reads, 4 rows of 64 bytes.
template <int DP> constexpr int k_pitch() { return DP * 2 + 16; }
template <int DP> constexpr int v_pitch() { return DP * 2 % 128 == 0 ? DP * 2 + 64 : DP * 2; }
// out = sum_s O_s 2^(m_s - m) / sum_s l_s 2^(m_s - m) over the `count` partial results of row r from slot `first` on, by
// one wave, 4 columns per lane.
template <typename T, int DP>
__device__ __forceinline__ void join_parts(const AttnDev& a, int b, int hk, int r, int first, int count) {
  const int lane = threadIdx.x % WAVE;
  const long long at0 = ((long long)first * a.HK + hk) * a.R + r, next = (long long)a.HK * a.R;
  float m = -__builtin_inff();
  for (int s = lane; s < count; s += WAVE) m = fmaxf(m, a.ml[2 * (at0 + s * next)]);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, WAVE));
  const float base = m == -__builtin_inff() ? 0.f : m;
  // Up to 128 columns the wave's halves take every other chunk.
  constexpr int HALVES = DP <= 128 ? 2 : 1;
  const int mine = HALVES == 2 ? lane >> 5 : 0, d = 4 * (HALVES == 2 ? lane & 31 : lane);
  const float* part = a.part + at0 * DP + min(d, DP - 4);
  f32x4 v = (f32x4){0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  for (int s0 = 0; s0 < count; s0 += WAVE) {
    // a lane's chunk of these 64: its factor and its part of the sum
    const bool in = s0 + lane < count;
    const long long at = at0 + (in ? s0 + lane : 0) * next;
    // not 0 for a chunk of this sequence: an infinity that its row sees stays one, whatever it weighs
    const float f = in ? fmaxf(__builtin_amdgcn_exp2f(a.ml[2 * at] - base), 1.4e-45f) : 0.f;
    l += in ? a.ml[2 * at + 1] * f : 0.f;
    const int n = min(WAVE, count - s0);
    for (int s = 0; s < n; s += 8) {
      constexpr int U = 8 / HALVES;
      f32x4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = *reinterpret_cast<const f32x4*>(part + (s0 + min(s + HALVES * u + mine, n - 1)) * next * DP);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = s + HALVES * u + mine;
        // the halves ask different lanes: what is shuffled must not depend on the asking lane's c
        const float g = __shfl(f, min(c, n - 1), WAVE);
        // past the last chunk its part is read again: left out by selection, as 0 times an infinity is none
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += c < n ? x[u][i] * g : 0.f;
      }
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) l += __shfl_xor(l, s, WAVE);
  if constexpr (HALVES == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = swap_add(v[i]);
  }
  if (HALVES == 2 && lane >= 32) return;
  if (d >= a.D) return;
  T* o = reinterpret_cast<T*>(a.out) + (long long)b * a.out_batch + (long long)(r / a.G) * a.out_node +
         (long long)(hk * a.G + r % a.G) * a.out_head + d;
  struct __attribute__((aligned(8))) { T e[4]; } w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w.e[i] = mean_out<T>(l == 0.f ? 0.f : v[i] / l, v[i]);
  __builtin_memcpy(__builtin_assume_aligned(o, 8), &w, 8);
}

constexpr int padded_dim(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256; }

// Bound by memory, the partial results' bytes (27 MB at 6656 rows in some 13 chunks: 10 us).
// Over a sequence's chunks, one wave per query row; rows of sequences of one chunk are done already.
template <typename T, int DP, int KT>
__global__ __launch_bounds__(BLOCK) void k_attn_join(AttnDev a, int rows) {
  const int lane = threadIdx.x % WAVE;
  // (b, hk, r) of this wave
  const int id = blockIdx.x * NWAVES + threadIdx.x / WAVE;
  if (id >= rows) return;
  const int r = id % a.R, hk = id / a.R % a.HK, b = id / a.R / a.HK;
  // the first slot of sequence b: the chunks before it
  auto tiles = [&](int i) { return i < a.B ? key_tiles<KT>(a, i) : 0; };
  auto sum = [&](int c, int end) {
    uint32_t n = 0;
    for (int i = lane; i < end; i += WAVE) n = lane_tiles(n, (tiles(i) + c - 1) / c);
    return sum_tiles(n);
  };
  const uint32_t slots = (uint32_t)a.slots;
  int c = max(1, (int)((sum(1, a.B) + slots - 1) / slots));
  while (c > 1 && sum(c, a.B) > slots) c += max(1, c >> 5);
  const int first = (int)sum(c, b), count = (tiles(b) + c - 1) / c;
  if (count == 1) return;
  join_parts<T, DP>(a, b, hk, r, first, count);
}

}  // namespace

// How a call is cut: waves along the rows, row tiles and slots (chunks of all sequences;
// over a 4-bit cache spans of all sequences' tiles).
struct AttnPlan {
  int wq, row_tiles, slots;
};
AttnPlan attn4_plan(int cus, int HK, int rows, int B, int DP);
pi_status launch_attn4(pi_ctx* c, const AttnDev& a, const Kv4Dev& scales, int wq, bool f16);
constexpr int padded_dim4(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

}  // namespace pi
