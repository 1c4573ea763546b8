// Check of drafted tokens by rejection sampling (pi_verify).
//
// Which child of a node is taken depends on p(t) = exp((z_t - max) / T) / Z of its parent's row (Z:
// the row's sum), on the draft's q(t) and, after rejections, on c and the weight S that is left:
// after j of them the residual is max(p - c q, 0) / S with c_{j+1} = c_j + S_j,
// S_{j+1} = sum_t max(p - c_{j+1} q, 0). So no residual is ever stored: every pass recomputes it.
//
// The draws compare running sums over the vocabulary, whose steps are as small as 1e-6 of the
// whole, so a row that is drawn from, or whose residual is weighed, has its exponentials and
// sums in 64 bits (a 32-bit exponential alone would move one draw in some hundred). Most rows of
// a tree are only walked past: for them Z in 32 bits, off by less than 1e-5, decides, and a child
// whose test is nearer than that waits for its row's Z in 64 bits.
//
//   k_verify_rows   every row's maximum and 32-bit sum, in chunks of the vocabulary: the one pass
//                   over all logits, bound by memory. 512 rows of 131072 fp16 logits, 134 MB:
//                   29 us, 4.6 TB/s (72 us with all exponentials in 64 bits)
//   k_verify_pass   walks the tree as far as it can, then sums in 64 bits, in the same chunks, what
//                   the walk waits for: over the current row the exponentials (E), those of
//                   the tokens with p > c q (A) and these tokens' q (Q). Then Z = E and
//                   S = A / Z - c Q, exact to second order in the error of the 32-bit Z that
//                   chose the tokens. Every workgroup walks for itself, all alike, so that
//                   none waits for another. Launched a fixed number of times (they return at
//                   once where the sequence is done).
//   k_verify_end    a workgroup per sequence does whatever is left and draws the next token: the
//                   chunk by the chunks' weights, then the token inside it.
// The passes and the end are chains of dependent loads, sums over a workgroup and the walk: 14, 7
// and 12 us at 16 trees of 32 nodes, 8, 3 and 8 at one chain of 5.
#include <algorithm>
#include <new>

#include "pi_host.hpp"
#include "pi_types.hpp"

using namespace pi;

namespace {

constexpr int VF_CH = 4096;        // tokens per chunk
constexpr int VF_MAX_NODES = 256;
constexpr int VF_NT = 512;         // threads of a workgroup that walks: 8 tokens of a chunk each
constexpr double VF_NEAR = 2e-5;   // a test with a 32-bit Z decides beyond this distance, relative to p

struct VfPart {   // a chunk of a row, in 32 bits
  float m, s;     // maximum, sum of exp((z - m) / T)
  int32_t at;     // the maximum's lowest index (greedy rows only)
  int32_t pad;
};
struct VfRow {    // a row; for a node also its own token's exp((z - m) / T) and q under its parent
  double s, et;
  float m, qt;
  int32_t at, pad;
};
struct VfBin {    // a chunk of the current row, in 64 bits
  double e, a, q;
};
enum { WAIT_REST = 0, WAIT_DRAW = 1, DONE = 2, DONE_PLAIN = 5 };
struct VfState {
  double c, left, z;  // z: the current row's sum in 64 bits, 0 before it is known
  int32_t cur, next, depth;
  int32_t stage;      // WAIT_*: for a pass; DONE + i: ended, the weights to draw from in bins i
};

}  // namespace

struct pi_verifier {
  pi_ctx* ctx;
  int vocab, max_batch, max_nodes, chunks;
  uint8_t* ws;
  VfPart* part;     // [B][N][chunks]
  VfRow* rows;      // [B][N]
  VfState* state;   // [2][B], by the parity of the pass
  VfBin* bins;      // [3][B][chunks]: two passes' by parity; the last kernel's own
};

namespace {

struct VfDev {
  const void* logits;
  const float* q;
  long long lb, ln, qb, qn;
  const int32_t *tokens, *parents;
  const float *u, *u_next, *temp;
  int32_t *nodes, *out, *n;
  int B, N, V, chunks;
  VfPart* part;
  VfRow* rows;
  VfState* state;
  VfBin* bins;
};

// NaN to -inf, +inf to the largest finite value
__device__ __forceinline__ float clean(float z) { return fminf(fmaxf(z, -__builtin_inff()), 3.4028234663852886e38f); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(half_t v) { return (float)v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return (float)v; }

// 8 logits from index i of a row (rows start at any element), -inf past its end
template <typename T>
__device__ __forceinline__ void logits8(const T* row, int i, int V, float (&o)[8]) {
  if (i + 8 <= V) {
    T v[8];
    __builtin_memcpy(v, row + i, sizeof v);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = clean(to_f32(v[j]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = i + j < V ? clean(to_f32(row[min(i + j, V - 1)])) : -__builtin_inff();
  }
}

// 2^t for t <= 0, and 2^-1000 for all below that: 2^f of the fraction (|f| <= 1/2) by the polynomial
// of degree 9 through the Chebyshev points of that interval, off by at most 3e-14.
__device__ __forceinline__ double pow2_floor(double t) {
  const double magic = 6755399441055744.0;  // 1.5 * 2^52: the sum's low bits are t's nearest whole number
  const double c = fmax(t, -1000.0);
  const double k = c + magic;
  const double f = c - (k - magic);
  double r = 1.0205905413765595e-07;
  r = fma(r, f, 1.325964524488711e-06);
  r = fma(r, f, 1.5252672924850737e-05);
  r = fma(r, f, 0.0001540343375125101);
  r = fma(r, f, 0.0013333558200794592);
  r = fma(r, f, 0.009618129193934313);
  r = fma(r, f, 0.05550410866465167);
  r = fma(r, f, 0.2402265069564034);
  r = fma(r, f, 0.6931471805599462);
  r = fma(r, f, 1.0);
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, r) + (__builtin_bit_cast(uint64_t, k) << 52));
}
__device__ __forceinline__ double pow2(double t) {
  const double r = pow2_floor(t);
  return t > -1000.0 ? r : 0.0;
}
// exp((z - m) / T), given it = log2(e) / T; z <= m, m finite
__device__ __forceinline__ double expw(float z, float m, double it) { return pow2(((double)z - (double)m) * it); }

// v of the lane that a data-parallel move brings it from, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Inclusive running sum over the wave's lanes: within rows of 16 by shifts of 1, 2, 4 and 8, then the
// sums of the rows before (row_bcast 15 and 31). A quarter of the latency of lane permutes.
__device__ __forceinline__ double wave_scan_d(double v) {
  v += moved<0x111, 0xF>(v);
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);
  v += moved<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ double wave_sum_d(double v) {  // the same on every lane
  const uint64_t b = __builtin_bit_cast(uint64_t, wave_scan_d(v));
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, WAVE - 1), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), WAVE - 1);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The same for floats: sum and maximum over the wave, the same on every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v, float none) {
  return u2f(__builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
}
template <typename F>
__device__ __forceinline__ float wave_fold(float v, float none, F f) {
  v = f(v, moved<0x111, 0xF>(v, none));
  v = f(v, moved<0x112, 0xF>(v, none));
  v = f(v, moved<0x114, 0xF>(v, none));
  v = f(v, moved<0x118, 0xF>(v, none));
  v = f(v, moved<0x142, 0xA>(v, none));
  v = f(v, moved<0x143, 0xC>(v, none));
  return u2f((uint32_t)__builtin_amdgcn_readlane(__builtin_bit_cast(int, v), WAVE - 1));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_fold(v, -__builtin_inff(), [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_fold(v, 0.f, [](float a, float b) { return a + b; });
}

// Sums over the workgroup's NT threads, the same on every thread; red: 3 NT / WAVE doubles.
template <int NT>
__device__ __forceinline__ VfBin block_sum(VfBin v, VfBin* red) {
  v = VfBin{wave_sum_d(v.e), wave_sum_d(v.a), wave_sum_d(v.q)};
  __syncthreads();
  if (threadIdx.x % WAVE == 0) red[threadIdx.x / WAVE] = v;
  __syncthreads();
  VfBin s{0.0, 0.0, 0.0};
#pragma unroll
  for (int i = 0; i < NT / WAVE; ++i) s = VfBin{s.e + red[i].e, s.a + red[i].a, s.q + red[i].q};
  return s;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const VfDev& p, int b, int i) {
  return static_cast<const T*>(p.logits) + (long long)b * p.lb + (long long)i * p.ln;
}
// log2(e) / T; 0: greedy. An infinite temperature's is a number that no logit's distance makes visible
// but that leaves -inf at -inf.
__device__ __forceinline__ double inv_temp(const VfDev& p, int b) {
  const float t = p.temp == nullptr ? 1.f : p.temp[b];
  return t == __builtin_inff() ? 1e-300 : t > 0.f ? 1.4426950408889634 / (double)t : 0.0;
}
__device__ __forceinline__ VfBin* bins_of(const VfDev& p, int which, int b) {
  return p.bins + ((long long)which * p.B + b) * p.chunks;
}

struct VfShared {
  double et[VF_MAX_NODES], rs[VF_MAX_NODES];
  float m[VF_MAX_NODES], u[VF_MAX_NODES], qt[VF_MAX_NODES];
  int32_t at[VF_MAX_NODES], par[VF_MAX_NODES], tok[VF_MAX_NODES];
  VfState st;
  VfBin red[VF_NT / WAVE];
  double target, before;
  int32_t pick, last;
  int32_t again;      // the residual's weight is needed once more, now that Z is known in 64 bits
};

// 8 tokens of the current row from i on: exp((z - m) / T), the draft's q (0 without one), and a bit
// for each token that the draw may give: without a q, not the children's.
template <typename T>
__device__ __forceinline__ uint32_t row8(const VfDev& p, const VfShared& s, int b, double it, int i, double (&e)[8],
                                         float (&q)[8]) {
  const int cur = s.st.cur;
  float z[8];
  logits8(row_of<T>(p, b, cur), i, p.V, z);
  if (p.q != nullptr) {
    const float* qr = p.q + (long long)b * p.qb + (long long)cur * p.qn;
    if (i + 8 <= p.V) {
      __builtin_memcpy(q, qr + i, sizeof q);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = i + j < p.V ? qr[i + j] : 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = 0.f;
  }
  const float m = s.m[cur];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = expw(z[j], m, it);
  uint32_t may = 0xFF;
  if (p.q == nullptr)
    for (int k = cur + 1; k < p.N; ++k) {
      const int t = s.tok[k] - i;
      if (s.par[k] == cur && t >= 0 && t < 8) may &= ~(1u << t);
    }
  return may;
}

// 8 tokens' part of a chunk's sums.
template <typename T>
__device__ __forceinline__ void bin8(const VfDev& p, const VfShared& s, int b, double it, int i, VfBin* v) {
  if (i >= p.V) return;
  double e[8];
  float q[8];
  const uint32_t may = row8<T>(p, s, b, it, i, e, q);
  const double iz = 1.0 / (s.st.z > 0.0 ? s.st.z : s.rs[s.st.cur]), c = s.st.c;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = ((may >> j) & 1) && e[j] * iz > c * (double)q[j];
    v->e += e[j];
    v->a += in ? e[j] : 0.0;
    v->q += in ? (double)q[j] : 0.0;
  }
}

// A chunk's sums by the workgroup's NT threads, the same on every thread.
template <typename T, int NT>
__device__ __forceinline__ VfBin bin_block(const VfDev& p, VfShared& s, int b, double it, int chunk) {
  VfBin v{0.0, 0.0, 0.0};
#pragma unroll
  for (int g = 0; g < VF_CH / 8; g += NT)
    if (NT <= VF_CH / 8 || threadIdx.x < VF_CH / 8) bin8<T>(p, s, b, it, chunk * VF_CH + (g + (int)threadIdx.x) * 8, &v);
  return block_sum<NT>(v, s.red);
}

// The same by one wave.
template <typename T>
__device__ __forceinline__ VfBin bin_wave(const VfDev& p, const VfShared& s, int b, double it, int chunk) {
  VfBin v{0.0, 0.0, 0.0};
#pragma unroll 2
  for (int g = 0; g < VF_CH / 8; g += WAVE) bin8<T>(p, s, b, it, chunk * VF_CH + (g + (int)threadIdx.x % WAVE) * 8, &v);
  return VfBin{wave_sum_d(v.e), wave_sum_d(v.a), wave_sum_d(v.q)};
}

// This thread's first chunk of a pass's sums.
__device__ __forceinline__ VfBin first_bin(const VfDev& p, const VfBin* bins) {
  return (int)threadIdx.x < p.chunks ? bins[threadIdx.x] : VfBin{0.0, 0.0, 0.0};
}

// The sums of the pass that the walk waited for: Z and the residual's weight. `v`: first_bin. The tokens
// of the residual were chosen by the 32-bit Z. The error of that Z, relative to Z, bounds what wrongly
// chosen tokens weigh: nothing beside the residual, but where the draft is the target to within a few
// roundings. A residual below 2^20 times the error is summed again, by the 64-bit Z.
template <int NT>
__device__ __forceinline__ void join_bins(const VfDev& p, VfShared& s, const VfBin* bins, VfBin v) {
  for (int k = threadIdx.x + NT; k < p.chunks; k += NT) v = VfBin{v.e + bins[k].e, v.a + bins[k].a, v.q + bins[k].q};
  v = block_sum<NT>(v, s.red);
  if (threadIdx.x == 0) {
    const double left = s.st.c > 0.0 ? fmax(v.a / v.e - s.st.c * v.q, 0.0) : 1.0;
    s.again = s.st.z == 0.0 && s.st.c > 0.0 && left * v.e < 0x1p20 * fabs(s.rs[s.st.cur] - v.e);
    s.st.z = v.e;
    s.st.left = left;
  }
  __syncthreads();
}

// Draw the next token at node s.st.cur and write the sequence's outputs. All VF_NT threads.
template <typename T>
__device__ __forceinline__ void finish(const VfDev& p, VfShared& s, int b, double it) {
  constexpr int NT = VF_NT;
  const int cur = s.st.cur, lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  const int depth = s.st.depth;  // nodes of the path; its nodes are written already
  static_assert(VF_MAX_NODES <= NT, "a thread per node");
  const int i1 = threadIdx.x + 1, node1 = i1 < depth ? p.nodes[(long long)b * p.N + i1] : -1;
  int next = -1;
  if (s.st.stage == DONE_PLAIN) {
    if (it == 0.0) next = s.at[cur];
  } else {
    const VfBin* bins = bins_of(p, s.st.stage - DONE, b);
    const float un = p.u_next[b];
    VfBin sum{0.0, 0.0, 0.0};  // of this thread's chunks, the first of which stays in registers
    if ((int)threadIdx.x < p.chunks) sum = bins[threadIdx.x];
    const VfBin own = sum;
    for (int k = threadIdx.x + NT; k < p.chunks; k += NT) sum = VfBin{sum.e + bins[k].e, sum.a + bins[k].a, sum.q + bins[k].q};
    sum = block_sum<NT>(sum, s.red);
    // the chunks' weights: of what is left, or of p where nothing is
    const double iz = 1.0 / sum.e, c = p.q != nullptr ? s.st.c : 0.0;
    const bool left = sum.a * iz - c * sum.q > 0.0;
    auto weight = [&](int k) {
      const VfBin v = k == (int)threadIdx.x ? own : bins[k];
      return left ? fmax(v.a * iz - c * v.q, 0.0) : v.e * iz;
    };
    if (threadIdx.x == 0) {
      s.before = 0.0;
      s.pick = 0x7FFFFFFF;
      s.last = -1;
    }
    // inclusive sum over the workgroup of one value per thread, from `carry` on
    auto scan = [&](double v, double* carry) {
      const double incl = wave_scan_d(v);
      __syncthreads();
      if (lane == WAVE - 1) s.red[wave].e = incl;
      __syncthreads();
      double run = *carry;
      for (int i = 0; i < NT / WAVE; ++i) {
        if (i < wave) run += s.red[i].e;
        *carry += s.red[i].e;
      }
      return run + incl;
    };
    // the chunk whose running sum passes the target, or the last one with any weight
    const double v0 = (int)threadIdx.x < p.chunks ? weight(threadIdx.x) : 0.0;
    double total = 0.0;
    const double run0 = scan(v0, &total);
    for (int k0 = NT; k0 < p.chunks; k0 += NT) {
      const int k = k0 + (int)threadIdx.x;
      scan(k < p.chunks ? weight(k) : 0.0, &total);
    }
    const double target = (double)un * total;
    double carry = 0.0;
    for (int k0 = 0; k0 < p.chunks; k0 += NT) {
      const int k = k0 + (int)threadIdx.x;
      const double v = k0 == 0 ? v0 : k < p.chunks ? weight(k) : 0.0;
      const double run = k0 == 0 && p.chunks <= NT ? run0 : scan(v, &carry);
      if (v > 0.0 && run > target) atomicMin(&s.pick, k);
      if (v > 0.0) atomicMax(&s.last, k);
      __syncthreads();
      const int pick = s.pick;
      if (k == pick) s.before = run - v;
      if (pick != 0x7FFFFFFF) break;
    }
    __syncthreads();
    const int chunk = s.pick != 0x7FFFFFFF ? s.pick : s.last;
    const double rest = target - s.before;
    __syncthreads();
    if (threadIdx.x == 0) {
      s.pick = 0x7FFFFFFF;
      s.last = -1;
    }
    if (chunk >= 0) {  // the token: 8 per thread in order, threads in order
      double w[8], all = 0.0;
      int lastw = -1;
      const int i = chunk * VF_CH + (int)threadIdx.x * 8;
      const bool in = threadIdx.x < VF_CH / 8 && i < p.V;
      if (in) {
        double e[8];
        float q[8];
        const uint32_t may = row8<T>(p, s, b, it, i, e, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = !left ? e[j] * iz : (may >> j) & 1 ? fmax(e[j] * iz - c * (double)q[j], 0.0) : 0.0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!in) w[j] = 0.0;
        all += w[j];
        if (w[j] > 0.0) lastw = i + j;
      }
      double none = 0.0;
      double run = scan(all, &none) - all;
      int mine = 0x7FFFFFFF;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        run += w[j];
        if (w[j] > 0.0 && run > rest) mine = min(mine, i + j);
      }
      if (mine != 0x7FFFFFFF) atomicMin(&s.pick, mine);
      if (lastw >= 0) atomicMax(&s.last, lastw);
      __syncthreads();
      next = s.pick != 0x7FFFFFFF ? s.pick : s.last;
    }
  }
  const int k = threadIdx.x;
  if (k < p.N) {
    p.out[(long long)b * p.N + k] = node1 >= 0 ? s.tok[node1] : k + 1 == depth ? next : -1;
    if (k >= depth) p.nodes[(long long)b * p.N + k] = -1;
  }
  if (threadIdx.x == 0) p.n[b] = depth;
}

// Walk on from s.st until a pass is needed or no child is left to try. All threads; the first wave
// walks, all its lanes on the same values. `src`: the bins of the pass just joined, if any;
// `write`: the path goes to memory.
__device__ __forceinline__ void walk(const VfDev& p, VfShared& s, int b, double it, int src, bool write) {
  __syncthreads();
  if (threadIdx.x < WAVE) {
    const int lane = threadIdx.x;
    int cur = s.st.cur, next = s.st.next, depth = s.st.depth;
    double c = s.st.c, left = s.st.left, z = s.st.z;
    bool end = true;
    for (int g = next / WAVE; g * WAVE < p.N;) {
      const int i0 = g * WAVE + lane;
      uint64_t kids = __ballot(i0 < p.N && i0 >= next && s.par[i0] == cur);
      if (kids == 0) {
        ++g;
        continue;
      }
      const int i = g * WAVE + __ffsll((unsigned long long)kids) - 1;
      const double sum = z > 0.0 ? z : s.rs[cur], u = (double)s.u[i], qt = (double)s.qt[i];
      const double pt = it == 0.0 ? (s.tok[i] == s.at[cur] ? 1.0 : 0.0) : sum > 0.0 ? s.et[i] / sum : 0.0;
      bool again = false;  // without a q: an earlier child's token
      if (p.q == nullptr)
        for (int k0 = 0; k0 < i; k0 += WAVE) {
          const int k = k0 + lane;
          again = again || __any(k < i && s.par[k] == cur && s.tok[k] == s.tok[i]);
        }
      const double lhs = p.q != nullptr ? u * left * qt : u * left, rhs = p.q != nullptr ? fmax(pt - c * qt, 0.0) : pt;
      if (it != 0.0 && z == 0.0 && pt > 0.0 && !again && fabs(lhs - rhs) <= VF_NEAR * (pt + (p.q != nullptr ? 0.0 : u))) {
        next = cur + 1;  // the row again, with its sum in 64 bits
        c = 0.0;
        left = 1.0;
        end = false;
        break;
      }
      next = i + 1;
      // without a q no probability is above 1, whatever the roundings of what is left of it
      const bool take = !again && lhs < rhs && (p.q != nullptr || u < 1.0);
      if (take) {
        cur = i;
        c = 0.0;
        left = 1.0;
        z = 0.0;
        if (write && lane == 0) p.nodes[(long long)b * p.N + depth] = i;
        ++depth;
      } else if (p.q != nullptr) {
        c += left;
        if (it == 0.0) {  // all weight at one token
          const int a = s.at[cur];
          left = a >= 0 ? fmax(1.0 - c * (double)p.q[(long long)b * p.qb + (long long)cur * p.qn + a], 0.0) : 0.0;
        } else if (left > 0.0 && sum > 0.0) {
          end = false;
          break;
        }
      } else if (!again) {
        left = fmax(left - pt, 0.0);
      }
      g = next / WAVE;
    }
    int stage = WAIT_REST;
    if (end) {
      if (it == 0.0 || s.rs[cur] == 0.0) stage = DONE_PLAIN;
      else if (p.q != nullptr && c > 0.0) stage = DONE + src;
      else stage = WAIT_DRAW;
    }
    if (lane == 0) s.st = VfState{c, left, z, cur, next, depth, stage};
  }
  __threadfence_block();
  __syncthreads();
}

// Bound by memory. CW waves share a chunk: with 4 each has 16 logits per lane and the waves' sums
// are joined in LDS; with 1 a lane has 64, which spreads the wave's sums and the loads' latency
// over more logits.
template <typename T, int CW>
__global__ __launch_bounds__(BLOCK) void k_verify_rows(VfDev p) {
  __shared__ VfPart w[NWAVES];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
  const int chunk = CW == 1 ? (int)blockIdx.x * NWAVES + wave : (int)blockIdx.x, node = blockIdx.y, b = blockIdx.z;
  if (CW == 1 && chunk >= p.chunks) return;
  const double itd = inv_temp(p, b);
  // Twice log2(e) / T, not 0, whose product with -inf is a NaN, for half the distance of a logit from the
  // maximum: that of two finite logits may lie beyond fp32's range where a hot row's weights do not.
  const float it2 = fmaxf(fminf((float)(2.0 * itd), 3e38f), 1.4e-45f);
  auto weight = [&](float z, float m) { return __builtin_amdgcn_exp2f(__builtin_fmaf(z, 0.5f, -0.5f * m) * it2); };
  const T* row = row_of<T>(p, b, node);
  constexpr int G = VF_CH / (8 * WAVE * CW);
  const int i0 = chunk * VF_CH + (CW == 1 ? lane : (int)threadIdx.x) * 8;
  constexpr int STEP = 8 * WAVE * CW;
  T raw[G][8];  // as stored: half the registers, twice the waves
  float m = -__builtin_inff();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int i = i0 + g * STEP;
    if (i + 8 <= p.V) {
      __builtin_memcpy(raw[g], row + i, sizeof raw[g]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[g][j] = i + j < p.V ? row[min(i + j, p.V - 1)] : (T)-__builtin_inff();
    }
  }
  auto z = [&](int g, int j) { return clean(to_f32(raw[g][j])); };
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, z(g, j));
  m = wave_max(m);
  float sum = 0.f;
  int at = 0x7FFFFFFF;
  if (m > -__builtin_inff()) {
    if (itd != 0.0) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[j & 3] += weight(z(g, j), m);
      sum = wave_sum((part[0] + part[1]) + (part[2] + part[3]));
    } else {
#pragma unroll
      for (int g = G - 1; g >= 0; --g)
#pragma unroll
        for (int j = 7; j >= 0; --j)
          if (z(g, j) == m) at = i0 + g * STEP + j;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) at = min(at, __shfl_xor(at, o, WAVE));
    }
  }
  VfPart o{m, sum, at, 0};
  if (CW > 1) {
    if (lane == 0) w[wave] = o;
    __syncthreads();
    if (threadIdx.x != 0) return;
    o = w[0];
#pragma unroll
    for (int k = 1; k < CW; ++k)
      if (w[k].m > o.m || (w[k].m == o.m && w[k].at < o.at)) {
        o.m = w[k].m;
        o.at = w[k].at;
      }
    o.s = 0.f;
#pragma unroll
    for (int k = 0; k < CW; ++k)
      if (w[k].s > 0.f) o.s += w[k].s * weight(w[k].m, o.m);
  }
  if (CW == 1 ? lane == 0 : true) p.part[((long long)b * p.N + node) * p.chunks + chunk] = o;
}

// The tree into LDS.
__device__ __forceinline__ void load_nodes(const VfDev& p, VfShared& s, int b) {
  const int i = threadIdx.x;
  if (i < p.N) {
    const long long at = (long long)b * p.N + i;
    const int par = p.parents[at];
    s.par[i] = i > 0 && par >= 0 && par < i ? par : -1;
    s.tok[i] = p.tokens[at];
    s.u[i] = p.u[at];
  }
}

// The first pass's start: all rows' sums in LDS (and, from one workgroup, in memory).
template <typename T>
__device__ __forceinline__ void join_rows(const VfDev& p, VfShared& s, int b, double it, bool write) {
  const int lane = threadIdx.x % WAVE;
  load_nodes(p, s, b);
  __syncthreads();
  float zt = 0.f, qt = 0.f;  // this node's token under its parent, loaded early
  bool has = false;
  const int i = threadIdx.x;
  if (i < p.N) {
    const int par = s.par[i], t = s.tok[i];
    has = par >= 0 && (unsigned)t < (unsigned)p.V;
    if (has) {
      zt = to_f32(row_of<T>(p, b, par)[t]);
      if (p.q != nullptr) qt = p.q[(long long)b * p.qb + (long long)par * p.qn + t];
    }
  }
  // a wave per row joins its chunks, in a fixed order; 4 rows' loads at once
  constexpr int NW = VF_NT / WAVE, U = 4;
  const int wave = threadIdx.x / WAVE;
  const VfPart none{-__builtin_inff(), 0.f, 0x7FFFFFFF, 0};
  for (int r0 = wave; r0 < p.N; r0 += U * NW) {
    VfPart o[U];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int r = r0 + n * NW;
      o[n] = none;
      if (r < p.N && lane < p.chunks) o[n] = p.part[((long long)b * p.N + r) * p.chunks + lane];
    }
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int r = r0 + n * NW;
      if (r >= p.N) break;
      const VfPart* part = p.part + ((long long)b * p.N + r) * p.chunks;
      float m = o[n].m;
      for (int k = lane + WAVE; k < p.chunks; k += WAVE) m = fmaxf(m, part[k].m);
      m = wave_max(m);
      int at = o[n].m == m ? o[n].at : 0x7FFFFFFF;
      double sum = o[n].s > 0.f ? (double)o[n].s * expw(o[n].m, m, it) : 0.0;
      for (int k = lane + WAVE; k < p.chunks; k += WAVE) {
        const VfPart x = part[k];
        if (x.m == m) at = min(at, x.at);
        if (x.s > 0.f) sum += (double)x.s * expw(x.m, m, it);
      }
      sum = wave_sum_d(sum);
      if (it == 0.0) {  // greedy rows only have it
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) at = min(at, __shfl_xor(at, d, WAVE));
      }
      if (lane == 0) {
        s.m[r] = m;
        s.at[r] = at == 0x7FFFFFFF ? -1 : at;
        s.rs[r] = sum;
      }
    }
  }
  __syncthreads();
  if (i < p.N) {
    const double et = has && s.m[s.par[i]] > -__builtin_inff() ? expw(clean(zt), s.m[s.par[i]], it) : 0.0;
    s.et[i] = et;
    s.qt[i] = qt;
    if (write) p.rows[(long long)b * p.N + i] = VfRow{s.rs[i], et, s.m[i], qt, s.at[i], 0};
  }
  if (i == 0) {
    s.st = VfState{0.0, 1.0, 0.0, 0, 1, 1, WAIT_REST};
    if (write) p.nodes[(long long)b * p.N] = 0;
  }
}

// What the passes before `pass` left, into LDS.
__device__ __forceinline__ void load_state(const VfDev& p, VfShared& s, int b, int pass) {
  load_nodes(p, s, b);
  const int i = threadIdx.x;
  if (i < p.N) {
    const VfRow r = p.rows[(long long)b * p.N + i];
    s.rs[i] = r.s;
    s.et[i] = r.et;
    s.qt[i] = r.qt;
    s.m[i] = r.m;
    s.at[i] = r.at;
  }
  if (i == 0) s.st = p.state[(long long)(pass & 1) * p.B + b];
  __syncthreads();
}

// Pass `pass`; FIRST: pass 0, which joins the rows' sums.
template <typename T, bool FIRST>
__global__ __launch_bounds__(VF_NT) void k_verify_pass(VfDev p, int pass) {
  constexpr int NT = VF_NT;
  __shared__ VfShared s;
  const int chunk = blockIdx.x, b = blockIdx.y;
  const bool first = chunk == 0;
  const double it = inv_temp(p, b);
  VfState* now = p.state + (long long)((pass + 1) & 1) * p.B + b;
  if constexpr (FIRST) {
    join_rows<T>(p, s, b, it, first);
    walk(p, s, b, it, 0, first);
  } else {
    const int src = (pass - 1) & 1;
    const VfBin v = first_bin(p, bins_of(p, src, b));  // all loads before the first is waited for
    load_state(p, s, b, pass);
    if (s.st.stage != WAIT_REST) {
      if (first && threadIdx.x == 0) {
        *now = s.st;
        if (s.st.stage == WAIT_DRAW) now->stage = DONE + src;
      }
      return;
    }
    join_bins<NT>(p, s, bins_of(p, src, b), v);
    if (!s.again) walk(p, s, b, it, src, first);
  }
  if (first && threadIdx.x == 0) *now = s.st;
  if (s.st.stage >= DONE) return;
  const VfBin v = bin_block<T, NT>(p, s, b, it, chunk);
  if (threadIdx.x == 0) bins_of(p, pass & 1, b)[chunk] = v;
}

template <typename T>
__global__ __launch_bounds__(VF_NT) void k_verify_end(VfDev p, int passes) {
  __shared__ VfShared s;
  const int b = blockIdx.x;
  const double it = inv_temp(p, b);
  load_state(p, s, b, passes);
  int src = (passes - 1) & 1;
  // at most one round per node and two more per row: each consumes a child or settles a row's sum
  while (s.st.stage < DONE) {
    if (s.st.stage == WAIT_DRAW) {
      __syncthreads();
      if (threadIdx.x == 0) s.st.stage = DONE + src;
      __syncthreads();
      break;
    }
    join_bins<VF_NT>(p, s, bins_of(p, src, b), first_bin(p, bins_of(p, src, b)));
    if (!s.again) walk(p, s, b, it, src, true);
    if (s.st.stage >= DONE) break;
    src = 2;
    for (int k = threadIdx.x / WAVE; k < p.chunks; k += VF_NT / WAVE) {
      const VfBin v = bin_wave<T>(p, s, b, it, k);
      if (threadIdx.x % WAVE == 0) bins_of(p, 2, b)[k] = v;
    }
    __threadfence_block();
    __syncthreads();
  }
  finish<T>(p, s, b, it);
}

template <typename T>
pi_status launch_verify(pi_ctx* c, const VfDev& p) {
  // a wave per chunk where that many waves fill the chip (8 per SIMD) all the same
  if ((long long)p.chunks * p.N * p.B >= (long long)c->cus * 32)
    PI_HIP(c, launch_k(c, 0, k_verify_rows<T, 1>, dim3((p.chunks + NWAVES - 1) / NWAVES, p.N, p.B), 0, p));
  else
    PI_HIP(c, launch_k(c, 0, k_verify_rows<T, NWAVES>, dim3(p.chunks, p.N, p.B), 0, p));
  // A pass costs some 2 us where it finds nothing to do; what is left after the last one k_verify_end does
  // on one CU, at 63 us a residual of 131072 tokens and 12 of 32000. The more nodes there are in all, the
  // likelier is a path with many rejections. Means over 36 draws (the longest of them), us, with 2, 4 and
  // 6 passes: one chain of 5, 32000 tokens: 31.9, 35.5 (all that it can take); one tree of 16: 34.4, 37.9,
  // 41.5; 131072 tokens: 39.8 (105), 40.0 (47), 43.8; one tree of 32, 32000 tokens: 35.8 (94), 38.3 (70),
  // 41.6 (60); 4 trees of 32: 45.8, 44.6, 48.4; 131072 tokens: 76 (187), 51 (62), 56; 16 of 32: 150 (223),
  // 81 (89), 86; 32 of 32: 202, 127, 132; 8 of 64: 162 (279), 91 (162), 85 (95); 64 of 8: 147, 106, 113.
  // Without a q one pass is enough but for tests too near to call.
  const int most = p.N * p.B > 16 ? 4 : 2;
  const int passes = p.q == nullptr ? 1 : std::min(most, std::max(1, p.N - 1));
  PI_HIP(c, launch_kb(c, 0, k_verify_pass<T, true>, dim3(p.chunks, p.B), VF_NT, 0, p, 0));
  for (int i = 1; i < passes; ++i) PI_HIP(c, launch_kb(c, 0, k_verify_pass<T, false>, dim3(p.chunks, p.B), VF_NT, 0, p, i));
  PI_HIP(c, launch_kb(c, 0, k_verify_end<T>, dim3(p.B), VF_NT, 0, p, passes));
  return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_verifier_create(pi_ctx* ctx, int32_t vocab, int32_t max_batch, int32_t max_nodes, pi_verifier** out) {
  if (ctx == nullptr || out == nullptr) return PI_ERR_INVALID;
  *out = nullptr;
  if (vocab < 1 || max_batch < 1 || max_nodes < 1)
    return fail(ctx, PI_ERR_INVALID, "bad limits: vocab %d, %d sequences, %d nodes", vocab, max_batch, max_nodes);
  if (max_nodes > VF_MAX_NODES || max_batch > 65535 || vocab > (1 << 30))
    return fail(ctx, PI_ERR_UNSUPPORTED, "limits: vocab 2^30, 65535 sequences, %d nodes", VF_MAX_NODES);
  const int chunks = (vocab + VF_CH - 1) / VF_CH;
  const size_t rows = (size_t)max_batch * max_nodes;
  const size_t o_rows = sizeof(VfPart) * rows * chunks, o_state = o_rows + sizeof(VfRow) * rows,
               o_bins = o_state + 2 * sizeof(VfState) * max_batch,
               bytes = o_bins + 3 * sizeof(VfBin) * max_batch * chunks;
  PI_HIP(ctx, hipSetDevice(ctx->device));
  uint8_t* ws = nullptr;
  if (hipMalloc(reinterpret_cast<void**>(&ws), bytes) != hipSuccess) {
    (void)hipGetLastError();
    return fail(ctx, PI_ERR_OOM, "verifier scratch of %zu bytes", bytes);
  }
  pi_verifier* v = new (std::nothrow) pi_verifier{
      ctx, vocab, max_batch, max_nodes, chunks, ws, reinterpret_cast<VfPart*>(ws), reinterpret_cast<VfRow*>(ws + o_rows),
      reinterpret_cast<VfState*>(ws + o_state), reinterpret_cast<VfBin*>(ws + o_bins)};
  if (v == nullptr) {
    (void)hipFree(ws);
    return fail(ctx, PI_ERR_OOM, "host allocation failed");
  }
  ctx_retain(ctx);
  *out = v;
  return PI_OK;
}

void pi_verifier_destroy(pi_verifier* ver) {
  if (ver == nullptr) return;
  (void)hipSetDevice(ver->ctx->device);
  (void)hipFree(ver->ws);
  ctx_release(ver->ctx);
  delete ver;
}

pi_status pi_verify(pi_ctx* ctx, pi_verifier* ver, const pi_verify_args* args) {
  if (ctx == nullptr) return PI_ERR_INVALID;
  if (ver == nullptr) return fail(ctx, PI_ERR_INVALID, "ver is NULL");
  if (ver->ctx != ctx) return fail(ctx, PI_ERR_INVALID, "ver belongs to another context");
  if (args == nullptr) return fail(ctx, PI_ERR_INVALID, "args is NULL");
  const pi_verify_args& a = *args;
  if (a.B < 1 || a.N < 1 || a.B > ver->max_batch || a.N > ver->max_nodes)
    return fail(ctx, PI_ERR_INVALID, "B %d, N %d outside 1..%d, 1..%d", a.B, a.N, ver->max_batch, ver->max_nodes);
  if (a.dtype != PI_T_F32 && a.dtype != PI_T_F16 && a.dtype != PI_T_BF16)
    return fail(ctx, PI_ERR_INVALID, "logits: unknown dtype %d", a.dtype);
  if (a.logits == nullptr || a.tokens == nullptr || a.parents == nullptr || a.u == nullptr || a.u_next == nullptr ||
      a.nodes == nullptr || a.out == nullptr || a.n == nullptr)
    return fail(ctx, PI_ERR_INVALID, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(a.logits) & (a.dtype == PI_T_F32 ? 3u : 1u))
    return fail(ctx, PI_ERR_INVALID, "logits is not aligned to its elements");
  for (const void* q : {(const void*)a.q, (const void*)a.tokens, (const void*)a.parents, (const void*)a.u,
                        (const void*)a.u_next, (const void*)a.temperature, (const void*)a.nodes, (const void*)a.out,
                        (const void*)a.n})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return fail(ctx, PI_ERR_INVALID, "a pointer is not 4-byte aligned");
  PI_HIP(ctx, hipSetDevice(ctx->device));
  const VfDev p{a.logits, a.q, a.logits_batch, a.logits_node, a.q_batch, a.q_node, a.tokens, a.parents, a.u, a.u_next,
                a.temperature, a.nodes, a.out, a.n, a.B, a.N, ver->vocab, ver->chunks, ver->part, ver->rows, ver->state,
                ver->bins};
  switch (a.dtype) {
    case PI_T_F32: return launch_verify<float>(ctx, p);
    case PI_T_F16: return launch_verify<half_t>(ctx, p);
    default: return launch_verify<bf16_t>(ctx, p);
  }
}

}  // extern "C"
