// Check of drafted tokens by rejection sampling (pi_verify).
//
// Which child of a node is taken depends on p(t) = exp((z_t - max) / T) / sum of its parent's row,
// on the draft's q(t) and, after rejections, on c and the weight S that is left: after j of
// them the residual is max(p - c q, 0) / S with c_{j+1} = c_j + S_j, S_{j+1} = sum_t max(p - c_{j+1} q, 0).
// So no residual is ever stored: every pass recomputes it from the logits.
//
//   k_verify_rows   every row's maximum and sum, in chunks of the vocabulary
//   k_verify_walk   a workgroup per sequence joins the chunks and walks the tree from its root, as
//                   far as it can without a residual's weight
//   k_verify_rest   the weight of one residual per sequence, in the same chunks. Every workgroup
//                   first joins the chunks of the pass before and walks on, all alike, so that
//                   no workgroup waits for another. Launched a fixed number of times (they
//                   return at once where the sequence is done), then k_verify_end does
//                   whatever is left. Vocabularies of few chunks have no such launch: the walk's
//                   workgroup takes the residuals itself, a chunk per wave.
// A walk that ends draws the next token: the chunk by the chunks' sums, then the token inside it.
//
// The draws compare running sums over the vocabulary, whose steps are as small as 1e-6 of the
// whole: exponentials and sums are in 64 bits throughout (a 32-bit exponential alone would move
// one draw in some hundred).
#include <algorithm>
#include <new>

#include "pi_host.hpp"
#include "pi_types.hpp"

using namespace pi;

namespace {

constexpr int VF_CH = 4096;        // tokens per chunk: 16 per thread of a workgroup, 64 per lane of a wave
constexpr int VF_MAX_NODES = 256;
constexpr int VF_RESTS = 4;        // launches of k_verify_rest, where there are any
constexpr int VF_NT = 1024;        // threads of the walk's workgroup
constexpr int VF_OWN_CHUNKS = VF_NT / WAVE;  // up to so many chunks the walk's workgroup does all itself

struct VfPart {   // a chunk of a row
  double s;       // sum of exp((z - m) / T)
  float m;        // maximum
  int32_t at;     // its lowest index (greedy rows only)
};
struct VfRow {    // a row; for a node also its own token's p and q under its parent
  double s, pt, qt;
  float m;
  int32_t at;
};
struct VfState {
  double c, left;
  int32_t cur, next, depth;
  int32_t done;   // 1: the walk ended; 2, 3: with the weights of a pass of that parity
};

}  // namespace

struct pi_verifier {
  pi_ctx* ctx;
  int vocab, max_batch, max_nodes, chunks;
  uint8_t* ws;
  VfPart* part;     // [B][N][chunks]
  VfRow* rows;      // [B][N]
  VfState* state;   // [2][B], by the parity of the pass
  double* rest;     // [3][B][chunks]: two passes' weights; the walk's own
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
  double* rest;
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

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, WAVE);
  return v;
}

// Sum over the workgroup's NT threads, the same on every thread; red: NT / WAVE doubles.
template <int NT>
__device__ __forceinline__ double block_sum_d(double v, double* red) {
  v = wave_sum_d(v);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) red[threadIdx.x / WAVE] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NT / WAVE; ++i) s += red[i];
  return s;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const VfDev& p, int b, int i) {
  return static_cast<const T*>(p.logits) + (long long)b * p.lb + (long long)i * p.ln;
}
__device__ __forceinline__ double inv_temp(const VfDev& p, int b) {  // log2(e) / T; 0: greedy
  const float t = p.temp == nullptr ? 1.f : p.temp[b];
  return t > 0.f ? 1.4426950408889634 / (double)t : 0.0;
}
// Weights of a pass (0, 1, by its parity) or of the walk itself (2).
__device__ __forceinline__ double* rest_of(const VfDev& p, int which, int b) {
  return p.rest + ((long long)which * p.B + b) * p.chunks;
}

struct VfShared {
  double pt[VF_MAX_NODES], qt[VF_MAX_NODES], rs[VF_MAX_NODES];
  float m[VF_MAX_NODES], u[VF_MAX_NODES];
  int32_t at[VF_MAX_NODES], par[VF_MAX_NODES], tok[VF_MAX_NODES];
  VfState st;
  double red[VF_NT / WAVE];
  double target, before;
  int32_t pick, last;
};

// The weights that are left, from token i on: p, p - c q or p without the children's tokens.
enum { REST_P = 0, REST_Q = 1, REST_KIDS = 2 };
template <typename T>
__device__ __forceinline__ void rest8(const VfDev& p, const VfShared& s, int b, int kind, double it, int i, double (&w)[8]) {
  const int cur = s.st.cur;
  float z[8], q[8];
  logits8(row_of<T>(p, b, cur), i, p.V, z);
  if (kind == REST_Q) {
    const float* qr = p.q + (long long)b * p.qb + (long long)cur * p.qn;
    if (i + 8 <= p.V) {
      __builtin_memcpy(q, qr + i, sizeof q);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = i + j < p.V ? qr[i + j] : 0.f;
    }
  }
  const float m = s.m[cur];
  const double is = 1.0 / s.rs[cur];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = expw(z[j], m, it) * is;
  if (kind == REST_Q) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < p.V) w[j] = fmax(w[j] - s.st.c * (double)q[j], 0.0);
  } else if (kind == REST_KIDS) {
    for (int k = cur + 1; k < p.N; ++k) {
      const int t = s.tok[k] - i;
      if (s.par[k] == cur && t >= 0 && t < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (t == j) w[j] = 0.0;
      }
    }
  }
}

// A chunk's weight, by one wave (part `k` of `of`); the same on every lane.
template <typename T>
__device__ __forceinline__ double rest_wave(const VfDev& p, const VfShared& s, int b, int kind, double it, int chunk, int k = 0,
                                            int of = 1) {
  double v = 0.0, w[8];
  const int each = VF_CH / (8 * WAVE) / of;
#pragma unroll 4
  for (int g = k * each; g < (k + 1) * each; ++g) {
    const int i = chunk * VF_CH + (g * WAVE + (int)threadIdx.x % WAVE) * 8;
    if (i < p.V) {
      rest8<T>(p, s, b, kind, it, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v += w[j];
    }
  }
  return wave_sum_d(v);
}

// Draw the next token at node s.st.cur and write the sequence's outputs. All NT threads; `bins`:
// the chunks' weights of the residual that is left, where the walk ended on one.
template <typename T, int NT>
__device__ __forceinline__ void finish(const VfDev& p, VfShared& s, int b, double it, const double* bins) {
  const int cur = s.st.cur, lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  int next = -1;
  if (it == 0.0) {
    next = s.at[cur];
  } else if (s.rs[cur] > 0.0) {
    double* own = rest_of(p, 2, b);
    int kind = p.q != nullptr ? (s.st.c > 0.0 ? REST_Q : REST_P) : REST_KIDS;
    const VfPart* part = p.part + ((long long)b * p.N + cur) * p.chunks;
    auto own_bins = [&]() {  // p itself, from the rows' pass
      for (int k = threadIdx.x; k < p.chunks; k += NT)
        own[k] = part[k].s > 0.0 ? part[k].s * expw(part[k].m, s.m[cur], it) / s.rs[cur] : 0.0;
      __threadfence_block();
      __syncthreads();
      bins = own;
    };
    if (kind != REST_Q) own_bins();
    if (kind == REST_KIDS) {  // the chunks that lose a token are summed again, a wave per child
      int nth = 0;
      for (int k = cur + 1; k < p.N; ++k) {
        if (s.par[k] != cur || (unsigned)s.tok[k] >= (unsigned)p.V || nth++ % (NT / WAVE) != wave) continue;
        const int ch = s.tok[k] / VF_CH;
        const double v = rest_wave<T>(p, s, b, kind, it, ch);
        if (lane == 0) own[ch] = v;  // children of one chunk write the same
      }
      __threadfence_block();
      __syncthreads();
    }
    for (int attempt = 0; attempt < 2; ++attempt) {
      double total = 0.0;
      for (int k = threadIdx.x; k < p.chunks; k += NT) total += bins[k];
      total = block_sum_d<NT>(total, s.red);
      if (threadIdx.x == 0) {
        s.target = (double)p.u_next[b] * total;
        s.before = 0.0;
        s.pick = 0x7FFFFFFF;
        s.last = -1;
      }
      __syncthreads();
      if (total > 0.0 || attempt == 1) break;
      kind = REST_P;
      own_bins();
    }
    // the chunk whose running sum passes the target, or the last one with any weight
    const double target = s.target;
    double carry = 0.0;
    for (int k0 = 0; k0 < p.chunks; k0 += NT) {
      const int k = k0 + (int)threadIdx.x;
      const double v = k < p.chunks ? bins[k] : 0.0;
      double incl = v;
#pragma unroll
      for (int o = 1; o < WAVE; o <<= 1) {
        const double t = __shfl_up(incl, o, WAVE);
        if (lane >= o) incl += t;
      }
      __syncthreads();
      if (lane == WAVE - 1) s.red[wave] = incl;
      __syncthreads();
      double run = carry;
      for (int i = 0; i < NT / WAVE; ++i) {
        if (i < wave) run += s.red[i];
        carry += s.red[i];
      }
      run += incl;
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
    if (chunk >= 0) {  // the token: TPT tokens per thread in order, threads in order
      constexpr int TPT = VF_CH / NT < 8 ? 8 : VF_CH / NT;
      double w[TPT], sum = 0.0;
      int lastw = -1;
      const int i0 = chunk * VF_CH + (int)threadIdx.x * TPT;
#pragma unroll
      for (int g = 0; g < TPT; g += 8) {
        double w8[8];
        const bool in = threadIdx.x * TPT < VF_CH && i0 + g < p.V;
        if (in) rest8<T>(p, s, b, kind, it, i0 + g, w8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[g + j] = in ? w8[j] : 0.0;
          sum += w[g + j];
          if (w[g + j] > 0.0) lastw = i0 + g + j;
        }
      }
      double incl = sum;
#pragma unroll
      for (int o = 1; o < WAVE; o <<= 1) {
        const double t = __shfl_up(incl, o, WAVE);
        if (lane >= o) incl += t;
      }
      if (lane == WAVE - 1) s.red[wave] = incl;
      __syncthreads();
      double run = incl - sum;
      for (int i = 0; i < wave; ++i) run += s.red[i];
      int mine = 0x7FFFFFFF;
#pragma unroll
      for (int j = 0; j < TPT; ++j) {
        run += w[j];
        if (w[j] > 0.0 && run > rest) mine = min(mine, i0 + j);
      }
      if (mine != 0x7FFFFFFF) atomicMin(&s.pick, mine);
      if (lastw >= 0) atomicMax(&s.last, lastw);
      __syncthreads();
      next = s.pick != 0x7FFFFFFF ? s.pick : s.last;
    }
  }
  const int depth = s.st.depth;  // nodes of the path; its nodes are written already
  for (int k = threadIdx.x; k < p.N; k += NT) {
    int o = -1;
    if (k + 1 < depth) o = s.tok[p.nodes[(long long)b * p.N + k + 1]];
    else if (k + 1 == depth) o = next;
    p.out[(long long)b * p.N + k] = o;
    if (k >= depth) p.nodes[(long long)b * p.N + k] = -1;
  }
  if (threadIdx.x == 0) p.n[b] = depth;
}

// Walk on from s.st until a residual's weight is needed or no child is left to try (s.st.done).
// All threads; the first wave walks, all its lanes on the same values. `write`: the path goes to
// memory.
__device__ __forceinline__ void walk(const VfDev& p, VfShared& s, int b, double it, bool write) {
  __syncthreads();
  if (threadIdx.x < WAVE) {
    const int lane = threadIdx.x;
    int cur = s.st.cur, next = s.st.next, depth = s.st.depth;
    double c = s.st.c, left = s.st.left;
    bool end = true;
    for (int g = next / WAVE; g * WAVE < p.N;) {
      const int i0 = g * WAVE + lane;
      uint64_t kids = __ballot(i0 < p.N && i0 >= next && s.par[i0] == cur);
      if (kids == 0) {
        ++g;
        continue;
      }
      const int i = g * WAVE + __ffsll((unsigned long long)kids) - 1;
      next = i + 1;
      const double pt = s.pt[i], u = (double)s.u[i];
      bool take;
      if (p.q != nullptr) {
        const double qt = s.qt[i];
        take = u * left * qt < fmax(pt - c * qt, 0.0);
        if (!take) {
          c += left;
          if (it == 0.0) {  // all weight at one token
            const int a = s.at[cur];
            left = a >= 0 ? fmax(1.0 - c * (double)p.q[(long long)b * p.qb + (long long)cur * p.qn + a], 0.0) : 0.0;
          } else if (left > 0.0) {
            end = false;
          }
        }
      } else {
        bool again = false;
        for (int k0 = 0; k0 < i; k0 += WAVE) {
          const int k = k0 + lane;
          again = again || __any(k < i && s.par[k] == cur && s.tok[k] == s.tok[i]);
        }
        take = !again && u * left < pt;
        if (!take && !again) left -= pt;
      }
      if (take) {
        cur = i;
        c = 0.0;
        left = 1.0;
        if (write && lane == 0) p.nodes[(long long)b * p.N + depth] = i;
        ++depth;
      }
      if (!end) break;
      g = next / WAVE;
    }
    if (lane == 0) s.st = VfState{c, left, cur, next, depth, end ? 1 : 0};
  }
  __threadfence_block();
  __syncthreads();
}

// What is left to do for a sequence, by its own workgroup: walk on, with the residuals of `bins`
// where the state waits for one.
template <typename T>
__device__ __forceinline__ void to_the_end(const VfDev& p, VfShared& s, int b, double it, const double* bins) {
  // at most one round per node: each consumes a child
  while (!s.st.done) {
    if (bins == nullptr) {
      double* own = rest_of(p, 1, b);
      constexpr int NW = VF_NT / WAVE;
      const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
      const int of = p.chunks <= NW / 8 ? 8 : p.chunks <= NW / 4 ? 4 : p.chunks <= NW / 2 ? 2 : 1;  // waves per chunk
      if (of == 1) {
        for (int k = wave; k < p.chunks; k += NW) {
          const double v = rest_wave<T>(p, s, b, REST_Q, it, k);
          if (lane == 0) own[k] = v;
        }
      } else {
        const double v = wave / of < p.chunks ? rest_wave<T>(p, s, b, REST_Q, it, wave / of, wave % of, of) : 0.0;
        __syncthreads();
        if (lane == 0) s.red[wave] = v;
        __syncthreads();
        if ((int)threadIdx.x < p.chunks) {
          double t = 0.0;
          for (int k = 0; k < of; ++k) t += s.red[threadIdx.x * of + k];
          own[threadIdx.x] = t;
        }
      }
      __threadfence_block();
      __syncthreads();
      bins = own;
    }
    double left = 0.0;
    for (int k = threadIdx.x; k < p.chunks; k += VF_NT) left += bins[k];
    left = block_sum_d<VF_NT>(left, s.red);
    if (threadIdx.x == 0) s.st.left = left;
    walk(p, s, b, it, true);
    if (!s.st.done) bins = nullptr;
  }
  finish<T, VF_NT>(p, s, b, it, bins);
}

// Bound by memory and by the exponentials, about 20 instructions of 64 bits per logit. CW waves
// share a chunk: with 4 each has 16 logits per lane and the waves' sums are joined in LDS; with 1
// a lane has 64, which spreads the wave's sums and the loads' latency over more logits.
template <typename T, int CW>
__global__ __launch_bounds__(BLOCK) void k_verify_rows(VfDev p) {
  __shared__ VfPart w[NWAVES];
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
  const int chunk = CW == 1 ? (int)blockIdx.x * NWAVES + wave : (int)blockIdx.x, node = blockIdx.y, b = blockIdx.z;
  if (CW == 1 && chunk >= p.chunks) return;
  const double it = inv_temp(p, b);
  const T* row = row_of<T>(p, b, node);
  constexpr int G = VF_CH / (8 * WAVE * CW);
  const int i0 = chunk * VF_CH + (CW == 1 ? lane : (int)threadIdx.x) * 8;
  constexpr int STEP = 8 * WAVE * CW;
  float z[G][8];
  float m = -__builtin_inff();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (i0 + g * STEP < p.V) {
      logits8(row, i0 + g * STEP, p.V, z[g]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[g][j] = -__builtin_inff();
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, z[g][j]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, WAVE));
  double sum = 0.0;
  int at = 0x7FFFFFFF;
  if (m > -__builtin_inff()) {
    if (it != 0.0) {
      // a weight below 2^-1000 of the largest counts as that: it does not change the sum
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += pow2_floor(((double)z[g][j] - (double)m) * it);
      sum = wave_sum_d(sum);
    } else {
#pragma unroll
      for (int g = G - 1; g >= 0; --g)
#pragma unroll
        for (int j = 7; j >= 0; --j)
          if (z[g][j] == m) at = i0 + g * STEP + j;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) at = min(at, __shfl_xor(at, o, WAVE));
    }
  }
  VfPart o{sum, m, at};
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
    o.s = 0.0;
    if (it != 0.0 && o.m > -__builtin_inff()) {
#pragma unroll
      for (int k = 0; k < CW; ++k) o.s += w[k].s * expw(w[k].m, o.m, it);
    }
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

// With `all` the sequence is brought to its end here.
template <typename T>
__global__ __launch_bounds__(VF_NT) void k_verify_walk(VfDev p, bool all) {
  __shared__ VfShared s;
  const int b = blockIdx.x, lane = threadIdx.x % WAVE;
  const double it = inv_temp(p, b);
  load_nodes(p, s, b);
  float zt = -__builtin_inff(), qv = 0.f;  // this node's token under its parent, loaded early
  bool has = false;
  if ((int)threadIdx.x < p.N) {
    const int par = s.par[threadIdx.x], t = s.tok[threadIdx.x];
    has = par >= 0 && (unsigned)t < (unsigned)p.V;
    if (has) {
      zt = clean(to_f32(row_of<T>(p, b, par)[t]));
      if (p.q != nullptr) qv = p.q[(long long)b * p.qb + (long long)par * p.qn + t];
    }
  }
  // a wave per row joins its chunks, in a fixed order
  for (int i = threadIdx.x / WAVE; i < p.N; i += VF_NT / WAVE) {
    const VfPart* part = p.part + ((long long)b * p.N + i) * p.chunks;
    float m = -__builtin_inff();
    double sum = 0.0;
    int at = 0x7FFFFFFF;
    if (p.chunks <= WAVE) {
      const VfPart o = lane < p.chunks ? part[lane] : VfPart{0.0, -__builtin_inff(), 0x7FFFFFFF};
      m = o.m;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, WAVE));
      if (o.m == m) at = o.at;
      if (o.s > 0.0) sum = o.s * expw(o.m, m, it);
    } else {
      for (int k = lane; k < p.chunks; k += WAVE) m = fmaxf(m, part[k].m);
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, WAVE));
      for (int k = lane; k < p.chunks; k += WAVE) {
        const VfPart o = part[k];
        if (o.m == m) at = min(at, o.at);
        if (o.s > 0.0) sum += o.s * expw(o.m, m, it);
      }
    }
    sum = wave_sum_d(sum);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) at = min(at, __shfl_xor(at, d, WAVE));
    if (lane == 0) {
      s.m[i] = m;
      s.at[i] = at == 0x7FFFFFFF ? -1 : at;
      s.rs[i] = sum;
    }
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i < p.N) {
    const int par = s.par[i];
    double pt = 0.0;
    if (has) {
      if (it == 0.0) pt = s.tok[i] == s.at[par] ? 1.0 : 0.0;
      else if (s.rs[par] > 0.0) pt = expw(zt, s.m[par], it) * (1.0 / s.rs[par]);
    }
    const double qt = (double)qv;
    s.pt[i] = pt;
    s.qt[i] = qt;
    if (!all) p.rows[(long long)b * p.N + i] = VfRow{s.rs[i], pt, qt, s.m[i], s.at[i]};
  }
  if (threadIdx.x == 0) {
    s.st = VfState{0.0, 1.0, 0, 1, 1, 0};
    p.nodes[(long long)b * p.N] = 0;
  }
  walk(p, s, b, it, true);
  if (all) to_the_end<T>(p, s, b, it, nullptr);
  else if (threadIdx.x == 0) p.state[b] = s.st;
}

// What the walk left, into LDS; `pass`: how many passes were before.
__device__ __forceinline__ void load_state(const VfDev& p, VfShared& s, int b, int pass) {
  load_nodes(p, s, b);
  const int i = threadIdx.x;
  if (i < p.N) {
    const VfRow r = p.rows[(long long)b * p.N + i];
    s.rs[i] = r.s;
    s.pt[i] = r.pt;
    s.qt[i] = r.qt;
    s.m[i] = r.m;
    s.at[i] = r.at;
  }
  if (i == 0) s.st = p.state[(long long)(pass & 1) * p.B + b];
  __syncthreads();
}

// Pass `pass` (from 0 on) over residuals: the walk goes on with the weights of the pass before.
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_verify_rest(VfDev p, int pass) {
  __shared__ VfShared s;
  const int chunk = blockIdx.x, b = blockIdx.y;
  const bool first = chunk == 0;
  VfState* now = p.state + (long long)((pass + 1) & 1) * p.B + b;
  if (p.state[(long long)(pass & 1) * p.B + b].done) {
    if (first && threadIdx.x == 0) *now = p.state[(long long)(pass & 1) * p.B + b];
    return;
  }
  load_state(p, s, b, pass);
  const double it = inv_temp(p, b);
  if (pass > 0) {
    const double* bins = rest_of(p, (pass - 1) & 1, b);
    double left = 0.0;
    for (int k = threadIdx.x; k < p.chunks; k += BLOCK) left += bins[k];
    left = block_sum_d<BLOCK>(left, s.red);
    if (threadIdx.x == 0) s.st.left = left;
    walk(p, s, b, it, first);
    if (s.st.done) {
      if (first && threadIdx.x == 0) {
        *now = s.st;
        now->done = 2 + ((pass - 1) & 1);
      }
      return;
    }
  }
  double v = 0.0, w[8];
#pragma unroll
  for (int g = 0; g < VF_CH / (8 * BLOCK); ++g) {
    const int i = chunk * VF_CH + (g * BLOCK + (int)threadIdx.x) * 8;
    if (i < p.V) {
      rest8<T>(p, s, b, REST_Q, it, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v += w[j];
    }
  }
  v = block_sum_d<BLOCK>(v, s.red);
  if (threadIdx.x == 0) {
    rest_of(p, pass & 1, b)[chunk] = v;
    if (first) *now = s.st;
  }
}

template <typename T>
__global__ __launch_bounds__(VF_NT) void k_verify_end(VfDev p, int passes) {
  __shared__ VfShared s;
  const int b = blockIdx.x;
  load_state(p, s, b, passes);
  to_the_end<T>(p, s, b, inv_temp(p, b), rest_of(p, s.st.done > 1 ? s.st.done - 2 : (passes - 1) & 1, b));
}

template <typename T>
pi_status launch_verify(pi_ctx* c, const VfDev& p) {
  // a wave per chunk where that many waves fill the chip (8 per SIMD) all the same
  if ((long long)p.chunks * p.N * p.B >= (long long)c->cus * 32)
    PI_HIP(c, launch_k(c, 0, k_verify_rows<T, 1>, dim3((p.chunks + NWAVES - 1) / NWAVES, p.N, p.B), 0, p));
  else
    PI_HIP(c, launch_k(c, 0, k_verify_rows<T, NWAVES>, dim3(p.chunks, p.N, p.B), 0, p));
  const bool all = p.q == nullptr || p.N == 1 || p.chunks <= VF_OWN_CHUNKS;
  PI_HIP(c, launch_kb(c, 0, k_verify_walk<T>, dim3(p.B), VF_NT, 0, p, all));
  if (all) return PI_OK;
  const int passes = std::min(VF_RESTS, p.N - 1);
  for (int i = 0; i < passes; ++i) PI_HIP(c, launch_k(c, 0, k_verify_rest<T>, dim3(p.chunks, p.B), 0, p, i));
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
               o_rest = o_state + 2 * sizeof(VfState) * max_batch,
               bytes = o_rest + 3 * sizeof(double) * max_batch * chunks;
  PI_HIP(ctx, hipSetDevice(ctx->device));
  uint8_t* ws = nullptr;
  if (hipMalloc(reinterpret_cast<void**>(&ws), bytes) != hipSuccess) {
    (void)hipGetLastError();
    return fail(ctx, PI_ERR_OOM, "verifier scratch of %zu bytes", bytes);
  }
  pi_verifier* v = new (std::nothrow) pi_verifier{
      ctx, vocab, max_batch, max_nodes, chunks, ws, reinterpret_cast<VfPart*>(ws), reinterpret_cast<VfRow*>(ws + o_rows),
      reinterpret_cast<VfState*>(ws + o_state), reinterpret_cast<double*>(ws + o_rest)};
  if (v == nullptr) {
    (void)hipFree(ws);
    return fail(ctx, PI_ERR_OOM, "host allocation failed");
  }
  *out = v;
  return PI_OK;
}

void pi_verifier_destroy(pi_verifier* ver) {
  if (ver == nullptr) return;
  (void)hipSetDevice(ver->ctx->device);
  (void)hipFree(ver->ws);
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
                ver->rest};
  switch (a.dtype) {
    case PI_T_F32: return launch_verify<float>(ctx, p);
    case PI_T_F16: return launch_verify<half_t>(ctx, p);
    default: return launch_verify<bf16_t>(ctx, p);
  }
}

}  // extern "C"
