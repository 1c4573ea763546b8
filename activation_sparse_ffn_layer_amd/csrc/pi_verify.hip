// Check of drafted tokens by rejection sampling (pi_verify).
//
// Which child of a node is taken depends on p(t) = exp((z_t - max) / T) / sum of its parent's row,
// on the draft's q(t) and, after rejections, on c and the weight S that is left: after j of
// them the residual is max(p - c q, 0) / S with c_{j+1} = c_j + S_j, S_{j+1} = sum_t max(p - c_{j+1} q, 0).
// So no residual is ever stored: every pass recomputes it from the logits.
//
//   k_verify_rows   every row's maximum and sum, in chunks of the vocabulary. The last workgroup
//                   of a sequence to finish walks the tree from its root, as far as it can
//                   without a residual's weight.
//   k_verify_rest   the weight of one residual per sequence, in the same chunks; its last
//                   workgroup walks on. Launched a fixed number of times (they return at once
//                   where the sequence is done), then k_verify_end does whatever is left.
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

constexpr int VF_CH = 4096;       // tokens per chunk: 16 per thread
constexpr int VF_MAX_NODES = 256; // one thread per node
constexpr int VF_RESTS = 4;       // launches of k_verify_rest

struct VfPart {   // a chunk of a row
  double s;       // sum of exp((z - m) / T)
  float m;        // maximum
  int32_t at;     // its lowest index
};
struct VfRow {    // a row; for a node also its own token's p and q under its parent
  double s, pt, qt;
  float m;
  int32_t at;
};
struct VfState {
  double c, left;
  int32_t cur, next, depth, done;
};

}  // namespace

struct pi_verifier {
  pi_ctx* ctx;
  int vocab, max_batch, max_nodes, chunks;
  uint8_t* ws;
  VfPart* part;     // [B][N][chunks]
  VfRow* rows;      // [B][N]
  VfState* state;   // [B]
  double* rest;     // [B][chunks]
  uint32_t* count;  // [B], zero between calls
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
  uint32_t* count;
};

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

__device__ __forceinline__ double shfl_xor_d(double v, int o) { return __shfl_xor(v, o, WAVE); }

// Sum over the workgroup, the same on every thread; red: NWAVES doubles.
__device__ __forceinline__ double block_sum_d(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += shfl_xor_d(v, o);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) red[threadIdx.x / WAVE] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NWAVES; ++i) s += red[i];
  return s;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const VfDev& p, int b, int i) {
  return static_cast<const T*>(p.logits) + (long long)b * p.lb + (long long)i * p.ln;
}
__device__ __forceinline__ double inv_temp(const VfDev& p, int b) {  // 0: greedy
  const float t = p.temp == nullptr ? 1.f : p.temp[b];
  return t > 0.f ? 1.0 / (double)t : 0.0;
}
__device__ __forceinline__ double expw(float z, float m, double it) { return exp(((double)z - (double)m) * it); }

struct VfShared {
  double pt[VF_MAX_NODES], qt[VF_MAX_NODES], rs[VF_MAX_NODES];
  float m[VF_MAX_NODES], u[VF_MAX_NODES];
  int32_t at[VF_MAX_NODES], par[VF_MAX_NODES], tok[VF_MAX_NODES];
  VfState st;
  double red[NWAVES];
  double pre[NWAVES + 1];
  int32_t pick, last;
  int final_;
};

// The weights that are left at the end of a walk, from token i on: p, p - c q or p without the
// children's tokens.
enum { REST_P = 0, REST_Q = 1, REST_KIDS = 2 };
template <typename T>
__device__ __forceinline__ void rest8(const VfDev& p, const VfShared& s, int b, int kind, double it, int i, double (&w)[8]) {
  const int cur = s.st.cur;
  float z[8];
  logits8(row_of<T>(p, b, cur), i, p.V, z);
  const float m = s.m[cur];
  const double is = 1.0 / s.rs[cur];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = expw(z[j], m, it) * is;
  if (kind == REST_Q) {
    const float* q = p.q + (long long)b * p.qb + (long long)cur * p.qn;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < p.V) w[j] = fmax(w[j] - s.st.c * (double)q[i + j], 0.0);
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

// A chunk's weight; a thread's 16 tokens are consecutive.
template <typename T>
__device__ __forceinline__ double rest_chunk(const VfDev& p, VfShared& s, int b, int kind, double it, int chunk) {
  double v = 0.0, w[8];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int i = chunk * VF_CH + threadIdx.x * 16 + g * 8;
    if (i < p.V) {
      rest8<T>(p, s, b, kind, it, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v += w[j];
    }
  }
  return block_sum_d(v, s.red);
}

// Draw the next token at node s.st.cur and write the sequence's outputs. All threads.
template <typename T>
__device__ void finish(const VfDev& p, VfShared& s, int b, double it) {
  const int cur = s.st.cur;
  int next = -1;
  if (it == 0.0) {
    next = s.at[cur];
  } else if (s.rs[cur] > 0.0) {
    double* bins = p.rest + (long long)b * p.chunks;
    int kind = p.q != nullptr ? (s.st.c > 0.0 ? REST_Q : REST_P) : REST_KIDS;
    const VfPart* part = p.part + ((long long)b * p.N + cur) * p.chunks;
    auto own_bins = [&]() {  // p itself, from the rows' pass
      for (int k = threadIdx.x; k < p.chunks; k += BLOCK)
        bins[k] = part[k].s > 0.0 ? part[k].s * expw(part[k].m, s.m[cur], it) / s.rs[cur] : 0.0;
    };
    if (kind == REST_P) own_bins();
    if (kind == REST_KIDS) {
      own_bins();
      for (int k = cur + 1; k < p.N; ++k) {  // the chunks that lose a token are summed again
        if (s.par[k] != cur || (unsigned)s.tok[k] >= (unsigned)p.V) continue;
        const int ch = s.tok[k] / VF_CH;
        const double v = rest_chunk<T>(p, s, b, kind, it, ch);
        if (threadIdx.x == 0) bins[ch] = v;
      }
    }
    __threadfence_block();
    __syncthreads();
    // the chunk: one wave runs along the bins
    for (int attempt = 0; attempt < 2; ++attempt) {
      double total = 0.0;
      for (int k = threadIdx.x; k < p.chunks; k += BLOCK) total += bins[k];
      total = block_sum_d(total, s.red);
      if (total > 0.0) break;
      __syncthreads();
      kind = REST_P;
      own_bins();
      __threadfence_block();
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      double total = 0.0;
      for (int k = 0; k < p.chunks; ++k) total += bins[k];
      const double target = (double)p.u_next[b] * total;
      double cum = 0.0, before = 0.0;
      int pick = -1, last = -1;
      double last_before = 0.0;
      for (int k = 0; k < p.chunks && pick < 0; ++k) {
        const double v = bins[k];
        if (v > 0.0) {
          last = k;
          last_before = cum;
        }
        if (cum + v > target) {
          pick = k;
          before = cum;
        }
        cum += v;
      }
      s.pick = pick >= 0 ? pick : last;
      s.pre[0] = target - (pick >= 0 ? before : last_before);
      s.last = -1;
    }
    __syncthreads();
    // the token: each thread's 16 in order, threads in order
    const int chunk = s.pick;
    const double target = s.pre[0];
    __syncthreads();
    double w[2][8], sum = 0.0;
    int lastw = -1;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int i = chunk * VF_CH + threadIdx.x * 16 + g * 8;
      if (i < p.V) rest8<T>(p, s, b, kind, it, i, w[g]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i >= p.V) w[g][j] = 0.0;
        sum += w[g][j];
        if (w[g][j] > 0.0) lastw = i + j;
      }
    }
    double incl = sum;
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) {
      const double t = __shfl_up(incl, o, WAVE);
      if (lane >= o) incl += t;
    }
    if (lane == WAVE - 1) s.red[wave] = incl;
    if (threadIdx.x == 0) s.pick = 0x7FFFFFFF;
    __syncthreads();
    double run = incl - sum;
    for (int i = 0; i < wave; ++i) run += s.red[i];
    int mine = 0x7FFFFFFF;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        run += w[g][j];
        if (w[g][j] > 0.0 && run > target) mine = min(mine, chunk * VF_CH + (int)threadIdx.x * 16 + g * 8 + j);
      }
    if (mine != 0x7FFFFFFF) atomicMin(&s.pick, mine);
    if (lastw >= 0) atomicMax(&s.last, lastw);
    __syncthreads();
    next = s.pick != 0x7FFFFFFF ? s.pick : s.last;
  }
  const int depth = s.st.depth;  // nodes of the path; its nodes are written already
  for (int k = threadIdx.x; k < p.N; k += BLOCK) {
    int o = -1;
    if (k + 1 < depth) o = s.tok[p.nodes[(long long)b * p.N + k + 1]];
    else if (k + 1 == depth) o = next;
    p.out[(long long)b * p.N + k] = o;
    if (k >= depth) p.nodes[(long long)b * p.N + k] = -1;
  }
  if (threadIdx.x == 0) p.n[b] = depth;
}

// Walk on from s.st until a residual's weight is needed (returns false) or no child is left to
// try (true). All lanes of one wave, on the same values.
__device__ __forceinline__ bool walk(const VfDev& p, VfShared& s, int b, double it) {
  const int lane = threadIdx.x % WAVE;
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
      if (lane == 0) p.nodes[(long long)b * p.N + depth] = i;
      ++depth;
    }
    if (!end) break;
    g = next / WAVE;
  }
  if (lane == 0) s.st = VfState{c, left, cur, next, depth, end ? 1 : 0};
  return end;
}

// Is this workgroup the last of `of` to arrive at the sequence's counter? Its writes are
// visible to the last one, and the others' to it.
__device__ __forceinline__ bool last_one(uint32_t* count, uint32_t of, int32_t* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t n = __hip_atomic_fetch_add(count, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    *flag = n + 1 == of;
    if (n + 1 == of) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!*flag) return false;
  __threadfence();
  return true;
}

// Walk on and, where the walk ends, finish; the state goes back to memory.
template <typename T>
__device__ void go_on(const VfDev& p, VfShared& s, int b, double it) {
  __syncthreads();
  if (threadIdx.x < WAVE) walk(p, s, b, it);
  __threadfence_block();
  __syncthreads();
  if (s.st.done) finish<T>(p, s, b, it);
  if (threadIdx.x == 0) p.state[b] = s.st;
}

// The tree and the rows' statistics into LDS.
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

template <typename T>
__global__ __launch_bounds__(BLOCK) void k_verify_rows(VfDev p) {
  __shared__ VfShared s;
  __shared__ float rm[NWAVES];
  __shared__ int32_t ri[NWAVES];
  const int chunk = blockIdx.x, node = blockIdx.y, b = blockIdx.z;
  const double it = inv_temp(p, b);
  const T* row = row_of<T>(p, b, node);
  float z[2][8];
  float m = -__builtin_inff();
  int at = -1;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int i = chunk * VF_CH + g * (VF_CH / 2) + threadIdx.x * 8;
    if (i < p.V) {
      logits8(row, i, p.V, z[g]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[g][j] = -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (z[g][j] > m) {
        m = z[g][j];
        at = i + j;
      }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float m2 = __shfl_xor(m, o, WAVE);
    const int a2 = __shfl_xor(at, o, WAVE);
    if (m2 > m || (m2 == m && (unsigned)a2 < (unsigned)at)) {
      m = m2;
      at = a2;
    }
  }
  if (threadIdx.x % WAVE == 0) {
    rm[threadIdx.x / WAVE] = m;
    ri[threadIdx.x / WAVE] = at;
  }
  __syncthreads();
  m = rm[0];
  at = ri[0];
#pragma unroll
  for (int w = 1; w < NWAVES; ++w)
    if (rm[w] > m || (rm[w] == m && (unsigned)ri[w] < (unsigned)at)) {
      m = rm[w];
      at = ri[w];
    }
  double sum = 0.0;
  if (it != 0.0 && at >= 0) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += expw(z[g][j], m, it);
  }
  sum = block_sum_d(sum, s.red);
  if (threadIdx.x == 0) p.part[((long long)b * p.N + node) * p.chunks + chunk] = VfPart{sum, m, at};
  if (!last_one(p.count + b, (uint32_t)(p.chunks * p.N), &s.pick)) return;

  // every row of the sequence is there: the rows' own statistics, a thread per node
  load_nodes(p, s, b);
  const int i = threadIdx.x;
  if (i < p.N) {
    const VfPart* part = p.part + ((long long)b * p.N + i) * p.chunks;
    float rmax = -__builtin_inff();
    int rat = -1;
    for (int k = 0; k < p.chunks; ++k)
      if (part[k].m > rmax) {
        rmax = part[k].m;
        rat = part[k].at;
      }
    double rs = 0.0;
    if (it != 0.0)
      for (int k = 0; k < p.chunks; ++k)
        if (part[k].s > 0.0) rs += part[k].s * expw(part[k].m, rmax, it);
    s.m[i] = rmax;
    s.at[i] = rat;
    s.rs[i] = rs;
  }
  __syncthreads();
  if (i < p.N) {
    const int par = s.par[i], t = s.tok[i];
    double pt = 0.0, qt = 0.0;
    if (par >= 0 && (unsigned)t < (unsigned)p.V) {
      if (it == 0.0) pt = t == s.at[par] ? 1.0 : 0.0;
      else if (s.rs[par] > 0.0) pt = expw(clean(to_f32(row_of<T>(p, b, par)[t])), s.m[par], it) * (1.0 / s.rs[par]);
      if (p.q != nullptr) qt = (double)p.q[(long long)b * p.qb + (long long)par * p.qn + t];
    }
    s.pt[i] = pt;
    s.qt[i] = qt;
    p.rows[(long long)b * p.N + i] = VfRow{s.rs[i], pt, qt, s.m[i], s.at[i]};
  }
  if (threadIdx.x == 0) {
    s.st = VfState{0.0, 1.0, 0, 1, 1, 0};
    p.nodes[(long long)b * p.N] = 0;
  }
  go_on<T>(p, s, b, it);
}

// What the rows' pass left, into LDS.
__device__ __forceinline__ void load_state(const VfDev& p, VfShared& s, int b) {
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
  if (i == 0) s.st = p.state[b];
  __syncthreads();
}

template <typename T>
__global__ __launch_bounds__(BLOCK) void k_verify_rest(VfDev p) {
  __shared__ VfShared s;
  const int chunk = blockIdx.x, b = blockIdx.y;
  if (p.state[b].done) return;
  load_state(p, s, b);
  const double it = inv_temp(p, b);
  const double v = rest_chunk<T>(p, s, b, REST_Q, it, chunk);
  double* bins = p.rest + (long long)b * p.chunks;
  if (threadIdx.x == 0) bins[chunk] = v;
  if (!last_one(p.count + b, (uint32_t)p.chunks, &s.pick)) return;
  double left = 0.0;
  for (int k = threadIdx.x; k < p.chunks; k += BLOCK) left += bins[k];
  left = block_sum_d(left, s.red);
  if (threadIdx.x == 0) s.st.left = left;
  go_on<T>(p, s, b, it);
}

template <typename T>
__global__ __launch_bounds__(BLOCK) void k_verify_end(VfDev p) {
  __shared__ VfShared s;
  const int b = blockIdx.x;
  if (p.state[b].done) return;
  load_state(p, s, b);
  const double it = inv_temp(p, b);
  double* bins = p.rest + (long long)b * p.chunks;
  // at most one round per node: each consumes a child
  while (!s.st.done) {
    for (int k = 0; k < p.chunks; ++k) {
      const double v = rest_chunk<T>(p, s, b, REST_Q, it, k);
      if (threadIdx.x == 0) bins[k] = v;
    }
    __threadfence_block();
    __syncthreads();
    double left = 0.0;
    for (int k = threadIdx.x; k < p.chunks; k += BLOCK) left += bins[k];
    left = block_sum_d(left, s.red);
    __syncthreads();
    if (threadIdx.x == 0) s.st.left = left;
    go_on<T>(p, s, b, it);
    __syncthreads();
  }
}

template <typename T>
pi_status launch_verify(pi_ctx* c, const VfDev& p) {
  PI_HIP(c, launch_k(c, 0, k_verify_rows<T>, dim3(p.chunks, p.N, p.B), 0, p));
  if (p.q == nullptr) return PI_OK;
  for (int i = 0; i < std::min(VF_RESTS, p.N - 1); ++i)
    PI_HIP(c, launch_k(c, 0, k_verify_rest<T>, dim3(p.chunks, p.B), 0, p));
  if (p.N - 1 > VF_RESTS) PI_HIP(c, launch_k(c, 0, k_verify_end<T>, dim3(p.B), 0, p));
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
               o_rest = o_state + sizeof(VfState) * max_batch, o_count = o_rest + sizeof(double) * max_batch * chunks,
               bytes = o_count + sizeof(uint32_t) * max_batch;
  PI_HIP(ctx, hipSetDevice(ctx->device));
  uint8_t* ws = nullptr;
  if (hipMalloc(reinterpret_cast<void**>(&ws), bytes) != hipSuccess) {
    (void)hipGetLastError();
    return fail(ctx, PI_ERR_OOM, "verifier scratch of %zu bytes", bytes);
  }
  if (hipMemset(ws + o_count, 0, bytes - o_count) != hipSuccess) {
    (void)hipFree(ws);
    return fail(ctx, PI_ERR_HIP, "clearing the verifier's counters failed");
  }
  pi_verifier* v = new (std::nothrow) pi_verifier{
      ctx, vocab, max_batch, max_nodes, chunks, ws, reinterpret_cast<VfPart*>(ws), reinterpret_cast<VfRow*>(ws + o_rows),
      reinterpret_cast<VfState*>(ws + o_state), reinterpret_cast<double*>(ws + o_rest),
      reinterpret_cast<uint32_t*>(ws + o_count)};
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
                ver->rest, ver->count};
  switch (a.dtype) {
    case PI_T_F32: return launch_verify<float>(ctx, p);
    case PI_T_F16: return launch_verify<half_t>(ctx, p);
    default: return launch_verify<bf16_t>(ctx, p);
  }
}

}  // extern "C"
