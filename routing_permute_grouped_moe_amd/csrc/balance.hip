// The router's auxiliary losses: balance (per sequence) and z, with per-expert
// counts, and their gradient together with the gates'.
//
//   balance = 1/N sum_s n_s sum_e f_se P_se = E / (k N) sum_s 1/n_s sum_e c_se Q_se,
//   with Q_se the sum of p_te over the tokens of s that count
//   dlogits = p (g - sum p g + 2 w_z dloss/N lse),  g = w_balance dloss/N f + dgate
//
// Forward: one pass over the logits.  Blocks of tokens leave, for each sequence
// that they meet, a row of partial sums (Q fp32, c int32, sum lse^2, n); what a
// sequence's rows add up to is summed in fp64 in the order of the blocks, so the
// bits are the same on every run.  Block b's row for sequence s is b + s: along
// the tokens b and s only grow and one of them grows from row to row, so the rows
// are distinct and at most blocks + S.  Few tokens are one block, which leaves
// the outputs themselves.
// Measured: 65521 tokens of 256 experts 21 us (67 MB, 3.2 TB/s; the pass over the
// logits 15, the sums 5.5), 8192 tokens in 13 sequences 13 us, 256 tokens of 8
// experts, in one launch, 5.3 us: trips to memory one after the other (a
// sequence's ends, the rows, the parts).
#include "reduce.hpp"
#include "validate.hpp"

namespace {

constexpr int BAL_NT = 1024;                  // forward
constexpr int BAL_WAVES = BAL_NT / MOE_WAVE;
constexpr int BAL_BWD_NT = 256;
// sequences from which on each is added by a wave, not a workgroup (8192 tokens of 256
// experts in 24 sequences: 17.2 and 14.3 us, in 64 17.8 and 17.5, in 1000 32 and 75; their
// lengths are not known to the host, and where one has nearly all tokens the workgroup wins:
// 8192 tokens behind 63 sequences of one 85 and 66 us, 65536 tokens 155 and 134, most of it
// the first block's 64 sequences one after the other)
constexpr int BAL_MANY = 64;
constexpr int BAL_MAX_S = 65535;              // sequences
// rounds of a block, at most: a lane adds that many probabilities in fp32, 18 more additions
// join lanes and waves, the rest is fp64 (2^26 tokens of 3 experts have 4608 blocks so; in 256
// their probabilities, added 4096 times, were off by 430 roundings)
constexpr int BAL_CHAIN = 240;
constexpr uint32_t BAL_OOB = 0xffffffffu;     // past every tensor: reads zeros

// Lanes of a token in the forward: a wave has one of many experts, or several of
// few, whose sums over lanes then cost as much as one's (65536 tokens of 64
// experts: 19.5 -> 13.1 us, 65521 of 256 22.3 -> 21.0; four of 256 a wave 21.6).
int bal_lanes(int E) { return E <= 64 ? 16 : E <= 256 ? 32 : 64; }
// Tokens of a block: 256 blocks, one for each CU, or as many times 256 as keep a block's
// rounds of its waves at BAL_CHAIN; few tokens in few sequences are one block.
bool bal_one(int T, int E, int S) { return T <= 4 * (BAL_NT / bal_lanes(E)) && S <= 16; }
int bal_block_tokens(int T, int E, int S) {
  if (bal_one(T, E, S)) return T > 0 ? T : 1;
  const int round = BAL_NT / bal_lanes(E);
  const long long per = ((long long)T + 255) / 256;
  const long long rounds = (per + round - 1) / round, times = (rounds + BAL_CHAIN - 1) / BAL_CHAIN;
  return times > 0 ? (int)((rounds + times - 1) / times) * round : round;
}
int bal_blocks(int T, int E, int S) {
  const int tb = bal_block_tokens(T, E, S);
  return T > 0 ? (int)(((long long)T + tb - 1) / tb) : 1;
}

struct BalWs {
  size_t q, c, z, n, term, total;
};
BalWs bal_ws(int T, int E, int S) {
  BalWs w = {};
  if (bal_one(T, E, S)) return w;
  const size_t rows = (size_t)bal_blocks(T, E, S) + S, cg = (E + MOE_WAVE - 1) / MOE_WAVE;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  w.q = 256;                                  // (in front: the count of workgroups that are done)
  w.c = w.q + up(rows * E * 4);
  w.z = w.c + up(rows * E * 4);
  w.n = w.z + up(rows * 8);
  w.term = w.n + up(rows * 4);
  w.total = w.term + up((size_t)S * (cg + 1) * 8);
  return w;
}

struct BalArgs {
  const float* logits; const int32_t* idx; const uint8_t* keep; const int32_t* seq;
  int T, E, k, S, tb, one;
  int* done; float* q; int32_t* c; double* z; int32_t* n; double* term;
  float w_balance, w_z;
  float* loss; int32_t* counts; int32_t* tokens; float* prob;
};

__device__ __forceinline__ int bal_seq(const int32_t* seq, int s, int T) {
  const int v = seq[s];
  return v < 0 ? 0 : v > T ? T : v;
}
// First sequence that ends behind token t (S if none does), by a whole wave: 64
// ends at a time cut the range to a 64th, so that 64 sequences take one trip to
// memory where halving takes six.
__device__ __forceinline__ int bal_first(const int32_t* seq, int S, int T, int t) {
  const int lane = threadIdx.x % MOE_WAVE;
  int lo = 0, len = S;                        // it is in [lo, lo + len]
  while (len > 0) {
    const int step = (len + MOE_WAVE - 1) / MOE_WAVE;
    const int at = lo + (lane + 1) * step - 1;   // the last of the lane's run
    const bool before = at < lo + len && bal_seq(seq, at + 1, T) <= t;
    const int runs = __popcll(__ballot(before));
    const int from = runs * step;             // runs that end before t are behind us
    lo += from;
    len = len - from < step - 1 ? len - from : step - 1;
  }
  return lo;
}

// A token's softmax over its lanes: v <- exp(v - max), m the maximum and s their
// sum (s = 0 where all logits are -inf; NaN where there is a NaN or +inf).
// FAST: the exponential by the hardware's exp2, off by 2.4 |x| + 2 roundings (expf
// and its range reduction are half of the forward's instructions, and the forward
// of many tokens is bound by them: 65521 tokens of 256 experts 24 us so, 18 with
// exp2); the backward keeps moe_route_bwd's expf and its bits.
template <int TPR, int V, bool FAST>
__device__ __forceinline__ void bal_softmax(float (&v)[V], int E, float& m, float& s) {
  const int lane = threadIdx.x % TPR;
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = lane + i * TPR < E ? v[i] : -INFINITY;
    m = fmaxf(m, v[i]);
  }
  m = lanes_max<TPR>(m);
  m = m == -INFINITY ? 0.f : m;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // (a lane without an expert holds -inf: 0, or NaN where the sum is one anyway)
    if constexpr (FAST) v[i] = __builtin_amdgcn_exp2f((v[i] - m) * 1.44269504f);
    else v[i] = lane + i * TPR < E ? expf(v[i] - m) : 0.f;
    s += v[i];
  }
  s = lanes_sum<TPR>(s);
}

template <int TPR, int V>
__global__ __launch_bounds__(BAL_NT) void balance_part_kernel(BalArgs a) {
  constexpr int PER = MOE_WAVE / TPR, ROUND = BAL_WAVES * PER;   // tokens of a wave, of all
  constexpr int U = V >= 8 ? 1 : 2;           // rounds in flight
  __shared__ float q_s[BAL_WAVES][V * TPR];
  __shared__ int c_s[V * TPR];
  __shared__ double z_s[BAL_WAVES];
  __shared__ int n_s[BAL_WAVES];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x % MOE_WAVE / TPR;
  const int wave = uniform((int)(threadIdx.x / MOE_WAVE));
  const int E = a.E, b = blockIdx.x;
  const int t0 = b * a.tb, t1 = a.T - t0 < a.tb ? a.T : t0 + a.tb;
  uint32_t off[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + i * TPR;
    off[i] = e < E ? ((uint32_t)sub * (uint32_t)E + e) * 4u : BAL_OOB;
  }
  const uint32_t ioff = lane < a.k ? ((uint32_t)sub * (uint32_t)a.k + lane) * 4u : BAL_OOB;
  if (b == 0 && threadIdx.x == 0 && !a.one) *a.done = 0;
  double all_b = 0, all_z = 0;                // (one block: the losses)
  int all_n = 0;
  int s = a.one || !a.seq ? 0 : uniform(bal_first(a.seq, a.S, a.T, t0));
  for (; s < a.S; ++s) {
    int lo = a.seq ? bal_seq(a.seq, s, a.T) : 0, hi = a.seq ? bal_seq(a.seq, s + 1, a.T) : a.T;
    if (lo >= t1 && !a.one) break;
    lo = lo < t0 ? t0 : lo;
    hi = hi > t1 ? t1 : hi;
    if (lo >= hi && !a.one) continue;
    for (int e = threadIdx.x; e < E; e += BAL_NT) c_s[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    double z = 0;
    int n = 0;
    for (int base = lo + wave * PER; base < hi; base += ROUND * U) {
      float v[U][V];
      int e0[U];
      bool use[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {           // rows tu .. tu + PER - 1, as far as there are
        const int tu = uniform(base + u * ROUND), left = hi - tu < PER ? hi - tu : PER;
        const uint32_t rows = left > 0 ? (uint32_t)left * 4u : 0u;
        const long long from = left > 0 ? tu : 0;
        const auto rl = make_rsrc(a.logits + from * E, rows * (uint32_t)E);
        const auto ri = make_rsrc(a.idx + from * a.k, rows * (uint32_t)a.k);
#pragma unroll
        for (int i = 0; i < V; ++i) v[u][i] = __uint_as_float(buf_load4(rl, off[i]));
        e0[u] = (int)buf_load4(ri, ioff);
        e0[u] = lane < a.k ? e0[u] : -1;
        use[u] = sub < left;
        if (a.keep && use[u]) use[u] = a.keep[tu + sub] != 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (base + u * ROUND >= hi) break;
        float m, sum;
        bal_softmax<TPR, V, true>(v[u], E, m, sum);
        use[u] = use[u] && !(sum == 0.f);
        if (use[u]) {
          // (the hardware's reciprocal and log2, each off by a rounding at most: sum is in
          // [1, E], where neither needs the range steps of a division and of logf)
          const float inv = __builtin_amdgcn_rcpf(sum);
          const float lse = fmaf(__builtin_amdgcn_logf(sum), 0.693147181f, m);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(v[u][i], inv, acc[i]);
          z += (double)lse * lse;
          ++n;
          if (e0[u] >= 0 && e0[u] < E) atomicAdd(&c_s[e0[u]], 1);
          const long long t = base + u * ROUND + sub;
          for (int j = lane + TPR; j < a.k; j += TPR) {
            const int e = a.idx[t * a.k + j];
            if (e >= 0 && e < E) atomicAdd(&c_s[e], 1);
          }
        }
      }
    }
    // the tokens of a wave, then the waves
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (TPR <= 32) acc[i] = add_swap32(acc[i]);
      if constexpr (TPR <= 16) acc[i] = add_swap16(acc[i]);
      q_s[wave][lane + i * TPR] = acc[i];
    }
    z = lanes_sum64(lane == 0 ? z : 0.0);
    n = lanes_sum_int(lane == 0 ? n : 0);
    if (threadIdx.x % MOE_WAVE == 0) { z_s[wave] = z; n_s[wave] = n; }
    __syncthreads();
    z = 0, n = 0;
#pragma unroll
    for (int w = 0; w < BAL_WAVES; ++w) { z += z_s[w]; n += n_s[w]; }
    const long long row = a.one ? s : b + s;
    double part = 0;
    for (int e = threadIdx.x; e < E; e += BAL_NT) {
      float q = 0.f;
#pragma unroll
      for (int w = 0; w < BAL_WAVES; ++w) q += q_s[w][e];
      const int c = c_s[e];
      if (a.one) {
        a.counts[row * E + e] = c;
        if (a.prob) a.prob[row * E + e] = n > 0 ? (float)((double)q / n) : 0.f;
        if (n > 0) part += (double)c * q / n;
      } else {
        a.q[row * E + e] = q;
        a.c[row * E + e] = c;
      }
    }
    if (a.one) {
      all_b += part;
      all_z += z;
      all_n += n;
      if (threadIdx.x == 0) a.tokens[s] = n;
    } else if (threadIdx.x == 0) {
      a.z[row] = z;
      a.n[row] = n;
    }
    __syncthreads();
  }
  if (!a.one) return;
  all_b = lanes_sum64(all_b);
  if (threadIdx.x % MOE_WAVE == 0) z_s[wave] = all_b;
  __syncthreads();
  if (threadIdx.x != 0) return;
  all_b = 0;
#pragma unroll
  for (int w = 0; w < BAL_WAVES; ++w) all_b += z_s[w];
  const double d = all_n > 0 ? all_n : 1;
  all_b *= a.E / (a.k * d);
  all_z /= d;
  a.loss[0] = (float)all_b;
  a.loss[1] = (float)all_z;
  a.loss[2] = (float)(a.w_balance * all_b + a.w_z * all_z);
  a.tokens[a.S] = all_n;
}

template <typename T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Rows of a sequence: counts, probabilities and its part of the losses, for 64
// experts by PER waves, each its share of the rows; 16 / PER sequences a workgroup.
// The workgroup that is done last adds the parts, in their order.
template <int PER>
__global__ __launch_bounds__(BAL_NT) void balance_sum_kernel(BalArgs a) {
  constexpr int SEQ = BAL_WAVES / PER;
  __shared__ double q_s[BAL_WAVES][MOE_WAVE], z_s[BAL_WAVES], b_s[BAL_WAVES];
  __shared__ int c_s[BAL_WAVES][MOE_WAVE];
  __shared__ long long n_s[BAL_WAVES];
  __shared__ int last;
  const int lane = threadIdx.x % MOE_WAVE, wave = uniform((int)(threadIdx.x / MOE_WAVE));
  const int s = blockIdx.y * SEQ + wave / PER, mine = wave % PER;
  const int E = a.E, e = blockIdx.x * MOE_WAVE + lane, cg = gridDim.x;
  int lo = 0, hi = s < a.S ? a.T : 0;
  if (a.seq && s < a.S) lo = bal_seq(a.seq, s, a.T), hi = bal_seq(a.seq, s + 1, a.T);
  const int b0 = lo / a.tb, b1 = lo < hi ? (hi - 1) / a.tb + 1 : b0;
  double q = 0, z = 0;
  int c = 0;
  long long n = 0;
  if (e < E)
#pragma unroll 4
    for (int b = b0 + mine; b < b1; b += PER) {
      const long long at = (long long)(b + s) * E + e;
      q += a.q[at];
      c += a.c[at];
    }
  for (int b = b0 + mine * MOE_WAVE + lane; b < b1; b += PER * MOE_WAVE) {
    z += a.z[b + s];
    n += a.n[b + s];
  }
  z = lanes_sum64(z);
  n = lanes_sum_int((int)n);
  if constexpr (PER > 1) {
    q_s[wave][lane] = q;
    c_s[wave][lane] = c;
    if (lane == 0) { z_s[wave] = z; n_s[wave] = n; }
    __syncthreads();
    q = 0, z = 0, c = 0, n = 0;
    if (mine == 0)
#pragma unroll
      for (int w = 0; w < PER; ++w) {
        q += q_s[wave + w][lane];
        c += c_s[wave + w][lane];
        z += z_s[wave + w];
        n += n_s[wave + w];
      }
  }
  if (mine == 0 && s < a.S) {
    if (e < E) {
      a.counts[(long long)s * E + e] = c;
      if (a.prob) a.prob[(long long)s * E + e] = n > 0 ? (float)(q / n) : 0.f;
    }
    const double part = lanes_sum64(e < E && n > 0 ? c * q / n : 0.0);
    if (lane == 0) {
      // written at device scope, past this XCD's L2, and complete before the count
      put(a.term + (long long)s * cg + blockIdx.x, part);
      if (blockIdx.x == 0) {
        put(a.term + (long long)a.S * cg + s, z);
        put(a.tokens + s, (int)n);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           (int)(gridDim.x * gridDim.y) - 1;
  __syncthreads();
  if (!last) return;
  double b = 0;
  z = 0, n = 0;
  for (long long i = threadIdx.x; i < (long long)a.S * cg; i += BAL_NT) b += get(a.term + i);
  for (int i = threadIdx.x; i < a.S; i += BAL_NT) {
    z += get(a.term + (long long)a.S * cg + i);
    n += get(a.tokens + i);
  }
  b = lanes_sum64(b);
  z = lanes_sum64(z);
  n = lanes_sum_int((int)n);
  if (lane == 0) { b_s[wave] = b; z_s[wave] = z; n_s[wave] = n; }
  __syncthreads();
  if (threadIdx.x != 0) return;
  b = 0, z = 0, n = 0;
#pragma unroll
  for (int w = 0; w < BAL_WAVES; ++w) { b += b_s[w]; z += z_s[w]; n += n_s[w]; }
  const double d = n > 0 ? (double)n : 1.0;
  b *= a.E / (a.k * d);
  z /= d;
  a.loss[0] = (float)b;
  a.loss[1] = (float)z;
  a.loss[2] = (float)(a.w_balance * b + a.w_z * z);
  a.tokens[a.S] = (int)n;
}

struct BalBwd {
  const float* logits; const int32_t* idx; const float* dgate; const uint8_t* keep;
  const int32_t* seq; const int32_t* counts; const int32_t* tokens; const float* dloss;
  int T, E, k, S;
  float w_balance, w_z;
  float* dlogits;
};

// Bound by the row's trip to memory at few tokens, by memory at many.  A wave has
// one token of many experts or several of few (four tokens a wave in
// turn, all their rows in flight, end later: 8192 tokens of 256 experts 10.5 us,
// so 7.6; 65521 tokens 38.2 and 39.3).  Streaming stores: 7.5 -> 6.7 us at 8192
// tokens, 38.5 -> 34.7 at 65521 (3.9 TB/s).
template <int TPR, int V>
__global__ __launch_bounds__(BAL_BWD_NT) void balance_bwd_kernel(BalBwd a) {
  constexpr int PER = MOE_WAVE / TPR, WAVES = BAL_BWD_NT / MOE_WAVE;
  __shared__ float dp_s[WAVES][PER][V * TPR];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x % MOE_WAVE / TPR, E = a.E;
  const int wave = uniform((int)(threadIdx.x / MOE_WAVE));
  const int t0 = (blockIdx.x * WAVES + wave) * PER, t = t0 + sub;
  if (t0 >= a.T) return;                      // whole waves; no block barrier below
  // the wave's rows, as far as there are
  const uint32_t bytes = (uint32_t)(a.T - t0 < PER ? a.T - t0 : PER) * (uint32_t)E * 4u;
  const auto rl = make_rsrc(a.logits + (long long)t0 * E, bytes);
  const auto rd = make_rsrc(a.dlogits + (long long)t0 * E, bytes);
  uint32_t off[V];
  float v[V], g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + i * TPR;
    off[i] = e < E ? ((uint32_t)sub * (uint32_t)E + e) * 4u : BAL_OOB;
    v[i] = __uint_as_float(buf_load4(rl, off[i]));
  }
  const bool pair = a.dgate && t < a.T && lane < a.k;
  const int e0 = pair ? a.idx[(long long)t * a.k + lane] : -1;
  const float d0 = pair ? a.dgate[(long long)t * a.k + lane] : 0.f;
  bool counts = t < a.T && !(a.keep && a.keep[t] == 0);
  int s = 0;
  if (a.seq) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int of = bal_first(a.seq, a.S, a.T, t0 + j);
      s = sub == j ? of : s;
    }
    counts = counts && s < a.S && bal_seq(a.seq, s, a.T) <= t;
    s = s < a.S ? s : 0;
  }
  const int N = a.tokens[a.S], n = a.tokens[s];
  const float per = (a.dloss ? a.dloss[0] : 1.f) / (float)(N > 0 ? N : 1);
  const float fs = a.w_balance * per * ((float)E / ((float)a.k * (float)(n > 0 ? n : 1)));
  if constexpr (TPR == MOE_WAVE) {            // (the sequence's row is the wave's)
    const auto rc = make_rsrc(a.counts + (long long)uniform(s) * E, (uint32_t)E * 4u);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = counts ? fs * (float)(int)buf_load4(rc, off[i]) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      g[i] = counts && off[i] != BAL_OOB ? fs * (float)a.counts[(long long)s * E + lane + i * TPR]
                                         : 0.f;
  }
  if (a.dgate) {
    float* const dp = dp_s[wave][sub];
#pragma unroll
    for (int i = 0; i < V; ++i) dp[lane + i * TPR] = 0.f;
    wave_lds_sync();
    // chosen experts of a token are distinct, so these writes never collide
    if (e0 >= 0 && e0 < E) dp[e0] = d0;
    for (int j = lane + TPR; j < a.k && t < a.T; j += TPR) {
      const int e = a.idx[(long long)t * a.k + j];
      if (e >= 0 && e < E) dp[e] = a.dgate[(long long)t * a.k + j];
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] += dp[lane + i * TPR];
  }
  float m, sum, acc = 0.f, zs = 0.f;
  bal_softmax<TPR, V, false>(v, E, m, sum);
  const bool some = !(sum == 0.f);
  const float inv = some ? 1.0f / sum : 0.f;
  if (a.w_z != 0.f && some && counts) zs = 2.f * a.w_z * per * (m + logf(sum));
#pragma unroll
  for (int i = 0; i < V; ++i) acc += v[i] * inv * g[i];
  acc = lanes_sum<TPR>(acc);
  // a token that does not count and has no gates' gradient has zeros: its logits may be
  // NaN or infinite, and 0 times its probabilities is NaN then
  uint32_t some_g = counts;
#pragma unroll
  for (int i = 0; i < V; ++i) some_g |= __float_as_uint(g[i]) << 1;
  const unsigned long long lanes = ~0ull >> (MOE_WAVE - TPR) << sub * TPR;
  const bool none = (__ballot(some_g != 0) & lanes) == 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
    buf_store4_nt(rd, off[i], none ? 0u : __float_as_uint(v[i] * inv * (g[i] - acc + zs)));
}

template <int TPR, int V>
void launch_part(const BalArgs& a, int blocks, hipStream_t s) {
  hipLaunchKernelGGL((balance_part_kernel<TPR, V>), dim3(blocks), dim3(BAL_NT), 0, s, a);
}
template <int TPR, int V>
void launch_bwd(const BalBwd& a, hipStream_t s) {
  constexpr int G = BAL_BWD_NT / TPR;
  hipLaunchKernelGGL((balance_bwd_kernel<TPR, V>), dim3((a.T + G - 1) / G), dim3(BAL_BWD_NT), 0, s,
                     a);
}

int bal_checks(const char* fn, int T, int E, int k, int S) {
  MOE_TRY(moe_need_nonneg(T, fn, "T"));
  MOE_TRY(moe_need_ek(E, k, fn));
  if (S < 1) return moe_fail(MOE_ERR_INVALID_ARG, "%s: S = %d sequences", fn, S);
  if (S > BAL_MAX_S)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: S = %d above %d", fn, S, BAL_MAX_S);
  MOE_TRY(moe_need_elems(T, E, 4, fn, "logits"));
  // (and rows of partial sums where blocks are 256; where they are more T is in the millions)
  MOE_TRY(moe_need_elems((long long)S + 256, E, 4, fn, "counts"));
  return MOE_OK;
}

// Forward and backward take the same tokens.  The backward's launch has 16 lanes or more for
// each and ends at 2^32 of them, so below 2^28; 2^27 is half of that.
int bal_need_tokens(const char* fn, int T) {
  if (T < 1 << 27) return MOE_OK;
  return moe_fail(MOE_ERR_UNSUPPORTED, "%s: T = %d, above the limit", fn, T);
}

}  // namespace

extern "C" size_t moe_balance_loss_workspace_bytes(int T, int E, int k, int S) {
  if (bal_checks("moe_balance_loss_workspace_bytes", T, E, k, S) != MOE_OK) return 0;
  return bal_ws(T, E, S).total;
}

extern "C" int moe_balance_loss(const float* logits, const int32_t* idx, const uint8_t* keep,
                                const int32_t* seq, int T, int E, int k, int S, float w_balance,
                                float w_z, float* loss, int32_t* counts, int32_t* tokens,
                                float* prob, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* fn = "moe_balance_loss";
  MOE_TRY(bal_checks(fn, T, E, k, S));
  MOE_TRY(bal_need_tokens(fn, T));
  if (T > 0) {
    MOE_TRY(moe_need_ptr(logits, fn, "logits", 4));
    MOE_TRY(moe_need_ptr(idx, fn, "idx", 4));
  }
  if (seq == nullptr && S != 1)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: %d sequences without seq", fn, S);
  MOE_TRY(moe_opt_ptr(seq, fn, "seq", 4));
  MOE_TRY(moe_need_ptr(loss, fn, "loss", 4));
  MOE_TRY(moe_need_ptr(counts, fn, "counts", 4));
  MOE_TRY(moe_need_ptr(tokens, fn, "tokens", 4));
  MOE_TRY(moe_opt_ptr(prob, fn, "prob", 4));
  const BalWs lay = bal_ws(T, E, S);
  if (lay.total > 0) MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  if (ws_bytes < lay.total)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                    lay.total);
  const MoeRange in[] = {{logits, 4LL * T * E, "logits"}, {idx, 4LL * T * k, "idx"},
                         {keep, T, "keep"}, {seq, 4LL * (S + 1), "seq"}},
                 outs[] = {{loss, 12, "loss"}, {counts, 4LL * S * E, "counts"},
                           {tokens, 4LL * (S + 1), "tokens"}, {prob, 4LL * S * E, "prob"},
                           {lay.total > 0 ? ws : nullptr, (long long)lay.total, "ws"}};
  for (int i = 0; i < 5; ++i) {
    const char* with = moe_shares(outs[i], {in[0], in[1], in[2], in[3]});
    for (int j = 0; j < i && with == nullptr; ++j) with = moe_shares(outs[i], {outs[j]});
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: %s needs a buffer of its own, it overlaps %s", fn,
                      outs[i].name, with);
  }
  char* const w = (char*)ws;
  const bool one = bal_one(T, E, S);
  BalArgs a = {logits, idx, keep, seq, T, E, k, S, bal_block_tokens(T, E, S), one, (int*)w,
               (float*)(w + lay.q), (int32_t*)(w + lay.c), (double*)(w + lay.z),
               (int32_t*)(w + lay.n), (double*)(w + lay.term), w_balance, w_z,
               loss, counts, tokens, prob};
  hipStream_t s = (hipStream_t)stream;
  const int blocks = bal_blocks(T, E, S);
  if (E <= 16) launch_part<16, 1>(a, blocks, s);
  else if (E <= 32) launch_part<16, 2>(a, blocks, s);
  else if (E <= 64) launch_part<16, 4>(a, blocks, s);
  else if (E <= 128) launch_part<32, 4>(a, blocks, s);
  else if (E <= 256) launch_part<32, 8>(a, blocks, s);
  else if (E <= 512) launch_part<64, 8>(a, blocks, s);
  else launch_part<64, 16>(a, blocks, s);
  MOE_TRY(moe_check_launch(fn));
  if (one) return MOE_OK;
  // (of many sequences each has few rows, where all of them are 256 and one a sequence)
  const int cg = (E + MOE_WAVE - 1) / MOE_WAVE;
  if (S < BAL_MANY || (blocks > 256 && S < blocks))
    hipLaunchKernelGGL(balance_sum_kernel<BAL_WAVES>, dim3(cg, S), dim3(BAL_NT), 0, s, a);
  else
    hipLaunchKernelGGL(balance_sum_kernel<1>, dim3(cg, (S + BAL_WAVES - 1) / BAL_WAVES),
                       dim3(BAL_NT), 0, s, a);
  return moe_check_launch(fn);
}

extern "C" int moe_balance_loss_bwd(const float* logits, const int32_t* idx, const float* dgate,
                                    const uint8_t* keep, const int32_t* seq,
                                    const int32_t* counts, const int32_t* tokens, int T, int E,
                                    int k, int S, float w_balance, float w_z, const float* dloss,
                                    float* dlogits, moe_stream_t stream) {
  const char* fn = "moe_balance_loss_bwd";
  MOE_TRY(bal_checks(fn, T, E, k, S));
  MOE_TRY(bal_need_tokens(fn, T));
  if (T == 0) return MOE_OK;
  MOE_TRY(moe_need_ptr(logits, fn, "logits", 4));
  if (dgate != nullptr) MOE_TRY(moe_need_ptr(idx, fn, "idx", 4));
  MOE_TRY(moe_opt_ptr(dgate, fn, "dgate", 4));
  if (seq == nullptr && S != 1)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: %d sequences without seq", fn, S);
  MOE_TRY(moe_opt_ptr(seq, fn, "seq", 4));
  MOE_TRY(moe_need_ptr(counts, fn, "counts", 4));
  MOE_TRY(moe_need_ptr(tokens, fn, "tokens", 4));
  MOE_TRY(moe_opt_ptr(dloss, fn, "dloss", 4));
  MOE_TRY(moe_need_ptr(dlogits, fn, "dlogits", 4));
  const char* with =
      moe_shares({dlogits, 4LL * T * E, "dlogits"},
                 {{logits, 4LL * T * E, "logits"},
                  {dgate ? idx : nullptr, 4LL * T * k, "idx"},
                  {dgate, 4LL * T * k, "dgate"},
                  {keep, T, "keep"},
                  {seq, 4LL * (S + 1), "seq"},
                  {counts, 4LL * S * E, "counts"},
                  {tokens, 4LL * (S + 1), "tokens"},
                  {dloss, 4, "dloss"}});
  if (with != nullptr)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: dlogits needs a buffer of its own, it overlaps %s",
                    fn, with);
  BalBwd a = {logits, idx, dgate, keep, seq, counts, tokens, dloss, T, E, k, S,
              w_balance, w_z, dlogits};
  hipStream_t s = (hipStream_t)stream;
  // (lanes and values of a lane as moe_route_bwd has them, for its sums' bits)
  if (E <= 16) launch_bwd<16, 1>(a, s);
  else if (E <= 32) launch_bwd<32, 1>(a, s);
  else if (E <= 64) launch_bwd<64, 1>(a, s);
  else if (E <= 128) launch_bwd<64, 2>(a, s);
  else if (E <= 256) launch_bwd<64, 4>(a, s);
  else if (E <= 512) launch_bwd<64, 8>(a, s);
  else launch_bwd<64, 16>(a, s);
  return moe_check_launch(fn);
}
