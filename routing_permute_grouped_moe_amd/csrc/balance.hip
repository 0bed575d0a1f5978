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
// are distinct and at most blocks + S.
#include "validate.hpp"

namespace {

constexpr int BAL_WAVES = 4;
constexpr int BAL_NT = BAL_WAVES * MOE_WAVE;
constexpr int BAL_MAX_S = 65535;              // sequences: a grid's second dimension

int bal_block_tokens(int T) {
  const int most = 512;                       // blocks
  int tb = BAL_WAVES;
  while (((long long)T + tb - 1) / tb > most) tb *= 2;
  return tb;
}
int bal_blocks(int T) {
  const int tb = bal_block_tokens(T);
  return (int)(((long long)T + tb - 1) / tb);
}
int bal_width(int E) {
  int v = 1;
  while (v * MOE_WAVE < E) v *= 2;
  return v;
}

struct BalWs {
  size_t q, c, z, n, term, total;
};
BalWs bal_ws(int T, int E, int S) {
  const size_t rows = (size_t)bal_blocks(T) + S, cg = (E + MOE_WAVE - 1) / MOE_WAVE;
  BalWs w;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  w.q = 0;
  w.c = up(rows * E * 4);
  w.z = w.c + up(rows * E * 4);
  w.n = w.z + up(rows * 8);
  w.term = w.n + up(rows * 4);
  w.total = w.term + up((size_t)S * (cg + 1) * 8);
  return w;
}

struct BalArgs {
  const float* logits; const int32_t* idx; const uint8_t* keep; const int32_t* seq;
  int T, E, k, S, tb;
  float* q; int32_t* c; double* z; int32_t* n; double* term;
  float w_balance, w_z;
  float* loss; int32_t* counts; int32_t* tokens; float* prob;
};

__device__ __forceinline__ int bal_seq(const int32_t* seq, int s, int T) {
  const int v = seq[s];
  return v < 0 ? 0 : v > T ? T : v;
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, MOE_WAVE);
  return v;
}

// First sequence that ends behind token t (S if none does).
__device__ __forceinline__ int bal_first(const int32_t* seq, int S, int T, int t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (bal_seq(seq, mid + 1, T) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// One row's softmax: v <- exp(v - max), its sum's reciprocal (0 for a row of -inf
// alone) and the log of the sum; whether one logit is not -inf.
template <int V>
__device__ __forceinline__ bool bal_softmax(const float* row, int E, float (&v)[V], float& inv,
                                            float& lse) {
  const int lane = threadIdx.x % MOE_WAVE;
  float m = -INFINITY;
  bool some = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + i * MOE_WAVE;
    v[i] = e < E ? row[e] : -INFINITY;
    some |= !(v[i] == -INFINITY);     // (a NaN is one)
    m = fmaxf(m, v[i]);
  }
  some = __ballot(some) != 0;
  m = some ? wave_max(m) : 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = lane + i * MOE_WAVE < E ? expf(v[i] - m) : 0.f;
    s += v[i];
  }
  s = wave_sum(s);
  inv = some ? 1.0f / s : 0.f;
  lse = m + logf(s);
  return some;
}

template <int V>
__global__ __launch_bounds__(BAL_NT) void balance_part_kernel(BalArgs a) {
  __shared__ float q_s[BAL_WAVES][V * MOE_WAVE];
  __shared__ int c_s[V * MOE_WAVE];
  __shared__ double z_s[BAL_WAVES];
  __shared__ int n_s[BAL_WAVES];
  const int lane = threadIdx.x % MOE_WAVE, wave = threadIdx.x / MOE_WAVE;
  const int E = a.E, b = blockIdx.x;
  const int t0 = b * a.tb, t1 = a.T - t0 < a.tb ? a.T : t0 + a.tb;
  int s = a.seq ? bal_first(a.seq, a.S, a.T, t0) : 0;
  for (; s < a.S; ++s) {
    int lo = a.seq ? bal_seq(a.seq, s, a.T) : 0, hi = a.seq ? bal_seq(a.seq, s + 1, a.T) : a.T;
    if (lo >= t1) break;
    lo = lo < t0 ? t0 : lo;
    hi = hi > t1 ? t1 : hi;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < E; e += BAL_NT) c_s[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    double z = 0;
    int n = 0;
    for (int t = lo + wave; t < hi; t += BAL_WAVES) {
      if (a.keep && a.keep[t] == 0) continue;
      float v[V], inv, lse;
      if (!bal_softmax<V>(a.logits + (long long)t * E, E, v, inv, lse)) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += v[i] * inv;
      z += (double)lse * lse;
      ++n;
      for (int j = lane; j < a.k; j += MOE_WAVE) {
        const int e = a.idx[(long long)t * a.k + j];
        if (e >= 0 && e < E) atomicAdd(&c_s[e], 1);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) q_s[wave][lane + i * MOE_WAVE] = acc[i];
    if (lane == 0) { z_s[wave] = z; n_s[wave] = n; }
    __syncthreads();
    const long long row = b + s;
    for (int e = threadIdx.x; e < E; e += BAL_NT) {
      float q = 0.f;
#pragma unroll
      for (int w = 0; w < BAL_WAVES; ++w) q += q_s[w][e];
      a.q[row * E + e] = q;
      a.c[row * E + e] = c_s[e];
    }
    if (threadIdx.x == 0) {
      double zz = 0;
      int nn = 0;
#pragma unroll
      for (int w = 0; w < BAL_WAVES; ++w) { zz += z_s[w]; nn += n_s[w]; }
      a.z[row] = zz;
      a.n[row] = nn;
    }
    __syncthreads();
  }
}

// Rows of a sequence: counts, probabilities and its part of the losses, 64
// experts a workgroup, a quarter of the rows a wave.
__global__ __launch_bounds__(BAL_NT) void balance_sum_kernel(BalArgs a) {
  __shared__ double q_s[BAL_WAVES][MOE_WAVE], z_s[BAL_WAVES];
  __shared__ int c_s[BAL_WAVES][MOE_WAVE], n_s[BAL_WAVES];
  const int lane = threadIdx.x % MOE_WAVE, wave = threadIdx.x / MOE_WAVE;
  const int s = blockIdx.y, E = a.E, e = blockIdx.x * MOE_WAVE + lane;
  const int lo = a.seq ? bal_seq(a.seq, s, a.T) : 0, hi = a.seq ? bal_seq(a.seq, s + 1, a.T) : a.T;
  const int b0 = lo / a.tb, b1 = lo < hi ? (hi - 1) / a.tb + 1 : b0;
  double q = 0, z = 0;
  int c = 0, n = 0;
  for (int b = b0 + wave; b < b1; b += BAL_WAVES) {
    const long long row = b + s;
    if (e < E) {
      q += a.q[row * E + e];
      c += a.c[row * E + e];
    }
  }
  for (int b = b0 + threadIdx.x; b < b1; b += BAL_NT) {
    z += a.z[b + s];
    n += a.n[b + s];
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, MOE_WAVE);
  z = wave_sum64(z);
  q_s[wave][lane] = q;
  c_s[wave][lane] = c;
  if (lane == 0) { z_s[wave] = z; n_s[wave] = n; }
  __syncthreads();
  if (wave != 0) return;
  q = 0, z = 0, c = 0, n = 0;
#pragma unroll
  for (int w = 0; w < BAL_WAVES; ++w) {
    q += q_s[w][lane];
    c += c_s[w][lane];
    z += z_s[w];
    n += n_s[w];
  }
  if (e < E) {
    a.counts[(long long)s * E + e] = c;
    if (a.prob) a.prob[(long long)s * E + e] = n > 0 ? (float)(q / n) : 0.f;
  }
  const double part = wave_sum64(e < E && n > 0 ? c * q / n : 0.0);
  if (lane == 0) {
    a.term[(long long)s * gridDim.x + blockIdx.x] = part;
    if (blockIdx.x == 0) {
      a.term[(long long)a.S * gridDim.x + s] = z;
      a.tokens[s] = n;
    }
  }
}

__global__ __launch_bounds__(BAL_NT) void balance_loss_kernel(BalArgs a, int cg) {
  __shared__ double b_s[BAL_WAVES], z_s[BAL_WAVES];
  __shared__ long long n_s[BAL_WAVES];
  const int lane = threadIdx.x % MOE_WAVE, wave = threadIdx.x / MOE_WAVE;
  double b = 0, z = 0;
  long long n = 0;
  for (long long i = threadIdx.x; i < (long long)a.S * cg; i += BAL_NT) b += a.term[i];
  for (int s = threadIdx.x; s < a.S; s += BAL_NT) {
    z += a.term[(long long)a.S * cg + s];
    n += a.tokens[s];
  }
  b = wave_sum64(b);
  z = wave_sum64(z);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, MOE_WAVE);
  if (lane == 0) { b_s[wave] = b; z_s[wave] = z; n_s[wave] = n; }
  __syncthreads();
  if (threadIdx.x != 0) return;
  b = 0, z = 0, n = 0;
#pragma unroll
  for (int w = 0; w < BAL_WAVES; ++w) { b += b_s[w]; z += z_s[w]; n += n_s[w]; }
  const double d = n > 0 ? (double)n : 1.0;
  b = b * a.E / (a.k * d);
  z = z / d;
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

template <int V>
__global__ __launch_bounds__(BAL_NT) void balance_bwd_kernel(BalBwd a) {
  __shared__ float dp_s[BAL_WAVES][V * MOE_WAVE];
  const int lane = threadIdx.x % MOE_WAVE, wave = threadIdx.x / MOE_WAVE, E = a.E;
  const int t = blockIdx.x * BAL_WAVES + wave;
  if (t >= a.T) return;  // whole wave leaves together; no block barrier below
  float* dp = dp_s[wave];
  if (a.dgate) {
#pragma unroll
    for (int i = 0; i < V; ++i) dp[lane + i * MOE_WAVE] = 0.f;
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_wave_barrier();
    // chosen experts of a token are distinct, so these writes never collide
    for (int j = lane; j < a.k; j += MOE_WAVE) {
      const int e = a.idx[(long long)t * a.k + j];
      if (e >= 0 && e < E) dp[e] = a.dgate[(long long)t * a.k + j];
    }
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_wave_barrier();
  }
  float v[V], inv, lse;
  bool counts = bal_softmax<V>(a.logits + (long long)t * E, E, v, inv, lse);
  if (a.keep && a.keep[t] == 0) counts = false;
  int s = 0;
  if (a.seq) {
    s = bal_first(a.seq, a.S, a.T, t);
    counts = counts && s < a.S && bal_seq(a.seq, s, a.T) <= t;
  }
  float fs = 0.f, zs = 0.f;
  if (counts) {
    const float dl = a.dloss ? a.dloss[0] : 1.f;
    const int N = a.tokens[a.S], n = a.tokens[s];
    const float per = dl / (float)(N > 0 ? N : 1);
    fs = a.w_balance * per * ((float)E / ((float)a.k * (float)(n > 0 ? n : 1)));
    zs = 2.f * a.w_z * per * lse;
  }
  const int32_t* c = a.counts + (long long)(counts ? s : 0) * E;
  float g[V], acc = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + i * MOE_WAVE;
    g[i] = counts && e < E ? fs * (float)c[e] : 0.f;
    if (a.dgate) g[i] += dp[e];
    acc += v[i] * inv * g[i];
  }
  acc = wave_sum(acc);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + i * MOE_WAVE;
    if (e < E) a.dlogits[(long long)t * E + e] = v[i] * inv * (g[i] - acc + zs);
  }
}

template <int V>
void launch_part(const BalArgs& a, int blocks, hipStream_t s) {
  hipLaunchKernelGGL(balance_part_kernel<V>, dim3(blocks), dim3(BAL_NT), 0, s, a);
}
template <int V>
void launch_bwd(const BalBwd& a, hipStream_t s) {
  hipLaunchKernelGGL(balance_bwd_kernel<V>, dim3((a.T + BAL_WAVES - 1) / BAL_WAVES), dim3(BAL_NT),
                     0, s, a);
}

int bal_checks(const char* fn, int T, int E, int k, int S) {
  MOE_TRY(moe_need_nonneg(T, fn, "T"));
  MOE_TRY(moe_need_ek(E, k, fn));
  if (S < 1) return moe_fail(MOE_ERR_INVALID_ARG, "%s: S = %d sequences", fn, S);
  if (S > BAL_MAX_S)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: S = %d above %d", fn, S, BAL_MAX_S);
  MOE_TRY(moe_need_elems(T, E, 4, fn, "logits"));
  // (rows of partial sums: at most 512 and one a sequence)
  MOE_TRY(moe_need_elems((long long)S + 512, E, 4, fn, "counts"));
  return MOE_OK;
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
  MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  const BalWs lay = bal_ws(T, E, S);
  if (ws_bytes < lay.total)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                    lay.total);
  const MoeRange in[] = {{logits, 4LL * T * E, "logits"}, {idx, 4LL * T * k, "idx"},
                         {keep, T, "keep"}, {seq, 4LL * (S + 1), "seq"}},
                 outs[] = {{loss, 12, "loss"}, {counts, 4LL * S * E, "counts"},
                           {tokens, 4LL * (S + 1), "tokens"}, {prob, 4LL * S * E, "prob"},
                           {ws, (long long)lay.total, "ws"}};
  for (int i = 0; i < 5; ++i) {
    const char* with = moe_shares(outs[i], {in[0], in[1], in[2], in[3]});
    for (int j = 0; j < i && with == nullptr; ++j) with = moe_shares(outs[i], {outs[j]});
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: %s needs a buffer of its own, it overlaps %s", fn,
                      outs[i].name, with);
  }
  char* const w = (char*)ws;
  BalArgs a = {logits, idx, keep, seq, T, E, k, S, bal_block_tokens(T),
               (float*)(w + lay.q), (int32_t*)(w + lay.c), (double*)(w + lay.z),
               (int32_t*)(w + lay.n), (double*)(w + lay.term), w_balance, w_z,
               loss, counts, tokens, prob};
  hipStream_t s = (hipStream_t)stream;
  const int blocks = bal_blocks(T);
  if (blocks > 0) {
    switch (bal_width(E)) {
      case 1: launch_part<1>(a, blocks, s); break;
      case 2: launch_part<2>(a, blocks, s); break;
      case 4: launch_part<4>(a, blocks, s); break;
      case 8: launch_part<8>(a, blocks, s); break;
      default: launch_part<16>(a, blocks, s); break;
    }
    MOE_TRY(moe_check_launch(fn));
  }
  const int cg = (E + MOE_WAVE - 1) / MOE_WAVE;
  hipLaunchKernelGGL(balance_sum_kernel, dim3(cg, S), dim3(BAL_NT), 0, s, a);
  MOE_TRY(moe_check_launch(fn));
  hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(BAL_NT), 0, s, a, cg);
  return moe_check_launch(fn);
}

extern "C" int moe_balance_loss_bwd(const float* logits, const int32_t* idx, const float* dgate,
                                    const uint8_t* keep, const int32_t* seq,
                                    const int32_t* counts, const int32_t* tokens, int T, int E,
                                    int k, int S, float w_balance, float w_z, const float* dloss,
                                    float* dlogits, moe_stream_t stream) {
  const char* fn = "moe_balance_loss_bwd";
  MOE_TRY(bal_checks(fn, T, E, k, S));
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
  switch (bal_width(E)) {
    case 1: launch_bwd<1>(a, s); break;
    case 2: launch_bwd<2>(a, s); break;
    case 4: launch_bwd<4>(a, s); break;
    case 8: launch_bwd<8>(a, s); break;
    default: launch_bwd<16>(a, s); break;
  }
  return moe_check_launch(fn);
}
