// Layer norm and RMS norm of rows, with the residual sum in front, and their
// gradients:
//   h = x + residual,  q = (h - m) rstd,  y = q w + bias
//   g = dy w,  dx = rstd (g - mean(g) - q mean(g q)) + dh,  dw = sum dy q,  db = sum dy
//
// Bound by HBM: every row is read once and stays in registers between its sums,
// as 16-byte chunks of the storage type; the weight stays in registers from row
// to row, and the next row is on its way while this one's sums are made.  The
// backward keeps a column's part of dw and db in registers too; each workgroup
// leaves one row of them, and a second launch adds those rows in fp64, in order.
// Measured among calls back to back (one MI355X, where a 1 GiB copy moves 5.1 TB/s):
// 8192 x 7680 bf16 with a residual 85 us (5.9 TB/s), its backward 91 us (5.5 TB/s; 5 us
// of it the second launch); backwards of 4095 x 2048 fp32 and of 131071 x 128 bf16,
// 100 MB each, 20.0 and 20.7 us; one row of 7680 3 us.  (Times beside the choices below
// are of the step that made them.)
#include "reduce.hpp"
#include "validate.hpp"

namespace {

constexpr int NORM_MAX_H = 16384;
constexpr uint32_t NORM_OOB = 0x80000000u;   // past every row: reads zeros, stores are dropped

// TPR threads hold a row, C chunks of 16 bytes each; rows of less than a
// workgroup share one.  PRE: registers suffice for the next row and the weight.
template <typename T, int TPR, int C, int THREADS>
struct Rows {
  static constexpr int VEC = Elem<T>::VEC;
  static constexpr int NT = THREADS;
  static constexpr int G = NT / TPR;         // rows at a time
  static constexpr int WAVES = NT / MOE_WAVE;
  static constexpr bool PRE = !(TPR == 1024 && C * VEC >= 16);
};

// The sums of two values over the threads of a row, in all of them; `turn` flips
// from call to call, so that one barrier a call is enough.
template <int TPR, int WAVES>
__device__ __forceinline__ void row_sums(float& a, float& b, float2 (*red)[WAVES], int& turn) {
  constexpr int N = TPR < MOE_WAVE ? TPR : MOE_WAVE;
  a = lanes_sum<N>(a);
  b = lanes_sum<N>(b);
  if constexpr (TPR > MOE_WAVE) {
    const int wave = threadIdx.x / MOE_WAVE, first = wave / (TPR / MOE_WAVE) * (TPR / MOE_WAVE);
    if ((threadIdx.x & 63) == 0) red[turn][wave] = float2{a, b};
    __syncthreads();
    a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / MOE_WAVE; ++w) {
      a += red[turn][first + w].x;
      b += red[turn][first + w].y;
    }
    turn ^= 1;
  }
}
template <int TPR, int WAVES>
__device__ __forceinline__ float row_sum(float a, float2 (*red)[WAVES], int& turn) {
  constexpr int N = TPR < MOE_WAVE ? TPR : MOE_WAVE;
  a = lanes_sum<N>(a);
  if constexpr (TPR > MOE_WAVE) {
    const int wave = threadIdx.x / MOE_WAVE, first = wave / (TPR / MOE_WAVE) * (TPR / MOE_WAVE);
    if ((threadIdx.x & 63) == 0) red[turn][wave].x = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / MOE_WAVE; ++w) a += red[turn][first + w].x;
    turn ^= 1;
  }
  return a;
}

template <bool STREAM>
__device__ __forceinline__ u32x4 row_load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return STREAM ? buf_load16_nt(r, off) : buf_load16(r, off);
}

struct NormArgs {
  const void* x; const void* residual; const float* w; const float* bias;
  void* h; void* y; float* mean; float* rstd;
  int M, H, rms;
  float eps, inv_h;
};

template <typename T, int TPR, int C, int NT_, bool STREAM>
__global__ __launch_bounds__(NT_) void norm_kernel(NormArgs a) {
  using R = Rows<T, TPR, C, NT_>;
  constexpr int VEC = R::VEC, ES = sizeof(T);
  __shared__ float2 red[2][R::WAVES];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int n = a.H / VEC;                   // chunks of a row
  const uint32_t rb = (uint32_t)a.H * ES;
  uint32_t off[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = lane + i * TPR;
    off[i] = c < n ? (uint32_t)grp * rb + (uint32_t)c * 16u : NORM_OOB;
  }
  float w[C][VEC], b[C][VEC];
  const auto rw = make_rsrc(a.w, (uint32_t)a.H * 4u);
  const auto rbias = make_rsrc(a.bias, a.bias ? (uint32_t)a.H * 4u : 0u);
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      const uint32_t o = ((uint32_t)(lane + i * TPR) * VEC + j) * 4u;
      unpack16(buf_load16(rw, o), &w[i][j], float());
      unpack16(buf_load16(rbias, o), &b[i][j], float());
    }
  auto rows = [&](const void* p, int r0) {   // the rows from r0 on (no memory: none)
    const int m = r0 < a.M && p != nullptr ? (a.M - r0 < R::G ? a.M - r0 : R::G) : 0;
    return make_rsrc((const char*)p + (m ? (long long)r0 * rb : 0), (uint32_t)m * rb);
  };
  u32x4 x[C], res[C];
  auto fetch = [&](int r0) {
    const auto rx = rows(a.x, r0), rr = rows(a.residual, r0);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      x[i] = row_load<STREAM>(rx, off[i]);
      res[i] = row_load<STREAM>(rr, off[i]);
    }
  };
  const int step = gridDim.x * R::G;
  int turn = 0;
  int r0 = blockIdx.x * R::G;
  fetch(r0);
  for (; r0 < a.M; r0 += step) {
    // (no fma but where it says so: the mean is a product, and as part of one it would be
    // another mean)
#pragma clang fp contract(off)
    u32x4 h[C];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[VEC], q[VEC];
      unpack16(x[i], v, T());
      unpack16(res[i], q, T());
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] += q[j];
      h[i] = pack16(v, T());
      unpack16(h[i], v, T());                // the norm of the sum as it is stored
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[j];
    }
    fetch(r0 + step);                        // in flight during the sums
    const float m0 = a.rms ? 0.f : row_sum<TPR>(s, red, turn) * a.inv_h;
    float mean = m0, d2 = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[VEC], e = 0.f;
      unpack16(h[i], v, T());
#pragma unroll
      for (int j = 0; j < VEC; ++j) e = fmaf(v[j] - m0, v[j] - m0, e);
      d2 += off[i] != NORM_OOB ? e : 0.f;
    }
    float var = row_sum<TPR>(d2, red, turn) * a.inv_h;
    // Where the mean is beyond twice the deviations its rounding counts, and the mean of
    // what is left corrects it: m + E[d], E[d^2] - E[d]^2.  (In every row that would take
    // 2 us of the 88 of 8192 x 7680, 5 of the 52 without a residual.)
    if (!a.rms && m0 * m0 > 4.f * var) {
      float d1 = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float v[VEC], f = 0.f;
        unpack16(h[i], v, T());
#pragma unroll
        for (int j = 0; j < VEC; ++j) f += v[j] - m0;
        d1 += off[i] != NORM_OOB ? f : 0.f;
      }
      d1 = row_sum<TPR>(d1, red, turn) * a.inv_h;
      mean = m0 + d1;
      var -= d1 * d1;
      var = var < 0.f ? 0.f : var;
    }
    const float rstd = 1.0f / sqrtf(var + a.eps);
    const auto rh = rows(a.h, r0), ry = rows(a.y, r0);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[VEC];
      unpack16(h[i], v, T());
      buf_store16_nt(rh, off[i], h[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = fmaf((v[j] - mean) * rstd, w[i][j], b[i][j]);
      buf_store16_nt(ry, off[i], pack16(v, T()));
    }
    if (lane == 0 && r0 + grp < a.M) {
      if (a.mean && !a.rms) a.mean[r0 + grp] = mean;
      if (a.rstd) a.rstd[r0 + grp] = rstd;
    }
  }
}

struct NormBwdArgs {
  const void* dy; const void* h; const void* dh; const float* w; const float* mean;
  const float* rstd;
  void* dx; float* dw; float* db; float* part;
  int M, H, rms, parts;
  float inv_h;
};

template <typename T, int TPR, int C, int NT_, bool STREAM>
__global__ __launch_bounds__(NT_) void norm_bwd_kernel(NormBwdArgs a) {
  using R = Rows<T, TPR, C, NT_>;
  constexpr int VEC = R::VEC, ES = sizeof(T);
  constexpr bool PRE = R::PRE;
  __shared__ float2 red[2][R::WAVES];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int n = a.H / VEC;
  const uint32_t rb = (uint32_t)a.H * ES;
  uint32_t off[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = lane + i * TPR;
    off[i] = c < n ? (uint32_t)grp * rb + (uint32_t)c * 16u : NORM_OOB;
  }
  float w[PRE ? C : 1][VEC], dw[C][VEC], db[C][VEC];
  const auto rw = make_rsrc(a.w, (uint32_t)a.H * 4u);
  auto wo = [&](int i, int j) { return ((uint32_t)(lane + i * TPR) * VEC + j) * 4u; };
  auto weight = [&](int i) -> const float (&)[VEC] {   // (where registers are short: read again)
    if constexpr (PRE) {
      return w[i];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j += 4) unpack16(buf_load16(rw, wo(i, j)), &w[0][j], float());
      return w[0];
    }
  };
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      if (PRE) unpack16(buf_load16(rw, wo(i, j)), &w[i][j], float());
#pragma unroll
      for (int l = 0; l < 4; ++l) dw[i][j + l] = 0.f, db[i][j + l] = 0.f;
    }
  auto rows = [&](const void* p, int r0) {
    const int m = r0 < a.M && p != nullptr ? (a.M - r0 < R::G ? a.M - r0 : R::G) : 0;
    return make_rsrc((const char*)p + (m ? (long long)r0 * rb : 0), (uint32_t)m * rb);
  };
  u32x4 y[C], x[C];
  float mean, rstd;
  auto fetch = [&](int r0) {
    const auto ry = rows(a.dy, r0), rx = rows(a.h, r0);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      y[i] = row_load<STREAM>(ry, off[i]);
      x[i] = row_load<STREAM>(rx, off[i]);
    }
    const int r = r0 + grp;
    mean = !a.rms && r < a.M ? a.mean[r] : 0.f;
    rstd = r < a.M ? a.rstd[r] : 0.f;
  };
  const int step = gridDim.x * R::G;
  int turn = 0;
  int r0 = blockIdx.x * R::G;
  fetch(r0);
  for (; r0 < a.M; r0 += step) {
    float s1 = 0.f, s2 = 0.f;
    u32x4 yc[C], xc[C], ac[C];
    const float m = mean, rs = rstd;
    // (asked for here and not with the next row: 95 us, 99 with it)
    const auto ra = rows(a.dx ? a.dh : nullptr, r0);
#pragma unroll
    for (int i = 0; i < C; ++i) ac[i] = row_load<STREAM>(ra, off[i]);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      yc[i] = y[i], xc[i] = x[i];
      float dy[VEC], q[VEC];
      unpack16(yc[i], dy, T());
      unpack16(xc[i], q, T());
      const float(&wi)[VEC] = weight(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        q[j] = (q[j] - m) * rs;
        const float g = dy[j] * wi[j];
        s1 += g;
        s2 = fmaf(g, q[j], s2);
        dw[i][j] = fmaf(dy[j], q[j], dw[i][j]);
        db[i][j] += dy[j];
      }
    }
    if (PRE) fetch(r0 + step);               // in flight during the sums
    row_sums<TPR>(s1, s2, red, turn);
    s1 = a.rms ? 0.f : s1 * a.inv_h;
    s2 *= a.inv_h;
    const auto rx = rows(a.dx, r0);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float dy[VEC], q[VEC], v[VEC];
      unpack16(yc[i], dy, T());
      unpack16(xc[i], q, T());
      unpack16(ac[i], v, T());
      const float(&wi)[VEC] = weight(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        q[j] = (q[j] - m) * rs;
        v[j] = fmaf(rs, dy[j] * wi[j] - s1 - q[j] * s2, v[j]);
      }
      buf_store16_nt(rx, off[i], pack16(v, T()));
    }
    if (!PRE) fetch(r0 + step);
  }
  if (a.part == nullptr) return;
  float* const part = a.part + (long long)blockIdx.x * 2 * a.H;
  const auto rp = make_rsrc(part, (uint32_t)a.H * 8u);
  if constexpr (R::G > 1) {                  // rows side by side: lanes of a wave, then the waves
    constexpr int PER = TPR < MOE_WAVE ? 1 : TPR / MOE_WAVE;   // waves of a row
    __shared__ float sum[2][TPR * C * VEC];
    if constexpr (TPR < MOE_WAVE) {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
#pragma unroll
          for (int o = TPR; o < MOE_WAVE; o *= 2) {
            dw[i][j] += __shfl_xor(dw[i][j], o, MOE_WAVE);
            db[i][j] += __shfl_xor(db[i][j], o, MOE_WAVE);
          }
    }
    for (int v = 0; v < R::WAVES / PER; ++v) {
      if ((int)(threadIdx.x / MOE_WAVE) / PER == v && (threadIdx.x & 63) < TPR) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int c = (lane + i * TPR) * VEC + j;
            sum[0][c] = v ? sum[0][c] + dw[i][j] : dw[i][j];
            sum[1][c] = v ? sum[1][c] + db[i][j] : db[i][j];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.H; c += R::NT) {
      part[c] = sum[0][c];
      part[a.H + c] = sum[1][c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (off[i] == NORM_OOB) continue;
#pragma unroll
      for (int j = 0; j < VEC; j += 4) {
        const uint32_t o = ((uint32_t)(lane + i * TPR) * VEC + j) * 4u;
        buf_store16(rp, o, pack16(&dw[i][j], float()));
        buf_store16(rp, o + (uint32_t)a.H * 4u, pack16(&db[i][j], float()));
      }
    }
  }
}

// The workgroups' sums, in their order: 32 columns a workgroup, a 32nd of the
// rows a thread.
constexpr int SUM_COLS = 32, SUM_ROWS = 32;
__global__ __launch_bounds__(SUM_COLS* SUM_ROWS) void norm_sum_kernel(NormBwdArgs a) {
  __shared__ double red[SUM_ROWS][SUM_COLS];
  const int col = threadIdx.x % SUM_COLS, row = threadIdx.x / SUM_COLS;
  const int c = blockIdx.x * SUM_COLS + col;   // of [dw | db]
  double s = 0;
  if (c < 2 * a.H)
#pragma unroll 8
    for (int p = row; p < a.parts; p += SUM_ROWS) s += a.part[(long long)p * 2 * a.H + c];
  red[row][col] = s;
  __syncthreads();
  if (row != 0 || c >= 2 * a.H) return;
#pragma unroll
  for (int r = 1; r < SUM_ROWS; ++r) s += red[r][col];
  if (c < a.H) {
    if (a.dw) a.dw[c] = (float)s;
  } else if (a.db) {
    a.db[c - a.H] = (float)s;
  }
}

// ---------------------------------------------------------------- host

struct Shape {
  int tpr, c, nt;   // as Rows
  int waves;        // resident in a CU
};

// Threads of a row by its 16-byte chunks.  Where 64 lanes hold a row in two chunks
// they do, without a barrier (1000 x 1024 bf16: 3.1 us, 3.8 with 256 threads a
// row); from 256 chunks on 256 threads and more (8 x 2048 bf16: 2.5 us, 3.0 by a
// wave; 8192 x 4096: 50 us at two chunks a thread, 53 by a wave), and two chunks a
// thread rather than four (8192 x 7680: 91 us, 95 with four, 90 to 94 with one).  Workgroups
// of a CU: enough rows in flight, which are 8 waves with a residual (91 us, 95 at
// 16) and 16 without (52 us, 69 at 8).
Shape norm_shape(int chunks, bool residual) {
  if (chunks <= 8) return {8, 1, 256, 16};
  if (chunks <= 16) return {16, 1, 256, 16};
  if (chunks <= 32) return {32, 1, 256, 16};
  if (chunks <= 64) return {64, 1, 256, 16};
  if (chunks <= 128) return {64, 2, 256, 16};
  const int waves = residual ? 8 : 16;
  if (chunks <= 256) return {256, 1, 256, waves};
  if (chunks <= 512) return {256, 2, 256, waves};
  if (chunks <= 1024) return {512, 2, 512, waves};
  if (chunks <= 2048) return {512, 4, 512, waves};
  return {1024, 4, 1024, 16};
}
// The backward: a workgroup's last row of sums is written and read again, so few
// large workgroups, 8 waves a CU (8192 x 7680: 95 us, 101 at 16; 4095 x 2048 fp32:
// 21 us, 23 in workgroups of 256 at 16 waves, 28 with one chunk a thread at 8),
// but for rows of one chunk a thread, whose registers are few (131071 x 128: 21.6
// us, 22.2 at 8 waves).  Above 1024 chunks 1024 threads without the next row.
Shape norm_bwd_shape(int chunks) {
  if (chunks <= 8) return {8, 1, 512, 16};
  if (chunks <= 16) return {16, 1, 512, 16};
  if (chunks <= 32) return {32, 1, 512, 16};
  if (chunks <= 64) return {64, 1, 512, 16};
  if (chunks <= 128) return {64, 2, 512, 8};
  if (chunks <= 256) return {128, 2, 512, 8};
  if (chunks <= 512) return {256, 2, 512, 8};
  if (chunks <= 1024) return {512, 2, 512, 8};
  if (chunks <= 2048) return {1024, 2, 1024, 16};
  return {1024, 4, 1024, 16};
}
// Workgroups, as many as are resident, or as many times that as keep a thread's rows at
// `chain`.
int norm_blocks(int M, Shape s, long long chain) {
  const long long G = s.nt / s.tpr, most = (long long)moe_cu_count() * s.waves * MOE_WAVE / s.nt;
  const long long need = (M + G - 1) / G, per = (need + most - 1) / most;
  if (per == 0) return 0;
  const long long times = (per + chain - 1) / chain, each = (per + times - 1) / times;
  return (int)((need + each - 1) / each);
}
// Rows whose part of dw and db a thread adds in fp32, at most; 10 more additions join the
// rows of a workgroup, and the workgroups' sums are fp64.  (Alike in 2^27 rows of 8 values,
// 4096 a thread, they were off by 890 roundings.)
constexpr int NORM_CHAIN = 240;
int norm_parts(int M, int H, int dt) {
  return norm_blocks(M, norm_bwd_shape(H * moe_dt_bytes(dt) / 16), NORM_CHAIN);
}

#define NORM_SHAPES(X)                                                                    \
  X(8, 1, 256) X(16, 1, 256) X(32, 1, 256) X(64, 1, 256) X(64, 2, 256) X(256, 1, 256)     \
  X(256, 2, 256) X(512, 2, 512) X(512, 4, 512) X(1024, 4, 1024)
#define NORM_BWD_SHAPES(X)                                                                \
  X(8, 1, 512) X(16, 1, 512) X(32, 1, 512) X(64, 1, 512) X(64, 2, 512) X(128, 2, 512)     \
  X(256, 2, 512) X(512, 2, 512) X(1024, 2, 1024) X(1024, 4, 1024)

// (rows of bf16 end at 2048 chunks)
template <typename T, bool STREAM>
int norm_launch(const NormArgs& a, Shape s, hipStream_t st) {
  const dim3 grid(norm_blocks(a.M, s, a.M));
#define X(P, N, TH)                                                                        \
  if constexpr (P * N * Elem<T>::VEC <= NORM_MAX_H)                                        \
    if (s.tpr == P && s.c == N)                                                            \
      hipLaunchKernelGGL((norm_kernel<T, P, N, TH, STREAM>), grid, dim3(TH), 0, st, a);
  NORM_SHAPES(X)
#undef X
  return moe_check_launch("moe_norm");
}
template <typename T, bool STREAM>
int norm_bwd_launch(const NormBwdArgs& a, Shape s, hipStream_t st) {
  const dim3 grid(a.parts);
#define X(P, N, TH)                                                                        \
  if constexpr (P * N * Elem<T>::VEC <= NORM_MAX_H)                                        \
    if (s.tpr == P && s.c == N)                                                            \
      hipLaunchKernelGGL((norm_bwd_kernel<T, P, N, TH, STREAM>), grid, dim3(TH), 0, st, a);
  NORM_BWD_SHAPES(X)
#undef X
  return moe_check_launch("moe_norm_bwd");
}

// A call whose rows, read and written, are more than the 256 MB memory-side cache
// holds reads them with the streaming policy (8192 x 7680, forward: 87 us, 91
// without; 4095 x 2048 fp32, which the cache holds, 16 us with it and 12 without),
// in a kernel of its own: with a branch between the two kinds of load the backward
// of 8192 x 7680 took 105 us, so 95.  Stores are streaming always (87 and 94 us).
bool norm_streams(long long bytes) { return bytes > (256LL << 20); }

int norm_checks(const char* fn, int dt, int M, int H, int kind) {
  MOE_TRY(moe_need_dt(dt, fn));
  MOE_TRY(moe_need_nonneg(M, fn, "M"));
  if (H < 8 || H % 8 != 0 || H > NORM_MAX_H)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: H = %d is no multiple of 8 in [8, %d]", fn, H,
                    NORM_MAX_H);
  if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: kind %d is none of the MOE_NORM values", fn, kind);
  return moe_need_elems(M, H, moe_dt_bytes(dt), fn, "x");
}

}  // namespace

extern "C" int moe_norm(const void* x, const void* residual, int dt, int M, int H, int kind,
                        float eps, const float* w, const float* bias, void* h, void* y,
                        float* mean, float* rstd, moe_stream_t stream) {
  const char* fn = "moe_norm";
  MOE_TRY(norm_checks(fn, dt, M, H, kind));
  if (!(eps > 0.f && eps < INFINITY))
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: eps = %g is not positive and finite", fn, eps);
  if (h != nullptr && residual == nullptr)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: h without a residual is x", fn);
  if (M == 0) return MOE_OK;
  MOE_TRY(moe_need_ptr(x, fn, "x"));
  MOE_TRY(moe_opt_ptr(residual, fn, "residual"));
  MOE_TRY(moe_need_ptr(w, fn, "w"));
  MOE_TRY(moe_opt_ptr(bias, fn, "bias"));
  MOE_TRY(moe_opt_ptr(h, fn, "h"));
  MOE_TRY(moe_need_ptr(y, fn, "y"));
  MOE_TRY(moe_opt_ptr(mean, fn, "mean", 4));
  MOE_TRY(moe_opt_ptr(rstd, fn, "rstd", 4));
  const long long mh = (long long)M * H * moe_dt_bytes(dt);
  const MoeRange rx = {x, mh, "x"}, rr = {residual, mh, "residual"}, rw = {w, 4LL * H, "w"},
                 rb = {bias, 4LL * H, "bias"}, rh = {h, mh, "h"}, ry = {y, mh, "y"},
                 rm = {mean, 4LL * M, "mean"}, rs = {rstd, 4LL * M, "rstd"};
  const char* out = "y";
  const char* with = moe_shares(ry, {rx, rr, rw, rb, rh});
  if (with == nullptr) {   // (an element of h is written by the thread that read it)
    out = "h";
    with = moe_shares(rh, {rw, rb, h != x ? rx : MoeRange{}, h != residual ? rr : MoeRange{}});
  }
  if (with == nullptr) {
    out = "mean";
    with = moe_shares(rm, {rx, rr, rw, rb, rh, ry});
  }
  if (with == nullptr) {
    out = "rstd";
    with = moe_shares(rs, {rx, rr, rw, rb, rh, ry, rm});
  }
  if (with != nullptr)
    return moe_fail(MOE_ERR_INVALID_ARG,
                    "%s: %s overlaps %s (h alone may be x's or the residual's buffer)", fn, out,
                    with);
  NormArgs a = {x, residual, w, bias, h, y, mean, rstd, M, H, kind == MOE_NORM_RMS,
                eps, 1.0f / H};
  hipStream_t s = (hipStream_t)stream;
  const Shape shape = norm_shape(H * moe_dt_bytes(dt) / 16, residual != nullptr);
  const bool far = norm_streams(mh * (2 + (residual != nullptr) + (h != nullptr)));
  if (dt == MOE_BF16)
    return far ? norm_launch<bf16_t, true>(a, shape, s) : norm_launch<bf16_t, false>(a, shape, s);
  return far ? norm_launch<float, true>(a, shape, s) : norm_launch<float, false>(a, shape, s);
}

extern "C" size_t moe_norm_bwd_workspace_bytes(int M, int H, int dt) {
  if (norm_checks("moe_norm_bwd_workspace_bytes", dt, M, H, MOE_NORM_LAYER) != MOE_OK) return 0;
  return ((size_t)norm_parts(M, H, dt) * 2 * H * 4 + 255) / 256 * 256;
}

extern "C" int moe_norm_bwd(const void* dy, const void* h, const void* dh, int dt, int M, int H,
                            int kind, const float* w, const float* mean, const float* rstd,
                            void* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                            moe_stream_t stream) {
  const char* fn = "moe_norm_bwd";
  MOE_TRY(norm_checks(fn, dt, M, H, kind));
  MOE_TRY(moe_opt_ptr(dx, fn, "dx"));
  MOE_TRY(moe_opt_ptr(dw, fn, "dw"));
  MOE_TRY(moe_opt_ptr(db, fn, "db"));
  const bool sums = dw != nullptr || db != nullptr;
  const size_t need = sums ? moe_norm_bwd_workspace_bytes(M, H, dt) : 0;
  if (M > 0) {
    MOE_TRY(moe_need_ptr(dy, fn, "dy"));
    MOE_TRY(moe_need_ptr(h, fn, "h"));
    MOE_TRY(moe_opt_ptr(dh, fn, "dh"));
    MOE_TRY(moe_need_ptr(w, fn, "w"));
    if (kind == MOE_NORM_LAYER) MOE_TRY(moe_need_ptr(mean, fn, "mean", 4));
    MOE_TRY(moe_need_ptr(rstd, fn, "rstd", 4));
    if (sums) {
      MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
      if (ws_bytes < need)
        return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                        need);
    }
  }
  const long long mh = (long long)M * H * moe_dt_bytes(dt);
  const MoeRange rdy = {dy, mh, "dy"}, rh = {h, mh, "h"},
                 rdh = {dh, mh, "dh"}, rw = {w, 4LL * H, "w"},
                 rm = {kind == MOE_NORM_LAYER ? mean : nullptr, 4LL * M, "mean"},
                 rr = {rstd, 4LL * M, "rstd"},
                 outs[] = {{dx, mh, "dx"}, {dw, 4LL * H, "dw"}, {db, 4LL * H, "db"},
                           {sums ? ws : nullptr, (long long)need, "ws"}};
  for (int i = 0; i < 4; ++i) {
    const char* with = moe_shares(outs[i], {rdy, rh, rw, rm, rr});
    if (with == nullptr && !(i == 0 && dx == dh)) with = moe_shares(outs[i], {rdh});
    for (int j = 0; j < i && with == nullptr; ++j) with = moe_shares(outs[i], {outs[j]});
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s (dx alone may be dh's buffer)", fn,
                      outs[i].name, with);
  }
  NormBwdArgs a = {dy, h, dh, w, mean, rstd, dx, dw, db, sums ? (float*)ws : nullptr, M, H,
                   kind == MOE_NORM_RMS, norm_parts(M, H, dt), 1.0f / H};
  hipStream_t s = (hipStream_t)stream;
  if (M > 0 && (dx != nullptr || sums)) {
    const Shape shape = norm_bwd_shape(H * moe_dt_bytes(dt) / 16);
    const bool far = norm_streams(mh * (2 + (dx != nullptr) + (dx != nullptr && dh != nullptr)));
    const int st = dt == MOE_BF16 ? far ? norm_bwd_launch<bf16_t, true>(a, shape, s)
                                        : norm_bwd_launch<bf16_t, false>(a, shape, s)
                   : far          ? norm_bwd_launch<float, true>(a, shape, s)
                                  : norm_bwd_launch<float, false>(a, shape, s);
    MOE_TRY(st);
  }
  if (!sums) return MOE_OK;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((2 * H + SUM_COLS - 1) / SUM_COLS),
                     dim3(SUM_COLS * SUM_ROWS), 0, s, a);
  return moe_check_launch(fn);
}
