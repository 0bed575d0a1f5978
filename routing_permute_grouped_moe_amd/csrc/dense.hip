// Dense products too small for the grouped GEMM's 256 x 256 tiles: with few
// of those, most of the 256 CUs would idle, so these run on 128 x 128 or
// 64 x 64 tiles and, where that still leaves CUs idle, in K slices whose fp32
// partial sums a second launch adds in slice order and finishes.
//
//   linear fwd   y = act(x W^T + b) + residual     both operands K-contiguous
//   linear bwd   dx = dz W, dW = dz^T x            one launch for both products
//
// A workgroup of 4 waves (2 x 2) owns a BT x BT tile; K runs in steps of 128
// bytes (64 bf16, 32 fp32) through a ring of LDS stages filled by direct
// copies (lds_copy.hpp).  K-contiguous operands sit in LDS as BT rows of 128
// bytes, 16-byte chunk c of row r in slot c ^ ((r >> 1) & 7), so 16 rows read
// at once cover all banks; MN-contiguous operands sit as rows of K, bf16 ones
// read with the transposing LDS read, their chunks moved so that its four
// rows fall into distinct banks.
#include <type_traits>

#include "act.hpp"
#include "lds_copy.hpp"
#include "validate.hpp"

namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4* lds_bf16x4_t;

constexpr uint32_t D_OOB = 0x80000000u;   // past every operand (all below 2 GiB)
constexpr int D_ROWB = 128;               // bytes of a K step along K
constexpr int D_GROUPS = 4;               // 32 x 32 MFMA groups per K step (16 bf16 or 8 fp32 of K)

// One product C[M,N] (+ epilogue) in S slices of kslice along K.
struct DenseArgs {
  const void* A; const void* B;   // A_MN: A[k][m], else A[m][k]; B alike with n
  int lda, ldb, M, N, K;
  int mt, nt, S, kslice;          // tiles, slices, K of a slice (a multiple of a step)
  void* C;                        // [M][N]
  float* part;                    // [S][M][N] partial sums (S > 1)
  const float* bias; const void* res; void* z; int act;   // epilogue (nullable, fwd)
};

// Per tile size: stages of the ring
// (two workgroups of 64 KB fit a CU, and one multiplies while the other waits
// for its copies: with three stages, one to a CU, 2000 x 8192 x 2048 took 116 us
// instead of 83)
template <int BT> constexpr int D_STAGES = BT == 128 ? 2 : 4;
template <int BT> constexpr int D_OPB = BT * D_ROWB;      // bytes of an operand's stage
template <int BT> constexpr int D_RING = D_STAGES<BT> * 2 * D_OPB<BT>;

__device__ __forceinline__ int kchunk(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }
// MN-major rows of K: BT bf16 are 16 (or 8) chunks; fp32 rows are read word by word
template <int BT>
__device__ __forceinline__ int mchunk_bf16(int k, int chunk) {
  if constexpr (BT == 128) return chunk ^ ((k & 3) << 2);
  else return chunk ^ (((k >> 1) & 1) << 2);
}

template <typename T, bool MN, int BT>
__device__ __forceinline__ void copy_offsets(int mn0, int lim, int ld, uint32_t (&off)[BT / 32]) {
  constexpr int ES = sizeof(T), VEC = 16 / ES;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < BT / 32; ++j) {
    const int q = wave * (BT / 32) + j;     // 1 KB of the stage
    if constexpr (!MN) {
      const int row = q * 8 + (lane >> 3);
      const int chunk = kchunk(row, lane & 7);
      off[j] = mn0 + row < lim ? (uint32_t)((mn0 + row) * ld * ES + chunk * 16) : D_OOB;
    } else {
      constexpr int CPR = BT / VEC;         // 16-byte chunks per K row
      const int at = q * 64 + lane, k = at / CPR;
      int chunk = at % CPR;
      if constexpr (ES == 2) chunk = mchunk_bf16<BT>(k, chunk);
      const int mn = mn0 + chunk * VEC;
      off[j] = mn < lim ? (uint32_t)((k * ld + mn) * ES) : D_OOB;
    }
  }
}

// Fragment of 32 rows (or columns) from r0 on, K group g: lane l has row
// r0 + l % 32, 16 bytes of K from 16 (2 g + l / 32) on.
template <typename T, bool MN, int BT>
__device__ __forceinline__ u32x4 dense_frag(const char* st, int r0, int g) {
  const int lane = threadIdx.x & 63;
  if constexpr (!MN) {
    const int row = r0 + (lane & 31);
    return *(const u32x4*)(st + row * D_ROWB + (kchunk(row, 2 * g + (lane >> 5)) << 4));
  } else if constexpr (sizeof(T) == 2) {
    const int grp = lane >> 4, i = lane & 15;
    const int col = r0 + (grp & 1) * 16 + 4 * (i & 3);
    const int kb = g * 16 + (grp >> 1) * 8 + (i >> 2);
    const char* p0 = st + kb * (BT * 2) + (mchunk_bf16<BT>(kb, col >> 3) << 4) + (col & 7) * 2;
    const char* p1 =
        st + (kb + 4) * (BT * 2) + (mchunk_bf16<BT>(kb + 4, col >> 3) << 4) + (col & 7) * 2;
    const u32x2 lo =
        __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t)p0));
    const u32x2 hi =
        __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t)p1));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  } else {
    const int k = 8 * g + 4 * (lane >> 5), r = r0 + (lane & 31);
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *(const uint32_t*)(st + ((k + i) * BT + r) * 4);
    return v;
  }
}

__device__ __forceinline__ f32x16 dense_mma(const u32x4& a, const u32x4& b, f32x16 c, bf16_t) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 dense_mma(const u32x4& a, const u32x4& b, f32x16 c, float) {
  const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i], fb[i], c, 0, 0, 0);
  return c;
}

// bias, activation, residual on 4 sums of row m, columns n .. n + 3
template <typename T>
__device__ __forceinline__ void dense_finish(const DenseArgs& a, int m, int n, f32x4 v) {
  const long long at = (long long)m * a.N + n;
  auto store = [&](void* p, const f32x4& s) {
    if constexpr (sizeof(T) == 2) {
      u32x2 o;
      o.x = f32_to_bf16(s.x) | (f32_to_bf16(s.y) << 16);
      o.y = f32_to_bf16(s.z) | (f32_to_bf16(s.w) << 16);
      *(u32x2*)((T*)p + at) = o;
    } else {
      *(f32x4*)((T*)p + at) = s;
    }
  };
  if (a.bias != nullptr) v += *(const f32x4*)(a.bias + n);
  if (a.z != nullptr) store(a.z, v);
  if (a.act != MOE_ACT_NONE)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], a.act);
  if (a.res != nullptr) {
    if constexpr (sizeof(T) == 2) {
      const u32x2 r = *(const u32x2*)((const T*)a.res + at);
      v += f32x4{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                 __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u)};
    } else {
      v += *(const f32x4*)((const T*)a.res + at);
    }
  }
  store(a.C, v);
}

// Tile (m0, n0), K from k0 on: sums, then the epilogue or the partial store.
template <typename T, bool A_MN, bool B_MN, int BT>
__device__ __forceinline__ void dense_tile(const DenseArgs& a, int m0, int n0, int slice,
                                           char* smem) {
  constexpr int ES = sizeof(T), BK = D_ROWB / ES, NS = D_STAGES<BT>, OPB = D_OPB<BT>;
  constexpr int F = BT / 64;            // 32 x 32 fragments along a wave's tile
  constexpr int CP = BT / 32;           // copies per operand per wave per step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * (BT / 2), wn = (wave & 1) * (BT / 2);
  const int k0 = slice * a.kslice, k1 = min(a.K, k0 + a.kslice), kn = k1 - k0;
  auto rsrc = [&](const void* p, bool mn, int ld, int rows) {
    const char* b = (const char*)p + (long long)(mn ? (long long)k0 * ld : k0) * ES;
    const long long n = mn ? (long long)kn * ld : (long long)(rows - 1) * ld + kn;
    return raw_rsrc(b, (uint32_t)(n * ES));
  };
  const i32x4 ra = rsrc(a.A, A_MN, a.lda, a.M), rb = rsrc(a.B, B_MN, a.ldb, a.N);
  uint32_t offa[CP], offb[CP];
  copy_offsets<T, A_MN, BT>(m0, a.M, a.lda, offa);
  copy_offsets<T, B_MN, BT>(n0, a.N, a.ldb, offb);
  const int sa = A_MN ? a.lda * BK * ES : D_ROWB, sb = B_MN ? a.ldb * BK * ES : D_ROWB;
  const int steps = (kn + BK - 1) / BK;
  const uint32_t base = lds_addr(smem) + wave * CP * 1024;
  // (steps past the last copy through an empty range, so that the wait counts
  // hold for every step)
  auto issue = [&](int kt) {
    const uint32_t st = base + (uint32_t)(kt % NS) * (2 * OPB);
    const int live = uniform(kt < steps ? -1 : 0);
    const i32x4 va = {uniform(ra.x), uniform(ra.y), uniform(ra.z & live), MOE_RSRC_DW3};
    const i32x4 vb = {uniform(rb.x), uniform(rb.y), uniform(rb.z & live), MOE_RSRC_DW3};
#pragma unroll
    for (int j = 0; j < CP; ++j) dma16(va, st + j * 1024, offa[j], kt * sa & live);
#pragma unroll
    for (int j = 0; j < CP; ++j) dma16(vb, st + OPB + j * 1024, offb[j], kt * sb & live);
  };
  f32x16 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
#pragma unroll
  for (int kt = 0; kt < NS - 1; ++kt) issue(kt);
  for (int kt = 0; kt < steps; ++kt) {
    wait_vm<(NS - 2) * 2 * CP>();
    __syncthreads();   // step kt has landed for every wave; step kt - 1's stage is free
    issue(kt + NS - 1);
    const char* st = smem + (kt % NS) * (2 * OPB);
    // two sets of fragments in turn: a group's reads go between the MFMAs of the
    // group before (pinned by scheduling barriers), so that only the first
    // group of a step waits for its own
    u32x4 fa[2][F], fb[2][F];
    auto load = [&](int g, int q) {   // read q of group g: A fragments, then B
      if (q < F) fa[g & 1][q] = dense_frag<T, A_MN, BT>(st, wm + 32 * q, g);
      else fb[g & 1][q - F] = dense_frag<T, B_MN, BT>(st + OPB, wn + 32 * (q - F), g);
    };
#pragma unroll
    for (int q = 0; q < 2 * F; ++q) load(0, q);
#pragma unroll
    for (int g = 0; g < D_GROUPS; ++g)
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) {
          acc[i][j] = dense_mma(fb[g & 1][j], fa[g & 1][i], acc[i][j], T());
          __builtin_amdgcn_sched_barrier(0);
          const int q = i * F + j;    // F^2 MFMAs carry the next group's 2 F reads
          if (g + 1 < D_GROUPS) {
            if constexpr (F == 1) {
              load(g + 1, 0);
              load(g + 1, 1);
            } else if (q < 2 * F) {
              load(g + 1, q);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
  }
  wait_vm<0>();
  __syncthreads();   // the ring is free: each wave turns its tile through its own part of it
  // register r of fragment (i, j): row 32 i + lane % 32, column 32 j + 8 (r / 4)
  // + 4 (lane / 32) + r % 4 (the B fragment is the MFMA's first operand)
  constexpr int WB = BT / 2, PITCH = WB + 4;
  float* const ep = (float*)smem + wave * (32 * PITCH);
#pragma unroll
  for (int i = 0; i < F; ++i) {
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(ep + (lane & 31) * PITCH + 32 * j + 8 * q + 4 * (lane >> 5)) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    // (one wave's own words: its LDS accesses stay in order)
    __builtin_amdgcn_wave_barrier();
    constexpr int CPR = WB / 4, RPP = 64 / CPR;   // chunks of 4 columns per row, rows per pass
#pragma unroll
    for (int p = 0; p < 32 / RPP; ++p) {
      const int r = p * RPP + lane / CPR, c = (lane % CPR) * 4;
      const f32x4 v = *(const f32x4*)(ep + r * PITCH + c);
      const int m = m0 + wm + 32 * i + r, n = n0 + wn + c;
      if (m < a.M && n < a.N) {
        if (a.S > 1) *(f32x4*)(a.part + ((long long)slice * a.M + m) * a.N + n) = v;
        else dense_finish<T>(a, m, n, v);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Unit u of a product: M tiles of a column panel one after the other, then
// the panels, then the slices.
template <typename T, bool A_MN, bool B_MN, int BT>
__device__ __forceinline__ void dense_unit(const DenseArgs& a, int u, char* smem) {
  const int per = a.mt * a.nt;
  const int slice = uniform(u / per), t = uniform(u % per);
  dense_tile<T, A_MN, B_MN, BT>(a, uniform(t % a.mt) * BT, uniform(t / a.mt) * BT, slice, smem);
}

// Workgroup b runs on XCD b % 8: consecutive units go to one XCD, so the
// tiles that share a weight panel share its L2.
__device__ __forceinline__ int xcd_unit(int b, int total) {
  const int per = total / 8, rest = total % 8;
  const int x = b % 8, i = b / 8;
  return x * per + min(x, rest) + i;
}

template <typename T, int BT>
__global__ __launch_bounds__(256) void dense_fwd_kernel(DenseArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[D_RING<BT>];
  dense_unit<T, false, false, BT>(a, xcd_unit(blockIdx.x, gridDim.x), smem);
}

// db = sum of the blocks' column sums of dz: four threads a column, each over a
// quarter of the blocks in order, then the four in order.  Workgroup b takes 64
// columns (N is a multiple of 64).
struct DbArgs {
  const float* sums; int parts, N; float* db;
};
__device__ __forceinline__ void dense_db(const DbArgs& a, int b, double* red) {
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6, n = b * 64 + c;
  const int per = (a.parts + 3) / 4, p1 = min(a.parts, (q + 1) * per);
  double s = 0;
#pragma unroll 8
  for (int p = q * per; p < p1; ++p) s += a.sums[(long long)p * a.N + n];
  red[q * 64 + c] = s;
  __syncthreads();
  if (q == 0) a.db[n] = (float)(((red[c] + red[64 + c]) + red[128 + c]) + red[192 + c]);
}
__global__ __launch_bounds__(256) void dense_db_kernel(DbArgs a) {
  __shared__ double red[256];
  dense_db(a, blockIdx.x, red);
}

// dx (A = dz K-contiguous, B = W with rows along K) and dW (both operands
// with rows along K): units of dx first; then the bias gradient
template <typename T, int BT>
__global__ __launch_bounds__(256) void dense_bwd_kernel(DenseArgs dx, DenseArgs dw, DbArgs db) {
  __shared__ __attribute__((aligned(1024))) char smem[D_RING<BT>];
  const int n = dx.S * dx.mt * dx.nt, units = n + dw.S * dw.mt * dw.nt;
  if ((int)blockIdx.x >= units) {
    dense_db(db, blockIdx.x - units, (double*)smem);
    return;
  }
  const int u = xcd_unit(blockIdx.x, units);
  if (u < n) dense_unit<T, false, true, BT>(dx, u, smem);
  else dense_unit<T, true, true, BT>(dw, u - n, smem);
}

// Sum of the slices' partials in slice order, then the epilogue: 4 columns
// per thread; workgroups [0, n0) finish product a, the rest product b.
template <typename T>
__global__ __launch_bounds__(256) void dense_sum_kernel(DenseArgs a, DenseArgs b, int n0) {
  const bool second = (int)blockIdx.x >= n0;
  const DenseArgs& p = second ? b : a;
  const long long q = (long long)(blockIdx.x - (second ? n0 : 0)) * 256 + threadIdx.x;
  const long long mn = (long long)p.M * p.N;
  if (q * 4 >= mn) return;
  const f32x4* src = (const f32x4*)p.part + q;
  f32x4 v = src[0];
  for (int s = 1; s < p.S; ++s) v += src[s * (mn / 4)];
  dense_finish<T>(p, (int)(q * 4 / p.N), (int)(q * 4 % p.N), v);
}

// ---------------------------------------------------------------- host side

constexpr int D_MAX_S = 16;

// Tile size: 128 x 128 tiles move half the bytes per flop of 64 x 64 ones, so
// bf16 takes them as soon as there are 32.  In fp32, at a sixteenth of the
// matrix rate, the bytes matter less than an even share of the work: 1000 x 1024
// x 1024 (64 large tiles) takes 31 us on small ones and 34 on large, 600 x 2048 x
// 1600 (80) takes 60 and 48.
int plan_tile(long long M, long long N, int es) {
  return ((M + 127) / 128) * ((N + 127) / 128) >= (es == 4 ? 72 : 32) ? 128 : 64;
}

// tiles of a product; returns their number times K
double plan_tiles(DenseArgs& a, int bt) {
  a.mt = (a.M + bt - 1) / bt;
  a.nt = (a.N + bt - 1) / bt;
  return (double)a.mt * a.nt * a.K;
}
// K of a slice, for a launch of `work` tiles times K in all: 512 slices, two
// workgroups a CU, while they stay long enough to be worth their ramp and their
// partial sums (419 x 2048 x 8192: 28 us with 8 slices a tile, 30 with 4), else
// one a CU (128 x 8192 x 2048: 17 us with 4 slices, 21 with 8).  Both products
// of a backward are cut to the same length: 700 x 2048 x 1600 in fp32 takes 98
// us so, 248 when each is given half of the chip.
double plan_length(double work, int es) {
  const double two = es == 2 ? 640 : 256, least = es == 2 ? 256 : 64;
  double l = work / 512;
  if (l < two) l = work / 256;
  return l > least ? l : least;
}
void plan_slices(DenseArgs& a, int es, double length, double round) {
  const int bk = D_ROWB / es;
  int s = (int)(a.K / length + round);
  s = s < D_MAX_S ? s : D_MAX_S;
  s = s > 1 ? s : 1;
  a.kslice = ((a.K + s - 1) / s + bk - 1) / bk * bk;
  if (a.kslice < bk) a.kslice = bk;              // (no rows: K = 0)
  a.S = a.K > 0 ? (a.K + a.kslice - 1) / a.kslice : 1;
}

DenseArgs fwd_args(int M, int N, int K, int dt) {
  DenseArgs a = {};
  a.M = M; a.N = N; a.K = K; a.lda = K; a.ldb = K;
  const int es = moe_dt_bytes(dt);
  const double work = plan_tiles(a, plan_tile(M, N, es));
  plan_slices(a, es, plan_length(work, es), 1e-6);   // (no more than that)
  return a;
}

struct BwdPlan {
  int bt;
  DenseArgs dx, dw;
};
BwdPlan bwd_args(int M, int N, int K, int dt, bool dx_only) {
  BwdPlan p = {};
  const int es = moe_dt_bytes(dt);
  p.bt = plan_tile(dx_only ? M : M + N, K, es);
  p.dx.M = M; p.dx.N = K; p.dx.K = N; p.dx.lda = N; p.dx.ldb = K;
  p.dw.M = N; p.dw.N = K; p.dw.K = M; p.dw.lda = N; p.dw.ldb = K;
  double work = plan_tiles(p.dx, p.bt);
  if (!dx_only) work += plan_tiles(p.dw, p.bt);
  const double length = plan_length(work, es);
  plan_slices(p.dx, es, length, 0.5);
  plan_slices(p.dw, es, length, 0.5);
  return p;
}

size_t part_bytes(const DenseArgs& a) {
  return a.S > 1 ? (size_t)a.S * a.M * a.N * 4 : 0;
}

}  // namespace

size_t moe_dense_fwd_bytes(int M, int N, int K, int dt) {
  return part_bytes(fwd_args(M, N, K, dt));
}

size_t moe_dense_bwd_bytes(int M, int N, int K, int dt, bool dx_only) {
  const BwdPlan p = bwd_args(M, N, K, dt, dx_only);
  return part_bytes(p.dx) + (dx_only ? 0 : part_bytes(p.dw));
}

int moe_dense_fwd(const void* x, int dt, int M, int N, int K, const void* w, const float* bias,
                  int act, const void* residual, void* z, void* y, void* ws, hipStream_t s) {
  const char* fn = "moe_linear";
  DenseArgs a = fwd_args(M, N, K, dt);
  a.A = x; a.B = w; a.C = y; a.part = (float*)ws;
  a.bias = bias; a.res = residual; a.z = z; a.act = act;
  const dim3 grid(a.S * a.mt * a.nt), block(256);
  const bool big = plan_tile(M, N, moe_dt_bytes(dt)) == 128;
  if (dt == MOE_BF16) {
    if (big) hipLaunchKernelGGL((dense_fwd_kernel<bf16_t, 128>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((dense_fwd_kernel<bf16_t, 64>), grid, block, 0, s, a);
  } else {
    if (big) hipLaunchKernelGGL((dense_fwd_kernel<float, 128>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((dense_fwd_kernel<float, 64>), grid, block, 0, s, a);
  }
  MOE_TRY(moe_check_launch(fn));
  if (a.S == 1) return MOE_OK;
  const int n0 = (int)(((long long)M * N / 4 + 255) / 256);
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(dense_sum_kernel<bf16_t>, dim3(n0), block, 0, s, a, a, n0);
  else
    hipLaunchKernelGGL(dense_sum_kernel<float>, dim3(n0), block, 0, s, a, a, n0);
  return moe_check_launch(fn);
}

int moe_dense_db(const float* sums, int parts, int N, float* db, hipStream_t s) {
  hipLaunchKernelGGL(dense_db_kernel, dim3(N / 64), dim3(256), 0, s, DbArgs{sums, parts, N, db});
  return moe_check_launch("moe_linear_bwd");
}

int moe_dense_bwd(const void* dz, const void* x, const void* w, int dt, int M, int N, int K,
                  void* dx, void* dw, bool dx_only, const float* sums,
                  int parts, float* db, void* ws, hipStream_t s) {
  const char* fn = "moe_linear_bwd";
  BwdPlan p = bwd_args(M, N, K, dt, dx_only);
  DenseArgs &a = p.dx, &b = p.dw;
  a.A = dz; a.B = w; a.C = dx; a.part = (float*)ws;
  b.A = dz; b.B = x; b.C = dw; b.part = (float*)((char*)ws + part_bytes(a));
  if (dx == nullptr) a.mt = a.nt = 0;   // no units, no sums
  if (dw == nullptr) b.mt = b.nt = 0;
  const DbArgs c = {sums, parts, N, db};
  const dim3 grid(a.S * a.mt * a.nt + b.S * b.mt * b.nt + (db != nullptr ? N / 64 : 0)), block(256);
  if (grid.x == 0) return MOE_OK;
  if (dt == MOE_BF16) {
    if (p.bt == 128) hipLaunchKernelGGL((dense_bwd_kernel<bf16_t, 128>), grid, block, 0, s, a, b, c);
    else hipLaunchKernelGGL((dense_bwd_kernel<bf16_t, 64>), grid, block, 0, s, a, b, c);
  } else {
    if (p.bt == 128) hipLaunchKernelGGL((dense_bwd_kernel<float, 128>), grid, block, 0, s, a, b, c);
    else hipLaunchKernelGGL((dense_bwd_kernel<float, 64>), grid, block, 0, s, a, b, c);
  }
  MOE_TRY(moe_check_launch(fn));
  auto blocks = [](const DenseArgs& q) {
    return q.mt > 0 && q.S > 1 ? (int)(((long long)q.M * q.N / 4 + 255) / 256) : 0;
  };
  const int n0 = blocks(a), n1 = blocks(b);
  if (n0 + n1 == 0) return MOE_OK;
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(dense_sum_kernel<bf16_t>, dim3(n0 + n1), block, 0, s, a, b, n0);
  else
    hipLaunchKernelGGL(dense_sum_kernel<float>, dim3(n0 + n1), block, 0, s, a, b, n0);
  return moe_check_launch(fn);
}

int moe_dense_sum(const float* part, int S, int M, int N, int dt, void* out, hipStream_t s) {
  DenseArgs a = {};
  a.M = M; a.N = N; a.S = S; a.part = const_cast<float*>(part); a.C = out;
  const int n0 = (int)(((long long)M * N / 4 + 255) / 256);
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(dense_sum_kernel<bf16_t>, dim3(n0), dim3(256), 0, s, a, a, n0);
  else
    hipLaunchKernelGGL(dense_sum_kernel<float>, dim3(n0), dim3(256), 0, s, a, a, n0);
  return moe_check_launch("moe_linear_bwd");
}
