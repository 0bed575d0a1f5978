// A matrix product with bias, activation and residual in its epilogue, and
// its gradients:
//   z = x W^T + b,  y = act(z) + residual           (x [M,K], W [N,K])
//   dz = dy * act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
// Few rows (decode batches) run as a stream of W (stream.hpp); large products
// run on the grouped GEMM's 256 x 256 tiles (gmm.hip), those between on
// smaller tiles (dense.hip).  The epilogues take the bias, activation and
// residual, and the two products of the backward share one launch.  What is here: the few-row kernel, the elementwise half of the
// backward, the checks and the choice between the kernels.
#include <type_traits>

#include "act.hpp"
#include "stream.hpp"
#include "validate.hpp"

namespace {

constexpr int LIN_FEW_ROWS = 64;    // most rows of the streaming kernel
#ifndef LIN_TILES
#define LIN_TILES 192
#endif
constexpr int LIN_BIG_TILES = LIN_TILES;   // 256 x 256 tiles from which the large-tile kernels run
constexpr int LIN_NW = 8;
constexpr int LIN_NT = 64 * LIN_NW;

struct LinArgs {
  const void* x; const void* w; const float* bias; const void* residual;
  void* z; void* y;
  int M, N, K, act;
};

template <typename T>
__device__ __forceinline__ float lin_load(const void* p, long long i) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(((const T*)p)[i]);
  else return ((const T*)p)[i];
}
template <typename T>
__device__ __forceinline__ void lin_store(void* p, long long i, float v) {
  if constexpr (sizeof(T) == 2) ((T*)p)[i] = (T)f32_to_bf16(v);
  else ((T*)p)[i] = v;
}

// 16 output columns per workgroup, all rows (at most 16 MT): every weight is
// read once.
template <typename T, int MT>
__global__ __launch_bounds__(LIN_NT) void linear_rows_kernel(LinArgs a) {
  constexpr int ES = sizeof(T);
  __shared__ float red[LIN_NW * 256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16;
  const uint32_t rowb = (uint32_t)(a.K * ES), k16 = (uint32_t)(lane >> 4) * 16u;
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc((const char*)a.w + (long long)n0 * a.K * ES, 16u * rowb);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)a.M * rowb);
  const uint32_t woff[1] = {(uint32_t)(lane & 15) * rowb + k16};
  uint32_t aoff[1][MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    aoff[0][m] = (uint32_t)min(m * 16 + (lane & 15), a.M - 1) * rowb + k16;
  f32x4 acc[MT][1];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0] = f32x4{0, 0, 0, 0};
  stream_product<T, MT, 1, 1, STREAM_CS<MT>, LIN_NW, 2>(acc, wr, woff, xr, aoff, a.K * ES, wave);
  stream_reduce<MT, 1, LIN_NW>(acc, red, [&](int mt, int m, int c, const float* v) {
    const int r = mt * 16 + m, n = n0 + c;
    if (r >= a.M) return;
    const long long at = (long long)r * a.N + n;
    const float z = a.bias != nullptr ? v[0] + a.bias[n] : v[0];
    if (a.z != nullptr) lin_store<T>(a.z, at, z);
    float y = act_value(z, a.act);
    if (a.residual != nullptr) y += lin_load<T>(a.residual, at);
    lin_store<T>(a.y, at, y);
  });
}

template <typename T>
int launch_rows(const LinArgs& a, hipStream_t s, const char* fn) {
  const dim3 grid(a.N / 16), block(LIN_NT);
  if (a.M <= 16) hipLaunchKernelGGL((linear_rows_kernel<T, 1>), grid, block, 0, s, a);
  else if (a.M <= 32) hipLaunchKernelGGL((linear_rows_kernel<T, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((linear_rows_kernel<T, 4>), grid, block, 0, s, a);
  return moe_check_launch(fn);
}

// ---------------------------------------------------------------- dz and db
// dz = dy act'(z) and, per block of rows, the column sums of the unrounded
// dz.  A thread owns 8 columns (16 bytes of bf16) and walks the block's rows
// 8 apart; the 8 threads of a column chunk are summed through LDS in order.
constexpr int DZ_COLS = 256;   // columns of a workgroup: 32 threads of 8
constexpr int DZ_MAX_PARTS = 128;

int dz_rows(int M) {           // rows of a block: at least 64, at most 128 blocks
  const int r = (M + DZ_MAX_PARTS - 1) / DZ_MAX_PARTS;
  return r < 64 ? 64 : (r + 7) / 8 * 8;
}

template <typename T>
__global__ __launch_bounds__(256) void linear_dz_kernel(const T* __restrict__ dy,
                                                        const T* __restrict__ z,
                                                        T* __restrict__ dz,
                                                        float* __restrict__ part, int M, int N,
                                                        int act, int rows) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ float red[8][DZ_COLS];
  const int cc = threadIdx.x & 31, rr = threadIdx.x >> 5;
  const int c = blockIdx.x * DZ_COLS + cc * 8;
  const int m0 = blockIdx.y * rows, m1 = min(M, m0 + rows);
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  if (c < N)
    for (int m = m0 + rr; m < m1; m += 8) {
      const long long at = (long long)m * N + c;
      float d[8], v[8];
#pragma unroll
      for (int q = 0; q < 8; q += VEC) unpack16(*(const u32x4*)(dy + at + q), d + q, T());
      if (z != nullptr) {
#pragma unroll
        for (int q = 0; q < 8; q += VEC) unpack16(*(const u32x4*)(z + at + q), v + q, T());
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= act_slope(v[i], act);
#pragma unroll
        for (int q = 0; q < 8; q += VEC) *(u32x4*)(dz + at + q) = pack16(d + q, T());
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
    }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rr][cc * 8 + i] = sum[i];
  __syncthreads();
  const int n = blockIdx.x * DZ_COLS + threadIdx.x;
  if (n < N) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += red[r][threadIdx.x];
    part[(long long)blockIdx.y * N + n] = s;
  }
}

// db = sum of the blocks' column sums, in block order
__global__ __launch_bounds__(256) void linear_db_kernel(const float* __restrict__ part, int parts,
                                                        int N, float* __restrict__ db) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  double s = 0;
  for (int p = 0; p < parts; ++p) s += part[(long long)p * N + n];
  db[n] = (float)s;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// 256 x 256 tiles of an M x N product
long long big_tiles(long long M, long long N) { return ((M + 255) / 256) * ((N + 255) / 256); }
bool fwd_big(int M, int N) { return big_tiles(M, N) >= LIN_BIG_TILES; }
bool bwd_big(int M, int N, int K) { return big_tiles(M, K) + big_tiles(N, K) >= LIN_BIG_TILES; }

size_t fwd_ws(int M, int N, int K, int dt) {
  return M <= LIN_FEW_ROWS || fwd_big(M, N) ? 0 : round256(moe_dense_fwd_bytes(M, N, K, dt));
}

struct BwdWs {
  size_t part, dz, dense, total;
  int rows, parts;
};
BwdWs bwd_ws(int M, int N, int K, int dt, int act) {
  BwdWs w;
  w.rows = dz_rows(M);
  w.parts = (M + w.rows - 1) / w.rows;
  w.part = 0;
  w.dz = round256((size_t)w.parts * N * 4);
  w.dense = w.dz + (act == MOE_ACT_NONE ? 0 : round256((size_t)M * N * moe_dt_bytes(dt)));
  w.total = w.dense + (bwd_big(M, N, K) ? 0 : round256(moe_dense_bwd_bytes(M, N, K, dt)));
  if (w.total == 0) w.total = 256;
  return w;
}

int lin_checks(const char* fn, int dt, int M, int N, int K, int act) {
  MOE_TRY(moe_need_dt(dt, fn));
  MOE_TRY(moe_need_nonneg(M, fn, "M"));
  MOE_TRY(moe_need_mult64(N, fn, "N"));
  MOE_TRY(moe_need_mult64(K, fn, "K"));
  if (act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: act %d is none of the MOE_ACT values", fn, act);
  const int es = moe_dt_bytes(dt);
  MOE_TRY(moe_need_elems(M, K, es, fn, "x"));
  MOE_TRY(moe_need_elems(M, N, es, fn, "y"));
  MOE_TRY(moe_need_elems(N, K, es, fn, "w"));
  return MOE_OK;
}

// the tile kernels' byte offsets stay below the one that stands for "no load"
int lin_tile_checks(const char* fn, int dt, int M, int N, int K) {
  const long long es = moe_dt_bytes(dt), most = 0x80000000LL;
  if ((long long)M * K * es >= most || (long long)M * N * es >= most ||
      (long long)N * K * es >= most)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: x, w or y of 2 GiB or more (M=%d N=%d K=%d)", fn, M,
                    N, K);
  return MOE_OK;
}

}  // namespace

extern "C" size_t moe_linear_workspace_bytes(int M, int N, int K, int dt) {
  if (lin_checks("moe_linear_workspace_bytes", dt, M, N, K, MOE_ACT_NONE) != MOE_OK) return 0;
  return fwd_ws(M, N, K, dt);
}

extern "C" int moe_linear(const void* x, int dt, int M, int N, int K, const void* w,
                          const float* bias, int act, const void* residual, void* z, void* y,
                          void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* fn = "moe_linear";
  MOE_TRY(lin_checks(fn, dt, M, N, K, act));
  if (M == 0) return MOE_OK;
  MOE_TRY(moe_need_ptr(x, fn, "x"));
  MOE_TRY(moe_need_ptr(w, fn, "w"));
  MOE_TRY(moe_opt_ptr(bias, fn, "bias"));
  MOE_TRY(moe_opt_ptr(residual, fn, "residual"));
  MOE_TRY(moe_opt_ptr(z, fn, "z"));
  MOE_TRY(moe_need_ptr(y, fn, "y"));
  if (y == x || z == x || (z != nullptr && (z == y || z == residual)))
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: y and z need buffers of their own (y may be residual's)",
                    fn);
  hipStream_t s = (hipStream_t)stream;
  if (M <= LIN_FEW_ROWS) {
    LinArgs a = {x, w, bias, residual, z, y, M, N, K, act};
    return dt == MOE_BF16 ? launch_rows<bf16_t>(a, s, fn) : launch_rows<float>(a, s, fn);
  }
  MOE_TRY(lin_tile_checks(fn, dt, M, N, K));
  const size_t need = fwd_ws(M, N, K, dt);
  if (need > 0) MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  if (ws_bytes < need)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes, need);
  if (!fwd_big(M, N))
    return moe_dense_fwd(x, dt, M, N, K, w, bias, act, residual, z, y, ws, s);
  return moe_gmm_linear_fwd(x, dt, M, N, K, w, bias, act, residual, z, y, s);
}

extern "C" size_t moe_linear_bwd_workspace_bytes(int M, int N, int K, int dt, int act) {
  if (lin_checks("moe_linear_bwd_workspace_bytes", dt, M, N, K, act) != MOE_OK) return 0;
  return bwd_ws(M, N, K, dt, act).total;
}

extern "C" int moe_linear_bwd(const void* dy, const void* z, const void* x, const void* w, int dt,
                              int M, int N, int K, int act, void* dx, void* dw, float* db,
                              void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* fn = "moe_linear_bwd";
  MOE_TRY(lin_checks(fn, dt, M, N, K, act));
  MOE_TRY(lin_tile_checks(fn, dt, M, N, K));
  MOE_TRY(moe_opt_ptr(dx, fn, "dx"));
  MOE_TRY(moe_opt_ptr(dw, fn, "dw"));
  MOE_TRY(moe_opt_ptr(db, fn, "db"));
  const BwdWs lay = bwd_ws(M, N, K, dt, act);
  if (M > 0) {
    MOE_TRY(moe_need_ptr(dy, fn, "dy"));
    if (act != MOE_ACT_NONE) MOE_TRY(moe_need_ptr(z, fn, "z"));
    if (dw != nullptr) MOE_TRY(moe_need_ptr(x, fn, "x"));
    if (dx != nullptr) MOE_TRY(moe_need_ptr(w, fn, "w"));
    if (dx != nullptr && (dx == dy || dx == z || dx == x))
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: dx needs a buffer of its own", fn);
    MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
    if (ws_bytes < lay.total)
      return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                      lay.total);
  }
  if (dx == nullptr && dw == nullptr && db == nullptr) return MOE_OK;
  hipStream_t s = (hipStream_t)stream;
  const void* dz = dy;
  if (M > 0 && (act != MOE_ACT_NONE || db != nullptr)) {
    void* out = act != MOE_ACT_NONE ? (char*)ws + lay.dz : nullptr;
    const void* zz = act != MOE_ACT_NONE ? z : nullptr;
    float* part = db != nullptr ? (float*)((char*)ws + lay.part) : nullptr;
    const dim3 grid((N + DZ_COLS - 1) / DZ_COLS, lay.parts);
    if (dt == MOE_BF16)
      hipLaunchKernelGGL(linear_dz_kernel<bf16_t>, grid, dim3(256), 0, s, (const bf16_t*)dy,
                         (const bf16_t*)zz, (bf16_t*)out, part, M, N, act, lay.rows);
    else
      hipLaunchKernelGGL(linear_dz_kernel<float>, grid, dim3(256), 0, s, (const float*)dy,
                         (const float*)zz, (float*)out, part, M, N, act, lay.rows);
    MOE_TRY(moe_check_launch(fn));
    if (out != nullptr) dz = out;
  }
  if (db != nullptr) {
    hipLaunchKernelGGL(linear_db_kernel, dim3((N + 255) / 256), dim3(256), 0, s,
                       (const float*)((char*)ws + lay.part), M > 0 ? lay.parts : 0, N, db);
    MOE_TRY(moe_check_launch(fn));
  }
  if (M > 0 && !bwd_big(M, N, K))
    return moe_dense_bwd(dz, x, w, dt, M, N, K, dx, dw, (char*)ws + lay.dense, s);
  return moe_gmm_linear_bwd(dz, x, w, dt, M, N, K, dx, dw, s);
}
