// A matrix product with bias, activation and residual in its epilogue, and
// its gradients:
//   z = x W^T + b,  y = act(z) + residual           (x [M,K], W [N,K])
//   dz = dy * act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
// Few rows (decode batches) run as a stream of W (stream.hpp); large products
// run on the grouped GEMM's 256 x 256 tiles (gmm.hip), those between on
// smaller tiles (dense.hip).  The epilogues take the bias, activation and
// residual, and the two products of the backward share one launch.  What is
// here: the few-row kernel, the elementwise half of the backward, the checks
// and the choice between the kernels.
#include <type_traits>

#include "act.hpp"
#include "stream.hpp"
#include "validate.hpp"

namespace {

// Rows of the streaming kernel, at most: up to 16 it always runs; up to 64 but
// where N is short and K long, for then its workgroups, one per 16 columns, are
// few and read for long, and the K slices of dense.hip end sooner (37 x 2048 x
// 7680: 18.3 us streaming, 12.6 in slices; 64 x 4096 x 4096: 13.8 and 14.7; 33 x
// 2048 x 2048 fp32: 12.1 and 13.1; 17 x 1024 x 1024: 7.8 and 11.6).
bool few_rows(int M, int N, int K, int dt) {
  return M <= 16 || (M <= 64 && (N >= 4096 || (long long)K * moe_dt_bytes(dt) <= 8192));
}
constexpr int LIN_NW = 4;
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

// NT x 16 output columns per workgroup and all rows, at most 8 AC: every weight
// is read once.  The four waves split K (stream.hpp) and keep D steps of copies
// in flight each, AC of them for the rows' operand; their partial tiles are
// summed through LDS in wave order (the same bits on every run).  Rows of a
// 16-row tile beyond 8 AC hold whatever the LDS held: their results are dropped.
template <typename T, int AC, int NT, int D>
__global__ __launch_bounds__(LIN_NT) void linear_rows_kernel(LinArgs a) {
  constexpr int ES = sizeof(T), MT = (AC + 1) / 2, OPS = 2 * NT + AC;
  constexpr int SLOT = (NT + MT) * STREAM_TILE;
  __shared__ __attribute__((aligned(1024))) char smem[LIN_NW * D * SLOT];
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  const int n0 = blockIdx.x * 16 * NT;
  const int ld = a.K * ES, steps = (ld / STREAM_STEP - wave + LIN_NW - 1) / LIN_NW;
  const i32x4 rw = raw_rsrc((const char*)a.w + (long long)n0 * ld, 16u * NT * (uint32_t)ld);
  const i32x4 rx = raw_rsrc(a.x, (uint32_t)a.M * (uint32_t)ld);
  uint32_t wo[2], xo[AC];
#pragma unroll
  for (int j = 0; j < 2; ++j) wo[j] = (uint32_t)(stream_row(j) * ld) + stream_chunk(j);
#pragma unroll
  for (int j = 0; j < AC; ++j)
    xo[j] = stream_row(j) < a.M ? (uint32_t)(stream_row(j) * ld) + stream_chunk(j & 1) : STREAM_OOB;
  char* const ring = smem + wave * D * SLOT;
  const uint32_t lds = lds_addr(ring);
  int k = wave * STREAM_STEP, left = steps;
  uint32_t slot = 0;
  // (steps past the last go through an empty range, so that every step waits
  // for the same number of copies)
  auto copy = [&]() {
    const int live = uniform(left > 0 ? -1 : 0);
    const i32x4 w = {uniform(rw.x), uniform(rw.y), uniform(rw.z & live), MOE_RSRC_DW3};
    const i32x4 x = {uniform(rx.x), uniform(rx.y), uniform(rx.z & live), MOE_RSRC_DW3};
    const uint32_t p = (uint32_t)uniform((int)(lds + slot));
    const int k0 = uniform(k & live);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        dma16_nt(w, p + t * STREAM_TILE + j * 1024, wo[j], (k0 + t * 16 * ld) & live);
#pragma unroll
    for (int j = 0; j < AC; ++j) dma16(x, p + NT * STREAM_TILE + j * 1024, xo[j], k0);
    slot = (uint32_t)uniform((int)(slot + SLOT == D * SLOT ? 0 : slot + SLOT));
    k = uniform(k + LIN_NW * STREAM_STEP);
    left = uniform(left + live);
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
  const int f[2] = {stream_frag(0), stream_frag(1)};
#pragma unroll
  for (int d = 0; d < D - 1; ++d) copy();
  uint32_t rs = 0;
  for (int i = 0; i < steps; ++i) {
    copy();                        // into the slot read last
    vm_drain<(D - 1) * OPS>();
    const char* p = ring + rs;
    rs = (uint32_t)uniform((int)(rs + SLOT == D * SLOT ? 0 : rs + SLOT));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 w[NT], x[MT];
#pragma unroll
      for (int t = 0; t < NT; ++t) w[t] = *(const u32x4*)(p + t * STREAM_TILE + f[h]);
#pragma unroll
      for (int m = 0; m < MT; ++m) x[m] = *(const u32x4*)(p + (NT + m) * STREAM_TILE + f[h]);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = stream_mma(x[m], w[t], acc[m][t], T());
    }
    lds_drain();                   // the slot is read
  }
  vm_drain<0>();                   // (empty copies)
  __syncthreads();
  // partial tiles: [wave][tile][register][lane]
  float* const red = (float*)smem;
  static_assert(MT * NT * 1024 <= D * SLOT, "partial tiles fit the ring");
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[((wave * MT + m) * NT + t) * 256 + q * 64 + lane] = acc[m][t][q];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NT * 256; i += LIN_NT) {
    float v = red[i];
#pragma unroll
    for (int w = 1; w < LIN_NW; ++w) v += red[w * MT * NT * 256 + i];
    // register q of lane l: row 4 (l / 16) + q, column l % 16
    const int tile = i >> 8, q = (i >> 6) & 3, l = i & 63;
    const int r = tile / NT * 16 + 4 * (l >> 4) + q, n = n0 + tile % NT * 16 + (l & 15);
    if (r >= a.M) continue;
    const long long at = (long long)r * a.N + n;
    const float z = a.bias != nullptr ? v + a.bias[n] : v;
    if (a.z != nullptr) lin_store<T>(a.z, at, z);
    float y = act_value(z, a.act);
    if (a.residual != nullptr) y += lin_load<T>(a.residual, at);
    lin_store<T>(a.y, at, y);
  }
}

template <typename T, int AC, int NT, int D>
int launch_rows(const LinArgs& a, hipStream_t s, const char* fn) {
  hipLaunchKernelGGL((linear_rows_kernel<T, AC, NT, D>), dim3(a.N / (16 * NT)), dim3(LIN_NT), 0, s,
                     a);
  return moe_check_launch(fn);
}

// Two 16-column tiles per workgroup halve what is read of x, once there are
// columns enough to fill most of the chip that way (24 x 7680 x 7680: 23.8 us,
// one tile 29.7; 64 x 4096 x 4096: 17.9, one tile 13.8).
constexpr int LIN_TWO_N = 6144;
template <typename T>
int linear_rows(const LinArgs& a, hipStream_t s, const char* fn) {
  const bool two = a.M > 16 && a.N >= LIN_TWO_N;
  if (a.M <= 8) return launch_rows<T, 1, 1, 5>(a, s, fn);
  if (a.M <= 16) return launch_rows<T, 2, 1, 5>(a, s, fn);
  if (a.M <= 32)
    return two ? launch_rows<T, 4, 2, 4>(a, s, fn) : launch_rows<T, 4, 1, 3>(a, s, fn);
  if (a.M <= 48)
    return two ? launch_rows<T, 6, 2, 3>(a, s, fn) : launch_rows<T, 6, 1, 2>(a, s, fn);
  return two ? launch_rows<T, 8, 2, 3>(a, s, fn) : launch_rows<T, 8, 1, 2>(a, s, fn);
}

// ---------------------------------------------------------------- dz and db
// dz is rounded to the storage type, as every matrix that the matrix cores read
// here is: in bf16 that is half a step more in dx and dW (0.0023 of their size
// off instead of 0.0017), and holding dz as two bf16 would double both products,
// which are all of the time of a large call.  db sums the unrounded values.
//
// dz = dy act'(z) and, per block of rows, the column sums of the unrounded
// dz.  A thread owns 8 columns (16 bytes of bf16) and walks the block's rows
// 8 apart; the 8 threads of a column chunk are summed through LDS in order.
constexpr int DZ_COLS = 256;   // columns of a workgroup: 32 threads of 8
constexpr int DZ_MAX_PARTS = 128;

// Rows of a block, a multiple of the 8 threads that share a column chunk: as few
// as give 512 workgroups work, at most 128 blocks.
int dz_rows(int M, int N) {
  const int cols = (N + DZ_COLS - 1) / DZ_COLS;
  const int want = (512 + cols - 1) / cols;               // blocks
  const int parts = want < DZ_MAX_PARTS ? want : DZ_MAX_PARTS;
  const int r = (M + parts - 1) / parts;
  return r < 8 ? 8 : (r + 7) / 8 * 8;
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

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// The 256 x 256 tiles of the grouped GEMM (bf16; in fp32 the smaller ones are
// faster throughout) pay once there are enough of them for the 256 CUs.
// Measured, smaller tiles against these: 2048 x 4096 x 4096 (128 tiles) 73 and
// 137 us, 2000 x 8192 x 2048 (256) 83 and 83, 4096^3 (256) 146 and 135, 8191 x
// 2048 x 7680 (256) 308 and 236.
constexpr int LIN_BIG_TILES = 192;
long long big_tiles(long long M, long long N) { return ((M + 255) / 256) * ((N + 255) / 256); }
bool fwd_big(int M, int N, int dt) {
  return dt == MOE_BF16 && big_tiles(M, N) >= LIN_BIG_TILES;
}

// The backward's two products share a launch, so what counts is their tiles
// together.  Where a dx tile (N deep) would take more than 3 times a workgroup's
// share of the work, dx goes to the smaller tiles in slices, in a launch of its
// own (1000 x 7680 x 2048: 100 us, 203 together, 177 all in smaller tiles; 200 x
// 8192 x 8192: 122, 236 and 324), and where a dW tile (M deep) would take more
// than its share, M is cut into `runs` (8192 x 2048 x 2048: 228 us, 302 in one
// run).
struct BwdBig {
  bool dx, dw;    // these tiles for this product
  int runs;
};
BwdBig bwd_big(int M, int N, int K, int dt) {
  const long long tx = big_tiles(M, K), tw = big_tiles(N, K);
  const double share = ((double)tx * N + (double)tw * M) / 256;   // in K elements
  BwdBig b = {false, false, 1};
  if (dt != MOE_BF16 || tx + tw < LIN_BIG_TILES) return b;
  b.dx = N <= 3 * share;
  b.dw = b.dx || tw >= LIN_BIG_TILES;
  while (b.dx && b.runs < 8 && M / b.runs > 1.3 * share && M / b.runs >= 1024) b.runs *= 2;
  return b;
}

size_t fwd_ws(int M, int N, int K, int dt) {
  return few_rows(M, N, K, dt) || fwd_big(M, N, dt) ? 0
                                                    : round256(moe_dense_fwd_bytes(M, N, K, dt));
}

struct BwdWs {
  size_t part, dz, dense, total;
  int rows, parts;
  BwdBig big;
};
BwdWs bwd_ws(int M, int N, int K, int dt, int act) {
  BwdWs w;
  w.rows = dz_rows(M, N);
  w.parts = (M + w.rows - 1) / w.rows;
  w.part = 0;
  w.dz = round256((size_t)w.parts * N * 4);
  w.dense = w.dz + (act == MOE_ACT_NONE ? 0 : round256((size_t)M * N * moe_dt_bytes(dt)));
  w.big = bwd_big(M, N, K, dt);
  w.total = w.dense + round256(!w.big.dx ? moe_dense_bwd_bytes(M, N, K, dt, w.big.dw)
                               : w.big.runs > 1 ? (size_t)w.big.runs * N * K * 4 : 0);
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
  const bool few = few_rows(M, N, K, dt);
  if (!few) MOE_TRY(lin_tile_checks(fn, dt, M, N, K));
  const size_t need = fwd_ws(M, N, K, dt);
  if (need > 0) MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  if (ws_bytes < need)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes, need);
  // (the products read x and W to the end of the launch; a residual that y is
  // written over is read by the thread that writes, so only element for element)
  const long long es = moe_dt_bytes(dt), mn = (long long)M * N * es;
  const MoeRange rx = {x, (long long)M * K * es, "x"}, rw = {w, (long long)N * K * es, "w"},
                 rb = {bias, 4LL * N, "bias"}, rr = {residual, mn, "residual"}, rz = {z, mn, "z"},
                 ry = {y, mn, "y"}, rs = {need > 0 ? ws : nullptr, (long long)need, "ws"};
  const char* with = moe_shares(ry, {rx, rw, rb, rz, rs});
  if (with == nullptr && residual != y) with = moe_shares(ry, {rr});
  const char* out = "y";
  if (with == nullptr) {
    with = moe_shares(rz, {rx, rw, rb, rr, rs});
    out = "z";
  }
  if (with == nullptr) {
    with = moe_shares(rs, {rx, rw, rb, rr});
    out = "ws";
  }
  if (with != nullptr)
    return moe_fail(MOE_ERR_INVALID_ARG,
                    "%s: %s overlaps %s (y and z need buffers of their own; y may be residual's)", fn,
                    out, with);
  hipStream_t s = (hipStream_t)stream;
  if (few) {
    LinArgs a = {x, w, bias, residual, z, y, M, N, K, act};
    return dt == MOE_BF16 ? linear_rows<bf16_t>(a, s, fn) : linear_rows<float>(a, s, fn);
  }
  if (!fwd_big(M, N, dt))
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
    // (both products read dy or dz, and x or W, to the end of the launch, and
    // the outputs are written side by side)
    const long long es = moe_dt_bytes(dt), mn = (long long)M * N * es, mk = (long long)M * K * es,
                    nk = (long long)N * K * es;
    const MoeRange rdy = {dy, mn, "dy"}, rz = {z, mn, "z"}, rx = {x, mk, "x"}, rw = {w, nk, "w"},
                   outs[] = {{dx, mk, "dx"}, {dw, nk, "dw"}, {db, 4LL * N, "db"}};
    for (int i = 0; i < 3; ++i) {
      const char* with = moe_shares(outs[i], {rdy, rz, rx, rw});
      for (int j = 0; j < i && with == nullptr; ++j) with = moe_shares(outs[i], {outs[j]});
      if (with != nullptr)
        return moe_fail(MOE_ERR_INVALID_ARG, "%s: %s needs a buffer of its own, it overlaps %s", fn,
                        outs[i].name, with);
    }
    MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
    if (ws_bytes < lay.total)
      return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                      lay.total);
    const bool any = dx != nullptr || dw != nullptr || db != nullptr;
    const char* with = any ? moe_shares({ws, (long long)lay.total, "ws"},
                                        {rdy, rz, rx, rw, outs[0], outs[1], outs[2]}) : nullptr;
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: ws overlaps %s", fn, with);
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
  const float* const sums = (const float*)((char*)ws + lay.part);
  const int parts = M > 0 ? lay.parts : 0;
  char* const dense = (char*)ws + lay.dense;
  if (M > 0 && !lay.big.dx) {
    MOE_TRY(moe_dense_bwd(dz, x, w, dt, M, N, K, dx, lay.big.dw ? nullptr : dw, lay.big.dw, sums,
                          parts, db, dense, s));
    if (!lay.big.dw) return MOE_OK;
    dx = nullptr;
  } else if (db != nullptr) {
    MOE_TRY(moe_dense_db(sums, parts, N, db, s));
  }
  const int runs = M > 0 ? lay.big.runs : 1;
  MOE_TRY(moe_gmm_linear_bwd(dz, x, w, dt, M, N, K, dx, dw, runs, (float*)dense, s));
  return runs > 1 && dw != nullptr ? moe_dense_sum((const float*)dense, runs, N, K, dt, dw, s)
                                   : MOE_OK;
}
