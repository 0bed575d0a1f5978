// The whole expert layer for a few tokens (serving): router projection,
// softmax top-k, the chosen SwiGLU experts, the shared expert, the
// gate-weighted sum and the residual.  For at most 128 tokens the layer is a
// stream of the chosen experts' weights; sorting rows into groups, as the
// training path does, would be latency only, so the rows of an expert are
// found from the token's choices directly and the products read tokens in
// place (stream.hpp).
#include <type_traits>

#include "route_select.hpp"
#include "stream.hpp"
#include "validate.hpp"

namespace {

constexpr int DEC_MAX_T = 128;       // tokens of a call
constexpr int DEC_MAX_PAIRS = 4096;  // (token, slot) pairs of a call
constexpr int DEC_NW = 8;            // waves of a workgroup of the expert products
constexpr int DEC_NT = 64 * DEC_NW;
constexpr int DEC_GU = 16;           // gate/up columns of a unit (16 gate and 16 up rows of W13)
constexpr int DEC_DN = 32;           // output columns of a unit of the second product
constexpr int RT_NW = 4;             // waves of a router workgroup
constexpr int RT_COLS = 16;          // experts of a router workgroup
constexpr int RT_MAX_S = 32;         // K slices of the router product

typedef double f64x4 __attribute__((ext_vector_type(4)));

struct DecArgs {
  const void* x; const float* wg; const float* bias;
  int T, H, I, E, k, g0, G, shared;
  const void* w13; const void* w2; const void* ws13; const void* ws2; const void* residual;
  float* logits; int32_t* idx; float* gate; void* y;
  int S;              // K slices of the router product (0: logits are an input)
  double* part;       // [S][T][E] partial logits
  void* act;          // [planes][T k + T][I] activations, shared rows last
  float* yp;          // [T k + T][H] expert outputs
};

// 8 elements of T as fp32, from byte offset off
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t off, float* v, bf16_t) {
  unpack16(buf_load16(r, off), v, bf16_t());
}
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t off, float* v, float) {
  unpack16(buf_load16(r, off), v, 0.f);
  unpack16(buf_load16(r, off + 16), v + 4, 0.f);
}

// ---------------------------------------------------------------- router
// part[s][t][e] = sum over the K slice s of x[t, h] Wg[h, e], in fp64: a
// product of an fp32 and a bf16 (or fp32) value is exact there, so the logits
// are rounded once, to fp32, and experts whose logits nearly tie are ordered
// as their exact values are.  Work is 16 experts x one K slice per workgroup;
// lane l of a wave holds Wg[h0 + 8 (l / 16) + i][l % 16] and x[l % 16][..] for
// i = 0..7, eight MFMAs of 4 K values each.  MT: 16-token tiles.
template <typename T, int MT>
__global__ __launch_bounds__(64 * RT_NW) void decode_router_kernel(DecArgs a) {
  constexpr int ES = sizeof(T);
  __shared__ double red[RT_NW][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, kg = lane >> 4;
  const int e0 = blockIdx.x * RT_COLS, slice = blockIdx.y;
  const int e = min(e0 + c, a.E - 1);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)((long long)a.T * a.H * ES));
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.wg, clamp_bytes((long long)a.H * a.E * 4));
  f64x4 acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f64x4{0, 0, 0, 0};
  // steps of 32 K values, dealt to the waves of all slices in turn
  const int nw = a.S * RT_NW;
  for (int s = slice * RT_NW + wave; s < a.H / 32; s += nw) {
    const int h = s * 32 + 8 * kg;
    float w[8], x[MT][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = __uint_as_float(buf_load4(wr, (uint32_t)((h + i) * a.E + e) * 4u));
#pragma unroll
    for (int m = 0; m < MT; ++m)
      load8(xr, (uint32_t)(min(m * 16 + c, a.T - 1) * a.H + h) * ES, x[m], T());
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[m] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[m][i], (double)w[i], acc[m], 0, 0,
                                                      0);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][r][lane] = acc[m][r];
    __syncthreads();
    // register r of the fp64 tile: row 4 r + lane / 16, column lane % 16
    const int r = threadIdx.x >> 6;
    double s = red[0][r][lane];
#pragma unroll
    for (int w = 1; w < RT_NW; ++w) s += red[w][r][lane];
    const int t = m * 16 + 4 * r + (lane >> 4);
    if (t < a.T && e0 + c < a.E) a.part[((long long)slice * a.T + t) * a.E + e0 + c] = s;
  }
}

// One wave per token: the logits (sum of the partials and the bias, rounded
// once to fp32), the k largest and their softmax weights.
template <int V>
__device__ __forceinline__ void decode_route_token(const DecArgs& a, int t) {
  const int lane = threadIdx.x & 63;
  float v[V];
  uint32_t key[V];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + i * MOE_WAVE;
    v[i] = -INFINITY;
    if (e < a.E) {
      if (a.S > 0) {
        double s = 0;
        for (int p = 0; p < a.S; ++p) s += a.part[((long long)p * a.T + t) * a.E + e];
        if (a.bias != nullptr) s += (double)a.bias[e];
        v[i] = (float)s;
        a.logits[(long long)t * a.E + e] = v[i];
      } else {
        v[i] = a.logits[(long long)t * a.E + e];
      }
    }
    key[i] = e < a.E ? route_key(v[i]) : 0u;
    m = fmaxf(m, v[i]);
  }
  m = wave_max(m);
  const bool none = m == -INFINITY;   // every expert masked: gates of zero, not NaN
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += lane + i * MOE_WAVE < a.E ? expf(v[i] - m) : 0.f;
  s = wave_sum(s);
  const float inv = 1.0f / s;
  route_select<V>(key, a.k, [&](int slot, int i) {
    a.idx[(long long)t * a.k + slot] = lane + i * MOE_WAVE;
    a.gate[(long long)t * a.k + slot] = none ? 0.f : expf(v[i] - m) * inv;
  });
}

template <int V>
__global__ __launch_bounds__(256) void decode_route_kernel(DecArgs a) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < a.T) decode_route_token<V>(a, t);
}

// ---------------------------------------------------------------- experts
struct DecLds {
  int16_t loc[DEC_MAX_PAIRS];   // window index of each pair's expert, -1 outside it
  int16_t list[MOE_MAX_E];      // window indices of the experts some token chose, ascending
  int n_list;
  int rows[DEC_MAX_T];          // rows of the current unit: pair indices, or T k + token
  int n_rows;
  float red[DEC_NW * 2 * 256];
};

// loc and list of the call, by every workgroup for itself.
__device__ __forceinline__ void decode_plan(const DecArgs& a, DecLds& l) {
  const int P = a.T * a.k;
  int* const flag = (int*)l.red;
  for (int g = threadIdx.x; g < a.G; g += DEC_NT) flag[g] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += DEC_NT) {
    const int g = a.idx[p] - a.g0;
    const bool in = g >= 0 && g < a.G;
    l.loc[p] = in ? (int16_t)g : (int16_t)-1;
    if (in) flag[g] = 1;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int n = 0;
    for (int g0 = 0; g0 < a.G; g0 += 64) {
      const int g = g0 + threadIdx.x;
      const bool on = g < a.G && flag[g];
      const unsigned long long b = __ballot(on);
      if (on) l.list[n + __popcll(b & ((1ull << threadIdx.x) - 1))] = (int16_t)g;
      n += __popcll(b);
    }
    if (threadIdx.x == 0) l.n_list = n;
  }
  __syncthreads();
}

// Rows of the unit's expert: window index g, or the shared expert (g < 0).
// Begins and ends with a barrier.
__device__ __forceinline__ void decode_rows(const DecArgs& a, DecLds& l, int g) {
  __syncthreads();
  const int P = a.T * a.k;
  if (g < 0) {
    for (int t = threadIdx.x; t < a.T; t += DEC_NT) l.rows[t] = P + t;
    if (threadIdx.x == 0) l.n_rows = a.T;
  } else if (threadIdx.x < 64) {
    int n = 0;
    for (int p0 = 0; p0 < P; p0 += 64) {
      const int p = p0 + threadIdx.x;
      const bool on = p < P && l.loc[p] == g;
      const unsigned long long b = __ballot(on);
      // (a token chooses an expert once, so at most T <= DEC_MAX_T rows)
      if (on) l.rows[n + __popcll(b & ((1ull << threadIdx.x) - 1))] = p;
      n += __popcll(b);
    }
    if (threadIdx.x == 0) l.n_rows = n;
  }
  __syncthreads();
}

// silu(g) u; the sum of two bf16 that the second product reads carries 16
// bits of it, so its rounding does not show beside that of the result
__device__ __forceinline__ float decode_swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

template <typename T> constexpr int DEC_PLANES = sizeof(T) == 2 ? 2 : 1;

// act[row, i0 .. i0 + 15] of the unit's rows.
template <typename T, int MT>
__device__ __forceinline__ void decode_gateup(const DecArgs& a, DecLds& l, int g, int i0) {
  constexpr int ES = sizeof(T);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int P = a.T * a.k, n = l.n_rows;
  const char* w = (g < 0 ? (const char*)a.ws13 : (const char*)a.w13 + (long long)g * 2 * a.I * a.H * ES) +
                  (long long)i0 * a.H * ES;
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(w, (uint32_t)((long long)(2 * a.I - i0) * a.H * ES));
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)((long long)a.T * a.H * ES));
  const uint32_t k16 = (uint32_t)(lane >> 4) * 16u;
  const uint32_t row0 = (uint32_t)(lane & 15) * (uint32_t)(a.H * ES) + k16;
  const uint32_t woff[2] = {row0, row0 + (uint32_t)a.I * (uint32_t)(a.H * ES)};
  uint32_t aoff[1][MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = l.rows[min(m * 16 + (lane & 15), n - 1)];
    const int t = r >= P ? r - P : r / a.k;
    aoff[0][m] = (uint32_t)t * (uint32_t)(a.H * ES) + k16;
  }
  f32x4 acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4{0, 0, 0, 0};
  stream_product<T, MT, 2, 1, STREAM_CS<MT>, DEC_NW, 2>(acc, wr, woff, xr, aoff, a.H * ES, wave);
  T* const act = (T*)a.act;
  stream_reduce<MT, 2, DEC_NW>(acc, l.red, [&](int mt, int m, int c, const float* v) {
    const int r = mt * 16 + m;
    if (r >= n) return;
    const float s = decode_swiglu(v[0], v[1]);
    const long long at = (long long)l.rows[r] * a.I + i0 + c;
    if constexpr (sizeof(T) == 2) {
      const uint32_t hi = f32_to_bf16(s);
      act[at] = (T)hi;
      act[(long long)(P + a.T) * a.I + at] = (T)f32_to_bf16(s - bf16_to_f32(hi));
    } else {
      act[at] = s;
    }
  });
}

// yp[row, h0 .. h0 + 31] of the unit's rows.
template <typename T, int MT>
__device__ __forceinline__ void decode_down(const DecArgs& a, DecLds& l, int g, int h0) {
  constexpr int ES = sizeof(T), AP = DEC_PLANES<T>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int P = a.T * a.k, n = l.n_rows;
  const char* w = (g < 0 ? (const char*)a.ws2 : (const char*)a.w2 + (long long)g * a.H * a.I * ES) +
                  (long long)h0 * a.I * ES;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(w, (uint32_t)((long long)(a.H - h0) * a.I * ES));
  const long long plane = (long long)(P + a.T) * a.I * ES;
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.act, (uint32_t)(AP * plane));
  const uint32_t k16 = (uint32_t)(lane >> 4) * 16u, rowb = (uint32_t)(a.I * ES);
  const uint32_t woff[2] = {(uint32_t)(lane & 15) * rowb + k16, (uint32_t)(16 + (lane & 15)) * rowb + k16};
  uint32_t aoff[AP][MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int p = 0; p < AP; ++p)
      aoff[p][m] = (uint32_t)l.rows[min(m * 16 + (lane & 15), n - 1)] * rowb + k16 +
                   (uint32_t)(p * plane);
  f32x4 acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4{0, 0, 0, 0};
  stream_product<T, MT, 2, AP, STREAM_CS<MT>, DEC_NW, 2>(acc, wr, woff, ar, aoff, a.I * ES, wave);
  stream_reduce<MT, 2, DEC_NW>(acc, l.red, [&](int mt, int m, int c, const float* v) {
    const int r = mt * 16 + m;
    if (r >= n) return;
    float* const out = a.yp + (long long)l.rows[r] * a.H + h0 + c;
    out[0] = v[0];
    out[16] = v[1];
  });
}

// run f<MT> with the fewest 16-row tiles that hold the unit's rows
template <typename F>
__device__ __forceinline__ void decode_by_tiles(int n, F&& f) {
  if (n <= 16) f(std::integral_constant<int, 1>{});
  else if (n <= 32) f(std::integral_constant<int, 2>{});
  else if (n <= 64) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

template <typename T, bool DOWN>
__global__ __launch_bounds__(DEC_NT) void decode_expert_kernel(DecArgs a) {
  __shared__ DecLds l;
  decode_plan(a, l);
  const int per = DOWN ? a.H / DEC_DN : a.I / DEC_GU;
  const int total = (l.n_list + a.shared) * per;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int s = u / per, b = u % per;
    const int g = s < l.n_list ? l.list[s] : -1;
    decode_rows(a, l, g);
    decode_by_tiles(l.n_rows, [&](auto mt) {
      constexpr int MT = decltype(mt)::value;
      if constexpr (DOWN) decode_down<T, MT>(a, l, g, b * DEC_DN);
      else decode_gateup<T, MT>(a, l, g, b * DEC_GU);
    });
  }
}

// y[t, h] = residual + shared + sum_j gate yp[t, j], in that order
template <typename T>
__global__ __launch_bounds__(256) void decode_combine_kernel(DecArgs a) {
  const int h = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (h >= a.H) return;
  const long long at = (long long)t * a.H + h;
  float s = 0.f;
  if (a.residual != nullptr) {
    if constexpr (sizeof(T) == 2) s = bf16_to_f32(((const T*)a.residual)[at]);
    else s = ((const T*)a.residual)[at];
  }
  if (a.shared) s += a.yp[((long long)a.T * a.k + t) * a.H + h];
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j, g = a.idx[p] - a.g0;
    if (g >= 0 && g < a.G) s += a.gate[p] * a.yp[(long long)p * a.H + h];
  }
  if constexpr (sizeof(T) == 2) ((T*)a.y)[at] = (T)f32_to_bf16(s);
  else ((T*)a.y)[at] = s;
}

// ---------------------------------------------------------------- host side

// K slices of the router product: enough workgroups for the chip, each wave
// at least one step of 32
int router_slices(int H, int E) {
  const int blocks = (E + RT_COLS - 1) / RT_COLS;
  int s = (256 + blocks - 1) / blocks;
  const int most = (H / 32 + RT_NW - 1) / RT_NW;
  s = s < most ? s : most;
  return s < RT_MAX_S ? s : RT_MAX_S;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct DecWs {
  size_t part, act, yp, total;   // byte offsets
};
DecWs decode_ws(int T, int H, int I, int E, int k, int dt) {
  DecWs w;
  const size_t rows = (size_t)T * k + T;
  w.part = 0;
  w.act = w.part + round256((size_t)router_slices(H, E) * T * E * 8);
  w.yp = w.act + round256(rows * I * 4);   // two bf16 planes, or one fp32
  w.total = w.yp + round256(rows * H * 4);
  (void)dt;
  return w;
}

int decode_shape(const char* fn, int T, int H, int I, int E, int k, int dt) {
  MOE_TRY(moe_need_dt(dt, fn));
  MOE_TRY(moe_need_nonneg(T, fn, "T"));
  MOE_TRY(moe_need_ek(E, k, fn));
  MOE_TRY(moe_need_mult64(H, fn, "H"));
  MOE_TRY(moe_need_mult64(I, fn, "I"));
  if (T > DEC_MAX_T)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: T = %d above the %d tokens of a call", fn, T,
                    DEC_MAX_T);
  if ((long long)T * k > DEC_MAX_PAIRS)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: T k = %lld above %d pairs", fn, (long long)T * k,
                    DEC_MAX_PAIRS);
  // byte offsets within one expert's weights and within the workspace's rows are 32-bit, below
  // the offset that stands for "no load"
  const long long es = moe_dt_bytes(dt), rows = (long long)T * k + T;
  if (2LL * I * H * es >= 0x80000000LL || rows * I * 4 >= 0x80000000LL ||
      (long long)T * H * es >= 0x80000000LL || 4LL * H * E >= 0x80000000LL)
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: an operand of 2 GiB or more (T=%d H=%d I=%d E=%d)",
                    fn, T, H, I, E);
  return MOE_OK;
}

template <typename T>
int decode_launch(const DecArgs& a, hipStream_t s, const char* fn) {
  if (a.S > 0) {
    const dim3 grid((a.E + RT_COLS - 1) / RT_COLS, a.S), block(64 * RT_NW);
    if (a.T <= 16) hipLaunchKernelGGL((decode_router_kernel<T, 1>), grid, block, 0, s, a);
    else if (a.T <= 64) hipLaunchKernelGGL((decode_router_kernel<T, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((decode_router_kernel<T, 8>), grid, block, 0, s, a);
    MOE_TRY(moe_check_launch(fn));
  }
  const dim3 rg((a.T + 3) / 4), rb(256);
  switch (route_width(a.E)) {
    case 1: hipLaunchKernelGGL(decode_route_kernel<1>, rg, rb, 0, s, a); break;
    case 2: hipLaunchKernelGGL(decode_route_kernel<2>, rg, rb, 0, s, a); break;
    case 4: hipLaunchKernelGGL(decode_route_kernel<4>, rg, rb, 0, s, a); break;
    case 8: hipLaunchKernelGGL(decode_route_kernel<8>, rg, rb, 0, s, a); break;
    default: hipLaunchKernelGGL(decode_route_kernel<16>, rg, rb, 0, s, a); break;
  }
  MOE_TRY(moe_check_launch(fn));
  const int P = a.T * a.k;
  const long long experts = (P < a.G ? P : a.G) + a.shared;   // most that can be active
  const int cus = moe_cu_count();
  auto grid = [&](long long units) {
    return dim3((unsigned)(units < 1 ? 1 : units < 2LL * cus ? units : 2LL * cus));
  };
  hipLaunchKernelGGL((decode_expert_kernel<T, false>), grid(experts * (a.I / DEC_GU)),
                     dim3(DEC_NT), 0, s, a);
  MOE_TRY(moe_check_launch(fn));
  hipLaunchKernelGGL((decode_expert_kernel<T, true>), grid(experts * (a.H / DEC_DN)),
                     dim3(DEC_NT), 0, s, a);
  MOE_TRY(moe_check_launch(fn));
  hipLaunchKernelGGL(decode_combine_kernel<T>, dim3((a.H + 255) / 256, a.T), dim3(256), 0, s, a);
  return moe_check_launch(fn);
}

}  // namespace

extern "C" size_t moe_decode_workspace_bytes(int T, int H, int I, int E, int k, int dt) {
  if (decode_shape("moe_decode_workspace_bytes", T, H, I, E, k, dt) != MOE_OK) return 0;
  return decode_ws(T, H, I, E, k, dt).total;
}

extern "C" int moe_decode(const void* x, int dt, const float* wg, const float* bias, int T, int H,
                          int I, int E, int k, int g0, int G, const void* w13, const void* w2,
                          const void* ws13, const void* ws2, const void* residual, float* logits,
                          int32_t* idx, float* gate, void* y, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  const char* fn = "moe_decode";
  MOE_TRY(decode_shape(fn, T, H, I, E, k, dt));
  MOE_TRY(moe_need_nonneg(g0, fn, "g0"));
  MOE_TRY(moe_need_nonneg(G, fn, "G"));
  if ((long long)g0 + G > E)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: window [%d, %d + %d) beyond E = %d", fn, g0, g0, G,
                    E);
  if ((ws13 == nullptr) != (ws2 == nullptr))
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: ws13 and ws2 come together", fn);
  if (wg == nullptr && bias != nullptr)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: bias without wg (logits are an input)", fn);
  if (T == 0) return MOE_OK;
  MOE_TRY(moe_need_ptr(x, fn, "x"));
  MOE_TRY(moe_opt_ptr(wg, fn, "wg"));
  MOE_TRY(moe_opt_ptr(bias, fn, "bias", 4));
  if (G > 0) {
    MOE_TRY(moe_need_ptr(w13, fn, "w13"));
    MOE_TRY(moe_need_ptr(w2, fn, "w2"));
  }
  MOE_TRY(moe_opt_ptr(ws13, fn, "ws13"));
  MOE_TRY(moe_opt_ptr(ws2, fn, "ws2"));
  MOE_TRY(moe_opt_ptr(residual, fn, "residual"));
  MOE_TRY(moe_need_ptr(logits, fn, "logits", 4));
  MOE_TRY(moe_need_ptr(idx, fn, "idx", 4));
  MOE_TRY(moe_need_ptr(gate, fn, "gate", 4));
  MOE_TRY(moe_need_ptr(y, fn, "y"));
  if (y == x)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: y is x's buffer (it may be residual's)", fn);
  MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  const DecWs w = decode_ws(T, H, I, E, k, dt);
  if (ws_bytes < w.total)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                    w.total);
  DecArgs a = {};
  a.x = x; a.wg = wg; a.bias = bias;
  a.T = T; a.H = H; a.I = I; a.E = E; a.k = k; a.g0 = g0; a.G = G;
  a.shared = ws13 != nullptr;
  a.w13 = w13; a.w2 = w2; a.ws13 = ws13; a.ws2 = ws2; a.residual = residual;
  a.logits = logits; a.idx = idx; a.gate = gate; a.y = y;
  a.S = wg != nullptr ? router_slices(H, E) : 0;
  a.part = (double*)((char*)ws + w.part);
  a.act = (char*)ws + w.act;
  a.yp = (float*)((char*)ws + w.yp);
  return dt == MOE_BF16 ? decode_launch<bf16_t>(a, (hipStream_t)stream, fn)
                        : decode_launch<float>(a, (hipStream_t)stream, fn);
}
