// Layer norm and RMS norm of rows, with the residual sum in front, and their
// gradients:
//   h = x + residual,  q = (h - m) rstd,  y = q w + bias
//   g = dy w,  dx = rstd (g - mean(g) - q mean(g q)) + dh,  dw = sum dy q,  db = sum dy
#include "validate.hpp"

namespace {

constexpr int NORM_NT = 256;
constexpr int NORM_WAVES = NORM_NT / MOE_WAVE;
constexpr int NORM_MAX_H = 16384;
constexpr int NORM_PARTS = 256;   // row runs of the weight gradient, at most

template <typename T>
__device__ __forceinline__ float norm_load(const void* p, long long i) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(((const T*)p)[i]);
  else return ((const T*)p)[i];
}
template <typename T>
__device__ __forceinline__ float norm_store(void* p, long long i, float v) {
  if constexpr (sizeof(T) == 2) {
    const T b = (T)f32_to_bf16(v);
    ((T*)p)[i] = b;
    return bf16_to_f32(b);
  } else {
    ((T*)p)[i] = v;
    return v;
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  __syncthreads();
  if (threadIdx.x % MOE_WAVE == 0) red[threadIdx.x / MOE_WAVE] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NORM_WAVES; ++w) s += red[w];
  return s;
}

struct NormArgs {
  const void* x; const void* residual; const float* w; const float* bias;
  void* h; void* y; float* mean; float* rstd;
  int M, H, rms;
  float eps;
};

template <typename T>
__global__ __launch_bounds__(NORM_NT) void norm_kernel(NormArgs a) {
  __shared__ float red[NORM_WAVES];
  const long long r0 = (long long)blockIdx.x * a.H;
  auto at = [&](int i) {
    float v = norm_load<T>(a.x, r0 + i);
    if (a.residual) {
      v += norm_load<T>(a.residual, r0 + i);
      if constexpr (sizeof(T) == 2) v = bf16_to_f32(f32_to_bf16(v));
    }
    return v;
  };
  float s = 0.f;
  for (int i = threadIdx.x; i < a.H; i += NORM_NT) s += at(i);
  const float mean = a.rms ? 0.f : block_sum(s, red) / a.H;
  float q = 0.f;
  for (int i = threadIdx.x; i < a.H; i += NORM_NT) {
    const float d = at(i) - mean;
    q += d * d;
  }
  const float rstd = 1.0f / sqrtf(block_sum(q, red) / a.H + a.eps);
  for (int i = threadIdx.x; i < a.H; i += NORM_NT) {
    const float v = at(i);
    if (a.h) norm_store<T>(a.h, r0 + i, v);
    const float y = (v - mean) * rstd * a.w[i];
    norm_store<T>(a.y, r0 + i, a.bias ? y + a.bias[i] : y);
  }
  if (threadIdx.x == 0) {
    if (a.mean && !a.rms) a.mean[blockIdx.x] = mean;
    if (a.rstd) a.rstd[blockIdx.x] = rstd;
  }
}

struct NormBwdArgs {
  const void* dy; const void* h; const void* dh; const float* w; const float* mean;
  const float* rstd;
  void* dx; float* dw; float* db; float* part;
  int M, H, rms, parts;
};

template <typename T>
__global__ __launch_bounds__(NORM_NT) void norm_dx_kernel(NormBwdArgs a) {
  __shared__ float red[NORM_WAVES];
  const long long r0 = (long long)blockIdx.x * a.H;
  const float mean = a.rms ? 0.f : a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < a.H; i += NORM_NT) {
    const float g = norm_load<T>(a.dy, r0 + i) * a.w[i];
    s1 += g;
    s2 += g * ((norm_load<T>(a.h, r0 + i) - mean) * rstd);
  }
  s1 = a.rms ? 0.f : block_sum(s1, red) / a.H;
  s2 = block_sum(s2, red) / a.H;
  for (int i = threadIdx.x; i < a.H; i += NORM_NT) {
    const float g = norm_load<T>(a.dy, r0 + i) * a.w[i];
    const float q = (norm_load<T>(a.h, r0 + i) - mean) * rstd;
    float v = rstd * (g - s1 - q * s2);
    if (a.dh) v += norm_load<T>(a.dh, r0 + i);
    norm_store<T>(a.dx, r0 + i, v);
  }
}

template <typename T>
__global__ __launch_bounds__(NORM_NT) void norm_dw_kernel(NormBwdArgs a) {
  const int c = blockIdx.x * NORM_NT + threadIdx.x;
  if (c >= a.H) return;
  float dw = 0.f, db = 0.f;
  for (int r = blockIdx.y; r < a.M; r += gridDim.y) {
    const float d = norm_load<T>(a.dy, (long long)r * a.H + c);
    const float m = a.rms ? 0.f : a.mean[r];
    dw += d * ((norm_load<T>(a.h, (long long)r * a.H + c) - m) * a.rstd[r]);
    db += d;
  }
  a.part[(long long)blockIdx.y * 2 * a.H + c] = dw;
  a.part[((long long)blockIdx.y * 2 + 1) * a.H + c] = db;
}

__global__ __launch_bounds__(NORM_NT) void norm_dw_sum_kernel(NormBwdArgs a) {
  const int c = blockIdx.x * NORM_NT + threadIdx.x;
  if (c >= a.H) return;
  double dw = 0, db = 0;
  for (int p = 0; p < a.parts; ++p) {
    dw += a.part[(long long)p * 2 * a.H + c];
    db += a.part[((long long)p * 2 + 1) * a.H + c];
  }
  if (a.dw) a.dw[c] = (float)dw;
  if (a.db) a.db[c] = (float)db;
}

int norm_parts(int M) { return M < NORM_PARTS ? M : NORM_PARTS; }

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
  NormArgs a = {x, residual, w, bias, h, y, mean, rstd, M, H, kind == MOE_NORM_RMS, eps};
  hipStream_t s = (hipStream_t)stream;
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(norm_kernel<bf16_t>, dim3(M), dim3(NORM_NT), 0, s, a);
  else
    hipLaunchKernelGGL(norm_kernel<float>, dim3(M), dim3(NORM_NT), 0, s, a);
  return moe_check_launch(fn);
}

extern "C" size_t moe_norm_bwd_workspace_bytes(int M, int H, int dt) {
  if (norm_checks("moe_norm_bwd_workspace_bytes", dt, M, H, MOE_NORM_LAYER) != MOE_OK) return 0;
  return ((size_t)norm_parts(M) * 2 * H * 4 + 255) / 256 * 256;
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
  NormBwdArgs a = {dy, h, dh, w, mean, rstd, dx, dw, db, (float*)ws, M, H, kind == MOE_NORM_RMS,
                   norm_parts(M)};
  hipStream_t s = (hipStream_t)stream;
  const int cols = (H + NORM_NT - 1) / NORM_NT;
  if (M > 0 && sums) {
    const dim3 grid(cols, a.parts);
    if (dt == MOE_BF16)
      hipLaunchKernelGGL(norm_dw_kernel<bf16_t>, grid, dim3(NORM_NT), 0, s, a);
    else
      hipLaunchKernelGGL(norm_dw_kernel<float>, grid, dim3(NORM_NT), 0, s, a);
    MOE_TRY(moe_check_launch(fn));
  }
  if (sums) {
    hipLaunchKernelGGL(norm_dw_sum_kernel, dim3(cols), dim3(NORM_NT), 0, s, a);
    MOE_TRY(moe_check_launch(fn));
  }
  if (M == 0 || dx == nullptr) return MOE_OK;
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(norm_dx_kernel<bf16_t>, dim3(M), dim3(NORM_NT), 0, s, a);
  else
    hipLaunchKernelGGL(norm_dx_kernel<float>, dim3(M), dim3(NORM_NT), 0, s, a);
  return moe_check_launch(fn);
}
