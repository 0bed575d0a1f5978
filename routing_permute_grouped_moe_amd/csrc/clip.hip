// The norm of many gradients together and of each, and clipping by it.
//   norm = sqrt(sum g^2) or max |g|;  out = min(1, max_norm / (norm + 1e-6)) g, or g
//   where max_norm is infinite
//
// Gradients are cut into chunks of one length; a workgroup takes one.  Which
// chunk belongs to which gradient stands in a table that travels with the
// launch's arguments (no copy to the device, and a captured launch keeps its
// own).  A chunk's sum is kept in fp64 -- squares of every fp32 value are in its
// range -- and a last launch adds the chunks in order.
// Bound by HBM: 425 M gradients in bf16 (0.85 GB) have their norm in 134 us, 6.3
// TB/s; clipped into fp32 417 us more, 6.1 TB/s, in bf16 272, 6.2 TB/s, where a copy
// moves 5.1.  (Chunks taken in reverse to find the end of the norm's pass in the
// cache, plain loads and plain stores gave nothing.)
#include <algorithm>
#include <new>

#include "validate.hpp"

namespace {

constexpr int CLIP_NT = 256;
constexpr int CLIP_WAVES = CLIP_NT / MOE_WAVE;
constexpr int CLIP_SUM_NT = 1024;
constexpr int NORM_TABLE = 176;           // gradients of one launch: tables below 4 KB
constexpr int CLIP_TABLE = 128;
// Elements of a chunk, at least, and chunks, at most (but for one a gradient).  The
// norm's are few, for a launch adds them (425 M bf16: 134 us at 4096, 138 at 2048 and
// at 32768).  What is scaled is cut as fine as a workgroup's two rounds of loads: then
// what runs at one time lies together in memory (into fp32 417 us; 434 at 8192
// elements a chunk, 454 at 16384, 483 at 52000; into bf16 272, 276, 281 and 316).
constexpr long long NORM_CHUNK = 2048, CLIP_CHUNK = 4096;
constexpr long long NORM_CHUNKS = 4096, CLIP_CHUNKS = 1 << 23;
// chunks, at most, where each workgroup that scales adds the parts itself, instead of
// a launch between (a call on 6 gradients of 32768 values: 12.1 us, 14.5 with the
// launch; 1 M values 11.5 and 14.4, 4 M values 23 and 14.3)
constexpr long long FUSED_CHUNKS = 512;

static_assert((CLIP_CHUNKS + CLIP_TABLE) * CLIP_NT < (1LL << 32), "a launch ends at 2^32 threads");

struct NormTable {
  const void* g[NORM_TABLE];
  unsigned long long n[NORM_TABLE];   // elements; top bit: bf16
  int first[NORM_TABLE + 1];          // first chunk
  int count;
};
// The same in memory, of any length.
struct NormList {
  const void** g; unsigned long long* n; int* first;
  int count;
};
struct ClipTable {
  const void* g[CLIP_TABLE];
  void* out[CLIP_TABLE];
  unsigned long long n[CLIP_TABLE];   // elements; top bits: g is bf16, out is bf16
  int first[CLIP_TABLE + 1];
  int count;
};
constexpr unsigned long long G_BF16 = 1ull << 63, OUT_BF16 = 1ull << 62,
                             N_MASK = OUT_BF16 - 1;

// 16 bytes, aligned to an element only
typedef unsigned int u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
// (streaming: read once here, written for whoever comes later)
__device__ __forceinline__ u32x4 load16(const float* p) {
  return __builtin_nontemporal_load((const u32x4_a4*)p);
}
__device__ __forceinline__ u32x4 load16(const bf16_t* p) {
  return __builtin_nontemporal_load((const u32x4_a2*)p);
}
__device__ __forceinline__ void store16(float* p, u32x4 v) {
  __builtin_nontemporal_store(v, (u32x4_a4*)p);
}
__device__ __forceinline__ void store16(bf16_t* p, u32x4 v) {
  __builtin_nontemporal_store(v, (u32x4_a2*)p);
}
__device__ __forceinline__ void load_vec(const float* p, float (&v)[4]) {
  unpack16(load16(p), v, float());
}
__device__ __forceinline__ void load_vec(const bf16_t* p, float (&v)[8]) {
  unpack16(load16(p), v, bf16_t());
}
__device__ __forceinline__ void load_vec(const bf16_t* p, float (&v)[4]) {
  const u32x2 x = __builtin_nontemporal_load((const u32x2_a2*)p);
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { *p = (bf16_t)f32_to_bf16(v); }

// The gradient that chunk c belongs to: the last whose first chunk is not behind
// it, by a whole wave, 64 entries at a time.
template <typename Table>
__device__ __forceinline__ int grad_of(const Table& t, int c) {
  const int lane = threadIdx.x % MOE_WAVE;
  int lo = 0, len = t.count;                  // it is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + MOE_WAVE - 1) / MOE_WAVE, at = lane * step;
    const bool mine = at < len && t.first[lo + at] <= c;
    int runs = __popcll(__ballot(mine));
    runs = runs > 0 ? runs - 1 : 0;
    lo += runs * step;
    len = len - runs * step < step ? len - runs * step : step;
  }
  return uniform(lo);
}

// (a NaN is larger than any number)
__device__ __forceinline__ double max_nan(double a, double b) { return a >= b || a != a ? a : b; }

template <bool MAX>
__device__ __forceinline__ double join(double a, double b) { return MAX ? max_nan(a, b) : a + b; }
template <bool MAX>
__device__ __forceinline__ double wave_join(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = join<MAX>(v, __shfl_xor(v, o, MOE_WAVE));
  return v;
}
template <bool MAX>
__device__ __forceinline__ double take(double acc, float v) {
  return MAX ? max_nan(acc, fabs((double)v)) : fma((double)v, (double)v, acc);
}

// The squares (or the largest) of n values, this thread's part of them: four
// loads in flight, four chains of additions.
template <bool MAX, typename T>
__device__ __forceinline__ double chunk_sum(const T* g, long long n) {
  constexpr int VEC = Elem<T>::VEC, STEP = CLIP_NT * VEC, U = 4;
  double acc[U] = {0, 0, 0, 0};
  const long long whole = n / VEC * VEC;
  long long i = (long long)threadIdx.x * VEC;
  auto add = [&](double& to, const u32x4& x) {
    float v[VEC];
    unpack16(x, v, T());
#pragma unroll
    for (int j = 0; j < VEC; ++j) to = take<MAX>(to, v[j]);
  };
  for (; i + (U - 1) * STEP < whole; i += U * STEP) {
    u32x4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = load16(g + i + u * STEP);
#pragma unroll
    for (int u = 0; u < U; ++u) add(acc[u], x[u]);
  }
  for (; i < whole; i += STEP) add(acc[0], load16(g + i));
  if (whole + threadIdx.x < n) acc[1] = take<MAX>(acc[1], load1(g + whole + threadIdx.x));
  return join<MAX>(join<MAX>(acc[0], acc[1]), join<MAX>(acc[2], acc[3]));
}

// A table's entries, into memory.
__global__ __launch_bounds__(CLIP_NT) void grad_table_kernel(NormTable t, int at, NormList to) {
  const int i = threadIdx.x;
  if (i < t.count) {
    to.g[at + i] = t.g[i];
    to.n[at + i] = t.n[i];
  }
  if (i <= t.count) to.first[at + i] = t.first[i];
}
static_assert(NORM_TABLE < CLIP_NT, "a thread an entry");

// first: the table's first chunks go there, for the launch that adds the parts.
template <bool MAX, typename Table>
__global__ __launch_bounds__(CLIP_NT) void grad_part_kernel(Table t, long long chunk, double* part,
                                                            int* first) {
  __shared__ double red[CLIP_WAVES];
  const int c = blockIdx.x, i = grad_of(t, c);
  if (first != nullptr && c == 0 && threadIdx.x <= (unsigned)t.count)
    first[threadIdx.x] = t.first[threadIdx.x];
  const unsigned long long word = t.n[i];
  const long long n = (long long)(word & N_MASK), at = (long long)(c - t.first[i]) * chunk;
  const long long len = n - at < chunk ? n - at : chunk;
  double v = word & G_BF16 ? chunk_sum<MAX>((const bf16_t*)t.g[i] + at, len)
                           : chunk_sum<MAX>((const float*)t.g[i] + at, len);
  v = wave_join<MAX>(v);
  if (threadIdx.x % MOE_WAVE == 0) red[threadIdx.x / MOE_WAVE] = v;
  __syncthreads();
  if (threadIdx.x == 0 && len > 0) {          // (no chunk: one workgroup, for `first`)
    v = red[0];
#pragma unroll
    for (int w = 1; w < CLIP_WAVES; ++w) v = join<MAX>(v, red[w]);
    part[c] = v;
  }
}

// A thread adds a gradient of few chunks, a wave one of many (a wave for each of 700
// gradients: 25 us, so 4.8).  Of more than FEW chunks are at most NORM_CHUNKS / FEW,
// since there are at most NORM_CHUNKS chunks and one a gradient.
constexpr int FEW = 16, MANY = NORM_CHUNKS / (FEW - 1) + 8;
template <bool MAX>
__device__ __forceinline__ double grad_total(const double* part, const int* first, int count,
                                             float* norms) {
  constexpr int WAVES = CLIP_SUM_NT / MOE_WAVE;
  __shared__ double red[WAVES];
  __shared__ int found, list[MANY], sorted[MANY];
  const int lane = threadIdx.x % MOE_WAVE, wave = threadIdx.x / MOE_WAVE;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  double all = 0;
  for (int i = threadIdx.x; i < count; i += CLIP_SUM_NT) {
    const int c0 = first[i], c1 = first[i + 1];
    if (c1 - c0 > FEW) {
      const int at = atomicAdd(&found, 1);
      if (at < MANY) list[at] = i;
      continue;
    }
    double v = 0;
#pragma unroll 4
    for (int c = c0; c < c1; ++c) v = join<MAX>(v, part[c]);
    all = join<MAX>(all, v);
    if (norms) norms[i] = (float)(MAX ? v : sqrt(v));
  }
  __syncthreads();
  const int many = found < MANY ? found : MANY;
  if (threadIdx.x < many) {                   // in their order, whoever came first
    const int mine = list[threadIdx.x];
    int at = 0;
    for (int j = 0; j < many; ++j) at += list[j] < mine;
    sorted[at] = mine;
  }
  __syncthreads();
  all = wave_join<MAX>(all);
  for (int j = wave; j < many; j += WAVES) {
    const int i = sorted[j], c1 = first[i + 1];
    double v = 0;
#pragma unroll 8
    for (int c = first[i] + lane; c < c1; c += MOE_WAVE) v = join<MAX>(v, part[c]);
    v = wave_join<MAX>(v);
    all = join<MAX>(all, v);
    if (norms && lane == 0) norms[i] = (float)(MAX ? v : sqrt(v));
  }
  if (lane == 0) red[wave] = all;
  __syncthreads();
  all = red[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) all = join<MAX>(all, red[w]);
  return all;
}

template <bool MAX>
__global__ __launch_bounds__(CLIP_SUM_NT) void grad_norm_kernel(const double* part,
                                                                const int* first, int count,
                                                                float* norm, float* norms,
                                                                double* total) {
  const double all = grad_total<MAX>(part, first, count, norms);
  if (threadIdx.x == 0) {
    norm[0] = (float)(MAX ? all : sqrt(all));
    if (total) total[0] = all;
  }
}

// n values times c.  A thread's store is 16 bytes and a wave's 1 KB without
// gaps, whatever a thread loads for it (bf16 to fp32 with 32 bytes a thread, whose
// streaming stores leave gaps: 700 us in place of 485, both in long chunks).  Two
// loads in flight: 417 us, 448 with four, 442 with one.
template <int NT, typename G, typename O>
__device__ __forceinline__ void scale_chunk(const G* g, O* out, long long n, float c) {
  constexpr int VEC = Elem<O>::VEC, STEP = NT * VEC, U = 2;
  const long long whole = n / VEC * VEC;
  long long i = (long long)threadIdx.x * VEC;
  auto put = [&](O* to, float (&v)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] *= c;
    store16(to, pack16(v, O()));
  };
  for (; i + (U - 1) * STEP < whole; i += U * STEP) {
    float v[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) load_vec(g + i + u * STEP, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) put(out + i + u * STEP, v[u]);
  }
  for (; i < whole; i += STEP) {
    float v[VEC];
    load_vec(g + i, v);
    put(out + i, v);
  }
  if (whole + threadIdx.x < n)
    store1(out + whole + threadIdx.x, load1(g + whole + threadIdx.x) * c);
}

// Chunk b of the table, scaled for a norm.
template <int NT>
__device__ __forceinline__ void clip_chunk(const ClipTable& t, int b, long long chunk, float norm,
                                           float max_norm) {
  const int i = grad_of(t, b);
  float c = max_norm / (norm + 1e-6f);
  // (a NaN norm stays one; no limit scales nothing, an infinite norm either)
  c = c > 1.f || (max_norm == INFINITY && norm == norm) ? 1.f : c;
  if (c == 1.f && t.out[i] == t.g[i]) return;
  const unsigned long long word = t.n[i];
  const long long n = (long long)(word & N_MASK), at = (long long)(b - t.first[i]) * chunk;
  const long long len = n - at < chunk ? n - at : chunk;
  if (!(word & G_BF16))
    scale_chunk<NT>((const float*)t.g[i] + at, (float*)t.out[i] + at, len, c);
  else if (word & OUT_BF16)
    scale_chunk<NT>((const bf16_t*)t.g[i] + at, (bf16_t*)t.out[i] + at, len, c);
  else
    scale_chunk<NT>((const bf16_t*)t.g[i] + at, (float*)t.out[i] + at, len, c);
}
__global__ __launch_bounds__(CLIP_NT) void grad_clip_kernel(ClipTable t, long long chunk,
                                                            const float* norm, float max_norm) {
  clip_chunk<CLIP_NT>(t, blockIdx.x, chunk, norm[0], max_norm);
}
// The same, and the norm from its parts, by every workgroup for itself.
template <bool MAX>
__global__ __launch_bounds__(CLIP_SUM_NT) void grad_norm_clip_kernel(
    ClipTable t, long long chunk, const double* part, const int* first, float* norm, float* norms,
    float max_norm) {
  const bool one = blockIdx.x == 0;
  const double all = grad_total<MAX>(part, first, t.count, one ? norms : nullptr);
  const float by = (float)(MAX ? all : sqrt(all));
  if (one && threadIdx.x == 0) norm[0] = by;
  if ((int)blockIdx.x < t.first[t.count])     // (no chunk: one workgroup, for the norm)
    clip_chunk<CLIP_SUM_NT>(t, blockIdx.x, chunk, by, max_norm);
}

// Elements of a chunk: a multiple of the least.
long long chunk_of(const moe_grad* g, int count, long long least, long long most) {
  long long n = 0;
  for (int i = 0; i < count; ++i) n += g[i].n;
  const long long c = (n + most - 1) / most;
  return c < least ? least : (c + least - 1) / least * least;
}
long long chunks_of(const moe_grad* g, int count, long long chunk) {
  long long c = 0;
  for (int i = 0; i < count; ++i) c += (g[i].n + chunk - 1) / chunk;
  return c;
}

int grad_checks(const char* fn, const moe_grad* g, int count, bool outs) {
  MOE_TRY(moe_need_nonneg(count, fn, "count"));
  if (count > 0 && g == nullptr) return moe_fail(MOE_ERR_INVALID_ARG, "%s: grads is NULL", fn);
  if (count > (1 << 20))
    return moe_fail(MOE_ERR_UNSUPPORTED, "%s: %d gradients, above the limit", fn, count);
  for (int i = 0; i < count; ++i) {
    if (g[i].n < 0 || g[i].n >= (1LL << 40))
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: gradient %d has %lld elements", fn, i, g[i].n);
    MOE_TRY(moe_need_dt(g[i].dt, fn));
    if (outs && g[i].out_dt != MOE_F32 && g[i].out_dt != g[i].dt)
      return moe_fail(MOE_ERR_INVALID_ARG,
                      "%s: out %d has dtype %d, neither its gradient's nor MOE_F32", fn, i,
                      g[i].out_dt);
    if (g[i].n == 0) continue;
    MOE_TRY(moe_need_ptr(g[i].g, fn, "a gradient", moe_dt_bytes(g[i].dt)));
    if (outs) {
      MOE_TRY(moe_need_ptr(g[i].out, fn, "an out", moe_dt_bytes(g[i].out_dt)));
      if (g[i].out == g[i].g && g[i].out_dt != g[i].dt)
        return moe_fail(MOE_ERR_INVALID_ARG, "%s: out %d overlaps its gradient, of another type",
                        fn, i);
    }
  }
  return MOE_OK;
}

// An out that shares memory with another gradient or out (in place: its own).
struct Span {
  uintptr_t lo, hi;
  int i;
  bool written;
  bool operator<(const Span& o) const { return lo < o.lo; }
};
int clip_overlaps(const char* fn, const moe_grad* g, int count) {
  Span* s = new (std::nothrow) Span[2 * (size_t)count];
  if (s == nullptr) return moe_fail(MOE_ERR_UNSUPPORTED, "%s: no host memory", fn);
  int m = 0;
  for (int i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t p = (uintptr_t)g[i].g, o = (uintptr_t)g[i].out;
    s[m++] = {o, o + (uintptr_t)g[i].n * moe_dt_bytes(g[i].out_dt), i, true};
    if (o != p) s[m++] = {p, p + (uintptr_t)g[i].n * moe_dt_bytes(g[i].dt), i, false};
  }
  std::sort(s, s + m);
  uintptr_t any = 0, written = 0;     // ends of what began before
  int st = MOE_OK;
  for (int j = 0; j < m && st == MOE_OK; ++j) {
    if (s[j].lo < (s[j].written ? any : written))
      st = moe_fail(MOE_ERR_INVALID_ARG, "%s: the memory of %s %d is also another's", fn,
                    s[j].written ? "out" : "gradient", s[j].i);
    any = std::max(any, s[j].hi);
    if (s[j].written) written = std::max(written, s[j].hi);
  }
  delete[] s;
  return st;
}

// part [chunks] fp64, first [count + 1], and beyond a table's length g, n [count]
struct NormWs {
  long long chunk, chunks;
  size_t first, g, n, total;
};
NormWs norm_ws(const moe_grad* grads, int count) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  NormWs w;
  w.chunk = chunk_of(grads, count, NORM_CHUNK, NORM_CHUNKS);
  w.chunks = chunks_of(grads, count, w.chunk);
  w.first = up((size_t)w.chunks * 8);
  w.g = w.first + up((size_t)(count + 1) * 4);
  const size_t list = count > NORM_TABLE ? up((size_t)count * 8) : 0;
  w.n = w.g + list;
  w.total = w.n + list;
  return w;
}

int norm_checks(const char* fn, const moe_grad* grads, int count, int kind, const float* norm,
                const float* norms, const double* total, const void* ws, size_t ws_bytes,
                const NormWs& lay) {
  if (kind != MOE_GRAD_L2 && kind != MOE_GRAD_MAX)
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: kind %d is none of the MOE_GRAD values", fn, kind);
  MOE_TRY(moe_need_ptr(norm, fn, "norm", 4));
  MOE_TRY(moe_opt_ptr(norms, fn, "norms", 4));
  MOE_TRY(moe_opt_ptr(total, fn, "total", 8));
  MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  if (ws_bytes < lay.total)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                    lay.total);
  const MoeRange outs[] = {{norm, 4, "norm"}, {norms, 4LL * count, "norms"}, {total, 8, "total"},
                           {ws, (long long)lay.total, "ws"}};
  for (int i = 0; i < 4; ++i) {
    const char* with = nullptr;
    for (int j = 0; j < i && with == nullptr; ++j) with = moe_shares(outs[i], {outs[j]});
    for (int j = 0; j < count && with == nullptr; ++j)
      with = moe_shares(outs[i], {{grads[j].g, grads[j].n * moe_dt_bytes(grads[j].dt),
                                   "a gradient"}});
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: %s needs a buffer of its own, it overlaps %s", fn,
                      outs[i].name, with);
  }
  return MOE_OK;
}
int clip_checks(const char* fn, const moe_grad* grads, int count, const float* norm,
                float max_norm) {
  if (!(max_norm >= 0.f))
    return moe_fail(MOE_ERR_INVALID_ARG, "%s: max_norm = %g is negative or NaN", fn, max_norm);
  MOE_TRY(moe_need_ptr(norm, fn, "norm", 4));
  for (int i = 0; i < count; ++i)
    if (moe_shares({grads[i].out, grads[i].n * moe_dt_bytes(grads[i].out_dt), "out"},
                   {{norm, 4, "norm"}}))
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: out %d overlaps norm", fn, i);
  return clip_overlaps(fn, grads, count);
}

// The parts of the norm, in ws.
int launch_parts(const char* fn, const moe_grad* grads, int count, bool max, const NormWs& lay,
                 void* ws, hipStream_t s) {
  double* const part = (double*)ws;
  int* const first = (int*)((char*)ws + lay.first);
  NormList list = {(const void**)((char*)ws + lay.g), (unsigned long long*)((char*)ws + lay.n),
                   first, count};
  // (gradients that are all empty have a workgroup, for `first`)
  const dim3 grid(lay.chunks > 0 ? (unsigned)lay.chunks : 1);
  int at = 0;
  for (int g0 = 0; g0 < count; g0 += NORM_TABLE) {
    NormTable t;
    t.count = std::min(NORM_TABLE, count - g0);
    for (int i = 0; i < t.count; ++i) {
      const moe_grad& g = grads[g0 + i];
      t.g[i] = g.g;
      t.n[i] = (unsigned long long)g.n | (g.dt == MOE_BF16 ? G_BF16 : 0);
      t.first[i] = at;
      at += (int)((g.n + lay.chunk - 1) / lay.chunk);
    }
    t.first[t.count] = at;
    if (count > NORM_TABLE)
      hipLaunchKernelGGL(grad_table_kernel, dim3(1), dim3(CLIP_NT), 0, s, t, g0, list);
    else if (max)
      hipLaunchKernelGGL((grad_part_kernel<true, NormTable>), grid, dim3(CLIP_NT), 0, s, t,
                         lay.chunk, part, first);
    else
      hipLaunchKernelGGL((grad_part_kernel<false, NormTable>), grid, dim3(CLIP_NT), 0, s, t,
                         lay.chunk, part, first);
    MOE_TRY(moe_check_launch(fn));
  }
  if (count <= NORM_TABLE) return MOE_OK;
  // more gradients than a table holds: tables into memory, then one launch for all
  // (700 gradients of 40000 values: 32 us, where a launch a table takes 65)
  if (max)
    hipLaunchKernelGGL((grad_part_kernel<true, NormList>), grid, dim3(CLIP_NT), 0, s, list,
                       lay.chunk, part, nullptr);
  else
    hipLaunchKernelGGL((grad_part_kernel<false, NormList>), grid, dim3(CLIP_NT), 0, s, list,
                       lay.chunk, part, nullptr);
  return moe_check_launch(fn);
}
int launch_norm(const char* fn, int count, bool max, const NormWs& lay, void* ws, float* norm,
                float* norms, double* total, hipStream_t s) {
  const double* const part = (const double*)ws;
  const int* const first = (const int*)((char*)ws + lay.first);
  if (max)
    hipLaunchKernelGGL(grad_norm_kernel<true>, dim3(1), dim3(CLIP_SUM_NT), 0, s, part, first,
                       count, norm, norms, total);
  else
    hipLaunchKernelGGL(grad_norm_kernel<false>, dim3(1), dim3(CLIP_SUM_NT), 0, s, part, first,
                       count, norm, norms, total);
  return moe_check_launch(fn);
}

ClipTable clip_table(const moe_grad* grads, int count, long long chunk) {
  ClipTable t;
  t.count = count;
  t.first[0] = 0;
  for (int i = 0; i < count; ++i) {
    t.g[i] = grads[i].g;
    t.out[i] = grads[i].out;
    t.n[i] = (unsigned long long)grads[i].n | (grads[i].dt == MOE_BF16 ? G_BF16 : 0) |
             (grads[i].out_dt == MOE_BF16 ? OUT_BF16 : 0);
    t.first[i + 1] = t.first[i] + (int)((grads[i].n + chunk - 1) / chunk);
  }
  return t;
}
int launch_clip(const char* fn, const moe_grad* grads, int count, const float* norm,
                float max_norm, hipStream_t s) {
  const long long chunk = chunk_of(grads, count, CLIP_CHUNK, CLIP_CHUNKS);
  for (int g0 = 0; g0 < count; g0 += CLIP_TABLE) {
    const ClipTable t = clip_table(grads + g0, std::min(CLIP_TABLE, count - g0), chunk);
    if (t.first[t.count] == 0) continue;
    hipLaunchKernelGGL(grad_clip_kernel, dim3(t.first[t.count]), dim3(CLIP_NT), 0, s, t, chunk,
                       norm, max_norm);
    MOE_TRY(moe_check_launch(fn));
  }
  return MOE_OK;
}

}  // namespace

extern "C" size_t moe_grad_norm_workspace_bytes(const moe_grad* grads, int count) {
  if (grad_checks("moe_grad_norm_workspace_bytes", grads, count, false) != MOE_OK) return 0;
  return norm_ws(grads, count).total;
}

extern "C" int moe_grad_norm(const moe_grad* grads, int count, int kind, float* norm, float* norms,
                             double* total, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* fn = "moe_grad_norm";
  MOE_TRY(grad_checks(fn, grads, count, false));
  const NormWs lay = norm_ws(grads, count);
  MOE_TRY(norm_checks(fn, grads, count, kind, norm, norms, total, ws, ws_bytes, lay));
  hipStream_t s = (hipStream_t)stream;
  const bool max = kind == MOE_GRAD_MAX;
  MOE_TRY(launch_parts(fn, grads, count, max, lay, ws, s));
  return launch_norm(fn, count, max, lay, ws, norm, norms, total, s);
}

extern "C" int moe_grad_clip(const moe_grad* grads, int count, const float* norm, float max_norm,
                             moe_stream_t stream) {
  const char* fn = "moe_grad_clip";
  MOE_TRY(grad_checks(fn, grads, count, true));
  MOE_TRY(clip_checks(fn, grads, count, norm, max_norm));
  return launch_clip(fn, grads, count, norm, max_norm, (hipStream_t)stream);
}

extern "C" int moe_grad_norm_clip(const moe_grad* grads, int count, int kind, float max_norm,
                                  float* norm, float* norms, void* ws, size_t ws_bytes,
                                  moe_stream_t stream) {
  const char* fn = "moe_grad_norm_clip";
  MOE_TRY(grad_checks(fn, grads, count, true));
  const NormWs lay = norm_ws(grads, count);
  MOE_TRY(norm_checks(fn, grads, count, kind, norm, norms, nullptr, ws, ws_bytes, lay));
  MOE_TRY(clip_checks(fn, grads, count, norm, max_norm));
  for (int i = 0; i < count; ++i) {   // (the parts and the norms are read while outs are written)
    const char* with = moe_shares(
        {grads[i].out, grads[i].n * moe_dt_bytes(grads[i].out_dt), "out"},
        {{norms, 4LL * count, "norms"}, {ws, (long long)lay.total, "ws"}});
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: out %d overlaps %s", fn, i, with);
  }
  hipStream_t s = (hipStream_t)stream;
  const bool max = kind == MOE_GRAD_MAX;
  MOE_TRY(launch_parts(fn, grads, count, max, lay, ws, s));
  if (count > CLIP_TABLE || lay.chunks > FUSED_CHUNKS) {
    MOE_TRY(launch_norm(fn, count, max, lay, ws, norm, norms, nullptr, s));
    return launch_clip(fn, grads, count, norm, max_norm, s);
  }
  const ClipTable t = clip_table(grads, count, lay.chunk);
  const double* const part = (const double*)ws;
  const int* const first = (const int*)((char*)ws + lay.first);
  const dim3 grid(lay.chunks > 0 ? (unsigned)lay.chunks : 1);
  if (max)
    hipLaunchKernelGGL(grad_norm_clip_kernel<true>, grid, dim3(CLIP_SUM_NT), 0, s, t, lay.chunk,
                       part, first, norm, norms, max_norm);
  else
    hipLaunchKernelGGL(grad_norm_clip_kernel<false>, grid, dim3(CLIP_SUM_NT), 0, s, t, lay.chunk,
                       part, first, norm, norms, max_norm);
  return moe_check_launch(fn);
}
