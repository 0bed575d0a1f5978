// The whole expert layer for a few tokens (serving): router projection,
// softmax top-k, the chosen SwiGLU experts, the shared expert, the
// gate-weighted sum and the residual.
//
// For at most 128 tokens the layer is a stream of the chosen experts' weights,
// with the multiplications in its shade (2 m flops per weight for m rows, far
// below the 300 flops per byte at which the matrix cores and HBM balance).  An
// expert's weights are read once for every block of its rows: 16 or 32 rows of
// W13 (gateup_tiles below), 16 of W2, so once where it serves at most 16 tokens;
// the shared expert's W2 is asked for 8 times at 128 tokens.  (128 tokens of 64
// experts, 6 each: 1.31 GB from the fabric, 1.11 without re-reads.)  Sorting rows
// into groups, as the training path does, would be latency only: the rows of an
// expert are found from the tokens' choices directly and the products read tokens
// in place.  Two launches up to 8 tokens, three above:
//  1. the router product in K slices (and the second launch's counters set
//     to zero);
//  2. everything else in one persistent launch of one workgroup per CU, whose
//     units of work -- route a few tokens, 16 gate/up columns of an expert, 32
//     output columns of an expert -- are drawn from one counter in an order in
//     which a unit depends on earlier ones only;
//  3. above 8 tokens (or 256 pairs), the gate-weighted sum.
#include <type_traits>

#include "lds_copy.hpp"
#include "route_select.hpp"
#include "stream.hpp"
#include "validate.hpp"

namespace {

constexpr int DEC_MAX_T = 128;       // tokens of a call
constexpr int DEC_MAX_PAIRS = 2048;  // (token, slot) pairs of a call
constexpr int DEC_SW = 4;            // streaming waves of a workgroup of the second launch
constexpr int DEC_NT = 64 * (DEC_SW + 2);   // and one that schedules, one that finishes tiles
constexpr int DEC_GU = 16;           // gate/up columns of a unit (16 gate and 16 up rows of W13)
constexpr int DEC_DN = 32;           // output columns of a unit of the second product
constexpr int RT_NW = 4;             // waves of a router workgroup
constexpr int RT_COLS = 16;          // experts of a router workgroup
constexpr int RT_MAX_S = 32;         // K slices of the router product

typedef double f64x4 __attribute__((ext_vector_type(4)));

struct DecArgs {
  const void* x; const float* wg; const float* bias;
  int T, H, I, E, k, g0, G, shared;
  int gu_tiles;       // row tiles of a gate/up unit: 1 or 2
  const void* w13; const void* w2; const void* ws13; const void* ws2; const void* residual;
  float* logits; int32_t* idx; float* gate; void* y;
  int S;              // K slices of the router product (0: logits are an input)
  double* part;       // [S][T][E] partial logits
  void* act;          // [planes][T k + T][I] activations, shared rows last
  float* yp;          // [T k + T][H] expert outputs
  // counters, zero when the second launch starts: the next unit, tokens
  // routed, whether a wait for that was given up, finished gate/up units of each
  // expert (window index; the shared expert last), finished units of each block of
  // DEC_DN output columns.  All but the last lie a cache line apart: on one line
  // with the others, a look at an expert's counter waited for everyone's draws
  // (128 tokens: 323 us so, 267 apart)
  int* next; int* routed; int* unrouted; int* act_done; int* col_done;
  int* go;            // one word a cache line for each workgroup: 0, DEC_GO or DEC_GO_LOST
  int n_count;        // all of them, from next on
  unsigned long long wait_ticks;   // after which a wait is given up
};

// 8 elements of T as fp32, from byte offset off
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t off, float* v, bf16_t) {
  unpack16(buf_load16(r, off), v, bf16_t());
}
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t off, float* v, float) {
  unpack16(buf_load16(r, off), v, 0.f);
  unpack16(buf_load16(r, off + 16), v + 4, 0.f);
}

// The second launch's counters (workgroup b of n, 256 threads).
__device__ __forceinline__ void decode_clear(const DecArgs& a, int b, int n) {
  for (int i = b * 256 + threadIdx.x; i < a.n_count; i += n * 256) a.next[i] = 0;
}
__global__ __launch_bounds__(256) void decode_clear_kernel(DecArgs a) {
  decode_clear(a, blockIdx.x, gridDim.x);
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
  decode_clear(a, blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y);
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

// Device-scope stores and loads: data that another workgroup of the same
// launch reads.  A store goes through this XCD's L2; it is visible to whoever
// learns, through a counter raised after the store completed, that it is there
// and then drops what its own caches may hold (acquire).
__device__ __forceinline__ void dev_store(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void dev_store(int32_t* p, int32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void dev_store(bf16_t* p, uint32_t v) {
  __hip_atomic_store(p, (bf16_t)v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int dev_load(const int* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void dev_add(int* p, int v) {
  __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One wave per token: the logits (sum of the partials and the bias, rounded
// once to fp32), the k largest and their softmax weights.
// emit(slot, expert, gate) for each; keep: the logits are written out.
template <int V, typename Emit>
__device__ __forceinline__ void decode_route_token(const DecArgs& a, int t, bool keep,
                                                   Emit&& emit) {
  const int lane = threadIdx.x & 63;
  float v[V];
  uint32_t key[V];
  float m = -INFINITY;
  if (a.S > 0) {
    // all loads of a batch of slices in flight
    double s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + i * MOE_WAVE;
      s[i] = a.bias != nullptr && e < a.E ? (double)a.bias[e] : 0.0;
    }
    constexpr int B = V == 1 ? 32 : V == 2 ? 16 : V == 4 ? 16 : 2;
    for (int p = 0; p < a.S; p += B) {
      double d[V][B];
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < B; ++q)
          d[i][q] = a.part[((long long)min(p + q, a.S - 1) * a.T + t) * a.E +
                           min(lane + i * MOE_WAVE, a.E - 1)];
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < B; ++q) s[i] += p + q < a.S ? d[i][q] : 0.0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + i * MOE_WAVE;
      v[i] = e < a.E ? (float)s[i] : -INFINITY;
      if (keep && e < a.E) a.logits[(long long)t * a.E + e] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + i * MOE_WAVE;
      v[i] = e < a.E ? a.logits[(long long)t * a.E + e] : -INFINITY;
    }
  }
  bool masked = true;   // (fmaxf passes NaN over: m alone does not tell)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = lane + i * MOE_WAVE < a.E ? route_key(v[i]) : 0u;
    m = fmaxf(m, v[i]);
    masked = masked && v[i] == -INFINITY;
  }
  m = wave_max(m);
  const bool none = __all(masked);   // every expert masked: gates of zero, not NaN
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += lane + i * MOE_WAVE < a.E ? expf(v[i] - m) : 0.f;
  s = wave_sum(s);
  const float inv = 1.0f / s;
  route_select<V>(key, a.k, [&](int slot, int i) {
    emit(slot, lane + i * MOE_WAVE, none ? 0.f : expf(v[i] - m) * inv);
  });
}

// ---------------------------------------------------------------- experts
// The second launch.  A workgroup has four streaming waves, one that schedules
// and one that finishes tiles; they meet in LDS words only, never at a
// barrier, so the stream of weights does not stop between units.
//
// Streaming.  A unit is 32 weight rows (two 16-row tiles) times at most 16
// rows of the other operand (32 in the gate/up units of calls whose experts
// have many rows: each unit reads its weights again).  K runs in steps of 128 bytes of a row (64 bf16,
// 32 fp32) dealt to the four waves in turn; a step's weights and operand rows
// go HBM -> LDS in copies of whole lines (stream.hpp) into a ring that belongs
// to the wave alone, several steps ahead.  The stream is one flat sequence of
// steps, unit after unit: at the end of a unit the waves leave their partial
// tiles in LDS while the next one's steps are on their way.  A wave has a SIMD
// to itself, so a branch costs it as much as a dozen instructions, and a step
// has 590 ns at HBM's rate (16 KB for the four waves): every step is the same
// few copies, reads and MFMAs, and while there is nothing to copy the copies
// go through an empty range, whose zeros add nothing to whatever tile is next.
//
// Finishing.  The finishing wave adds the four partial tiles in wave order
// (the same bits on every run), applies silu(g) u or stores the rows of the
// second product, and raises the unit's counter.
//
// Scheduling.  Units are numbered [route][shared gate/up][gate/up of each
// chosen expert][second product, same order].  A unit waits only for units of
// lower numbers, and numbers are drawn in order by running workgroups, so the
// lowest unfinished unit never waits: no residency of the grid is assumed.
// For few tokens every workgroup routes them itself (they cost each about a
// microsecond) instead of waiting for the one that would.
constexpr int DEC_ROWS = 16;         // operand rows of a tile; of a unit, but for gate/up ones of 32
constexpr int DEC_DESCS = 4;
constexpr int DEC_PAGE = 2048;       // a 16-row tile of a step
constexpr int DEC_PAGES = 16;        // of a streaming wave's ring
constexpr int DEC_OWN_T = 8;         // tokens, and pairs, that every workgroup routes itself
constexpr int DEC_OWN_PAIRS = 256;
constexpr unsigned DEC_WAIT_US = 1000000;   // a wait longer than this is given up (moe_decode_wait_limit)
constexpr unsigned DEC_TICKS_PER_US = 100;   // of the constant 100 MHz clock
constexpr unsigned DEC_STEP_US = 100;        // most that a look of a wait counts for
constexpr int DEC_GO = 1, DEC_GO_LOST = 2;   // a workgroup's word: activations complete, or given up

enum { U_GATEUP = 0, U_DOWN = 1, U_ROUTE = 2, U_SUM = 3, U_EXIT = 4 };

// words of a descriptor (a wave reads them all at once, one a lane)
enum {
  W_KIND = 0,
  W_AT,                  // A tiles (operand copies of 16 rows)
  W_MT,                  // row tiles of the result
  W_PACKED,              // rows 8-15 are the low halves of rows 0-7
  W_STEPS,               // K steps of 128 bytes
  W_N,                   // rows
  W_SLOT,                // counter the unit raises (expert, or column block)
  W_COL,                 // first gate/up or output column
  W_WLO, W_WHI, W_WBYTES,   // weights: address and extent
  W_ALO, W_AHI, W_ABYTES,   // and the A operand's
  W_LDW, W_TILE1,        // bytes of a weight row, and from the first tile to the second
  W_WORDS = 16           // (all of them)
};

struct DecDesc {
  int word[W_WORDS];
  uint32_t arow[2 * 16];       // byte offset of each A row
  int rows[2 * DEC_ROWS];      // pair indices, or T k + token
};

struct DecLds {
  char ring[DEC_SW][DEC_PAGES * DEC_PAGE];
  float red[2][DEC_SW][2 * 256];   // partial tiles, of units of even and of odd number (units of
                                   // two row tiles take both)
  int16_t order[DEC_MAX_PAIRS];    // pairs of the window, expert by expert
  int cur[(MOE_MAX_E + 3) / 2];    // while that is built: two counters a word; then pre_g
  int16_t list[MOE_MAX_E + 1];     // experts some token chose, ascending; the shared one first (-1)
  int16_t first[MOE_MAX_E + 2];    // their places in order
  int16_t pre[MOE_MAX_E + 2];      // row blocks before each, of second-product units
  int16_t own_idx[DEC_OWN_PAIRS];  // choices and gates, where every workgroup routes itself
  float own_gate[DEC_OWN_PAIRS];
  DecDesc desc[DEC_DESCS];
  // words the waves meet in
  int ready;                       // descriptors written, their A operands there
  int early;                       // one written whose A operand is not there yet: its number + 1
  int parts[DEC_SW];               // units whose partial tiles each streaming wave has left
  int taken;                       // units whose partial tiles were read
  int done;                        // units finished
  int per_col;                     // units of a column block
  int lost;                        // a wait was given up: what it waited for is not there
};
static_assert(sizeof(DecLds) <= 160 * 1024, "LDS of a CU");

__device__ __forceinline__ int lds_peek(const int* p) {
  return *(const volatile int*)p;
}
__device__ __forceinline__ void lds_post(int* p, int v) {   // (by one lane)
  *(volatile int*)p = v;
}
// wait until *p >= v: another wave of the workgroup raises it
__device__ __forceinline__ void lds_wait(const int* p, int v) {
  while (uniform(lds_peek(p)) < v) __builtin_amdgcn_s_sleep(1);
  asm volatile("" ::: "memory");
}
// row blocks of an expert with m rows, in units of `tiles` row tiles
__device__ __forceinline__ int row_blocks(int m, int tiles) {
  return (m + DEC_ROWS * tiles - 1) >> (tiles == 2 ? 5 : 4);
}

// A wait for other workgroups, bounded by the time that this one ran: a step from
// look to look counts DEC_STEP_US at most, so that the time in which the whole
// queue was suspended does not (looks are a few microseconds apart).
struct DecWait {
  unsigned long long last = wall_clock64(), spent = 0;
  bool late = false;
};
// After a look that found nothing: give up?  Only if the look before was late
// already, so that one look at least follows the last of the time.
__device__ __forceinline__ bool dec_give_up(DecWait& w, unsigned long long limit) {
  if (w.late) return true;
  const unsigned long long now = wall_clock64(), step = now - w.last;
  w.last = now;
  w.spent += step < DEC_STEP_US * DEC_TICKS_PER_US ? step : DEC_STEP_US * DEC_TICKS_PER_US;
  w.late = w.spent >= limit;
  return false;
}

template <typename T> constexpr int DEC_PLANES = sizeof(T) == 2 ? 2 : 1;

__device__ __host__ __forceinline__ bool dec_own(int T, int k) {
  return T <= DEC_OWN_T && T * k <= DEC_OWN_PAIRS;
}

// ---- the scheduling wave

// The launch's arguments where they lie, read again where they are used: held
// in scalar registers across the scheduler's loop they would spill.
typedef const __attribute__((address_space(4))) DecArgs DecConst;

// Tables of the call, from the tokens' choices: the list of chosen experts
// (shared first), the row blocks before each, and the pairs expert by expert
// (in any order within one: a row's result does not depend on its place).
// Returns the length of the list.
__device__ __forceinline__ int decode_tables(DecConst& a, DecLds& l) {
  const int lane = threadIdx.x & 63, P = a.T * a.k;
  const bool own = dec_own(a.T, a.k);
  if (P <= 64 && a.T <= DEC_ROWS) {
    // a pair a lane, sorted by counting; an expert has one row block at most
    // (0.4 us, the general way below 2.4)
    constexpr int NONE = 0x7fff;
    int g = NONE, rank = lane;
    if (lane < P) {
      g = (own ? (int)l.own_idx[lane] : a.idx[lane]) - a.g0;
      if (g < 0 || g >= a.G) g = NONE;
      rank = 0;
    }
    for (int j = 0; j < P; ++j) {
      const int o = __builtin_amdgcn_readlane(g, j);
      rank += lane < P && (o < g || (o == g && j < lane)) ? 1 : 0;
    }
    const int n_in = __popcll(__ballot(g != NONE));
    if (g != NONE) l.order[rank] = (int16_t)lane;
    const int sorted = __builtin_amdgcn_ds_permute(rank * 4, g);
    const int left = __shfl_up(sorted, 1, 64);
    const bool head = sorted != NONE && (lane == 0 || left != sorted);
    const unsigned long long b = __ballot(head);
    const int n0 = a.shared ? 1 : 0, n = n0 + __popcll(b);
    int16_t* const pre_g = (int16_t*)l.cur;
    if (a.shared && lane == 0) {
      l.list[0] = -1;
      l.first[0] = l.pre[0] = pre_g[0] = 0;
    }
    if (head) {
      const int at = n0 + __popcll(b & ((1ull << lane) - 1));
      l.list[at] = (int16_t)sorted;
      l.first[at] = (int16_t)lane;
      l.pre[at] = pre_g[at] = (int16_t)at;
    }
    if (lane == 0) {
      l.first[n] = (int16_t)n_in;
      l.pre[n] = pre_g[n] = (int16_t)n;
      l.per_col = n;
    }
    lds_drain();
    return n;
  }
  for (int g = lane; g < (a.G + 1) / 2; g += 64) l.cur[g] = 0;
  lds_drain();
  // counter of expert g: a half of a word (at most 2048 pairs in all)
  auto add = [&](int g, int v) {
    return (atomicAdd(&l.cur[g >> 1], v << ((g & 1) * 16)) >> ((g & 1) * 16)) & 0xffff;
  };
  auto pairs = [&](auto&& f) {   // f(pair, window index) for every pair of the window
    for (int p0 = 0; p0 < P; p0 += 64 * 8) {
      int e[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int p = min(p0 + q * 64 + lane, P - 1);
        e[q] = own ? (int)l.own_idx[p & (DEC_OWN_PAIRS - 1)] : a.idx[p];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int p = p0 + q * 64 + lane, g = e[q] - a.g0;
        if (p < P && g >= 0 && g < a.G) f(p, g);
      }
    }
    lds_drain();
  };
  pairs([&](int, int g) { add(g, 1); });
  int n = 0, blocks = 0, rows = 0;
  if (a.shared) {
    if (lane == 0) {
      l.list[0] = -1;
      l.first[0] = 0;
      l.pre[0] = 0;
    }
    n = 1;
    blocks = row_blocks(a.T, 1);
  }
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const int g = g0 + lane;
    const int m = g < a.G ? (l.cur[g >> 1] >> ((g & 1) * 16)) & 0xffff : 0;
    const unsigned long long b = __ballot(m > 0);
    int incl = m | row_blocks(m, 1) << 16;   // both sums at once
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    if (m > 0) {
      const int at = n + __popcll(b & ((1ull << lane) - 1));
      l.list[at] = (int16_t)g;
      l.first[at] = (int16_t)(rows + (incl & 0xffff) - m);
      l.pre[at] = (int16_t)(blocks + (incl >> 16) - row_blocks(m, 1));
      add(g, rows + (incl & 0xffff) - 2 * m);   // m counted there -> its first place
    }
    const int all = __shfl(incl, 63, 64);
    n += __popcll(b);
    rows += all & 0xffff;
    blocks += all >> 16;
  }
  if (lane == 0) {
    l.first[n] = (int16_t)rows;
    l.pre[n] = (int16_t)blocks;
    l.per_col = blocks;
  }
  lds_drain();
  pairs([&](int p, int g) { l.order[add(g, 1)] = (int16_t)p; });
  // row blocks of gate/up units before each (the counters are done with)
  int16_t* const pre_g = (int16_t*)l.cur;
  int before = 0;
  for (int s0 = 0; s0 <= n; s0 += 64) {
    const int s = s0 + lane;
    const int m = s >= n ? 0 : (a.shared && s == 0) ? a.T : l.first[s + 1] - l.first[s];
    int incl = row_blocks(m, a.gu_tiles);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    if (s <= n) pre_g[s] = (int16_t)(before + incl - row_blocks(m, a.gu_tiles));
    before += __shfl(incl, 63, 64);
  }
  lds_drain();
  return n;
}

template <typename T>
__device__ __forceinline__ void decode_schedule(DecLds& l) {
  constexpr int ES = sizeof(T), PL = DEC_PLANES<T>;
  const int lane = threadIdx.x & 63;
  DecConst* args = (DecConst*)__builtin_amdgcn_kernarg_segment_ptr();
  int n_list = -1, n_gu = 0, n_dn = 0;
  const int16_t* const pre_g = (const int16_t*)l.cur;
  bool go = false;       // the activations are complete
  bool pending = false, watch = false;   // not yet, and units wait for them; this wave looks
  bool lost = false;     // a wait was given up (calls that share a workspace): wait no more,
                         // and what this workgroup adds to the result is NaN
  auto draw = [&]() {
    int v = 0;
    if (lane == 0)
      v = __hip_atomic_fetch_add(args->next, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return v;
  };
  // two numbers are drawn ahead: they take microseconds under load (the second
  // one only when the first unit is on its way -- 256 workgroups start at once,
  // and their draws queue up)
  int held = draw(), held2 = 0;
  for (int seq = 0;; ++seq) {
    int u = uniform(held);
    // (kept in a vector register, and all that follows from it: the scheduling
    // arithmetic would not fit the scalar ones)
    asm volatile("" : "+v"(u));
    asm volatile("" : "+s"(args));
    DecConst& a = *args;
    const int P = a.T * a.k;
    const int n_route = dec_own(a.T, a.k) ? 0 : (a.T + DEC_SW - 1) / DEC_SW;
    const int per_g = a.I / DEC_GU, per_d = a.H / DEC_DN;
    const int n_shared = a.shared ? row_blocks(a.T, a.gu_tiles) * per_g : 0;
    lds_wait(&l.done, seq - DEC_DESCS + 1);   // the descriptor's last user is through
    DecDesc& d = l.desc[seq % DEC_DESCS];
    int kind, g = -2, s = 0, rb = 0, col = 0;
    if (u < n_route) {
      kind = U_ROUTE;
      col = u * DEC_SW;
    } else if (u < n_route + n_shared) {
      // (the shared expert needs no routing)
      const int v = u - n_route, nb = row_blocks(a.T, a.gu_tiles);
      kind = U_GATEUP;
      g = -1;
      rb = v % nb;
      col = v / nb * DEC_GU;
    } else {
      if (n_list < 0) {
        if (n_route > 0) {
          DecWait w;
          while (uniform(dev_load(a.routed)) < a.T) {
            lost = dec_give_up(w, args->wait_ticks);
            if (lost) break;
            __builtin_amdgcn_s_sleep(1);
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
          if (lost && lane == 0) dev_store(a.unrouted, 1);
        }
        if (!lost) {
          n_list = decode_tables(a, l);
          n_gu = pre_g[n_list] * per_g;
          n_dn = l.pre[n_list] * per_d;
        }
      }
      int v = u - n_route;
      if (lost && n_list < 0) {
        // Without every token's choices the numbers mean nothing: this workgroup
        // does no more, whoever waits for its units gives up in turn, and the
        // sum's launch makes all of y NaN.
        kind = U_EXIT;
      } else if (v < n_gu + n_dn) {
        kind = v < n_gu ? U_GATEUP : U_DOWN;
        const int per = v < n_gu ? per_g : per_d;
        const int16_t* const pre = v < n_gu ? pre_g : l.pre;
        if (v >= n_gu) v -= n_gu;
        // place in the list: the last with pre * per <= v
        for (int s0 = 0; s0 < n_list; s0 += 64) {
          const unsigned long long le =
              __ballot(s0 + lane < n_list && pre[s0 + lane] * per <= v);
          if (le) s = s0 + 63 - __builtin_clzll(le);
        }
        g = l.list[s];
        const int nb = pre[s + 1] - pre[s];
        v -= pre[s] * per;
        rb = v % nb;
        col = v / nb * (kind == U_GATEUP ? DEC_GU : DEC_DN);
      } else if (n_dn == 0 && v < per_d && n_route == 0) {
        kind = U_SUM;    // nothing but the residual
        col = v * DEC_DN;
      } else {
        kind = U_EXIT;
      }
    }
    if (kind <= U_DOWN) {
      const bool down = kind == U_DOWN;
      const int mt = down ? 1 : a.gu_tiles, most = DEC_ROWS * mt, r0 = rb * most;
      int n, row = 0;
      if (g < 0) {
        n = min(most, a.T - r0);
        row = P + r0 + min(lane, n - 1);
      } else {
        const int f = l.first[s] + r0;
        n = min(most, l.first[s + 1] - f);
        row = l.order[f + min(lane, n - 1)];
      }
      if (lane < n) d.rows[lane] = row;
      // (packed or not goes by the call: one number of tiles all through a phase)
      const bool two = down && PL == 2;
      const bool packed = two && a.T <= 8;
      const int at = two && !packed ? 2 : mt;
      const uint32_t plane = (uint32_t)(P + a.T) * (uint32_t)(a.I * ES);
      // A row `lane`: packed tiles hold the high halves in rows 0-7 and the low
      // ones in rows 8-15; else the tile of the low halves follows
      const int per_plane = packed ? 8 : 16 * mt;
      // (padding rows lie out of range: they read as zeros and move nothing)
      const int mine = __shfl(row, min(lane % per_plane, n - 1), 64);
      const int tok = mine >= P ? mine - P : mine / a.k;
      if (lane < 16 * at)
        d.arow[lane] = lane % per_plane >= n ? STREAM_OOB
                       : down ? (uint32_t)mine * (uint32_t)(a.I * ES) + lane / per_plane * plane
                              : (uint32_t)tok * (uint32_t)(a.H * ES);
      const long long ld = (long long)(down ? a.I : a.H) * ES;
      const char* base =
          down ? (g < 0 ? (const char*)a.ws2 : (const char*)a.w2 + (long long)g * a.H * ld)
               : (g < 0 ? (const char*)a.ws13 : (const char*)a.w13 + (long long)g * 2 * a.I * ld);
      const unsigned long long w = (unsigned long long)(base + col * ld);
      const unsigned long long x = (unsigned long long)(down ? a.act : a.x);
      if (lane == 0) {
        d.word[W_AT] = at;
        d.word[W_MT] = mt;
        d.word[W_PACKED] = packed;
        d.word[W_STEPS] = (int)(ld / 128);
        d.word[W_N] = n;
        d.word[W_SLOT] = down ? col / DEC_DN : (g < 0 ? a.G : g);
        d.word[W_WLO] = (int)(uint32_t)w;
        d.word[W_WHI] = (int)(w >> 32) & 0xffff;
        d.word[W_WBYTES] = (int)((down ? DEC_DN : a.I + DEC_GU) * ld);
        d.word[W_ALO] = (int)(uint32_t)x;
        d.word[W_AHI] = (int)(x >> 32) & 0xffff;
        d.word[W_ABYTES] = (int)(down ? plane * PL : (uint32_t)(a.T * a.H * ES));
        d.word[W_LDW] = (int)ld;
        d.word[W_TILE1] = (int)((down ? 16 : a.I) * ld);
      }
    }
    if (lane == 0) {
      d.word[W_KIND] = kind;
      d.word[W_COL] = col;
    }
    lds_drain();
    // A unit of the second product needs its expert's activations, and those of
    // the experts at the head of the list are long there when its last gate/up
    // units still run: one look at the expert's counter (and at this workgroup's
    // word, below) lets such a unit go ahead (one token of 7680 x 2048, 8 experts
    // and the shared one: 174 us without, 162 with it; 61 tokens: 460 and 447).
    const bool ask = kind == U_DOWN && !go && !pending;
    bool there = false;
    if (uniform(ask)) {
      const int v = dev_load(lane == 1 ? a.go + blockIdx.x * 32 : a.act_done + 32 * (g < 0 ? a.G : g));
      const int need = lane == 1 ? 1 : (pre_g[s + 1] - pre_g[s]) * per_g;
      const unsigned long long ok = __ballot(lane < 2 && v >= need);
      there = ok != 0;
      go = (ok & 2) != 0;
      if (__ballot(lane == 1 && v == DEC_GO_LOST)) {
        lost = true;
        if (lane == 0) lds_post(&l.lost, 1);   // (before this unit is)
      }
      if (there) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    }
    // The first one whose expert is not there waits for all of them: for few
    // tokens its weights may come in before that, as many as the rings hold, and
    // the unit behind it is looked up (one token of 2048 x 1408, 6 experts: 49.2 us
    // without either, 47.0 with them; 61 tokens of 7680 x 2048: 468 and 472, the
    // streams run dry to be started anew)
    const bool first = uniform(ask && (!there || u == n_route + n_gu));
    if (first) {
      pending = true;
      watch = u == n_route + n_gu;
      if (n_route == 0 && lane == 0 && !watch) lds_post(&l.early, seq + 1);
    }
    if (lane == 0 && (!pending || (first && there))) lds_post(&l.ready, seq + 1);
    if (!pending && uniform(kind) == U_EXIT) break;
    if (uniform(kind) != U_EXIT) {
      held = seq == 0 ? draw() : held2;
      held2 = draw();
    }
    if (!pending || (first && n_route == 0)) continue;
    // The second product begins when all activations are complete.  One
    // workgroup, whoever drew its first unit, watches the experts' counters (64
    // at a look) and tells each of the others on a line of its own: 256 of them
    // watching the same lines took so long for every look that the copies
    // queued behind it in their CUs' memory pipelines stood still.  (It copies
    // no weights early: its looks would queue behind them.)
    DecWait wait;
    if (watch) {
      int known = 0;
      while (known < n_list) {
        const int q = known + lane;
        bool there = false;
        if (q < n_list) {
          const int gq = l.list[q];
          there = dev_load(args->act_done + 32 * (gq < 0 ? args->G : gq)) >=
                  (pre_g[q + 1] - pre_g[q]) * (args->I / DEC_GU);
        }
        const unsigned long long no = ~__ballot(there);
        known += no ? __builtin_ctzll(no) : 64;
        if (known < n_list && !lost) lost = dec_give_up(wait, args->wait_ticks);
        if (lost) break;
      }
      // (given up: the others must not take incomplete activations for whole ones)
      const int word = lost ? DEC_GO_LOST : DEC_GO;
      for (int w = lane; w < (int)gridDim.x; w += 64) dev_store(args->go + w * 32, word);
    } else {
      int word;
      while ((word = uniform(dev_load(args->go + blockIdx.x * 32))) == 0 && !lost) {
        lost = dec_give_up(wait, args->wait_ticks);
        __builtin_amdgcn_s_sleep(2);
      }
      lost = lost || word == DEC_GO_LOST;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    go = true;
    pending = false;
    if (lost && lane == 0) lds_post(&l.lost, 1);
    if (lane == 0) lds_post(&l.ready, seq + 1);
    if (uniform(kind) == U_EXIT) break;
  }
}

// ---- the streaming waves

// The flat stream of one streaming wave over the units from seq on that have AT
// A tiles each, feeding MT row tiles of the result (A tile i adds to row tile
// i % MT); returns the number of the first unit that has not.  Steps are
// counted as they are copied (`put`) and read (`got`); a unit's tile is complete
// when got reaches the put at which its last step was copied.  The copies are
// at most one unit ahead.  early: the first unit's operand is not there yet.
template <typename T, int AT, int MT, bool OWN>
__device__ __forceinline__ int stream_units(DecLds& l, int seq, bool early) {
  constexpr int SIZE = 2 + AT, OPS = 4 + 2 * AT, D = DEC_PAGES / SIZE;
  constexpr int NEVER = 0x7fffffff;
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  char* const ring = l.ring[wave];
  const uint32_t lds = lds_addr(ring);
  // the unit being copied
  int at_unit = seq - 1, left = 0, end = NEVER;
  bool stop = false;
  int wlo = 0, whi = 0, wbytes = 0, alo = 0, ahi = 0, abytes = 0;
  uint32_t wo[2] = {0, 0}, ao[2 * AT];
#pragma unroll
  for (int j = 0; j < 2 * AT; ++j) ao[j] = 0;
  int tile1 = 0, k = 0;
  // the unit being read
  int got_end = NEVER;
  int put = 0, got = 0;
  uint32_t wslot = 0, rslot = 0;   // byte of the ring

  // on to the next unit, if it is known and its operand is there
  auto bind = [&](bool early) {
    const int u = at_unit + 1;
    if (u > seq + 1 || stop) return;
    if (!early && uniform(lds_peek(&l.ready)) <= u) {
      if constexpr (OWN) stop = uniform(lds_peek(&l.early)) == u + 1;   // (a stream of its own)
      return;
    }
    asm volatile("" ::: "memory");
    const DecDesc& d = l.desc[u % DEC_DESCS];
    const int word = d.word[lane % W_WORDS];
#pragma unroll
    for (int j = 0; j < 2 * AT; ++j) {
      const int r = stream_row(j);
      ao[j] = d.arow[r] + stream_chunk(j);
    }
    auto w = [&](int i) { return __builtin_amdgcn_readlane(word, i); };
    if (w(W_KIND) > U_DOWN || w(W_AT) != AT || w(W_MT) != MT) {
      stop = true;
      return;
    }
    wlo = w(W_WLO);
    whi = w(W_WHI);
    wbytes = w(W_WBYTES);
    alo = w(W_ALO);
    ahi = w(W_AHI);
    abytes = w(W_ABYTES);
    tile1 = w(W_TILE1);
    left = uniform((w(W_STEPS) - wave + DEC_SW - 1) / DEC_SW);
    k = wave * 128;
    const int ldw = w(W_LDW);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      wo[j] = (uint32_t)(stream_row(j) * ldw) + stream_chunk(j);
    }
    at_unit = u;
    end = put + left;
    if (u == seq) got_end = end;
  };
  // a step's copies: its weights, and (not `early`) its A rows
  auto copy = [&](auto with_a) {
    if (with_a() && left == 0) bind(false);
    const int live = uniform(left > 0 ? -1 : 0);
    const i32x4 rw = {uniform(wlo), uniform(whi), uniform(wbytes & live), MOE_RSRC_DW3};
    const i32x4 ra = {uniform(alo), uniform(ahi), uniform(abytes & live), MOE_RSRC_DW3};
    const uint32_t p = (uint32_t)uniform((int)(lds + wslot));
    const int k0 = uniform(k & live), k1 = uniform((k + tile1) & live);
    dma16_nt(rw, p, wo[0], k0);
    dma16_nt(rw, p + 1024, wo[1], k0);
    dma16_nt(rw, p + 2048, wo[0], k1);
    dma16_nt(rw, p + 3 * 1024, wo[1], k1);
    if constexpr (with_a())
#pragma unroll
      for (int j = 0; j < 2 * AT; ++j) dma16(ra, p + 4096 + j * 1024, ao[j], k0);
    wslot = (uint32_t)uniform((int)(wslot + SIZE * DEC_PAGE == D * SIZE * DEC_PAGE
                                        ? 0 : wslot + SIZE * DEC_PAGE));
    k = uniform(k + DEC_SW * 128);
    left = uniform(left + live);
    ++put;
  };
  f32x4 acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4{0, 0, 0, 0};
  const int f0 = stream_frag(0), f1 = stream_frag(1);
  if (OWN && early) {
    // the weights of as many steps as the ring holds, then, when it is there,
    // the operand; the loop below finds D steps copied either way
    bind(true);
    const int steps = left;
#pragma unroll 1
    for (int d = 0; d < D; ++d) copy(std::false_type());
    lds_wait(&l.ready, seq + 1);
#pragma unroll 1
    for (int d = 0; d < D; ++d) {
      const int live = uniform(d < steps ? -1 : 0);
      const i32x4 ra = {uniform(alo), uniform(ahi), uniform(abytes & live), MOE_RSRC_DW3};
      const uint32_t p = (uint32_t)uniform((int)(lds + d * SIZE * DEC_PAGE + 4096));
#pragma unroll
      for (int j = 0; j < 2 * AT; ++j)
        dma16(ra, p + j * 1024, ao[j], uniform((wave + d * DEC_SW) * 128 & live));
    }
    vm_drain<0>();
  } else {
#pragma unroll 1
    for (int d = 0; d < D; ++d) copy(std::true_type());
  }
  lds_wait(&l.taken, seq);         // (units of another kind may have used all of red)
  for (;;) {
    vm_drain<(D - 1) * OPS>();     // the oldest step has landed
    const char* p = ring + rslot;
    u32x4 w[2][2], x[2][AT];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      w[0][t] = *(const u32x4*)(p + t * DEC_PAGE + f0);
      w[1][t] = *(const u32x4*)(p + t * DEC_PAGE + f1);
    }
#pragma unroll
    for (int t = 0; t < AT; ++t) {
      x[0][t] = *(const u32x4*)(p + (2 + t) * DEC_PAGE + f0);
      x[1][t] = *(const u32x4*)(p + (2 + t) * DEC_PAGE + f1);
    }
    rslot = (uint32_t)uniform((int)(rslot + SIZE * DEC_PAGE == D * SIZE * DEC_PAGE
                                        ? 0 : rslot + SIZE * DEC_PAGE));
    ++got;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        acc[t % MT][0] = stream_mma(x[h][t], w[h][0], acc[t % MT][0], T());
        acc[t % MT][1] = stream_mma(x[h][t], w[h][1], acc[t % MT][1], T());
      }
    lds_drain();                   // the slot is read
    if (got >= got_end) {
      // (>: a unit without steps of this wave ends where it was bound)
      lds_wait(&l.taken, MT == 2 ? seq : seq - 1);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float* red = l.red[MT == 2 ? m : seq & 1][wave];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int q = 0; q < 4; ++q) red[t * 256 + q * 64 + lane] = acc[m][t][q];
          acc[m][t] = f32x4{0, 0, 0, 0};
        }
      }
      lds_drain();
      if (lane == 0) lds_post(&l.parts[wave], seq + 1);
      ++seq;
      got_end = at_unit == seq ? end : NEVER;
    }
    if (stop && at_unit < seq) break;
    copy(std::true_type());        // into the slot read last
  }
  vm_drain<0>();                   // (empty copies)
  return seq;
}

template <typename T, int V, bool OWN>
__device__ __forceinline__ void decode_stream(const DecArgs& a, DecLds& l) {
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  for (int seq = 0;;) {
    bool early = false;
    for (;;) {
      if (uniform(lds_peek(&l.ready)) > seq) break;
      if constexpr (OWN) early = uniform(lds_peek(&l.early)) == seq + 1;
      if (early) break;
      __builtin_amdgcn_s_sleep(1);
    }
    asm volatile("" ::: "memory");
    const DecDesc& d = l.desc[seq % DEC_DESCS];
    const int kind = uniform(d.word[W_KIND]);
    if (kind == U_EXIT) break;
    if (kind <= U_DOWN) {
      if constexpr (!OWN) {
        if (uniform(d.word[W_MT]) == 2) {
          seq = stream_units<T, 2, 2, false>(l, seq, early);
          continue;
        }
        if constexpr (DEC_PLANES<T> == 2)
          if (uniform(d.word[W_AT]) == 2) {
            seq = stream_units<T, 2, 1, false>(l, seq, early);
            continue;
          }
      }
      seq = stream_units<T, 1, 1, OWN>(l, seq, early);
      continue;
    }
    if constexpr (!OWN) {
      const int t = uniform(d.word[W_COL]) + wave;
      if (kind == U_ROUTE && t < a.T)
        decode_route_token<V>(a, t, true, [&](int slot, int e, float gate) {
          dev_store(a.idx + (long long)t * a.k + slot, e);
          dev_store(a.gate + (long long)t * a.k + slot, gate);
        });
      vm_drain<0>();
    }
    if (lane == 0) lds_post(&l.parts[wave], seq + 1);
    ++seq;
  }
}

// ---- the finishing wave

constexpr float BF16_MAX = 0x1.fep127f;

// silu(g) u; the sum of two bf16 that the second product reads carries 16
// bits of it, so its rounding does not show beside that of the result
__device__ __forceinline__ float decode_swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

template <typename T>
__device__ __forceinline__ float elem_load(const void* p, long long i) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(((const T*)p)[i]);
  else return ((const T*)p)[i];
}
template <typename T>
__device__ __forceinline__ void elem_store(void* p, long long i, float v) {
  if constexpr (sizeof(T) == 2) ((T*)p)[i] = (T)f32_to_bf16(v);
  else ((T*)p)[i] = v;
}

// residual + shared + sum_j gate yp[t, j], in that order; pair(p) gives a
// pair's expert and gate.  (For a pair outside the window row 0 is read, and not
// added: a branch for each would have every load waited for in turn.)  A gate of
// zero adds nothing either: a masked expert, there to fill the k slots, may hold
// infinities or NaN.
template <typename T, typename Pair>
__device__ __forceinline__ float decode_sum(const DecArgs& a, int t, int h, Pair&& pair) {
  float s = a.residual != nullptr ? elem_load<T>(a.residual, (long long)t * a.H + h) : 0.f;
  if (a.shared) s += a.yp[((long long)a.T * a.k + t) * a.H + h];
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    float gate[8], v[8];
    bool in[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int p = t * a.k + min(j0 + q, a.k - 1);
      int e;
      pair(p, e, gate[q]);
      in[q] = j0 + q < a.k && e >= a.g0 && e - a.g0 < a.G;
      v[q] = a.yp[(long long)(in[q] ? p : 0) * a.H + h];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s += in[q] && gate[q] != 0.f ? gate[q] * v[q] : 0.f;
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void decode_finish(const DecArgs& a, DecLds& l) {
  const int lane = threadIdx.x & 63, P = a.T * a.k;
  // the last unit of a column block sums it, where no wait precedes the tables
  // and the choices are at hand; else the sum is a launch of its own
  const bool fused = dec_own(a.T, a.k);
  const long long plane = (long long)(P + a.T) * a.I;
  auto sum_block = [&](int col, int n) {
#pragma unroll 1
    for (int t0 = 0; t0 < a.T; t0 += 2) {
      const int t = t0 + (lane >> 5), h = col + (lane & 31);
      const float s = decode_sum<T>(a, min(t, a.T - 1), h, [&](int p, int& e, float& w) {
        e = l.own_idx[p & (DEC_OWN_PAIRS - 1)];
        w = l.own_gate[p & (DEC_OWN_PAIRS - 1)];
      });
      if (t < n) elem_store<T>(a.y, (long long)t * a.H + h, s);
    }
  };
  // Once for nothing, while the first unit streams: a first pass through this
  // code waits for every line of it, 4 us that would end the call.
  if (fused) sum_block(0, 0);
  for (int seq = 0;; ++seq) {
    lds_wait(&l.ready, seq + 1);
    const DecDesc& d = l.desc[seq % DEC_DESCS];
    const int word = d.word[lane % W_WORDS];
    auto w = [&](int i) { return __builtin_amdgcn_readlane(word, i); };
    const int kind = w(W_KIND), col = w(W_COL);
    if (kind == U_EXIT) break;
#pragma unroll
    for (int w = 0; w < DEC_SW; ++w) lds_wait(&l.parts[w], seq + 1);
    if (kind <= U_DOWN) {
      const int n = w(W_N);
      const bool packed = w(W_PACKED);
      const int mt = w(W_MT);
      const bool lost = uniform(lds_peek(&l.lost)) != 0;   // NaN, not a wrong answer
      float v[2][2][4];   // [row tile][weight tile][register]
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (m < mt) {
          const int b = mt == 2 ? m : seq & 1;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float s = l.red[b][0][t * 256 + q * 64 + lane];
#pragma unroll
              for (int z = 1; z < DEC_SW; ++z) s += l.red[b][z][t * 256 + q * 64 + lane];
              v[m][t][q] = s;
            }
        }
      lds_drain();
      if (lane == 0) lds_post(&l.taken, seq + 1);
      // register q: row 4 (lane / 16) + q, column lane % 16
      const int c = lane & 15;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (m < mt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float s0 = v[m][0][q], s1 = v[m][1][q];
            if (packed) {   // rows 8-15: the low halves' part of rows 0-7
              s0 += __shfl_xor(s0, 32, 64);
              s1 += __shfl_xor(s1, 32, 64);
            }
            const int r = 16 * m + 4 * (lane >> 4) + q;
            if (r >= n || (packed && lane >= 32)) continue;
            const int row = d.rows[r];
            if (kind == U_GATEUP) {
              const float s = decode_swiglu(s0, s1);
              const long long at = (long long)row * a.I + col + c;
              if constexpr (sizeof(T) == 2) {
                // (held to the finite values: with hi an infinity, s - hi would be NaN or
                // the opposite one; so an infinite s is lo's, and NaN too)
                const uint32_t hi = f32_to_bf16(fminf(fmaxf(s, -BF16_MAX), BF16_MAX));
                dev_store((bf16_t*)a.act + at, hi);
                dev_store((bf16_t*)a.act + plane + at, f32_to_bf16(s - bf16_to_f32(hi)));
              } else {
                dev_store((float*)a.act + at, s);
              }
            } else {
              if (lost) s0 = s1 = __uint_as_float(0x7fc00000u);
              float* out = a.yp + (long long)row * a.H + col + c;
              dev_store(out, s0);
              dev_store(out + 16, s1);
            }
          }
      vm_drain<0>();   // the stores are out: the unit counts
      if (kind == U_GATEUP) {
        if (lane == 0) dev_add(a.act_done + 32 * w(W_SLOT), 1);
      } else if (fused) {
        int before = 0;
        if (lane == 0)
          before = __hip_atomic_fetch_add(a.col_done + w(W_SLOT), 1, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
        if (uniform(before) == uniform(lds_peek(&l.per_col)) - 1) {
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
          sum_block(col, a.T);
        }
      }
    } else {
      if (lane == 0) lds_post(&l.taken, seq + 1);
      if (kind == U_ROUTE) {
        if (lane == 0) dev_add(a.routed, min(DEC_SW, a.T - col));
      } else {
        sum_block(col, a.T);
      }
    }
    if (lane == 0) lds_post(&l.done, seq + 1);
  }
}

template <typename T, int V, bool OWN>
__global__ __launch_bounds__(DEC_NT) void decode_kernel(DecArgs a) {
  __shared__ __attribute__((aligned(1024))) DecLds l;
  if (threadIdx.x < DEC_SW) l.parts[threadIdx.x] = 0;
  if (threadIdx.x == 0) l.ready = l.early = l.taken = l.done = l.lost = 0;
  const int wave = uniform((int)(threadIdx.x >> 6));
  if constexpr (OWN) {
    const bool keep = blockIdx.x == 0;   // (one of them writes the choices out)
    for (int t = wave; t < a.T; t += DEC_SW + 2)
      decode_route_token<V>(a, t, keep, [&](int slot, int e, float gate) {
        const int p = t * a.k + slot;
        l.own_idx[p & (DEC_OWN_PAIRS - 1)] = (int16_t)e;
        l.own_gate[p & (DEC_OWN_PAIRS - 1)] = gate;
        if (keep) {
          a.idx[p] = e;
          a.gate[p] = gate;
        }
      });
  }
  __syncthreads();
  if (wave < DEC_SW) {
    decode_stream<T, V, OWN>(a, l);
    return;
  }
  if (wave == DEC_SW) decode_schedule<T>(l);
  else decode_finish<T>(a, l);
}

// the sum as a launch of its own, for more tokens than one wave should add; NaN
// where some workgroup gave up its wait for the routing
template <typename T>
__global__ __launch_bounds__(256) void decode_sum_kernel(DecArgs a) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= a.H) return;
  const float s = decode_sum<T>(a, blockIdx.y, h, [&](int p, int& e, float& w) {
    e = a.idx[p];
    w = a.gate[p];
  });
  elem_store<T>(a.y, (long long)blockIdx.y * a.H + h,
                *a.unrouted == 0 ? s : __uint_as_float(0x7fc00000u));
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

// Row tiles of the gate/up units: two where an expert is likely to have more
// rows than one tile holds (its mean over 8, or the shared expert's all): its
// weights are then read once, not once a tile.  us with one tile and with two
// (bf16; H x I, experts, k):
//   shared expert    7680 x 2048, 32 of 256, 8: 17 tokens 253, 248; 64 462, 450; 128 574, 548
//                    7168 x 2048, 16 of 256, 8: 17 tokens 122, 115; 128 335, 313
//                    4096 x 1024, 16, 2: 24 tokens 88.0, 89.5; 64 103, 102; 128 146, 128
//                    1024 x 512, 128, 8: 17 tokens 98, 98.5; 128 140.7, 142.8
//   mean of 8        4096 x 2048, 8, 2: 99.6, 101.6; 4096 x 1024, 16, 2: 100.4, 103.6
//   12               105.7, 108.5 (4096 x 1024, 16, 2); 4096 x 2048, 32, 4: 322, 303
//   16               4096 x 2048, 8, 2: 125, 120; 32, 4: 398, 340; 4096 x 1024, 16, 2: 128, 125
constexpr int GU_MEAN = 8;
int gateup_tiles(bool shared, int T, int E, int k) {
  return T > 16 && (shared || T * k > GU_MEAN * E) ? 2 : 1;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct DecWs {
  size_t count, part, act, yp, total;   // byte offsets
  int n_count;
};
DecWs decode_ws(int T, int H, int I, int E, int k) {
  DecWs w;
  const size_t rows = (size_t)T * k + T;
  // a cache line for each of the three scalars and each expert of the window and
  // the shared one, an int per column block, a cache line per workgroup
  w.n_count = (96 + 32 * (E + 1) + H / DEC_DN + 31) / 32 * 32 + 32 * moe_cu_count();
  w.count = 0;
  w.part = w.count + round256((size_t)w.n_count * 4);
  w.act = w.part + round256((size_t)router_slices(H, E) * T * E * 8);
  w.yp = w.act + round256(rows * I * 4);   // two bf16 planes, or one fp32
  w.total = w.yp + round256(rows * H * 4);
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
  } else {
    hipLaunchKernelGGL(decode_clear_kernel, dim3((a.n_count + 255) / 256), dim3(256), 0, s, a);
  }
  MOE_TRY(moe_check_launch(fn));
  // one workgroup per CU (its LDS fills one), no more than there can be units
  const long long P = (long long)a.T * a.k;
  const long long experts = (P < a.G ? P : a.G) + a.shared;
  const long long units = experts * (a.I / DEC_GU + a.H / DEC_DN) + a.H / DEC_DN;
  const int cus = moe_cu_count();
  const dim3 grid((unsigned)(units < cus ? units : cus)), block(DEC_NT);
  auto launch = [&](auto own) {
    constexpr bool OWN = decltype(own)::value;
    switch (route_width(a.E)) {
      case 1: hipLaunchKernelGGL((decode_kernel<T, 1, OWN>), grid, block, 0, s, a); break;
      case 2: hipLaunchKernelGGL((decode_kernel<T, 2, OWN>), grid, block, 0, s, a); break;
      case 4: hipLaunchKernelGGL((decode_kernel<T, 4, OWN>), grid, block, 0, s, a); break;
      default: hipLaunchKernelGGL((decode_kernel<T, 16, OWN>), grid, block, 0, s, a); break;
    }
  };
  if (dec_own(a.T, a.k)) launch(std::true_type{});
  else launch(std::false_type{});
  MOE_TRY(moe_check_launch(fn));
  if (dec_own(a.T, a.k)) return MOE_OK;
  hipLaunchKernelGGL(decode_sum_kernel<T>, dim3((a.H + 255) / 256, a.T), dim3(256), 0, s, a);
  return moe_check_launch(fn);
}

}  // namespace

static thread_local unsigned g_wait_us = DEC_WAIT_US;

extern "C" void moe_decode_wait_limit(unsigned us) { g_wait_us = us; }

extern "C" size_t moe_decode_workspace_bytes(int T, int H, int I, int E, int k, int dt) {
  if (decode_shape("moe_decode_workspace_bytes", T, H, I, E, k, dt) != MOE_OK) return 0;
  return decode_ws(T, H, I, E, k).total;
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
  MOE_TRY(moe_need_ptr(ws, fn, "ws", 256));
  const DecWs w = decode_ws(T, H, I, E, k);
  if (ws_bytes < w.total)
    return moe_fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, ws_bytes,
                    w.total);
  const long long es = moe_dt_bytes(dt), th = (long long)T * H * es, ih = (long long)I * H * es;
  const MoeRange rx = {x, th, "x"}, rg = {wg, 4LL * H * E, "wg"}, rb = {bias, 4LL * E, "bias"},
                 r13 = {w13, 2 * G * ih, "w13"}, r2 = {w2, G * ih, "w2"},
                 rs13 = {ws13, 2 * ih, "ws13"}, rs2 = {ws2, ih, "ws2"}, rr = {residual, th, "residual"},
                 outs[] = {{y, th, "y"}, {logits, 4LL * T * E, "logits"}, {idx, 4LL * T * k, "idx"},
                           {gate, 4LL * T * k, "gate"}, {ws, (long long)w.total, "ws"}};
  for (int i = 0; i < 5; ++i) {
    // (given logits are an input: apart from the outputs only; y may be residual's very buffer)
    const bool out = i != 1 || wg != nullptr;
    const char* with = out ? moe_shares(outs[i], {rx, rg, rb, r13, r2, rs13, rs2}) : nullptr;
    if (with == nullptr && out && !(i == 0 && residual == y)) with = moe_shares(outs[i], {rr});
    for (int j = 0; j < i && with == nullptr; ++j) with = moe_shares(outs[i], {outs[j]});
    if (with != nullptr)
      return moe_fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s's buffer (y may be residual's)", fn,
                      outs[i].name, with);
  }
  DecArgs a = {};
  a.x = x; a.wg = wg; a.bias = bias;
  a.T = T; a.H = H; a.I = I; a.E = E; a.k = k; a.g0 = g0; a.G = G;
  a.shared = ws13 != nullptr;
  a.w13 = w13; a.w2 = w2; a.ws13 = ws13; a.ws2 = ws2; a.residual = residual;
  a.logits = logits; a.idx = idx; a.gate = gate; a.y = y;
  a.S = wg != nullptr ? router_slices(H, E) : 0;
  a.gu_tiles = gateup_tiles(a.shared != 0, T, E, k);
  a.n_count = w.n_count;
  a.wait_ticks = (unsigned long long)g_wait_us * DEC_TICKS_PER_US;
  a.next = (int*)((char*)ws + w.count);
  a.routed = a.next + 32;
  a.unrouted = a.next + 64;
  a.act_done = a.next + 96;
  a.col_done = a.act_done + 32 * (E + 1);
  a.go = a.next + (96 + 32 * (E + 1) + H / DEC_DN + 31) / 32 * 32;
  a.part = (double*)((char*)ws + w.part);
  a.act = (char*)ws + w.act;
  a.yp = (float*)((char*)ws + w.yp);
  return dt == MOE_BF16 ? decode_launch<bf16_t>(a, (hipStream_t)stream, fn)
                        : decode_launch<float>(a, (hipStream_t)stream, fn);
}
