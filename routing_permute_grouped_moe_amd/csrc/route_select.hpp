// Selection of the k largest logits of one token by one wavefront, shared by
// the routing call and the few-token layer.
#pragma once

#include "common.hpp"

// Order-preserving key of a finite logit: larger logit <-> larger key; -0 is
// taken as +0 so that equal logits have equal keys (ties go by index).
__device__ __forceinline__ uint32_t route_key(float v) {
  uint32_t u = __float_as_uint(v);
  u = (u == 0x80000000u) ? 0u : u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Top-k without cross-lane shuffles: the k-th largest key is found bit by bit
// from the top (a key bit is kept when at least k keys reach the prefix with
// it set; counts are wave ballots), the keys above it are chosen, and of the
// keys equal to it the ones with the lowest expert index fill the rest.  The
// slot of a chosen expert is the number of chosen experts ahead of it in the
// order (logit descending, index ascending) -- everything ahead of a chosen
// expert is chosen too.  Lane l's key i belongs to expert l + 64 i; padding
// (index >= E) holds key 0, below every finite logit's key, and k <= E.
// emit(slot, i) is called in the lane of each chosen expert.
template <int V, typename Emit>
__device__ __forceinline__ void route_select(const uint32_t (&key)[V], int k, Emit&& emit) {
  const int lane = threadIdx.x % MOE_WAVE;
  // the k-th largest key
  uint32_t K = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t c = K | (1u << b);
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) cnt += __popcll(__ballot(key[i] >= c));
    if (cnt >= k) K = c;
  }
  // chosen: keys above K, then ties at K by ascending index (i, then lane)
  int need = k;
#pragma unroll
  for (int i = 0; i < V; ++i) need -= __popcll(__ballot(key[i] > K));
  const unsigned long long below = (1ull << lane) - 1ull;
  bool sel[V];
  unsigned long long bsel[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const unsigned long long tie = __ballot(key[i] == K);
    sel[i] = key[i] > K || (key[i] == K && __popcll(tie & below) < need);
    const int nt = __popcll(tie);
    need -= need < nt ? need : nt;
    bsel[i] = __ballot(sel[i]);
  }
  // slots: chosen experts ahead of each chosen one
  int slot[V];
#pragma unroll
  for (int i = 0; i < V; ++i) slot[i] = 0;
#pragma unroll
  for (int i2 = 0; i2 < V; ++i2) {
    unsigned long long bm = bsel[i2];
    while (bm) {
      const int l2 = __builtin_ctzll(bm);
      bm &= bm - 1;
      const uint32_t k2 = (uint32_t)__builtin_amdgcn_readlane((int)key[i2], l2);
      const int e2 = l2 + i2 * MOE_WAVE;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + i * MOE_WAVE;
        slot[i] += (k2 > key[i]) || (k2 == key[i] && e2 < e);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (sel[i]) emit(slot[i], i);
}

// logits per lane of the kernel built for E <= 1024 experts: 1, 2, 4, 8 or 16
static inline int route_width(int E) {
  int v = 1;
  while (v * MOE_WAVE < E && v < 16) v *= 2;
  return v;
}
