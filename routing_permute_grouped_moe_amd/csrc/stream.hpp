// Products of a few rows with a long weight matrix: out[m, n] = sum_k a[m, k]
// w[n, k] for at most 128 rows m.  Such a product does 2 m flops for every
// weight it reads, far below the 300 flops per byte at which the matrix cores
// and HBM balance, so it is a stream of w, each byte read once, with the
// multiplications in its shade.
//
// K runs in steps of 128 bytes of a row (64 bf16, 32 fp32), dealt to the waves
// of a workgroup in turn.  A 16-row tile of a step (2 KB) goes HBM -> LDS in two
// copies of 8 whole 128-byte lines each, into a ring that belongs to one wave:
// read that way with the streaming policy HBM gives 7.0 TB/s here, against 5.1
// TB/s for loads straight into the MFMA's operand layout (16 rows x 64 bytes,
// 6.2 TB/s without the policy).  16-byte chunk c of row r sits in slot c ^ ((r
// >> 1) & 7) of its row, so the 16 rows of a fragment read hit all banks.
#pragma once

#include "lds_copy.hpp"

#define STREAM_STEP 128          // bytes of a row a step covers
#define STREAM_TILE 2048         // bytes of a 16-row tile of a step
#define STREAM_OOB 0x80000000u   // past every operand: reads zeros, moves nothing

// Byte offset of this lane's 16 bytes of copy j of a tile (rows 8 j .. 8 j + 7)
// within its row, and the row.
__device__ __forceinline__ int stream_row(int j) { return 8 * j + ((threadIdx.x & 63) >> 3); }
__device__ __forceinline__ uint32_t stream_chunk(int j) {
  const int r = stream_row(j);
  return (uint32_t)(((threadIdx.x & 7) ^ ((r >> 1) & 7)) << 4);
}
// Byte of this lane's 16 in a tile, for half h of a step: row lane % 16, chunk
// 4 h + lane / 16 -- the MFMA's operand layout.
__device__ __forceinline__ int stream_frag(int h) {
  const int lane = threadIdx.x & 63, r = lane & 15;
  return r * STREAM_STEP + (((4 * h + (lane >> 4)) ^ ((r >> 1) & 7)) << 4);
}

// A copy with the streaming policy, for what is read once.
__device__ __forceinline__ void dma16_nt(const i32x4& rs, uint32_t lds, uint32_t voff, int soff) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               :
               : "v"(voff), "s"(rs), "s"(uniform(soff)), "s"(uniform((int)lds))
               : "memory", "m0");
}

__device__ __forceinline__ void lds_drain() {   // this wave's LDS accesses have happened
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}
template <int n>
__device__ __forceinline__ void vm_drain() {    // all but n of its memory operations have
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

// Half a step of a 16 x 16 tile: lane l holds 16 bytes of row (or column) l % 16
// at K bytes 16 (l / 16).  The fp32 MFMA takes one float per lane, so its four
// MFMAs cover K in the order (l / 16, i) -- any order of K will do as long as
// both operands share it.
__device__ __forceinline__ f32x4 stream_mma(const u32x4& a, const u32x4& b, f32x4 c, bf16_t) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 stream_mma(const u32x4& a, const u32x4& b, f32x4 c, float) {
  const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i], fb[i], c, 0, 0, 0);
  return c;
}
