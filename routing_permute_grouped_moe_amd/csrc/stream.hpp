// Products of a few rows with a long weight matrix: out[m, n] = sum_k a[m, k]
// w[n, k] for at most 128 rows m.  Such a product does 2 m flops for every
// weight it reads, far below the 300 flops per byte at which the matrix cores
// and HBM balance, so it is a stream of w, each byte read once, with the
// multiplications in its shade.
//
// Weights go straight from HBM to registers in the layout the MFMA takes them
// in (no LDS round trip: nothing is shared between waves): a 16 x 16 output
// tile reads 16 weight rows, 64 bytes of each per K step (lane l: row l % 16,
// 16 bytes at 16 (l / 16)).  The waves of a workgroup split K in chunks of CS
// steps dealt in turn, so together they read consecutive bytes of each row;
// their partial tiles are summed through LDS in wave order, which makes the
// result the same bits on every run.  Padding rows of a 16-row tile repeat a
// valid row and are dropped at the end.
#pragma once

#include "common.hpp"

// bytes of one row one K step covers: 32 bf16 or 16 fp32
#define STREAM_STEP 64
#define STREAM_OOB 0x80000000u

// One K step of a 16 x 16 tile: lane l holds 16 bytes of row (or column)
// l % 16 at K bytes 16 (l / 16).  The fp32 MFMA takes one float per lane, so
// its four MFMAs cover K in the order (l / 16, i) -- any order of K will do
// as long as both operands share it.
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

// Registers of one chunk: NTL weight tiles and, for each of AP planes of the
// row operand (two for a value kept as a sum of two bf16), MT row tiles.
template <int MT, int NTL, int AP, int CS>
struct StreamChunk {
  u32x4 w[CS][NTL];
  u32x4 a[CS][AP][MT];
};

// acc[mt][nt] += the products of this wave's chunks.  woff / aoff: byte offset
// of each lane's row and 16-byte column within the two descriptors; kbytes:
// bytes of a row along K (a multiple of STREAM_STEP).  D chunks of loads are
// in flight; a chunk past the end loads through an out-of-range offset, which
// reads zeros and moves nothing, so that every step of the ring looks alike.
template <typename T, int MT, int NTL, int AP, int CS, int NW, int D>
__device__ __forceinline__ void stream_product(f32x4 (&acc)[MT][NTL], __amdgpu_buffer_rsrc_t wr,
                                               const uint32_t (&woff)[NTL],
                                               __amdgpu_buffer_rsrc_t ar,
                                               const uint32_t (&aoff)[AP][MT], int kbytes,
                                               int wave) {
  const int steps = kbytes / STREAM_STEP;
  const int chunks = (steps + CS - 1) / CS;
  const int iters = (chunks + NW - 1) / NW;
  StreamChunk<MT, NTL, AP, CS> ring[D];
  auto load = [&](StreamChunk<MT, NTL, AP, CS>& b, int it) {
    const int s0 = (it * NW + wave) * CS;
#pragma unroll
    for (int s = 0; s < CS; ++s) {
      const bool ok = s0 + s < steps;
      const uint32_t k = (uint32_t)(s0 + s) * STREAM_STEP;
#pragma unroll
      for (int n = 0; n < NTL; ++n) b.w[s][n] = buf_load16_nt(wr, ok ? woff[n] + k : STREAM_OOB);
#pragma unroll
      for (int p = 0; p < AP; ++p)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          b.a[s][p][m] = buf_load16(ar, ok ? aoff[p][m] + k : STREAM_OOB);
    }
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) load(ring[d], d);
  for (int it = 0; it < iters; it += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(ring[(d + D - 1) % D], it + d + D - 1);
      const StreamChunk<MT, NTL, AP, CS>& b = ring[d];
#pragma unroll
      for (int s = 0; s < CS; ++s)
#pragma unroll
        for (int p = 0; p < AP; ++p)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NTL; ++n)
              acc[m][n] = stream_mma(b.a[s][p][m], b.w[s][n], acc[m][n], T());
    }
  }
}

// Steps of a chunk by the row tiles it serves: fewer where the row operand
// takes more registers.
template <int MT> constexpr int STREAM_CS = MT <= 1 ? 4 : MT <= 2 ? 2 : 1;

// Partial tiles of the NW waves, summed in wave order: red holds
// [wave][NTL][256] floats; the value of row m, column n of tile (mt, nt) is
// handed to consume(mt, nt, m, n, sum) by one thread.  Begins and ends with a
// barrier.
template <int MT, int NTL, int NW, typename Consume>
__device__ __forceinline__ void stream_reduce(const f32x4 (&acc)[MT][NTL], float* red,
                                              Consume&& consume) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[((wave * NTL + nt) * 4 + r) * 64 + lane] = acc[mt][nt][r];
    __syncthreads();
    for (int q = threadIdx.x; q < 256; q += NW * 64) {
      float v[NTL];
#pragma unroll
      for (int nt = 0; nt < NTL; ++nt) {
        float s = red[nt * 256 + q];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[(w * NTL + nt) * 256 + q];
        v[nt] = s;
      }
      // q = 64 r + lane of the tile's holder: row 4 (lane / 16) + r, column lane % 16
      consume(mt, 4 * ((q & 63) >> 4) + (q >> 6), q & 15, v);
    }
  }
  __syncthreads();
}
