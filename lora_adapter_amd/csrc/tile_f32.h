// 64 x 64 tile of a float32 product on v_mfma_f32_32x32x2_f32, for layers in
// float32.  Internal to liblora (gfx950 only).
#pragma once

#include "gemm_tile.h"

namespace lora {
namespace {

constexpr int kF32K = 32;
struct F32Tile {
  float a[2][64][kF32K + 1], b[2][64][kF32K + 1];
};

// A 32 x 32 block of the tile for each of four waves: rows 32 (wave / 2), columns
// 32 (wave % 2), as the MFMA's registers hold them.  K in chunks of 32 through
// LDS, the next chunk's loads in flight while one feeds the MFMAs, one barrier a
// chunk.  a(r, k) and b(r, k) give 4 values along k; with kBAcross b(c, k) gives
// row k's columns c .. c + 3.  k_end - k_begin is a multiple of 32.
template <bool kBAcross, typename FA, typename FB>
__device__ __forceinline__ f32x16_t tile_f32(F32Tile &t, int k_begin, int k_end, const FA &fa, const FB &fb) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  f32x16_t acc = {};
  float4 va[2], vb[2];
  auto load = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (tid + i * 256) * 4;
      va[i] = fa(at / kF32K, k0 + at % kF32K);
      if constexpr (kBAcross) vb[i] = fb(at % 64, k0 + at / 64);
      else vb[i] = fb(at / kF32K, k0 + at % kF32K);
    }
  };
  auto put = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (tid + i * 256) * 4;
      float *p = &t.a[s][at / kF32K][at % kF32K];
      p[0] = va[i].x; p[1] = va[i].y; p[2] = va[i].z; p[3] = va[i].w;
      if constexpr (kBAcross) {
        const int c = at % 64, k = at / 64;
        t.b[s][c][k] = vb[i].x; t.b[s][c + 1][k] = vb[i].y; t.b[s][c + 2][k] = vb[i].z; t.b[s][c + 3][k] = vb[i].w;
      } else {
        float *q = &t.b[s][at / kF32K][at % kF32K];
        q[0] = vb[i].x; q[1] = vb[i].y; q[2] = vb[i].z; q[3] = vb[i].w;
      }
    }
  };
  const int ra = (wave >> 1) * 32 + (lane & 31), rb = (wave & 1) * 32 + (lane & 31), kh = lane >> 5;
  if (k_begin < k_end) {
    load(k_begin);
    put(0);
  }
  __syncthreads();
  int s = 0;
  for (int k0 = k_begin; k0 < k_end; k0 += kF32K, s ^= 1) {
    const bool more = k0 + kF32K < k_end;
    if (more) load(k0 + kF32K);
#pragma unroll
    for (int k = 0; k < kF32K; k += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(t.a[s][ra][k + kh], t.b[s][rb][k + kh], acc, 0, 0, 0);
    if (more) put(s ^ 1);
    __syncthreads();
  }
  return acc;
}

// Row and column, in the tile, of this lane's register v.
__device__ __forceinline__ int f32_row(int v) {
  return (int(threadIdx.x) >> 7) * 32 + (v >> 2) * 8 + (int(threadIdx.x & 63) >> 5) * 4 + (v & 3);
}
__device__ __forceinline__ int f32_col() { return (int(threadIdx.x >> 6) & 1) * 32 + int(threadIdx.x & 31); }

}  // namespace
}  // namespace lora
