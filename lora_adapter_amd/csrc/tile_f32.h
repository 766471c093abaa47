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
// LDS, one barrier (of LDS alone: the loads stay in flight) a chunk, the loads two
// chunks ahead: with few workgroups on a CU one chunk's 0.4 us of MFMAs does not
// cover a load.  a(r, k) and b(r, k) give
// 4 values along k; with kBAcross b(c, k) gives row k's columns c .. c + 3.
// k_end - k_begin is a multiple of 32.
template <bool kBAcross, typename FA, typename FB>
__device__ __forceinline__ f32x16_t tile_f32(F32Tile &t, int k_begin, int k_end, const FA &fa, const FB &fb) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  f32x16_t acc = {};
  if (k_begin >= k_end) return acc;
  const int last = k_end - kF32K;
  float4 va[2][2], vb[2][2];
  // of a chunk past the end: the last one, which no one reads
  auto load = [&](int b, int k) __attribute__((always_inline)) {
    const int k0 = min(k, last);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (tid + i * 256) * 4;
      va[b][i] = fa(at / kF32K, k0 + at % kF32K);
      if constexpr (kBAcross) vb[b][i] = fb(at % 64, k0 + at / 64);
      else vb[b][i] = fb(at / kF32K, k0 + at % kF32K);
    }
  };
  auto put = [&](int b, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (tid + i * 256) * 4;
      float *p = &t.a[s][at / kF32K][at % kF32K];
      p[0] = va[b][i].x; p[1] = va[b][i].y; p[2] = va[b][i].z; p[3] = va[b][i].w;
      if constexpr (kBAcross) {
        const int c = at % 64, k = at / 64;
        t.b[s][c][k] = vb[b][i].x; t.b[s][c + 1][k] = vb[b][i].y;
        t.b[s][c + 2][k] = vb[b][i].z; t.b[s][c + 3][k] = vb[b][i].w;
      } else {
        float *q = &t.b[s][at / kF32K][at % kF32K];
        q[0] = vb[b][i].x; q[1] = vb[b][i].y; q[2] = vb[b][i].z; q[3] = vb[b][i].w;
      }
    }
  };
  const int ra = (wave >> 1) * 32 + (lane & 31), rb = (wave & 1) * 32 + (lane & 31), kh = lane >> 5;
  load(0, k_begin);
  load(1, k_begin + kF32K);
  put(0, 0);
  load(0, k_begin + 2 * kF32K);
  lds_bar();
  // the chunk from kc, in stage s
  auto chunk = [&](int s, int kc) __attribute__((always_inline)) {
    // operands of 4 MFMAs at a time, the next four's reads under them
    float xa[2][4], xb[2][4];
    auto read = [&](int g) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        xa[g & 1][q] = t.a[s][ra][8 * g + 2 * q + kh];
        xb[g & 1][q] = t.b[s][rb][8 * g + 2 * q + kh];
      }
    };
    read(0);
#pragma unroll
    for (int g = 0; g < kF32K / 8; ++g) {
      if (g + 1 < kF32K / 8) read(g + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(xa[g & 1][q], xb[g & 1][q], acc, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    put(s ^ 1, s ^ 1);
    load(s ^ 1, kc + 3 * kF32K);
    lds_bar();
  };
  // (both chunks of a turn without a branch between them: past one the compiler
  // would wait for every load)
  int k0 = k_begin;
  for (; k0 + kF32K < k_end; k0 += 2 * kF32K) {
    chunk(0, k0);
    chunk(1, k0 + kF32K);
  }
  if (k0 < k_end) chunk(0, k0);
  return acc;
}

// Row and column, in the tile, of this lane's register v.
__device__ __forceinline__ int f32_row(int v) {
  return (int(threadIdx.x) >> 7) * 32 + (v >> 2) * 8 + (int(threadIdx.x & 63) >> 5) * 4 + (v & 3);
}
__device__ __forceinline__ int f32_col() { return (int(threadIdx.x >> 6) & 1) * 32 + int(threadIdx.x & 31); }

}  // namespace
}  // namespace lora
