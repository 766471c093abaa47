// One workgroup's part of a decode GEMM (few tokens, bf16): shared by gemm.hip
// and gated.hip.  Internal to liblora (gfx950 only).
#pragma once

#include "gemm_tile.h"

namespace lora {
namespace {

// ------------------------------------------------------------ decode GEMM
// Few tokens (M <= 128): the product is a stream of W (d_in x d_out bf16)
// through HBM, and every W byte is used by one wave only.  A workgroup owns
// 128 output columns (32 per wave) and KC = 512 of K, and issues its whole
// W share at once, straight into the MFMA B-operand registers (32 loads of
// 16 bytes per lane, nothing staged in LDS), so a 1-workgroup-per-CU grid
// keeps ~128 KiB per CU in flight.  The token rows (shared by the 4 waves)
// go through LDS.  K is permuted inside each 64-wide group so that a lane's
// W loads are 64 contiguous bytes: in step s, lanes 0-31 contract k = 8s..8s+7
// and lanes 32-63 k = 32+8s..32+8s+7; the X fragments read from LDS use the
// same permutation, so the sum is unchanged.  Partial sums of the K splits go
// to the workspace for the epilogue kernel.
constexpr int kDecodeKC = 512;   // K elements per decode workgroup

// One decode tile: columns bx*128 .. +127, token rows by*32*MB .., K chunk bz.
// xs: LDS of MB*32*kDecodeKC bf16 for the token rows.
template <int MB>
__device__ __forceinline__ void decode_tile(const GemmArgs &g, int bx, int by, int bz,
                                            uint16_t *xs) {
  constexpr int KC = kDecodeKC;
  constexpr int NG = KC / 64;                 // 64-wide K groups
  constexpr int BMr = MB * 32;
  // One token row of the K chunk = 64 slots of 16 bytes.  Row r keeps chunk c
  // in slot c ^ (r & 15): the 16 rows that one quarter of a wave's fragment
  // read touches at once (same chunk) cover the 64 banks exactly once.
  const uint16_t *X = static_cast<const uint16_t *>(g.X);
  const uint16_t *W = static_cast<const uint16_t *>(g.W);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = bx * 128 + wave * 32;
  const int m0 = by * BMr;
  const int k0 = bz * KC;
  const int ng = min(NG, (g.Kd - k0) / 64);
  const int half = lane >> 5;

  // All loads are unconditional, from clamped addresses, so none waits on a
  // branch: rows past M and columns past N only feed outputs that are never
  // stored, and K groups past the end are skipped by the MFMA loop.
  // The token rows (mostly L2) go first, straight into LDS: wave w copies
  // rows w, w+4, ...; lane l of a copy fills slot l of the row.  The copies
  // are issued from inline asm, so the compiler does not hold every LDS read
  // until all loads have landed; the W stream (HBM) follows, and the MFMAs
  // of each 64-wide K group start as soon as its W fragments are in.
#pragma unroll
  for (int i = 0; i < BMr / 4; ++i) {
    const int r = wave + 4 * i;
    const int row = min(m0 + r, g.M - 1);
    const int chunk = lane ^ (r & 15);
    const int col = min(chunk * 8, ng * 64 - 8);
    lds_dma16(X + int64_t(row) * g.Kd + k0 + col, lds_addr(xs + r * KC));
  }
  // W fragments: row n0 + lane%32, k0 + 64*grp + 32*half + [0, 32)
  uint4 wf[NG][4];
  const uint16_t *wrow = W + int64_t(min(n0 + (lane & 31), g.N - 1)) * g.Kd + k0 + half * 32;
#pragma unroll
  for (int gq = 0; gq < NG; ++gq)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      wf[gq][q] = *reinterpret_cast<const uint4 *>(wrow + min(gq, ng - 1) * 64 + q * 8);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<NG * 4>();   // this wave's token rows have landed (its W loads came after them)
  lds_bar();              // and every wave's
  f32x16_t acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[b][v] = 0.f;
#pragma unroll
  for (int gq = 0; gq < NG; ++gq) {
    if (gq < ng) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8_t bfrag;
        __builtin_memcpy(&bfrag, &wf[gq][s], 16);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int r = b * 32 + (lane & 31);
          const int chunk = (gq * 64 + half * 32 + s * 8) / 8;
          const bf16x8_t afrag =
              *reinterpret_cast<const bf16x8_t *>(xs + r * KC + ((chunk ^ (r & 15)) * 8));
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(afrag, bfrag, acc[b], 0, 0, 0);
        }
      }
    }
  }
  // partials are read once, by the epilogue: streaming (non-temporal) stores
  float *Pz = g.partial + int64_t(bz) * g.M * g.N;
  const int col = n0 + (lane & 31);
  if (col < g.N) {
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = m0 + b * 32 + (v >> 2) * 8 + half * 4 + (v & 3);
        if (row < g.M) __builtin_nontemporal_store(acc[b][v], Pz + int64_t(row) * g.N + col);
      }
  }
}

}  // namespace
}  // namespace lora
