// The K loop of a bf16 output tile over two LDS stages, for products whose
// operands are not plain rows of two matrices: the gated block (two weights
// side by side, or two products added along K) and the cross entropy (weights
// read along their other axis).  Internal to liblora (gfx950 only).
#pragma once

#include "gemm_tile.h"

namespace lora {
namespace {

typedef short v4i16_t __attribute__((ext_vector_type(4)));

// Where a tile's operands come from.  `copy(lds, kt, i)` issues copy i of the
// wave's TileCfg::LPW copies of K tile kt (64 of K) into the stage at LDS
// address lds; `frag(base, s, q)` reads fragment q (A blocks 0 .. TM-1, then B
// blocks) of 16-wide K step s from the stage at base.
//
// Rows of 64 of K, 128 bytes each, in tswz order: the A operand everywhere and
// the B operand of products with both sides along K.
template <typename C, int WN>
__device__ __forceinline__ bf16x8_t frag_rows(const char *base, int s, int row) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const bf16x8_t *>(base + row * C::ROWB + (tswz(lane & 31, 2 * s + (lane >> 5)) << 4));
}

// The loop: acc += A.B over nk K tiles.  The fragments of K step s + 1 are
// read from LDS while the MFMAs of step s run (two register sets); before the
// last step of a K tile one barrier frees the stage just read (the copies of
// the tile after next go into it, spread over that step's MFMAs) and publishes
// the next tile.  Each step's instructions are pinned in this order.  On
// return no copy is in flight and every wave is done with the stages.
template <int BM, int BN, int WM, int WN, typename P>
__device__ __forceinline__ void tile_loop(const P &p, char *smem, int nk,
                                          f32x16_t (&acc)[TileCfg<BM, BN, WM, WN>::TM]
                                                         [TileCfg<BM, BN, WM, WN>::TN]) {
  using C = TileCfg<BM, BN, WM, WN>;
  constexpr int TM = C::TM, TN = C::TN;
  char *const st0 = smem;
  char *const st1 = smem + C::STAGE;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  if (nk <= 0) return;

  bf16x8_t fa0[TM], fb0[TN], fa1[TM], fb1[TN];
  auto kstep = [&](auto mode, bf16x8_t (&xa)[TM], bf16x8_t (&xb)[TN], bf16x8_t (&ya)[TM],
                   bf16x8_t (&yb)[TN], const char *src, int s_next, char *dst,
                   int kn) __attribute__((always_inline)) {
    constexpr int MD = decltype(mode)::value;   // bit 0: read the next fragments, bit 1: copy tile kn
    constexpr int NM = TM * TN, NQ = TM + TN;
    static_assert(NQ <= NM, "one fragment read after each of the first MFMAs");
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      acc[m / TN][m % TN] =
          __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[m / TN], xb[m % TN], acc[m / TN][m % TN], 0, 0, 0);
      if constexpr ((MD & 1) != 0) {
        const int q = frag_order<TM, TN>(m);
        if (m < NQ) {
          if (q < TM) ya[q] = p.frag(src, s_next, q);
          else yb[q - TM] = p.frag(src, s_next, q);
        }
      }
      if constexpr ((MD & 2) != 0) {
#pragma unroll
        for (int c = m * C::LPW / NM; c < (m + 1) * C::LPW / NM; ++c) p.copy(lds_addr(dst), kn, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int c = 0; c < C::LPW; ++c) p.copy(lds_addr(st0), 0, c);
  if (nk > 1) {
#pragma unroll
    for (int c = 0; c < C::LPW; ++c) p.copy(lds_addr(st1), 1, c);
    wait_vmcnt<C::LPW>();
  } else {
    wait_vmcnt<0>();
  }
  lds_bar();
#pragma unroll
  for (int q = 0; q < TM + TN; ++q) {
    if (q < TM) fa0[q] = p.frag(st0, 0, q);
    else fb0[q - TM] = p.frag(st0, 0, q);
  }
  // past the end the body stays the same: the copy repeats the last tile into
  // a stage no one reads again, and the reads of nxt go unused
  for (int kt = 0; kt < nk; ++kt) {
    char *const cur = (kt & 1) ? st1 : st0;
    char *const nxt = (kt & 1) ? st0 : st1;
    kstep(std::integral_constant<int, 1>{}, fa0, fb0, fa1, fb1, cur, 1, cur, 0);
    kstep(std::integral_constant<int, 1>{}, fa1, fb1, fa0, fb0, cur, 2, cur, 0);
    kstep(std::integral_constant<int, 1>{}, fa0, fb0, fa1, fb1, cur, 3, cur, 0);
    wait_vmcnt<0>();   // tile kt + 1, the only copies in flight, has landed
    lds_bar();         // for every wave, and every wave has read cur
    kstep(std::integral_constant<int, 3>{}, fa1, fb1, fa0, fb0, nxt, 0, cur, min(kt + 2, nk - 1));
  }
  wait_vmcnt<0>();
  lds_bar();
}

// Output tile t of tiles_m x tiles_n for workgroup b: the workgroups that the
// hardware places on one XCD (ids equal mod 8) take consecutive tiles, walked
// 4 tile rows at a time.  False past the end.
__device__ __forceinline__ bool tile_of_workgroup(int b, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int per = (tiles_m * tiles_n + 7) / 8;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= tiles_m * tiles_n) return false;
  tile_coords(t, tiles_m, tiles_n, tm, tn);
  return true;
}

}  // namespace
}  // namespace lora
