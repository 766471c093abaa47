// The K loop of a bf16 output tile over two to four LDS stages, for the products of
// the gated block (two weights side by side, or two products added along K)
// and of the cross entropy (weights read along their other axis).
// Internal to liblora (gfx950 only).
//
// v_mfma_f32_16x16x32_bf16 with scalar-based copies: on 8192 x 8192 x 4096 a
// 256 x 256 tile of eight waves runs at 1480 TFLOP/s in a steady state, where
// 32x32x16 MFMAs and copies with 64-bit lane addresses reach 1270.  The card's
// power limit sets the clock there (1.7 of 2.4 GHz): the 16x16x32 form moves
// its accumulators a quarter as often per product, and a copy with a scalar
// base and a constant 32-bit lane offset has no address arithmetic.
#pragma once

#include "gemm_tile.h"

namespace lora {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));

// A tile of BM x BN over WM x WN waves, in blocks of 16 x 16, with NS LDS stages.
template <int BM_, int BN_, int WM_, int WN_, int NS_ = 2>
struct LoopCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int ROWB = 128;                     // bytes per row of 64 of K
  static constexpr int STAGE = (BM + BN) * ROWB;       // bytes per LDS stage
  static constexpr int TM = BM / (WM * 16), TN = BN / (WN * 16);
  static constexpr int A_INS = BM / 8 / NW, B_INS = BN / 8 / NW, LPW = A_INS + B_INS;
  static constexpr int LDS = NS * STAGE;
  static_assert(A_INS * 8 * NW == BM && B_INS * 8 * NW == BN, "tile rows / waves");
  static_assert(NS >= 2 && (NS - 1) * LPW < 64, "stages, and the copies that may be in flight");
};

// The shapes, one workgroup on a CU each, and the time of a K tile on a full card
// in units of about 0.17 us (measured with 64 K tiles: 107, 95, 62 and 40 us).
// The larger ones do more with what they read; which one is fastest depends on
// how well a problem's tiles divide into rounds of 256 CUs.
using Big = LoopCfg<256, 256, 2, 4>;
using Tall = LoopCfg<192, 256, 2, 4>;
using Mid = LoopCfg<128, 256, 2, 4, 3>;
using Small = LoopCfg<128, 128, 2, 2, 4>;
struct TileShape {
  int bm, bn, cost;
};
constexpr TileShape kTileShapes[4] = {{256, 256, 10}, {192, 256, 9}, {128, 256, 6}, {128, 128, 4}};
enum { kBig, kTall, kMid, kSmall };

// Tiles of an M x N output.
inline int64_t tile_count(int shape, int64_t M, int64_t N) {
  const TileShape &t = kTileShapes[shape];
  return ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
}
// The shape whose rounds over the CUs cost least; `more`: further workgroups in the launch.
inline int pick_shape(int64_t M, int64_t N, int64_t more = 0) {
  int best = 0;
  int64_t least = 0;
  for (int i = 0; i < 4; ++i) {
    const int64_t c = kTileShapes[i].cost * ((tile_count(i, M, N) + more + 255) / 256);
    if (i == 0 || c < least) {
      best = i;
      least = c;
    }
  }
  return best;
}

// One 16-byte copy per lane from base + off to LDS at lds + 16 lane; base and
// lds are the wave's.  (The s_nop: an LDS DMA needs a wait state after the scalar
// write of m0.  The readfirstlanes: a uniform value may have come out of vector
// arithmetic, where the compiler leaves it; of a scalar one they are nothing.)
__device__ __forceinline__ void lds_dma16_s(const void *ptr, uint32_t off, uint32_t lds) {
  const uint64_t p = reinterpret_cast<uint64_t>(ptr);
  const uint64_t base = uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(p)))) |
                        uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(p >> 32)))) << 32;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

// Where a lane's pieces of n copies' rows lie, from a base that moves along K:
// 32-bit byte offsets, or (kWide) 64 bits where the rows pass 2^32 bytes.
template <int n, bool kWide>
struct RowOffsets {
  uint32_t o[kWide ? 1 : n];
  int64_t w[kWide ? n : 1];
  __device__ __forceinline__ void set(int i, int64_t elements) {
    if constexpr (kWide) w[i] = elements;
    else o[i] = uint32_t(elements) * 2;
  }
  __device__ __forceinline__ void copy(const uint16_t *base, int i, uint32_t lds) const {
    if constexpr (kWide) lds_dma16(base + w[i], lds);
    else lds_dma16_s(base, o[i], lds);
  }
};

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6); }

// LDS slot of 16-byte chunk c (0 .. 7) of a tile row.  A 16-byte LDS read of a wave
// goes in four groups of 16 lanes, {0 .. 3, 12 .. 15, 20 .. 27}, {4 .. 11, 16 .. 19,
// 28 .. 31} and the same 32 higher; of a fragment's reads (rows lane % 16, chunk
// 4 s + lane / 16) each group then covers the 64 banks once.  (tswz, made for 32-row
// fragments, gives two lanes of a group the same banks here: SQ_LDS_BANK_CONFLICT 23 %
// of the cycles of a prefill instead of 0.6 %, and 2.5 to 4 % more cycles.  The time is
// the same: the power limit gives them back as clock.)
__device__ __forceinline__ int fswz(int row, int c) { return c ^ (row & 7); }

// Fragment of 16 rows from `row0` (a multiple of 16) of a stage whose rows are
// 64 of K in fswz order: lane (row lane % 16, k of 8 (lane / 16) .. + 7) of
// 32-wide K step s.
__device__ __forceinline__ bf16x8_t frag_rows(const char *base, int s, int row0) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const bf16x8_t *>(base + row0 * 128 + (lane & 15) * 128 +
                                             (fswz(lane & 15, 4 * s + (lane >> 4)) << 4));
}

// acc += A.B over nk K tiles of 64.  Src: `copy(lds, kt, i)` issues copy i of
// the wave's LPW copies of K tile kt into the stage at LDS address lds;
// `frag(base, s, q)` reads fragment q (A blocks 0 .. TM-1, then B blocks) of K
// step s from the stage at base.
// The fragments of a step are read from LDS while the MFMAs of the step before
// run (two register sets).  K tile kt lies in stage kt % NS.  Between the two
// steps of a K tile one barrier frees the stage just read (the copies of tile
// kt + NS go into it, spread over the second step's MFMAs) and publishes the
// next tile.  The instructions of a step are pinned in this order; every other
// row of blocks runs backwards, so that one operand of an MFMA is always the
// last one's.  On return no copy is in flight and every wave is done with the
// stages.
template <typename C, typename Src>
__device__ __forceinline__ void tile_loop(const Src &p, char *smem, int nk, f32x4_t (&acc)[C::TM][C::TN]) {
  constexpr int TM = C::TM, TN = C::TN, NM = TM * TN, NQ = TM + TN, LPW = C::LPW, NS = C::NS;
  const uint32_t l0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (nk <= 0) return;

  bf16x8_t fa0[TM], fb0[TN], fa1[TM], fb1[TN];
  // copies: mode 1 issues those of tile kn into the stage at `dst`
  auto step = [&](auto mode, bf16x8_t (&xa)[TM], bf16x8_t (&xb)[TN], bf16x8_t (&ya)[TM], bf16x8_t (&yb)[TN],
                  const char *src, int s, uint32_t dst, int kn) __attribute__((always_inline)) {
    constexpr bool kCopy = decltype(mode)::value != 0;
    // a fragment read after every kPer-th MFMA
    constexpr int kPer = NM >= 2 * NQ ? 2 : 1;
    static_assert(NM >= NQ, "a fragment read after an MFMA each");
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int i = m / TN, j = (i & 1) ? TN - 1 - m % TN : m % TN;
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[i], xb[j], acc[i][j], 0, 0, 0);
      if (m % kPer == 0 && m / kPer < NQ) {
        const int q = frag_order<TM, TN>(m / kPer);
        if (q < TM) ya[q] = p.frag(src, s, q);
        else yb[q - TM] = p.frag(src, s, q);
      }
      if constexpr (kCopy) {
#pragma unroll
        for (int c = m * LPW / NM; c < (m + 1) * LPW / NM; ++c) p.copy(dst, kn, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int t = 0; t < NS; ++t)
#pragma unroll
    for (int c = 0; c < LPW; ++c) p.copy(l0 + t * C::STAGE, min(t, nk - 1), c);
  wait_vmcnt<(NS - 1) * LPW>();
  lds_bar();
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    if (q < TM) fa0[q] = p.frag(smem, 0, q);
    else fb0[q - TM] = p.frag(smem, 0, q);
  }
  // past the end the body stays the same: the copies repeat the last tile into
  // stages that no one reads again, and the reads of the next stage go unused
  auto tile = [&](int kt, int cur, int nxt) __attribute__((always_inline)) {
    step(std::integral_constant<int, 0>{}, fa0, fb0, fa1, fb1, smem + cur * C::STAGE, 1, 0, 0);
    wait_vmcnt<(NS - 2) * LPW>();   // tile kt + 1 has landed
    lds_bar();                      // for every wave, and every wave has read tile kt
    step(std::integral_constant<int, 1>{}, fa1, fb1, fa0, fb0, smem + nxt * C::STAGE, 0, l0 + cur * C::STAGE,
         min(kt + NS, nk - 1));
  };
  int kt = 0;
  for (; kt + NS <= nk; kt += NS) {
#pragma unroll
    for (int u = 0; u < NS; ++u) tile(kt + u, u, (u + 1) % NS);
  }
#pragma unroll
  for (int u = 0; u < NS - 1; ++u)
    if (kt + u < nk) tile(kt + u, u, u + 1);
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

// The same for `splits` parts of K of each tile: the tiles of one part lie
// together, on XCDs that hold its rows of both operands.
__device__ __forceinline__ bool tile_of_workgroup(int b, int tiles_m, int tiles_n, int splits, int &tm, int &tn, int &z) {
  const int n = tiles_m * tiles_n, per = (n * splits + 7) / 8;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= n * splits) return false;
  z = __builtin_amdgcn_readfirstlane(t / n);
  tile_coords(t - z * n, tiles_m, tiles_n, tm, tn);
  return true;
}

// Row of the wave's part of the tile that lane's register v of block i holds,
// and its column in block j.
__device__ __forceinline__ int acc_row(int i, int v) { return i * 16 + (int(threadIdx.x & 63) >> 4) * 4 + v; }
__device__ __forceinline__ int acc_col(int j) { return j * 16 + int(threadIdx.x & 15); }

}  // namespace
}  // namespace lora
