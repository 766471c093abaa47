// The multi-adapter layer's products over e4m3 operands with one power-of-two
// scale per 128 of K (and, for the weight, per 128 x 128 block):
//   Y[t][n] = round( sum_b 2^(ex[t][b] + ew[n/128][b]) sum_{k in b} qx[t][k] qw[n][k] + expand )
// and the input gradient, the same product of the quantised dY rows with the
// codes of W^T.
//
// The scaled MFMA (v_mfma_scale_f32_32x32x64_f8f6f4, exponent bytes as its
// scale operands) multiplies at twice the bf16 rate and applies both scales
// itself, so one fp32 accumulator runs over the whole of K and no wave spends
// an instruction on scaling.  Inside one instruction the products are aligned
// to the largest of them before they are added, which cost 1.3e-5 (normal
// values) to 6e-5 (a few columns 40 times the rest) of the result's norm at K
// 64 .. 11008 (measured against 64 bits): a hundredth of the bf16 rounding
// that follows, but too much for an fp32 result.  fp32 layers therefore widen
// the codes to bf16 (exact) and run the bf16 MFMA (2e-7), each block's sum
// scaled as it is added to the fp32 total.
//
// Forms:
//   * split-K tiles of 128 columns by up to 128 rows (decode; fp32 layers of
//     any size by 32): the token rows are quantised by the workgroup that reads
//     them, straight into LDS, so a decode step has no quantising launch;
//   * 256 x 256 tiles with the LoRA expand in their epilogue, and 256 x 128
//     tiles that write fp32 partials: rows quantised ahead by one launch.
#include "gemm_tile.h"
#include "lora_internal.h"
#include "plan_build.h"
#include "quantise.h"
#include "shrink_units.h"

namespace lora {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kQDecodeKC = 512;           // K elements staged at a time (4 scale blocks)

__device__ __forceinline__ i32x8_t join32(uint4 a, uint4 b) {
  const i32x8_t r = {int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
  return r;
}

// Eight codes widened to bf16 (exact: 4 significant bits).
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(int(lo), false);
  const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(int(lo), true);
  const f32x2_t c = __builtin_amdgcn_cvt_pk_f32_fp8(int(hi), false);
  const f32x2_t d = __builtin_amdgcn_cvt_pk_f32_fp8(int(hi), true);
  const uint4 w = make_uint4(f2bf2(a[0], a[1]), f2bf2(b[0], b[1]), f2bf2(c[0], c[1]), f2bf2(d[0], d[1]));
  bf16x8_t r;
  __builtin_memcpy(&r, &w, 16);
  return r;
}

// cbsz = blgp = 0: both operands e4m3; SA, SB: the byte of each scale word.
template <int SA, int SB>
__device__ __forceinline__ f32x16_t mfma_q(i32x8_t a, i32x8_t b, f32x16_t c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, SA, sa, SB, sb);
}

// ------------------------------------------------------------ split-K tiles
// Columns bx*128 .. +127 (32 per wave), rows by*32*MB .., K from bz*k_split.
// Per 512 of K: every lane issues its share of W (64 bytes of each 128-byte
// block: lanes 0-31 the first half, 32-63 the second, the same permutation of
// K in both operands) into registers, then the workgroup quantises its token
// rows into LDS while those loads are in flight.
// A row's 512 codes are 32 slots of 16 bytes, chunk c in slot c ^ (row & 15):
// the 16 rows that a quarter wave reads at once cover the 64 banks once.
template <typename E, int MB>
__device__ __forceinline__ void q_split_tile(const QGemmArgs &q, int bx, int by, int bz,
                                             uint8_t *xs, uint32_t *ss) {
  constexpr int KC = kQDecodeKC, NG = KC / kQBlock, BMr = MB * 32;
  constexpr bool kExact = sizeof(E) == 4;
  const GemmArgs &g = q.g;
  const E *X = static_cast<const E *>(g.X);
  const uint8_t *W = static_cast<const uint8_t *>(g.W);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
  const int n0 = bx * 128 + wave * 32, m0 = by * BMr;
  const int kp = int(q.ldb);                       // K, padded to whole blocks
  const int k1 = min(kp, (bz + 1) * g.k_split);
  const uint8_t *wrow = W + int64_t(min(n0 + (lane & 31), g.N - 1)) * q.ldb + half * 64;
  const uint8_t *srow = q.sb + int64_t(bx) * q.lsb;
  f32x16_t acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[b][v] = 0.f;
  for (int k0 = bz * g.k_split; k0 < k1; k0 += KC) {
    const int ng = min(NG, (k1 - k0) / kQBlock);
    uint4 wf[NG][4];
#pragma unroll
    for (int gq = 0; gq < NG; ++gq)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        wf[gq][c] = *reinterpret_cast<const uint4 *>(wrow + k0 + min(gq, ng - 1) * kQBlock + c * 16);
    const int sw = *reinterpret_cast<const int *>(srow + k0 / kQBlock);
    if (k0 > bz * g.k_split) __syncthreads();      // every wave is done with the last chunk
    // 16 lanes per (row, block): 8 elements each; rows past M are zero codes
#pragma unroll
    for (int i = 0; i < BMr / 4; ++i) {
      const int it = i * 16 + (tid >> 4);
      const int r = it >> 2, blk = it & 3;
      const int c8 = blk * kQBlock + (tid & 15) * 8;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (m0 + r < g.M && k0 + c8 < g.Kd) Elem<E>::load8(X + int64_t(m0 + r) * g.Kd + k0 + c8, v);
      const uint32_t byte = q_scale_byte(max16(abs_max8(v)));
      *reinterpret_cast<uint2 *>(xs + r * KC + (((c8 >> 4) ^ (r & 15)) << 4) + (c8 & 8)) =
          q_encode8(v, byte);
      if ((tid & 15) == 0) reinterpret_cast<uint8_t *>(ss)[r * 4 + blk] = uint8_t(byte);
    }
    __syncthreads();
    auto group = [&](auto gi) __attribute__((always_inline)) {
      constexpr int G = decltype(gi)::value;
      if (G >= ng) return;
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const int r = b * 32 + (lane & 31);
        uint4 xa[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          xa[c] = *reinterpret_cast<const uint4 *>(
              xs + r * KC + (((G * 8 + half * 4 + c) ^ (r & 15)) << 4));
        if constexpr (!kExact) {
          const int sa = int(ss[r]);
#pragma unroll
          for (int s = 0; s < 2; ++s)
            acc[b] = mfma_q<G, G>(join32(xa[2 * s], xa[2 * s + 1]), join32(wf[G][2 * s], wf[G][2 * s + 1]),
                               acc[b], sa, sw);
        } else {
          f32x16_t p;
#pragma unroll
          for (int v = 0; v < 16; ++v) p[v] = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(xa[c].x, xa[c].y),
                                                        widen8(wf[G][c].x, wf[G][c].y), p, 0, 0, 0);
            p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(xa[c].z, xa[c].w),
                                                        widen8(wf[G][c].z, wf[G][c].w), p, 0, 0, 0);
          }
          // a block of scale byte 255 has NaN codes, so its sum is NaN already
          const int ew = ((sw >> (8 * G)) & 0xff) - 254;
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int row = b * 32 + (v >> 2) * 8 + half * 4 + (v & 3);
            acc[b][v] += ldexpf(p[v], int((ss[row] >> (8 * G)) & 0xffu) + ew);
          }
        }
      }
    };
    group(std::integral_constant<int, 0>{});
    group(std::integral_constant<int, 1>{});
    group(std::integral_constant<int, 2>{});
    group(std::integral_constant<int, 3>{});
  }
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

template <typename E, int MB>
__global__ __launch_bounds__(256) void q_split_kernel(QGemmArgs q) {
  __shared__ __attribute__((aligned(16))) uint8_t xs[MB * 32 * kQDecodeKC];
  __shared__ uint32_t ss[MB * 32];
  q_split_tile<E, MB>(q, blockIdx.x, blockIdx.y, blockIdx.z, xs, ss);
}

// The same tiles with the plan built by the launch's first workgroup (in the
// LDS of the token rows) and, for bf16 decode batches, the per-slot shrink
// after the tiles, four workgroups per slot: a decode forward is then this
// launch and the epilogue.  No part reads what another writes.
constexpr size_t kQPlanLds = 32 << 10;    // at least this for the plan

template <int MB>
struct QSplitLds {
  static constexpr size_t XS = size_t(MB) * 32 * kQDecodeKC, SS = size_t(MB) * 32 * 4;
  static constexpr size_t TOTAL = XS + SS > kQPlanLds ? XS + SS : kQPlanLds;
};

template <typename E, int MB, bool kMask, bool kLds>
__global__ __launch_bounds__(256) void q_split_plan_kernel(QGemmArgs q, SlotShrinkArgs ss, PlanArgs pa,
                                                            int gx, int gy, int n_gemm) {
  using L = QSplitLds<MB>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[L::TOTAL];
  const int t = int(blockIdx.x) - 1;
  if (t < 0) {
    plan_build<kLds>(pa, reinterpret_cast<int *>(lds));
    return;
  }
  if (t < n_gemm) {
    q_split_tile<E, MB>(q, t % gx, (t / gx) % gy, t / (gx * gy), lds,
                        reinterpret_cast<uint32_t *>(lds + L::XS));
    return;
  }
  if constexpr (sizeof(E) == 2) slot_shrink_part<kMask>(ss, (t - n_gemm) / kSlotParts, (t - n_gemm) % kSlotParts);
}

// ------------------------------------------------------------ pipelined tiles
// Tiles of BM x BN over K tiles of 128 codes (one scale block, 128 bytes per
// row: the LDS layout of the bf16 tiles), WM x WN waves.  NS stages: before
// the second half of K tile kt one barrier frees the stage just read for tile
// kt + NS and publishes tile kt + 1, whose first fragments are read under the
// second half's MFMAs.  A fragment is 32 bytes per lane; the A fragments of
// the next half replace each A block's registers after its last MFMA, the B
// fragments alternate between two sets.
// Scales: a stage ends with the 256 rows' bytes of its K tile, copied with the
// codes (rows r, r + 32, r + 64, r + 96 of a group of 128 share a dword, so a
// lane reads one for its four A blocks); the weight's bytes of the tile's
// column blocks lie in an LDS table for the whole of K.  The loop has no
// branch: with one, the compiler sinks the MFMAs past the copies and the
// barrier they are to cover.
template <int BM, int BN, int NS>
struct QTileLds {
  static constexpr int STAGE = (BM + BN) * 128 + BM;
  static constexpr int TABLE = NS * STAGE;
  static constexpr int TOTAL = TABLE + (BN / 128) * kQTableBytes;
};

// global_load_lds_dword: each lane copies 4 bytes to LDS at lds + 4 * lane
// (waits and m0 as in lds_dma16).
__device__ __forceinline__ void lds_dma4(const void *gptr, uint32_t lds) {
  const uint32_t lds_s = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(gptr), "s"(lds_s)
               : "memory", "m0");
}

// The expand of the 32-row blocks that the fused epilogue leaves (ranks over
// 16, or several slots per token): MFMA passes of 16 rank rows, one slot and
// one adapter at a time, into accumulators of their own, then added to the
// staged base product (times the keep mask with kMask), rounded and stored.
// Returns the blocks left to expand_nonfinite (whose test of every B fragment
// takes 3 to 4 % of a call whose adapters are in any order: 8192 x 4096 -> 4096,
// 16 adapters of ranks 2 .. 64 510 -> 532 us; in runs of rank 64 271 -> 272).
// One rolled loop over the blocks, apart from the fused epilogue: inside its
// unrolled blocks the same code slowed the common ones (8192 x 4096 -> 11008,
// rank 16: 357 -> 449 us).
template <int BM, int BN, int WM, int WN, bool kMask>
__device__ __forceinline__ unsigned q_expand_wide(const GemmArgs &g,
                                                  f32x16_t (&acc)[TileCfg<BM, BN, WM, WN>::TM]
                                                                 [TileCfg<BM, BN, WM, WN>::TN],
                                                  char *lds0, char *lds1, int m0, int n0, unsigned blocks) {
  using C = TileCfg<BM, BN, WM, WN>;
  constexpr int TM = C::TM, TN = C::TN, WC = TN * 32, SC = WC + 4, LPR = WC / 8, RPS = 64 / LPR;
  static_assert((C::NW / 2) * 40 * SC * 4 <= C::STAGE && RPS <= 8, "staging must fit in LDS");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / WN, wn = wave % WN, frow = lane & 31, half = lane >> 5;
  const uint16_t *Bp = static_cast<const uint16_t *>(g.ex.b_pages);
  char *const mem = wave < C::NW / 2 ? lds0 : lds1;
  float *stage = reinterpret_cast<float *>(mem) + (wave % (C::NW / 2)) * 32 * SC;
  float *lstage = reinterpret_cast<float *>(mem) + (C::NW / 2) * 32 * SC + (wave % (C::NW / 2)) * 8 * SC;
  uint16_t *Y = static_cast<uint16_t *>(g.Y);
  const int cbase = n0 + wn * WC, vr = lane / LPR, vc = (lane % LPR) * 8;
  const bool c8 = cbase + vc + 8 <= g.N;
  int key_ps = -1, key_j = -1;               // adapter slice held in bfr
  bool b_dropped = false;                    // .. less its non-finite values
  unsigned nonfinite = 0;
  bf16x8_t bfr[TN] = {};
  auto put = [&](const f32x16_t (&a)[TN]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) stage[((v >> 2) * 8 + half * 4 + (v & 3)) * SC + j * 32 + frow] = a[j][v];
  };
#pragma unroll 1
  for (int i = 0; i < TM; ++i) {
    if (!((blocks >> i) & 1u)) continue;
    // (acc is addressed by constants only)
#pragma unroll
    for (int b = 0; b < TM; ++b)
      if (b == i) put(acc[b]);
    f32x16_t l[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) l[j] = f32x16_t{};
    const int rbase = m0 + wm * TM * 32 + i * 32;
#pragma unroll 1
    for (int k = 0; k < g.ex.K; ++k) {
      int4 sd = g.ex.slot_desc[int64_t(min(rbase + frow, g.M - 1)) * g.ex.K + k];
      if (rbase + frow >= g.M) sd.x = -1;
      unsigned long long pending = __ballot(sd.x >= 0) & 0xffffffffull;
      while (pending) {
        const int leader = __ffsll(pending) - 1;
        const int kps = __builtin_amdgcn_readfirstlane(__shfl(sd.w, leader, 64));
        const int kr = __builtin_amdgcn_readfirstlane(__shfl(sd.y, leader, 64));
        const bool mine = sd.x >= 0 && sd.w == kps && sd.y == kr;
        pending &= ~__ballot(mine);
#pragma unroll 1
        for (int jb = 0; jb < kr; jb += 16) {
          const int rc = min(16, kr - jb);
          // A operand: U of row frow (zero unless the row is on this
          // adapter), rank rows jb + 8*half .. +7, as bf16 hi + lo
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int ja = half * 8 + e;
            u[e] = mine ? g.ex.U[sd.z + jb + min(ja, rc - 1)] : 0.f;
            if (ja >= rc) u[e] = 0.f;
          }
          if (kps != key_ps || jb != key_j) {
            // B operand: lane (column frow of block j, rank rows jb + 8*half .. +7)
            const int pidl = g.ex.page_ids[kps + jb + min(lane, rc - 1)];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
              const int cj = min(cbase + j * 32 + frow, g.N - 1);
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const int ja = half * 8 + e;
                uint32_t lo = Bp[int64_t(__shfl(pidl, ja, 64)) * g.ex.d_out + cj];
                uint32_t hi = Bp[int64_t(__shfl(pidl, ja + 1, 64)) * g.ex.d_out + cj];
                if (ja >= rc) lo = 0;
                if (ja + 1 >= rc) hi = 0;
                w4[e >> 1] = lo | (hi << 16);
              }
              const uint4 packed = make_uint4(w4[0], w4[1], w4[2], w4[3]);
              __builtin_memcpy(&bfr[j], &packed, 16);
            }
            b_dropped = drop_nonfinite<TN>(bfr);
            key_ps = kps;
            key_j = jb;
          }
          if (b_dropped) nonfinite |= 1u << i;
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const uint32_t h2 = f2bf2(u[e], u[e + 1]);
            hw[e >> 1] = h2;
            lw[e >> 1] = f2bf2(u[e] - bf_lo(h2), u[e + 1] - bf_hi(h2));
          }
          bf16x8_t ahi, alo;
          const uint4 ph = make_uint4(hw[0], hw[1], hw[2], hw[3]), pl = make_uint4(lw[0], lw[1], lw[2], lw[3]);
          __builtin_memcpy(&ahi, &ph, 16);
          __builtin_memcpy(&alo, &pl, 16);
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            l[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ahi, bfr[j], l[j], 0, 0, 0);
            l[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(alo, bfr[j], l[j], 0, 0, 0);
          }
        }
      }
    }
    // quarter qr: MFMA registers v = 4qr .. 4qr+3 hold rows 8qr .. 8qr+7
#pragma unroll
    for (int qr = 0; qr < 4; ++qr) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 4 * qr; v < 4 * qr + 4; ++v)
          lstage[(half * 4 + (v & 3)) * SC + j * 32 + frow] = l[j][v];
#pragma unroll
      for (int q = 0; q < 8 / RPS; ++q) {
        const int lr = q * RPS + vr, rr = qr * 8 + lr, row = rbase + rr;
        if (row >= g.M || !c8) continue;
        float b8[8], l8[8], v8[8];
        Elem<float>::load8(stage + rr * SC + vc, b8);
        Elem<float>::load8(lstage + lr * SC + vc, l8);
        uint2 mw = make_uint2(0x01010101u, 0x01010101u);
        if constexpr (kMask) mw = *reinterpret_cast<const uint2 *>(g.mask + int64_t(row) * g.N + cbase + vc);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t word = c < 4 ? mw.x : mw.y;
          v8[c] = kMask ? b8[c] + float((word >> (8 * (c & 3))) & 0xffu) * l8[c] : b8[c] + l8[c];
        }
        store8_nt(Y + int64_t(row) * g.N + cbase + vc, v8);
      }
    }
  }
  return nonfinite;
}

template <int BM, int BN, int WM, int WN, int NS, bool kFused, bool kMask = false>
__device__ __forceinline__ void q_tile_run(const QGemmArgs &q, char *smem, int m0, int n0, int kt0,
                                           int nk, int slot) {
  using C = TileCfg<BM, BN, WM, WN>;
  using Q = QTileLds<BM, BN, NS>;
  constexpr int TM = C::TM, TN = C::TN, NM = TM * TN, LPW = C::LPW + 1;
  static_assert(BM == 256 && (TM == 4 || TM == 2), "a lane's scale word holds its wave's row blocks");
  static_assert(BN % 128 == 0 && TN * 32 <= 128, "a wave's columns lie in one scale block");
  static_assert(NS >= 2 && (NS - 2) * LPW < 64, "stages / vmcnt range");
  const GemmArgs &g = q.g;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int frow = lane & 31, half = lane >> 5, lrow = lane >> 3;
  const uint8_t *abase = static_cast<const uint8_t *>(g.X) + int64_t(m0) * q.lda + int64_t(kt0) * kQBlock;
  const uint8_t *bbase = static_cast<const uint8_t *>(g.W) + int64_t(n0) * q.ldb + int64_t(kt0) * kQBlock;
  const uint8_t *sbase = q.sa + int64_t(kt0) * q.lsa + m0 + lane * 4;
  uint32_t aoff[C::A_INS], boff[C::B_INS];
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + lrow;
    aoff[i] = uint32_t(min(row, g.M - 1 - m0)) * uint32_t(q.lda) + tswz(row, lane & 7) * 16;
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = (wave * C::B_INS + i) * 8 + lrow;
    boff[i] = uint32_t(min(row, g.N - 1 - n0)) * uint32_t(q.ldb) + tswz(row, lane & 7) * 16;
  }
  // copy i of K tile kt: the wave's A rows, its B rows, the scale bytes (every
  // wave copies all 256, so that no wave has a branch of its own)
  auto dma_one = [&](char *base, int kt, int i) __attribute__((always_inline)) {
    const uint32_t lds = lds_addr(base);
    if (i < C::A_INS)
      lds_dma16(abase + kt * kQBlock + aoff[i], lds + (wave * C::A_INS + i) * 1024);
    else if (i < C::LPW)
      lds_dma16(bbase + kt * kQBlock + boff[i - C::A_INS],
                lds + BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
    else
      lds_dma4(sbase + int64_t(kt) * q.lsa, lds + C::STAGE);
  };

  EpiPre<TM> pre;
  if constexpr (kFused) epi_fetch_desc<BM, BN, WM, WN>(g, m0, pre);
  // the weight's scale bytes of the tile's column blocks, all of K
  for (int o = tid * 4; o < int(q.lsb) * (BN / 128); o += C::NT * 4) {
    const int blk = o / int(q.lsb), at = o % int(q.lsb);
    const int row = min(n0 / kQBlock + blk, (g.N - 1) / kQBlock);
    *reinterpret_cast<uint32_t *>(smem + Q::TABLE + blk * kQTableBytes + at) =
        *reinterpret_cast<const uint32_t *>(q.sb + row * q.lsb + at);
  }
  f32x16_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16_t{};

  i32x8_t fa[TM], fb0[TN], fb1[TN];
  auto frag = [&](const char *base, int s, int row) __attribute__((always_inline)) {
    const char *p = base + row * C::ROWB;
    const int c = tswz(frow, 4 * s + 2 * half);
    return join32(*reinterpret_cast<const uint4 *>(p + (c << 4)),
                  *reinterpret_cast<const uint4 *>(p + ((c ^ 1) << 4)));
  };
  auto frag_a = [&](const char *base, int s, int i) __attribute__((always_inline)) {
    return frag(base, s, wm * TM * 32 + i * 32 + frow);
  };
  auto frag_b = [&](const char *base, int s, int j) __attribute__((always_inline)) {
    return frag(base, s, BM + wn * TN * 32 + j * 32 + frow);
  };
  // (waves of two row blocks: the word's upper half for the odd ones)
  auto scale_a = [&](const char *base) __attribute__((always_inline)) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(base + C::STAGE + wm * TM / 4 * 128 + frow * 4);
    return int(TM == 4 ? w : w >> (16 * (wm & 1)));
  };
  const char *table = smem + Q::TABLE + (wn * TN * 32 / kQBlock) * kQTableBytes + kt0;
  // MFMAs of one half of a K tile from (fa, xb); the next half's fragments
  // come from src (half s_next), the copies of K tile kn go into dst (kCopy)
  auto kstep = [&](auto copy, i32x8_t (&xb)[TN], i32x8_t (&yb)[TN], const char *src, int s_next,
                   char *dst, int kn, int sa, int sb) __attribute__((always_inline)) {
    constexpr bool kCopy = decltype(copy)::value;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int i = m / TN, j = m % TN;
      switch (i) {
        case 0: acc[i][j] = mfma_q<0, 0>(fa[i], xb[j], acc[i][j], sa, sb); break;
        case 1: acc[i][j] = mfma_q<1, 0>(fa[i], xb[j], acc[i][j], sa, sb); break;
        case 2: acc[i][j] = mfma_q<2, 0>(fa[i], xb[j], acc[i][j], sa, sb); break;
        default: acc[i][j] = mfma_q<3, 0>(fa[i], xb[j], acc[i][j], sa, sb); break;
      }
      if (m < TN) yb[m] = frag_b(src, s_next, m);
      if (j == TN - 1) fa[i] = frag_a(src, s_next, i);
      if constexpr (kCopy) {
#pragma unroll
        for (int c = m * LPW / NM; c < (m + 1) * LPW / NM; ++c) dma_one(dst, kn, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int p = 0; p < NS; ++p) {
    // (past the end: the last tile again, into a stage that no one reads)
#pragma unroll
    for (int c = 0; c < LPW; ++c) dma_one(smem + p * Q::STAGE, min(p, nk - 1), c);
  }
  wait_vmcnt<0>();
  // the table is in LDS and every wave's first tiles have landed
  __syncthreads();
  if constexpr (kFused) epi_fetch_pid(g, pre);
  int sa = scale_a(smem), sb = uint8_t(table[0]);
#pragma unroll
  for (int i = 0; i < TM; ++i) fa[i] = frag_a(smem, 0, i);
#pragma unroll
  for (int j = 0; j < TN; ++j) fb0[j] = frag_b(smem, 0, j);
  int stage = 0;
  for (int kt = 0; kt < nk; ++kt) {
    char *const cur = smem + stage * Q::STAGE;
    stage = stage + 1 == NS ? 0 : stage + 1;
    char *const nxt = smem + stage * Q::STAGE;
    kstep(std::false_type{}, fb0, fb1, cur, 1, cur, 0, sa, sb);
    // tile kt + 1 has landed: everything but the copies of kt + 2 .. kt + NS - 1
    wait_vmcnt<(NS - 2) * LPW>();
    lds_bar();
    const int na = scale_a(nxt), nb = uint8_t(table[min(kt + 1, nk - 1)]);
    kstep(std::true_type{}, fb1, fb0, nxt, 0, cur, min(kt + NS, nk - 1), sa, sb);
    sa = na;
    sb = nb;
  }
  // the last copies have landed and every wave is done with the stages
  wait_vmcnt<0>();
  lds_bar();

  if constexpr (!kFused) {
    float *Pz = g.partial + int64_t(slot) * g.M * g.N;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int col = n0 + wn * TN * 32 + j * 32 + frow;
        if (col >= g.N) continue;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int row = m0 + wm * TM * 32 + i * 32 + (v >> 2) * 8 + half * 4 + (v & 3);
          if (row < g.M) __builtin_nontemporal_store(acc[i][j][v], Pz + int64_t(row) * g.N + col);
        }
      }
  } else {
    unsigned nf;
    const unsigned wide =
        fused_epilogue<BM, BN, WM, WN, kMask, true>(g, acc, smem, smem + C::STAGE, m0, n0, pre, nf);
    if (wide) nf |= q_expand_wide<BM, BN, WM, WN, kMask>(g, acc, smem, smem + C::STAGE, m0, n0, wide);
    if (nf) expand_nonfinite<TM, TN * 32, kMask>(g, m0 + wm * TM * 32, n0 + wn * TN * 32, nf);
  }
}

// Stream-K over g.sk_g workgroups: workgroup w takes the units (tile, K tile)
// [w U / G, (w + 1) U / G), the pieces as the epilogue counts them.
template <int BM, int BN, int WM, int WN, int NS>
__device__ __forceinline__ void q_stream_k(const QGemmArgs &q, char *smem, int w) {
  const GemmArgs &g = q.g;
  const int tiles_n = (g.N + BN - 1) / BN;
  const int ntiles = ((g.M + BM - 1) / BM) * tiles_n;
  const int KT = int(q.ldb) / kQBlock;
  const int64_t U = int64_t(ntiles) * KT;
  int64_t u = int64_t(w) * U / g.sk_g;
  const int64_t u1 = int64_t(w + 1) * U / g.sk_g;
  while (u < u1) {
    const int t = int(u / KT), kb = int(u % KT);
    const int ke = int(min<int64_t>(KT, kb + (u1 - u)));
    const int wf = int(((int64_t(t) * KT + 1) * g.sk_g - 1) / U);
    q_tile_run<BM, BN, WM, WN, NS, false>(q, smem, (t / tiles_n) * BM, (t % tiles_n) * BN, kb, ke - kb,
                                          w - wf);
    u += ke - kb;
  }
}

// Stream-K over workgroups 1 .. G, with the plan built by workgroup 0 in the
// LDS the others use for their stages.
template <int BM, int BN, int WM, int WN, int NS, bool kLds>
__global__ __launch_bounds__(WM * WN * 64, 1) void q_tile_plan_kernel(QGemmArgs q, PlanArgs pa) {
  __shared__ __attribute__((aligned(16))) char smem[QTileLds<BM, BN, NS>::TOTAL];
  if (blockIdx.x == 0) {
    plan_build<kLds>(pa, reinterpret_cast<int *>(smem));
    return;
  }
  q_stream_k<BM, BN, WM, WN, NS>(q, smem, int(blockIdx.x) - 1);
}

// Tiles as the bf16 form orders them (consecutive tiles on one XCD).  Split
// form: stream-K, or g.k_split of K per blockIdx.y.
template <int BM, int BN, int WM, int WN, int NS, bool kFused, bool kMask = false>
__global__ __launch_bounds__(WM * WN * 64, 1) void q_tile_kernel(QGemmArgs q) {
  __shared__ __attribute__((aligned(16))) char smem[QTileLds<BM, BN, NS>::TOTAL];
  const GemmArgs &g = q.g;
  const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
  const int ntiles = tiles_m * tiles_n;
  const int KT = int(q.ldb) / kQBlock;
  if constexpr (!kFused) {
    if (g.sk_g > 0) {
      q_stream_k<BM, BN, WM, WN, NS>(q, smem, int(blockIdx.x));
      return;
    }
  }
  const int per = (ntiles + 7) / 8;
  int b = int(blockIdx.x), half = -1;
  if constexpr (kFused && BN == 256) {
    // a grid larger than 8 * per asks for the last, partial round of tiles as
    // two 256 x 128 halves each (as in the bf16 tile kernel)
    const int nb = 8 * per, n_first = nb - nb % 256;
    if (int(gridDim.x) > nb && b >= n_first) {
      half = (b - n_first) & 1;
      b = n_first + (b - n_first) / 2;
    }
  }
  const int t = (b & 7) * per + (b >> 3);
  if (t >= ntiles) return;
  int tm, tn;
  tile_coords(t, tiles_m, tiles_n, tm, tn);
  const int k0 = blockIdx.y * (g.k_split / kQBlock);
  if (k0 >= KT) return;
  if constexpr (kFused && BN == 256) {
    if (half >= 0) {
      const int n0 = tn * BN + half * (BN / 2);
      if (n0 >= g.N) return;           // a half wholly past the last column
      q_tile_run<BM, BN / 2, 4, 2, NS, kFused, kMask>(q, smem, tm * BM, n0, k0,
                                                      min(KT - k0, g.k_split / kQBlock), blockIdx.y);
      return;
    }
  }
  q_tile_run<BM, BN, WM, WN, NS, kFused, kMask>(q, smem, tm * BM, tn * BN, k0,
                                                min(KT - k0, g.k_split / kQBlock), blockIdx.y);
}

}  // namespace

GemmConfig choose_quantised_gemm(int T, int few, int d_in, int d_out, int dtype) {
  GemmConfig c{};
  const int kb = int(q_row_bytes(d_in)) / kQBlock;
  if (dtype == LORA_F32 || T <= 128) {
    // decode: W streamed once, 512 of K per workgroup; with more tiles of
    // output (fp32 layers of many rows) a workgroup keeps more of K, down to
    // two workgroups per CU
    // (fp32: 32 rows always.  Their widened operands make a workgroup of 128
    // rows four times as long, and two of those are all that a CU holds: 669 x
    // 2496 -> 1472 63 -> 36 us, 3000 x 4096 -> 4096 733 -> 631 a forward)
    c.kind = 4; c.bn = 128;
    c.bm = T <= 32 || dtype == LORA_F32 ? 32 : (T <= 64 ? 64 : 128);
    const int chunks = (kb + 3) / 4;
    const int64_t tiles = int64_t((T + c.bm - 1) / c.bm) * ((d_out + 127) / 128);
    const int64_t want = (512 + tiles - 1) / tiles;
    const int splits = int(want < chunks ? want : chunks);
    const int per = (chunks + splits - 1) / splits;
    c.k_split = per * kQDecodeKC;
    c.splits = (chunks + per - 1) / per;
    return c;
  }
  // 256 x 256 tiles with the epilogue inside where they fill the GPU, or where
  // that is quicker for a prefill of few adapters.  With fewer tiles than CUs a
  // fused tile costs its CU 1.1 us per block of K whatever their number; the
  // split form spreads K over the GPU (6 ns a tile and block) but writes fp32
  // partials, reads them and finishes in a second launch (0.23 us a tile and 3
  // us).  Each adapter costs the fused epilogue a pass over the 32 rows that it
  // shares with others: nothing in runs of tokens, 3 us each in any order,
  // taken as 0.5.  Fused against split, whole calls, four adapters in runs: 80
  // tiles and 7 blocks of K (2048 x 832 -> 2496) 41 against 56 us, 128 and 32
  // (4096 x 4096 -> 2048) 81 against 105, 153 and 83 (the input gradient of
  // 4234 x 2304 -> 10560) 90 less; but 24 and 36 (2048 x 4544 -> 640) 78
  // against 60, 32 and 64 (2048 x 8192 -> 1024) 122 against 81.
  // (few counts the pool's adapters: the batch's own are known on the device
  // alone.)  From 256 tiles on the adapters are not asked for: in runs of four
  // 8192 x 11008 -> 4096 takes 400 us fused and 824 split, with 64 adapters of
  // ranks 2 .. 16 in any order 8192 x 4096 -> 4096 takes 353 and 388.  Blocks
  // that need q_expand_wide turn that round (two slots of rank 16: 488 and 426;
  // ranks 2 .. 64 of 16 adapters in any order: 536 and 461), but ranks are
  // known on the device alone too.
  const int64_t big = int64_t((T + 255) / 256) * ((d_out + 255) / 256);
  if (big >= 256 ||
      (few > 0 && T >= 1024 && big * (6 * kb + 230) + 3000 >= 1100 * int64_t(kb) + 500 * few)) {
    c.kind = 5; c.bm = 256; c.bn = 256;
    c.splits = 1; c.k_split = kb * kQBlock; c.fused = true;
    return c;
  }
  c.kind = 6; c.bm = 256; c.bn = 128;
  const int64_t tiles = int64_t((T + 255) / 256) * ((d_out + 127) / 128);
  const int64_t units = tiles * kb;
  constexpr int kWgs = 255;              // + 1 plan workgroup in launch_quantised_gemm_plan
  if (units >= 4 * kWgs) {
    const int64_t per = units / kWgs;
    c.sk = kWgs;
    c.k_split = kQBlock;
    c.splits = int((kb + per - 1) / per) + 1;
    return c;
  }
  const int64_t want = (kWgs + tiles - 1) / tiles;
  const int64_t most = kb / 4 > 1 ? kb / 4 : 1;        // every split keeps >= 512 of K
  const int splits = int(want < most ? want : most);
  const int per = (kb + splits - 1) / splits;
  c.k_split = per * kQBlock;
  c.splits = (kb + per - 1) / per;
  return c;
}

hipError_t launch_quantised_gemm(const GemmConfig &c, const QGemmArgs &q, int dtype, hipStream_t s) {
  const GemmArgs &g = q.g;
  if (c.kind == 4) {
    const dim3 grid((g.N + 127) / 128, (g.M + c.bm - 1) / c.bm, c.splits), block(256);
    if (dtype == LORA_F32) hipLaunchKernelGGL((q_split_kernel<float, 1>), grid, block, 0, s, q);
    else if (c.bm == 32) hipLaunchKernelGGL((q_split_kernel<uint16_t, 1>), grid, block, 0, s, q);
    else if (c.bm == 64) hipLaunchKernelGGL((q_split_kernel<uint16_t, 2>), grid, block, 0, s, q);
    else hipLaunchKernelGGL((q_split_kernel<uint16_t, 4>), grid, block, 0, s, q);
    return hipGetLastError();
  }
  if (dtype != LORA_BF16) return hipErrorInvalidConfiguration;
  const int tiles = ((g.M + c.bm - 1) / c.bm) * ((g.N + c.bn - 1) / c.bn);
  if (c.kind == 5) {
    unsigned gx = 8 * ((tiles + 7) / 8);
    const unsigned nf = gx - gx % 256, rem = gx - nf;
    if (nf > 0 && rem > 0 && rem <= 128) gx = nf + 2 * rem;
    const dim3 grid(gx);
    if (g.mask) hipLaunchKernelGGL((q_tile_kernel<256, 256, 2, 4, 2, true, true>), grid, dim3(512), 0, s, q);
    else hipLaunchKernelGGL((q_tile_kernel<256, 256, 2, 4, 2, true>), grid, dim3(512), 0, s, q);
    return hipGetLastError();
  }
  if (c.kind == 6 && !g.mask) {
    const dim3 grid = c.sk > 0 ? dim3(c.sk) : dim3(8 * ((tiles + 7) / 8), c.splits);
    hipLaunchKernelGGL((q_tile_kernel<256, 128, 2, 2, 3, false>), grid, dim3(256), 0, s, q);
    return hipGetLastError();
  }
  return hipErrorInvalidConfiguration;
}

bool quantised_gemm_plan_fusable(const GemmConfig &c) { return c.kind == 4 || (c.kind == 6 && c.sk > 0); }

size_t quantised_plan_lds_cap(const GemmConfig &c) {
  if (c.kind != 4) return QTileLds<256, 128, 3>::TOTAL;
  return c.bm == 32 ? QSplitLds<1>::TOTAL : c.bm == 64 ? QSplitLds<2>::TOTAL : QSplitLds<4>::TOTAL;
}

hipError_t launch_quantised_gemm_plan(const GemmConfig &c, const QGemmArgs &q, const SlotShrinkArgs *ss,
                                      const PlanLaunch &pl, int dtype, hipStream_t s) {
  const GemmArgs &g = q.g;
  if (!quantised_gemm_plan_fusable(c) || pl.lds_bytes > quantised_plan_lds_cap(c))
    return hipErrorInvalidConfiguration;
  if (c.kind == 6) {
    const dim3 grid(unsigned(1 + c.sk)), block(256);
    if (pl.lds) hipLaunchKernelGGL((q_tile_plan_kernel<256, 128, 2, 2, 3, true>), grid, block, 0, s, q, pl.a);
    else hipLaunchKernelGGL((q_tile_plan_kernel<256, 128, 2, 2, 3, false>), grid, block, 0, s, q, pl.a);
    return hipGetLastError();
  }
  const int gx = (g.N + 127) / 128, gy = (g.M + c.bm - 1) / c.bm;
  const int n_gemm = gx * gy * c.splits;
  const dim3 grid(unsigned(1 + n_gemm + (ss ? kSlotParts * ss->n_slots : 0))), block(256);
  const SlotShrinkArgs sa = ss ? *ss : SlotShrinkArgs{};
#define LORA_QP3(E, MB, M, L) \
  hipLaunchKernelGGL((q_split_plan_kernel<E, MB, M, L>), grid, block, 0, s, q, sa, pl.a, gx, gy, n_gemm)
#define LORA_QP2(E, MB, M) do { if (pl.lds) LORA_QP3(E, MB, M, true); else LORA_QP3(E, MB, M, false); } while (0)
#define LORA_QP(MB) \
  do { \
    if (sa.mask) LORA_QP2(uint16_t, MB, true); \
    else LORA_QP2(uint16_t, MB, false); \
  } while (0)
  if (dtype == LORA_F32) LORA_QP2(float, 1, false);
  else if (c.bm == 32) LORA_QP(1);
  else if (c.bm == 64) LORA_QP(2);
  else LORA_QP(4);
#undef LORA_QP
#undef LORA_QP2
#undef LORA_QP3
  return hipGetLastError();
}

}  // namespace lora
