// Device code shared by the tile GEMMs (gemm.hip: bf16 operands;
// gemm_quantised.hip: e4m3 operands): wide loads and stores, the LoRA expand
// of a row, LDS copies and waits, tile shapes and the fused epilogue.
// Internal to liblora (gfx950 only).
#pragma once

#include "lora_internal.h"

namespace lora {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------ vector loads/stores
template <typename E, int CPL> struct Cols;
template <> struct Cols<uint16_t, 1> {
  static __device__ __forceinline__ void load(const uint16_t *p, float v[1]) { v[0] = bf2f(*p); }
  static __device__ __forceinline__ void store(uint16_t *p, const float v[1]) { *p = f2bf(v[0]); }
};
template <> struct Cols<uint16_t, 2> {
  static __device__ __forceinline__ void load(const uint16_t *p, float v[2]) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    v[0] = bf_lo(w); v[1] = bf_hi(w);
  }
  static __device__ __forceinline__ void store(uint16_t *p, const float v[2]) {
    *reinterpret_cast<uint32_t *>(p) = f2bf2(v[0], v[1]);
  }
};
template <> struct Cols<uint16_t, 8> {
  static __device__ __forceinline__ void load(const uint16_t *p, float v[8]) { Elem<uint16_t>::load8(p, v); }
  static __device__ __forceinline__ void store(uint16_t *p, const float v[8]) {
    uint4 w;
    w.x = f2bf2(v[0], v[1]);
    w.y = f2bf2(v[2], v[3]);
    w.z = f2bf2(v[4], v[5]);
    w.w = f2bf2(v[6], v[7]);
    *reinterpret_cast<uint4 *>(p) = w;
  }
};
// 8 bf16 values, one 16-byte streaming store (Y is written once and not
// read back by the layer)
__device__ __forceinline__ void store8_nt(uint16_t *p, const float v[8]) {
  typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
  u32x4_t w;
  w.x = f2bf2(v[0], v[1]);
  w.y = f2bf2(v[2], v[3]);
  w.z = f2bf2(v[4], v[5]);
  w.w = f2bf2(v[6], v[7]);
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t *>(p));
}
template <> struct Cols<float, 8> {
  static __device__ __forceinline__ void load(const float *p, float v[8]) { Elem<float>::load8(p, v); }
  static __device__ __forceinline__ void store(float *p, const float v[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ void load_f8(const float *p, float v[8]) { Elem<float>::load8(p, v); }

// ------------------------------------------------------------ expand of one row
// v[c] += sum over the row's active slots k (in slot order) and rank rows j
// (ascending) of U[u_off[p] + j] * B_a[j][col + c].  Wave-uniform control flow:
// every lane handles the same row; lanes own consecutive columns.  `col` must
// be a valid column (callers clamp it and mask their store), so the B loads
// are unconditional and eight of them are in flight at a time.
// 8 consecutive elements held raw until used, so a batch of loads is in
// flight before the first conversion waits.
template <typename E> struct Raw8;
template <> struct Raw8<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void to8(float o[8]) const { Elem<uint16_t>::load8(reinterpret_cast<const uint16_t *>(&v), o); }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void to8(float o[8]) const {
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
};

// One row, 8 columns per lane.  Control data is gathered lane-parallel and
// broadcast: the row's slot descriptors ({pair, rank, u_off, page_start},
// lane k = slot k; the caller loads them, so their round trip can overlap
// its own loads), then the page ids and U values of up to 64 rank rows (lane
// j = row j), then the B rows stream in batches of 8, the next batch in
// flight while the current one is added.  Rank rows are added in ascending
// order, slot by slot.
template <typename E>
__device__ __forceinline__ int4 expand_row_desc(int t, const ExpandArgs &e) {
  int4 sd = make_int4(-1, 0, 0, 0);
  if (lane_id() < e.K) sd = e.slot_desc[t * e.K + lane_id()];
  return sd;
}

template <typename E>
__device__ __forceinline__ void expand_row8(float (&v)[8], int4 sd, int col, const ExpandArgs &e) {
  constexpr int NB = 8;                  // B rows per batch; two batches in flight
  const E *B = static_cast<const E *>(e.b_pages);
  const int lane = lane_id();
  for (int k = 0; k < e.K; ++k) {
    // the slot's descriptor, the same in every lane: scalar registers, so
    // that the loops below branch uniformly
    if (__builtin_amdgcn_readfirstlane(__shfl(sd.x, k, 64)) < 0) continue;
    const int r = __builtin_amdgcn_readfirstlane(__shfl(sd.y, k, 64));
    const int uo = __builtin_amdgcn_readfirstlane(__shfl(sd.z, k, 64));
    const int ps = __builtin_amdgcn_readfirstlane(__shfl(sd.w, k, 64));
    for (int jb = 0; jb < r; jb += 64) {
      const int nrb = min(64, r - jb);
      const int jl = jb + min(lane, nrb - 1);
      const int pid = e.page_ids[ps + jl];
      const float uv = e.U[uo + jl];
      Raw8<E> ba[NB], bb[NB];
      auto loadb = [&](Raw8<E> (&dst)[NB], int q0) {
#pragma unroll
        for (int q = 0; q < NB; ++q)
          dst[q].load(B + int64_t(__shfl(pid, min(q0 + q, nrb - 1), 64)) * e.d_out + col);
      };
      auto addb = [&](const Raw8<E> (&src)[NB], int q0) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          if (q0 + q < nrb) {
            float b[8];
            src[q].to8(b);
            const float uj = __shfl(uv, q0 + q, 64);
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = fmaf(uj, b[c], v[c]);
          }
        }
      };
      // both batches' loads are issued unconditionally (rows past nrb
      // re-read row nrb - 1, a cache hit, and are not added): a load under
      // a condition leaves the compiler unable to count what is in flight,
      // and it then waits for every load, the batch just issued included
      loadb(ba, 0);
      for (int q0 = 0; q0 < nrb; q0 += 2 * NB) {
        loadb(bb, q0 + NB);
        addb(ba, q0);
        loadb(ba, q0 + 2 * NB);
        addb(bb, q0 + NB);
      }
    }
  }
}

// Same sums in the same order, with the B slice of the last page range (rank
// <= RB) kept in registers: consecutive prefill rows usually share an adapter.
template <int CPL, int RB>
struct BCache {
  int ps, r;
  float b[RB][CPL];
};

template <int CPL, int RB>
__device__ __forceinline__ void expand_row_cached(float (&v)[CPL], int t, int col,
                                                  const ExpandArgs &e, BCache<CPL, RB> &cache) {
  const uint16_t *B = static_cast<const uint16_t *>(e.b_pages);
  for (int k = 0; k < e.K; ++k) {
    const int4 sd = e.slot_desc[t * e.K + k];
    if (sd.x < 0) continue;
    const int r = sd.y;
    const float *u = e.U + sd.z;
    const int32_t *pid = e.page_ids + sd.w;
    if (r <= RB) {
      if (sd.w != cache.ps || r != cache.r) {
        // rows past r reload row r-1; they are never used
#pragma unroll
        for (int j = 0; j < RB; ++j)
          Cols<uint16_t, CPL>::load(B + int64_t(pid[min(j, r - 1)]) * e.d_out + col, cache.b[j]);
        cache.ps = sd.w;
        cache.r = r;
      }
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        if (j < r) {
          const float uj = u[j];
#pragma unroll
          for (int c = 0; c < CPL; ++c) v[c] = fmaf(uj, cache.b[j][c], v[c]);
        }
      }
    } else {
      for (int j = 0; j < r; ++j) {
        float bv[CPL];
        Cols<uint16_t, CPL>::load(B + int64_t(pid[j]) * e.d_out + col, bv);
        const float uj = u[j];
#pragma unroll
        for (int c = 0; c < CPL; ++c) v[c] = fmaf(uj, bv[c], v[c]);
      }
    }
  }
}

__device__ __forceinline__ bool expand_enabled(const ExpandArgs &e) {
  return e.U != nullptr && int64_t(e.hdr[LORA_PH_RPAIRS]) <= e.u_cap;
}

// ------------------------------------------------------------ LDS copies and waits
// LDS byte address of a __shared__ object.
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (const __attribute__((address_space(3))) char *)(p)));
}

// global_load_lds_dwordx4: each of the 64 lanes copies 16 bytes from its
// global address to LDS at lds + 16 * lane.  Issued from inline asm so that
// the compiler does not put a blanket vmcnt(0) in front of every later LDS
// read (it cannot tell which LDS stage an in-flight copy writes); the
// instruction has no register result, and the kernel waits for these copies
// itself (wait_vmcnt) before the barrier that precedes reading the stage.
// On this architecture family an LDS DMA needs one wait state after a
// scalar write of m0, which the compiler cannot insert inside the asm
// block: the s_nop provides it.
__device__ __forceinline__ void lds_dma16(const void *gptr, uint32_t lds) {
  const uint32_t lds_s = __builtin_amdgcn_readfirstlane(lds);   // wave-uniform LDS base
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(gptr), "s"(lds_s)
               : "memory", "m0");
}

// s_waitcnt with only vmcnt constrained (gfx9 encoding: vmcnt bits 3:0 and 15:14).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Workgroup barrier for LDS only.  The stage copies are LDS DMA issued from
// inline asm, so every wave first waits (wait_vmcnt) for its own copies of a
// stage and then meets the others here; no global load in flight is waited
// for (__syncthreads() waits for all of them).
__device__ __forceinline__ void lds_bar() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------ tiles
// LDS slot of 16-byte chunk c (0..7) in tile row `row`.
__device__ __forceinline__ int tswz(int row, int c) { return c ^ (row & 7) ^ ((row >> 3) & 1); }

template <int BM, int BN, int WM, int WN>
struct TileCfg {
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int ROWB = 128;                        // bytes per 64-wide K row
  static constexpr int STAGE = (BM + BN) * ROWB;          // bytes per LDS stage
  static constexpr int TM = BM / (WM * 32), TN = BN / (WN * 32);
  static constexpr int A_INS = BM / 8 / NW, B_INS = BN / 8 / NW;
  static constexpr int LPW = A_INS + B_INS;               // loads per wave per stage
  static_assert(A_INS * 8 * NW == BM && B_INS * 8 * NW == BN, "tile rows / waves");
  static_assert(LPW < 64, "vmcnt field holds at most 63");
};

__device__ __forceinline__ void tile_coords(int T, int tiles_m, int tiles_n, int &tm, int &tn) {
  constexpr int G = 4;
  const int gsize = G * tiles_n;
  const int grp = T / gsize;
  const int first = grp * G;
  const int gm = min(G, tiles_m - first);
  const int in = T - grp * gsize;
  tm = first + in % gm;
  tn = in / gm;
}

// Operands of the fused epilogue's MFMA expand that do not depend on the
// product: the slot descriptors of the tile's rows and the page ids of the
// first adapter of the wave's first block.  They are fetched while the K loop
// runs (the descriptors before its first copies, the page ids once those have
// landed); after the loop each would be a round trip of its own with the MFMA
// pipe idle.  U is not held across the loop (32 more registers would spill):
// the epilogue issues it together with the B values, one round trip for both.
template <int TM>
struct EpiPre {
  int4 sd[TM];        // slot descriptor of row frow of each 32-row block
  int pid;            // lanes 0-15: page id of rank row `lane` of (kps, kr)
  int kps, kr;        // page start and rank of block 0's first adapter (-1: none)
};

// The descriptors (none when U is absent or K > 1: those tiles take the row
// path or no LoRA term).
template <int BM, int BN, int WM, int WN>
__device__ __forceinline__ void epi_fetch_desc(const GemmArgs &g, int m0,
                                               EpiPre<TileCfg<BM, BN, WM, WN>::TM> &p) {
  constexpr int TM = TileCfg<BM, BN, WM, WN>::TM;
  const int lane = threadIdx.x & 63, wm = (threadIdx.x >> 6) / WN;
  const bool want = g.ex.U != nullptr && g.ex.K == 1;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = m0 + wm * TM * 32 + i * 32 + (lane & 31);
    p.sd[i] = want ? g.ex.slot_desc[min(row, g.M - 1)] : make_int4(-1, 0, 0, 0);
    if (row >= g.M) p.sd[i].x = -1;
  }
  p.kps = -1;
  p.kr = -1;
  p.pid = 0;
}

// The page ids of block 0's first adapter (the load the epilogue would issue
// for it).
template <int TM>
__device__ __forceinline__ void epi_fetch_pid(const GemmArgs &g, EpiPre<TM> &p) {
  const int lane = threadIdx.x & 63;
  const unsigned long long m = __ballot(p.sd[0].x >= 0) & 0xffffffffull;
  if (m && expand_enabled(g.ex)) {
    const int leader = __ffsll(m) - 1;
    p.kps = __shfl(p.sd[0].w, leader, 64);
    p.kr = __shfl(p.sd[0].y, leader, 64);
    if (lane < 16) p.pid = g.ex.page_ids[p.kps + min(lane, p.kr - 1)];
  }
}

// An MFMA pass of the expand takes one adapter's B rows for all 32 rows of a
// block, with U = 0 in the rows of other adapters: an infinity or a NaN of B
// would reach those as 0 . inf.  The passes therefore run on B fragments whose
// non-finite values are zero (drop_nonfinite, when a fragment has any), and
// expand_nonfinite adds what was left out to the rows it belongs to.  The test
// is one dot product with zeros per pair of values, NaN if either is not
// finite (16 adapters in any order, 8192 x 4096 -> 4096, bf16: 314.3 -> 317.3 us
// of the call; 325 with integer compares; nothing measurable in runs).
template <int TN>
__device__ __forceinline__ bool drop_nonfinite(bf16x8_t (&b)[TN]) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t zero = {};
  uint32_t w[TN][4];
  float t[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    __builtin_memcpy(w[j], &b[j], 16);
    t[j] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bf16x2_t v;
      __builtin_memcpy(&v, &w[j][e], 4);
      t[j] = __builtin_amdgcn_fdot2_f32_bf16(v, zero, t[j], false);
    }
    if (j > 0) t[0] += t[j];
  }
  if (__builtin_expect(__ballot(t[0] != t[0]) == 0, 1)) return false;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // the exponents' carry: bits 15 and 31 of a half that is not finite
      const uint32_t x = (((w[j][e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15;
      w[j][e] &= ~((x << 16) - x);
    }
    __builtin_memcpy(&b[j], w[j], 16);
  }
  return true;
}

// Y += the products of U with the non-finite B values alone, for the 32-row
// blocks `blocks` (bit i: rows row0 + 32 i ..) and the wave's WC columns, which
// this wave has stored: each sum is an infinity or a NaN, so that the rounding
// of Y before it is no loss.
template <int TM, int WC, bool kMask>
__device__ __forceinline__ void expand_nonfinite(const GemmArgs &g, int row0, int cbase, unsigned blocks) {
  const int lane = threadIdx.x & 63;
  const uint16_t *Bp = static_cast<const uint16_t *>(g.ex.b_pages);
  __threadfence();                             // the lanes' stores of Y before the loads here
#pragma unroll 1
  for (int rr = 0; rr < TM * 32; ++rr) {
    const int row = row0 + rr;
    if (row >= g.M) break;
    if (!((blocks >> (rr >> 5)) & 1u)) continue;
#pragma unroll 1
    for (int c = cbase + lane; c < min(cbase + WC, g.N); c += 64) {
      float sum = 0.f;
      bool any = false;
#pragma unroll 1
      for (int k = 0; k < g.ex.K; ++k) {
        const int4 sd = g.ex.slot_desc[int64_t(row) * g.ex.K + k];
        if (sd.x < 0) continue;
#pragma unroll 1
        for (int j = 0; j < sd.y; ++j) {
          const uint16_t b = Bp[int64_t(g.ex.page_ids[sd.w + j]) * g.ex.d_out + c];
          if ((b & 0x7f80u) != 0x7f80u) continue;
          sum = fmaf(g.ex.U[sd.z + j], bf2f(b), sum);
          any = true;
        }
      }
      if (!any) continue;
      uint16_t *y = static_cast<uint16_t *>(g.Y) + int64_t(row) * g.N + c;
      if constexpr (kMask) sum *= float(g.mask[int64_t(row) * g.N + c]);
      *y = f2bf(bf2f(*y) + sum);
    }
  }
}

// Fused epilogue of a tile: add the expand to the fp32 accumulators, round
// once, store Y.
//   * One slot per token (K = 1) and ranks <= 16 -- prefill: the expand of a
//     32-row block is done by MFMAs, U_block (32 x r, fp32 split exactly into
//     bf16 hi + lo, error < 2^-16 of U) times the adapter's B slice (r x 32 per
//     MFMA block), accumulated into the base product's registers.  A block
//     spanning several adapters takes one pass per adapter, with the U rows
//     of the other adapters zero.  The B fragments of the last adapter are
//     kept, so a long segment loads them once.  The slot descriptors, U and
//     the first adapter's page ids come prefetched (EpiPre); B values are
//     the one round trip left after the K loop.
//   * Blocks with higher ranks or several slots per token add the expand row
//     by row (all lanes on one row).
//   * Every block is staged in LDS and stored with 16-byte stores when it
//     needs no row-by-row expand.
// The per-block loop is unrolled, so every block's accumulators, descriptors
// and U values are addressed by compile-time indices (a rolled loop that
// rotated the blocks down into position 0 needed 11 dwords of scratch per
// block for the rotation temporaries).
// kMask (the input gradient, whose LoRA term is multiplied by the keep mask
// g.mask [M][N]): the LoRA term is accumulated apart from the base product
// and added times the mask bytes, one rounding, as the split-K epilogue does.
// An MFMA block stages its base product first, accumulates the LoRA term in
// the same registers, and moves it through a second, 8-row staging region a
// quarter at a time; the row path keeps the term in registers of its own.
// kLeaveRows: blocks for the row path are left to the caller, which gets them
// as bits (bit i: 32-row block i of the wave).  nonfinite: the blocks, so, that
// the caller has to take to expand_nonfinite.
template <int BM, int BN, int WM, int WN, bool kMask, bool kLeaveRows = false>
__device__ __forceinline__ unsigned fused_epilogue(const GemmArgs &g,
                                               f32x16_t (&acc)[TileCfg<BM, BN, WM, WN>::TM]
                                                              [TileCfg<BM, BN, WM, WN>::TN],
                                               char *lds0, char *lds1, int m0, int n0,
                                               const EpiPre<TileCfg<BM, BN, WM, WN>::TM> &pre,
                                               unsigned &nonfinite) {
  using C = TileCfg<BM, BN, WM, WN>;
  constexpr int TM = C::TM, TN = C::TN;
  constexpr int WC = TN * 32;                // columns of this wave's sub-tile
  constexpr int SC = WC + 4;                 // staged floats per row (padded, 16-byte rows)
  constexpr int CPL = WC / 64;               // columns per lane in the row-by-row path
  static_assert(CPL == 1 || CPL == 2, "fused epilogue handles 64 or 128 columns per wave");
  static_assert(WC % 8 == 0 && 64 % (WC / 8) == 0, "16-byte store layout");
  // waves 0..NW/2-1 stage in lds0, the others in lds1
  static_assert((C::NW / 2) * (kMask ? 40 : 32) * SC * 4 <= C::STAGE, "staging must fit in LDS");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int frow = lane & 31, half = lane >> 5;
  const bool lora_on = expand_enabled(g.ex);
  const bool mfma_ok = lora_on && g.ex.K == 1;
  const uint16_t *Bp = static_cast<const uint16_t *>(g.ex.b_pages);

  // slot descriptor of row frow of every block (fetched during the K loop),
  // and that row's U values (rank rows 8*half .. +7), whose loads share their
  // round trip with the first B values
  const int4 (&sdv)[TM] = pre.sd;
  float uv[TM][8];
  unsigned rowwise = lora_on && !mfma_ok ? (1u << TM) - 1 : 0u;   // blocks for the row path
  if (mfma_ok) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const bool act = sdv[i].x >= 0;
      if (__ballot(act && sdv[i].y > 16) != 0) rowwise |= 1u << i;
      // 32 consecutive pairs of one adapter of rank 8 or 16 hold their U as
      // one run of 32 r floats: the wave loads it in 16-byte pieces (lane l
      // floats 8l .. 8l+7, i.e. row l r/8 ... ) and hands each row's values
      // to its lanes by shuffles.  Otherwise each lane loads its 8 values
      // one by one (every such load touches 16 cache lines).
      const int r0 = __shfl(sdv[i].y, 0, 64), z0 = __shfl(sdv[i].z, 0, 64);
      const int w0 = __shfl(sdv[i].w, 0, 64);
      const bool in_run = act && sdv[i].y == r0 && sdv[i].w == w0 && sdv[i].z == z0 + r0 * frow;
      const bool run = __ballot(!in_run) == 0 && (r0 == 8 || r0 == 16) &&
                       (reinterpret_cast<uintptr_t>(g.ex.U + z0) & 15) == 0;
      if (run) {
        const float4 *src = reinterpret_cast<const float4 *>(g.ex.U + z0) + 2 * min(lane, 4 * r0 - 1);
        const float4 lo4 = src[0], hi4 = src[1];
        const float v8[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
        // row frow's rank rows 8*half .. +7 sit in lane frow * r/8 + half
        const int from = min(frow * (r0 / 8) + half, 63);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __shfl(v8[e], from, 64);
          uv[i][e] = half * 8 < r0 ? x : 0.f;
        }
      } else {
        const int r = act ? min(sdv[i].y, 16) : 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ja = half * 8 + e;
          uv[i][e] = act ? g.ex.U[sdv[i].z + min(ja, r - 1)] : 0.f;
          if (ja >= r) uv[i][e] = 0.f;
        }
      }
    }
  }

  float *stage = reinterpret_cast<float *>(wave < C::NW / 2 ? lds0 : lds1) +
                 (wave % (C::NW / 2)) * 32 * SC;
  // kMask: 8 rows of the LoRA term, past every wave's staging region
  float *lstage = reinterpret_cast<float *>(wave < C::NW / 2 ? lds0 : lds1) +
                  (C::NW / 2) * 32 * SC + (wave % (C::NW / 2)) * 8 * SC;
  uint16_t *Y = static_cast<uint16_t *>(g.Y);
  const int cbase = n0 + wn * WC;
  // row-by-row path: lane owns CPL consecutive columns
  const int col_raw = cbase + lane * CPL;
  const bool col_ok = col_raw < g.N;
  const int col = col_ok ? col_raw : g.N - CPL;     // loads stay in bounds
  // 16-byte path: lane owns 8 columns of one of 64 / (WC / 8) rows per step
  constexpr int LPR = WC / 8, RPS = 64 / LPR;
  static_assert(RPS <= 8, "the kMask quarter holds 8 rows");
  const int vr = lane / LPR, vc = (lane % LPR) * 8;
  const bool c8 = cbase + vc + 8 <= g.N;
  BCache<CPL, 16> cache;
  cache.ps = -1;
  cache.r = -1;
  int bkey_ps = -1, bkey_r = -1;             // adapter slice held in bfr
  bool b_dropped = false;                    // .. less its non-finite values
  bf16x8_t bfr[TN] = {};
  nonfinite = 0;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (kLeaveRows && ((rowwise >> i) & 1u)) continue;
    bool lterm = false;                      // kMask: acc[i] holds the LoRA term
    if (mfma_ok && !((rowwise >> i) & 1u)) {
      // one MFMA pass per adapter present in the block (lanes 0-31 = rows)
      const int4 sd = sdv[i];
      unsigned long long pending = __ballot(sd.x >= 0) & 0xffffffffull;
      if constexpr (kMask) {
        lterm = pending != 0;
        if (lterm) {
          // the staging region is this wave's own (see below)
#pragma unroll
          for (int j = 0; j < TN; ++j) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const int r = (v >> 2) * 8 + half * 4 + (v & 3);
              stage[r * SC + j * 32 + frow] = acc[i][j][v];
            }
            acc[i][j] = f32x16_t{};
          }
        }
      }
      // A operand: U of row frow, rank rows 8*half .. +7, as bf16 hi + lo
      uint32_t hw[4], lw[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint32_t h2 = f2bf2(uv[i][e], uv[i][e + 1]);
        hw[e >> 1] = h2;
        lw[e >> 1] = f2bf2(uv[i][e] - bf_lo(h2), uv[i][e + 1] - bf_hi(h2));
      }
      while (pending) {
        const int leader = __ffsll(pending) - 1;
        const int kps = __shfl(sd.w, leader, 64), kr = __shfl(sd.y, leader, 64);
        const bool mine = sd.x >= 0 && sd.w == kps && sd.y == kr;
        pending &= ~__ballot(mine);
        if (kps != bkey_ps || kr != bkey_r) {
          // B operand: lane (column frow of block j, rank rows 8*half .. +7)
          int pidl = 0;
          if (kps == pre.kps && kr == pre.kr) pidl = pre.pid;
          else if (lane < 16) pidl = g.ex.page_ids[kps + min(lane, kr - 1)];
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const int cj = min(n0 + wn * TN * 32 + j * 32 + frow, g.N - 1);
            uint32_t w4[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int ja = half * 8 + e, jb = ja + 1;
              const int pa = __shfl(pidl, min(ja, 15), 64), pb = __shfl(pidl, min(jb, 15), 64);
              uint32_t lo = Bp[int64_t(pa) * g.ex.d_out + cj];
              uint32_t hi = Bp[int64_t(pb) * g.ex.d_out + cj];
              if (ja >= kr) lo = 0;
              if (jb >= kr) hi = 0;
              w4[e >> 1] = lo | (hi << 16);
            }
            const uint4 packed = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            __builtin_memcpy(&bfr[j], &packed, 16);
          }
          b_dropped = drop_nonfinite<TN>(bfr);
          bkey_ps = kps;
          bkey_r = kr;
        }
        if (b_dropped) nonfinite |= 1u << i;
        // zero unless the row is on this adapter
        bf16x8_t ahi, alo;
        const uint4 ph = mine ? make_uint4(hw[0], hw[1], hw[2], hw[3]) : make_uint4(0u, 0u, 0u, 0u);
        const uint4 pl = mine ? make_uint4(lw[0], lw[1], lw[2], lw[3]) : make_uint4(0u, 0u, 0u, 0u);
        __builtin_memcpy(&ahi, &ph, 16);
        __builtin_memcpy(&alo, &pl, 16);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ahi, bfr[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(alo, bfr[j], acc[i][j], 0, 0, 0);
        }
      }
    }
    // the staging region is this wave's own, and the K loop ended with a
    // workgroup barrier: no barrier here (LDS accesses of one wave stay in
    // order)
    if (!(kMask && lterm)) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int r = (v >> 2) * 8 + half * 4 + (v & 3);
          stage[r * SC + j * 32 + frow] = acc[i][j][v];
        }
    }
    const int rbase = m0 + wm * TM * 32 + i * 32;
    if (kMask && lterm) {
      // quarter qr: MFMA registers v = 4qr .. 4qr+3 hold rows 8qr .. 8qr+7
#pragma unroll
      for (int qr = 0; qr < 4; ++qr) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int v = 4 * qr; v < 4 * qr + 4; ++v)
            lstage[(half * 4 + (v & 3)) * SC + j * 32 + frow] = acc[i][j][v];
#pragma unroll
        for (int q = 0; q < 8 / RPS; ++q) {
          const int lr = q * RPS + vr;
          const int rr = qr * 8 + lr;
          const int row = rbase + rr;
          if (row < g.M && c8) {
            const float *sb = stage + rr * SC + vc, *sl = lstage + lr * SC + vc;
            const float4 b0 = *reinterpret_cast<const float4 *>(sb);
            const float4 b1 = *reinterpret_cast<const float4 *>(sb + 4);
            const float4 l0 = *reinterpret_cast<const float4 *>(sl);
            const float4 l1 = *reinterpret_cast<const float4 *>(sl + 4);
            const float b8[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
            const float l8[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
            const uint2 mw = *reinterpret_cast<const uint2 *>(g.mask + int64_t(row) * g.N + cbase + vc);
            float v8[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint32_t word = c < 4 ? mw.x : mw.y;
              v8[c] = b8[c] + float((word >> (8 * (c & 3))) & 0xffu) * l8[c];
            }
            store8_nt(Y + int64_t(row) * g.N + cbase + vc, v8);
          }
        }
      }
    } else if (kLeaveRows || !((rowwise >> i) & 1u)) {
#pragma unroll
      for (int rr0 = 0; rr0 < 32; rr0 += RPS) {
        const int rr = rr0 + vr;
        const int row = rbase + rr;
        if (row < g.M && c8) {
          const float4 lo = *reinterpret_cast<const float4 *>(stage + rr * SC + vc);
          const float4 hi = *reinterpret_cast<const float4 *>(stage + rr * SC + vc + 4);
          const float v8[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          store8_nt(Y + int64_t(row) * g.N + cbase + vc, v8);
        }
      }
    } else {
      for (int rr = 0; rr < 32; ++rr) {
        const int row = rbase + rr;
        if (row >= g.M) break;
        float v[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) v[c] = stage[rr * SC + lane * CPL + c];
        if constexpr (kMask) {
          float l[CPL];
#pragma unroll
          for (int c = 0; c < CPL; ++c) l[c] = 0.f;
          expand_row_cached<CPL, 16>(l, row, col, g.ex, cache);
          const uint8_t *mr = g.mask + int64_t(row) * g.N + col;
#pragma unroll
          for (int c = 0; c < CPL; ++c) v[c] += float(mr[c]) * l[c];
        } else {
          expand_row_cached<CPL, 16>(v, row, col, g.ex, cache);
        }
        if (col_ok) Cols<uint16_t, CPL>::store(Y + int64_t(row) * g.N + col, v);
      }
    }
  }
  return kLeaveRows ? rowwise : 0u;
}

// Fragment read slot i of a K step (A blocks 0 .. TM-1 are fragments
// 0 .. TM-1, B blocks TM ..): block (i, j) takes MFMA i * TN + j, so the
// next step needs A 0 and B 0 first, then B 1 .. TN-1, then A 1, A 2, ...;
// read in that order, one after each of the first TM + TN MFMAs of a step,
// every fragment has at least TM * TN - 2 MFMAs between its read and its
// first use.
template <int TM, int TN>
__device__ __forceinline__ constexpr int frag_order(int i) {
  return i == 0 ? 0 : i <= TN ? TM + i - 1 : i - TN;
}

// Wait until at most n (0 <= n <= NS - 2) K tiles' copies are still in flight.
template <int LPW, int NS>
__device__ __forceinline__ void wait_tiles(int n) {
  if constexpr (NS >= 4) {
    if (n >= 2) { wait_vmcnt<2 * LPW>(); return; }
  }
  if constexpr (NS >= 3) {
    if (n >= 1) { wait_vmcnt<LPW>(); return; }
  }
  wait_vmcnt<0>();
}

}  // namespace
}  // namespace lora
