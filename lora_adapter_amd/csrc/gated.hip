// The gated feed-forward block over two adapted projections, and its backward.
//
//   g = X.Wg + adapters,  u = X.Wu + adapters,  H = act(g) . u
//   dg = dH . u . act'(g),  du = dH . act(g)
//   dX = dg.Wg^T + du.Wu^T + mask . (G_g.A_g + G_u.A_u)
//
// The two projections share X, the routing and the page table.  A prefill
// computes a 256 x 128 tile of both at once: the B operand of a 256 x 256 tile
// holds 128 rows of each weight, 32 and 32 for each wave, so that a lane ends
// up with g and u of the same element and X is read once.  The adapters' terms
// join the accumulators as MFMA passes (gate and up in one pass), then
// activation, product and the one rounding happen on the way out.  Smaller
// batches take the split products of the single projections and an epilogue
// that finishes both.
#include "decode_tile.h"
#include "plan_build.h"
#include "shrink_units.h"
#include "tile_loop.h"

namespace lora {
namespace {

// ------------------------------------------------------------ activations
// kFast (bf16 layers): exponential and reciprocal by the hardware's
// instructions, relative error about 1e-7 (1 + |x|), far under a bf16 step.
template <bool kFast>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (kFast) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504088896340736f));
  return 1.f / (1.f + expf(-x));
}

// act(x), and act'(x) in `slope`.
template <int kAct, bool kFast>
__device__ __forceinline__ float activate(float x, float &slope) {
  if constexpr (kAct == LORA_ACT_SILU) {
    const float p = sigmoid<kFast>(x);
    slope = fmaf(x * p, 1.f - p, p);
    return x * p;
  } else if constexpr (kAct == LORA_ACT_GELU) {
    const float p = 0.5f * erfcf(x * -0.70710678118654752440f);
    slope = fmaf(x * 0.39894228040143267794f, expf(-0.5f * x * x), p);
    return x * p;
  } else {
    // (1 + tanh z) / 2 = sigmoid(2 z); past |x| = 100 both limits are reached,
    // and x^2 stays there so that the slope has no 0 . inf
    constexpr float k = 0.79788456080286535588f, c = 0.044715f;
    const float x2 = fminf(x * x, 1e4f), p = sigmoid<kFast>(2.f * k * x * fmaf(c, x2, 1.f));
    slope = fmaf(x * p, (1.f - p) * (2.f * k) * fmaf(3.f * c, x2, 1.f), p);
    return x * p;
  }
}

// ------------------------------------------------------------ adapters' terms
// Both projections' adapter terms of a 16-row block and the wave's 64
// accumulator columns as MFMA passes: for every slot, adapter and 16 rank rows,
// U times the pages' rows.  U (fp32; rows of other adapters zero) is bf16 hi
// in the first 16 of K and lo in the second (error < 2^-16 of U), against the
// page rows twice.  kPair (the forward): columns 0 .. 31 are the gate's c0 ..,
// 32 .. 63 the up projection's, the same c0 ...  Otherwise (dX) both
// projections' terms go into all of c0 .. c0 + 63.
// The page rows come in 16-byte loads through the wave's LDS, read transposed
// from there; the last adapter's fragments are kept, so that a run of blocks
// loads them once.
struct Terms {
  ExpandArgs ex;
  const float *U_up;
  const void *b_up;
};

constexpr int kTermLds = 4096;             // bytes of LDS per wave

template <bool kPair>
struct TermCache {
  static constexpr int NF = kPair ? 4 : 8;
  int key = -1;                            // first page id's place, or -1
  bool dropped = false;                    // its values that are not finite were left out
  bf16x8_t b[NF];                          // kPair: gate 0, 1, up 0, 1; else gate 0 .. 3, up 0 .. 3
};

// 8 bf16 values with those that are not finite zero; whether there were any.
__device__ __forceinline__ bool drop8(uint4 &w) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // the exponents' carry: bits 15 and 31 of a half that is not finite
    const uint32_t x = (((v[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15;
    any |= x;
    v[e] &= ~((x << 16) - x);
  }
  w = make_uint4(v[0], v[1], v[2], v[3]);
  return any != 0;
}

template <bool kPair>
__device__ __forceinline__ void load_terms(const Terms &e, char *lds, int at, int nr, int c0, int N,
                                           TermCache<kPair> &t) {
  constexpr int CPL = kPair ? 4 : 8;       // lanes along a page's columns
  constexpr int NL = kPair ? 1 : 2;        // loads of a projection
  constexpr int PITCH = CPL * 16, SIZE = 16 * PITCH;
  const int lane = threadIdx.x & 63, col = min(c0 + (lane % CPL) * 8, N - 8);
  uint4 v[2][NL];
#pragma unroll
  for (int h = 0; h < NL; ++h) {
    const int j = lane / CPL + h * (64 / CPL);
    const int64_t row = int64_t(e.ex.page_ids[at + min(j, nr - 1)]) * e.ex.d_out + col;
    v[0][h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(e.ex.b_pages) + row);
    v[1][h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(e.b_up) + row);
  }
  bool bad = false;
#pragma unroll
  for (int h = 0; h < NL; ++h) {
    const int j = lane / CPL + h * (64 / CPL);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (j >= nr) v[p][h] = make_uint4(0u, 0u, 0u, 0u);
      bad |= drop8(v[p][h]);
      *reinterpret_cast<uint4 *>(lds + p * SIZE + j * PITCH + (lane % CPL) * 16) = v[p][h];
    }
  }
  t.dropped = __ballot(bad) != 0;
  t.key = at;
  // B operand: lane (column lane % 16, rank rows 8 (lane / 16 % 2) .. + 7)
  constexpr int NB = kPair ? 2 : 4;        // blocks of a projection
  typedef __attribute__((address_space(3))) v4i16_t lds_v4;
  const int L = lane & 15, k = 8 * ((lane >> 4) & 1) + (L >> 2);
#pragma unroll
  for (int f = 0; f < 2 * NB; ++f) {
    const char *p = lds + (f / NB) * SIZE + k * PITCH + (f % NB) * 32 + (L & 3) * 8;
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p));
    const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p + 4 * PITCH));
    __builtin_memcpy(&t.b[f], &lo, 8);
    __builtin_memcpy(reinterpret_cast<char *>(&t.b[f]) + 8, &hi, 8);
  }
}

// Returns whether a page value that is not finite was left out of the block:
// it would reach other adapters' rows as 0 . inf.  terms_nonfinite adds those.
template <bool kPair>
__device__ __forceinline__ bool add_terms(const Terms &e, char *lds, int row0, int M, int c0, int N,
                                          f32x4_t (&acc)[4], TermCache<kPair> &t) {
  const int lane = threadIdx.x & 63, row = row0 + (lane & 15);
  bool dropped = false;
  for (int k = 0; k < e.ex.K; ++k) {
    int4 sd = make_int4(-1, 0, 0, 0);
    if (row < M) sd = e.ex.slot_desc[int64_t(row) * e.ex.K + k];
    unsigned long long pending = __ballot(sd.x >= 0) & 0xffffull;
    while (pending) {
      const int leader = __ffsll(pending) - 1;
      const int kps = __builtin_amdgcn_readfirstlane(__shfl(sd.w, leader, 64));
      const int kr = __builtin_amdgcn_readfirstlane(__shfl(sd.y, leader, 64));
      const bool mine = sd.x >= 0 && sd.w == kps && sd.y == kr;
      pending &= ~__ballot(mine);
      for (int jb = 0; jb < kr; jb += 16) {
        const int nr = min(16, kr - jb), j0 = 8 * ((lane >> 4) & 1);
        // A operand: lane (row lane % 16, rank rows j0 .. j0 + 7), hi or lo
        bf16x8_t u[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float *U = (p ? e.U_up : e.ex.U) + int64_t(sd.z) + jb;
          uint32_t w[4];
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = mine && j0 + q < nr ? U[j0 + q] : 0.f;
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const uint32_t h = f2bf2(v[q], v[q + 1]);
            w[q >> 1] = lane < 32 ? h : f2bf2(v[q] - bf_lo(h), v[q + 1] - bf_hi(h));
          }
          __builtin_memcpy(&u[p], w, 16);
        }
        if (t.key != kps + jb) load_terms<kPair>(e, lds, kps + jb, nr, c0, N, t);
        dropped |= t.dropped;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if constexpr (kPair) {
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[b >> 1], t.b[b], acc[b], 0, 0, 0);
          } else {
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[0], t.b[b], acc[b], 0, 0, 0);
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[1], t.b[4 + b], acc[b], 0, 0, 0);
          }
        }
      }
    }
  }
  return dropped;
}

// The common case (one slot for each token, ranks of at most 16): the tile's
// slot descriptors are fetched under the K loop, and U of all its rows goes to
// LDS at once, as the bf16 fragments of add_terms; block by block each of
// those is a round trip with the matrix cores idle (8192 x 4096 -> 11008, three
// outputs: 1403 -> 1240 us).
template <typename C>
struct TileTerms {
  int4 sd[C::BM];                          // .x < 0: no adapter
  uint16_t u[2][2][C::BM][16];             // [projection][hi, lo][row][rank row]
  int wide;                                // a rank over 16
};

// Slot descriptor of tile row threadIdx.x, or none.
template <typename C>
__device__ __forceinline__ int4 tile_desc(const ExpandArgs &ex, int m0, int M) {
  const int row = m0 + int(threadIdx.x);
  if (int(threadIdx.x) >= C::BM || row >= M || ex.K != 1 || ex.U == nullptr) return make_int4(-1, 0, 0, 0);
  return ex.slot_desc[row];
}

// After the K loop: fills t; false where the tile takes add_terms instead.
// t lies in the stages, which the loop has left.
template <typename C>
__device__ __forceinline__ bool tile_terms(const Terms &e, TileTerms<C> &t, int4 sd) {
  const int tid = threadIdx.x;
  if (tid == 0) t.wide = 0;
  lds_bar();
  if (tid < C::BM) {
    t.sd[tid] = sd;
    if (sd.x >= 0 && sd.y > 16) t.wide = 1;
  }
  lds_bar();
  if (__builtin_amdgcn_readfirstlane(t.wide)) return false;
  // a thread takes 8 rank rows of one token
  for (int at = tid; at < 2 * C::BM; at += C::NT) {
    const int r = at >> 1, j0 = (at & 1) * 8;
    const int4 d = t.sd[r];
    float v[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float *U = (p ? e.U_up : e.ex.U) + int64_t(d.z) + j0;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[p][q] = d.x >= 0 && j0 + q < d.y ? U[q] : 0.f;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        h[q >> 1] = f2bf2(v[p][q], v[p][q + 1]);
        l[q >> 1] = f2bf2(v[p][q] - bf_lo(h[q >> 1]), v[p][q + 1] - bf_hi(h[q >> 1]));
      }
      *reinterpret_cast<uint4 *>(&t.u[p][0][r][j0]) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4 *>(&t.u[p][1][r][j0]) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
  lds_bar();
  return true;
}

// add_terms from them; tr: the block's first row in the tile.
template <bool kPair, typename C>
__device__ __forceinline__ bool add_tile_terms(const Terms &e, const TileTerms<C> &tt, char *lds, int tr, int c0,
                                               int N, f32x4_t (&acc)[4], TermCache<kPair> &t) {
  const int lane = threadIdx.x & 63;
  const int4 sd = tt.sd[tr + (lane & 15)];
  bf16x8_t u[2];
#pragma unroll
  for (int p = 0; p < 2; ++p)
    u[p] = *reinterpret_cast<const bf16x8_t *>(&tt.u[p][lane >> 5][tr + (lane & 15)][8 * ((lane >> 4) & 1)]);
  bool dropped = false;
  unsigned long long pending = __ballot(sd.x >= 0) & 0xffffull;
  while (pending) {
    const int leader = __ffsll(pending) - 1;
    const int kps = __builtin_amdgcn_readfirstlane(__shfl(sd.w, leader, 64));
    const int kr = __builtin_amdgcn_readfirstlane(__shfl(sd.y, leader, 64));
    const bool mine = sd.x >= 0 && sd.w == kps && sd.y == kr;
    pending &= ~__ballot(mine);
    bf16x8_t um[2] = {u[0], u[1]};
    if (!mine) um[0] = um[1] = bf16x8_t{};
    if (t.key != kps) load_terms<kPair>(e, lds, kps, kr, c0, N, t);
    dropped |= t.dropped;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if constexpr (kPair) {
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(um[b >> 1], t.b[b], acc[b], 0, 0, 0);
      } else {
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(um[0], t.b[b], acc[b], 0, 0, 0);
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(um[1], t.b[4 + b], acc[b], 0, 0, 0);
      }
    }
  }
  return dropped;
}

// What add_terms left out: the products of U with the page values that are not
// finite, of token `row` at column col, for projection p.  Rare.
__device__ __forceinline__ float terms_nonfinite(const Terms &e, int row, int col, int p) {
  const float *U = p ? e.U_up : e.ex.U;
  const uint16_t *B = static_cast<const uint16_t *>(p ? e.b_up : e.ex.b_pages);
  float sum = 0.f;
#pragma unroll 1
  for (int k = 0; k < e.ex.K; ++k) {
    const int4 sd = e.ex.slot_desc[int64_t(row) * e.ex.K + k];
    if (sd.x < 0) continue;
#pragma unroll 1
    for (int j = 0; j < sd.y; ++j) {
      const uint16_t b = B[int64_t(e.ex.page_ids[sd.w + j]) * e.ex.d_out + col];
      if ((b & 0x7f80u) == 0x7f80u) sum = fmaf(U[int64_t(sd.z) + j], bf2f(b), sum);
    }
  }
  return sum;
}

// ------------------------------------------------------------ forward, tiles
// A rows of X by 32 rows of the gate's and 32 of the up projection's weight in
// turn.
template <typename C>
struct GatedSrc {
  static_assert(C::TN == 4, "32 columns of each projection per wave");
  const uint16_t *a, *b[2];
  uint32_t ao[C::A_INS], bo[C::B_INS];
  int wave, wm, wn;
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    if (i < C::A_INS) {
      lds_dma16_s(a + kt * 64, ao[i], lds + (wave * C::A_INS + i) * 1024);
    } else {
      const int ib = wave * C::B_INS + i - C::A_INS;     // 8 rows of the B tile, all of one weight
      lds_dma16_s(((ib >> 2) & 1 ? b[1] : b[0]) + kt * 64, bo[i - C::A_INS], lds + C::BM * C::ROWB + ib * 1024);
    }
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    return frag_rows(base, s, q < C::TM ? (wm * C::TM + q) * 16 : C::BM + (wn * C::TN + q - C::TM) * 16);
  }
};

template <typename C, int kAct>
__global__ __launch_bounds__(C::NT, 1) void gated_tile_kernel(GatedArgs g) {
  constexpr int SC = 64 + 4;                            // floats of a staged row: 32 of g, 32 of u
  constexpr int NO = C::BN / 2;                         // output columns of the tile
  constexpr int WLDS = 16 * SC * 4 + kTermLds;          // bytes of a wave's epilogue
  constexpr int TT = C::NW * WLDS;                      // the tile's terms lie behind those
  __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
  static_assert(TT % 16 == 0 && TT + sizeof(TileTerms<C>) <= 2 * C::STAGE, "staging must fit in LDS");
  int tm, tn;
  if (!tile_of_workgroup(blockIdx.x, (g.M + C::BM - 1) / C::BM, (g.N + NO - 1) / NO, tm, tn)) return;
  const int m0 = tm * C::BM, n0 = tn * NO;
  const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / C::WN, wn = wave % C::WN;

  GatedSrc<C> src;
  src.wave = wave; src.wm = wm; src.wn = wn;
  src.a = static_cast<const uint16_t *>(g.X) + int64_t(m0) * g.Kd;
#pragma unroll
  for (int p = 0; p < 2; ++p) src.b[p] = static_cast<const uint16_t *>(g.W[p]) + int64_t(n0) * g.Kd;
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
    src.ao[i] = (uint32_t(min(row, g.M - 1 - m0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8) * 2;
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = (wave * C::B_INS + i) * 8 + (lane >> 3);
    const int of = (row >> 6) * 32 + (row & 31);        // of its weight
    src.bo[i] = (uint32_t(min(of, g.N - 1 - n0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8) * 2;
  }
  const int4 sd = tile_desc<C>(g.ex, m0, g.M);
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, g.Kd / 64, acc);

  const Terms e{g.ex, g.U_up, g.b_up};
  const bool lora_on = expand_enabled(g.ex);
  TileTerms<C> &tt = *reinterpret_cast<TileTerms<C> *>(smem + TT);
  const bool common = lora_on && g.ex.K == 1 && tile_terms<C>(e, tt, sd);
  const int c0 = n0 + wn * 32;                          // the wave's output columns
  if (c0 >= g.N) return;
  float *stage = reinterpret_cast<float *>(smem + wave * WLDS);
  char *tlds = smem + wave * WLDS + 16 * SC * 4;
  TermCache<true> cache;
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int r0 = m0 + (wm * C::TM + i) * 16;
    bool dropped = false;
    if (common) dropped = add_tile_terms<true, C>(e, tt, tlds, (wm * C::TM + i) * 16, c0, g.N, acc[i], cache);
    else if (lora_on) dropped = add_terms<true>(e, tlds, r0, g.M, c0, g.N, acc[i], cache);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) stage[acc_row(0, v) * SC + acc_col(j)] = acc[i][j][v];
    if (dropped) {
#pragma unroll 1
      for (int rr = 0; rr < 16 && r0 + rr < g.M; ++rr)
        stage[rr * SC + lane] += terms_nonfinite(e, r0 + rr, c0 + (lane & 31), lane >> 5);
    }
    // a lane takes 8 columns of one of the rows
    const int rr = lane >> 2, row = r0 + rr, cc = (lane & 3) * 8;
    if (row >= g.M) continue;
    float gv[8], uv[8], h[8];
    Elem<float>::load8(stage + rr * SC + cc, gv);
    Elem<float>::load8(stage + rr * SC + 32 + cc, uv);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float slope;
      h[x] = activate<kAct, true>(gv[x], slope) * uv[x];
    }
    const int64_t at = int64_t(row) * g.N + c0 + cc;
    store8_nt(static_cast<uint16_t *>(g.H) + at, h);
    if (g.pre_gate) {
      store8_nt(static_cast<uint16_t *>(g.pre_gate) + at, gv);
      store8_nt(static_cast<uint16_t *>(g.pre_up) + at, uv);
    }
  }
}

// ------------------------------------------------------------ split forms
// Pieces of an output element: the K splits, or the stream-K workgroups that
// covered its tile.
__device__ __forceinline__ int pieces_of(int splits, int sk_g, int sk_kt, int bm, int bn, int M, int N, int row,
                                         int col) {
  if (sk_g <= 0) return splits;
  const int tiles_n = (N + bn - 1) / bn;
  const int t = (row / bm) * tiles_n + col / bn;
  const int64_t U = int64_t((M + bm - 1) / bm) * tiles_n * sk_kt;
  const int64_t x0 = int64_t(t) * sk_kt, x1 = x0 + sk_kt - 1;
  return int(((x1 + 1) * sk_g - 1) / U - ((x0 + 1) * sk_g - 1) / U) + 1;
}

// v += pieces of 8 columns of both products, 8 loads in flight.
__device__ __forceinline__ void add_pieces(const float *part, int np, int M, int N, int row, int col, float (&v)[8]) {
  for (int z0 = 0; z0 < np; z0 += 8) {
    Raw8<float> pr[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) pr[z].load(part + (int64_t(min(z0 + z, np - 1)) * M + row) * N + col);
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      if (z0 + z < np) {
        float o[8];
        pr[z].to8(o);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += o[c];
      }
    }
  }
}

// Decode: workgroup 0 builds the plan, then come the decode GEMM tiles of the
// gate's weight and of the up projection's, then the per-slot shrinks (four
// parts a slot) of both.  No part reads what another writes.
template <int MB, bool kMask, bool kLds>
__global__ __launch_bounds__(256) void gated_decode_plan_kernel(GemmArgs g0, GemmArgs g1, SlotShrinkArgs s0,
                                                                 SlotShrinkArgs s1, PlanArgs pa, int gx, int gy,
                                                                 int n_gemm) {
  __shared__ __attribute__((aligned(16))) uint16_t xs[MB * 32 * kDecodeKC];
  int b = int(blockIdx.x);
  if (b == 0) {
    plan_build<kLds>(pa, reinterpret_cast<int *>(xs));
    return;
  }
  b -= 1;
  if (b < 2 * n_gemm) {
    const int t = b < n_gemm ? b : b - n_gemm;
    decode_tile<MB>(b < n_gemm ? g0 : g1, t % gx, (t / gx) % gy, t / (gx * gy), xs);
    return;
  }
  b -= 2 * n_gemm;
  const int parts = kSlotParts * s0.n_slots, q = b < parts ? b : b - parts;
  slot_shrink_part<kMask>(b < parts ? s0 : s1, q / kSlotParts, q % kSlotParts);
}

template <int MB>
__global__ __launch_bounds__(256) void gated_decode_kernel(GemmArgs g0, GemmArgs g1) {
  __shared__ __attribute__((aligned(16))) uint16_t xs[MB * 32 * kDecodeKC];
  const int z = blockIdx.z >> 1;
  decode_tile<MB>(blockIdx.z & 1 ? g1 : g0, blockIdx.x, blockIdx.y, z, xs);
}

// Decode epilogue: a workgroup per row and 512 columns, its waves the two
// projections by halves of the pieces and of each slot's rank rows, joined
// through LDS.  A row's rank rows come one batch after another, so that the
// launch lasts as long as its longest chain: one wave for all four took 39 us
// at 48 tokens of two adapters of ranks 8 .. 64 (4096 -> 11008).
template <int kAct>
__global__ __launch_bounds__(256) void gated_decode_epilogue_kernel(GatedArgs g) {
  __shared__ __attribute__((aligned(16))) float part[4][512];
  const int lane = threadIdx.x & 63, wave = wave_id(), p = wave & 1, h = wave >> 1;
  const int row = blockIdx.y;
  const int col_raw = (blockIdx.x * 64 + lane) * 8, col = min(col_raw, g.N - 8);   // loads stay in bounds
  const bool lora_on = expand_enabled(g.ex);
  const int4 *desc = g.sdesc ? g.sdesc : g.ex.slot_desc;
  int4 sd = make_int4(-1, 0, 0, 0);
  if (lora_on && lane < g.ex.K) sd = desc[int64_t(row) * g.ex.K + lane];
  float v[8] = {};
  {
    // pieces h, h + 2, ..: up to 8 loads in flight
    const int np = (g.splits - h + 1) / 2;
    const float *src = g.part[p] + (int64_t(h) * g.M + row) * g.N + col;
    for (int z0 = 0; z0 < np; z0 += 8) {
      Raw8<float> pr[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) pr[z].load(src + 2 * int64_t(min(z0 + z, np - 1)) * g.M * g.N);
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        if (z0 + z < np) {
          float o[8];
          pr[z].to8(o);
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] += o[c];
        }
      }
    }
  }
  if (lora_on) {
    ExpandArgs e = g.ex;
    if (p) {
      e.U = g.U_up;
      e.b_pages = g.b_up;
    }
    int4 mine = sd;
    const int first = (sd.y + 1) / 2;
    if (h == 0) {
      mine.y = first;
    } else {
      mine.y = sd.y - first;
      mine.z += first;
      mine.w += first;
      if (mine.y == 0) mine.x = -1;
    }
    expand_row8<uint16_t>(v, mine, col, e);
  }
  Cols<float, 8>::store(&part[wave][lane * 8], v);
  __syncthreads();
  const int c = int(threadIdx.x) * 2, at_col = int(blockIdx.x) * 512 + c;
  if (at_col < g.N) {
    float gv[2], uv[2], o[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float slope;
      gv[x] = part[0][c + x] + part[2][c + x];
      uv[x] = part[1][c + x] + part[3][c + x];
      o[x] = activate<kAct, true>(gv[x], slope) * uv[x];
    }
    const int64_t at = int64_t(row) * g.N + at_col;
    Cols<uint16_t, 2>::store(static_cast<uint16_t *>(g.H) + at, o);
    if (g.pre_gate) {
      Cols<uint16_t, 2>::store(static_cast<uint16_t *>(g.pre_gate) + at, gv);
      Cols<uint16_t, 2>::store(static_cast<uint16_t *>(g.pre_up) + at, uv);
    }
  }
  if (g.sdesc == nullptr || blockIdx.x != 0) return;
  // the row's per-slot U to the places the plan gave its active slots
  int32_t *hdr = const_cast<int32_t *>(g.ex.hdr);
  if (!lora_on) {
    if (row == 0 && threadIdx.x == 0) atomicOr(hdr + LORA_PH_ERR, LORA_DEVERR_CAPACITY);
    return;
  }
  if (h) return;
  for (int k = 0; k < g.ex.K; ++k) {
    const int64_t i = int64_t(row) * g.ex.K + k;
    const int4 d = g.ex.slot_desc[i];
    if (d.x < 0) continue;
    const float *src = (p ? g.U_up : g.ex.U) + i * g.slot_stride;
    for (int j = lane; j < d.y; j += 64) g.u_out[p][d.z + j] = src[j];
  }
}

// One wave per row and 512 columns.
template <typename E, int NW, int kAct>
__global__ __launch_bounds__(NW * 64) void gated_epilogue_kernel(GatedArgs g) {
  const int lane = threadIdx.x & 63, row = blockIdx.y * NW + (threadIdx.x >> 6);
  if (row >= g.M) return;
  const int col_raw = (blockIdx.x * 64 + lane) * 8;
  const bool ok = col_raw < g.N;
  const int col = ok ? col_raw : g.N - 8;               // loads stay in bounds
  const bool lora_on = expand_enabled(g.ex);
  int4 sd = make_int4(-1, 0, 0, 0);
  if (lora_on) sd = expand_row_desc<E>(row, g.ex);
  const int np = pieces_of(g.splits, g.sk_g, g.sk_kt, g.bm, g.bn, g.M, g.N, row, col);
  float gv[8] = {}, uv[8] = {}, h[8];
  add_pieces(g.part[0], np, g.M, g.N, row, col, gv);
  add_pieces(g.part[1], np, g.M, g.N, row, col, uv);
  if (lora_on) {
    ExpandArgs eu = g.ex;
    eu.U = g.U_up;
    eu.b_pages = g.b_up;
    expand_row8<E>(gv, sd, col, g.ex);
    expand_row8<E>(uv, sd, col, eu);
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    float slope;
    h[x] = activate<kAct, sizeof(E) == 2>(gv[x], slope) * uv[x];
  }
  if (!ok) return;
  const int64_t at = int64_t(row) * g.N + col;
  Cols<E, 8>::store(static_cast<E *>(g.H) + at, h);
  if (g.pre_gate) {
    Cols<E, 8>::store(static_cast<E *>(g.pre_gate) + at, gv);
    Cols<E, 8>::store(static_cast<E *>(g.pre_up) + at, uv);
  }
}

// ------------------------------------------------------------ backward
template <typename E, int kAct>
__global__ __launch_bounds__(256) void gated_act_grad_kernel(const E *dH, const E *pg, const E *pu, E *dg, E *du,
                                                             int64_t n8) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n8) return;
  float h[8], g[8], u[8], a[8], b[8];
  Elem<E>::load8(dH + i * 8, h);
  Elem<E>::load8(pg + i * 8, g);
  Elem<E>::load8(pu + i * 8, u);
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    float slope;
    const float v = activate<kAct, sizeof(E) == 2>(g[x], slope);
    a[x] = h[x] * u[x] * slope;
    b[x] = h[x] * v;
  }
  Cols<E, 8>::store(dg + i * 8, a);
  Cols<E, 8>::store(du + i * 8, b);
}

// K tiles of dg.Wg^T, then those of du.Wu^T.
template <typename C>
struct GatedGradSrc {
  const uint16_t *a[2], *b[2];
  uint32_t ao[C::A_INS], bo[C::B_INS];
  int wave, wm, wn, kt1;
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    const bool p = kt >= kt1;
    const int k = (p ? kt - kt1 : kt) * 64;
    if (i < C::A_INS) {
      lds_dma16_s((p ? a[1] : a[0]) + k, ao[i], lds + (wave * C::A_INS + i) * 1024);
    } else {
      lds_dma16_s((p ? b[1] : b[0]) + k, bo[i - C::A_INS],
                  lds + C::BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
    }
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    return frag_rows(base, s, q < C::TM ? (wm * C::TM + q) * 16 : C::BM + (wn * C::TN + q - C::TM) * 16);
  }
};

template <typename C>
__global__ __launch_bounds__(C::NT, 1) void gated_grad_x_tile_kernel(GatedGradXArgs g) {
  constexpr int SC = 64 + 4;                            // a wave stages 16 rows, and those of the adapters' term
  constexpr int WLDS = 2 * 16 * SC * 4 + kTermLds;
  constexpr int TT = C::NW * WLDS;
  constexpr int LDS = TT + int(sizeof(TileTerms<C>)) > 2 * C::STAGE ? TT + int(sizeof(TileTerms<C>)) : 2 * C::STAGE;
  static_assert(C::TN == 4, "64 columns per wave");
  static_assert(TT % 16 == 0 && LDS <= 160 * 1024, "staging must fit in LDS");
  __shared__ __attribute__((aligned(16))) char smem[LDS];
  int tm, tn;
  if (!tile_of_workgroup(blockIdx.x, (g.M + C::BM - 1) / C::BM, (g.N + C::BN - 1) / C::BN, tm, tn)) return;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / C::WN, wn = wave % C::WN;
  GatedGradSrc<C> src;
  src.wave = wave; src.wm = wm; src.wn = wn;
  src.kt1 = g.Kd / 64;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    src.a[p] = static_cast<const uint16_t *>(g.dY[p]) + int64_t(m0) * g.Kd;
    src.b[p] = static_cast<const uint16_t *>(g.W[p]) + int64_t(n0) * g.Kd;
  }
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
    src.ao[i] = (uint32_t(min(row, g.M - 1 - m0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8) * 2;
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = (wave * C::B_INS + i) * 8 + (lane >> 3);
    src.bo[i] = (uint32_t(min(row, g.N - 1 - n0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8) * 2;
  }
  const int4 sd = tile_desc<C>(g.ex, m0, g.M);
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, 2 * src.kt1, acc);

  const Terms e{g.ex, g.U_up, g.b_up};
  const bool lora_on = expand_enabled(g.ex);
  TileTerms<C> &tt = *reinterpret_cast<TileTerms<C> *>(smem + TT);
  const bool common = lora_on && g.ex.K == 1 && tile_terms<C>(e, tt, sd);
  const int vr = lane >> 3, vc = (lane & 7) * 8, c0 = n0 + wn * 64;
  if (c0 >= g.N) return;
  float *stage = reinterpret_cast<float *>(smem + wave * WLDS), *lstage = stage + 16 * SC;
  char *tlds = smem + wave * WLDS + 2 * 16 * SC * 4;
  TermCache<false> cache;
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int r0 = m0 + (wm * C::TM + i) * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int v = 0; v < 4; ++v) stage[acc_row(0, v) * SC + acc_col(j)] = acc[i][j][v];
      acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    bool dropped = false;
    if (common) dropped = add_tile_terms<false, C>(e, tt, tlds, (wm * C::TM + i) * 16, c0, g.N, acc[i], cache);
    else if (lora_on) dropped = add_terms<false>(e, tlds, r0, g.M, c0, g.N, acc[i], cache);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) lstage[acc_row(0, v) * SC + acc_col(j)] = acc[i][j][v];
    if (dropped) {
#pragma unroll 1
      for (int rr = 0; rr < 16 && r0 + rr < g.M; ++rr)
        lstage[rr * SC + lane] += terms_nonfinite(e, r0 + rr, c0 + lane, 0) + terms_nonfinite(e, r0 + rr, c0 + lane, 1);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int rr = q * 8 + vr, row = r0 + rr;
      if (row >= g.M) continue;
      float b[8], l[8];
      Elem<float>::load8(stage + rr * SC + vc, b);
      Elem<float>::load8(lstage + rr * SC + vc, l);
      const int64_t at = int64_t(row) * g.N + c0 + vc;
      uint2 mw = make_uint2(0x01010101u, 0x01010101u);
      if (g.mask) mw = *reinterpret_cast<const uint2 *>(g.mask + at);
#pragma unroll
      for (int x = 0; x < 8; ++x)
        b[x] += float(((x < 4 ? mw.x : mw.y) >> (8 * (x & 3))) & 0xffu) * l[x];
      store8_nt(static_cast<uint16_t *>(g.dX) + at, b);
    }
  }
}

template <typename E, int NW>
__global__ __launch_bounds__(NW * 64) void gated_grad_x_epilogue_kernel(GatedGradXArgs g) {
  const int lane = threadIdx.x & 63, row = blockIdx.y * NW + (threadIdx.x >> 6);
  if (row >= g.M) return;
  const int col_raw = (blockIdx.x * 64 + lane) * 8;
  const bool ok = col_raw < g.N;
  const int col = ok ? col_raw : g.N - 8;
  const bool lora_on = expand_enabled(g.ex);
  int4 sd = make_int4(-1, 0, 0, 0);
  if (lora_on) sd = expand_row_desc<E>(row, g.ex);
  const int np = pieces_of(g.splits, g.sk_g, g.sk_kt, g.bm, g.bn, g.M, g.N, row, col);
  float v[8] = {}, l[8] = {};
  add_pieces(g.part[0], np, g.M, g.N, row, col, v);
  add_pieces(g.part[1], np, g.M, g.N, row, col, v);
  if (lora_on) {
    ExpandArgs eu = g.ex;
    eu.U = g.U_up;
    eu.b_pages = g.b_up;
    expand_row8<E>(l, sd, col, g.ex);
    expand_row8<E>(l, sd, col, eu);
    uint2 mw = make_uint2(0x01010101u, 0x01010101u);
    if (g.mask) mw = *reinterpret_cast<const uint2 *>(g.mask + int64_t(row) * g.N + col);
#pragma unroll
    for (int x = 0; x < 8; ++x)
      v[x] += float(((x < 4 ? mw.x : mw.y) >> (8 * (x & 3))) & 0xffu) * l[x];
  }
  if (ok) Cols<E, 8>::store(static_cast<E *>(g.dX) + int64_t(row) * g.N + col, v);
}

using Big = LoopCfg<256, 256, 2, 4>;
using Mid = LoopCfg<128, 128, 2, 2>;

template <typename E>
void launch_act_grad(const void *dH, const void *pg, const void *pu, int act, void *dg, void *du, int64_t n,
                     hipStream_t s) {
  const int64_t n8 = n / 8;
  const dim3 grid(unsigned((n8 + 255) / 256)), block(256);
  const E *h = static_cast<const E *>(dH), *g = static_cast<const E *>(pg), *u = static_cast<const E *>(pu);
  E *a = static_cast<E *>(dg), *b = static_cast<E *>(du);
  if (act == LORA_ACT_SILU)
    hipLaunchKernelGGL((gated_act_grad_kernel<E, LORA_ACT_SILU>), grid, block, 0, s, h, g, u, a, b, n8);
  else if (act == LORA_ACT_GELU)
    hipLaunchKernelGGL((gated_act_grad_kernel<E, LORA_ACT_GELU>), grid, block, 0, s, h, g, u, a, b, n8);
  else
    hipLaunchKernelGGL((gated_act_grad_kernel<E, LORA_ACT_GELU_TANH>), grid, block, 0, s, h, g, u, a, b, n8);
}

}  // namespace

bool gated_fused(int T, int d_out, int dtype) { return dtype == LORA_BF16 && T > 128; }

namespace {

template <typename C>
void launch_tiles(const GatedArgs &g, hipStream_t s) {
  const int tiles = ((g.M + C::BM - 1) / C::BM) * ((g.N + C::BN / 2 - 1) / (C::BN / 2));
  const dim3 grid(8 * unsigned((tiles + 7) / 8)), block(C::NT);
  if (g.act == LORA_ACT_SILU) hipLaunchKernelGGL((gated_tile_kernel<C, LORA_ACT_SILU>), grid, block, 0, s, g);
  else if (g.act == LORA_ACT_GELU) hipLaunchKernelGGL((gated_tile_kernel<C, LORA_ACT_GELU>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((gated_tile_kernel<C, LORA_ACT_GELU_TANH>), grid, block, 0, s, g);
}

}  // namespace

hipError_t launch_gated_tiles(const GatedArgs &g, hipStream_t s) {
  const int64_t big = int64_t((g.M + 255) / 256) * ((g.N + 127) / 128);
  if (big >= 256) launch_tiles<Big>(g, s);
  else launch_tiles<Mid>(g, s);
  return hipGetLastError();
}

hipError_t launch_gated_decode_plan(const GemmConfig &c, const GemmArgs (&g)[2], const SlotShrinkArgs (&ss)[2],
                                    const PlanLaunch &pl, hipStream_t s) {
  if (c.kind != 4 || pl.lds_bytes > plan_lds_cap(c)) return hipErrorInvalidConfiguration;
  const int gx = (g[0].N + 127) / 128, gy = (g[0].M + c.bm - 1) / c.bm, n_gemm = gx * gy * c.splits;
  const dim3 grid(unsigned(1 + 2 * n_gemm + 2 * kSlotParts * ss[0].n_slots)), block(256);
  const bool m = ss[0].mask != nullptr;
#define LORA_GD3(MB, M, L) \
  hipLaunchKernelGGL((gated_decode_plan_kernel<MB, M, L>), grid, block, 0, s, g[0], g[1], ss[0], ss[1], pl.a, gx, gy, n_gemm)
#define LORA_GD2(MB, M) do { if (pl.lds) LORA_GD3(MB, M, true); else LORA_GD3(MB, M, false); } while (0)
#define LORA_GD(MB) do { if (m) LORA_GD2(MB, true); else LORA_GD2(MB, false); } while (0)
  if (c.bm == 32) LORA_GD(1);
  else if (c.bm == 64) LORA_GD(2);
  else LORA_GD(4);
#undef LORA_GD
#undef LORA_GD2
#undef LORA_GD3
  return hipGetLastError();
}

hipError_t launch_gated_decode(const GemmConfig &c, const GemmArgs (&g)[2], hipStream_t s) {
  if (c.kind != 4) return hipErrorInvalidConfiguration;
  const dim3 grid((g[0].N + 127) / 128, (g[0].M + c.bm - 1) / c.bm, 2 * c.splits), block(256);
  if (c.bm == 32) hipLaunchKernelGGL(gated_decode_kernel<1>, grid, block, 0, s, g[0], g[1]);
  else if (c.bm == 64) hipLaunchKernelGGL(gated_decode_kernel<2>, grid, block, 0, s, g[0], g[1]);
  else hipLaunchKernelGGL(gated_decode_kernel<4>, grid, block, 0, s, g[0], g[1]);
  return hipGetLastError();
}

namespace {

template <int kAct>
void launch_epilogue(const GatedArgs &g, int dtype, hipStream_t s) {
  const unsigned n_x = unsigned((g.N + 511) / 512);
  if (dtype == LORA_BF16)
    hipLaunchKernelGGL(gated_decode_epilogue_kernel<kAct>, dim3(n_x, unsigned(g.M)), dim3(256), 0, s, g);
  else if (int64_t(n_x) * ((g.M + 3) / 4) < 256)      // one wave a workgroup where four leave CUs idle
    hipLaunchKernelGGL((gated_epilogue_kernel<float, 1, kAct>), dim3(n_x, unsigned(g.M)), dim3(64), 0, s, g);
  else
    hipLaunchKernelGGL((gated_epilogue_kernel<float, 4, kAct>), dim3(n_x, unsigned((g.M + 3) / 4)), dim3(256), 0, s, g);
}

}  // namespace

hipError_t launch_gated_epilogue(const GatedArgs &g, int dtype, hipStream_t s) {
  if (g.act == LORA_ACT_SILU) launch_epilogue<LORA_ACT_SILU>(g, dtype, s);
  else if (g.act == LORA_ACT_GELU) launch_epilogue<LORA_ACT_GELU>(g, dtype, s);
  else launch_epilogue<LORA_ACT_GELU_TANH>(g, dtype, s);
  return hipGetLastError();
}

hipError_t launch_gated_act_grad(const void *dH, const void *pre_gate, const void *pre_up, int act, void *d_gate,
                                 void *d_up, int64_t n, int dtype, hipStream_t s) {
  if (dtype == LORA_BF16) launch_act_grad<uint16_t>(dH, pre_gate, pre_up, act, d_gate, d_up, n, s);
  else launch_act_grad<float>(dH, pre_gate, pre_up, act, d_gate, d_up, n, s);
  return hipGetLastError();
}

bool gated_grad_x_fused(int T, int d_in, int dtype) {
  return dtype == LORA_BF16 && T > 128 && int64_t((T + 255) / 256) * ((d_in + 255) / 256) >= 192;
}

hipError_t launch_gated_grad_x_tiles(const GatedGradXArgs &g, hipStream_t s) {
  const int tiles = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  hipLaunchKernelGGL((gated_grad_x_tile_kernel<Big>), dim3(8 * unsigned((tiles + 7) / 8)), dim3(512), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_gated_grad_x_epilogue(const GatedGradXArgs &g, int dtype, hipStream_t s) {
  const unsigned n_x = unsigned((g.N + 511) / 512);
  const dim3 grid(n_x, unsigned((g.M + 3) / 4));
  if (dtype == LORA_BF16) hipLaunchKernelGGL((gated_grad_x_epilogue_kernel<uint16_t, 4>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((gated_grad_x_epilogue_kernel<float, 4>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace lora
