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
// Both projections' adapter terms of a 32-row block as MFMA passes: for every
// slot, adapter and 16 rank rows, U (fp32, as bf16 hi + lo, error < 2^-16 of
// U; rows of other adapters zero) times the pages' rows.  kBlocks 32-column
// blocks: block j takes projection kPair ? j : both.  kPair (the forward):
// acc[0] is the gate's, acc[1] the up projection's, both of column col[0].
// Otherwise (dX) both projections' terms go into both blocks, columns col[0]
// and col[1].  Returns whether a page value that is not finite was left out
// (see drop_nonfinite); terms_nonfinite adds those.
struct Terms {
  ExpandArgs ex;
  const float *U_up;
  const void *b_up;
};

template <bool kPair>
__device__ __forceinline__ bool add_terms(const Terms &e, int row, bool row_ok, const int (&col)[2],
                                          f32x16_t (&acc)[2]) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  bool dropped = false;
  for (int k = 0; k < e.ex.K; ++k) {
    int4 sd = make_int4(-1, 0, 0, 0);
    if (row_ok) sd = e.ex.slot_desc[int64_t(row) * e.ex.K + k];
    unsigned long long pending = __ballot(sd.x >= 0) & 0xffffffffull;
    while (pending) {
      const int leader = __ffsll(pending) - 1;
      const int kps = __builtin_amdgcn_readfirstlane(__shfl(sd.w, leader, 64));
      const int kr = __builtin_amdgcn_readfirstlane(__shfl(sd.y, leader, 64));
      const bool mine = sd.x >= 0 && sd.w == kps && sd.y == kr;
      pending &= ~__ballot(mine);
      for (int jb = 0; jb < kr; jb += 16) {
        const int nr = min(16, kr - jb);
        const int pid = e.ex.page_ids[kps + jb + min(lane & 15, nr - 1)];
        // lane (row lane % 32, or column): rank rows jb + 8 half .. + 7
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float *U = p ? e.U_up : e.ex.U;
          const uint16_t *B = static_cast<const uint16_t *>(p ? e.b_up : e.ex.b_pages);
          constexpr int NB = kPair ? 1 : 2;
          float uv[8];
          bf16x8_t bf[NB];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int j = half * 8 + q;
            uv[q] = mine && j < nr ? U[int64_t(sd.z) + jb + j] : 0.f;
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 8; q += 2) {
              const int ja = half * 8 + q;
              const int pa = __shfl(pid, ja, 64), pb = __shfl(pid, ja + 1, 64);
              uint32_t lo = B[int64_t(pa) * e.ex.d_out + col[b]], hi = B[int64_t(pb) * e.ex.d_out + col[b]];
              if (ja >= nr) lo = 0;
              if (ja + 1 >= nr) hi = 0;
              w[q >> 1] = lo | (hi << 16);
            }
            __builtin_memcpy(&bf[b], w, 16);
          }
          dropped |= drop_nonfinite<NB>(bf);
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const uint32_t h = f2bf2(uv[q], uv[q + 1]);
            hw[q >> 1] = h;
            lw[q >> 1] = f2bf2(uv[q] - bf_lo(h), uv[q + 1] - bf_hi(h));
          }
          bf16x8_t hi, lo;
          __builtin_memcpy(&hi, hw, 16);
          __builtin_memcpy(&lo, lw, 16);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            f32x16_t &a = acc[kPair ? p : b];
            a = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi, bf[b], a, 0, 0, 0);
            a = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo, bf[b], a, 0, 0, 0);
          }
        }
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
// turn (a wave's copies are all of one weight).
template <int BM, int BN, int WM, int WN>
struct GatedSrc {
  using C = TileCfg<BM, BN, WM, WN>;
  static_assert(C::B_INS * 8 == 32 && C::TN == 2, "a wave copies 32 rows of one weight");
  const uint16_t *a, *b;
  uint32_t ao[C::A_INS], bo[C::B_INS];
  int wave;
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    if (i < C::A_INS) lds_dma16(a + kt * 64 + ao[i], lds + (wave * C::A_INS + i) * 1024);
    else lds_dma16(b + kt * 64 + bo[i - C::A_INS], lds + BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    const int frow = threadIdx.x & 31, wm = wave / WN, wn = wave % WN;
    return frag_rows<C, WN>(base, s, q < C::TM ? (wm * C::TM + q) * 32 + frow
                                               : BM + (wn * C::TN + q - C::TM) * 32 + frow);
  }
};

template <int BM, int BN, int WM, int WN, int kAct>
__global__ __launch_bounds__(WM * WN * 64, 1) void gated_tile_kernel(GatedArgs g) {
  using C = TileCfg<BM, BN, WM, WN>;
  constexpr int SC = 64 + 4;                            // floats of a staged row: 32 of g, 32 of u
  constexpr int NO = BN / 2;                            // output columns of the tile
  __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
  static_assert(C::NW * 32 * SC * 4 <= 2 * C::STAGE, "staging must fit in LDS");
  int tm, tn;
  if (!tile_of_workgroup(blockIdx.x, (g.M + BM - 1) / BM, (g.N + NO - 1) / NO, tm, tn)) return;
  const int m0 = tm * BM, n0 = tn * NO;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / WN, wn = wave % WN;

  GatedSrc<BM, BN, WM, WN> src;
  src.wave = wave;
  src.a = static_cast<const uint16_t *>(g.X) + int64_t(m0) * g.Kd;
  src.b = static_cast<const uint16_t *>(g.W[wave & 1]) + int64_t(n0) * g.Kd;
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
    src.ao[i] = uint32_t(min(row, g.M - 1 - m0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8;
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = i * 8 + (lane >> 3);                // of the wave's 32
    src.bo[i] = uint32_t(min((wave >> 1) * 32 + row, g.N - 1 - n0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8;
  }
  f32x16_t acc[C::TM][C::TN];
  tile_loop<BM, BN, WM, WN>(src, smem, g.Kd / 64, acc);

  const Terms e{g.ex, g.U_up, g.b_up};
  const bool lora_on = expand_enabled(g.ex);
  const int frow = lane & 31, half = lane >> 5;
  const int c0 = n0 + wn * 32;                          // the wave's output columns
  const int col[2] = {min(c0 + frow, g.N - 1), 0};
  float *stage = reinterpret_cast<float *>(smem) + wave * 32 * SC;
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int r0 = m0 + (wm * C::TM + i) * 32;
    bool dropped = false;
    if (lora_on) dropped = add_terms<true>(e, r0 + frow, r0 + frow < g.M, col, acc[i]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        stage[((v >> 2) * 8 + half * 4 + (v & 3)) * SC + j * 32 + frow] = acc[i][j][v];
    if (dropped) {
#pragma unroll 1
      for (int rr = 0; rr < 32 && r0 + rr < g.M; ++rr)
        if (c0 + frow < g.N) stage[rr * SC + lane] += terms_nonfinite(e, r0 + rr, c0 + frow, half);
    }
    // a lane takes 8 columns of one of 16 rows
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int rr = q * 16 + (lane >> 2), row = r0 + rr, cc = (lane & 3) * 8;
      if (row >= g.M || c0 + cc >= g.N) continue;
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
template <int BM, int BN, int WM, int WN>
struct GatedGradSrc {
  using C = TileCfg<BM, BN, WM, WN>;
  const uint16_t *a[2], *b[2];
  uint32_t ao[C::A_INS], bo[C::B_INS];
  int wave, kt1;
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    const int p = kt >= kt1, k = (kt - (p ? kt1 : 0)) * 64;
    if (i < C::A_INS) lds_dma16((p ? a[1] : a[0]) + k + ao[i], lds + (wave * C::A_INS + i) * 1024);
    else lds_dma16((p ? b[1] : b[0]) + k + bo[i - C::A_INS], lds + BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    const int frow = threadIdx.x & 31, wm = wave / WN, wn = wave % WN;
    return frag_rows<C, WN>(base, s, q < C::TM ? (wm * C::TM + q) * 32 + frow
                                               : BM + (wn * C::TN + q - C::TM) * 32 + frow);
  }
};

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 1) void gated_grad_x_tile_kernel(GatedGradXArgs g) {
  using C = TileCfg<BM, BN, WM, WN>;
  constexpr int SC = 64 + 4, RS = 32 + 8;               // a wave stages 32 rows, and 8 of the adapters' term
  static_assert(C::TN == 2, "64 columns per wave");
  __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
  static_assert(C::NW * RS * SC * 4 <= 2 * C::STAGE, "staging must fit in LDS");
  int tm, tn;
  if (!tile_of_workgroup(blockIdx.x, (g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn)) return;
  const int m0 = tm * BM, n0 = tn * BN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / WN, wn = wave % WN;
  GatedGradSrc<BM, BN, WM, WN> src;
  src.wave = wave;
  src.kt1 = g.Kd / 64;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    src.a[p] = static_cast<const uint16_t *>(g.dY[p]) + int64_t(m0) * g.Kd;
    src.b[p] = static_cast<const uint16_t *>(g.W[p]) + int64_t(n0) * g.Kd;
  }
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
    src.ao[i] = uint32_t(min(row, g.M - 1 - m0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8;
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = (wave * C::B_INS + i) * 8 + (lane >> 3);
    src.bo[i] = uint32_t(min(row, g.N - 1 - n0)) * uint32_t(g.Kd) + tswz(row, lane & 7) * 8;
  }
  f32x16_t acc[C::TM][C::TN];
  tile_loop<BM, BN, WM, WN>(src, smem, 2 * src.kt1, acc);

  const Terms e{g.ex, g.U_up, g.b_up};
  const bool lora_on = expand_enabled(g.ex);
  const int frow = lane & 31, half = lane >> 5, vr = lane >> 3, vc = (lane & 7) * 8;
  const int c0 = n0 + wn * 64;
  const int col[2] = {min(c0 + frow, g.N - 1), min(c0 + 32 + frow, g.N - 1)};
  float *stage = reinterpret_cast<float *>(smem) + wave * RS * SC, *lstage = stage + 32 * SC;
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int r0 = m0 + (wm * C::TM + i) * 32;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        stage[((v >> 2) * 8 + half * 4 + (v & 3)) * SC + j * 32 + frow] = acc[i][j][v];
        acc[i][j][v] = 0.f;
      }
    bool dropped = false;
    if (lora_on) dropped = add_terms<false>(e, r0 + frow, r0 + frow < g.M, col, acc[i]);
    // the adapters' term a quarter of the rows at a time: MFMA registers
    // 4 q .. 4 q + 3 hold rows 8 q .. 8 q + 7
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = r0 + q * 8 + vr;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 4 * q; v < 4 * q + 4; ++v) lstage[(half * 4 + (v & 3)) * SC + j * 32 + frow] = acc[i][j][v];
      if (dropped) {
#pragma unroll 1
        for (int rr = 0; rr < 8 && r0 + q * 8 + rr < g.M; ++rr)
          if (c0 + lane < g.N)
            lstage[rr * SC + lane] += terms_nonfinite(e, r0 + q * 8 + rr, c0 + lane, 0) +
                                      terms_nonfinite(e, r0 + q * 8 + rr, c0 + lane, 1);
      }
      if (row < g.M && c0 + vc < g.N) {
        float b[8], l[8];
        Elem<float>::load8(stage + (q * 8 + vr) * SC + vc, b);
        Elem<float>::load8(lstage + vr * SC + vc, l);
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

template <typename E, int kAct>
void launch_epilogue_rows(const GatedArgs &g, hipStream_t s) {
  const unsigned n_x = unsigned((g.N + 511) / 512);
  // one wave a workgroup where four leave CUs idle
  if (int64_t(n_x) * ((g.M + 3) / 4) < 256)
    hipLaunchKernelGGL((gated_epilogue_kernel<E, 1, kAct>), dim3(n_x, unsigned(g.M)), dim3(64), 0, s, g);
  else
    hipLaunchKernelGGL((gated_epilogue_kernel<E, 4, kAct>), dim3(n_x, unsigned((g.M + 3) / 4)), dim3(256), 0, s, g);
}

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

bool gated_fused(int T, int d_out, int dtype) {
  return dtype == LORA_BF16 && T > 128 && int64_t((T + 255) / 256) * ((d_out + 127) / 128) >= 256;
}

hipError_t launch_gated_tiles(const GatedArgs &g, hipStream_t s) {
  const int tiles = ((g.M + 255) / 256) * ((g.N + 127) / 128);
  const dim3 grid(8 * unsigned((tiles + 7) / 8)), block(512);
  if (g.act == LORA_ACT_SILU)
    hipLaunchKernelGGL((gated_tile_kernel<256, 256, 2, 4, LORA_ACT_SILU>), grid, block, 0, s, g);
  else if (g.act == LORA_ACT_GELU)
    hipLaunchKernelGGL((gated_tile_kernel<256, 256, 2, 4, LORA_ACT_GELU>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((gated_tile_kernel<256, 256, 2, 4, LORA_ACT_GELU_TANH>), grid, block, 0, s, g);
  return hipGetLastError();
}

hipError_t launch_gated_epilogue(const GatedArgs &g, int dtype, hipStream_t s) {
  const bool bf = dtype == LORA_BF16;
  if (g.act == LORA_ACT_SILU) bf ? launch_epilogue_rows<uint16_t, LORA_ACT_SILU>(g, s) : launch_epilogue_rows<float, LORA_ACT_SILU>(g, s);
  else if (g.act == LORA_ACT_GELU) bf ? launch_epilogue_rows<uint16_t, LORA_ACT_GELU>(g, s) : launch_epilogue_rows<float, LORA_ACT_GELU>(g, s);
  else bf ? launch_epilogue_rows<uint16_t, LORA_ACT_GELU_TANH>(g, s) : launch_epilogue_rows<float, LORA_ACT_GELU_TANH>(g, s);
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
  hipLaunchKernelGGL((gated_grad_x_tile_kernel<256, 256, 2, 4>), dim3(8 * unsigned((tiles + 7) / 8)), dim3(512), 0, s, g);
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
