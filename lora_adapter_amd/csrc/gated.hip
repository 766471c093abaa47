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
// activation, product and the one rounding happen on the way out.  Batches of
// some hundred tokens leave both base products in memory, and the launch of the
// adapters' terms finishes them; up to 128 tokens take the split products of the
// single projections and an epilogue that finishes both.
#include "decode_tile.h"
#include "plan_build.h"
#include "shrink_units.h"
#include "tile_f32.h"
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
// Both projections' adapter terms of a tile as MFMA passes, a slot of the rows
// at a time: the tile's adapters are listed once, and each wave walks the list,
// 16 rank rows a pass, over those of its 16-row blocks that hold the adapter.
// A pass multiplies U (fp32; rows of other adapters zero), as bf16 hi in the
// first 16 of K and lo in the second (error < 2^-16 of U), by the page rows
// twice.  kPair (the forward): accumulator columns 0 .. 31 are the gate's c0 ..,
// 32 .. 63 the up projection's, the same c0 ...  Otherwise (dX) both
// projections' terms go into all of c0 .. c0 + 63.
// Page rows come in 16-byte loads, a pass ahead, through the wave's LDS, and are
// read transposed from there.  With one slot for each token the tile takes its
// rows in the plan's order, so that an adapter's tokens lie together and its
// pages are read by few tiles.
struct Terms {
  ExpandArgs ex;
  const float *U_up;
  const void *b_up;
};

constexpr int kTermLds = 4096;             // bytes of LDS per wave

template <typename C>
struct TileSegs {
  // page start (-1: none), rank, U offset and list entry of each row.  An adapter's
  // pages are its page start and rank: two may share the start.
  int ps[C::BM], rk[C::BM], z[C::BM], lead[C::BM];
  int l_ps[C::BM], l_r[C::BM], l_blocks[C::BM];
  int cnt[C::BM / 64], n;
};

// Slot descriptor k of tile row threadIdx.x, or none.
__device__ __forceinline__ int4 row_desc(const ExpandArgs &ex, const int *rows, int nrows, int k) {
  int4 sd = make_int4(-1, 0, 0, 0);
  if (int(threadIdx.x) < nrows && ex.U) sd = ex.slot_desc[int64_t(rows[threadIdx.x]) * ex.K + k];
  return sd;
}

// Lists the adapters of a slot of the tile's rows (sd: row_desc).  Every thread
// of the workgroup calls it.
template <typename C>
__device__ __forceinline__ void list_segs(TileSegs<C> &t, int4 sd) {
  const int r = threadIdx.x, lane = r & 63;
  lds_bar();                               // the last list is done with
  if (r < C::BM) {
    t.ps[r] = sd.x >= 0 ? sd.w : -1;
    t.rk[r] = sd.y;
    t.z[r] = sd.z;
    t.l_blocks[r] = 0;
  }
  lds_bar();
  int first = r;
  bool leads = false;
  if (r < C::BM && sd.x >= 0) {
    for (int i = 0; i < r; i += 4) {
      const int4 v = *reinterpret_cast<const int4 *>(&t.ps[i]), q = *reinterpret_cast<const int4 *>(&t.rk[i]);
      // (0: equal.  With && the compiler spills elsewhere in the tile of dX: 8192 tokens
      // 1395 -> 1500 us)
      const int m0 = (v.x ^ sd.w) | (q.x ^ sd.y), m1 = (v.y ^ sd.w) | (q.y ^ sd.y);
      const int m2 = (v.z ^ sd.w) | (q.z ^ sd.y), m3 = (v.w ^ sd.w) | (q.w ^ sd.y);
      if (m0 == 0 || m1 == 0 || m2 == 0 || m3 == 0) {
        first = i + (m0 == 0 ? 0 : m1 == 0 ? 1 : m2 == 0 ? 2 : 3);
        break;
      }
    }
    first = min(first, r);
    leads = first == r;
  }
  const unsigned long long m = __ballot(leads);
  if (r < C::BM && lane == 0) t.cnt[r >> 6] = __popcll(m);
  lds_bar();
  int at = __popcll(m & ((1ull << lane) - 1));
  for (int w = 0; w < (r >> 6) && w < C::BM / 64; ++w) at += t.cnt[w];
  if (leads) {
    t.lead[r] = at;
    t.l_ps[at] = sd.w;
    t.l_r[at] = sd.y;
  }
  if (r == 0) {
    int n = 0;
    for (int w = 0; w < C::BM / 64; ++w) n += t.cnt[w];
    t.n = n;
  }
  lds_bar();
  if (r < C::BM) {
    const int l = sd.x >= 0 ? t.lead[first] : -1;
    if (!leads) t.lead[r] = l;             // of rows that lead no list entry: no one else reads those
    if (l >= 0) atomicOr(&t.l_blocks[l], 1 << (r >> 4));
  }
  lds_bar();
}

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

// 8 floats from 4-byte aligned memory, of which the first `have` are there.
__device__ __forceinline__ void load8_tail(const float *p, int have, float (&v)[8]) {
  if (__ballot(have < 8) == 0) {
    __builtin_memcpy(v, p, 32);
    return;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = q < have ? p[q] : 0.f;
}

// acc += the listed terms for blocks blk0 .. blk0 + NB - 1 of the tile.  Returns the blocks (bit i: block blk0 + i)
// that a page value which is not finite was left out of: it would reach other
// adapters' rows as 0 . inf.  terms_nonfinite adds those.
template <bool kPair, typename C, int NB>
__device__ __forceinline__ unsigned add_segs(const Terms &e, const TileSegs<C> &t, char *lds, int blk0, int c0, int N,
                                             f32x4_t (&acc)[NB][4]) {
  constexpr int CPL = kPair ? 4 : 8;       // lanes along a page's columns
  constexpr int NL = kPair ? 1 : 2;        // loads of a projection
  constexpr int NF = kPair ? 2 : 4;        // fragments of a projection
  constexpr int PITCH = CPL * 16, SIZE = 16 * PITCH;
  const int lane = threadIdx.x & 63, col = min(c0 + (lane % CPL) * 8, N - 8);
  const int n = __builtin_amdgcn_readfirstlane(t.n), mine_mask = ((1 << NB) - 1) << blk0;
  const int total = e.ex.hdr[LORA_PH_RPAIRS];

  auto entry = [&](int li) __attribute__((always_inline)) {
    while (li < n && !(__builtin_amdgcn_readfirstlane(t.l_blocks[li]) & mine_mask)) ++li;
    return li;
  };
  // the pass after (li, jb)
  auto after = [&](int &li, int &jb) __attribute__((always_inline)) {
    jb += 16;
    if (jb >= __builtin_amdgcn_readfirstlane(t.l_r[li])) {
      jb = 0;
      li = entry(li + 1);
    }
  };
  auto ids = [&](int li, int jb, int (&id)[NL]) __attribute__((always_inline)) {
    const int nr = min(16, t.l_r[li] - jb), at = t.l_ps[li] + jb;
#pragma unroll
    for (int h = 0; h < NL; ++h) id[h] = e.ex.page_ids[at + min(lane / CPL + h * (64 / CPL), nr - 1)];
  };
  auto rows = [&](const int (&id)[NL], uint4 (&v)[2][NL]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < NL; ++h) {
      const int64_t at = int64_t(id[h]) * e.ex.d_out + col;
      v[0][h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(e.ex.b_pages) + at);
      v[1][h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(e.b_up) + at);
    }
  };

  unsigned dropped = 0;
  int li = entry(0), jb = 0;
  if (li >= n) return 0;
  int id[NL];
  uint4 v[2][NL], w[2][NL];
  ids(li, jb, id);
  rows(id, v);
  int lj = li, jj = jb;                    // the next pass
  after(lj, jj);
  if (lj < n) ids(lj, jj, id);
  while (true) {
    const bool more = lj < n;
    if (more) rows(id, w);
    int lk = lj, jk = jj;
    if (more) after(lk, jk);
    if (more && lk < n) ids(lk, jk, id);

    const int nr = min(16, __builtin_amdgcn_readfirstlane(t.l_r[li]) - jb), j0 = 8 * ((lane >> 4) & 1);
    const int blocks = __builtin_amdgcn_readfirstlane(t.l_blocks[li]) >> blk0;
    // page rows: to LDS, and back as the B operand (column lane % 16, rank rows j0 .. + 7)
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
    const bool any_bad = __ballot(bad) != 0;
    bf16x8_t b[2 * NF];
    typedef __attribute__((address_space(3))) v4i16_t lds_v4;
    const int L = lane & 15, kk = j0 + (L >> 2);
#pragma unroll
    for (int f = 0; f < 2 * NF; ++f) {
      const char *p = lds + (f / NF) * SIZE + kk * PITCH + (f % NF) * 32 + (L & 3) * 8;
      const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p));
      const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p + 4 * PITCH));
      __builtin_memcpy(&b[f], &lo, 8);
      __builtin_memcpy(reinterpret_cast<char *>(&b[f]) + 8, &hi, 8);
    }
    // U of two blocks in flight (one where both projections' fragments take the registers)
    constexpr int UB = kPair ? 2 : 1;
#pragma unroll
    for (int i0 = 0; i0 < NB; i0 += UB) {
      if (!((blocks >> i0) & ((1 << UB) - 1))) continue;
      float x[UB][2][8];
#pragma unroll
      for (int i = 0; i < UB; ++i) {
        // lane (row lane % 16, rank rows j0 .. j0 + 7); U's end may cut the 8 off
        const int r = (blk0 + i0 + i) * 16 + L, at = t.z[r] + jb + j0;
        const bool mine = ((blocks >> (i0 + i)) & 1) && t.lead[r] == li;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          load8_tail((p ? e.U_up : e.ex.U) + (mine ? at : 0), min(8, mine ? total - at : total), x[i][p]);
      }
#pragma unroll
      for (int i = 0; i < UB; ++i) {
        if (!((blocks >> (i0 + i)) & 1)) continue;
        if (any_bad) dropped |= 1u << (i0 + i);
        const bool mine = t.lead[(blk0 + i0 + i) * 16 + L] == li;
        bf16x8_t u[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t q4[4];
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const float x0 = mine && j0 + q < nr ? x[i][p][q] : 0.f, x1 = mine && j0 + q + 1 < nr ? x[i][p][q + 1] : 0.f;
            const uint32_t h = f2bf2(x0, x1);
            q4[q >> 1] = lane < 32 ? h : f2bf2(x0 - bf_lo(h), x1 - bf_hi(h));
          }
          __builtin_memcpy(&u[p], q4, 16);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f32x4_t &o = acc[i0 + i][c];
          if constexpr (kPair) {
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[c >> 1], b[c], o, 0, 0, 0);
          } else {
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[0], b[c], o, 0, 0, 0);
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[1], b[4 + c], o, 0, 0, 0);
          }
        }
      }
    }
    if (!more) return dropped;
    li = lj; jb = jj;
    lj = lk; jj = jk;
#pragma unroll
    for (int h = 0; h < NL; ++h) {
      v[0][h] = w[0][h];
      v[1][h] = w[1][h];
    }
  }
}

// The common case of a prefill (one slot for each token, ranks of at most 16):
// U of all the tile's rows goes to LDS at once, as the fragments of add_segs, and
// the blocks take theirs one by one, the last adapter's page rows kept in
// registers.  8192 tokens of four adapters in runs, 4096 -> 11008, three outputs:
// 1272 us, 1343 by add_segs.
template <bool kPair>
struct TermCache {
  static constexpr int NF = kPair ? 4 : 8;
  int key = -1, rank = 0;                  // the adapter's page start, or -1, and rank
  bool dropped = false;                    // its values that are not finite were left out
  bf16x8_t b[NF];                          // kPair: gate 0, 1, up 0, 1; else gate 0 .. 3, up 0 .. 3
};

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
  t.rank = nr;
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

template <typename C>
struct TileTerms {
  int4 sd[C::BM];                          // .x < 0: no adapter
  uint16_t u[2][2][C::BM][16];             // [projection][hi, lo][row][rank row]
  int wide;                                // a rank over 16
};

// Fills t (sd: row_desc, of slot 0); false where a rank is over 16.  Every thread
// of the workgroup calls it.
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

// The terms of the block from tile row tr; returns whether values that are not
// finite were left out.
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
    if (t.key != kps || t.rank != kr) load_terms<kPair>(e, lds, kps, kr, c0, N, t);
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

template <typename C>
struct TileLists {
  static constexpr int SIZE = int(sizeof(TileTerms<C>) > sizeof(TileSegs<C>) ? sizeof(TileTerms<C>) : sizeof(TileSegs<C>));
};

// The tokens of tile rows m0 ..: with one slot for each token those of the
// plan's pairs in its order, then the tokens without an active slot; else, or
// where `in_order` asks for it, in token order.  Returns their number.  Every thread of the workgroup calls it.
template <typename C>
__device__ __forceinline__ int tile_rows(const ExpandArgs &ex, const int32_t *slot_pos, int *rows, int *cnt, int m0,
                                         int M, bool in_order) {
  const int n = min(C::BM, M - m0), tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (ex.K != 1 || in_order) {
    if (tid < n) rows[tid] = m0 + tid;
    lds_bar();
    return n;
  }
  // (the pair's place exists in the plan, past its pairs too)
  const int P = ex.hdr[LORA_PH_PAIRS], t = ex.pair_tk[m0 + min(tid, n - 1)];
  if (tid < n && m0 + tid < P) rows[tid] = t;
  if (m0 + n > P) {
    int at = P - m0;                       // tile row of the next token without a pair
    for (int t0 = 0; t0 < M && at < n; t0 += C::NT) {
      const bool idle = t0 + tid < M && slot_pos[t0 + tid] < 0;
      const unsigned long long m = __ballot(idle);
      lds_bar();
      if (lane == 0) cnt[wave] = __popcll(m);
      lds_bar();
      int mine = at + __popcll(m & ((1ull << lane) - 1)), all = 0;
      for (int w = 0; w < C::NW; ++w) {
        if (w < wave) mine += cnt[w];
        all += cnt[w];
      }
      if (idle && mine >= 0 && mine < n) rows[mine] = t0 + tid;
      at += all;
    }
  }
  lds_bar();
  return n;
}

// What add_segs left out: the products of U with the page values that are not
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

// Whether the plan has a pair for one of token t's first n slots.
__device__ __forceinline__ bool any_slot(const int32_t *slot_pos, int t, int K, int n) {
  bool any = false;
  for (int k = 0; k < n; ++k) any |= slot_pos[int64_t(t) * K + k] >= 0;
  return any;
}
__device__ __forceinline__ bool any_slot(const int32_t *slot_pos, int t, int K) { return any_slot(slot_pos, t, K, K); }

// ------------------------------------------------------------ adapters' terms to memory
// Batches of some hundred tokens have few tiles and many adapters for each of
// them: walking those in the tiles is a chain of round trips (700 tokens of 96
// adapters of ranks 8 .. 64, 2240 -> 5824: 235 us for the tiles).  There the base
// products go to memory in float32 (which needs no plan: one workgroup of that
// launch builds it), and a launch of one-wave workgroups forms the terms
// sum_j U[u + j] . page_j[n] for slot k of the tokens and finishes what it can.
// A wave takes 16 pairs of the plan's order and 128 columns (64 of each
// projection), so that pages are read once for the pairs of an adapter among
// them, and there are thousands of waves.  It walks their adapters, 16 rank rows
// a pass, with the page ids two passes ahead and page rows and U one.
// Launched slot by slot (or for all at once, see launch_terms): a token's first active slot adds the base product's
// splits, its last one finishes (activation, product and rounding; for kSum,
// dX, both projections' terms under the mask and the rounding), the ones between
// leave the sum in split 0.  The first launch also finishes, 16 tokens a wave,
// those without an active slot.
// The products are MFMAs with the rows of other adapters zero, so that all runs
// of a window share accumulators: with a branch for each row and rank row, or
// every product on the vector units, that launch took 270 us and 73 without
// finishing anything, as MFMAs 45; with its epilogue it takes 49 (57 with the next
// pass's rows in registers instead of LDS: 138 of them instead of 99).
// bf16 pages: U as hi | lo against the rows twice, as in add_segs; float32 pages:
// v_mfma_f32_16x16x4_f32.
template <typename E, bool kPair> struct TermTile;
template <bool kPair> struct TermTile<uint16_t, kPair> {
  static constexpr int COLS = 128, NBLK = 8, NV = 4;
  uint4 v[NV];
  float u[kPair ? 2 : 1][8];
  // kPair: rank rows lane / 8 + 8 (h % 2) of projection h / 2, columns 8 (lane % 8) ..;
  // else of projection p rows lane / 16 + 4 h, columns 8 (lane % 16) ..  (page id in
  // the lane of the row's number)
  static __device__ __forceinline__ int row(int h) {
    const int lane = threadIdx.x;
    return kPair ? (lane >> 3) + 8 * (h & 1) : (lane >> 4) + 4 * h;
  }
  __device__ __forceinline__ void load(const void *const (&pages)[2], int p, int id, int c0, int N) {
    const int lane = threadIdx.x, col = min(c0 + (kPair ? lane & 7 : lane & 15) * 8, N - 8);
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const uint16_t *from = static_cast<const uint16_t *>((kPair ? h >> 1 : p) ? pages[1] : pages[0]);
      v[h] = *reinterpret_cast<const uint4 *>(from + int64_t(__shfl(id, row(h), 64)) * N + col);
    }
  }
  // the loaded pass to LDS and to the A operand; whether values that are not
  // finite were left out
  bf16x8_t a[kPair ? 2 : 1];
  __device__ __forceinline__ bool put(char *lds, int nr) {
    const int lane = threadIdx.x;
    bool bad = false;
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const int j = row(h), piece = kPair ? (lane & 7) + 8 * (h >> 1) : lane & 15;
      if (j >= nr) v[h] = make_uint4(0u, 0u, 0u, 0u);
      bad |= drop8(v[h]);
      *reinterpret_cast<uint4 *>(lds + j * 256 + (piece ^ ((j & 3) << 1)) * 16) = v[h];
    }
#pragma unroll
    for (int p = 0; p < (kPair ? 2 : 1); ++p) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        const uint32_t h = f2bf2(u[p][q], u[p][q + 1]);
        w[q >> 1] = lane < 32 ? h : f2bf2(u[p][q] - bf_lo(h), u[p][q + 1] - bf_hi(h));
      }
      __builtin_memcpy(&a[p], w, 16);
    }
    return __ballot(bad) != 0;
  }
  // acc += U.rows of the pass that was put
  __device__ __forceinline__ void mul(const char *lds, f32x4_t (&acc)[NBLK]) const {
    const int lane = threadIdx.x, L = lane & 15;
    typedef __attribute__((address_space(3))) v4i16_t lds_v4;
    const int k = 8 * ((lane >> 4) & 1) + (L >> 2);
#pragma unroll
    for (int b = 0; b < NBLK; ++b) {
      // 16-byte piece 2 b + L % 4 / 2 of row k, in slot ^ 2 (k % 4)
      const char *p = lds + k * 256 + ((2 * b + ((L & 3) >> 1)) ^ ((k & 3) << 1)) * 16 + (L & 1) * 8;
      const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p));
      const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p + 4 * 256));
      bf16x8_t f;
      __builtin_memcpy(&f, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char *>(&f) + 8, &hi, 8);
      acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[kPair ? b / 4 : 0], f, acc[b], 0, 0, 0);
    }
  }
  static __device__ __forceinline__ bool finite(uint16_t v) { return (v & 0x7f80u) != 0x7f80u; }
};
template <bool kPair> struct TermTile<float, kPair> {
  static constexpr int COLS = 64, NBLK = 4, NV = 16;
  float v[NV], x[NV];
  float u[kPair ? 2 : 1][8], a[kPair ? 2 : 1][4];
  // v[4 b + s]: rank row 4 s + lane / 16, column 16 b + lane % 16 (kPair: 16 (b % 2)
  // + lane % 16 of projection b / 2)
  __device__ __forceinline__ void load(const void *const (&pages)[2], int p, int id, int c0, int N) {
    const int lane = threadIdx.x;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t at = int64_t(__shfl(id, 4 * s + (lane >> 4), 64)) * N + (lane & 15);
#pragma unroll
      for (int b = 0; b < NBLK; ++b) {
        const float *from = static_cast<const float *>((kPair ? b >> 1 : p) ? pages[1] : pages[0]);
        v[4 * b + s] = from[at + min(c0 + 16 * (kPair ? b & 1 : b), N - 16)];
      }
    }
  }
  __device__ __forceinline__ bool put(char *, int nr) {
    const int lane = threadIdx.x;
    bool bad = false;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // u: ranks 8 (lane / 16 % 2) .. of row lane % 16; wanted: rank 4 s + lane / 16
#pragma unroll
      for (int p = 0; p < (kPair ? 2 : 1); ++p) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float t = __shfl(u[p][(4 * s + g) & 7], (lane & 15) + 16 * ((4 * s + g) >> 3), 64);
          if ((lane >> 4) == g) a[p][s] = t;
        }
      }
#pragma unroll
      for (int b = 0; b < NBLK; ++b) {
        float &o = x[4 * b + s];
        o = 4 * s + (lane >> 4) < nr ? v[4 * b + s] : 0.f;
        if (!(o - o == 0.f)) {
          bad = true;
          o = 0.f;
        }
      }
    }
    return __ballot(bad) != 0;
  }
  __device__ __forceinline__ void mul(const char *, f32x4_t (&acc)[NBLK]) const {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int b = 0; b < NBLK; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[kPair ? b / 2 : 0][s], x[4 * b + s], acc[b], 0, 0, 0);
  }
  static __device__ __forceinline__ bool finite(float v) { return v - v == 0.f; }
};

// v += the base product's sums at i, of all splits (`first`) or what an earlier
// slot left in split 0.
__device__ __forceinline__ void add_sums(const TermsArgs &a, int p, int64_t i, bool first, float (&v)[8]) {
  const int64_t n = int64_t(a.M) * a.N;
  const int splits = first ? a.splits : 1;
  for (int z0 = 0; z0 < splits; z0 += 4) {
    Raw8<float> pr[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) pr[z].load(a.sums[p] + int64_t(min(z0 + z, splits - 1)) * n + i);
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      if (z0 + z < splits) {
        float o[8];
        pr[z].to8(o);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += o[c];
      }
    }
  }
}

// 8 columns of a token, whose terms of this slot are in term[0] (kSum) or term[0]
// and term[1].
template <typename E, bool kSum>
__device__ __forceinline__ void finish8(const TermsArgs &a, int64_t i, bool first, bool last, float (&term)[2][8]) {
  if constexpr (kSum) {
    float v[8] = {};
    add_sums(a, 0, i, first, v);
    uint2 mw = make_uint2(0x01010101u, 0x01010101u);
    if (a.mask) mw = *reinterpret_cast<const uint2 *>(a.mask + i);
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] += float(((x < 4 ? mw.x : mw.y) >> (8 * (x & 3))) & 0xffu) * term[0][x];
    if (last) Cols<E, 8>::store(static_cast<E *>(a.dX) + i, v);
    else Cols<float, 8>::store(a.sums[0] + i, v);
  } else {
    add_sums(a, 0, i, first, term[0]);
    add_sums(a, 1, i, first, term[1]);
    if (!last) {
      Cols<float, 8>::store(a.sums[0] + i, term[0]);
      Cols<float, 8>::store(a.sums[1] + i, term[1]);
      return;
    }
    constexpr bool kFast = sizeof(E) == 2;
    float h[8], slope;
    if (a.act == LORA_ACT_SILU) {
#pragma unroll
      for (int x = 0; x < 8; ++x) h[x] = activate<LORA_ACT_SILU, kFast>(term[0][x], slope) * term[1][x];
    } else if (a.act == LORA_ACT_GELU) {
#pragma unroll
      for (int x = 0; x < 8; ++x) h[x] = activate<LORA_ACT_GELU, kFast>(term[0][x], slope) * term[1][x];
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) h[x] = activate<LORA_ACT_GELU_TANH, kFast>(term[0][x], slope) * term[1][x];
    }
    Cols<E, 8>::store(static_cast<E *>(a.H) + i, h);
    if (a.pre_gate) {
      Cols<E, 8>::store(static_cast<E *>(a.pre_gate) + i, term[0]);
      Cols<E, 8>::store(static_cast<E *>(a.pre_up) + i, term[1]);
    }
  }
}

constexpr int kWindowRows = 32768;                      // of the grid's second dimension

// kApart: all slots at once, each slot's terms to a.slots; terms_finish_kernel adds them.
template <typename E, bool kSum, bool kApart>
__global__ __launch_bounds__(64) void terms_kernel(TermsArgs a) {
  constexpr bool kPair = !kSum;
  constexpr int NP = kPair ? 2 : 1;
  using Tile = TermTile<E, kPair>;
  constexpr int COLS = Tile::COLS / NP;                 // output columns of the wave
  constexpr int SC = Tile::COLS + 4;                    // floats of a staged row: COLS of each projection
  __shared__ __attribute__((aligned(16))) char lds[16 * SC * 4];
  static_assert(sizeof(lds) >= 4096, "a pass's page rows");
  const int P = a.hdr[LORA_PH_PAIRS], total = a.hdr[LORA_PH_RPAIRS], lane = threadIdx.x;
  const int window = int(blockIdx.z) * kWindowRows + int(blockIdx.y), c0 = int(blockIdx.x) * COLS;
  const bool lora_on = int64_t(total) <= a.u_cap;
  if (window >= a.windows) {
    // tokens without an active slot
    const int t = (window - a.windows) * 16 + (lane >> 2);
    if (t >= a.M || (lora_on && any_slot(a.slot_pos, t, a.K))) return;
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) {
      const int col = c0 + h * 32 + (lane & 3) * 8;
      float zero[2][8] = {};
      if (col < a.N) finish8<E, kSum>(a, int64_t(t) * a.N + col, true, true, zero);
    }
    return;
  }
  const int p0 = window * 16, m = min(16, P - p0);
  if (m <= 0 || !lora_on) return;
  // lane l (mod 16): pair p0 + l
  const int pl = p0 + min(lane & 15, m - 1);
  const int tk = a.pair_tk[pl], ad = a.pair_adapter[pl], uo = a.u_off[pl];
  const int rk = a.rank[ad], pst = a.page_start[ad];
  const unsigned want = unsigned(__ballot(lane < m && (kApart || tk % a.K == a.k))) & 0xffffu;
  if (!want) return;
  auto lane_of = [&](int v, int l) __attribute__((always_inline)) { return __builtin_amdgcn_readlane(v, l); };
  // a pass: projection p (kPair: both), the run of pairs [i, j) of one adapter, rank rows jb ..
  struct Pass {
    int p, i, j, jb;
  };
  auto run_at = [&](Pass &x, int i) __attribute__((always_inline)) {
    // the next run from pair i that has a wanted pair
    while (i < m) {
      const int who = lane_of(ad, i);
      const unsigned same = unsigned(__ballot(lane < m && ad == who)) & 0xffffu;
      const int j = i + __popc(same >> i);         // pairs of an adapter lie together
      if (want & same) {
        x.i = i; x.j = j; x.jb = 0;
        return;
      }
      i = j;
    }
    x.i = x.j = m;
  };
  auto after = [&](Pass &x) __attribute__((always_inline)) {
    x.jb += 16;
    if (x.jb < lane_of(rk, x.i)) return;
    x.jb = 0;
    if (kSum && x.p == 0) {
      x.p = 1;
      return;
    }
    if (kSum) x.p = 0;
    run_at(x, x.j);
  };
  auto ids = [&](const Pass &x) __attribute__((always_inline)) {
    const int nr = min(16, lane_of(rk, x.i) - x.jb);
    return a.page_ids[lane_of(pst, x.i) + x.jb + min(lane & 15, nr - 1)];
  };
  auto fetch = [&](const Pass &x, int id, Tile &v) __attribute__((always_inline)) {
    v.load(a.pages, x.p, id, c0, a.N);
    // U of row lane % 16, ranks 8 (lane / 16 % 2) .. + 7 of the pass
    const int r = lane & 15, j0 = 8 * ((lane >> 4) & 1), nr = min(16, lane_of(rk, x.i) - x.jb);
    const bool mine = r >= x.i && r < x.j;
    const int at = uo + x.jb + j0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      load8_tail(((kPair ? p : x.p) ? a.U[1] : a.U[0]) + (mine ? at : 0), min(8, mine ? total - at : total), v.u[p]);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (!mine || j0 + q >= nr) v.u[p][q] = 0.f;
    }
  };

  Pass c, n1;
  c.p = 0;
  run_at(c, 0);
  n1 = c;
  Tile v;
  int id = ids(c);
  fetch(c, id, v);
  after(n1);
  if (n1.i < m) id = ids(n1);
  f32x4_t acc[Tile::NBLK];
#pragma unroll
  for (int b = 0; b < Tile::NBLK; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  bool dropped = false;
  while (true) {
    dropped |= v.put(lds, min(16, lane_of(rk, c.i) - c.jb));
    const bool more = n1.i < m;
    c = n1;
    if (more) {
      fetch(c, id, v);
      after(n1);
      if (n1.i < m) id = ids(n1);
    }
    v.mul(lds, acc);
    if (!more) break;
  }
  // through LDS, to lanes that hold 8 columns of a row
  float *stage = reinterpret_cast<float *>(lds);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int r = acc_row(0, x);
    const int rr = __shfl(rk, r, 64), ps = __shfl(pst, r, 64), at = __shfl(uo, r, 64);
#pragma unroll
    for (int b = 0; b < Tile::NBLK; ++b) {
      float y = acc[b][x];
      const int col = c0 + (acc_col(b) % COLS), p = acc_col(b) / COLS;
      if (dropped && r < m && col < a.N) {
        // the values left out: infinities and NaN
        for (int q = p; q < (kSum ? 2 : p + 1); ++q)
          for (int j = 0; j < rr; ++j) {
            const E z = static_cast<const E *>(a.pages[q])[int64_t(a.page_ids[ps + j]) * a.N + col];
            if (!Tile::finite(z)) y = fmaf(a.U[q][int64_t(at) + j], Elem<E>::to_f(z), y);
          }
      }
      stage[r * SC + acc_col(b)] = y;
    }
  }
  const int r = lane >> 2, my_tk = __shfl(tk, r, 64), t = my_tk / a.K;
  if (!((want >> r) & 1)) return;
  if constexpr (kApart) {
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) {
      const int cc = h * 32 + (lane & 3) * 8, col = c0 + cc;
      if (col >= a.N) continue;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        float term[8];
        Elem<float>::load8(stage + r * SC + p * COLS + cc, term);
        Cols<float, 8>::store(a.slots[p] + (int64_t(my_tk % a.K) * a.M + t) * a.N + col, term);
      }
    }
    return;
  }
  const bool first = !any_slot(a.slot_pos, t, a.K, a.k);
  bool last = true;
  for (int k = a.k + 1; k < a.K; ++k) last &= a.slot_pos[int64_t(t) * a.K + k] < 0;
#pragma unroll
  for (int h = 0; h < COLS / 32; ++h) {
    const int cc = h * 32 + (lane & 3) * 8, col = c0 + cc;
    if (col >= a.N) continue;
    float term[2][8];
#pragma unroll
    for (int p = 0; p < NP; ++p) Elem<float>::load8(stage + r * SC + p * COLS + cc, term[p]);
    finish8<E, kSum>(a, int64_t(t) * a.N + col, first, last, term);
  }
}

// What terms_kernel left apart: 8 columns of a token a thread, its slots in order.
template <typename E, bool kSum>
__global__ __launch_bounds__(256) void terms_finish_kernel(TermsArgs a) {
  const int64_t n = int64_t(a.M) * a.N, i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const int t = int(i / a.N);
  const bool lora_on = int64_t(a.hdr[LORA_PH_RPAIRS]) <= a.u_cap;
  float term[2][8] = {};
  for (int k = 0; lora_on && k < a.K; ++k) {
    if (a.slot_pos[int64_t(t) * a.K + k] < 0) continue;
#pragma unroll
    for (int p = 0; p < (kSum ? 1 : 2); ++p) {
      float x[8];
      Elem<float>::load8(a.slots[p] + k * n + i, x);
#pragma unroll
      for (int c = 0; c < 8; ++c) term[p][c] += x[c];
    }
  }
  finish8<E, kSum>(a, i, true, true, term);
}

// ------------------------------------------------------------ forward, tiles
// A rows of X by 32 rows of the gate's and 32 of the up projection's weight in
// turn.
template <typename C, bool kWide>
struct GatedSrc {
  static_assert(C::TN == 4, "32 columns of each projection per wave");
  const uint16_t *a, *b[2];
  RowOffsets<C::A_INS, kWide> ao;
  uint32_t bo[C::B_INS];
  int wave, wm, wn;
  // row_of(r): the token of tile row r
  template <typename F>
  __device__ __forceinline__ void set(const GatedArgs &g, int n0, const F &row_of) {
    const int lane = threadIdx.x & 63;
    wave = wave_id();
    wm = wave / C::WN;
    wn = wave % C::WN;
    a = static_cast<const uint16_t *>(g.X);
#pragma unroll
    for (int p = 0; p < 2; ++p) b[p] = static_cast<const uint16_t *>(g.W[p]) + int64_t(n0) * g.Kd;
#pragma unroll
    for (int i = 0; i < C::A_INS; ++i) {
      const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
      ao.set(i, int64_t(row_of(row)) * g.Kd + fswz(row, lane & 7) * 8);
    }
#pragma unroll
    for (int i = 0; i < C::B_INS; ++i) {
      const int row = (wave * C::B_INS + i) * 8 + (lane >> 3);
      const int of = (row >> 6) * 32 + (row & 31);        // of its weight
      bo[i] = (uint32_t(min(of, g.N - 1 - n0)) * uint32_t(g.Kd) + fswz(row, lane & 7) * 8) * 2;
    }
  }
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    if (i < C::A_INS) {
      ao.copy(a + kt * 64, i, lds + (wave * C::A_INS + i) * 1024);
    } else {
      const int ib = wave * C::B_INS + i - C::A_INS;     // 8 rows of the B tile, all of one weight
      lds_dma16_s(((ib >> 2) & 1 ? b[1] : b[0]) + kt * 64, bo[i - C::A_INS], lds + C::BM * C::ROWB + ib * 1024);
    }
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    return frag_rows(base, s, q < C::TM ? (wm * C::TM + q) * 16 : C::BM + (wn * C::TN + q - C::TM) * 16);
  }
};

template <typename C, bool kWide, int kAct>
__global__ __launch_bounds__(C::NT, 1) void gated_tile_kernel(GatedArgs g) {
  constexpr int SC = 64 + 4;                            // floats of a staged row: 32 of g, 32 of u
  constexpr int NO = C::BN / 2;                         // output columns of the tile
  constexpr int WLDS = 16 * SC * 4 + kTermLds;          // bytes of a wave's epilogue
  constexpr int TS = C::NW * WLDS;                      // the list of adapters lies behind those
  __shared__ __attribute__((aligned(16))) char smem[C::LDS];
  __shared__ int rows[C::BM], cnt[C::NW];
  static_assert(TS % 16 == 0 && TS + TileLists<C>::SIZE <= C::LDS, "staging must fit in LDS");
  int tm, tn;
  if (!tile_of_workgroup(blockIdx.x, (g.M + C::BM - 1) / C::BM, (g.N + NO - 1) / NO, tm, tn)) return;
  const int m0 = tm * C::BM, n0 = tn * NO;
  const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / C::WN, wn = wave % C::WN;
  const int nrows = tile_rows<C>(g.ex, g.slot_pos, rows, cnt, m0, g.M, false);

  GatedSrc<C, kWide> src;
  src.set(g, n0, [&](int row) { return rows[min(row, nrows - 1)]; });
  // fetched under the K loop
  const int4 sd0 = row_desc(g.ex, rows, nrows, 0);
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, g.Kd / 64, acc);

  const Terms e{g.ex, g.U_up, g.b_up};
  TileSegs<C> &segs = *reinterpret_cast<TileSegs<C> *>(smem + TS);
  const int c0 = n0 + wn * 32;                          // the wave's output columns
  const bool inside = c0 < g.N;
  float *stage = reinterpret_cast<float *>(smem + wave * WLDS);
  char *tlds = smem + wave * WLDS + 16 * SC * 4;
  unsigned dropped = 0;
  const bool lora_on = expand_enabled(g.ex);
  TileTerms<C> &tt = *reinterpret_cast<TileTerms<C> *>(smem + TS);
  const bool common = lora_on && g.ex.K == 1 && tile_terms<C>(e, tt, sd0);
  if (lora_on && !common) {
    for (int k = 0; k < g.ex.K; ++k) {
      list_segs<C>(segs, k ? row_desc(g.ex, rows, nrows, k) : sd0);
      if (inside) dropped |= add_segs<true, C, C::TM>(e, segs, tlds, wm * C::TM, c0, g.N, acc);
    }
  }
  if (!inside) return;
  TermCache<true> cache;
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int r0 = (wm * C::TM + i) * 16;
    if (common && add_tile_terms<true, C>(e, tt, tlds, r0, c0, g.N, acc[i], cache)) dropped |= 1u << i;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) stage[acc_row(0, v) * SC + acc_col(j)] = acc[i][j][v];
    if ((dropped >> i) & 1) {
#pragma unroll 1
      for (int rr = 0; rr < 16 && r0 + rr < nrows; ++rr)
        stage[rr * SC + lane] += terms_nonfinite(e, rows[r0 + rr], c0 + (lane & 31), lane >> 5);
    }
    // a lane takes 8 columns of one of the rows
    const int rr = lane >> 2, cc = (lane & 3) * 8;
    if (r0 + rr >= nrows) continue;
    float gv[8], uv[8], h[8];
    Elem<float>::load8(stage + rr * SC + cc, gv);
    Elem<float>::load8(stage + rr * SC + 32 + cc, uv);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float slope;
      h[x] = activate<kAct, true>(gv[x], slope) * uv[x];
    }
    const int64_t at = int64_t(rows[r0 + rr]) * g.N + c0 + cc;
    store8_nt(static_cast<uint16_t *>(g.H) + at, h);
    if (g.pre_gate) {
      store8_nt(static_cast<uint16_t *>(g.pre_gate) + at, gv);
      store8_nt(static_cast<uint16_t *>(g.pre_up) + at, uv);
    }
  }
}

// The base products alone, in float32 (no plan needed: where pa has one to build,
// the first workgroup does, so that its 12 .. 20 us lie under the product's).
template <typename C>
__global__ __launch_bounds__(C::NT, 1) void gated_base_tile_kernel(GatedArgs g, PlanArgs pa) {
  __shared__ __attribute__((aligned(16))) char smem[C::LDS];
  int b = blockIdx.x, tm, tn;
  if (pa.plan) {
    if (b == 0) {
      plan_build<true>(pa, reinterpret_cast<int *>(smem));
      return;
    }
    --b;
  }
  constexpr int NO = C::BN / 2;
  if (!tile_of_workgroup(b, (g.M + C::BM - 1) / C::BM, (g.N + NO - 1) / NO, tm, tn)) return;
  const int m0 = tm * C::BM, n0 = tn * NO;
  GatedSrc<C, false> src;
  src.set(g, n0, [&](int row) { return min(m0 + row, g.M - 1); });
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, g.Kd / 64, acc);
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = n0 + src.wn * 32 + acc_col(j & 1);
      if (col >= g.N) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = m0 + src.wm * C::TM * 16 + acc_row(i, v);
        if (row < g.M) g.sums[j >> 1][int64_t(row) * g.N + col] = acc[i][j][v];
      }
    }
}

// ------------------------------------------------------------ decode
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
// launch lasts as long as its longest chain: at 48 tokens of two adapters of ranks
// 8 .. 64 (4096 -> 11008) one wave for all four took 39 us, these 32, eight waves by
// quarters 35; pages and pieces are some 140 MB.
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

// ------------------------------------------------------------ float32
// The base products of 64 tokens by 32 output columns, of a split of K: the B side
// of a tile_f32 is 32 rows of each weight.  The plan as in gated_base_tile_kernel.
__global__ __launch_bounds__(256) void gated_base_f32_kernel(GatedArgs g, PlanArgs pa) {
  __shared__ F32Tile lds;
  int b = blockIdx.x;
  if (pa.plan) {
    if (b == 0) {
      plan_build<true>(pa, reinterpret_cast<int *>(&lds));
      return;
    }
    --b;
  }
  const int gx = g.N / 32, gy = (g.M + 63) / 64;
  const int n0 = b % gx * 32, m0 = b / gx % gy * 64, z = b / gx / gy, kt = g.Kd / 64;
  const float *X = static_cast<const float *>(g.X);
  const float *Wg = static_cast<const float *>(g.W[0]), *Wu = static_cast<const float *>(g.W[1]);
  const f32x16_t acc = tile_f32<false>(
      lds, int(int64_t(kt) * z / g.splits) * 64, int(int64_t(kt) * (z + 1) / g.splits) * 64,
      [&](int r, int k) { return *reinterpret_cast<const float4 *>(X + int64_t(min(m0 + r, g.M - 1)) * g.Kd + k); },
      [&](int r, int k) {
        return *reinterpret_cast<const float4 *>((r < 32 ? Wg : Wu) + int64_t(n0 + (r & 31)) * g.Kd + k);
      });
  float *out = (f32_col() < 32 ? g.sums[0] : g.sums[1]) + int64_t(z) * g.M * g.N + n0 + (f32_col() & 31);
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int row = m0 + f32_row(v);
    if (row < g.M) out[int64_t(row) * g.N] = acc[v];
  }
}

// ------------------------------------------------------------ backward
// d_gate and d_up, rounded to the layer's type: they are outputs, and lora_grad, the
// shrinks and dX's product all read them so, the MFMAs taking bf16 operands.  In dX
// each term then carries that half step too (bf16, 600 tokens: dX is 2.3e-3 of its norm
// from 64 bits, and 1.7e-3 with float32 ones, its own rounding).
template <typename E, int kAct>
__global__ __launch_bounds__(256) void gated_act_grad_kernel(const E *dH, const E *pg, const E *pu, E *dg, E *du,
                                                             int64_t n8) {
  const int64_t i = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
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
template <typename C, bool kWide>
struct GatedGradSrc {
  const uint16_t *a[2], *b[2];
  RowOffsets<C::A_INS, kWide> ao;
  uint32_t bo[C::B_INS];
  int wave, wm, wn, kt1;
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    const bool p = kt >= kt1;
    const int k = (p ? kt - kt1 : kt) * 64;
    if (i < C::A_INS) {
      ao.copy((p ? a[1] : a[0]) + k, i, lds + (wave * C::A_INS + i) * 1024);
    } else {
      lds_dma16_s((p ? b[1] : b[0]) + k, bo[i - C::A_INS],
                  lds + C::BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
    }
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    return frag_rows(base, s, q < C::TM ? (wm * C::TM + q) * 16 : C::BM + (wn * C::TN + q - C::TM) * 16);
  }
};

// Split z of kSplit takes a part of the K tiles and leaves float32 sums for
// terms_kernel; without kSplit dX itself, adapters' terms and all.
template <typename C, bool kSplit, bool kWide>
__global__ __launch_bounds__(C::NT, 1) void gated_grad_x_tile_kernel(GatedGradXArgs g) {
  constexpr int SC = 64 + 4;                            // a wave stages 16 rows, and those of the adapters' term
  constexpr int WLDS = 2 * 16 * SC * 4 + kTermLds;
  constexpr int TS = C::NW * WLDS;
  constexpr int NB = 2;                                 // blocks whose adapters' term is in registers
  static_assert(C::TN == 4 && C::TM % NB == 0, "64 columns per wave");
  constexpr int LDS = !kSplit && TS + TileLists<C>::SIZE > C::LDS ? TS + TileLists<C>::SIZE : C::LDS;
  static_assert(TS % 16 == 0 && LDS <= 156 * 1024, "staging must fit in LDS");
  __shared__ __attribute__((aligned(16))) char smem[LDS];
  __shared__ int rows[C::BM], cnt[C::NW];
  int tm, tn, z;
  if (!tile_of_workgroup(blockIdx.x, (g.M + C::BM - 1) / C::BM, (g.N + C::BN - 1) / C::BN, kSplit ? g.splits : 1, tm, tn,
                         z))
    return;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / C::WN, wn = wave % C::WN;
  const int nrows = tile_rows<C>(g.ex, g.slot_pos, rows, cnt, m0, g.M, kSplit);
  GatedGradSrc<C, kWide> src;
  src.wave = wave; src.wm = wm; src.wn = wn;
  const int kt = g.Kd / 64;
  // (scalar: the division is not, and the copies' bases have to be)
  const int kb = kSplit ? __builtin_amdgcn_readfirstlane(int(int64_t(2 * kt) * z / g.splits)) : 0;
  const int ke = kSplit ? __builtin_amdgcn_readfirstlane(int(int64_t(2 * kt) * (z + 1) / g.splits)) : 2 * kt;
  const int nk = ke - kb;
  src.kt1 = max(kt - kb, 0);                            // K tiles of the gate's product
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int k0 = p == 0 ? min(kb, kt - 1) : max(kb - kt, 0);
    src.a[p] = static_cast<const uint16_t *>(g.dY[p]) + k0 * 64;
    src.b[p] = static_cast<const uint16_t *>(g.W[p]) + int64_t(n0) * g.Kd + k0 * 64;
  }
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
    src.ao.set(i, int64_t(rows[min(row, nrows - 1)]) * g.Kd + fswz(row, lane & 7) * 8);
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = (wave * C::B_INS + i) * 8 + (lane >> 3);
    src.bo[i] = (uint32_t(min(row, g.N - 1 - n0)) * uint32_t(g.Kd) + fswz(row, lane & 7) * 8) * 2;
  }
  const int4 sd0 = kSplit ? make_int4(-1, 0, 0, 0) : row_desc(g.ex, rows, nrows, 0);
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, nk, acc);
  if constexpr (kSplit) {
    float *out = g.sums + int64_t(z) * g.M * g.N;
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j) {
        const int col = n0 + wn * C::TN * 16 + acc_col(j);
        if (col >= g.N) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = m0 + wm * C::TM * 16 + acc_row(i, v);
          if (row < g.M) out[int64_t(row) * g.N + col] = acc[i][j][v];
        }
      }
    return;
  }

  const Terms e{g.ex, g.U_up, g.b_up};
  TileSegs<C> &segs = *reinterpret_cast<TileSegs<C> *>(smem + TS);
  const bool lora_on = expand_enabled(g.ex);
  const int vr = lane >> 3, vc = (lane & 7) * 8, c0 = n0 + wn * 64;
  const bool inside = c0 < g.N;
  float *stage = reinterpret_cast<float *>(smem + wave * WLDS), *lstage = stage + 16 * SC;
  char *tlds = smem + wave * WLDS + 2 * 16 * SC * 4;
  TileTerms<C> &tt = *reinterpret_cast<TileTerms<C> *>(smem + TS);
  const bool common = lora_on && g.ex.K == 1 && tile_terms<C>(e, tt, sd0);
  TermCache<false> cache;
#pragma unroll
  for (int half = 0; half < C::TM / NB; ++half) {
    f32x4_t term[NB][4];
    unsigned dropped = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) term[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (lora_on && !common) {
      for (int k = 0; k < g.ex.K; ++k) {
        if (half == 0 || g.ex.K > 1) list_segs<C>(segs, k ? row_desc(g.ex, rows, nrows, k) : sd0);
        if (inside)
          dropped |= add_segs<false, C, NB>(e, segs, tlds, wm * C::TM + half * NB, c0, g.N, term);
      }
    }
    if (!inside) continue;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int r0 = (wm * C::TM + half * NB + i) * 16;
      if (common && add_tile_terms<false, C>(e, tt, tlds, r0, c0, g.N, term[i], cache)) dropped |= 1u << i;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          stage[acc_row(0, v) * SC + acc_col(j)] = acc[half * NB + i][j][v];
          lstage[acc_row(0, v) * SC + acc_col(j)] = term[i][j][v];
        }
      if ((dropped >> i) & 1) {
#pragma unroll 1
        for (int rr = 0; rr < 16 && r0 + rr < nrows; ++rr)
          lstage[rr * SC + lane] += terms_nonfinite(e, rows[r0 + rr], c0 + lane, 0) +
                                    terms_nonfinite(e, rows[r0 + rr], c0 + lane, 1);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int rr = q * 8 + vr;
        if (r0 + rr >= nrows) continue;
        float b[8], l[8];
        Elem<float>::load8(stage + rr * SC + vc, b);
        Elem<float>::load8(lstage + rr * SC + vc, l);
        const int64_t at = int64_t(rows[r0 + rr]) * g.N + c0 + vc;
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

// float32: the K range of split blockIdx.z, over both products.
__global__ __launch_bounds__(256) void gated_grad_x_f32_kernel(GatedGradXArgs g) {
  __shared__ F32Tile t;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, z = blockIdx.z, kt = 2 * (g.Kd / 64);
  const int kb = int(int64_t(kt) * z / g.splits) * 64, ke = int(int64_t(kt) * (z + 1) / g.splits) * 64;
  auto at = [&](const void *const (&m)[2], int row, int k) __attribute__((always_inline)) {
    const bool p = k >= g.Kd;
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p ? m[1] : m[0]) + int64_t(row) * g.Kd +
                                             (p ? k - g.Kd : k));
  };
  const f32x16_t acc = tile_f32<false>(
      t, kb, ke, [&](int r, int k) { return at(g.dY, min(m0 + r, g.M - 1), k); },
      [&](int r, int k) { return at(g.W, n0 + r, k); });
  float *out = g.sums + int64_t(z) * g.M * g.N;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int row = m0 + f32_row(v);
    if (row < g.M) out[int64_t(row) * g.N + n0 + f32_col()] = acc[v];
  }
}

template <typename E>
void launch_act_grad(const void *dH, const void *pg, const void *pu, int act, void *dg, void *du, int64_t n,
                     hipStream_t s) {
  // (a grid dimension holds less than 2^32 threads; a launch of more takes their number
  // modulo 2^32 and reports nothing)
  const int64_t n8 = n / 8, wgs = (n8 + 255) / 256, gx = wgs < (1 << 20) ? wgs : 1 << 20;
  const dim3 grid(unsigned(gx), unsigned((wgs + gx - 1) / gx)), block(256);
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

namespace {

template <bool kWide>
void launch_tiles(const GatedArgs &g, hipStream_t s) {
  const int tiles = int(tile_count(kBig, g.M, 2 * int64_t(g.N)));
  const dim3 grid(8 * unsigned((tiles + 7) / 8)), block(Big::NT);
  if (g.act == LORA_ACT_SILU)
    hipLaunchKernelGGL((gated_tile_kernel<Big, kWide, LORA_ACT_SILU>), grid, block, 0, s, g);
  else if (g.act == LORA_ACT_GELU)
    hipLaunchKernelGGL((gated_tile_kernel<Big, kWide, LORA_ACT_GELU>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((gated_tile_kernel<Big, kWide, LORA_ACT_GELU_TANH>), grid, block, 0, s, g);
}

template <typename C>
void launch_base(const GatedArgs &g, const PlanArgs &pa, int64_t tiles, hipStream_t s) {
  hipLaunchKernelGGL((gated_base_tile_kernel<C>), dim3(8 * unsigned((tiles + 7) / 8) + (pa.plan ? 1 : 0)), dim3(C::NT),
                     0, s, g, pa);
}

// Rows anywhere in [M][Kd]: 32-bit byte offsets reach them all, or not.
bool wide_rows(int64_t M, int64_t Kd) { return M * Kd >= (int64_t(1) << 31); }

}  // namespace

namespace {

template <typename E, bool kSum>
hipError_t run_terms(TermsArgs a, hipStream_t s) {
  constexpr int cols = kSum ? TermTile<E, false>::COLS : TermTile<E, true>::COLS / 2;
  const unsigned n_x = unsigned((a.N + cols - 1) / cols);
  const dim3 block(64);
  a.windows = int((int64_t(a.M) * a.K + 15) / 16);
  auto grid = [&](int rows) {
    return dim3(n_x, unsigned(rows < kWindowRows ? rows : kWindowRows), unsigned((rows + kWindowRows - 1) / kWindowRows));
  };
  if (a.slots[0]) {
    hipLaunchKernelGGL((terms_kernel<E, kSum, true>), grid(a.windows), block, 0, s, a);
    hipLaunchKernelGGL((terms_finish_kernel<E, kSum>), dim3(unsigned((int64_t(a.M) * a.N / 8 + 255) / 256)), dim3(256), 0,
                       s, a);
    return hipGetLastError();
  }
  for (a.k = 0; a.k < a.K; ++a.k)
    hipLaunchKernelGGL((terms_kernel<E, kSum, false>), grid(a.windows + (a.k == 0 ? (a.M + 15) / 16 : 0)), block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

// With one slot a launch, which finishes; with several and room for their terms
// two, that reads the pages once for all slots; else one for each slot
// (600 tokens of top 2, 5824 -> 2240: 26 us in two launches, 45 slot by slot; 333
// float32 tokens 16 and 21; with one slot, 700 tokens of 96 adapters, 60 and 49).
hipError_t launch_terms(const TermsArgs &a, bool sum, int dtype, hipStream_t s) {
  if (dtype == LORA_BF16) return sum ? run_terms<uint16_t, true>(a, s) : run_terms<uint16_t, false>(a, s);
  return sum ? run_terms<float, true>(a, s) : run_terms<float, false>(a, s);
}

bool gated_whole(int64_t M, int64_t Kd, int dtype, bool fused) { return dtype == LORA_BF16 && (fused || wide_rows(M, Kd)); }

hipError_t launch_gated(const GatedArgs &g, hipStream_t s) {
  if (wide_rows(g.M, g.Kd)) launch_tiles<true>(g, s);
  else launch_tiles<false>(g, s);
  return hipGetLastError();
}

// With at most `most` splits: 768 float32 workgroups, at least 4 K tiles of 64 each.
int gated_base_splits(int M, int N, int Kd, int dtype, int most) {
  if (dtype == LORA_BF16) return 1;
  const int64_t tiles = int64_t((M + 63) / 64) * (N / 32);
  int64_t n = 768 / tiles;
  if (n > Kd / 256) n = Kd / 256;
  if (n > most) n = most;
  return n < 1 ? 1 : int(n);
}

PlanLaunch gated_base_plan(const GatedArgs &g, int dtype, const int32_t *ids, const float *gates, int T, int K,
                           const PoolView &pool, int32_t *plan) {
  static const int nt[] = {Big::NT, Tall::NT, Mid::NT, Small::NT};
  static const size_t lds[] = {Big::LDS, Tall::LDS, Mid::LDS, Small::LDS};
  const int i = pick_shape(g.M, 2 * int64_t(g.N), 1);
  if (dtype == LORA_F32) return plan_setup(ids, gates, T, K, pool, plan, 256, sizeof(F32Tile));
  return plan_setup(ids, gates, T, K, pool, plan, nt[i], lds[i]);
}

hipError_t launch_gated_base(const GatedArgs &g, int dtype, const PlanArgs *plan, hipStream_t s) {
  PlanArgs pa{};
  if (plan) pa = *plan;
  if (dtype == LORA_F32) {
    const int64_t wgs = int64_t(g.N / 32) * ((g.M + 63) / 64) * g.splits + (plan ? 1 : 0);
    hipLaunchKernelGGL(gated_base_f32_kernel, dim3(unsigned(wgs)), dim3(256), 0, s, g, pa);
    return hipGetLastError();
  }
  const int i = pick_shape(g.M, 2 * int64_t(g.N), 1);
  const int64_t tiles = tile_count(i, g.M, 2 * int64_t(g.N));
  switch (i) {
    case kBig: launch_base<Big>(g, pa, tiles, s); break;
    case kTall: launch_base<Tall>(g, pa, tiles, s); break;
    case kMid: launch_base<Mid>(g, pa, tiles, s); break;
    default: launch_base<Small>(g, pa, tiles, s);
  }
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

hipError_t launch_gated_decode_epilogue(const GatedArgs &g, hipStream_t s) {
  const dim3 grid(unsigned((g.N + 511) / 512), unsigned(g.M)), block(256);
  if (g.act == LORA_ACT_SILU) hipLaunchKernelGGL(gated_decode_epilogue_kernel<LORA_ACT_SILU>, grid, block, 0, s, g);
  else if (g.act == LORA_ACT_GELU) hipLaunchKernelGGL(gated_decode_epilogue_kernel<LORA_ACT_GELU>, grid, block, 0, s, g);
  else hipLaunchKernelGGL(gated_decode_epilogue_kernel<LORA_ACT_GELU_TANH>, grid, block, 0, s, g);
  return hipGetLastError();
}

hipError_t launch_gated_act_grad(const void *dH, const void *pre_gate, const void *pre_up, int act, void *d_gate,
                                 void *d_up, int64_t n, int dtype, hipStream_t s) {
  if (dtype == LORA_BF16) launch_act_grad<uint16_t>(dH, pre_gate, pre_up, act, d_gate, d_up, n, s);
  else launch_act_grad<float>(dH, pre_gate, pre_up, act, d_gate, d_up, n, s);
  return hipGetLastError();
}

int gated_grad_x_splits(int T, int d_in, int d_out, int dtype) {
  const int64_t kt = 2 * int64_t(d_out / 64);
  int64_t tiles, want;
  if (dtype == LORA_BF16) {
    if (int64_t((T + 255) / 256) * ((d_in + 255) / 256) >= 192 || wide_rows(T, d_out)) return 0;
    // 128 x 256, one on a CU: a K tile takes 0.97 us, of 192 x 256 1.5 and of 256 x 256
    // 1.7, and smaller tiles divide the card better (600 tokens, 2240 wide: 41 us)
    tiles = int64_t((T + 127) / 128) * ((d_in + 255) / 256);
    want = 256;
  } else {
    tiles = int64_t((T + 63) / 64) * (d_in / 64);                  // several on a CU
    want = 512;
  }
  // at least 8 K tiles of 64 each
  int64_t s = want / (tiles > 0 ? tiles : 1);
  if (s > kt / 8) s = kt / 8;
  return s < 1 ? 1 : int(s);
}

hipError_t launch_gated_grad_x(const GatedGradXArgs &g, const TermsArgs &t, int dtype, hipStream_t s) {
  if (g.splits == 0) {
    const int tiles = ((g.M + 255) / 256) * ((g.N + 255) / 256);
    const dim3 grid(8 * unsigned((tiles + 7) / 8)), block(Big::NT);
    if (wide_rows(g.M, g.Kd)) hipLaunchKernelGGL((gated_grad_x_tile_kernel<Big, false, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((gated_grad_x_tile_kernel<Big, false, false>), grid, block, 0, s, g);
    return hipGetLastError();
  }
  if (dtype == LORA_F32) {
    hipLaunchKernelGGL(gated_grad_x_f32_kernel, dim3(unsigned(g.N / 64), unsigned((g.M + 63) / 64), unsigned(g.splits)),
                       dim3(256), 0, s, g);
  } else {
    const int tiles = ((g.M + 127) / 128) * ((g.N + 255) / 256);
    hipLaunchKernelGGL((gated_grad_x_tile_kernel<Mid, true, false>), dim3(8 * unsigned((tiles * g.splits + 7) / 8)),
                       dim3(Mid::NT), 0, s, g);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? launch_terms(t, true, dtype, s) : e;
}

}  // namespace lora
