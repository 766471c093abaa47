// Newton-Schulz orthogonalisation of adapter factors, and the optimiser step
// built on it.
//
// A factor is the r x d matrix N of one adapter's rank rows (its pages).  With
// X_0 = N / (|N|_F + eps) each step is X <- (a I + b G + c G^2) X, G = X X^T,
// which moves every singular value s to s (a + b s^2 + c s^4) and leaves the
// singular vectors.  All the polynomials are in the one matrix G_0 and
// commute, so with P_k = a I + b G_k + c G_k^2
//   G_{k+1} = P_k G_k P_k,   Q_{k+1} = P_k Q_k,   X_n = Q_n X_0:
// the steps run on r x r matrices alone, and N is read twice (once for G_0,
// once for the product with Q_n) instead of twice per step.
//
// G_0 squares the condition: a singular value of 1e-3 of the norm has the
// eigenvalue 1e-6, fp32 would know it to 6 %, and the steps amplify small
// values (3.44 each at the usual coefficients).  G and the r x r products
// therefore run in fp64 (v_mfma_f64_16x16x4_f64; products of fp32 inputs are
// exact there): against the steps in 64 bits the result is off by 1.3e-7 (four
// of rank 16) and 2.6e-7 (64 of ranks 8 .. 128) of its norm, where an fp32 Gram
// matrix gives 2e-5 .. 2e-4 and the steps themselves run in fp32 1.2e-6 and
// 4.6e-6.  Q N is fp32 (v_mfma_f32_16x16x4_f32).
//
// Launches: the Gram partials over column chunks (the optimiser step updates
// the momentum in the same pass); the steps, one workgroup per matrix of rank
// <= 64, all of it in LDS; the product with N (and the update of the pages).
// Ranks over 64 take the momentum and the r x r products in launches of their
// own, tiles of 32 x 32 over the GPU (14 for five steps).
#include "lora_internal.h"

namespace lora {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kSmall = 64;      // ranks whose steps run in one workgroup
constexpr int kBigMats = 5;     // r x r buffers of a matrix of rank over 64: G, P, Q and two spare

// The adapter of list entry m if it can be taken: in range, rank 1..max_rank,
// its page table consistent, and not listed before.  Called by every thread of
// a workgroup of 256; ends with the same answer in all of them.
__device__ __forceinline__ int orth_rank(const OrthArgs &a, int m, int *flag, int &adapter, int &ps) {
  adapter = a.adapters[m];
  ps = 0;
  if (adapter < 0 || adapter >= a.pool.n_adapters) return 0;
  const int r = a.pool.rank[adapter];
  ps = a.pool.page_start[adapter];
  if (r < 1 || r > a.max_rank || a.pool.page_start[adapter + 1] - ps != r || ps < 0 ||
      int64_t(ps) + r > a.pool.n_page_ids)
    return 0;
  __syncthreads();
  if (threadIdx.x == 0) *flag = 0;
  __syncthreads();
  bool bad = false;
  for (int j = threadIdx.x; j < m; j += 256) bad |= a.adapters[j] == adapter;
  for (int j = threadIdx.x; j < r; j += 256) {
    const int p = a.pool.page_ids[ps + j];
    bad |= p < 0 || p >= a.pool.n_pages;
  }
  if (bad) *flag = 1;
  __syncthreads();
  return *flag ? 0 : r;
}

// VC (4 or 8) columns of a row of the source, and (kStep) of the momentum,
// held raw until used, so that a step's loads are in flight under the step
// before.
template <bool kStep, int VC>
struct RawN {
  static constexpr int W = VC / 4;
  float4 g[W], m[kStep ? W : 1];
  __device__ __forceinline__ void load(const OrthFactor &f, int64_t at, bool on) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      g[w] = z;
      if constexpr (kStep) m[w] = z;
    }
    if (!on) return;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      g[w] = reinterpret_cast<const float4 *>(f.src + at)[w];
      if constexpr (kStep) m[w] = reinterpret_cast<const float4 *>(f.momentum + at)[w];
    }
  }
  // N from the gradient and the momentum (which kUpdate moves on first and
  // stores); else the source row
  template <bool kUpdate>
  __device__ __forceinline__ void value(const OrthFactor &f, const OrthArgs &a, int64_t at, bool on,
                                        float v[VC]) const {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float gv[4] = {g[w].x, g[w].y, g[w].z, g[w].w};
      if constexpr (!kStep) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * w + e] = gv[e];
      } else {
        float mv[4] = {m[w].x, m[w].y, m[w].z, m[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (kUpdate) mv[e] = a.mu * mv[e] + gv[e];
          v[4 * w + e] = a.nesterov ? gv[e] + a.mu * mv[e] : mv[e];
        }
        if (kUpdate && on)
          reinterpret_cast<float4 *>(f.momentum + at)[w] = make_float4(mv[0], mv[1], mv[2], mv[3]);
      }
    }
  }
};

// ------------------------------------------------------------ Gram partials
// Row blocks bi .. bi+NB-1 against bj .. bj+NB-1 (16 rows each, those past the
// rank left out) over columns [c0, c1).  A wave takes 32 columns of every 128,
// 4 VC at a time: lane l holds row l % 16 and VC columns of every block, one
// MFMA step per column of the VC (four columns each; the order of the sum over
// columns is free).  Pairs of different blocks take VC = 4: with 8 the second
// of two waves per SIMD would not fit the registers.  The four waves' sums are
// added in wave order through LDS.
template <int NB, bool kDiag, bool kStep, bool kUpdate>
__device__ __forceinline__ void gram_body(const OrthArgs &a, const OrthFactor &f, int r, int ps, int bi,
                                          int bj, int c0, int c1, double *out, double *red) {
  constexpr int NJ = kDiag ? 1 : NB, VC = kDiag ? 8 : 4, H = 8 / VC;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int nbj = min(NB, (r + 15) / 16 - bj);     // column blocks with rows of the matrix
  int64_t ri[NB], rj[NJ];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = (bi + i) * 16 + lr;
    ri[i] = row < r ? int64_t(a.pool.page_ids[ps + row]) * f.d + lg * VC : -1;
    if constexpr (!kDiag) {
      const int col = (bj + i) * 16 + lr;
      rj[i] = col < r ? int64_t(a.pool.page_ids[ps + col]) * f.d + lg * VC : -1;
    }
  }
  f64x4_t acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f64x4_t{0, 0, 0, 0};
  RawN<kStep, VC> x[NB], y[NJ];
  auto load = [&](int c) __attribute__((always_inline)) {
    const bool in = c < c1;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      x[i].load(f, ri[i] + c, in && ri[i] >= 0);
      if constexpr (!kDiag) y[i].load(f, rj[i] + c, in && rj[i] >= 0);
    }
  };
  // step s: columns of the wave's s-th group of 4 VC
  auto col_of = [&](int st) { return c0 + wave * 32 + (st / H) * 128 + (st % H) * (4 * VC); };
  load(col_of(0));
  for (int st = 0; col_of(st) < c1; ++st) {
    const int c = col_of(st);
    float xv[NB][VC], yv[NJ][VC];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      x[i].template value<kUpdate>(f, a, ri[i] + c, ri[i] >= 0, xv[i]);
      if constexpr (!kDiag) y[i].template value<false>(f, a, 0, false, yv[i]);
    }
    load(col_of(st + 1));
#pragma unroll
    for (int e = 0; e < VC; ++e) {
      double dx[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) dx[i] = double(xv[i][e]);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (NB > 1 && j >= nbj) break;
        const double dy = kDiag ? dx[j] : double(yv[kDiag ? 0 : j][e]);
#pragma unroll
        for (int i = 0; i < (kDiag ? j + 1 : NB); ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(dx[i], dy, acc[i][j], 0, 0, 0);
      }
    }
  }
  // acc element v of lane l: row 4 v + l / 16, column l % 16 of its block
  constexpr int S = 16 * NB;
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < (kDiag ? j + 1 : NB); ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            double *p = red + (i * 16 + 4 * v + lg) * S + j * 16 + lr;
            *p = w == 0 ? acc[i][j][v] : *p + acc[i][j][v];
          }
    }
    __syncthreads();
  }
  const int R = a.R;
  for (int e = threadIdx.x; e < S * S; e += 256) {
    // below the diagonal tiles: the mirror image, so that whole rows are read
    const int i = e / S, j = e % S;
    const int gi = bi * 16 + i, gj = bj * 16 + j;
    if (gi < R && gj < R) out[int64_t(gi) * R + gj] = red[kDiag && i / 16 > j / 16 ? j * S + i : e];
  }
}

// Grid: (column chunks x super-tiles, matrices).  Super-tiles are 64 x 64
// blocks (si <= sj) of the Gram matrix; ranks <= 64 have the first only.
// NBMAX: 16-row blocks of the largest rank, 8 for ranks over 64 (a launch of
// small ranks then keeps the registers, and the waves per SIMD, of its own).
template <bool kStep, int NBMAX>
__global__ __launch_bounds__(256, NBMAX <= 2 ? 4 : 2) void gram_kernel(OrthArgs a) {
  constexpr int S = 16 * (NBMAX < 4 ? NBMAX : 4);
  __shared__ double red[S * S];
  __shared__ int flag;
  const int m = blockIdx.y % a.M, fi = blockIdx.y / a.M;
  const OrthFactor &f = a.f[fi];
  int adapter, ps;
  const int r = orth_rank(a, m, &flag, adapter, ps);
  const int ck = blockIdx.x % a.chunks;
  int st = blockIdx.x / a.chunks;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.rec[blockIdx.y] = OrthRec{r, ps, 0.f, 1.f};
    if (fi == 0 && a.out_rank) a.out_rank[m] = r;
  }
  if (r == 0) return;
  const int c0 = int(int64_t(ck) * a.chunk_cols), c1 = min(f.d, c0 + a.chunk_cols);
  double *out = a.gram + (int64_t(blockIdx.y) * a.chunks + ck) * a.R * a.R;
  if (NBMAX == 1 || r <= 16) {
    if (st == 0) gram_body<1, true, kStep, kStep>(a, f, r, ps, 0, 0, c0, c1, out, red);
  } else if (NBMAX == 2 || r <= 32) {
    if constexpr (NBMAX >= 2)
      if (st == 0) gram_body<2, true, kStep, kStep>(a, f, r, ps, 0, 0, c0, c1, out, red);
  } else if (NBMAX == 4 || r <= kSmall) {
    if constexpr (NBMAX >= 4)
      if (st == 0) gram_body<4, true, kStep, kStep>(a, f, r, ps, 0, 0, c0, c1, out, red);
  } else if constexpr (NBMAX == 8) {
    // pair (si, sj), si <= sj, counted along columns sj
    int sj = 0;
    while (st > sj) { st -= sj + 1; ++sj; }
    if (sj * kSmall >= r) return;
    // the momentum of these ranks was moved on by its own launch
    if (st == sj) gram_body<4, true, kStep, false>(a, f, r, ps, st * 4, sj * 4, c0, c1, out, red);
    else gram_body<4, false, kStep, false>(a, f, r, ps, st * 4, sj * 4, c0, c1, out, red);
  }
}

// Momentum of the matrices of rank over 64 (their Gram super-tiles read a row
// several times, so it moves on in a launch of its own).  Grid: (columns,
// matrices, rows).
__global__ __launch_bounds__(256) void momentum_kernel(OrthArgs a) {
  __shared__ int flag;
  const int m = blockIdx.y % a.M;
  const OrthFactor &f = a.f[blockIdx.y / a.M];
  int adapter, ps;
  const int r = orth_rank(a, m, &flag, adapter, ps);
  if (r <= kSmall) return;
  const int col = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= f.d) return;
  for (int row = blockIdx.z; row < r; row += gridDim.z) {
    const int64_t at = int64_t(a.pool.page_ids[ps + row]) * f.d + col;
    RawN<true, 8> x;
    x.load(f, at, true);
    float v[8];
    x.value<true>(f, a, at, true, v);
  }
}

// ------------------------------------------------------------ the steps, rank <= 64
// inv from the trace of the summed Gram matrix: zero rows stay zero, a NaN or
// an infinity reaches every element.
__device__ __forceinline__ double norm_inv(double tr, float eps) {
  return tr == 0 ? 0.0 : 1.0 / (sqrt(tr) + double(eps));
}

// The factor of N in two parts: past 2^126 its reciprocal would be a subnormal
// float of few bits (16 x 8256 numbers up to 3e38 have a norm of 2^135: 4e-5).
__device__ __forceinline__ void store_inv(OrthRec &rec, double inv) {
  const bool far = inv > 0 && inv < 0x1p-64;
  rec.pre = far ? 0x1p-64f : 1.f;
  rec.inv = float(far ? inv * 0x1p64 : inv);
}

// Ranks <= 16: one 16 x 16 tile.  Element v of lane l of an MFMA result is row
// 4 v + l / 16, column l % 16; operand k of lane l is row l % 16, column 4 k +
// l / 16.  For a symmetric matrix these are the same value, so a result is the
// next product's operand as it stands: the steps are MFMAs of one wave and
// nothing else (a step: 1.2 -> 0.5 us; the launch of four rank-16 matrices,
// five steps with the sum of the partials before them: 5.8 .. 6.4 us).
__device__ __forceinline__ f64x4_t sym16(const f64x4_t &A, const f64x4_t &B) {
  f64x4_t c = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f64_16x16x4f64(A[k], B[k], c, 0, 0, 0);
  return c;
}

// All NW waves sum the chunks' partials (each its share, then in wave order);
// the first runs the steps.
template <int NW>
__device__ __forceinline__ void steps16(const OrthArgs &a, int mat, int r, double *lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, R = a.R;
  const int lr = lane & 15, lg = lane >> 4;
  const double *p = a.gram + int64_t(mat) * a.chunks * R * R;
  f64x4_t G = {0, 0, 0, 0};
  constexpr int CB = 6;                       // chunks whose loads are in flight together
  for (int c = wave; c < a.chunks; c += NW * CB) {
    double t[CB][4];
#pragma unroll
    for (int u = 0; u < CB; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        t[u][v] = p[int64_t(min(c + u * NW, a.chunks - 1)) * R * R + (4 * v + lg) * R + lr];
#pragma unroll
    for (int u = 0; u < CB; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) G[v] += c + u * NW < a.chunks ? t[u][v] : 0.0;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) lds[(wave * 4 + v) * 64 + lane] = G[v];
  __syncthreads();
  if (wave > 0) return;
  double tr = 0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int i = 4 * v + lg;
    double s = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += lds[(w * 4 + v) * 64 + lane];
    G[v] = i < r && lr < r ? s : 0.0;
    tr += i == lr ? G[v] : 0.0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  const double inv = norm_inv(tr, a.eps);
  if (lane == 0) store_inv(a.rec[mat], inv);
  f64x4_t Q, P;
#pragma unroll
  for (int v = 0; v < 4; ++v) G[v] *= inv * inv;
  for (int k = 0; k < a.steps; ++k) {
    const f64x4_t H = sym16(G, G);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      P[v] = (4 * v + lg == lr ? double(a.ca) : 0.0) + double(a.cb) * G[v] + double(a.cc) * H[v];
    if (k + 1 < a.steps) G = sym16(P, sym16(P, G));
    Q = k == 0 ? P : sym16(P, Q);
  }
  float *q = a.q + int64_t(mat) * R * R;
#pragma unroll
  for (int v = 0; v < 4; ++v) q[(4 * v + lg) * R + lr] = float(Q[v]);
}

// Larger: symmetric matrices of 16 NB rows in LDS, rows of S doubles (S = 16 NB
// + 2 puts the 16 rows x 2 columns that a half wave reads at once on distinct
// banks).  Both operands of a product are read along rows (they are
// symmetric); its upper tiles are taken by the waves in turn and stored with
// their mirror images.
template <int NB>
struct SymMat {
  static constexpr int n = 16 * NB, S = n + 2, SIZE = n * S, NT = NB * (NB + 1) / 2;
};

// CT tiles (ti, tj) of C = A . B; store(i, j, value, tile off the diagonal).
template <int NB, int CT, typename Store>
__device__ __forceinline__ void sym_tiles(const double *A, const double *B, const int (&ti)[CT],
                                          const int (&tj)[CT], const Store &store) {
  constexpr int S = SymMat<NB>::S;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const double *pa[CT], *pb[CT];
  f64x4_t acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    pa[c] = A + (ti[c] * 16 + lr) * S + lg;
    pb[c] = B + (tj[c] * 16 + lr) * S + lg;
    acc[c] = f64x4_t{0, 0, 0, 0};
  }
  // unrolled whole: in a loop the compiler moves every accumulator between the
  // two register files each time round, behind a drained pipe
#pragma unroll
  for (int k = 0; k < 4 * NB; ++k)
#pragma unroll
    for (int c = 0; c < CT; ++c)
      acc[c] = __builtin_amdgcn_mfma_f64_16x16x4f64(pa[c][4 * k], pb[c][4 * k], acc[c], 0, 0, 0);
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      store(ti[c] * 16 + 4 * v + lg, tj[c] * 16 + lr, acc[c][v], ti[c] != tj[c]);
}

// This wave's tiles w, w + NW, .. of a product (at most 2), without idle MFMAs
// for the waves that have fewer.
template <int NB, int NW>
struct MyTiles {
  int n, ti[2], tj[2];
  __device__ __forceinline__ MyTiles() {
    constexpr int NT = SymMat<NB>::NT;
    static_assert(NT <= 2 * NW, "at most two tiles a wave");
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    n = w >= NT ? 0 : (NT - 1 - w) / NW + 1;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      int t = min(w + c * NW, NT - 1), j = 0;
      while (t > j) { t -= j + 1; ++j; }
      ti[c] = t; tj[c] = j;
    }
  }
  template <typename Store>
  __device__ __forceinline__ void product(const double *A, const double *B, const Store &store) const {
    if (n == 2) {
      sym_tiles<NB, 2>(A, B, ti, tj, store);
    } else if (n == 1) {
      const int i1[1] = {ti[0]}, j1[1] = {tj[0]};
      sym_tiles<NB, 1>(A, B, i1, j1, store);
    }
  }
};

template <int NB, int NW>
__device__ __forceinline__ void steps_body(const OrthArgs &a, int mat, int r, double *lds) {
  using M = SymMat<NB>;
  constexpr int n = M::n, S = M::S, NTH = NW * 64;
  double *G = lds, *P = G + M::SIZE, *Q = P + M::SIZE, *T = Q + M::SIZE;
  const int tid = threadIdx.x, R = a.R;
  const MyTiles<NB, NW> mine;
  // the chunks' partials in order, the loads of all of a thread's elements
  // (and of several chunks) in flight together
  {
    constexpr int EP = n * n / NTH, CB = 16 / EP;
    const double *p[EP];
    double sum[EP];
#pragma unroll
    for (int q = 0; q < EP; ++q) {
      const int i = (tid + q * NTH) / n, j = (tid + q * NTH) % n;
      p[q] = a.gram + int64_t(mat) * a.chunks * R * R + int64_t(min(i, R - 1)) * R + min(j, R - 1);
      sum[q] = 0;
    }
    for (int c = 0; c < a.chunks; c += CB) {
      double t[CB][EP];
#pragma unroll
      for (int u = 0; u < CB; ++u)
#pragma unroll
        for (int q = 0; q < EP; ++q) t[u][q] = p[q][int64_t(min(c + u, a.chunks - 1)) * R * R];
#pragma unroll
      for (int u = 0; u < CB; ++u)
#pragma unroll
        for (int q = 0; q < EP; ++q) sum[q] += c + u < a.chunks ? t[u][q] : 0.0;
    }
#pragma unroll
    for (int q = 0; q < EP; ++q) {
      const int i = (tid + q * NTH) / n, j = (tid + q * NTH) % n;
      G[i * S + j] = i < r && j < r ? sum[q] : 0.0;
    }
  }
  __syncthreads();
  // the trace, the same in every wave
  double tr = (tid & 63) < n ? G[(tid & 63) * (S + 1)] : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  const double inv = norm_inv(tr, a.eps);
  if (tid == 0) store_inv(a.rec[mat], inv);
  __syncthreads();
  for (int e = tid; e < n * n; e += NTH) G[(e / n) * S + e % n] *= inv * inv;
  __syncthreads();
  const double ca = a.ca, cb = a.cb, cc = a.cc;
  auto put = [](double *D, int i, int j, double v, bool off) {
    D[i * S + j] = v;
    if (off) D[j * S + i] = v;
  };
  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    double *const F = k == 0 ? Q : P;       // the first factor is Q itself
    mine.product(G, G, [&](int i, int j, double v, bool off) {
      put(F, i, j, (i == j ? ca : 0.0) + cb * G[i * S + j] + cc * v, off);
    });
    __syncthreads();
    if (!last) {
      mine.product(F, G, [&](int i, int j, double v, bool off) { put(T, i, j, v, off); });
      __syncthreads();
      mine.product(F, T, [&](int i, int j, double v, bool off) { put(G, i, j, v, off); });
      __syncthreads();
    }
    if (k > 0) {
      // Q <- P Q by way of T (free again after the barrier)
      mine.product(P, Q, [&](int i, int j, double v, bool off) { put(T, i, j, v, off); });
      __syncthreads();
      double *const t = Q; Q = T; T = t;
    }
  }
  float *q = a.q + int64_t(mat) * R * R;
  for (int e = tid; e < n * n; e += NTH) {
    const int i = e / n, j = e % n;
    if (i < R && j < R) q[int64_t(i) * R + j] = float(Q[i * S + j]);
  }
}

// NBMAX: 16-row blocks of the largest rank (4: all that fit a workgroup).
template <int NBMAX>
__global__ __launch_bounds__(512) void steps_kernel(OrthArgs a) {
  __shared__ double steps_lds[NBMAX == 1 ? 8 * 256 : 4 * SymMat<NBMAX>::SIZE];
  const int mat = blockIdx.x, r = a.rec[mat].rank;
  if (r < 1 || r > kSmall) return;
  if (NBMAX == 1 || r <= 16) {
    steps16<8>(a, mat, r, steps_lds);
  } else if (NBMAX == 2 || r <= 32) {
    if constexpr (NBMAX >= 2) steps_body<2, 8>(a, mat, r, steps_lds);
  } else {
    if constexpr (NBMAX >= 4) steps_body<4, 8>(a, mat, r, steps_lds);
  }
}

// ------------------------------------------------------------ ranks over 64
// Sum of the chunks' partials, normalised.  Grid: (16-row strips of the 64 x 64
// blocks (si <= sj), matrices); blocks off the diagonal are stored with their
// mirror images.  Every workgroup takes the trace itself.
__global__ __launch_bounds__(256) void gram_sum_kernel(OrthArgs a) {
  const int mat = blockIdx.y, r = a.rec[mat].rank, R = a.R;
  if (r <= kSmall) return;
  __shared__ double part[256], turn[16][65];
  int si = blockIdx.x >> 2, sj = 0;
  while (si > sj) { si -= sj + 1; ++sj; }
  const int64_t n = int64_t(R) * R;
  const double *p = a.gram + int64_t(mat) * a.chunks * n;
  const int tid = threadIdx.x, i0 = si * kSmall + (blockIdx.x & 3) * 16, j = sj * kSmall + (tid & 63);
  if (i0 >= R) return;
  double t = 0, sum[4] = {0, 0, 0, 0};
  int64_t at[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) at[q] = int64_t(min(i0 + (tid >> 6) + 4 * q, R - 1)) * R + min(j, R - 1);
  // eight chunks' loads in flight, added in order
  for (int c = 0; c < a.chunks; c += 8) {
    double v[8][4], d[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const double *pc = p + int64_t(min(c + u, a.chunks - 1)) * n;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[u][q] = pc[at[q]];
      d[u] = pc[int64_t(min(tid, r - 1)) * (R + 1)];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = c + u < a.chunks;
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[q] += in ? v[u][q] : 0.0;
      t += in && tid < r ? d[u] : 0.0;
    }
  }
  for (int i = tid + 256; i < r; i += 256)
    for (int c = 0; c < a.chunks; ++c) t += p[int64_t(c) * n + int64_t(i) * (R + 1)];
  part[tid] = t;
  __syncthreads();
  // a fixed tree: the same trace in every workgroup
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) part[tid] += part[tid + o];
    __syncthreads();
  }
  const double inv = norm_inv(part[0], a.eps);
  if (blockIdx.x == 0 && tid == 0) store_inv(a.rec[mat], inv);
  double *G = a.big + int64_t(mat) * kBigMats * n;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int y = (tid >> 6) + 4 * q, i = i0 + y;
    // past the rank the partials were never written
    const double v = i < r && j < r ? sum[q] * (inv * inv) : 0.0;
    if (i < R && j < R) G[int64_t(i) * R + j] = v;
    turn[y][tid & 63] = v;
  }
  if (si == sj) return;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int x = (tid >> 4) + 16 * q, i = sj * kSmall + x, c = i0 + (tid & 15);
    if (i < R && c < R) G[int64_t(i) * R + c] = turn[tid & 15][x];
  }
}

// Products of symmetric R x R matrices of every matrix of rank over 64: upper
// tiles of 32 x 32 (one 16 x 16 block per wave), stored with their mirror
// images.  Both operands are read along rows, 64 columns at a time through LDS
// (coalesced; the next 64 in flight under the MFMAs; rows of 66 doubles as in
// sym_tiles).  Grid: (tiles, matrices, products).
struct SymOp {
  int A, B, C;            // buffers: C = A . B
  int poly;               // C = ca I + cb A + cc A . B
  int copy;               // also into this buffer (-1: none)
  int to_q;               // also, in fp32, into q
};

__global__ __launch_bounds__(256, 2) void sym_product_kernel(OrthArgs a, SymOp op0, SymOp op1) {
  constexpr int KB = 64, S = KB + 2;
  __shared__ double la[32 * S], lb[32 * S];
  const int mat = blockIdx.y, r = a.rec[mat].rank, R = a.R;
  if (r <= kSmall) return;
  const SymOp op = blockIdx.z == 0 ? op0 : op1;
  int t = blockIdx.x, tj = 0;
  while (t > tj) { t -= tj + 1; ++tj; }
  if (tj * 32 >= r) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  double *base = a.big + int64_t(mat) * kBigMats * R * R;
  const double *A = base + int64_t(op.A) * R * R, *B = base + int64_t(op.B) * R * R;
  // thread: row tid / 8 of both tiles, 8 columns of each 64
  const int row = tid >> 3, cc = (tid & 7) * 8;
  const double *ga = A + int64_t(min(t * 32 + row, R - 1)) * R, *gb = B + int64_t(min(tj * 32 + row, R - 1)) * R;
  const int n = (r + 15) / 16 * 16;
  double2 va[4], vb[4];
  auto load = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = min(k0 + cc + 2 * e, R - 2);     // past n: not used
      va[e] = *reinterpret_cast<const double2 *>(ga + c);
      vb[e] = *reinterpret_cast<const double2 *>(gb + c);
    }
  };
  load(0);
  const int i0 = t * 32 + (wave >> 1) * 16, j0 = tj * 32 + (wave & 1) * 16;
  double lin[4];                                     // the linear term's elements
#pragma unroll
  for (int v = 0; v < 4; ++v)
    lin[v] = op.poly ? A[int64_t(min(i0 + 4 * v + lg, R - 1)) * R + min(j0 + lr, R - 1)] : 0.0;
  f64x4_t acc = {0, 0, 0, 0};
  const double *pa = la + ((wave >> 1) * 16 + lr) * S + lg, *pb = lb + ((wave & 1) * 16 + lr) * S + lg;
  for (int k0 = 0; k0 < n; k0 += KB) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      la[row * S + cc + 2 * e] = va[e].x; la[row * S + cc + 2 * e + 1] = va[e].y;
      lb[row * S + cc + 2 * e] = vb[e].x; lb[row * S + cc + 2 * e + 1] = vb[e].y;
    }
    __syncthreads();
    if (k0 + KB < n) load(k0 + KB);
    const int kn = min(KB, n - k0);
    for (int k = 0; k < kn; k += 16)
#pragma unroll
      for (int u = 0; u < 16; u += 4)
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64(pa[k + u], pb[k + u], acc, 0, 0, 0);
    __syncthreads();
  }
  // the tile through LDS (rows of 33), so that it and its mirror image are
  // stored along rows
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int i = i0 + 4 * v + lg, j = j0 + lr;
    double x = acc[v];
    if (op.poly) x = (i == j ? double(a.ca) : 0.0) + double(a.cb) * lin[v] + double(a.cc) * x;
    la[((wave >> 1) * 16 + 4 * v + lg) * 33 + (wave & 1) * 16 + lr] = x;
  }
  __syncthreads();
  double *C = base + int64_t(op.C) * R * R;
  double *D = op.copy >= 0 ? base + int64_t(op.copy) * R * R : nullptr;
  float *q = a.q + int64_t(mat) * R * R;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    // u < 4: rows of the tile; u >= 4: rows of its mirror image
    const int e = (u & 3) * 256 + tid, y = e >> 5, x = e & 31;
    const bool mir = u >= 4;
    if (mir && t == tj) break;
    const int i = (mir ? tj : t) * 32 + y, j = (mir ? t : tj) * 32 + x;
    if (i >= R || j >= R) continue;
    const double val = mir ? la[x * 33 + y] : la[y * 33 + x];
    const int64_t at = int64_t(i) * R + j;
    C[at] = val;
    if (D) D[at] = val;
    if (op.to_q) q[at] = float(val);
  }
}

// ------------------------------------------------------------ the product with N
// Rows 16 ib .. of O = Q (N inv) for `chunks` runs of 256 columns: a wave takes
// 64 columns of a run, lane l the four columns 4 (l % 16) .. +3 of row l / 16
// of every four, so a load is 256 contiguous bytes per row; column tile e
// holds columns 4 c + e, and the four tiles' results are four consecutive
// columns again.  The rows come U groups of four at a time, the next groups
// (of the same run or the next) in flight under the MFMAs of these.  Q's
// columns and the rows' pages go through LDS, 128 of them at a time (up to
// rank 128 once for all the runs).
constexpr int kApplyRows = 128, kApplyQ = kApplyRows + 4;

template <int NB, bool kStep, typename E>
__device__ __forceinline__ void apply_body(const OrthArgs &a, const OrthFactor &f, const OrthRec &rc,
                                           int ib, const float *q, int col0, int chunks, float *lq, int *lp) {
  constexpr int U = 4;
  const int r = rc.rank, ps = rc.page_start;
  const float pre = rc.pre, inv = rc.inv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int R = a.R;
  auto column = [&](int ck) { return min(col0 + ck * 256 + wave * 64, f.d - 64) + lr * 4; };
  struct Rows {
    float4 x[U], m[kStep ? U : 1];
  };
  // groups k0 .. of the staged rows, columns of run ck; rows past the staged
  // ones repeat the last (they are cleared before use)
  auto load = [&](Rows &w, int ck, int k0, int n16) __attribute__((always_inline)) {
    const int col = column(ck);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = int64_t(lp[min(k0 + 4 * u + lg, n16 - 1)]) * f.d + col;
      w.x[u] = *reinterpret_cast<const float4 *>(f.src + at);
      if constexpr (kStep) w.m[u] = *reinterpret_cast<const float4 *>(f.momentum + at);
    }
  };
  f32x4_t acc[NB][4];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = f32x4_t{0, 0, 0, 0};
  };
  auto add = [&](const Rows &w, int k0, int nr, int n16) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 4 * u >= n16) break;
      const int k = k0 + 4 * u + lg;
      float4 v = w.x[u];
      if constexpr (kStep) {
        const float4 t = w.m[u];
        if (a.nesterov)
          v = make_float4(v.x + a.mu * t.x, v.y + a.mu * t.y, v.z + a.mu * t.z, v.w + a.mu * t.w);
        else
          v = t;
      }
      if (k >= nr) v = make_float4(0.f, 0.f, 0.f, 0.f);
      const float b[4] = {v.x * pre * inv, v.y * pre * inv, v.z * pre * inv, v.w * pre * inv};
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const float av = lq[(i * 16 + lr) * kApplyQ + k];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(av, b[e], acc[i][e], 0, 0, 0);
      }
    }
  };
  auto pages = [&](int r0, int nr, int n16) __attribute__((always_inline)) {
    if (tid < n16) lp[tid] = a.pool.page_ids[ps + r0 + min(tid, nr - 1)];
  };
  auto stage_q = [&](int r0, int nr, int n16) __attribute__((always_inline)) {
    for (int i = wave; i < NB * 16; i += 4) {
      const int qi = ib * 16 + i;
      for (int k = lane; k < n16; k += 64)
        lq[i * kApplyQ + k] = k < nr && qi < R ? q[int64_t(qi) * R + r0 + k] : 0.f;
    }
  };
  // acc element v of lane l: row 4 (l / 16) + v, column l % 16 of its tile
  auto store = [&](int ck) __attribute__((always_inline)) {
    if (col0 + ck * 256 + wave * 64 >= f.d) return;
    const int col = column(ck);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      // one row block at a time: its weights' registers are free for the next
      __builtin_amdgcn_sched_barrier(0);
      int64_t at[4];
      float4 mw[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = min((ib + i) * 16 + lg * 4 + v, r - 1);
        at[v] = int64_t(r <= kApplyRows ? lp[row] : a.pool.page_ids[ps + row]) * f.d + col;
        if constexpr (kStep) {
          if (f.master) {
            mw[v] = *reinterpret_cast<const float4 *>(f.master + at[v]);
          } else {
            const E *pg = static_cast<const E *>(f.pages) + at[v];
            mw[v] = make_float4(Elem<E>::load1(pg), Elem<E>::load1(pg + 1), Elem<E>::load1(pg + 2),
                                Elem<E>::load1(pg + 3));
          }
        }
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if ((ib + i) * 16 + lg * 4 + v >= r) continue;
        const float o[4] = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
        if constexpr (!kStep) {
          *reinterpret_cast<float4 *>(f.out + at[v]) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
          float w[4] = {mw[v].x, mw[v].y, mw[v].z, mw[v].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = w[e] * f.keep - f.lr * o[e];
          if (f.master) *reinterpret_cast<float4 *>(f.master + at[v]) = make_float4(w[0], w[1], w[2], w[3]);
          E *pg = static_cast<E *>(f.pages) + at[v];
          if constexpr (sizeof(E) == 2)
            *reinterpret_cast<uint2 *>(pg) = make_uint2(f2bf2(w[0], w[1]), f2bf2(w[2], w[3]));
          else
            *reinterpret_cast<float4 *>(pg) = make_float4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  };
  Rows w0;
  if (r <= kApplyRows) {
    const int n16 = (r + 15) / 16 * 16;
    pages(0, r, n16);
    __syncthreads();
    stage_q(0, r, n16);
    __syncthreads();
    for (int ck = 0; ck < chunks; ++ck) {
      clear();
      for (int k0 = 0; k0 < n16; k0 += 4 * U) {
        load(w0, ck, k0, n16);
        add(w0, k0, r, n16);
      }
      store(ck);
    }
    return;
  }
  for (int ck = 0; ck < chunks; ++ck) {
    clear();
    for (int r0 = 0; r0 < r; r0 += kApplyRows) {
      const int nr = min(kApplyRows, r - r0), n16 = (nr + 15) / 16 * 16;
      __syncthreads();                         // the last rows and Q are done with
      pages(r0, nr, n16);
      __syncthreads();
      stage_q(r0, nr, n16);
      __syncthreads();
      for (int k0 = 0; k0 < n16; k0 += 4 * U) {
        load(w0, ck, k0, n16);
        add(w0, k0, nr, n16);
      }
    }
    store(ck);
  }
}

// Grid: (runs of a.apply_chunks x 256 columns, matrices, row blocks of 64).
template <bool kStep, typename E>
__global__ __launch_bounds__(256, 4) void orth_apply_kernel(OrthArgs a) {
  __shared__ float lq[kSmall * kApplyQ];
  __shared__ int lp[kApplyRows];
  const OrthRec rc = a.rec[blockIdx.y];
  const OrthFactor &f = a.f[blockIdx.y / a.M];
  const int ib = blockIdx.z * 4;
  const int col0 = blockIdx.x * a.apply_chunks * 256;
  if (rc.rank <= ib * 16 || col0 >= f.d) return;
  const int chunks = min(a.apply_chunks, (f.d - col0 + 255) / 256);
  const float *q = a.q + int64_t(blockIdx.y) * a.R * a.R;
  const int left = rc.rank - ib * 16;         // output rows from ib * 16
  if (left <= 16) apply_body<1, kStep, E>(a, f, rc, ib, q, col0, chunks, lq, lp);
  else if (left <= 32) apply_body<2, kStep, E>(a, f, rc, ib, q, col0, chunks, lq, lp);
  else apply_body<4, kStep, E>(a, f, rc, ib, q, col0, chunks, lq, lp);
}

int orth_r(int max_rank) { return (max_rank + 15) / 16 * 16; }

// Column chunks of the Gram launch: about four workgroups per CU, at least 256
// columns each (two steps of each wave); twelve where ranks go over 64, whose
// pairs of blocks take unlike times.
int orth_chunk_cols(int64_t mats, int max_rank, int d) {
  const int s = (max_rank + kSmall - 1) / kSmall;
  const int64_t per = mats * (s * (s + 1) / 2);
  const int64_t want = ((max_rank > kSmall ? 12 : 4) * 256 + per - 1) / per;
  int64_t cols = (d + want - 1) / want;
  cols = (cols + 127) / 128 * 128;
  return int(cols < 256 ? 256 : cols);
}

int orth_chunks(int64_t mats, int max_rank, int d) {
  const int c = orth_chunk_cols(mats, max_rank, d);
  return (d + c - 1) / c;
}

size_t pad256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Workspace: records, Q (fp32), Gram partials, and for ranks over 64 the r x r
// matrices.
size_t orth_workspace_bytes(int M, int factors, int max_rank, int d) {
  const int64_t mats = int64_t(M) * factors;
  const size_t RR = size_t(orth_r(max_rank)) * orth_r(max_rank);
  size_t b = pad256(size_t(mats) * sizeof(OrthRec)) + pad256(size_t(mats) * RR * 4) +
             pad256(size_t(mats) * orth_chunks(mats, max_rank, d) * RR * 8);
  if (max_rank > kSmall) b += pad256(size_t(mats) * kBigMats * RR * 8);
  return b;
}

hipError_t launch_orthogonal(OrthArgs a, int factors, bool step, int dtype, void *ws, hipStream_t s) {
  const int64_t mats = int64_t(a.M) * factors;
  int d = a.f[0].d;
  if (factors > 1 && a.f[1].d > d) d = a.f[1].d;
  a.R = orth_r(a.max_rank);
  a.chunk_cols = orth_chunk_cols(mats, a.max_rank, d);
  a.chunks = orth_chunks(mats, a.max_rank, d);
  const size_t RR = size_t(a.R) * a.R;
  char *p = static_cast<char *>(ws);
  a.rec = reinterpret_cast<OrthRec *>(p);
  p += pad256(size_t(mats) * sizeof(OrthRec));
  a.q = reinterpret_cast<float *>(p);
  p += pad256(size_t(mats) * RR * 4);
  a.gram = reinterpret_cast<double *>(p);
  p += pad256(size_t(mats) * a.chunks * RR * 8);
  a.big = reinterpret_cast<double *>(p);
  const bool big = a.max_rank > kSmall;
  const int st = (a.max_rank + kSmall - 1) / kSmall;
  if (big && step) {
    const int rows = a.max_rank < 128 ? a.max_rank : 128;
    hipLaunchKernelGGL(momentum_kernel, dim3(unsigned((d / 8 + 255) / 256), unsigned(mats), unsigned(rows)),
                       dim3(256), 0, s, a);
  }
  const dim3 gg(unsigned(a.chunks * (st * (st + 1) / 2)), unsigned(mats));
#define LORA_GRAM(NB) \
  do { \
    if (step) hipLaunchKernelGGL((gram_kernel<true, NB>), gg, dim3(256), 0, s, a); \
    else hipLaunchKernelGGL((gram_kernel<false, NB>), gg, dim3(256), 0, s, a); \
  } while (0)
  if (a.max_rank <= 16) LORA_GRAM(1);
  else if (a.max_rank <= 32) LORA_GRAM(2);
  else if (!big) LORA_GRAM(4);
  else LORA_GRAM(8);
#undef LORA_GRAM
  if (a.max_rank <= 16) hipLaunchKernelGGL(steps_kernel<1>, dim3(unsigned(mats)), dim3(512), 0, s, a);
  else if (a.max_rank <= 32) hipLaunchKernelGGL(steps_kernel<2>, dim3(unsigned(mats)), dim3(512), 0, s, a);
  else hipLaunchKernelGGL(steps_kernel<4>, dim3(unsigned(mats)), dim3(512), 0, s, a);
  if (big) {
    hipLaunchKernelGGL(gram_sum_kernel, dim3(unsigned(4 * (st * (st + 1) / 2)), unsigned(mats)), dim3(256), 0, s, a);
    const int t32 = (a.R + 31) / 32;
    const unsigned tiles = unsigned(t32 * (t32 + 1) / 2);
    auto products = [&](const SymOp &x, const SymOp &y, unsigned n) {
      hipLaunchKernelGGL(sym_product_kernel, dim3(tiles, unsigned(mats), n), dim3(256), 0, s, a, x, y);
    };
    int Q = 2, Qn = 3;                         // buffers 0 G, 1 P, 4 P G
    for (int k = 0; k < a.steps; ++k) {
      const bool last = k + 1 == a.steps;
      // P (the first step's is Q too)
      const SymOp poly{0, 0, 1, 1, k == 0 ? Q : -1, last && k == 0};
      products(poly, poly, 1);
      // P G and the next Q in one launch, then G <- P (P G)
      const SymOp pg{1, 0, 4, 0, -1, 0}, pq{1, Q, Qn, 0, -1, last}, ppg{1, 4, 0, 0, -1, 0};
      if (!last && k > 0) products(pg, pq, 2);
      else if (!last) products(pg, pg, 1);
      else if (k > 0) products(pq, pq, 1);
      if (k > 0) { const int t = Q; Q = Qn; Qn = t; }
      if (!last) products(ppg, ppg, 1);
    }
  }
  // about 8192 workgroups: enough to even out unlike ranks, few enough that Q
  // is staged for several runs of columns where matrices are many
  const int64_t runs = (d + 255) / 256, all = runs * mats * st;
  a.apply_chunks = int(all / 8192 < 1 ? 1 : all / 8192 > runs ? runs : all / 8192);
  const dim3 ga(unsigned((runs + a.apply_chunks - 1) / a.apply_chunks), unsigned(mats), unsigned(st));
  if (!step) hipLaunchKernelGGL((orth_apply_kernel<false, float>), ga, dim3(256), 0, s, a);
  else if (dtype == LORA_BF16) hipLaunchKernelGGL((orth_apply_kernel<true, uint16_t>), ga, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((orth_apply_kernel<true, float>), ga, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace lora
