// Softmax cross entropy of a large vocabulary, with the gradient of the hidden
// states, without the logits.
//
//   l_v = scale . X_t.W_v,   loss_t = w_t (log sum_v e^{l_v} - l_y)
//   dX_t = w_t scale (sum_v p_v W_v - W_y),   p = softmax(l)
//
// In base 2, L = l log2 e, with a whole number ref near the target's L_y:
//   e_v = 2^{L_v - ref},  S = sum over v != y of e_v,  q = S / e_y
//   loss = w ln(1 + q),   dX = w scale / (S + e_y) . (sum over v != y of e_v W_v - S W_y)
// The target's term stands apart: where p_y is near 1, both results come from
// S alone and keep their relative precision.  A row's largest L is at least
// L_y, so that nothing that counts underflows against ref; a 64-column piece
// of a row whose largest L - ref is over 64 takes a further shift of its own
// (a whole number, so that putting the pieces on one shift later is exact).
//
// So the products run once each: the first launch of a block of tokens leaves
// e in bf16 (float32 layers: float32), with no common reference to wait for, and
// the sums of each piece; a small one makes S, the loss and the two coefficients
// of each row; the second product is e.W, split along the vocabulary.  bf16 is what
// its MFMAs take: each e is off by 2^-8 of itself at most and S is not, so that
// dX is off by 2^-8 |w scale| sum over v != y of p_v |W_v| beside its own
// rounding, as much where W_y and the likely rows are alike and the two sums
// nearly cancel.  Memory is bounded by taking the tokens in blocks (kBlockBytes of
// e, and of the float32 sums of dX).  Tokens without a target are left out before
// the first product, by a list of the others.
#include <algorithm>

#include "tile_f32.h"
#include "tile_loop.h"

namespace lora {
namespace {

constexpr int kSub = 64;                               // columns of one piece of a row
constexpr size_t kBlockBytes = size_t(512) << 20;      // e, and the sums of dX, of one block of tokens
constexpr int kMaxSplits = 64;                         // whose sums one thread adds up
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMaxExp = 64.f;                        // a piece's exponents over this are shifted

struct CeWs {
  int32_t *count;      // [1] tokens with a target
  int32_t *rows;       // [T] those tokens, ascending
  double *ly;          // [T] the tokens' target's logit in base 2
  float2 *coef;        // [T] (w scale / Z, -w scale S / Z)
  float2 *part;        // [block][pieces] (sum, shift)
  void *e;             // [block][lde]
  float *acc;          // [splits][block][d]
  int block, pieces, splits;
  int shape;           // of the second product's tiles (bf16)
  int64_t lde;
  size_t bytes;
};

struct CeArgs {
  CrossEntropyArgs a;
  CeWs w;
  int row0;            // first row (of the list) of this block
};

__device__ __forceinline__ int block_rows(const CeArgs &c) { return min(c.w.block, c.w.count[0] - c.row0); }

// ref of a row, from its target's logit
__device__ __forceinline__ float ref_of(double ly) {
  const float r = float(rint(ly));
  return r - r == 0.f ? r : 0.f;
}

// ------------------------------------------------------------ rows
__device__ __forceinline__ bool ce_listed(const CeArgs &c, int t) {
  const int y = c.a.targets[t];
  return y >= 0 && y < c.a.V && !(c.a.weights && c.a.weights[t] == 0.f);
}

// Workgroup 0: the list of tokens that have a target and a weight.  Beside it,
// four waves per token: the target's logit of a listed one (float64 sums: both
// results hang on it), the zero loss and gradient of another.  (As launches one
// after the other 48 us at 8192 tokens, as one 29; at 1024 tokens 6.6, 10 with a
// wave per token.)
template <typename E>
__global__ __launch_bounds__(1024) void ce_rows_kernel(CeArgs c) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, T = c.a.T;
  if (blockIdx.x == 0) {
    __shared__ int sums[16];
    const int per = (T + 1023) / 1024, t0 = min(tid * per, T), t1 = min(t0 + per, T);
    int n = 0;
    for (int t = t0; t < t1; ++t) n += ce_listed(c, t) ? 1 : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    int at = incl - n;
    for (int w = 0; w < wave; ++w) at += sums[w];
    for (int t = t0; t < t1; ++t)
      if (ce_listed(c, t)) c.w.rows[at++] = t;
    if (tid == 1023) c.w.count[0] = at;
    return;
  }
  // a quarter of the row for each of four waves
  __shared__ double part[16];
  const int t = (int(blockIdx.x) - 1) * 4 + (wave >> 2), q = wave & 3, d = c.a.d;
  const bool listed = t < T && ce_listed(c, t);
  double sum = 0.0;
  if (listed) {
    const E *x = static_cast<const E *>(c.a.X) + int64_t(t) * d;
    const E *w = static_cast<const E *>(c.a.W) + int64_t(c.a.targets[t]) * d;
    for (int i = (q * 64 + lane) * 8; i < d; i += 2048) {
      float xv[8], wv[8];
      Elem<E>::load8(x + i, xv);
      Elem<E>::load8(w + i, wv);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fma(double(xv[k]), double(wv[k]), sum);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  } else if (t < T) {
    if (q == 0 && lane == 0) c.a.loss[t] = c.a.targets[t] >= c.a.V ? __builtin_nanf("") : 0.f;
    const float z[8] = {};
    for (int i = (q * 64 + lane) * 8; c.a.dX && i < d; i += 2048)
      Cols<E, 8>::store(static_cast<E *>(c.a.dX) + int64_t(t) * d + i, z);
  }
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  if (listed && q == 0 && lane == 0) {
    sum = (part[wave] + part[wave + 1]) + (part[wave + 2] + part[wave + 3]);
    c.w.ly[t] = sum * double(c.a.logit_scale) * 1.4426950408889634074;
  }
}

// ------------------------------------------------------------ first product
// 8 logits of one row (list entry r, columns col .. col + 7 of a 64-column
// piece that 8 neighbouring lanes share) to e: the piece's sum and shift, and
// with a gradient e itself.  Columns past V and the target's count as nothing.
// Every lane of the wave calls this.
template <typename E>
__device__ __forceinline__ void ce_store8(const CeArgs &c, float (&v)[8], int lr, bool row_ok, int col, float ref,
                                          int y) {
  const float s2 = c.a.logit_scale * kLog2e;
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = col + k < c.a.V ? fmaf(v[k], s2, -ref) : -INFINITY;
    top = fmaxf(top, v[k]);
  }
  float shift = 0.f;
  if (__ballot(row_ok && top > kMaxExp)) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    // an infinity keeps its place: the row's sum then is no number
    shift = top > kMaxExp && top < INFINITY ? ceilf(top) : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] -= shift;
  }
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = __builtin_amdgcn_exp2f(v[k]);
    if (col + k == y) v[k] = 0.f;
    sum += v[k];
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor(sum, o, 64);
  if (!row_ok) return;
  if (c.a.dX && col < c.w.lde) Cols<E, 8>::store(static_cast<E *>(c.w.e) + int64_t(lr) * c.w.lde + col, v);
  if ((threadIdx.x & 7) == 0 && col / kSub < c.w.pieces)
    c.w.part[int64_t(lr) * c.w.pieces + col / kSub] = make_float2(sum, shift);
}

// Rows of the list, anywhere in X, by rows of W, both along d.
template <typename C, bool kWide>
struct LogitsSrc {
  const uint16_t *X, *W;
  RowOffsets<C::A_INS, kWide> ao;
  uint32_t bo[C::B_INS];
  int wave, wm, wn;
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    if (i < C::A_INS) {
      ao.copy(X + kt * 64, i, lds + (wave * C::A_INS + i) * 1024);
    } else {
      lds_dma16_s(W + kt * 64, bo[i - C::A_INS], lds + C::BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
    }
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    return frag_rows(base, s, q < C::TM ? (wm * C::TM + q) * 16 : C::BM + (wn * C::TN + q - C::TM) * 16);
  }
};

template <typename C, bool kWide>
__global__ __launch_bounds__(C::NT, 1) void ce_logits_kernel(CeArgs c) {
  constexpr int WC = C::TN * 16, SC = WC + 4;
  static_assert(WC == kSub, "one piece per wave");
  static_assert(C::NW * 32 * SC * 4 <= C::LDS && C::TM % 2 == 0, "staging must fit in LDS");
  __shared__ __attribute__((aligned(16))) char smem[C::LDS];
  const int M = block_rows(c);
  int tm, tn;
  if (M <= 0 || !tile_of_workgroup(blockIdx.x, (M + C::BM - 1) / C::BM, (c.a.V + C::BN - 1) / C::BN, tm, tn)) return;
  const int m0 = tm * C::BM, n0 = tn * C::BN, d = c.a.d;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / C::WN, wn = wave % C::WN, lrow = lane >> 3;

  LogitsSrc<C, kWide> src;
  src.wave = wave; src.wm = wm; src.wn = wn;
  src.X = static_cast<const uint16_t *>(c.a.X);
  src.W = static_cast<const uint16_t *>(c.a.W) + int64_t(n0) * d;
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + lrow;
    src.ao.set(i, int64_t(c.w.rows[c.row0 + min(m0 + row, M - 1)]) * d + fswz(row, lane & 7) * 8);
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int row = (wave * C::B_INS + i) * 8 + lrow;
    src.bo[i] = (uint32_t(min(row, c.a.V - 1 - n0)) * uint32_t(d) + fswz(row, lane & 7) * 8) * 2;
  }
  // ref and target of the tile's rows, fetched under the K loop: as loads of
  // the epilogue they were a third of it
  __shared__ float s_ref[C::BM];
  __shared__ int s_y[C::BM];
  float ref = 0.f;
  int y = -1;
  if (int(threadIdx.x) < C::BM) {
    const int t = c.w.rows[c.row0 + min(m0 + int(threadIdx.x), M - 1)];
    ref = ref_of(c.w.ly[t]);
    y = c.a.targets[t];
  }
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, d / 64, acc);
  if (int(threadIdx.x) < C::BM) {
    s_ref[threadIdx.x] = ref;
    s_y[threadIdx.x] = y;
  }
  lds_bar();

  // through the wave's own LDS, to lanes that hold 8 columns of a row
  float *stage = reinterpret_cast<float *>(smem) + wave * 32 * SC;
  const int vr = lane >> 3, col = n0 + wn * WC + (lane & 7) * 8;
#pragma unroll
  for (int i = 0; i < C::TM; i += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) stage[acc_row(h, v) * SC + acc_col(j)] = acc[i + h][j][v];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int tr = (wm * C::TM + i) * 16 + q * 8 + vr, lr = m0 + tr;
      const float4 lo = *reinterpret_cast<const float4 *>(stage + (q * 8 + vr) * SC + (lane & 7) * 8);
      const float4 hi = *reinterpret_cast<const float4 *>(stage + (q * 8 + vr) * SC + (lane & 7) * 8 + 4);
      float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      ce_store8<uint16_t>(c, x, lr, lr < M, col, s_ref[tr], s_y[tr]);
    }
  }
}

// ------------------------------------------------------------ float32
__global__ __launch_bounds__(256) void ce_logits_f32_kernel(CeArgs c) {
  __shared__ F32Tile lds;
  __shared__ __attribute__((aligned(16))) float stage[64][64 + 4];
  const int M = block_rows(c), d = c.a.d;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  if (m0 >= M) return;
  const float *X = static_cast<const float *>(c.a.X), *W = static_cast<const float *>(c.a.W);
  // ref and target of the tile's rows, as in ce_logits_kernel
  __shared__ float s_ref[64];
  __shared__ int s_y[64];
  float ref = 0.f;
  int y = -1;
  if (threadIdx.x < 64) {
    const int t = c.w.rows[c.row0 + min(m0 + int(threadIdx.x), M - 1)];
    ref = ref_of(c.w.ly[t]);
    y = c.a.targets[t];
  }
  // the thread's two rows of X: the list is read once, not with every chunk's loads
  int64_t x_row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    x_row[i] = int64_t(c.w.rows[c.row0 + min(m0 + int(threadIdx.x) / 8 + 32 * i, M - 1)]) * d;
  const f32x16_t acc = tile_f32<false>(
      lds, 0, d,
      [&](int r, int k) { return *reinterpret_cast<const float4 *>(X + (r < 32 ? x_row[0] : x_row[1]) + k); },
      [&](int r, int k) { return *reinterpret_cast<const float4 *>(W + int64_t(min(n0 + r, c.a.V - 1)) * d + k); });
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int v = 0; v < 16; ++v) stage[f32_row(v)][f32_col()] = acc[v];
  if (threadIdx.x < 64) {
    s_ref[threadIdx.x] = ref;
    s_y[threadIdx.x] = y;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int rr = q * 32 + (threadIdx.x >> 3), lr = m0 + rr;
    const bool ok = lr < M;
    float x[8];
    Elem<float>::load8(&stage[rr][(lane & 7) * 8], x);
    ce_store8<float>(c, x, lr, ok, n0 + (lane & 7) * 8, s_ref[rr], s_y[rr]);
  }
}

// ------------------------------------------------------------ rows' sums
// One workgroup per row: its pieces on one shift, the loss and the
// coefficients of its gradient.
template <typename E>
__global__ __launch_bounds__(256) void ce_row_kernel(CeArgs c) {
  __shared__ float red[2][4];
  const int lr = blockIdx.x;
  if (lr >= block_rows(c)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float2 *part = c.w.part + int64_t(lr) * c.w.pieces;
  float R = 0.f;
  for (int i = tid; i < c.w.pieces; i += 256) R = fmaxf(R, part[i].y);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) R = fmaxf(R, __shfl_xor(R, o, 64));
  if (lane == 0) red[0][wave] = R;
  __syncthreads();
  R = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  float S = 0.f;
  for (int i = tid; i < c.w.pieces; i += 256) {
    const float2 p = part[i];
    S += R > 0.f ? p.x * exp2f(p.y - R) : p.x;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) S += __shfl_xor(S, o, 64);
  if (lane == 0) red[1][wave] = S;
  __syncthreads();
  S = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  if (R > 0.f && c.a.dX) {
    E *e = static_cast<E *>(c.w.e) + int64_t(lr) * c.w.lde;
    for (int64_t i = tid * 8; i < c.w.lde; i += 256 * 8) {
      const float f = exp2f(part[i / kSub].y - R);
      if (f == 1.f) continue;
      float v[8];
      Elem<E>::load8(e + i, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= f;
      Cols<E, 8>::store(e + i, v);
    }
  }
  if (tid != 0) return;
  const int r = c.row0 + lr, t = c.w.rows[r];
  const float w = c.a.weights ? c.a.weights[t] : 1.f;
  const double ly = c.w.ly[t], up = double(ref_of(ly)) + double(R) - ly;   // ref + R - L_y
  const double ey = exp2(-up);                    // the target's e on the row's shift
  double loss, z = double(S) + ey;
  if (!(S < INFINITY) || !(ly < double(INFINITY))) loss = z = __builtin_nan("");
  else if (up > 900.0) loss = log(double(S)) + up * 0.69314718055994530942;
  else loss = log1p(double(S) * exp2(up));
  c.a.loss[t] = float(double(w) * loss);
  const double k = double(w) * double(c.a.logit_scale) / z;
  c.w.coef[r] = make_float2(float(k), float(-k * double(S)));
}

// ------------------------------------------------------------ second product
// e [rows][lde] along the vocabulary by W [V][d] across it.  A K tile of W is
// 64 rows of BN columns in LDS, 16-byte piece p of row k in slot
// p ^ (2 (k % 4) + 8 (k / 8 % 2)): the transposing reads of a fragment take
// rows k .. k + 3 and k + 8 .. k + 11 by 32 bytes at once, which then cover the
// 64 banks once.  Rows past V meet zeros of e.
__device__ __forceinline__ int exp_swz(int k) { return ((k & 3) << 1) | (((k >> 3) & 1) << 3); }

template <typename C>
struct ExpSrc {
  static_assert(C::BN == 256, "a row of the B tile is 512 bytes");
  const uint16_t *e, *W;              // from the split's first K tile
  uint32_t ao[C::A_INS], brow[C::B_INS], bcol[C::B_INS];
  uint32_t pitch;                     // bytes of a row of W
  int wave, wm, wn, last;             // last: V - 1, from the first K tile
  __device__ __forceinline__ void copy(uint32_t lds, int kt, int i) const {
    if (i < C::A_INS) {
      lds_dma16_s(e + kt * 64, ao[i], lds + (wave * C::A_INS + i) * 1024);
    } else {
      const uint32_t top = uint32_t(min(last - kt * 64, 63)) * pitch;   // the last row's offset in this K tile
      const uint32_t off = min(brow[i - C::A_INS], top) + bcol[i - C::A_INS];
      lds_dma16_s(reinterpret_cast<const char *>(W) + int64_t(kt) * 64 * pitch, off,
                  lds + C::BM * C::ROWB + (wave * C::B_INS + i - C::A_INS) * 1024);
    }
  }
  __device__ __forceinline__ bf16x8_t frag(const char *base, int s, int q) const {
    if (q < C::TM) return frag_rows(base, s, (wm * C::TM + q) * 16);
    // lane (column lane % 16, k of 8 (lane / 16) .. + 7): two transposing
    // reads.  In each group of 16 lanes, lane L gives the address of row L / 4
    // of a 4-row block, columns 4 (L % 4) .. + 3, and receives column L of the
    // 4 rows.
    const int lane = threadIdx.x & 63, L = lane & 15, cb = (wn * C::TN + q - C::TM) * 16 + 4 * (L & 3);
    const int kk = 32 * s + 8 * (lane >> 4) + (L >> 2);
    const char *p = base + C::BM * C::ROWB + kk * 512 + (((cb >> 3) ^ exp_swz(kk)) << 4) + (cb & 7) * 2;
    typedef __attribute__((address_space(3))) v4i16_t lds_v4;
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p));
    const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(p + 4 * 512));
    bf16x8_t f;
    __builtin_memcpy(&f, &lo, 8);
    __builtin_memcpy(reinterpret_cast<char *>(&f) + 8, &hi, 8);
    return f;
  }
};

// K tiles of split z of n
__device__ __forceinline__ void split_range(int kt, int splits, int z, int &k0, int &nk) {
  // scalar: the division is not, and the copies' bases have to be
  const int b = __builtin_amdgcn_readfirstlane(int(int64_t(kt) * z / splits));
  k0 = b * 64;
  nk = __builtin_amdgcn_readfirstlane(int(int64_t(kt) * (z + 1) / splits)) - b;
}

template <typename C>
__global__ __launch_bounds__(C::NT, 1) void ce_grad_kernel(CeArgs c) {
  __shared__ __attribute__((aligned(16))) char smem[C::LDS];
  const int M = block_rows(c), d = c.a.d;
  int tm, tn, z;
  if (M <= 0 || !tile_of_workgroup(blockIdx.x, (M + C::BM - 1) / C::BM, (d + C::BN - 1) / C::BN, c.w.splits, tm, tn, z))
    return;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int lane = threadIdx.x & 63, wave = wave_id();
  int k0, nk;
  split_range(int(c.w.lde / 64), c.w.splits, z, k0, nk);
  ExpSrc<C> src;
  src.wave = wave; src.wm = wave / C::WN; src.wn = wave % C::WN;
  src.last = c.a.V - 1 - k0;
  src.pitch = uint32_t(d) * 2;
  src.e = static_cast<const uint16_t *>(c.w.e) + int64_t(m0) * c.w.lde + k0;
  src.W = static_cast<const uint16_t *>(c.a.W) + int64_t(k0) * d;
#pragma unroll
  for (int i = 0; i < C::A_INS; ++i) {
    const int row = (wave * C::A_INS + i) * 8 + (lane >> 3);
    src.ao[i] = (uint32_t(min(row, M - 1 - m0)) * uint32_t(c.w.lde) + fswz(row, lane & 7) * 8) * 2;
  }
#pragma unroll
  for (int i = 0; i < C::B_INS; ++i) {
    const int k = 2 * (wave * C::B_INS + i) + (lane >> 5);
    src.brow[i] = uint32_t(k) * src.pitch;
    src.bcol[i] = uint32_t(min(n0 + ((lane & 31) ^ exp_swz(k)) * 8, d - 8)) * 2;
  }
  f32x4_t acc[C::TM][C::TN];
  tile_loop<C>(src, smem, nk, acc);
  float *out = c.w.acc + int64_t(z) * c.w.block * d;
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j) {
      const int col = n0 + src.wn * C::TN * 16 + acc_col(j);
      if (col >= d) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int lr = m0 + src.wm * C::TM * 16 + acc_row(i, v);
        if (lr < M) __builtin_nontemporal_store(acc[i][j][v], out + int64_t(lr) * d + col);
      }
    }
}

__global__ __launch_bounds__(256) void ce_grad_f32_kernel(CeArgs c) {
  __shared__ F32Tile lds;
  const int M = block_rows(c), d = c.a.d;
  // (rows last: those past the list's end would leave their CUs' places empty)
  const int m0 = blockIdx.z * 64, n0 = blockIdx.x * 64, z = blockIdx.y;
  if (m0 >= M) return;
  const float *e = static_cast<const float *>(c.w.e), *W = static_cast<const float *>(c.a.W);
  int k0, nk;
  split_range(int(c.w.lde / 64), c.w.splits, z, k0, nk);
  const f32x16_t acc = tile_f32<true>(
      lds, k0, k0 + nk * 64,
      [&](int r, int k) { return *reinterpret_cast<const float4 *>(e + int64_t(min(m0 + r, M - 1)) * c.w.lde + k); },
      [&](int n, int k) { return *reinterpret_cast<const float4 *>(W + int64_t(min(k, c.a.V - 1)) * d + n0 + n); });
  float *out = c.w.acc + int64_t(z) * c.w.block * d;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int lr = m0 + f32_row(v);
    if (lr < M) out[int64_t(lr) * d + n0 + f32_col()] = acc[v];
  }
}

// dX of one row's 2048 columns from blockIdx.y: the splits' sums in order, the
// target's term, one rounding.
template <typename E>
__global__ __launch_bounds__(256) void ce_finish_kernel(CeArgs c) {
  const int lr = blockIdx.x, d = c.a.d, i = (int(blockIdx.y) * 256 + int(threadIdx.x)) * 8;
  if (lr >= block_rows(c) || i >= d) return;
  const int r = c.row0 + lr, t = c.w.rows[r];
  const float2 k = c.w.coef[r];
  const int64_t pitch = int64_t(c.w.block) * d;
  const float *src = c.w.acc + int64_t(lr) * d + i;
  float v[8], w[8];
  Elem<float>::load8(src, v);
  Elem<E>::load8(static_cast<const E *>(c.a.W) + int64_t(c.a.targets[t]) * d + i, w);
  for (int z0 = 1; z0 < c.w.splits; z0 += 4) {
    Raw8<float> pr[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) pr[z].load(src + min(z0 + z, c.w.splits - 1) * pitch);
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      if (z0 + z < c.w.splits) {
        float o[8];
        pr[z].to8(o);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += o[q];
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = fmaf(k.x, v[q], k.y * w[q]);
  Cols<E, 8>::store(static_cast<E *>(c.a.dX) + int64_t(t) * d + i, v);
}

size_t up(size_t x) { return (x + 255) & ~size_t(255); }

CeWs ce_layout(char *ws, int T, int V, int d, int dtype, bool grad) {
  CeWs w{};
  const size_t e = dtype == LORA_BF16 ? 2 : 4;
  const int tile = dtype == LORA_BF16 ? 256 : 64;
  w.lde = (int64_t(V) + 63) / 64 * 64;
  w.pieces = int(w.lde / kSub);
  // rows of a block: as many as kBlockBytes hold of the exponentials and, with a gradient,
  // of its float32 sums, the blocks alike.  (Several splits take 64 MiB of sums at most:
  // they are for outputs of few tiles.)
  int64_t most = int64_t(kBlockBytes / std::max(size_t(w.lde) * e, grad ? size_t(d) * 4 : 0)) / tile * tile;
  if (most < tile) most = tile;
  const int64_t blocks = (T + most - 1) / most;
  int64_t rows = blocks > 0 ? (T + blocks - 1) / blocks : 1;
  rows = (rows + tile - 1) / tile * tile;
  w.block = int(rows < T ? rows : T);
  size_t at = 0;
  auto take = [&](size_t n) { char *p = ws ? ws + at : nullptr; at += up(n); return p; };
  w.count = reinterpret_cast<int32_t *>(take(4));
  w.rows = reinterpret_cast<int32_t *>(take(size_t(T) * 4));
  w.ly = reinterpret_cast<double *>(take(size_t(T) * 8));
  w.coef = reinterpret_cast<float2 *>(take(size_t(T) * 8));
  w.part = reinterpret_cast<float2 *>(take(size_t(w.block) * size_t(w.pieces) * 8));
  if (grad) {
    const int64_t kt = w.lde / 64;
    auto split = [&](int64_t tiles, int64_t fill, int64_t least) {
      int64_t n = fill / (tiles > 0 ? tiles : 1);
      if (n > kt / least) n = kt / least;
      if (n > kMaxSplits) n = kMaxSplits;
      return int(n < 1 ? 1 : n);
    };
    if (dtype == LORA_BF16) {
      // the K tiles of a workgroup's share, and what its sums cost at 4 TB/s
      // written and read once more
      double least = 0.0;
      for (int i = kBig; i <= kMid; ++i) {
        const int64_t tiles = tile_count(i, w.block, d);
        const int n = split(tiles, 256, 8);
        const double rounds = double((tiles * n + 255) / 256) * double((kt + n - 1) / n);
        const double us = 0.17 * kTileShapes[i].cost * rounds + 2.0 * n * double(w.block) * d * 4.0 / 4e6;
        if (i == kBig || us < least) {
          least = us;
          w.shape = i;
          w.splits = n;
        }
      }
    } else {
      w.splits = split(int64_t((w.block + 63) / 64) * (d / 64), 768, 4);   // several on a CU
    }
    w.e = take(size_t(w.block) * size_t(w.lde) * e);
    w.acc = reinterpret_cast<float *>(take(size_t(w.splits) * size_t(w.block) * size_t(d) * 4));
  }
  w.bytes = at;
  return w;
}

template <typename C>
void launch_logits(const CeArgs &c, int rows, hipStream_t s) {
  const int tiles = ((rows + C::BM - 1) / C::BM) * ((c.a.V + C::BN - 1) / C::BN);
  const dim3 grid(8 * unsigned((tiles + 7) / 8));
  if (int64_t(c.a.T) * c.a.d < (int64_t(1) << 31))
    hipLaunchKernelGGL((ce_logits_kernel<C, false>), grid, dim3(C::NT), 0, s, c);
  else
    hipLaunchKernelGGL((ce_logits_kernel<C, true>), grid, dim3(C::NT), 0, s, c);
}

template <typename C>
void launch_grad(const CeArgs &c, int rows, hipStream_t s) {
  const int tiles = ((rows + C::BM - 1) / C::BM) * ((c.a.d + C::BN - 1) / C::BN);
  hipLaunchKernelGGL((ce_grad_kernel<C>), dim3(8 * unsigned((tiles * c.w.splits + 7) / 8)), dim3(C::NT), 0, s, c);
}

template <typename E>
hipError_t run(CeArgs c, hipStream_t s) {
  constexpr bool bf = sizeof(E) == 2;
  const int T = c.a.T, V = c.a.V, d = c.a.d;
  hipLaunchKernelGGL(ce_rows_kernel<E>, dim3(unsigned(1 + (T + 3) / 4)), dim3(1024), 0, s, c);
  for (int r0 = 0; r0 < T; r0 += c.w.block) {
    c.row0 = r0;
    const int rows = T - r0 < c.w.block ? T - r0 : c.w.block;
    if (bf) {
      switch (pick_shape(rows, V)) {
        case kBig: launch_logits<Big>(c, rows, s); break;
        case kTall: launch_logits<Tall>(c, rows, s); break;
        case kMid: launch_logits<Mid>(c, rows, s); break;
        default: launch_logits<Small>(c, rows, s);
      }
    } else {
      hipLaunchKernelGGL(ce_logits_f32_kernel, dim3(unsigned((V + 63) / 64), unsigned((rows + 63) / 64)), dim3(256), 0,
                         s, c);
    }
    hipLaunchKernelGGL(ce_row_kernel<E>, dim3(unsigned(rows)), dim3(256), 0, s, c);
    if (c.a.dX) {
      if (bf) {
        switch (c.w.shape) {
          case kBig: launch_grad<Big>(c, rows, s); break;
          case kTall: launch_grad<Tall>(c, rows, s); break;
          default: launch_grad<Mid>(c, rows, s);
        }
      } else {
        hipLaunchKernelGGL(ce_grad_f32_kernel, dim3(unsigned(d / 64), unsigned(c.w.splits), unsigned((rows + 63) / 64)),
                           dim3(256), 0, s, c);
      }
      hipLaunchKernelGGL(ce_finish_kernel<E>, dim3(unsigned(rows), unsigned((d + 2047) / 2048)), dim3(256), 0, s, c);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

}  // namespace

size_t cross_entropy_workspace_bytes(int T, int V, int d, int dtype, bool grad) {
  return ce_layout(nullptr, T, V, d, dtype, grad).bytes;
}

hipError_t launch_cross_entropy(const CrossEntropyArgs &a, int dtype, void *ws, hipStream_t s) {
  CeArgs c{};
  c.a = a;
  c.w = ce_layout(static_cast<char *>(ws), a.T, a.V, a.d, dtype, a.dX != nullptr);
  return dtype == LORA_BF16 ? run<uint16_t>(c, s) : run<float>(c, s);
}

}  // namespace lora
