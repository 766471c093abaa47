// Gradient norms of adapters over many layers, and clipping.
//
//   n_a^2 = sum over layers of |dA_a|^2 + |dB_a|^2,   out <- g . min(1, max_norm / n)
//
// with n the adapter's own norm or that of all listed adapters together.
// Squares and sums are float64: a float32 square overflows past 1.8e19, and
// float64 costs nothing beside the loads.  Every partial sum has a place of
// its own and is added in a fixed order, so results are deterministic.
//
// Two passes of one workgroup for some rows of a (listed adapter, layer's
// factor): squares, then the product with the coefficient.  Between them one
// workgroup per adapter adds its partials; of few partials each workgroup of
// the second pass adds them itself instead, its row's loads in flight (4
// adapters of rank 16, 20 MB: two launches 17 us, four 24).  Bytes bound it:
// each row is read twice and written once, four 16-byte loads of a thread in
// flight, the second pass from the last row back (48 adapters, 1 GB: 195 + 340
// us, 5.2 and 6.0 TB/s; from the first row on, one load in flight and a
// workgroup for each row 240 + 368).
#include "lora_internal.h"

namespace lora {
namespace {

constexpr int kThreads = 256;

// Sum over the workgroup, the same order every time; valid in every thread.
__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// Four pieces of a row to this thread: columns c, c + 4 kThreads, .. while they
// are below d (past it: zeros, which the caller does not store).
constexpr int kPieces = 4, kStep = kThreads * 4;
__device__ __forceinline__ void load_pieces(const float *row, int c, int d, float4 (&v)[kPieces]) {
#pragma unroll
  for (int u = 0; u < kPieces; ++u)
    v[u] = c + u * kStep < d ? *reinterpret_cast<const float4 *>(row + c + u * kStep) : make_float4(0.f, 0.f, 0.f, 0.f);
}

// The rank of list entry m in layer l if its pages can be taken (0: not): the
// adapter in range, rank 1..max_rank, its page table consistent, and not
// listed before.  The same answer in every thread.  v: the first pieces of its
// row y in factor f (if it has one), whose loads go out before the rest of the
// table is looked at.
__device__ __forceinline__ int clip_rank(const ClipArgs &a, const ClipLayer &l, int m, int f, int y, int &ps,
                                         float4 (&v)[kPieces]) {
  const int ad = a.adapters[m];
  ps = 0;
  if (ad < 0 || ad >= l.n_adapters) return 0;
  const int r = l.rank[ad];
  ps = l.page_start[ad];
  const int pe = l.page_start[ad + 1];
  bool bad = r < 1 || r > a.max_rank || pe - ps != r || ps < 0 || int64_t(ps) + r > l.n_page_ids;
  if (bad) return 0;
  const int own = l.page_ids[ps + (y < r ? y : 0)];
  for (int j = threadIdx.x; j < m; j += kThreads) bad |= a.adapters[j] == ad;
  for (int j = threadIdx.x; j < r; j += kThreads) {
    const int p = l.page_ids[ps + j];
    bad |= p < 0 || p >= l.n_pages;
  }
  if (y < r && own >= 0 && own < l.n_pages)
    load_pieces(l.grad[f] + int64_t(own) * l.d[f], threadIdx.x * 4, l.d[f], v);
  return __syncthreads_or(bad) ? 0 : r;
}

// Workgroup (y, m, 2 l + f): rows y, y + Y, .. of entry m in factor f of layer l.
__global__ __launch_bounds__(kThreads) void clip_square_kernel(ClipArgs a) {
  __shared__ double red[4];
  const int m = blockIdx.y, z = blockIdx.z, y = blockIdx.x, Y = gridDim.x;
  const ClipLayer &l = a.layer[z >> 1];
  const int f = z & 1, d = l.d[f];
  int ps;
  float4 v[kPieces] = {};
  const int r = clip_rank(a, l, m, f, y, ps, v);
  double sum[kPieces] = {};
  for (int j = y; j < r; j += Y) {
    const float *row = l.grad[f] + int64_t(l.page_ids[ps + j]) * d;
    for (int c = threadIdx.x * 4; c < d; c += kPieces * kStep) {
      if (j != y || c >= kPieces * kStep) load_pieces(row, c, d, v);
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        sum[u] = fma(double(v[u].x), double(v[u].x), sum[u]);
        sum[u] = fma(double(v[u].y), double(v[u].y), sum[u]);
        sum[u] = fma(double(v[u].z), double(v[u].z), sum[u]);
        sum[u] = fma(double(v[u].w), double(v[u].w), sum[u]);
      }
    }
  }
  const double all = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]), red);
  if (threadIdx.x == 0) a.part[(int64_t(m) * a.factors + a.first + z) * Y + y] = all;
}

__device__ __forceinline__ double sum_of(const double *v, int64_t n, double *red) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += v[i];
  return block_sum(sum, red);
}

// Workgroup m: the square of entry m's norm from its partials.
__global__ __launch_bounds__(kThreads) void clip_norm_kernel(ClipArgs a) {
  __shared__ double red[4];
  const int m = blockIdx.x;
  const double sum = sum_of(a.part + m * a.parts, a.parts, red);
  if (threadIdx.x == 0) {
    a.square[m] = sum;
    a.norm[m] = float(sqrt(sum));
  }
}

__global__ __launch_bounds__(kThreads) void clip_total_kernel(ClipArgs a) {
  __shared__ double red[4];
  const double sum = sum_of(a.square, a.M, red);
  if (threadIdx.x == 0) a.norm[a.M] = float(sqrt(sum));
}

// The rows of clip_square_kernel times the coefficient, the last ones first:
// they are what the cache still holds.  With kPart each workgroup adds
// the partials itself, its row's loads in flight; otherwise clip_norm_kernel
// has.  The workgroups of an entry's first row write the norms.  A norm that is
// not finite, as the float that is written, clips nothing: the gradients stay what
// they are, and the norm says so.
template <bool kPart>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipArgs a) {
  __shared__ double red[4];
  const int y = gridDim.x - 1 - blockIdx.x, m = gridDim.y - 1 - blockIdx.y, z = gridDim.z - 1 - blockIdx.z;
  const ClipLayer &l = a.layer[z >> 1];
  const int f = z & 1, d = l.d[f], Y = gridDim.x;
  const bool first = y == 0 && a.first + z == 0;
  int ps;
  float4 v[kPieces] = {};
  const int r = clip_rank(a, l, m, f, y, ps, v);
  if (y >= r && !first) return;
  double square = 0.0, total = 0.0;
  if (kPart) {
    if (first || !a.together) square = sum_of(a.part + m * a.parts, a.parts, red);
    if ((first && m == 0) || a.together) total = sum_of(a.part, a.parts * a.M, red);
  } else {
    square = a.square[m];
    if ((first && m == 0) || a.together) total = sum_of(a.square, a.M, red);
  }
  if (first && threadIdx.x == 0) {
    if (kPart) a.norm[m] = float(sqrt(square));
    if (m == 0) a.norm[a.M] = float(sqrt(total));
  }
  const double n = sqrt(a.together ? total : square);
  const bool clips = n > double(a.max_norm) && float(n) < INFINITY;
  if (l.out[f] == l.grad[f] && !clips) return;
  // the factor stays float64: it may be under float32's normal numbers, whose few bits
  // (none under 2^-149) would be all that the results had
  const double coef = clips ? double(a.max_norm) / n : 1.0;
  for (int j = y; j < r; j += Y) {
    const int64_t at = int64_t(l.page_ids[ps + j]) * d;
    for (int c = threadIdx.x * 4; c < d; c += kPieces * kStep) {
      if (j != y || c >= kPieces * kStep) load_pieces(l.grad[f] + at, c, d, v);
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        v[u].x = float(v[u].x * coef); v[u].y = float(v[u].y * coef);
        v[u].z = float(v[u].z * coef); v[u].w = float(v[u].w * coef);
        if (c + u * kStep < d) *reinterpret_cast<float4 *>(l.out[f] + at + c + u * kStep) = v[u];
      }
    }
  }
}

// Workgroups along the rank rows, one row each until they make 2^15: the
// 1 GB above takes 638, 585, 553, 547 and 589 us with 2^12, 13, 14, 15 and 17.
int clip_rows(int n_layers, int M, int max_rank) {
  const int64_t pairs = int64_t(n_layers) * 2 * M;
  int64_t y = (int64_t(1) << 15) / (pairs > 0 ? pairs : 1);
  if (y < 1) y = 1;
  return int(y < max_rank ? y : max_rank);
}

// Partials of all entries up to which every workgroup of the second pass adds
// its entry's itself, and one (or, with one norm for all, each) adds them all: 8
// loads of a thread, below the launches between the passes.  7 layers of 1024 ->
// 1024, a norm for each entry: 896 partials 10.5 us against 12.7 with the launches,
// 1792 13.3 and 14.4, 3584 21.9 and 21.4; of 1024 -> 2048, 28672 138 and 117.
constexpr int64_t kOwnParts = 2048;

}  // namespace

size_t clip_workspace_bytes(int n_layers, int M, int max_rank) {
  return (size_t(n_layers) * 2 * size_t(clip_rows(n_layers, M, max_rank)) + 1) * size_t(M) * sizeof(double);
}

hipError_t launch_clip(const ClipLayer *layers, int n_layers, ClipArgs a, void *ws, hipStream_t s) {
  const int Y = clip_rows(n_layers, a.M, a.max_rank);
  a.square = static_cast<double *>(ws);
  a.part = a.square + a.M;
  a.factors = 2 * n_layers;
  a.parts = int64_t(a.factors) * Y;
  bool store = a.max_norm < INFINITY;
  for (int i = 0; i < n_layers; ++i)
    for (int f = 0; f < 2; ++f) store |= layers[i].out[f] != layers[i].grad[f];
  store = store && a.M > 0 && n_layers > 0;
  const bool own = store && a.parts * a.M <= kOwnParts;
  const int chunks = a.M > 0 ? (n_layers + kClipLayers - 1) / kClipLayers : 0;
  auto chunk = [&](int i) {
    const int l0 = i * kClipLayers, nl = n_layers - l0 < kClipLayers ? n_layers - l0 : kClipLayers;
    for (int q = 0; q < nl; ++q) a.layer[q] = layers[l0 + q];
    a.first = 2 * l0;
    return dim3(unsigned(Y), unsigned(a.M), unsigned(2 * nl));
  };
  for (int i = 0; i < chunks; ++i) {
    const dim3 grid = chunk(i);
    hipLaunchKernelGGL(clip_square_kernel, grid, dim3(kThreads), 0, s, a);
  }
  if (!own) {
    if (a.M > 0) hipLaunchKernelGGL(clip_norm_kernel, dim3(unsigned(a.M)), dim3(kThreads), 0, s, a);
    if (!store) hipLaunchKernelGGL(clip_total_kernel, dim3(1), dim3(kThreads), 0, s, a);
  }
  for (int i = chunks; store && i-- > 0;) {
    const dim3 grid = chunk(i);
    if (own) hipLaunchKernelGGL(clip_scale_kernel<true>, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(clip_scale_kernel<false>, grid, dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace lora
