// Gradient norms of adapters over many layers, and clipping.
//
//   n_a^2 = sum over layers of |dA_a|^2 + |dB_a|^2,   out <- g . min(1, max_norm / n)
//
// with n the adapter's own norm or that of all listed adapters together.
// Squares and sums are float64: a float32 square overflows past 1.8e19, and
// float64 costs nothing beside the loads.  Every partial sum has a place of
// its own and is added in a fixed order, so results are deterministic.
//
// Launches: one workgroup per (rank row, listed adapter, layer's factor)
// squares its row; one workgroup per adapter adds that adapter's partials; one
// workgroup per row again multiplies and stores.  Bytes bound it: each row is
// read twice (the second time from the 256 MB cache when the gradients fit
// it) and written once.
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

// The rank of list entry m in layer l if its pages can be taken (0: not): the
// adapter in range, rank 1..max_rank, its page table consistent, and not
// listed before.  The same answer in every thread.
__device__ __forceinline__ int clip_rank(const ClipArgs &a, const ClipLayer &l, int m, int &ps) {
  const int ad = a.adapters[m];
  ps = 0;
  if (ad < 0 || ad >= l.n_adapters) return 0;
  const int r = l.rank[ad];
  ps = l.page_start[ad];
  const int pe = l.page_start[ad + 1];
  bool bad = r < 1 || r > a.max_rank || pe - ps != r || ps < 0 || int64_t(ps) + r > l.n_page_ids;
  for (int j = threadIdx.x; j < m; j += kThreads) bad |= a.adapters[j] == ad;
  if (!bad) {
    for (int j = threadIdx.x; j < r; j += kThreads) {
      const int p = l.page_ids[ps + j];
      bad |= p < 0 || p >= l.n_pages;
    }
  }
  return __syncthreads_or(bad) ? 0 : r;
}

// Workgroup (y, m, 2 l + f): rows y, y + Y, .. of entry m in factor f of layer l.
__global__ __launch_bounds__(kThreads) void clip_square_kernel(ClipArgs a) {
  __shared__ double red[4];
  const int m = blockIdx.y, z = blockIdx.z, y = blockIdx.x, Y = gridDim.x;
  const ClipLayer &l = a.layer[z >> 1];
  const int f = z & 1, d = l.d[f];
  int ps;
  const int r = clip_rank(a, l, m, ps);
  double sum = 0.0;
  for (int j = y; j < r; j += Y) {
    const float *row = l.grad[f] + int64_t(l.page_ids[ps + j]) * d;
    for (int c = threadIdx.x * 4; c < d; c += kThreads * 4) {
      const float4 v = *reinterpret_cast<const float4 *>(row + c);
      sum = fma(double(v.x), double(v.x), sum);
      sum = fma(double(v.y), double(v.y), sum);
      sum = fma(double(v.z), double(v.z), sum);
      sum = fma(double(v.w), double(v.w), sum);
    }
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) a.part[(int64_t(m) * a.factors + a.first + z) * Y + y] = sum;
}

// Workgroup m: the square of entry m's norm from its partials.
__global__ __launch_bounds__(kThreads) void clip_norm_kernel(ClipArgs a, int Y) {
  __shared__ double red[4];
  const int m = blockIdx.x;
  const int64_t n = int64_t(a.factors) * Y;
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += a.part[m * n + i];
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) {
    a.square[m] = sum;
    a.norm[m] = float(sqrt(sum));
  }
}

__device__ __forceinline__ double total_square(const ClipArgs &a, double *red) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.M; i += kThreads) sum += a.square[i];
  return block_sum(sum, red);
}

__global__ __launch_bounds__(kThreads) void clip_total_kernel(ClipArgs a) {
  __shared__ double red[4];
  const double sum = total_square(a, red);
  if (threadIdx.x == 0) a.norm[a.M] = float(sqrt(sum));
}

// The rows of clip_square_kernel times the coefficient.  A norm that is not
// finite clips nothing: the gradients stay what they are, and the norm says so.
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipArgs a) {
  __shared__ double red[4];
  const int m = blockIdx.y, z = blockIdx.z;
  const ClipLayer &l = a.layer[z >> 1];
  const int f = z & 1, d = l.d[f];
  int ps;
  const int r = clip_rank(a, l, m, ps);
  if (int(blockIdx.x) >= r) return;
  const double n = sqrt(a.together ? total_square(a, red) : a.square[m]);
  const float coef = n > double(a.max_norm) && n < double(INFINITY) ? float(double(a.max_norm) / n) : 1.f;
  const bool same = l.out[f] == l.grad[f];
  if (same && coef == 1.f) return;
  for (int j = blockIdx.x; j < r; j += gridDim.x) {
    const int64_t at = int64_t(l.page_ids[ps + j]) * d;
    const float *row = l.grad[f] + at;
    float *out = l.out[f] + at;
    for (int c = threadIdx.x * 4; c < d; c += kThreads * 4) {
      float4 v = *reinterpret_cast<const float4 *>(row + c);
      v.x *= coef; v.y *= coef; v.z *= coef; v.w *= coef;
      *reinterpret_cast<float4 *>(out + c) = v;
    }
  }
}

// Workgroups along the rank rows: one row each unless that makes too many.
int clip_rows(int n_layers, int M, int max_rank) {
  const int64_t pairs = int64_t(n_layers) * 2 * M;
  int64_t y = (int64_t(1) << 17) / (pairs > 0 ? pairs : 1);
  if (y < 1) y = 1;
  return int(y < max_rank ? y : max_rank);
}

}  // namespace

size_t clip_workspace_bytes(int n_layers, int M, int max_rank) {
  return (size_t(n_layers) * 2 * size_t(clip_rows(n_layers, M, max_rank)) + 1) * size_t(M) * sizeof(double);
}

hipError_t launch_clip(const ClipLayer *layers, int n_layers, ClipArgs a, void *ws, hipStream_t s) {
  const int Y = clip_rows(n_layers, a.M, a.max_rank);
  a.square = static_cast<double *>(ws);
  a.part = a.square + a.M;
  a.factors = 2 * n_layers;
  bool store = a.max_norm < INFINITY;
  for (int i = 0; i < n_layers; ++i)
    for (int f = 0; f < 2; ++f) store |= layers[i].out[f] != layers[i].grad[f];
  for (int pass = 0; pass < 2; ++pass) {
    for (int l0 = 0; a.M > 0 && l0 < n_layers; l0 += kClipLayers) {
      const int nl = n_layers - l0 < kClipLayers ? n_layers - l0 : kClipLayers;
      for (int i = 0; i < nl; ++i) a.layer[i] = layers[l0 + i];
      a.first = 2 * l0;
      const dim3 grid(unsigned(Y), unsigned(a.M), unsigned(2 * nl));
      if (pass == 0) hipLaunchKernelGGL(clip_square_kernel, grid, dim3(kThreads), 0, s, a);
      else if (store) hipLaunchKernelGGL(clip_scale_kernel, grid, dim3(kThreads), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (pass == 0 && a.M > 0) {
      hipLaunchKernelGGL(clip_norm_kernel, dim3(unsigned(a.M)), dim3(kThreads), 0, s, a, Y);
    }
    if (pass == 0) {
      hipLaunchKernelGGL(clip_total_kernel, dim3(1), dim3(kThreads), 0, s, a);
    }
  }
  return hipGetLastError();
}

}  // namespace lora
