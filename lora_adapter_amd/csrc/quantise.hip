// Quantisation to e4m3 with one power-of-two scale per block: rows (one scale
// per 128 columns: activations and gradients) and weights (one scale per 128 x
// 128 block, so that the codes of W and of W^T are the same and the input
// gradient runs over the very weight that the forward used).
#include "plan_build.h"
#include "quantise.h"

namespace lora {
namespace {

// Chunks w, w + stride, .. (NC of them; chunk = 512 columns of a row, 8
// elements per lane), their loads in flight together; 16 lanes share a block.
// Columns past d are zero codes.  kTiled: scale bytes laid out for the tile
// GEMM (q_tile_scale_at), else in rows.
template <typename E, bool kTiled, int NC>
__device__ __forceinline__ void quantise_chunks(const E *X, int T, int d, int chunks, uint8_t *codes,
                                                uint8_t *scale, int64_t w, int64_t stride) {
  const int lane = threadIdx.x & 63;
  const int64_t total = int64_t(T) * chunks;
  const int64_t ld = q_row_bytes(d), ls = q_scale_bytes(d);
  float v[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t wc = w + c * stride, t = wc / chunks;
    const int col = int(wc % chunks) * 512 + lane * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
    if (wc < total && col < d) Elem<E>::load8(X + t * d + col, v[c]);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t wc = w + c * stride, t = wc / chunks;
    if (wc >= total) return;
    const int col = int(wc % chunks) * 512 + lane * 8;
    const uint32_t byte = q_scale_byte(max16(abs_max8(v[c])));
    // (past d: zero in a block of scale byte 255 too)
    if (col < ld)
      *reinterpret_cast<uint2 *>(codes + t * ld + col) = col < d ? q_encode8(v[c], byte) : make_uint2(0, 0);
    const int blk = col / kQBlock;
    if ((lane & 15) != 0) continue;
    if constexpr (kTiled) {
      if (col < ld) scale[q_tile_scale_at(T, t, blk)] = uint8_t(byte);
    } else {
      if (blk < ls) scale[t * ls + blk] = col < ld ? uint8_t(byte) : uint8_t(0);
    }
  }
}

template <typename E, bool kTiled>
__global__ __launch_bounds__(256) void quantise_rows_kernel(const E *X, int T, int d, int chunks,
                                                            uint8_t *codes, uint8_t *scale) {
  const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  quantise_chunks<E, kTiled, 1>(X, T, d, chunks, codes, scale, wg * 4 + (threadIdx.x >> 6), 0);
}

// The rows quantised while the launch's first workgroup builds the batch's
// plan (neither needs the other).  The others keep two to a CU (the plan's LDS)
// and walk the chunks, four loads of each wave in flight.
template <bool kLds>
__global__ __launch_bounds__(kPlanThreads) void quantise_plan_kernel(const uint16_t *X, int T, int d,
                                                                     int chunks, uint8_t *codes,
                                                                     uint8_t *scale, PlanArgs pa) {
  extern __shared__ int qp_dyn[];
  if (blockIdx.x == 0) {
    plan_build<kLds>(pa, qp_dyn);
    return;
  }
  constexpr int W = kPlanThreads / 64, NC = 4;
  const int64_t waves = int64_t(gridDim.x - 1) * W, total = int64_t(T) * chunks;
  for (int64_t w = int64_t(blockIdx.x - 1) * W + (threadIdx.x >> 6); w < total; w += NC * waves)
    quantise_chunks<uint16_t, true, NC>(X, T, d, chunks, codes, scale, w, waves);
}

// 4 x 4 bytes turned: o[j] = byte j of each of d[0..3].
__device__ __forceinline__ void turn4(const uint32_t d[4], uint32_t o[4]) {
  const uint32_t a = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u);
  const uint32_t b = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
  const uint32_t e = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
  o[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(e, c, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(e, c, 0x07060302u);
}

// One workgroup per 128 x 128 block: 16 lanes per row, 16 rows at a time, the
// whole block in registers between its largest magnitude and its codes; the
// codes of W^T go through LDS as dwords of four columns.
template <typename E>
__global__ __launch_bounds__(256) void quantise_weight_kernel(const E *W, int d_out, int d_in,
                                                              uint8_t *q_t, uint8_t *q,
                                                              uint8_t *scale, uint8_t *scale_t) {
  constexpr int S = kQBlock / 4 + 1;                 // dwords per staged row (padded)
  __shared__ uint32_t tile[kQBlock * S];
  __shared__ uint32_t wmax[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int r0 = blockIdx.y * kQBlock, c0 = blockIdx.x * kQBlock;
  const int rr = tid >> 4, cc = (tid & 15) * 8;
  const int64_t ld = q_row_bytes(d_in), ldt = q_row_bytes(d_out);
  const bool c_ok = c0 + cc < d_in;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + rr + 16 * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    if (c_ok && r < d_out) Elem<E>::load8(W + int64_t(r) * d_in + c0 + cc, v[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_max8(v[i]));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o, 64)));
  if (lane == 0) wmax[tid >> 6] = m;
  __syncthreads();
  m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const uint32_t byte = q_scale_byte(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rr + 16 * i;
    uint2 w = q_encode8(v[i], byte);
    // a NaN block's padding stays zero
    if (!c_ok || r0 + r >= d_out) w = make_uint2(0, 0);
    if (r0 + r < d_out) *reinterpret_cast<uint2 *>(q_t + int64_t(r0 + r) * ld + c0 + cc) = w;
    tile[r * S + cc / 4] = w.x;
    tile[r * S + cc / 4 + 1] = w.y;
  }
  if (tid == 0) {
    const int64_t ls = q_scale_bytes(d_in), lst = q_scale_bytes(d_out);
    const int nbi = gridDim.x, nbo = gridDim.y;
    scale[blockIdx.y * ls + blockIdx.x] = uint8_t(byte);
    if (int(blockIdx.x) == nbi - 1)
      for (int64_t b = nbi; b < ls; ++b) scale[blockIdx.y * ls + b] = 0;
    if (scale_t) {
      scale_t[blockIdx.x * lst + blockIdx.y] = uint8_t(byte);
      if (int(blockIdx.y) == nbo - 1)
        for (int64_t b = nbo; b < lst; ++b) scale_t[blockIdx.x * lst + b] = 0;
    }
  }
  if (!q) return;
  __syncthreads();
  // lane -> 16 rows rg and 4 columns cg: 8 lanes write 128 bytes of one row of W^T
  const int rg = tid & 7, cg = tid >> 3;
  uint32_t o[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t d[4], t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = tile[(rg * 16 + k * 4 + i) * S + cg];
    turn4(d, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j][k] = t[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = c0 + cg * 4 + j;
    if (c < d_in)
      *reinterpret_cast<uint4 *>(q + int64_t(c) * ldt + r0 + rg * 16) =
          make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
  }
}

}  // namespace

hipError_t launch_quantise_rows(const void *X, int dtype, int T, int d, uint8_t *codes,
                                uint8_t *scale, bool tiled, hipStream_t s) {
  // whole scale rows: the padding bytes past the last block are written too
  const int chunks = int((q_scale_bytes(d) + 3) / 4);
  // (a grid dimension holds less than 2^32 threads)
  const int64_t wgs = (int64_t(T) * chunks + 3) / 4, gx = wgs < (1 << 20) ? wgs : 1 << 20;
  const dim3 grid(unsigned(gx), unsigned((wgs + gx - 1) / gx)), block(256);
  const uint16_t *xb = static_cast<const uint16_t *>(X);
  const float *xf = static_cast<const float *>(X);
  if (dtype == LORA_BF16 && tiled)
    hipLaunchKernelGGL((quantise_rows_kernel<uint16_t, true>), grid, block, 0, s, xb, T, d, chunks, codes, scale);
  else if (dtype == LORA_BF16)
    hipLaunchKernelGGL((quantise_rows_kernel<uint16_t, false>), grid, block, 0, s, xb, T, d, chunks, codes, scale);
  else if (!tiled)
    hipLaunchKernelGGL((quantise_rows_kernel<float, false>), grid, block, 0, s, xf, T, d, chunks, codes, scale);
  else
    return hipErrorInvalidConfiguration;
  return hipGetLastError();
}

hipError_t launch_quantise_plan(const void *X, int T, int d, uint8_t *codes, uint8_t *scale,
                                const PlanLaunch &pl, hipStream_t s) {
  const int chunks = int((q_scale_bytes(d) + 3) / 4);
  constexpr int W = kPlanThreads / 64;
  const int64_t wgs = (int64_t(T) * chunks + W - 1) / W;
  const dim3 grid(unsigned(1 + (wgs < 510 ? wgs : 510))), block(kPlanThreads);
  const uint16_t *x = static_cast<const uint16_t *>(X);
  if (pl.lds_bytes > kQPlanRowsLds) return hipErrorInvalidConfiguration;
  if (pl.lds)
    hipLaunchKernelGGL(quantise_plan_kernel<true>, grid, block, pl.lds_bytes, s, x, T, d, chunks, codes, scale, pl.a);
  else
    hipLaunchKernelGGL(quantise_plan_kernel<false>, grid, block, pl.lds_bytes, s, x, T, d, chunks, codes, scale, pl.a);
  return hipGetLastError();
}

hipError_t launch_quantise_weight(const void *W_t, int dtype, int d_out, int d_in, uint8_t *q_t,
                                  uint8_t *q, uint8_t *scale, uint8_t *scale_t, hipStream_t s) {
  const dim3 grid(unsigned((d_in + kQBlock - 1) / kQBlock), unsigned((d_out + kQBlock - 1) / kQBlock));
  if (dtype == LORA_BF16)
    hipLaunchKernelGGL(quantise_weight_kernel<uint16_t>, grid, dim3(256), 0, s,
                       static_cast<const uint16_t *>(W_t), d_out, d_in, q_t, q, scale, scale_t);
  else
    hipLaunchKernelGGL(quantise_weight_kernel<float>, grid, dim3(256), 0, s,
                       static_cast<const float *>(W_t), d_out, d_in, q_t, q, scale, scale_t);
  return hipGetLastError();
}

}  // namespace lora
