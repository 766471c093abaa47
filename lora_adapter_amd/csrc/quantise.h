// e4m3 codes with power-of-two block scales: the scale rule and the encoding,
// shared by the quantising kernels and the GEMMs that quantise their rows.
// Internal to liblora (gfx950 only).
#pragma once

#include "lora_internal.h"

namespace lora {

constexpr int kQBlock = 128;              // columns (and, for weights, rows) per scale
constexpr int kQTableBytes = 4096;        // a weight row's scale bytes in the tile GEMM's LDS table
constexpr int kQMaxWidth = kQTableBytes * kQBlock;

// Bytes of a row of codes (a multiple of the block) and of a row of scale
// bytes (a multiple of 4, so that a dword holds four blocks' scales).
__host__ __device__ inline int64_t q_row_bytes(int64_t d) { return (d + kQBlock - 1) / kQBlock * kQBlock; }
__host__ __device__ inline int64_t q_scale_bytes(int64_t d) {
  return ((d + kQBlock - 1) / kQBlock + 3) / 4 * 4;
}

// Scale bytes of quantised rows as the tile GEMM copies them: one run per K
// tile (block) of the rows padded to whole tiles of 256; in each group of 128
// rows, rows r, r + 32, r + 64 and r + 96 share a dword.
__host__ __device__ inline int64_t q_tile_rows(int64_t T) { return (T + 255) / 256 * 256; }
__host__ __device__ inline int64_t q_tile_scale_at(int64_t T, int64_t t, int64_t blk) {
  return blk * q_tile_rows(T) + (t & ~int64_t(127)) + (t & 31) * 4 + ((t >> 5) & 3);
}

namespace {

// Scale byte of a block from the bits of its largest magnitude: e + 127 for
// the smallest e >= -126 with amax <= 448 . 2^e (448 = 1.75 . 2^8, so e is the
// exponent of amax less 8, one more when its mantissa is over 1.75); 255 for a
// block that holds an infinity or a NaN.  A power of two, so x / 2^e is exact
// and each code is one rounding of x; the MFMA applies it without arithmetic
// of the wave's own.
__device__ __forceinline__ uint32_t q_scale_byte(uint32_t amax_bits) {
  const int ex = int(amax_bits >> 23);
  if (ex == 255) return 255;
  return uint32_t(max(1, ex - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0)));
}

// 2^-e of a scale byte 1 .. 247 (normal).
__device__ __forceinline__ float q_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Eight values to e4m3 codes under a scale byte (v_cvt_pk_fp8_f32: nearest
// even; |v . 2^-e| <= 448, so nothing overflows).  A block without a scale
// (byte 255) takes NaN codes.
__device__ __forceinline__ uint2 q_encode8(const float v[8], uint32_t byte) {
  if (byte == 255) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  const float s = q_inv_scale(byte);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * s, v[1] * s, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * s, v[3] * s, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * s, v[5] * s, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * s, v[7] * s, hi, true);
  return make_uint2(uint32_t(lo), uint32_t(hi));
}

__device__ __forceinline__ uint32_t abs_max8(const float v[8]) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

// Largest of 16 consecutive lanes (a DPP row), in every one of them: row
// rotations by 8, 4, 2 and 1, no trip through LDS.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x128, 0xf, 0xf, false)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x124, 0xf, 0xf, false)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x122, 0xf, 0xf, false)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x121, 0xf, 0xf, false)));
  return v;
}

}  // namespace

hipError_t launch_quantise_rows(const void *X, int dtype, int T, int d, uint8_t *codes,
                                uint8_t *scale, bool tiled, hipStream_t s);
// bf16 rows in the tile layout, with the plan built by one more workgroup (of
// kPlanThreads threads) in up to kQPlanRowsLds of LDS (every workgroup of the
// launch has that LDS: two of them to a CU).
constexpr size_t kQPlanRowsLds = 72 << 10;
hipError_t launch_quantise_plan(const void *X, int T, int d, uint8_t *codes, uint8_t *scale,
                                const PlanLaunch &pl, hipStream_t s);
hipError_t launch_quantise_weight(const void *W_t, int dtype, int d_out, int d_in, uint8_t *q_t,
                                  uint8_t *q, uint8_t *scale, uint8_t *scale_t, hipStream_t s);

}  // namespace lora
