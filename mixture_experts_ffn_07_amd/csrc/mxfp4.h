// MXFP4 rows: E2M1 codes, two to a byte (the even element in the low four bits), with one
// E8M0 scale per 32 elements: the rule that moe_quantize_mxfp4 and the MXFP4 experts share.
#pragma once

#include "common.h"

namespace moe {

// MX scale exponent of a block for E2M1 codes (OCP Microscaling v1.0): s = floor(log2(amax))
// - 2, clamped to [-127, 127]; amax = 0 gives -127.  (mx_scale_exp subtracts 8, E4M3's.)
__device__ __forceinline__ int mx4_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (u == 0) return -127;
  const int fl = (u >> 23) == 0 ? (31 - __clz(u)) - 149 : static_cast<int>(u >> 23) - 127;
  const int s = fl - 2;
  return s < -127 ? -127 : s;                              // (fl <= 127: never above 125)
}

// Four FP32 -> four E2M1 codes in the low 16 bits, the first in the lowest: the hardware
// conversion, to the nearest, ties to even, saturating at +-6, sign kept; checked against
// the definition on every border between codes, its neighbours and 4000 random values.
__device__ __forceinline__ uint32_t f32x4_to_e2m1x4(float a, float b, float c, float d) {
  uint32_t v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, 1.0f, 0);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, c, d, 1.0f, 1);
  return v;
}

// Block-scaled MFMA with E2M1 weights (operand a) and activations b of E2M1 (A4) or E4M3,
// 16x16x128, taking byte SEL of the lanes' scale registers.  Lane (r, g) = (lane % 16,
// lane / 16) holds of row r the 32 codes of one block in its first 16 bytes (E2M1), or
// (E4M3) in bytes 0..15 half g & 1 of the block of lanes g >> 1, in bytes 16..31 the same
// half of the block of lanes 2 + (g >> 1); the scale of lane (r, g) is that of row r's
// block in lanes g.  Which 32 columns of K a lane's block is, is free as long as both
// operands agree.  Products of E2M1 add up exactly while they span less than 24 bits.  With
// an E4M3 operand the instruction adds runs of eight neighbours along K, each on a grid of
// 2^-13 of the power of two of its largest product (lower bits are cut off, towards zero),
// and the runs and the accumulator as FP32: measured with one product per run exact to
// 2^-22, with random ones off by up to 2^-11.8 of the sum of their magnitudes and 2^-10.9 of
// the largest; at the worst 7 * 2^-13 of each run's largest.  Both shapes do so, and E4M3
// times E4M3 (common.h) does the same.
template <bool A4, int SEL>
__device__ __forceinline__ f32x4 mfma_mx4_16(i32x4 a, i32x8 b, int sa, int sb, f32x4 c) {
  const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b, c, 4, A4 ? 4 : 0, SEL, sa, SEL, sb);
}

// E4M3 codes in two: high keeps those of 2 and above (bit 6 set), low the others, zeros in each other's
// places.  A run of the instruction's holds either without a bit below its grid: low are multiples of
// 2^-9 below 2, high of 2^-2 up to 448, times weights that are multiples of 2^-1 up to 6, so products
// are multiples of 2^-10 and of 2^-3 beside largest ones whose grids are 2^-11 and 2^-3.  The product
// with both, one after the other, is exact to FP32 (measured 2^-21.5 of the summed magnitudes).
__device__ __forceinline__ void split_e4m3(int v, int& low, int& high) {
  const uint32_t m = static_cast<uint32_t>(v) & 0x40404040u;
  const int keep = static_cast<int>(m << 1 | ((m << 1) - (m >> 6)));      // 0xFF in their bytes
  high = v & keep;
  low = v & ~keep;
}

}  // namespace moe
