// INT8 rows with one FP32 scale each: the rule that moe_quantize_int8, the norm's INT8
// output and the INT8 experts share.
#pragma once

#include "common.h"

namespace moe {

// INT8 rows: scale = amax / 127, code = v * (127 / amax) to the nearest even.  A
// row below 2^-100 everywhere takes scale 0 and codes 0: 127 / amax would leave
// FP32's range not far below (amax < 3.8e-37), and no activation lives there.
constexpr float kInt8Tiny = 7.888609052210118e-31f;      // 2^-100
__device__ __forceinline__ float int8_scale(float amax) {
  return amax < kInt8Tiny ? 0.f : amax / 127.0f;
}
__device__ __forceinline__ float int8_inverse(float amax) {
  return amax < kInt8Tiny ? 0.f : 127.0f / amax;
}
// Four values' codes, code t in byte t; the clamp is for v * inv a hair above 127.
__device__ __forceinline__ uint32_t int8_codes4(float a, float b, float c, float d, float inv) {
  const float v[4] = {a, b, c, d};
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = static_cast<int>(rintf(__builtin_amdgcn_fmed3f(v[i] * inv, -127.f, 127.f)));
    w |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * i);
  }
  return w;
}

}  // namespace moe
