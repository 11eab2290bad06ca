// quantize.cuh -- e4m3 values and their blocks' scales (device helpers).
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace recattn {

constexpr float kFloatMax = 3.402823466e38f;

// The scale for a block whose largest finite value is `top`, and its reciprocal: 448 = 1.75 2^8.
__device__ __forceinline__ float block_scale(float top, float& inverse) {
  const uint32_t bits = __float_as_uint(top);
  int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < 1 ? 1 : e;  // 2^-126: both the scale and its reciprocal are normal
  if (top == 0.f) e = 127;
  inverse = __uint_as_float((uint32_t)(254 - e) << 23);
  return __uint_as_float((uint32_t)e << 23);
}
__device__ __forceinline__ float finite_size(float v) {
  const float a = fabsf(v);
  return a <= kFloatMax ? a : 0.f;
}
// The larger of a size and a value's, NaN if the value is one.
__device__ __forceinline__ float largest_or_nan(float top, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(v)));
  return r;
}
__device__ __forceinline__ uint32_t pack2_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Four values in e4m3; one that is not finite (fine: there is none) becomes NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d, bool fine) {
  if (!fine) {
    const auto keep = [](float v) { return fabsf(v) <= kFloatMax ? v : __uint_as_float(0x7fffffffu); };
    a = keep(a), b = keep(b), c = keep(c), d = keep(d);
  }
  return pack2_e4m3(a, b) | pack2_e4m3(c, d) << 16;
}

}  // namespace recattn
