// What the kernels that choose experts compare and score with
// (route_select.cu, few_route.cu).
#pragma once

#include "common.cuh"

namespace moe {

// Order-preserving key of the result of an fp32 addition: larger value,
// larger key; NaN (an addition's NaN is positive) above +inf.  0 is below
// every value's key.
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// 1 / d rounded to nearest, for 1 <= d < 2^120: a Newton step in fused
// multiply-adds from an approximation within a unit of the last place
// (Markstein, IBM J. Res. Dev. 34, 1990).  A GPU test compares it with the
// quotient for the d of every fp32 logit.
__device__ __forceinline__ float reciprocal(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return fmaf(r, fmaf(-d, r, 1.f), r);
}

// 1 / (1 + exp(-z)), each step rounded to fp32.  NEAR: z >= kNearest.
constexpr float kNearest = -80.f;
template <bool NEAR = false>
__device__ __forceinline__ float sigmoid(float z) {
  const float d = 1.f + expf(-z);
  return NEAR || d <= 0x1p119f ? reciprocal(d) : __frcp_rn(d);
}

}  // namespace moe
