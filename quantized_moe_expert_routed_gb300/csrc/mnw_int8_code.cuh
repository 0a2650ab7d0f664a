// mnw_int8_code.cuh -- INT8 codes of values by their group's scale.
#pragma once

namespace mnw {

// clamp(rne(y / s)), s = max|y| / 127 of the group and rs = 1 / s.  y * rs is
// within 2^-16 of y / s (two roundings of a value below 128), so it rounds to
// the same integer unless it lies that close to a half; there, and where rs is
// infinite or y not finite, the division decides.
__device__ __forceinline__ int int8_code(float y, float s, float rs) {
  const float r = y * rs;
  const float n = rintf(r);
  if (fabsf(fabsf(r - n) - 0.5f) < 0x1p-14f || !(fabsf(r) < 128.f))
    return max(-127, min(127, __float2int_rn(__fdiv_rn(y, s))));
  return max(-127, min(127, static_cast<int>(n)));
}

}  // namespace mnw
