// e4m3 codes from fp32 values and a block's floored magnitude (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "fp8_internal.h"

namespace moe {

// Four fp32 values -> four e4m3 codes (low byte first).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// The floored block magnitude: a NaN stays a NaN.
__device__ __forceinline__ float floor_amax(uint32_t bits) {
  const float m = __uint_as_float(bits);
  return m < kAmaxFloor ? kAmaxFloor : m;
}

// Largest magnitude of eight values as the bits of an fp32 number.
__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ u32x2 codes8(const float (&f)[8], float r) {
  return u32x2{pack_e4m3(f[0] * r, f[1] * r, f[2] * r, f[3] * r), pack_e4m3(f[4] * r, f[5] * r, f[6] * r, f[7] * r)};
}

}  // namespace moe
