// Device helpers of the attention kernels: matrix-core wrappers for 16-bit values of
// either kind, their conversion from fp32, and LDS reads that transpose.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "wave_ops.h"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// 16-bit values of one kind: their products, their rounding (nearest even) and the bits
// that all are set in an infinity or a NaN.
template <bool F16>
struct Half {
  static constexpr uint32_t kExponent = F16 ? 0x7C00 : 0x7F80;
  // The weights of a softmax are formed as 2^(s - m), m = the largest s so far - kLift, and that
  // may lag kLag behind: the largest is 2^kLift to 2^(kLift + kLag).  fp16 holds up to 2^16 and
  // loses bits below 2^-14, so its weights stand high in that range: those below 2^-21 of the
  // largest are off by 2^-32 of it at most (without the lift, 2^-14 and 2^-25: 16384 keys of
  // 2^-25 each beside one of 1 were lost, 2^-11 of the sum).
  static constexpr float kLift = F16 ? 7.f : 0.f, kLag = 8.f;
  // The logarithm of the sum of the weights 2^(s - m), base e.
  static __device__ __forceinline__ float log_of_sum(float m, float sum) {
    return sum == 0.f ? -INFINITY : (m + kLift) * kLn2 + logf(sum * (F16 ? 0x1p-7f : 1.f));
  }
  // D = A(32 x 16) B(16 x 32) + C.  Lane l supplies row l % 32 of A and column l % 32 of
  // B, k 8 (l / 32) .. + 7; it holds column l % 32 of D, row 8 (i / 4) + 4 (l / 32) + i % 4 in element i.
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (F16)
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                    0, 0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                     0, 0, 0);
  }
  // D = A(16 x 32) B(32 x 16) + C.  Lane l supplies row l % 16 of A and column l % 16 of B,
  // k 8 (l / 16) .. + 7; it holds column l % 16 of D, row 4 (l / 16) + i in element i.
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (F16)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                    0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                     0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    if constexpr (F16)
      return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, f16x2_t));
    else
      return f32x2_to_bf16x2(lo, hi);
  }
  static __device__ __forceinline__ float widen(uint32_t bits) {
    return F16 ? f16_to_f32(bits & 0xFFFFu) : __uint_as_float(bits << 16);
  }
};

// The other half of the wave: both halves' values of v, the lower lanes' first.
__device__ __forceinline__ f32x2_t both_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f32x2_t{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// Sums over the lanes up to each.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += shifted<kDppShr1, 0xF>(v);
  v += shifted<kDppShr2, 0xF>(v);
  v += shifted<kDppShr4, 0xF>(v);
  v += shifted<kDppShr8, 0xF>(v);
  v += shifted<kDppBcast15, 0xA>(v);
  return v + shifted<kDppBcast31, 0xC>(v);
}

// a / b, in 32 bits where these do.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Reads four rows of 16 values transposed: within 16 lanes, lane i gives the address of
// values 4 (i % 4) .. + 3 of row i / 4 and gets value i of the four rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)(p)));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, -1, 0x00027000);
}
// 16 bytes a lane to LDS, lane after lane from dst on.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t src, uint32_t lane_off, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16, (int)lane_off, 0, 0, 0);
}

}  // namespace moe
