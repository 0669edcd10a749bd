// Block-scaled 8-bit product for gfx950:
//   y[t, n] = sum over groups g of 128 of  sa[t, g] sw[n / 128, g] S(t, n, g),
//   S(t, n, g) = sum over k in g of a[t, k] w[n, k]
// with e4m3 a and w.  The scales are fp32 and differ per token, so each S is a
// matrix-core sum of its own, scaled and added in fp32 outside.  Tokens sit on
// the matrix core's columns: a lane's results belong to one token and, a 16-row
// tile lying inside one 128-row block of w, share one scale product.
//
// Two ways to form S, chosen by the output's type:
//   bf16  v_mfma_f32_16x16x128_f8f6f4.  It adds eight neighbouring products at a
//         time after cutting them at 2^-13 of the largest of the eight (measured:
//         a product 2^-13 of the largest counts, one of 2^-14 does not), then
//         adds in fp32: at most 7 2^-13 of that largest product is lost per eight.
//         On normal data S is off by 1.6e-5 of its size, a hundredth of the
//         output's own rounding.
//   fp32  e4m3 widened to bf16 (exact) and v_mfma_f32_16x16x32_bf16, whose products
//         are exact and whose sums are fp32 (4e-9 on the same data), at half the
//         matrix rate.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "fp8_internal.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// D = A(16 x 128) B(128 x 16), fp32, both operands e4m3.  Lane l supplies row
// l % 16 of A and column l % 16 of B; the order of K inside the group is free
// as long as both operands use the same one.
__device__ __forceinline__ f32x4 mfma_f8_16(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Lane quarter q's 32 bytes of one group: bytes 16 q .. + 15 and 64 + 16 q .. + 15.
__device__ __forceinline__ i32x8 load_frag(const uint8_t* row, int q) {
  const u32x4 lo = *(const u32x4*)(row + 16 * q), hi = *(const u32x4*)(row + 64 + 16 * q);
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Four e4m3 codes -> four bf16 (exact).
__device__ __forceinline__ u32x2 widen_f8x4(int v) {
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true))};
}

// One lane's 32 values of a group as the matrix cores take them.
template <bool F32>
struct Frag {
  i32x8 v;
  __device__ __forceinline__ void set(i32x8 codes) { v = codes; }
};
template <>
struct Frag<true> {
  u32x4 v[4];
  __device__ __forceinline__ void set(i32x8 codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x2 lo = widen_f8x4(codes[2 * i]), hi = widen_f8x4(codes[2 * i + 1]);
      v[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
};
__device__ __forceinline__ f32x4 group_product(const Frag<false>& w, const Frag<false>& a) {
  return mfma_f8_16(w.v, a.v, f32x4{0.f, 0.f, 0.f, 0.f});
}
__device__ __forceinline__ f32x4 group_product(const Frag<true>& w, const Frag<true>& a) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = mfma16(w.v[i], a.v[i], s);
  return s;
}

constexpr int kLinThreads = 256;

// 64 rows of w (16 a wave) and 64 tokens per block.
template <bool F32>
__global__ __launch_bounds__(kLinThreads) void fp8_linear_kernel(F8LinearArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 64 + 16 * wave, m0 = (int64_t)blockIdx.y * 64;
  if (n0 >= p.N) return;
  const int groups = p.K / kF8Group;
  const uint8_t* w = p.w + min(n0 + c, p.N - 1) * p.K;
  const float* sw = p.w_scales + n0 / kF8Group * groups;
  const uint8_t* a[4];
  const float* sa[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = min(m0 + 16 * i + c, p.M - 1);
    a[i] = p.a + t * p.K;
    sa[i] = p.a_scales + t * groups;
  }
  f32x4 acc[4] = {};
  for (int g = 0; g < groups; ++g) {
    Frag<F32> wf, af;
    wf.set(load_frag(w + g * kF8Group, q));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      af.set(load_frag(a[i] + g * kF8Group, q));
      const f32x4 s = group_product(wf, af);
      const float f = sa[i][g] * sw[g];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += s[j] * f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = m0 + 16 * i + c, n = n0 + 4 * q;
    if (t >= p.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= p.N) continue;
      if (F32) ((float*)p.y)[t * p.ldy + n + j] = acc[i][j];
      else ((uint16_t*)p.y)[t * p.ldy + n + j] = (uint16_t)f32_to_bf16(acc[i][j]);
    }
  }
}

}  // namespace

hipError_t launch_fp8_linear(const F8LinearArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64));
  auto kernel = a.f32 ? fp8_linear_kernel<true> : fp8_linear_kernel<false>;
  kernel<<<grid, kLinThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
