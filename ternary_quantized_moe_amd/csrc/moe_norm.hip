// The 8-bit quantizer and the residual RMS norm for gfx950.
//
// Both write e4m3 codes with one fp32 scale per block of 128: for a block whose
// largest magnitude is m, floored at 1e-30 so that neither the scale nor its
// reciprocal leaves the normal range,
//   scale = m / 448,   code = e4m3(v * (448 / m))   to nearest even.
// |v| (448 / m) is at most 448 (1 + 2^-23), which rounds to 448, so no code
// overflows.  A block with a NaN gets a NaN scale (magnitudes are compared as
// integers, in which a NaN is above every number).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.h"
#include "fp8_internal.h"
#include "wave_ops.h"

namespace moe {

namespace {

// Largest of an unsigned value over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, (uint32_t)dpp_row_i32<kDppXor1>((int)v));
  v = max(v, (uint32_t)dpp_row_i32<kDppXor2>((int)v));
  v = max(v, (uint32_t)dpp_row_i32<kDppHalfMirror>((int)v));
  return max(v, (uint32_t)dpp_row_i32<kDppMirror>((int)v));
}

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

template <bool F16>
__device__ __forceinline__ void widen8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = F16 ? f16_to_f32(v[i] & 0xFFFFu) : __uint_as_float(v[i] << 16);
    f[2 * i + 1] = F16 ? f16_to_f32(v[i] >> 16) : __uint_as_float(v[i] & 0xFFFF0000u);
  }
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

// A launch holds fewer than 2^32 threads along x: more blocks than 2^20 go on along y.
dim3 grid_of(int64_t blocks) {
  const int64_t x = blocks < 1 << 20 ? blocks : 1 << 20;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t block_number() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// ------------------------------------------------------------------ quantizer
constexpr int kQThreads = 256;

// One scale per row and group of 128: 16 lanes hold a group, eight values each.
// Bound by HBM for many rows: 16384 x 2048 takes 16.8 us (6.0 TB/s with what the
// Infinity Cache holds of it), 4096 x 2048 6.2 us (4.1 TB/s); 64 x 4096 is one
// launch, 2.3 us.
template <bool F16>
__global__ __launch_bounds__(kQThreads) void fp8_quantize_rows_kernel(const u32x4* __restrict__ x, int64_t n8,
                                                                      u32x2* __restrict__ q,
                                                                      float* __restrict__ scales) {
  const int64_t i = block_number() * kQThreads + threadIdx.x;
  if (i >= n8) return;  // n8 is a multiple of 16: whole groups leave together
  float f[8];
  widen8<F16>(x[i], f);
  const float m = floor_amax(row_max_u32(amax8(f)));
  q[i] = codes8(f, kE4m3Max / m);
  if ((i & 15) == 0) scales[i >> 4] = m / kE4m3Max;
}

// One scale per 128 x 128 block: a block of threads holds it in registers, so it is
// read once.  Bound by HBM: 50304 x 2048 takes 54.4 us, 5.7 TB/s with what the
// Infinity Cache still holds of it.
template <bool F16>
__global__ __launch_bounds__(kQThreads) void fp8_quantize_tiles_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                       int cols, uint8_t* __restrict__ q,
                                                                       float* __restrict__ scales) {
  constexpr int PER = kF8Group * kF8Group / 8 / kQThreads;  // 16-byte pieces per thread
  __shared__ uint32_t part[kQThreads / 64];
  const int groups = cols / kF8Group;
  const int64_t block = block_number(), rb = block / groups;
  if (rb * kF8Group >= rows) return;
  const int g = (int)(block - rb * groups);
  const int c = threadIdx.x & 15;
  const int64_t r0 = rb * kF8Group + (threadIdx.x >> 4);
  float f[PER][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t r = r0 + i * (kQThreads / 16);
    u32x4 v = {0, 0, 0, 0};
    if (r < rows) v = *(const u32x4*)(x + r * cols + g * kF8Group + 8 * c);
    widen8<F16>(v, f[i]);
    m = max(m, amax8(f[i]));
  }
  m = row_max_u32(m);
  m = max(max((uint32_t)__builtin_amdgcn_readlane((int)m, 0), (uint32_t)__builtin_amdgcn_readlane((int)m, 16)),
          max((uint32_t)__builtin_amdgcn_readlane((int)m, 32), (uint32_t)__builtin_amdgcn_readlane((int)m, 48)));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 64; ++w) m = max(m, part[w]);
  const float a = floor_amax(m), inv = kE4m3Max / a;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t r = r0 + i * (kQThreads / 16);
    if (r < rows) *(u32x2*)(q + r * cols + g * kF8Group + 8 * c) = codes8(f[i], inv);
  }
  if (threadIdx.x == 0) scales[rb * groups + g] = a / kE4m3Max;
}

// ------------------------------------------------------------------ RMS norm
// y = h / sqrt(mean(h^2) + eps) * g with h = x + residual in fp32.  One block
// per row; thread t holds values 8 (t + i threads) .. + 7, so 16 lanes of a DPP
// row hold one group of 128.  The row is read once, before anything is written,
// so the outputs may be the inputs.  Bound by HBM: 16384 x 2048 with a residual
// to codes and the sum takes 39.8 us, 5.9 TB/s likewise; one row 2.3 us.
template <int VPT>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a) {
  __shared__ float part[16];
  const int64_t token = block_number(), row = token * a.d;
  if (token >= a.T) return;
  const int threads = blockDim.x, n8 = a.d / 8;
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int p = threadIdx.x + i * threads;
    u32x4 v = {0, 0, 0, 0};
    if (p < n8) v = *(const u32x4*)(a.x + row + 8 * p);
    widen8<false>(v, h[i]);
    if (a.residual) {
      float r[8];
      u32x4 w = {0, 0, 0, 0};
      if (p < n8) w = *(const u32x4*)(a.residual + row + 8 * p);
      widen8<false>(w, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += r[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) ss += __shfl_xor(ss, o, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
  __syncthreads();
  ss = part[0];
  for (int w = 1; w < threads / 64; ++w) ss += part[w];
  const float rs = 1.0f / sqrtf(ss / (float)a.d + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int p = threadIdx.x + i * threads;
    if (p >= n8) continue;  // d is a multiple of 128: whole groups stay together
    if (a.sum)
      *(u32x4*)(a.sum + row + 8 * p) = u32x4{f32x2_to_bf16x2(h[i][0], h[i][1]), f32x2_to_bf16x2(h[i][2], h[i][3]),
                                             f32x2_to_bf16x2(h[i][4], h[i][5]), f32x2_to_bf16x2(h[i][6], h[i][7])};
    const f32x4 g0 = *(const f32x4*)(a.weight + 8 * p), g1 = *(const f32x4*)(a.weight + 8 * p + 4);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rs * (j < 4 ? g0[j & 3] : g1[j & 3]);
    if (a.y)
      *(u32x4*)(a.y + row + 8 * p) = u32x4{f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]),
                                           f32x2_to_bf16x2(y[4], y[5]), f32x2_to_bf16x2(y[6], y[7])};
    if (a.q) {
      const float m = floor_amax(row_max_u32(amax8(y)));
      *(u32x2*)(a.q + row + 8 * p) = codes8(y, kE4m3Max / m);
      if ((p & 15) == 0) a.scales[(row + 8 * p) / kF8Group] = m / kE4m3Max;
    }
  }
}

}  // namespace

hipError_t launch_fp8_quantize(bool f16, const uint16_t* x, int64_t rows, int cols, int block_rows, uint8_t* q,
                               float* scales, hipStream_t stream) {
  if (block_rows == 1) {
    const int64_t n8 = rows * (int64_t)cols / 8;
    const dim3 blocks = grid_of((n8 + kQThreads - 1) / kQThreads);
    auto kernel = f16 ? fp8_quantize_rows_kernel<true> : fp8_quantize_rows_kernel<false>;
    kernel<<<blocks, kQThreads, 0, stream>>>((const u32x4*)x, n8, (u32x2*)q, scales);
  } else {
    const dim3 blocks = grid_of((rows + kF8Group - 1) / kF8Group * (cols / kF8Group));
    auto kernel = f16 ? fp8_quantize_tiles_kernel<true> : fp8_quantize_tiles_kernel<false>;
    kernel<<<blocks, kQThreads, 0, stream>>>(x, rows, cols, q, scales);
  }
  return hipGetLastError();
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
  const int n8 = a.d / 8;
  const int threads = std::min(1024, (n8 + 63) / 64 * 64);
  const int vpt = (n8 + threads - 1) / threads;
  auto kernel = vpt == 1 ? rms_norm_kernel<1> : vpt == 2 ? rms_norm_kernel<2> : rms_norm_kernel<4>;
  kernel<<<grid_of(a.T), threads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
