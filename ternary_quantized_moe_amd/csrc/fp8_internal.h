// Internal interface of the operators between a residual stream and the next
// token: the e4m3 quantizer, the residual RMS norm, the block-scaled product
// and the sampler.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kF8Group = 128;            // values per scale along a row
constexpr float kE4m3Max = 448.0f;       // largest e4m3 value
constexpr float kAmaxFloor = 1e-30f;     // keeps a block's scale and its reciprocal normal numbers
constexpr int kNormMaxD = 32768;         // widest row the norm keeps in registers
constexpr int kLinearMaxK = 1 << 22;     // 256 rows of it stay inside 32 bits
constexpr int64_t kLinearMaxOut = (int64_t)1 << 37;  // with m, n <= 2^29 a launch of fewer than 2^32 threads
constexpr int64_t kSampleMaxVocab = 1 << 21, kSampleMaxBatch = 1 << 22;  // at most 2^30 chunks of a row

// e4m3 codes and scales of a [rows x cols] bf16 (f16 = false) or fp16 matrix,
// one scale per block_rows (1 or 128) x 128 block.
hipError_t launch_fp8_quantize(bool f16, const uint16_t* x, int64_t rows, int cols, int block_rows, uint8_t* q,
                               float* scales, hipStream_t stream);

struct NormArgs {
  const uint16_t* x;         // bf16 [T x d]
  const uint16_t* residual;  // bf16 [T x d] or NULL
  int64_t T;
  int d;
  const float* weight;       // [d]
  float eps;
  uint16_t* sum;             // bf16 x + residual, or NULL
  uint16_t* y;               // bf16, or NULL
  uint8_t* q;                // e4m3 with scales [T x d / 128], or NULL
  float* scales;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

struct F8LinearArgs {
  const uint8_t* a;       // e4m3 [M x K]
  const float* a_scales;  // [M x K / 128]
  int64_t M;
  const uint8_t* w;       // e4m3 [N x K]
  const float* w_scales;  // [ceil(N / 128) x K / 128]
  int64_t N;
  int K;
  bool f32;               // y is fp32 (else bf16)
  void* y;                // [M x ldy]
  int64_t ldy;
};
hipError_t launch_fp8_linear(const F8LinearArgs& a, hipStream_t stream);

enum SampleType { kSampleF32 = 0, kSampleBf16 = 1, kSampleF16 = 2 };
struct SampleArgs {
  const void* logits;  // [B x V], row stride ld elements
  int64_t B;
  int V;
  int64_t ld;
  const float* temperature;  // per row, or NULL (1)
  const int32_t* top_k;      // per row, or NULL (off)
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* tokens;
  float* probs;              // or NULL
};
int64_t sample_workspace_bytes(int64_t B, int V);
hipError_t launch_sample(SampleType type, const SampleArgs& a, void* ws, hipStream_t stream);

}  // namespace moe
