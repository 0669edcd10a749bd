// The sampler for gfx950: temperature, top-k, top-p and min-p from a given
// uniform number per row.
//
// The tokens of a row are ordered by falling logit, equal logits by rising
// index; token i weighs w_i = exp((l_i - l_max) / T).  Every filter keeps a
// prefix of that order: top-k the first k; top-p the shortest prefix that holds
// top_p of the mass the top-k left; min-p the tokens with w_i >= min_p.  The
// answer is the first token whose cumulative weight exceeds u times the mass of
// what is left.
//
// Weights are evaluated in fp64 and summed as 64-bit integers in units of
// 2^-42 of the largest, so the sums do not depend on their order and a decision
// is the same for every launch shape; a token below half a unit (e^-29.8 of the
// most likely one) has no mass.  Up to 2^21 tokens a sum stays below 2^63.
//
// A place in the order is found by radix descent on the logits' ordered bits,
// 11 + 11 + 10 of them: a histogram of counts and masses over the digit of the
// tokens that share the higher digits, a scan from the top, and the digit where
// the target is reached.  After three digits the logit is exact, its tokens
// weigh the same, and the place among them is a division.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "fp8_internal.h"

namespace moe {

namespace {

constexpr int kSampThreads = 1024;
constexpr int kSampWaves = kSampThreads / 64;
constexpr int kRadix = 2048;
constexpr double kMassUnit = 4398046511104.0;  // 2^42

template <int TYPE>
struct Logit;
template <>
struct Logit<kSampleF32> {
  typedef float T;
  static __device__ __forceinline__ float f32(float v) { return v; }
};
template <>
struct Logit<kSampleBf16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float f32(uint16_t v) { return bf16_to_f32(v); }
};
template <>
struct Logit<kSampleF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float f32(uint16_t v) { return f16_to_f32(v); }
};

// Ordered bits of a logit: larger logits have larger keys, -0 the key of +0 and
// a NaN that of -inf.
__device__ __forceinline__ uint32_t key_of(float v) {
  v = v != v ? -__builtin_inff() : v + 0.0f;
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

struct Weigher {
  double top, t;
  uint32_t top_key;
  __device__ __forceinline__ double weight(uint32_t key) const {
    return key == top_key ? 1.0 : key == kKeyNegInf ? 0.0 : exp(((double)logit_of(key) - top) / t);
  }
  __device__ __forceinline__ uint64_t mass(uint32_t key) const {
    return (uint64_t)(weight(key) * kMassUnit + 0.5);
  }
};

// The tokens up to a place in the order: keys above `key`, and at `key` the
// indices up to `last`; of those the ones with weight >= floor.
struct Prefix {
  uint32_t key;
  int last;
  double floor;
  __device__ __forceinline__ bool has(uint32_t k, int i) const { return k > key || (k == key && i <= last); }
};

struct Shared {
  uint32_t count[kRadix];
  uint64_t mass[kRadix];
  uint64_t wave_mass[kSampWaves];
  uint32_t wave_count[kSampWaves];
  uint64_t before_mass;
  uint32_t before_count, digit;
  int found;
};

__device__ __forceinline__ uint64_t scan_u64(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t t = __shfl_up(v, o, 64);
    if (lane >= o) v += t;
  }
  return v;
}
__device__ __forceinline__ uint32_t scan_u32(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t t = __shfl_up(v, o, 64);
    if (lane >= o) v += t;
  }
  return v;
}

template <int TYPE>
struct Row {
  typedef Logit<TYPE> L;
  const typename L::T* p;
  int V;
  Shared& s;
  __device__ __forceinline__ uint32_t key(int i) const { return key_of(L::f32(p[i])); }

  // The largest key and the lowest index that has it.
  __device__ void top(uint32_t& key_out, int& index_out) {
    uint64_t best = 0;  // key, then the complement of the index
    for (int i = threadIdx.x; i < V; i += kSampThreads) {
      const uint64_t v = (uint64_t)key(i) << 32 | (uint32_t)~i;
      best = v > best ? v : best;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      const uint64_t v = __shfl_xor(best, o, 64);
      best = v > best ? v : best;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.wave_mass[threadIdx.x >> 6] = best;
    __syncthreads();
    for (int w = 0; w < kSampWaves; ++w) best = s.wave_mass[w] > best ? s.wave_mass[w] : best;
    key_out = (uint32_t)(best >> 32);
    index_out = (int)~(uint32_t)best;
  }

  // Mass of a prefix's tokens with weight >= floor.
  __device__ uint64_t total(const Weigher& w, const Prefix& in) {
    uint64_t m = 0;
    for (int i = threadIdx.x; i < V; i += kSampThreads) {
      const uint32_t k = key(i);
      if (in.has(k, i)) {
        const double x = w.weight(k);
        if (x >= in.floor || k == w.top_key) m += (uint64_t)(x * kMassUnit + 0.5);
      }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) m += __shfl_xor(m, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.wave_mass[threadIdx.x >> 6] = m;
    __syncthreads();
    m = 0;
    for (int i = 0; i < kSampWaves; ++i) m += s.wave_mass[i];
    return m;
  }

  // The place in the order where `target` (>= 1) is reached among the tokens of
  // `in`: the target-th token (COUNT) or the first with cumulative mass >=
  // target.  The target is at most the prefix's whole count or mass.
  template <bool COUNT>
  __device__ Prefix find(const Weigher& w, const Prefix& in, uint64_t target) {
    uint32_t prefix = 0;
    uint64_t before_mass = 0;
    uint32_t before_count = 0, ties = 0;
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const uint32_t digits = level == 2 ? 1024u : 2048u;
      for (int b = threadIdx.x; b < kRadix; b += kSampThreads) {
        s.count[b] = 0;
        s.mass[b] = 0;
      }
      if (threadIdx.x == 0) s.digit = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < V; i += kSampThreads) {
        const uint32_t k = key(i);
        if (level && (level == 1 ? k >> 21 : k >> 10) != prefix) continue;
        if (!in.has(k, i)) continue;
        const uint32_t b = digits - 1 - ((k >> shift) & (digits - 1));  // larger keys first
        atomicAdd(&s.count[b], 1u);
        if (!COUNT) {
          const double x = w.weight(k);
          if (x >= in.floor || k == w.top_key)
            atomicAdd((unsigned long long*)&s.mass[b], (unsigned long long)(x * kMassUnit + 0.5));
        }
      }
      __syncthreads();
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b0 = 2 * threadIdx.x;
      const uint32_t c0 = s.count[b0], c1 = s.count[b0 + 1];
      const uint64_t m0 = s.mass[b0], m1 = s.mass[b0 + 1];
      uint32_t ci = scan_u32(c0 + c1, lane);
      uint64_t mi = scan_u64(m0 + m1, lane);
      if (lane == 63) {
        s.wave_count[wave] = ci;
        s.wave_mass[wave] = mi;
      }
      __syncthreads();
      for (int i = 0; i < wave; ++i) {
        ci += s.wave_count[i];
        mi += s.wave_mass[i];
      }
      const uint32_t ce = before_count + ci - c0 - c1;
      const uint64_t me = before_mass + mi - m0 - m1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t cb = h ? ce + c0 : ce, c = h ? c1 : c0;
        const uint64_t mb = h ? me + m0 : me, m = h ? m1 : m0;
        if (COUNT ? (cb < target && cb + (uint64_t)c >= target) : (mb < target && mb + m >= target)) {
          s.digit = digits - 1 - (uint32_t)(b0 + h);
          s.before_count = cb;
          s.before_mass = mb;
          s.found = (int)c;
        }
      }
      __syncthreads();
      prefix = level == 0 ? s.digit : level == 1 ? prefix << 11 | s.digit : prefix << 10 | s.digit;
      before_count = s.before_count;
      before_mass = s.before_mass;
      ties = (uint32_t)s.found;
      __syncthreads();
    }
    // `ties` tokens have the key `prefix`: the place is the nth of them
    uint32_t nth;
    if (COUNT) {
      nth = (uint32_t)target - before_count;
    } else {
      const uint64_t m = w.mass(prefix), need = target - before_mass;
      nth = (uint32_t)((need + m - 1) / m);
    }
    (void)ties;
    Prefix out;
    out.key = prefix;
    out.floor = in.floor;
    out.last = nth_at(prefix, nth);
    return out;
  }

  // The index of the nth (>= 1) token with this key, by rising index.
  __device__ int nth_at(uint32_t k, uint32_t nth) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) s.found = V - 1;
    uint32_t seen = 0;
    for (int i0 = 0; i0 < V; i0 += kSampThreads) {
      const int i = i0 + threadIdx.x;
      const bool hit = i < V && key(i) == k;
      const uint64_t votes = __ballot(hit);
      __syncthreads();
      if (lane == 0) s.wave_count[wave] = (uint32_t)__popcll(votes);
      __syncthreads();
      uint32_t before = seen, all = 0;
      for (int w = 0; w < kSampWaves; ++w) {
        if (w < wave) before += s.wave_count[w];
        all += s.wave_count[w];
      }
      before += (uint32_t)__popcll(votes & ((1ull << lane) - 1));
      if (hit && before + 1 == nth) s.found = i;
      seen += all;
      if (seen >= nth) break;
    }
    __syncthreads();
    const int f = s.found;
    __syncthreads();
    return f;
  }
};

template <int TYPE>
__global__ __launch_bounds__(kSampThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared s;
  typedef Logit<TYPE> L;
  const int64_t b = blockIdx.x;
  Row<TYPE> row{(const typename L::T*)a.logits + b * a.ld, a.V, s};
  Weigher w;
  int token;
  row.top(w.top_key, token);
  w.top = (double)logit_of(w.top_key);
  w.t = a.temperature ? (double)a.temperature[b] : 1.0;
  double prob = 1.0;
  if (w.top_key == kKeyNegInf) {
    token = -1;
    prob = 0.0;
  } else if (w.t > 0.0) {
    Prefix keep{0, a.V - 1, 0.0};
    const int k = a.top_k ? a.top_k[b] : 0;
    if (k > 0 && k < a.V) keep = row.template find<true>(w, keep, (uint64_t)k);
    const double p = a.top_p ? (double)a.top_p[b] : 1.0;
    if (p < 1.0) {
      const uint64_t all = row.total(w, keep);
      const double x = ceil(p * (double)all);
      keep = row.template find<false>(w, keep, x >= 1.0 ? (uint64_t)x : 1);
    }
    const double mp = a.min_p ? (double)a.min_p[b] : 0.0;
    if (mp > 0.0) keep.floor = mp;
    const uint64_t all = row.total(w, keep);
    const double x = floor((double)a.u[b] * (double)all) + 1.0;
    const uint64_t target = x >= (double)all ? all : x >= 1.0 ? (uint64_t)x : 1;
    const Prefix at = row.template find<false>(w, keep, target);
    token = at.last;
    prob = w.weight(at.key) / ((double)all / kMassUnit);
  }
  if (threadIdx.x == 0) {
    a.tokens[b] = token;
    if (a.probs) a.probs[b] = (float)prob;
  }
}

}  // namespace

int64_t sample_workspace_bytes(int64_t B, int V) {
  (void)B;
  (void)V;
  return 0;
}

hipError_t launch_sample(SampleType type, const SampleArgs& a, void* ws, hipStream_t stream) {
  (void)ws;
  auto kernel = type == kSampleF32 ? sample_kernel<kSampleF32> : type == kSampleBf16 ? sample_kernel<kSampleBf16>
                                                                                     : sample_kernel<kSampleF16>;
  kernel<<<(unsigned)a.B, kSampThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
