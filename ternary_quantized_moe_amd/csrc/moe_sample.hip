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
// Weights are evaluated in fp64 and summed as 64-bit integers, in units of 2^-35
// relative to a bin of 1 / 16 nat; the bins' sums are added in fp64 in one fixed
// order.
// Two launches.  The scan reads the logits once (HBM floor 6.5 us at 64 x 131072
// fp32, 14.6 us measured: some 30 vector instructions a token for its bin, weight and
// place bound it beside the read) and leaves 512-bin histograms and lists of
// tokens by bin; the choice works on those alone (22.8 us there, one block a row:
// a chain of dependent steps, each a memory's or a barrier's latency; 12.0 us for
// 1 x 50304).
//
// Rows off the grid of bins (an infinite logit, l / T beyond some 2^18) take radix descents on the logits' ordered bits,
// 11 + 11 + 10 of them, with units of 2^-42 of the largest weight: a histogram of
// counts and masses over the digit of the tokens that share the higher digits, a
// scan from the top, and the digit where the target is reached.  After three digits
// the logit is exact, its tokens weigh the same, and the place among them is a
// division.  One block re-reads its row for each digit: 64 x 131072 with top-p takes
// 690 us there (11 on the grid).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "fp8_internal.h"

namespace moe {

namespace {

constexpr int kSampThreads = 512;  // two blocks a CU, as registers and LDS allow
constexpr int kSampWaves = kSampThreads / 64;
constexpr int kRadix = 2048;
constexpr double kMassUnit = 4398046511104.0;  // 2^42

template <int TYPE>
struct Logit;
template <>
struct Logit<kSampleF32> {
  typedef float T;
  static constexpr int kDead = 0;  // low bits of an ordered key that say nothing
  static __device__ __forceinline__ float f32(float v) { return v; }
};
template <>
struct Logit<kSampleBf16> {
  typedef uint16_t T;
  static constexpr int kDead = 16;
  static __device__ __forceinline__ float f32(uint16_t v) { return bf16_to_f32(v); }
};
template <>
struct Logit<kSampleF16> {
  typedef uint16_t T;
  static constexpr int kDead = 13;
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

// A step of a scan over a wave: combine(v, w) where w is v of the lane that the step
// looks back at, or `none`.  Six of them, without a trip through LDS.
template <class V, class Combine>
__device__ __forceinline__ V scan_wave(V v, V none, Combine combine) {
  union Bits {
    V v;
    int w[sizeof(V) / 4];
  };
  auto step = [&](auto ctrl, auto rows) {
    Bits in, out;
    in.v = v;
    out.v = none;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(V) / 4); ++i)
      out.w[i] = __builtin_amdgcn_update_dpp(out.w[i], in.w[i], decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    v = combine(v, out.v);
  };
  typedef std::integral_constant<int, 0xF> All;
  step(std::integral_constant<int, 0x111>(), All());  // row_shr:1, 2, 4, 8: rows of 16
  step(std::integral_constant<int, 0x112>(), All());
  step(std::integral_constant<int, 0x114>(), All());
  step(std::integral_constant<int, 0x118>(), All());
  step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xA>());  // lane 15 of a row to the next
  step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xC>());  // lane 31 to the upper half
  return v;
}
template <class V>
__device__ __forceinline__ V scan_sum(V v) {
  return scan_wave(v, (V)0, [](V a, V b) { return a + b; });
}
__device__ __forceinline__ uint64_t last_lane(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), 63) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t wave_max(uint64_t v) { return last_lane(scan_wave(v, (uint64_t)0, max_u64)); }

template <int TYPE>
struct Row {
  typedef Logit<TYPE> L;
  const typename L::T* p;
  int V;
  Shared& s;
  __device__ __forceinline__ uint32_t key(int i) const { return key_of(L::f32(p[i])); }

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
    uint32_t before_count = 0;
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
      constexpr int PER = kRadix / kSampThreads;
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b0 = PER * threadIdx.x;
      uint32_t c = 0;
      uint64_t m = 0;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        c += s.count[b0 + h];
        m += s.mass[b0 + h];
      }
      uint32_t ci = scan_sum(c);
      uint64_t mi = scan_sum(m);
      if (lane == 63) {
        s.wave_count[wave] = ci;
        s.wave_mass[wave] = mi;
      }
      __syncthreads();
      for (int i = 0; i < wave; ++i) {
        ci += s.wave_count[i];
        mi += s.wave_mass[i];
      }
      uint32_t cb = before_count + ci - c;
      uint64_t mb = before_mass + mi - m;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        c = s.count[b0 + h];
        m = s.mass[b0 + h];
        if (COUNT ? (cb < target && cb + (uint64_t)c >= target) : (mb < target && mb + m >= target)) {
          s.digit = digits - 1 - (uint32_t)(b0 + h);
          s.before_count = cb;
          s.before_mass = mb;
        }
        cb += c;
        mb += m;
      }
      __syncthreads();
      prefix = level == 0 ? s.digit : level == 1 ? prefix << 11 | s.digit : prefix << 10 | s.digit;
      before_count = s.before_count;
      before_mass = s.before_mass;
      __syncthreads();
    }
    // the place is the nth of the tokens with the key `prefix`
    uint32_t nth;
    if (COUNT) {
      nth = (uint32_t)target - before_count;
    } else {
      const uint64_t m = w.mass(prefix), need = target - before_mass;
      nth = (uint32_t)((need + m - 1) / m);
    }
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

// The first of `all` units (from 1) with which a mass reaches `target` (`over`: exceeds
// it); the last one if none does.  A whole number of units above 2^53 has no room for
// one more in a double.
__device__ __forceinline__ uint64_t first_unit(double target, bool over, uint64_t all) {
  if (target >= (double)all) return all;
  if (!(target > 0.0)) return 1;
  const uint64_t n = over ? (uint64_t)target + 1 : (uint64_t)ceil(target);
  return n < all ? n : all;
}

// The whole row by radix descents alone: right for every row, and taken where the
// histogram below does not hold the answer.
template <int TYPE>
__device__ void solve_by_radix(Row<TYPE>& row, Weigher& w, int k, double p, double mp, double u, int& token,
                               double& prob) {
  Prefix keep{0, row.V - 1, 0.0};
  if (k > 0 && k < row.V) keep = row.template find<true>(w, keep, (uint64_t)k);
  if (p < 1.0) {
    const uint64_t all = row.total(w, keep);
    keep = row.template find<false>(w, keep, first_unit(p * (double)all, false, all));
  }
  if (mp > 0.0) keep.floor = mp;
  const uint64_t all = row.total(w, keep);
  const uint64_t target = first_unit(u * (double)all, true, all);
  const Prefix at = row.template find<false>(w, keep, target);
  token = at.last;
  prob = w.weight(at.key) / ((double)all / kMassUnit);
}

// ------------------------------------------------------------------ histograms
// One read of the logits: blocks take a chunk of a row each, keep it in registers
// for its largest value, and count it into 512 bins of 1 / 16 nat below that, on a
// grid that all chunks of the row share: bin floor(16 l / T), in fp64 (in fp32 a
// rounding moves an edge by up to half a bin near 2^22, and the polynomial below is
// left to extrapolate: weights off by 6e-9).  A bin holds a count and a mass: the
// weight of a token relative to the bin's upper edge lies in (e^-1/16, 1] and
// becomes an integer of 35 bits, so a chunk's sums are exact in whatever order they
// come, count and mass in one 64-bit number.  32 nats below the chunk's largest value a token has no mass (2^-46 of it).
// The chunk's tokens are also written down by bin (their places in the chunk, in no
// order within a bin), so that whoever wants a bin's tokens need not search the row;
// with a top-k only as many bins as hold the chunk's own first k.
constexpr int kBins = 512;
constexpr double kPerNat = 16.0, kBinUnit = 34359738368.0;  // 2^35
constexpr int kCountShift = 50;                            // 2^13 tokens of about 2^35 below it
constexpr int kScanThreads = 256;
constexpr double kFarthestBin = 4194304.0;                 // 2^22: the places of tokens are good to 2^-31 of a bin up to it

// Whether a chunk with this top bin is counted, and whether a row with it is answered
// from its chunks' bins: all within its reach are counted then.
__device__ __forceinline__ bool chunk_on_grid(double edge) { return fabs(edge) <= kFarthestBin; }
__device__ __forceinline__ bool row_on_grid(double edge) { return edge >= kBins - kFarthestBin && edge <= kFarthestBin; }

struct ChunkHead {
  uint64_t top;  // largest key, then the complement of its lowest index
  double edge;   // number of the top bin
};

// l / T on the grid: the bin number, and the weight in units of 2^-35 relative to
// the bin's upper edge.
struct Grid {
  double per;  // 16 / T
  __device__ __forceinline__ explicit Grid(float t) : per(kPerNat / (double)t) {}
  __device__ __forceinline__ double bin(float l) const { return floor((double)l * per); }
  // Place in the bin, from 0 to 1: the product is not rounded again.
  __device__ __forceinline__ double in_bin(float l, double bin) const { return fma((double)l, per, -bin); }
  // COUNTED: with 2^50 on top.  The polynomial of degree 4 that meets
  // 2^35 e^((y - 1) / 16) at the Chebyshev nodes of y in [0, 1] is off by 0.52 units
  // at most.  Adding 2^52 leaves the rounded integer in a double's low bits and takes
  // the constant's 0.27 with it: 1.29 units in all, 4e-11 of the lightest weight.
  template <bool COUNTED>
  __device__ __forceinline__ uint64_t unit(float l, double bin) const {
    const double y = in_bin(l, bin);
    double e = 21174.08417495729;
    e = fma(e, y, 1312820.8186157919);
    e = fma(e, y, 63043148.908760265);
    e = fma(e, y, 2017374165.4019043);
    e = fma(e, y, 32277987058.26685 + 4503599627370496.0 + (COUNTED ? 1125899906842624.0 : 0.0));
    return (uint64_t)__double_as_longlong(e) & ~(0xFFFull << 52);
  }
};

// VE neighbouring logits of a row from index i on; past the row -inf.
template <int TYPE>
struct Vec {
  static constexpr int VE = TYPE == kSampleF32 ? 4 : 8;
  float v[VE];
  __device__ __forceinline__ void load(const void* row, int i, int V) {
    typedef typename Logit<TYPE>::T T;
    const T* p = (const T*)row + i;
    if (i + VE <= V) {
      if (TYPE == kSampleF32) {
        const u32x4_a4 w = *(const u32x4_a4*)p;
#pragma unroll
        for (int k = 0; k < VE; ++k) v[k] = __uint_as_float(w[k & 3]);
      } else {  // rows of 16-bit logits are only 2-byte aligned
        typedef u32x4 __attribute__((aligned(2))) u32x4_a2;
        const u32x4 w = *(const u32x4_a2*)p;
#pragma unroll
        for (int k = 0; k < VE; ++k) v[k] = Logit<TYPE>::f32((T)(w[(k / 2) & 3] >> (16 * (k & 1))));
      }
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) v[k] = i + k < V ? Logit<TYPE>::f32(p[k]) : -__builtin_inff();
    }
  }
};

// The workspace: one of each per chunk.
struct Chunks {
  int n, len;       // chunks of a row, tokens in a chunk
  ChunkHead* heads;
  uint64_t* hists;  // [kBins] count and units of each bin below the chunk's top one
  uint16_t* ends;   // [kBins] where a bin's tokens end among the chunk's
  uint16_t* tokens; // [len] places in the chunk, by bin
};

template <int TYPE, int PT>
__global__ __launch_bounds__(kScanThreads) void sample_scan_kernel(SampleArgs a, Chunks ws) {
  constexpr int VE = Vec<TYPE>::VE, N = PT / VE, LEN = kScanThreads * PT, WAVES = kScanThreads / 64;
  static_assert(kBins == 2 * kScanThreads, "two bins a thread");
  __shared__ uint64_t hist[kBins + 64];
  __shared__ uint32_t begin[kBins + 64];
  __shared__ float tops[WAVES];
  __shared__ uint32_t counts[WAVES];
  __shared__ int end_bin, end_count, top_index;
  __shared__ __attribute__((aligned(16))) uint16_t places[LEN + 64];
  const int64_t b = blockIdx.x / ws.n;
  const int chunk = (int)(blockIdx.x - b * ws.n), base = chunk * LEN, tid = threadIdx.x, lane = tid & 63;
  const void* row = (const typename Logit<TYPE>::T*)a.logits + b * a.ld;
  Vec<TYPE> x[N];
#pragma unroll
  for (int j = 0; j < N; ++j) x[j].load(row, base + (j * kScanThreads + tid) * VE, a.V);
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  const int k = a.top_k ? a.top_k[b] : 0;
  // the largest value, then the lowest index that has it; a comparison passes over every
  // NaN (a maximum answers a signalling one with a NaN)
  float mine = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) mine = x[j].v[e] > mine ? x[j].v[e] : mine;
  float top = mine;
  top = scan_wave(top, -__builtin_inff(), [](float p, float q) { return fmaxf(p, q); });
  if (lane == 63) tops[tid >> 6] = top;
  if (tid == 0) top_index = 0x7FFFFFFF;
  hist[tid] = 0;
  hist[tid + kScanThreads] = 0;
  __syncthreads();
  top = tops[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) top = fmaxf(top, tops[w]);
  if (mine == top) {
    int first = 0x7FFFFFFF;
#pragma unroll
    for (int j = N - 1; j >= 0; --j)
#pragma unroll
      for (int e = VE - 1; e >= 0; --e)
        if (x[j].v[e] == top) first = base + (j * kScanThreads + tid) * VE + e;
    atomicMin(&top_index, first);
  }
  const Grid grid(t);
  const double edge = grid.bin(top);
  const bool counted = t > 0.f && k != 1 && chunk_on_grid(edge);
  // the first token needs no histogram; a grid too far out is not exact
  if (counted) {
    // a token's value gives way to its seat: its bin and its number there.  What is too far below the top
    // has one in the bins behind, one for each lane of a wave
    const double nowhere = (double)(kBins + lane), edge52 = edge + 4503599627370496.0;  // 2^52: see below
#pragma unroll
    for (int j = 0; j < N; ++j) {
      uint32_t at[VE];
      uint64_t was[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float l = x[j].v[e];
        const double bin = grid.bin(l);
        // edge - bin as the low bits of a double; a NaN is passed over
        at[e] = (uint32_t)__double_as_longlong(fmin(edge52 - bin, nowhere + 4503599627370496.0));
        was[e] = atomicAdd((unsigned long long*)&hist[at[e]], (unsigned long long)grid.template unit<true>(l, bin));
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) x[j].v[e] = __uint_as_float(at[e] << 16 | (uint32_t)(was[e] >> kCountShift));
    }
  }
  __syncthreads();
  if (tid == 0) ws.heads[blockIdx.x] = ChunkHead{(uint64_t)key_of(top) << 32 | (uint32_t)~top_index, edge};
  if (!counted) return;
  const uint64_t h0 = hist[2 * tid], h1 = hist[2 * tid + 1];
  const uint32_t c0 = (uint32_t)(h0 >> kCountShift), c1 = (uint32_t)(h1 >> kCountShift);
  uint32_t ci = scan_sum(c0 + c1);
  if (lane == 63) counts[tid >> 6] = ci;
  if (tid == 0) end_bin = kBins;
  __syncthreads();
  for (int w = 0; w < tid >> 6; ++w) ci += counts[w];
  const uint32_t b1 = ci - c1, b0 = b1 - c0;
  begin[2 * tid] = b0;
  begin[2 * tid + 1] = b1;
  if (tid == kScanThreads - 1) end_count = (int)ci;
  __syncthreads();
  if (k > 0) {  // past the chunk's own first k nothing is the row's
    const uint32_t n = (uint32_t)k;
    if (b0 < n && b1 >= n) {
      end_bin = 2 * tid + 1;
      end_count = (int)b1;
    }
    if (b1 < n && ci >= n) {
      end_bin = 2 * tid + 2;
      end_count = (int)ci;
    }
  }
  const int64_t at = (int64_t)blockIdx.x * kBins + 2 * tid;
  *(u32x4*)(ws.hists + at) = u32x4{(uint32_t)h0, (uint32_t)(h0 >> 32), (uint32_t)h1, (uint32_t)(h1 >> 32)};
  *(uint32_t*)(ws.ends + at) = b1 | ci << 16;
  __syncthreads();
  const uint32_t limit = (uint32_t)end_bin << 16;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint32_t to[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) to[e] = begin[__float_as_uint(x[j].v[e]) >> 16];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const uint32_t seat = __float_as_uint(x[j].v[e]);
      places[seat < limit ? to[e] + (seat & 0xFFFFu) : LEN + lane] = (uint16_t)((j * kScanThreads + tid) * VE + e);
    }
  }
  __syncthreads();
  u32x4* out = (u32x4*)(ws.tokens + (int64_t)blockIdx.x * LEN);
  for (int i = tid; i < (end_count + 7) / 8; i += kScanThreads) out[i] = ((const u32x4*)places)[i];
}

// ------------------------------------------------------------------ the choice
// One block per row: the chunks' histograms added up say in which bin of the order
// each filter ends and the answer lies; a border bin's tokens are fetched from the
// chunks' lists.  A place within a bin is found among its tokens: each counts what
// stands before it, at most 128 of them; a fuller bin is first divided by the order
// of its tokens (logit, then index), 1024 ways.  Up to 4096 tokens are kept in LDS
// for that, more are read from the chunks' lists every time.  Only rows off the grid
// (an infinite logit, a temperature near 0) go through the radix descents.
constexpr int kList = 4096;  // tokens kept
constexpr int kPrefix = 1024;  // as many are fetched where later borders may need them
constexpr int kFew = 128, kPartBits = 10, kParts = 1 << kPartBits;
constexpr int kNearChunks = 32;  // of a row, for the ends of their bins to be in LDS
constexpr int kMaxChunks = (int)(kSampleMaxVocab / (kScanThreads * 32));

struct Pick {
  union {
    Shared radix;
    struct {
      uint64_t order[kList];
      uint64_t hist[kParts];
      uint32_t parts[kParts];
    } s;
  };
  struct __attribute__((aligned(16))) Few {
    uint64_t order, units;
  } few[kFew];
  uint32_t count[kBins];  // tokens in the bins up to and with this one
  double mass[kBins];     // and their mass, in units of the top bin
  double unit[kBins];     // a unit of mass of a bin, in units of the top bin
  uint64_t units[kBins];  // a bin's units
  uint64_t wave_u64[kSampWaves];
  double wave_f64[kSampWaves];
  uint32_t wave_u32[kSampWaves];
  short dist[kMaxChunks];    // bins between the row's top and a chunk's, kBins for a chunk out of reach
  uint64_t before, answer;
  uint32_t before_count, bin_count;
  uint64_t heavy[3];
  int found[3];  // answers of three searches for a bin in turn
  int n, part, n_few;
};

template <int TYPE>
struct Picker {
  typedef Logit<TYPE> L;
  const void* row;
  int V;
  const Chunks& ws;  // this row's
  Pick& s;
  Grid grid;
  float top;    // the row's largest logit
  double edge;  // its bin
  int here;    // the fetched bin
  bool kept;   // whether its tokens are in the list, which holds the bins
  int list_from, list_to;
  uint16_t* ends;  // [n x kBins] where a row's bin ends in a chunk's list, in LDS
  bool near;       // if there is room for it
  int index_bits;  // of a token's index
  int turn;        // which of s.found the next search writes

  // 1 for the largest logit, from an exact difference for the others
  __device__ __forceinline__ double weight(float l) const {
    return exp(((double)l - (double)top) * (grid.per / kPerNat));
  }

  // The row's running counts and masses from the chunks' histograms; `e` is the top
  // bin of the thread's own chunk, if it has one.
  __device__ void merge(double e) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    static_assert(kMaxChunks <= kSampThreads, "a thread a chunk");
    if (t < ws.n) {
      const double d = edge - e;  // a chunk too far out has no histogram
      s.dist[t] = (short)(chunk_on_grid(e) && d < (double)kBins ? (int)d : kBins);
    }
    __syncthreads();
    static_assert(kBins == kSampThreads, "a bin a thread");
    uint64_t m = 0;
    uint32_t c = 0;
    for (int i0 = 0; i0 < ws.n; i0 += 16) {  // 16 chunks' numbers on their way at once
      uint64_t h[16];
      uint32_t end[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int i = min(i0 + q, ws.n - 1);
        const int64_t at = (int64_t)i * kBins + max(t - s.dist[i], 0);
        h[q] = ws.hists[at];
        end[q] = ws.ends[at];
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int i = min(i0 + q, ws.n - 1);
        const bool in = i == i0 + q && t >= s.dist[i];
        m += in ? h[q] & ((1ull << kCountShift) - 1) : 0;
        c += in ? (uint32_t)(h[q] >> kCountShift) : 0;
        if (near && i == i0 + q) ends[i * kBins + t] = in ? end[q] : 0;
      }
    }
    // e^(difference of the upper edges); 1 for the top bin, whose sums and shares are
    // therefore exact up to 2^53: tokens that weigh the same are counted
    const double unit = exp(-(double)t / kPerNat);
    uint32_t ci = scan_sum(c);
    // The lanes' sums are rounded in different orders: one can lie below its
    // predecessor's, or an empty bin's above it.  Their running maximum over the bins
    // with tokens never falls and rises at bins with tokens alone; adding the waves
    // before, in one order for all, keeps that.
    double mi = scan_sum((double)m * unit);
    mi = scan_wave(c ? mi : 0.0, 0.0, [](double p, double q) { return fmax(p, q); });
    if (lane == 63) {
      s.wave_u32[wave] = ci;
      s.wave_f64[wave] = mi;
    }
    __syncthreads();
    double waves = 0.0;
    for (int i = 0; i < wave; ++i) {
      ci += s.wave_u32[i];
      waves += s.wave_f64[i];
    }
    s.count[t] = ci;
    s.mass[t] = waves + mi;
    s.unit[t] = unit;
    s.units[t] = m;
    if (t < 3) s.found[t] = kBins;
    __syncthreads();
  }
  __device__ __forceinline__ uint32_t count_before(int b) const { return b ? s.count[b - 1] : 0; }
  __device__ __forceinline__ double mass_before(int b) const { return b ? s.mass[b - 1] : 0.0; }

  // First bin whose running count reaches k (kBins if none does), or whose running
  // mass reaches `target` (`over`: exceeds it; the last bin with tokens if none does).
  // Either has tokens: counts and masses rise nowhere else.
  // The searches take the three places of s.found in turn.  One that ends sets the
  // next one's place back, before its barrier: that place was read before the barrier
  // of the search in between, and is written after this one.
  __device__ int found_bin() {
    const int next = turn == 2 ? 0 : turn + 1;
    if (threadIdx.x == 0) s.found[next] = kBins;
    __syncthreads();
    const int f = s.found[turn];
    turn = next;
    return f;
  }
  __device__ int bin_of_count(uint32_t k) {
    const int t = threadIdx.x;
    if (s.count[t] >= k && count_before(t) < k) s.found[turn] = t;
    return found_bin();
  }
  __device__ int bin_of_mass(double target, bool over) {
    const int t = threadIdx.x;
    auto reached = [&](int i) { return over ? s.mass[i] > target : s.mass[i] >= target; };
    if (s.count[t] > count_before(t) &&
        (reached(t) ? t == 0 || !reached(t - 1) : s.count[t] == s.count[kBins - 1]))
      s.found[turn] = t;
    return found_bin();
  }

  // A token's place in the order as a number that rises along it: the complement of
  // the key without its dead bits, then the index.
  __device__ __forceinline__ uint64_t order_of(float l, int token) const {
    return (uint64_t)(~key_of(l) >> L::kDead) << index_bits | (uint32_t)token;
  }
  __device__ __forceinline__ float logit_at(uint64_t order) const {
    const uint32_t k = ~((uint32_t)(order >> index_bits) << L::kDead);  // dead bits set
    return logit_of(k & 0x80000000u ? k & ~0u << L::kDead : k);
  }
  __device__ __forceinline__ int token_at(uint64_t order) const { return (int)(order & ((1u << index_bits) - 1)); }

  // Every token of the bins from `b0` to `b` from the chunks' lists: begin(n) is called
  // by the lanes of a chunk with its n tokens and says the number of its first,
  // use(number, o) with each token's place in the order.
  template <class Begin, class Use>
  __device__ __forceinline__ void read_tokens(int b0, int b, Begin begin, Use use) {
    const int lanes = ws.n > 16 ? 16 : ws.n > 8 ? 32 : 64;  // of a chunk
    const int lane = threadIdx.x & (lanes - 1);
    for (int i = threadIdx.x / lanes; i < ws.n; i += kSampThreads / lanes) {
      int first, n;
      if (near) {
        first = b0 ? ends[i * kBins + b0 - 1] : 0;
        n = ends[i * kBins + b] - first;
      } else {
        const int d = s.dist[i];
        const uint16_t* e = ws.ends + (int64_t)i * kBins - d;
        first = b0 > d ? e[b0 - 1] : 0;
        n = (b >= d ? e[b] : 0) - first;
      }
      if (n == 0) continue;
      const uint16_t* from = ws.tokens + (int64_t)i * ws.len + first;
      const int to = begin(n, lanes);
      for (int j = lane; j < n; j += 4 * lanes) {  // four at a time on their way
        int token[4];
        float l[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) token[q] = i * ws.len + from[min(j + q * lanes, n - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q) l[q] = L::f32(((const typename L::T*)row)[token[q]]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q * lanes < n) use(to + j + q * lanes, order_of(l[q], token[q]));
      }
    }
  }

  // Makes bin b the one that the functions below look at.  The list holds the bins up
  // to the first border that is asked for if that is possible: later borders lie
  // before it.
  __device__ void fetch(int b) {
    here = b;
    if (kept && b >= list_from && b <= list_to) return;
    __syncthreads();
    const int n = (int)(s.count[b] - count_before(b));
    list_from = s.count[b] <= (uint32_t)kPrefix ? 0 : b;
    list_to = b;
    kept = n <= kList;
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    if (kept) {
      read_tokens(
          list_from, b,
          [&](int more, int lanes) {
            int to = 0;
            if ((threadIdx.x & (lanes - 1)) == 0) to = atomicAdd(&s.n, more);
            return __shfl(to, threadIdx.x & 63 & -lanes, 64);
          },
          [&](int at, uint64_t o) { s.s.order[at] = o; });
      __syncthreads();
    }
  }
  // Every token of the fetched bin.
  template <class Use>
  __device__ __forceinline__ void each(Use use) {
    if (kept) {
      for (int i = threadIdx.x; i < s.n; i += kSampThreads) {
        const uint64_t o = s.s.order[i];
        if (list_from == list_to || edge - grid.bin(logit_at(o)) == (double)here) use(o);
      }
    } else {
      read_tokens(here, here, [](int, int) { return 0; }, [&](int, uint64_t o) { use(o); });
    }
  }

  __device__ __forceinline__ uint64_t unit_at(uint64_t order) const {
    const float l = logit_at(order);
    return grid.template unit<false>(l, grid.bin(l));
  }

  // The token of the fetched bin with which its count (COUNT) or its units of mass
  // first reach `target` (from 1 to the whole); `cum` receives the units up to and
  // with it.
  template <bool COUNT>
  __device__ uint64_t select(uint64_t target, uint64_t& cum) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    uint64_t lo = 0, hi = ~0ull, before_units = 0;
    // where the bin's tokens should lie; the end parts take what does not
    const double slack = 1.0 / (1 << 20), b0 = edge - (double)here, b1 = b0 + 1.0;
    uint64_t from = order_of((float)((b1 + fabs(b1) * slack) / grid.per), 0),
             to = order_of((float)((b0 - fabs(b0) * slack) / grid.per), (1 << index_bits) - 1);
    if (from > to) {
      from = 0;
      to = hi;
    }
    uint32_t left = s.count[here] - count_before(here), before_count = 0;
    while (left > (uint32_t)kFew) {
      for (int i = t; i < kParts; i += kSampThreads) {
        s.s.hist[i] = 0;
        s.s.parts[i] = 0;
      }
      if (t == 0) s.bin_count = 0;  // the loop ends even if the logits change under it
      __syncthreads();
      const int shift = max(0, 64 - kPartBits - __clzll(to - from));
      const int parts = (int)((to - from) >> shift) + 1;  // at most kParts
      each([&](uint64_t o) {
        if (o >= lo && o <= hi) {
          const int part = o <= from ? 0 : o >= to ? parts - 1 : (int)((o - from) >> shift);
          atomicAdd((unsigned long long*)&s.s.hist[part], (unsigned long long)unit_at(o));
          atomicAdd(&s.s.parts[part], 1u);
        }
      });
      __syncthreads();
      constexpr int PER = kParts / kSampThreads;
      uint64_t m = 0;
      uint32_t c = 0;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        m += s.s.hist[PER * t + h];
        c += s.s.parts[PER * t + h];
      }
      uint64_t e = scan_sum(m);
      uint32_t f = scan_sum(c);
      if (lane == 63) {
        s.wave_u64[wave] = e;
        s.wave_u32[wave] = f;
      }
      __syncthreads();
      for (int w = 0; w < wave; ++w) {
        e += s.wave_u64[w];
        f += s.wave_u32[w];
      }
      e += before_units - m;
      f += before_count - c;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        m = s.s.hist[PER * t + h];
        c = s.s.parts[PER * t + h];
        if (COUNT ? (f < target && f + (uint64_t)c >= target) : (e < target && e + m >= target)) {
          s.part = PER * t + h;
          s.before = e;
          s.before_count = f;
          s.bin_count = c;
        }
        e += m;
        f += c;
      }
      __syncthreads();
      const int part = s.part;
      left = s.bin_count;
      before_units = s.before;
      before_count = s.before_count;
      if (part > 0) lo = from + ((uint64_t)part << shift);
      if (part < parts - 1) hi = from + ((uint64_t)(part + 1) << shift) - 1;
      from = lo;
      to = hi;
      __syncthreads();
    }
    // at most kFew are left: each counts what stands before it
    if (t == 0) s.n_few = 0;
    __syncthreads();
    each([&](uint64_t o) {
      if (o >= lo && o <= hi) s.few[min(atomicAdd(&s.n_few, 1), kFew - 1)] = Pick::Few{o, unit_at(o)};
    });
    __syncthreads();
    const int few = min(s.n_few, kFew);
    // as many lanes to a token as there are, up to a wave
    const int per = few > 1 ? max(0, min(6, __clz(few - 1) - 23)) : 6;
    const int i0 = t & ((1 << per) - 1);
    if (t >> per < few) {
      const uint64_t o = s.few[t >> per].order, m = s.few[t >> per].units;
      uint64_t c = 0;
      uint32_t r = 0;
#pragma unroll 4
      for (int i = i0; i < few; i += 1 << per) {
        const Pick::Few f = s.few[i];
        const bool first = f.order < o;
        r += first ? 1 : 0;
        c += first ? f.units : 0;
      }
      for (int x = 1; x < 1 << per; x <<= 1) {
        r += __shfl_xor(r, x, 64);
        c += __shfl_xor(c, x, 64);
      }
      const uint64_t was = COUNT ? before_count + (uint64_t)r : before_units + c, is = was + (COUNT ? 1 : m);
      if (i0 == 0 && was < target && is >= target) {
        s.answer = o;
        s.before = before_units + c + m;
      }
    }
    __syncthreads();
    cum = s.before;
    const uint64_t o = s.answer;
    __syncthreads();
    return o;
  }

  // The filters and the choice.
  __device__ void choose(int k, double p, double mp, double u, int& token, double& prob) {
    // what is kept: the bins before `end`, and of bin `end` the tokens up to `last`,
    // which hold `part` of its units (none of them if it is 0; never so for the first
    // bin, which has the largest logit); `held_mass` is the mass of it all
    uint64_t last = ~0ull, part = 0;
    int end = kBins;
    double held_mass = s.mass[kBins - 1];
    if (k > 0 && k < V) {
      const int b = bin_of_count((uint32_t)k);
      if (b < kBins) {  // else the tokens beyond the bins have no mass
        fetch(b);
        last = select<true>((uint64_t)k - count_before(b), part);
        end = b;
        held_mass = mass_before(b) + (double)part * s.unit[b];
      }
    }
    // the place in the order where the mass reaches (exceeds) a target below `held_mass`,
    // which is therefore not in a bin `end` of which nothing is kept
    auto place = [&](double target, bool over, int& bin, uint64_t& at, uint64_t& cum) {
      bin = min(bin_of_mass(target, over), end);
      fetch(bin);
      const double in = (target - mass_before(bin)) / s.unit[bin];
      at = select<false>(first_unit(in, over, bin == end ? part : s.units[bin]), cum);
    };
    if (p < 1.0) {
      int bin;
      uint64_t at, cum;
      place(p > 0.0 ? p * held_mass : 0.0, false, bin, at, cum);
      end = bin;
      last = at;
      part = cum;
      held_mass = mass_before(end) + (double)part * s.unit[end];
    }
    if (mp > 0.0) {
      // the bin that weight mp falls into; rounding may put it into a neighbour
      const double floor_w = mp < 1.0 ? mp : 1.0;
      const int near_bin = (int)fmin(fmax(-floor(grid.in_bin(top, edge) + log(floor_w) * kPerNat), 0.0), (double)kBins);
      const int first = max(0, near_bin - 1), far = min(min(near_bin + 1, end), kBins - 1);
      bool found = false;
      if (first <= far) {
        if (threadIdx.x < 3) s.heavy[threadIdx.x] = 0;
        if (threadIdx.x == 0) s.answer = 0;
        __syncthreads();
        auto weigh = [&](uint64_t o) {
          const float l = logit_at(o);
          const int bin = (int)fmin(edge - grid.bin(l), (double)kBins);
          if (bin >= first && (bin < end || o <= last) && bin <= far && weight(l) >= floor_w) {
            atomicAdd((unsigned long long*)&s.heavy[bin - first], (unsigned long long)unit_at(o));
            atomicMax((unsigned long long*)&s.answer, (unsigned long long)o);
          }
        };
        if (kept && list_from <= first && far <= list_to)
          for (int i = threadIdx.x; i < s.n; i += kSampThreads) weigh(s.s.order[i]);
        else
          read_tokens(first, far, [](int, int) { return 0; }, [&](int, uint64_t o) { weigh(o); });
        __syncthreads();
        for (int bin = first; bin <= far && !found; ++bin) {
          const uint64_t heavy = s.heavy[bin - first];
          if (heavy < (bin == end ? part : s.units[bin])) {  // this bin holds the border
            found = true;
            end = bin;
            part = heavy;
            last = s.answer;  // the last heavy token lies here if any does
            held_mass = mass_before(bin) + (double)heavy * s.unit[bin];
          }
        }
        __syncthreads();
      }
      if (!found && end > near_bin + 1) {  // no token near the border: nothing beyond it stays
        end = min(near_bin + 2, kBins);
        part = 0;
        held_mass = s.mass[end - 1];
      }
    }
    int bin;
    uint64_t at, cum;
    if (!(u >= 0.0)) u = 0.0;
    if (u < 1.0) {
      place(u * held_mass, true, bin, at, cum);
    } else {  // the last token with mass, by units and counts: a small one does not show in the sums
      bin = part > 0 ? end : bin_of_count(s.count[end - 1]);
      fetch(bin);
      at = select<false>(bin == end ? part : s.units[bin], cum);
    }
    token = token_at(at);
    // a unit of the top bin: e^(its upper edge - top) 2^-35
    prob = weight(logit_at(at)) / (held_mass * (exp((1.0 - grid.in_bin(top, edge)) / kPerNat) / kBinUnit));
  }
};

template <int TYPE>
__global__ __launch_bounds__(kSampThreads, 4) void sample_pick_kernel(SampleArgs a, Chunks ws) {
  __shared__ Pick s;
  extern __shared__ uint16_t ends[];
  typedef Logit<TYPE> L;
  const int64_t b = blockIdx.x;
  ws.heads += b * ws.n;
  ws.hists += b * ws.n * kBins;
  ws.ends += b * ws.n * kBins;
  ws.tokens += b * ws.n * ws.len;
  // everything the row is told, read at once
  const float t = a.temperature ? a.temperature[b] : 1.0f, pf = a.top_p ? a.top_p[b] : 1.0f,
              mpf = a.min_p ? a.min_p[b] : 0.0f, uf = a.u[b];
  const int k = a.top_k ? a.top_k[b] : 0;
  uint64_t best = 0;
  double chunk_edge = 0.0;
  if ((int)threadIdx.x < ws.n) {
    const ChunkHead h = ws.heads[threadIdx.x];
    best = h.top;
    chunk_edge = h.edge;
  }
  best = wave_max(best);
  if ((threadIdx.x & 63) == 0) s.wave_u64[threadIdx.x >> 6] = best;
  __syncthreads();
  for (int w = 0; w < kSampWaves; ++w) best = max_u64(best, s.wave_u64[w]);
  __syncthreads();
  const uint32_t top_key = (uint32_t)(best >> 32);
  int token = (int)~(uint32_t)best;
  double prob = 1.0;
  if (top_key == kKeyNegInf) {
    token = -1;
    prob = 0.0;
  } else if (t > 0.f && k != 1) {
    const double p = (double)pf, mp = (double)mpf, u = (double)uf;
    const float top = logit_of(top_key);
    Picker<TYPE> pick{(const typename L::T*)a.logits + b * a.ld, a.V, ws, s, Grid(t), top, 0.0, -1, false, 0, 0,
                      ends, ws.n <= kNearChunks, 32 - __clz(a.V | 1), 0};
    pick.edge = pick.grid.bin(top);
    if (row_on_grid(pick.edge)) {
      pick.merge(chunk_edge);
      pick.choose(k, p, mp, u, token, prob);
    } else {
      Row<TYPE> row{(const typename L::T*)a.logits + b * a.ld, a.V, s.radix};
      Weigher w{(double)top, (double)t, top_key};
      solve_by_radix(row, w, k, p, mp, u, token, prob);
    }
  }
  if (threadIdx.x == 0) {
    a.tokens[b] = token;
    if (a.probs) a.probs[b] = (float)prob;
  }
}

int chunks_of(int V, int pt) { return (V + kScanThreads * pt - 1) / (kScanThreads * pt); }
// Logits per thread of a scan block: 8 where that is enough for 1024 blocks at most
// and 16 chunks a row (which the choice reads at once: 1 x 50304 takes 17.2 us in 13
// chunks, 18.5 in 25), else 16 or 32.
int scan_pt(int64_t B, int V) {
  int pt = 8;
  while (pt < 32 && (chunks_of(V, pt) > 16 || B * chunks_of(V, pt) > 1024)) pt *= 2;
  return pt;
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// The chunks' places in a workspace, and its size.
Chunks chunks_in(char* ws, int64_t B, int V, int64_t& bytes) {
  Chunks c;
  const int pt = scan_pt(B, V);
  c.len = kScanThreads * pt;
  c.n = chunks_of(V, pt);
  const int64_t n = B * c.n;
  int64_t at = 0;
  c.heads = (ChunkHead*)(ws + at); at += up256(n * (int64_t)sizeof(ChunkHead));
  c.hists = (uint64_t*)(ws + at); at += n * kBins * 8;
  c.ends = (uint16_t*)(ws + at); at += n * kBins * 2;
  c.tokens = (uint16_t*)(ws + at); at += n * c.len * 2;
  bytes = at;
  return c;
}

template <int TYPE>
hipError_t launch_type(const SampleArgs& a, void* ws, hipStream_t stream) {
  int64_t bytes;
  const Chunks c = chunks_in((char*)ws, a.B, a.V, bytes);
  auto scan = c.len == 8 * kScanThreads    ? sample_scan_kernel<TYPE, 8>
              : c.len == 16 * kScanThreads ? sample_scan_kernel<TYPE, 16>
                                           : sample_scan_kernel<TYPE, 32>;
  scan<<<(unsigned)(a.B * c.n), kScanThreads, 0, stream>>>(a, c);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = c.n <= kNearChunks ? (size_t)c.n * kBins * 2 : 0;
  sample_pick_kernel<TYPE><<<(unsigned)a.B, kSampThreads, lds, stream>>>(a, c);
  return hipGetLastError();
}

}  // namespace

int64_t sample_workspace_bytes(int64_t B, int V) {
  int64_t bytes;
  chunks_in(nullptr, B, V, bytes);
  return bytes;
}

hipError_t launch_sample(SampleType type, const SampleArgs& a, void* ws, hipStream_t stream) {
  return type == kSampleF32 ? launch_type<kSampleF32>(a, ws, stream)
         : type == kSampleBf16 ? launch_type<kSampleBf16>(a, ws, stream)
                               : launch_type<kSampleF16>(a, ws, stream);
}

}  // namespace moe
