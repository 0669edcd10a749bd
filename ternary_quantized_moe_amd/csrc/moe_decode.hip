// Attention of one new token of every sequence over a paged cache, for gfx950:
//   y_h = sum_j p_hj v_j,   p_hj = exp(s_hj - m_h) / sum_j exp(s_hj - m_h),   s_hj = scale q_h k_j
// over the lengths[b] cached tokens j of sequence b.  Every key and value is read once for
// each 16 query heads that share it, so HBM bounds it (with up to 16 heads a key head; of 64, a
// token of 131072, whose keys and values are 67 MB, takes 48 us, 13 of them for that much).
//
// The tiles (a few dozen tokens for each wave of a block) of all sequences stand in one
// row, which the workers of a kv head share equally, however ragged the lengths are; a
// worker takes a run of tiles that may begin and end inside a sequence.  What it has of
// a sequence that others share goes to the workspace as (m, l, sum), and a second launch
// joins these in the order of the workers.
//
// A wave copies 32 or 64 tokens of keys and values into LDS of its own by loads that go there
// directly, some tiles ahead, and needs no barrier until a sequence ends and the waves
// join.  Every lane finds its token's row by itself, so pages may have any size (a second way
// for tiles within a page, with one address for all lanes, won 0.5% there and lost 1.5%
// elsewhere).  Scores are formed transposed, S^T = K Q^T, with the query heads on the matrix
// core's columns (16 of them; fewer leave columns idle, which HBM hides); the softmax is
// then within a lane and the four lanes of a column, and P stands as the second operand
// of y^T = V^T P^T, whose first is read from LDS transposed.  P is rounded to 16 bits for
// the matrix cores (half a step of itself, as y's own rounding; in fp16 2^-32 of the largest
// where that is more).
// e4m3 codes are widened exactly; a key's scale multiplies its scores, a value's scale
// the weights before they are rounded, in fp16 relative to the largest such product.
//
// Of 64 sequences of up to 8192 tokens, 32 heads over 8 of 128, it reads 974 MB in 176 us
// (5.5 TB/s; some of that is in the Infinity Cache), of one of 131072 268 MB in 54 us, the
// join with it (46 where that cache holds more of it), of 256 of up to 3001 in e4m3 832 MB in
// 162 us (5.1 TB/s), in fp16 over e4m3 in 167.  One sequence of 77 tokens is a launch and a
// chain of latencies: 9 us, of which finding the place takes 0.9, the page numbers 0.3, each of
// its two tiles 1.4 to ask for and 0.9 to go through, the join of the waves and the store 1.5.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attention_device.h"
#include "attention_internal.h"

namespace moe {

namespace {

// One a CU: its tiles fill the LDS (512: 256 sequences in e4m3 177 us, 165 with 256).  Groups of
// heads share them equally, so numbers that do not divide it leave some CUs idle.
constexpr int kBlocks = 256;
constexpr int kHeadTile = 16;  // query heads of a block

template <int D>
constexpr int kWaves = D == 256 ? 2 : 4;  // two tiles of each wave fit the LDS
// Tokens of a wave's tile: what a wave does between a tile's arrival and its end is a chain
// of latencies, so a tile has 64 tokens where these are short (64 channels, or 8 bits) and
// 32 otherwise (256 sequences of up to 3001 in e4m3 165 us, 178 with 32; 16 of up to 2000, 16
// heads of 64, 20 us and 22).
template <bool F8, int D>
constexpr int kTileTokens = F8 || D == 64 ? 64 : 32;

int64_t groups_of(int heads, int kv_heads) {
  return (int64_t)kv_heads * ((heads / kv_heads + kHeadTile - 1) / kHeadTile);
}
int64_t record_floats(int D) { return kHeadTile * D + 2 * kHeadTile; }
int64_t workers_of(int64_t groups) { return std::max<int64_t>(1, kBlocks / groups); }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

struct DecodeWork {
  int groups, per_kv;  // groups of query heads, and those of one kv head
  int workers;
  float* parts;   // [groups x workers x 2] records: sums [16 x D], m [16], l [16]
  int2* shared;   // [B]: first and last worker of a sequence
};

// Piece p (16 bytes) of row r of a tile is kept at place p ^ f(r) of the row, which
// spreads the rows that are read together over all banks.
template <int ROW>
__device__ __forceinline__ int swizzle(int r) {
  return ROW == 64 ? (r >> 2) & 3 : ROW == 128 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3) : (r & 3) << 2 | ((r >> 2) & 3);
}

// A number at an address that the whole wave shares, read past the vector loads in flight:
// those are waited for in order, and waiting for one waits for the tiles before it.
__device__ __forceinline__ int scalar_load(const int32_t* p) {
  return *(const int32_t __attribute__((address_space(4)))*)(uintptr_t)p;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Loads that go to LDS, lane after lane from dst on (the same in the whole wave).  They are
// written out, since the compiler waits for every such load of its own before any read of
// LDS, the tiles in flight among them; they write no register, and what needs them waits for
// them here.  Between m0 and its use stands one wait state.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is set by every statement that uses it
__device__ __forceinline__ uint32_t lds_address(uint8_t* p) {
  return (uint32_t)uniform((int)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)p);
}
// 16 or 4 bytes a lane from the lane's address.
__device__ __forceinline__ void copy16_to_lds(const void* src, uint8_t* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_address(dst)), "v"(src)
               : "memory", "m0");
}
__device__ __forceinline__ void copy4_to_lds(const void* src, uint8_t* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds_address(dst)), "v"(src)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Four e4m3 codes -> four 16-bit values (exact).
template <bool F16>
__device__ __forceinline__ u32x2 widen4(uint32_t v) {
  if constexpr (F16)
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)v, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)v, 1.0f, true))};
  else
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v, 1.0f, true))};
}

// The value of the four lanes of a column, 16 apart, joined.
template <class F>
__device__ __forceinline__ float over_column(float v, F f) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const f32x2_t h = both_halves(f(__uint_as_float(r[0]), __uint_as_float(r[1])));
  return f(h.x, h.y);
}

// Reads eight rows of 16 bytes transposed: within 16 lanes, lane i gives the address of
// bytes 8 (i % 2) .. + 7 of row i / 2 and gets byte i of the eight rows.
__device__ __forceinline__ u32x2 read_transposed8(const uint8_t* p) {
  typedef int i32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)(p)));
}

template <bool F16, bool F8, int D>
struct Decode {
  using H = Half<F16>;
  static constexpr int W = kWaves<D>, ROW = D * (F8 ? 1 : 2), kKeys = kTileTokens<F8, D>, PER = ROW / 16;
  static constexpr int kTile = kKeys * ROW, ST = kKeys / 16;  // ST: score tiles
  static constexpr int kLoads = kTile / 1024, kPerStage = 2 * kLoads + (F8 ? 2 : 0);
  static constexpr int kStage = 2 * kTile + (F8 ? 8 * kKeys : 0);
  static constexpr int kFit = 126 * 1024 / (W * kStage), kStages = kFit > 4 ? 4 : kFit < 2 ? 2 : kFit;
  static constexpr int kBlockKeys = W * kKeys;
  static constexpr int kRecord = 64 * (D / 4 + 2);  // floats of a wave's state
  static constexpr int QS = D / 32, DT = D / 16;
  // What is rounded to 16 bits is a weight times its value's scale, which may lie anywhere in
  // fp32, while fp16 has 30 exponents.  So there the sums of the values have a reference n of
  // their own beside m: they are formed of p scale 2^(m - n), the largest of which so far
  // lies between 2^7 and 2^15 (256 sequences of up to 3001 in fp16 over e4m3 167 us; the products as
  // they are, which small scales make zeros of, 162 us).
  static constexpr bool kOwnRange = F16 && F8;

  const DecodeArgs& a;
  int lane, wave, col, quad, kv;
  uint8_t* mine;
  u32x4 q[QS];
  f32x4 o[DT];
  float m, l, n;
  bool bad;

  __device__ __forceinline__ Decode(const DecodeArgs& args) : a(args) {}

  // A place in the row of all tiles.
  struct Walk {
    int b, tile, tiles, len;
    int64_t left;
  };
  __device__ __forceinline__ int tiles_of(int len) const {
    return max(1, (int)(((uint32_t)len + (kBlockKeys - 1)) / kBlockKeys));
  }
  __device__ __forceinline__ int length(int64_t b) const {
    const int64_t room = (int64_t)a.c.width * a.c.P;
    return (int)min((int64_t)max(a.lengths[b], 0), room);
  }
  __device__ __forceinline__ void enter(Walk& w) const {
    const int64_t room = (int64_t)a.c.width * a.c.P;
    w.len = (int)min((int64_t)max(scalar_load(a.lengths + w.b), 0), room);
    w.tiles = tiles_of(w.len);
  }
  __device__ __forceinline__ void step(Walk& w) const {
    if (--w.left > 0 && ++w.tile == w.tiles) {
      w.tile = 0;
      ++w.b;
      enter(w);
    }
  }

  static constexpr int ROWS = 64 / PER;  // rows of a load
  __device__ __forceinline__ int first_of(const Walk& w) const { return w.tile * kBlockKeys + wave * kKeys; }
  __device__ __forceinline__ const int32_t* table_of(const Walk& w) const { return a.c.tables + (int64_t)w.b * a.c.width; }

  // The page of every token goes to LDS, lane after lane, ahead of its tile.
  __device__ __forceinline__ void pages_to_lds(const Walk& w, uint8_t* dst) const {
    const int key = min(first_of(w) + (lane & (kKeys - 1)), max(w.len - 1, 0));
    copy4_to_lds(a.c.width > 0 ? table_of(w) + (key >> a.c.shift) : a.lengths, dst);
  }

  // The wave's tile into LDS.  Rows behind the last token repeat it; they are masked.  A
  // page that is none makes the sequence's results NaN and is read as page 0.
  __device__ __forceinline__ bool stage(int first, int len, int page, uint8_t* dst) const {
    const int last = max(len - 1, 0);
    const bool wrong = page < 0 || page >= a.c.n_pages || a.c.width == 0;
    if (wrong) page = 0;
    const int place = min(first + (lane & (kKeys - 1)), last) & (a.c.P - 1);  // of the lane's token in its page
    const int64_t mine = ((int64_t)page * a.c.kv_heads + kv) * a.c.P + place;  // the lane's token's row of the cache
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * ROWS + lane / PER;
      const int64_t at = __shfl(mine, row, 64) * ROW + 16 * ((lane % PER) ^ swizzle<ROW>(row));
      copy16_to_lds((const uint8_t*)a.c.k + at, dst + i * 1024);
      copy16_to_lds((const uint8_t*)a.c.v + at, dst + kTile + i * 1024);
    }
    if (F8) {  // the scales: the keys', then the values'
      copy4_to_lds(a.c.k_scales + mine, dst + 2 * kTile);
      copy4_to_lds(a.c.v_scales + mine, dst + 2 * kTile + 256);
    }
    return wrong && len > 0;
  }

  // The queries of sequence b.
  __device__ __forceinline__ void fetch(int64_t b, int head0, int heads, u32x4 (&to)[QS]) const {
    const uint16_t* p = a.q.p + b * a.q.token + (head0 + min(col, heads - 1)) * a.q.head;
#pragma unroll
    for (int k = 0; k < QS; ++k)
      to[k] = *(const u32x4*)(p + (F8 ? 64 * (k / 2) + 16 * quad + 8 * (k & 1) : 32 * k + 8 * quad));
  }
  __device__ __forceinline__ void begin() {
    m = n = -INFINITY;
    l = 0.f;
    bad = false;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x4{};
  }

  __device__ __forceinline__ void tile(const uint8_t* ks, int first, int len, float c) {
    const uint8_t* vs = ks + kTile;
    // All of the tile's keys are read before the first product: the reads' latencies then
    // run side by side.
    constexpr int KP = F8 ? D / 64 : QS;  // pieces of a row a lane reads
    u32x4 kf[ST][KP];
#pragma unroll
    for (int t = 0; t < ST; ++t) {
      const int row = 16 * t + col, at = row * ROW, f = swizzle<ROW>(row);
#pragma unroll
      for (int k = 0; k < KP; ++k) kf[t][k] = *(const u32x4*)(ks + at + 16 * ((4 * k + quad) ^ f));
    }
    f32x4 k_scale[ST], v_scale[ST];
    if (F8) {
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        k_scale[t] = *(const f32x4*)(ks + 2 * kTile + 4 * (16 * t + 4 * quad));
        v_scale[t] = *(const f32x4*)(ks + 2 * kTile + 4 * kKeys + 4 * (16 * t + 4 * quad));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    f32x4 s[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t) s[t] = f32x4{};
#pragma unroll
    for (int k = 0; k < KP; ++k)
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const u32x4 v = kf[t][k];
        if (F8) {
          const u32x2 w0 = widen4<F16>(v.x), w1 = widen4<F16>(v.y), w2 = widen4<F16>(v.z), w3 = widen4<F16>(v.w);
          s[t] = H::mfma16(u32x4{w0.x, w0.y, w1.x, w1.y}, q[2 * k], s[t]);
          s[t] = H::mfma16(u32x4{w2.x, w2.y, w3.x, w3.y}, q[2 * k + 1], s[t]);
        } else {
          s[t] = H::mfma16(v, q[k], s[t]);
        }
      }
    // So are the values of the first 32 tokens, beside the softmax.
    constexpr int VR = F8 ? 1 : 2;  // reads of a fragment
    u32x2 vf[DT][VR];
    auto read_values = [&](int h) {
      const uint8_t* half = vs + 32 * h * ROW;
      if (F8) {
        const int j = col >> 1, row = 16 * (j / 4) + 4 * quad + (j & 3), f = swizzle<ROW>(row);
#pragma unroll
        for (int d = 0; d < DT; ++d) vf[d][0] = read_transposed8(half + row * ROW + 16 * (d ^ f) + 8 * (col & 1));
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = 16 * t + 4 * quad + (col >> 2);
          const int at = row * ROW + 16 * (((col & 3) >> 1) ^ swizzle<ROW>(row)) + 8 * (col & 1);
#pragma unroll
          for (int d = 0; d < DT; ++d) vf[d][VR - 1 < t ? VR - 1 : t] = read_transposed(half + (at ^ (d << 5)));
        }
      }
    };
    __builtin_amdgcn_sched_barrier(0);
    read_values(0);
    __builtin_amdgcn_sched_barrier(0);
    if (F8) {
#pragma unroll
      for (int t = 0; t < ST; ++t) s[t] *= k_scale[t];
    }
    const int there = len - first;  // tokens of the tile that exist
    const bool whole = there >= kKeys;
    if (!whole) {
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * t + 4 * quad + i >= there) s[t][i] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][i]);
    top = over_column(top, [](float x, float y) { return fmaxf(x, y); }) * c;
    if (__any(top > m + (H::kLift + H::kLag))) {  // the maximum that is subtracted may lag behind
      const float now = fmaxf(m, top - H::kLift), f = now == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
      if (!kOwnRange) scale_sums(f);
    }
    const float off = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(s[t][i] * c - off);
        l += s[t][i];
      }
    if (F8) {
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] *= whole || 16 * t + 4 * quad + i < there ? v_scale[t][i] : 0.f;
    }
    if (kOwnRange) {
      // Products below 2^-33 count as that: their sums stay far below what fp16 holds.
      float big = 0x1p-33f;
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) big = fmaxf(big, __builtin_fabsf(s[t][i]));
      big = over_column(big, [](float x, float y) { return fmaxf(x, y); });
      const float at = __builtin_amdgcn_logf(big) + m;  // base 2
      if (__any(at > n + (H::kLift + H::kLag))) {
        const float now = fmaxf(n, at - H::kLift);
        scale_sums(now == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(n - now));
        n = now;
      }
      const float f = n == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - n);
#pragma unroll
      for (int t = 0; t < ST; ++t) s[t] *= f;
    }
    // k slot 8 quad + e of a product over 32 tokens is token 16 (e / 4) + 4 quad + e % 4.
    // Values behind the last token become zeros: they may hold anything.
#pragma unroll
    for (int h = 0; h < ST / 2; ++h) {
      const f32x4 &s0 = s[2 * h], &s1 = s[2 * h + 1];
      const u32x4 p = {H::pack(s0[0], s0[1]), H::pack(s0[2], s0[3]), H::pack(s1[0], s1[1]), H::pack(s1[2], s1[3])};
      u32x4 keep = {~0u, ~0u, ~0u, ~0u};
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 32 * h + 16 * (e / 2) + 4 * quad + 2 * (e & 1);
          keep[e] = (row < there ? 0xFFFFu : 0u) | (row + 1 < there ? 0xFFFF0000u : 0u);
        }
      }
      if (h) {
        __builtin_amdgcn_sched_barrier(0);
        read_values(h);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        u32x2 lo = vf[d][0], hi = vf[d][VR - 1];
        if (F8) {
          hi = widen4<F16>(lo.y);
          lo = widen4<F16>(lo.x);
        }
        u32x4 w = {lo.x, lo.y, hi.x, hi.y};
        if (!whole) w &= keep;
        o[d] = H::mfma16(w, p, o[d]);
      }
    }
  }

  __device__ __forceinline__ void scale_sums(float f) {
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] *= f;
  }

  // The waves' shares of a sequence, joined in wave 0: half of them hand theirs over, and
  // so on.
  __device__ __forceinline__ void join(float* room) {
    if (kOwnRange) scale_sums(n == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(n - m));
    l = over_column(l, [](float x, float y) { return x + y; });
    if (__any(bad)) l = NAN;
#pragma unroll
    for (int n = W / 2; n; n /= 2) {
      float* at = room + (wave % n) * kRecord;
      f32x4* const sums = (f32x4*)at + lane;
      at += 256 * DT + lane;
      if (wave >= n && wave < 2 * n) {
#pragma unroll
        for (int d = 0; d < DT; ++d) sums[64 * d] = o[d];
        at[0] = m;
        at[64] = l;
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (wave < n) {
        const float m2 = at[0], l2 = at[64], now = fmaxf(m, m2);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - now);
        const float f2 = m2 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m2 - now);
        m = now;
        l = (l == 0.f ? 0.f : l * f) + (l2 == 0.f ? 0.f : l2 * f2);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = o[d] * f + sums[64 * d] * f2;
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
  }
};

template <bool F16, bool F8, int D>
__global__ __launch_bounds__(64 * kWaves<D>) void attention_decode_kernel(DecodeArgs a, DecodeWork work) {
  using W = Decode<F16, F8, D>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W::W * W::kStages * (W::kStage + 256)];
  __shared__ __attribute__((aligned(16))) float room[W::W / 2 * W::kRecord];
  W w(a);
  w.lane = threadIdx.x & 63;
  w.wave = uniform(threadIdx.x >> 6);
  w.col = w.lane & 15;
  w.quad = w.lane >> 4;
  const int group = blockIdx.x % work.groups, worker = blockIdx.x / work.groups;
  w.kv = group / work.per_kv;
  const int shared = a.heads / a.c.kv_heads;
  const int head0 = w.kv * shared + group % work.per_kv * kHeadTile, heads = min(kHeadTile, shared - (head0 - w.kv * shared));

  // The tiles of all sequences, and the sequence in which this worker's begin: every wave
  // for itself, 64 sequences at a time (of fewer than 2^25 tiles each).
  typename W::Walk now;
  int64_t total = 0, before = 0, each = 0;
  int extra = 0;  // a worker has `each` tiles, the first `extra` ones one more
  {
    int len = 0;
    uint32_t n = 0, upto = 0;
    auto chunk = [&](int64_t b0) {
      const int64_t b = b0 + w.lane;
      len = b < a.B ? w.length(b) : 0;
      n = b < a.B ? w.tiles_of(len) : 0;
      upto = wave_scan(n);
      return (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    };
    for (int64_t b0 = 0; b0 < a.B; b0 += 64) total += chunk(b0);
    each = quotient(total, work.workers);
    extra = (int)(total - each * work.workers);
    if (each == 0 && worker >= extra) return;
    before = each * worker + min(worker, extra);
    int64_t base = 0;
    for (int64_t b0 = 0;; b0 += 64) {
      if (a.B > 64) {
        const uint32_t all = chunk(b0);
        if (before - base >= all) {
          base += all;
          continue;
        }
      }
      const int l = __builtin_ctzll(__ballot((uint32_t)(before - base) < upto));
      now.b = (int)b0 + l;
      now.len = __builtin_amdgcn_readlane(len, l);
      now.tiles = __builtin_amdgcn_readlane((int)n, l);
      now.tile = (int)(before - base) - (__builtin_amdgcn_readlane((int)upto, l) - now.tiles);
      break;
    }
  }
  now.left = each + (worker < extra);
  typename W::Walk far = now;  // the tile whose page numbers are asked for next

  w.mine = lds + w.wave * W::kStages * W::kStage;
  const float c = a.scale * kLog2e;
  constexpr int AHEAD = W::kStages - 1;
  uint32_t wrong = 0;  // a bit for each buffer: its tile's page is none
  // A tile's page numbers are asked for behind the loads of the tile AHEAD + 1 before it, and so
  // are there when the one AHEAD before it is: nothing waits for them alone (256 sequences in e4m3
  // 162 us, 163.5 with the numbers asked for ahead of the loads of the tile before).
  uint8_t* const ids = lds + W::W * W::kStages * W::kStage + w.wave * (W::kStages * 256);
  int first_at[AHEAD + 1], len_at[AHEAD + 1];  // of the tiles to load next
  int slot = 0;                                // the buffers of the next one
  int64_t to_load = now.left;
#pragma unroll
  for (int i = 0; i <= AHEAD; ++i) {
    first_at[i] = w.first_of(far);
    len_at[i] = far.len;
    w.pages_to_lds(far, ids + 256 * i);
    w.step(far);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  auto load_next = [&] {
    --to_load;
    const int page = *(const int*)(ids + 256 * slot + 4 * w.lane);
    const bool bad = w.stage(first_at[0], len_at[0], page, w.mine + slot * W::kStage);
    wrong = (wrong & ~(1u << slot)) | (uint32_t)bad << slot;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      first_at[i] = first_at[i + 1];
      len_at[i] = len_at[i + 1];
    }
    first_at[AHEAD] = w.first_of(far);
    len_at[AHEAD] = far.len;
    w.pages_to_lds(far, ids + 256 * slot);
    w.step(far);
    slot = slot == AHEAD ? 0 : slot + 1;
  };
  for (int i = 0; i < AHEAD && to_load > 0; ++i) load_next();
  w.fetch(now.b, head0, heads, w.q);
  // the queries are waited for here: in the loop, waiting for them would wait for the tiles in flight
#pragma unroll
  for (int k = 0; k < W::QS; ++k) asm volatile("" : "+v"(w.q[k]));
  w.begin();
  int from = now.tile;  // the first tile of the present sequence that this worker has
  int64_t tile0 = before - now.tile;  // the number of the sequence's first tile
  bool first_part = true;
  int at = 0;           // the buffer of the present tile
  for (;;) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (to_load > 0) {
      load_next();
      // what came before the last AHEAD tiles and their page numbers is there
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(AHEAD * (W::kPerStage + 1)) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    w.bad |= wrong >> at & 1;
    const bool last = now.left == 1, ends = now.tile + 1 == now.tiles;
    u32x4 next_q[W::QS];
    if (!last && ends) w.fetch(now.b + 1, head0, heads, next_q);
    const int first = now.tile * W::kBlockKeys + w.wave * W::kKeys;
    if (first < now.len) w.tile(w.mine + at * W::kStage, first, now.len, c);
    at = at == AHEAD ? 0 : at + 1;
    if (last || ends) {
      w.join(room);
      const bool whole = from == 0 && ends;
      if (w.wave == 0) {
        if (whole) {
          const float inv = w.l == 0.f ? 0.f : 1.f / w.l;
          if (w.col < heads) {
            const int64_t row = (int64_t)now.b * a.heads + head0 + w.col;
            uint16_t* y = a.y + row * D + 4 * w.quad;
#pragma unroll
            for (int d = 0; d < W::DT; ++d)
              *(u32x2*)(y + 16 * d) = u32x2{W::H::pack(w.o[d].x * inv, w.o[d].y * inv),
                                            W::H::pack(w.o[d].z * inv, w.o[d].w * inv)};
            if (a.lse && w.quad == 0) a.lse[row] = W::H::log_of_sum(w.m, w.l);
          }
        } else {
          float* part = work.parts + (((int64_t)group * work.workers + worker) * 2 + (first_part ? 0 : 1)) *
                                         (kHeadTile * D + 2 * kHeadTile);
#pragma unroll
          for (int d = 0; d < W::DT; ++d) *(f32x4*)(part + w.col * D + 16 * d + 4 * w.quad) = w.o[d];
          if (w.quad == 0) {
            part[kHeadTile * D + w.col] = w.m;
            part[kHeadTile * D + kHeadTile + w.col] = w.l;
          }
        }
        // the worker that has a sequence's first tile says who else has some of it
        if (work.workers > 1 && group == 0 && from == 0 && w.lane == 0) {
          const int64_t t = tile0 + now.tiles - 1, more = extra * (each + 1);
          const int64_t to = t < more ? quotient(t, each + 1) : extra + quotient(t - more, each);
          work.shared[now.b] = int2{first_part ? worker : ~worker, (int)to};
        }
      }
      if (last) return;
      first_part = false;
      from = 0;
      tile0 += now.tiles;
      w.begin();
#pragma unroll
      for (int k = 0; k < W::QS; ++k) {
        w.q[k] = next_q[k];
        asm volatile("" : "+v"(w.q[k]));
      }
    }
    w.step(now);
  }
}

// The shares of a sequence that several workers have, one block for each query head.
template <bool F16, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(DecodeArgs a, DecodeWork work) {
  constexpr int PER = D / 4, SETS = 256 / PER;
  __shared__ f32x4 sums[256];
  __shared__ float weights[SETS];
  const int64_t b = blockIdx.y;
  const int head = blockIdx.x;
  const int2 who = work.shared[b];
  const int w0 = who.x < 0 ? ~who.x : who.x, n = who.y - w0 + 1;
  if (n <= 1) return;
  const int shared = a.heads / a.c.kv_heads, kv = head / shared, in_kv = head - kv * shared;
  const int group = kv * work.per_kv + in_kv / kHeadTile, row = in_kv % kHeadTile;
  constexpr int64_t RECORD = kHeadTile * D + 2 * kHeadTile;
  const float* base = work.parts + ((int64_t)group * work.workers + w0) * 2 * RECORD;
  auto record = [&](int i) { return base + (2 * i + (i == 0 && who.x < 0 ? 1 : 0)) * RECORD; };
  // A thread's first records are asked for ahead of the maximum, kDeep together (one sequence of
  // 131072 54 us, 56 with one record after the other; batches, which have few, alike).
  constexpr int kDeep = 8;
  const int set = threadIdx.x / PER, d = threadIdx.x % PER;
  float m[kDeep], w[kDeep];
  f32x4 v[kDeep];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (i0 + u * SETS >= n) break;
      const float* r = record(i0 + u * SETS);
      m[u] = r[kHeadTile * D + row];
      w[u] = r[kHeadTile * D + kHeadTile + row];
      v[u] = *(const f32x4*)(r + row * D + 4 * d);
    }
  };
  fetch(set);
  float top = -INFINITY;
  for (int i = threadIdx.x & 63; i < n; i += 64) top = fmaxf(top, record(i)[kHeadTile * D + row]);
#pragma unroll
  for (int s = 32; s; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  for (int i0 = set;;) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (i0 + u * SETS >= n) continue;
      const float f = m[u] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[u] - top);
      l += w[u] == 0.f ? 0.f : w[u] * f;
      sum += v[u] * f;
    }
    i0 += kDeep * SETS;
    if (i0 >= n) break;
    fetch(i0);
  }
  sums[threadIdx.x] = sum;
  if (d == 0) weights[set] = l;
  __syncthreads();
  if (set) return;
#pragma unroll
  for (int i = 1; i < SETS; ++i) {
    sum += sums[i * PER + d];
    l += weights[i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t out = b * a.heads + head;
  *(u32x2*)(a.y + out * D + 4 * d) = u32x2{Half<F16>::pack(sum.x * inv, sum.y * inv), Half<F16>::pack(sum.z * inv, sum.w * inv)};
  if (a.lse && d == 0) a.lse[out] = Half<F16>::log_of_sum(top, l);
}

template <bool F16, bool F8, int D>
hipError_t launch(const DecodeArgs& a, DecodeWork w, hipStream_t stream) {
  // at most a worker a tile that can be there
  const int64_t room = std::min<int64_t>((int64_t)a.c.width * a.c.P, 0x7FFFFFFF);
  constexpr int KEYS = Decode<F16, F8, D>::kBlockKeys;
  const int64_t most = a.B * std::max<int64_t>(1, (room + KEYS - 1) / KEYS);
  w.workers = (int)std::min<int64_t>(w.workers, most);
  // Two tiles are gone through in less time than a second launch takes (77 tokens 11 us, 14).
  if (most <= 2) w.workers = 1;
  attention_decode_kernel<F16, F8, D><<<(unsigned)(w.groups * w.workers), 64 * kWaves<D>, 0, stream>>>(a, w);
  if (w.workers > 1)
    attention_join_kernel<F16, D><<<dim3((unsigned)a.heads, (unsigned)a.B), 256, 0, stream>>>(a, w);
  return hipGetLastError();
}

}  // namespace

int64_t decode_workspace_bytes(int64_t B, int heads, int kv_heads, int D) {
  const int64_t groups = groups_of(heads, kv_heads), workers = workers_of(groups);
  if (workers == 1) return 0;
  return up256(groups * workers * 2 * record_floats(D) * 4) + up256(B * 8);
}

hipError_t launch_attention_decode(const DecodeArgs& a, void* ws, hipStream_t stream) {
  DecodeWork w{};
  w.groups = (int)groups_of(a.heads, a.c.kv_heads);
  w.per_kv = w.groups / a.c.kv_heads;
  w.workers = (int)workers_of(w.groups);
  w.parts = (float*)ws;
  w.shared = (int2*)((char*)ws + up256((int64_t)w.groups * w.workers * 2 * record_floats(a.c.D) * 4));
  const bool f8 = a.c.k_scales != nullptr;
  auto by_dim = [&](auto f16, auto e4m3) {
    constexpr bool F = decltype(f16)::value, E = decltype(e4m3)::value;
    return a.c.D == 64 ? launch<F, E, 64>(a, w, stream) : a.c.D == 128 ? launch<F, E, 128>(a, w, stream)
                                                                      : launch<F, E, 256>(a, w, stream);
  };
  if (a.f16) return f8 ? by_dim(std::true_type{}, std::true_type{}) : by_dim(std::true_type{}, std::false_type{});
  return f8 ? by_dim(std::false_type{}, std::true_type{}) : by_dim(std::false_type{}, std::false_type{});
}

}  // namespace moe
