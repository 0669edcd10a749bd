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
//         output's own rounding, which is why fewer bits than fp32's are taken here;
//         an eight whose largest products cancel loses what they hid.  (The other
//         8-bit instructions, 16x16x32 and 32x32x16, cut the same and run at a third
//         to a half of the rate.)
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
typedef float f32x16 __attribute__((ext_vector_type(16)));

// D = A(16 x 128) B(128 x 16), fp32, both operands e4m3.  Lane l supplies row
// l % 16 of A and column l % 16 of B; the order of K inside the group is free
// as long as both operands use the same one.
__device__ __forceinline__ f32x4 mfma_f8_16(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Four e4m3 codes -> four bf16 (exact).
__device__ __forceinline__ u32x2 widen_f8x4(int v) {
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true))};
}

// One lane's 32 values of a group: as codes for the 8-bit instruction, widened, or
// as codes that are widened with every use.
enum { kCodes, kWide, kWidenLater };
template <int MODE>
struct Frag {
  i32x8 v;
  __device__ __forceinline__ void set(i32x8 codes) { v = codes; }
};
template <>
struct Frag<kWide> {
  u32x4 v[4];
  __device__ __forceinline__ void set(i32x8 codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x2 lo = widen_f8x4(codes[2 * i]), hi = widen_f8x4(codes[2 * i + 1]);
      v[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
};
__device__ __forceinline__ f32x4 group_product(const Frag<kCodes>& w, const Frag<kCodes>& a) {
  return mfma_f8_16(w.v, a.v, f32x4{0.f, 0.f, 0.f, 0.f});
}
__device__ __forceinline__ f32x4 group_product(const Frag<kWide>& w, const Frag<kWide>& a) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = mfma16(w.v[i], a.v[i], s);
  return s;
}

// ------------------------------------------------------------------ tiled kernel
// A block computes BN rows of w times BM tokens, a wave WTN x WTM of them as 32 x
// 32 matrix-core tiles.  One group of every row of the block, BN + BM rows of 128
// bytes, is staged in LDS by loads that go there directly; two buffers, so the
// next group arrives while this one is multiplied.
// 4096 x 8192 x 4096 (tokens x rows x K) to bf16: 137 us, 2010 TFLOP/s, the matrix
// cores busy 47% of the time, the rest the staging and the reads of LDS beside
// them (1.9 us a group, its products 0.9).  1 x 50304 x 2048 to fp32, 128 x 32
// tiles: 19.7 us, 5.2 TB/s of weights.
//
// A staging load writes 64 consecutive pieces of 16 bytes, eight rows, in lane
// order, so the swizzle that keeps the reads off each other's banks is in the
// lane's source address: piece p of row r is kept at place p ^ f(r) of the row,
// f(r) = r % 8 ^ r / 8 % 2, which is distinct over eight consecutive rows and over
// the even and the odd rows of sixteen.
__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

__device__ __forceinline__ f32x16 mfma_f8_32(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x16 half_product(const Frag<kCodes>& w, const Frag<kCodes>& a, f32x16 c) {
  return mfma_f8_32(w.v, a.v, c);
}
__device__ __forceinline__ f32x16 half_product(const Frag<kWide>& w, const Frag<kWide>& a, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma32(w.v[i], a.v[i], c);
  return c;
}
__device__ __forceinline__ f32x16 half_product(const Frag<kWidenLater>& w, const Frag<kWidenLater>& a, f32x16 c) {
  Frag<kWide> wide_w, wide_a;
  wide_w.set(w.v);
  wide_a.set(a.v);
  return half_product(wide_w, wide_a, c);
}

// A number that the compiler no longer knows: what is computed from it is not kept
// over a loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Lane l's 32 bytes of half h of a staged row: pieces 4 h + 2 (l / 32) and the
// next.  `at`: the place of half 0's first piece; the others differ from it in one
// or two address bits.
__device__ __forceinline__ int staged_at(int row, int q) { return row * kF8Group + 16 * ((2 * q) ^ swizzle(row)); }
template <int MODE>
__device__ __forceinline__ Frag<MODE> staged_frag(const uint8_t* buf, int at, int h) {
  const u32x4 lo = *(const u32x4*)(buf + (at ^ 64 * h)), hi = *(const u32x4*)(buf + (at ^ (64 * h + 16)));
  Frag<MODE> r;
  r.set(i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w});
  return r;
}

// A buffer descriptor over the bytes from p on (the lanes' offsets stay inside),
// or over none (bytes = 0): loads through that one touch no memory.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes = -1) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00027000);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t src, uint32_t lane_off, int off, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16, (int)lane_off, off, 0, 0);
}

template <int BN, int BM, int WTN, int WTM, int NB, bool F32>
struct Tile {
  static constexpr int kWavesN = BN / WTN, kWaves = kWavesN * (BM / WTM), kThreads = 64 * kWaves;
  static constexpr int TN = WTN / 32, TM = WTM / 32;
  // a single tile uses its operands once: widened with the use, they are not waited for when they are read
  // (1 x 50304 x 2048 to fp32)
  static constexpr int kMode = !F32 ? kCodes : TN * TM == 1 ? kWidenLater : kWide;
  static constexpr int kLoads = (BN + BM) / 8 / kWaves;  // staging loads of a wave per group
  static constexpr int kPerTile = TN * TM > 1 ? 2 * kLoads / (TN * TM) : kLoads;  // ... and behind a tile's product
  static constexpr int kBufBytes = (BN + BM) * kF8Group;

  f32x16 acc[TN][TM], t[2];
  Frag<kMode> fa[TM][2], fw[2][2];
  float s[TM], raw[NB][TM];  // the pending products' scales; the tokens' scales of the groups in the buffers
  const uint8_t *w, *a;
  int lane, wave, wn, wm, K, groups, last_n, last_m;
  int at_w, at_a;  // the lane's places in the wave's first 32 rows of w and of a (a tile's rows keep the swizzle)

  // A wave's loads: eight rows each, kWaves chunks apart (a multiple of 16 rows:
  // one swizzle for all).  Rows past the matrix repeat its last row; their results
  // are not stored.  Past the last group nothing is loaded, without a branch: one
  // would let the compiler move the additions behind it past it, and keep every
  // product.  The lanes' offsets are made anew each time: kept, they would take
  // eight registers that the products need.
  __device__ __forceinline__ void stage(uint8_t* buf, int g, int first = 0, int last = kLoads) const {
    const int tid = opaque(threadIdx.x), row0 = tid >> 3, piece = 16 * ((tid & 7) ^ swizzle(row0));
    const int bytes = __builtin_amdgcn_readfirstlane((g - groups) >> 31);
    const __amdgpu_buffer_rsrc_t from_w = buffer_of(w, bytes), from_a = buffer_of(a, bytes);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < first || i >= last) continue;
      const bool of_w = i * kWaves < BN / 8;
      const int row = min(row0 + (i * kWaves * 8 - (of_w ? 0 : BN)), of_w ? last_n : last_m);
      load_to_lds(of_w ? from_w : from_a, __umul24(row, K) + piece, g * kF8Group, buf + (wave + i * kWaves) * 1024);
    }
  }

  __device__ __forceinline__ void scale_add(int i, int j, const f32x16& t, float s) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][j][e] += t[e] * s;
  }

  __device__ __forceinline__ void read_w(const uint8_t* buf, int i, Frag<kMode> (&f)[2]) const {
    const int at = opaque(at_w);
#pragma unroll
    for (int h = 0; h < 2; ++h) f[h] = staged_frag<kMode>(buf + 32 * kF8Group * i, at, h);
  }
  __device__ __forceinline__ void read_a(const uint8_t* buf, int j) {
    const int at = opaque(at_a);
#pragma unroll
    for (int h = 0; h < 2; ++h) fa[j][h] = staged_frag<kMode>(buf + (BN + 32 * j) * kF8Group, at, h);
  }

  // The wave's results through LDS: token rows of WTN results, pieces of 16 bytes
  // kept at place p ^ token % pieces so that neither side meets in a bank, then 16
  // bytes a lane, whole rows a wave.
  __device__ __forceinline__ void store(const F8LinearArgs& p, uint8_t* buf, int64_t m, int64_t n) const {
    constexpr int SIZE = F32 ? 4 : 2, PER = 16 / SIZE, PIECES = WTN / PER;
    static_assert(WTM * WTN * SIZE * (kWaves / 2) <= kBufBytes, "the waves' shares fit");
    uint8_t* mine = buf + (wave % (kWaves / 2)) * (WTM * WTN * SIZE);
    const int c = lane & 31, q = lane >> 5;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int token = 32 * j + c;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = 32 * i + 8 * e + 4 * q, piece = (at / PER) ^ (token % PIECES);
          const f32x4 v = {acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
          uint8_t* to = mine + token * (WTN * SIZE) + 16 * piece + (at % PER) * SIZE;
          if (F32) *(f32x4*)to = v;
          else *(u32x2*)to = u32x2{f32x2_to_bf16x2(v.x, v.y), f32x2_to_bf16x2(v.z, v.w)};
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const bool whole = p.ldy % PER == 0 && (uintptr_t)p.y % 16 == 0;
    const int piece = lane % PIECES;
    const int64_t col = n + piece * PER;
#pragma unroll
    for (int k = 0; k < WTM * PIECES / 64; ++k) {
      const int token = lane / PIECES + k * (64 / PIECES);
      const u32x4 v = *(const u32x4*)(mine + token * (WTN * SIZE) + 16 * (piece ^ (token % PIECES)));
      if (m + token >= p.M) continue;
      uint8_t* to = (uint8_t*)p.y + ((m + token) * p.ldy + col) * SIZE;
      if (whole && col + PER <= p.N) {
        *(u32x4*)to = v;
      } else {
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          if (col + x >= p.N) break;
          if (F32) ((uint32_t*)to)[x] = v[x];
          else ((uint16_t*)to)[x] = (uint16_t)(v[x / 2] >> (16 * (x & 1)));
        }
      }
    }
  }

  // Group g, whose bytes are in `now`, its tokens' operands and the first of w's
  // already read.  A 32 x 32 tile's product is scaled and added while the matrix
  // core works on the next one.  When the last row of tiles has begun, every read
  // of `now` has been made and the next group's bytes have arrived in `then`: the
  // block meets at the one barrier and `now` takes the loads of group g + NB, a few
  // behind each of the next tiles' products, half a group's worth of them (all at
  // once they cost 10%: they stand in the way of the reads); `last` takes the rest
  // of those that the group before began.  The next group's first operands are
  // read behind the last tiles' products.  The scheduling barriers keep the
  // compiler from issuing all products first, whose results would not fit the
  // registers.
  template <int SLOT, class Meet, class Scales>
  __device__ __forceinline__ void step(uint8_t* now, uint8_t* then, uint8_t* last, int g, float sw, Meet meet,
                                       Scales read_scales) {
    constexpr int N = TN * TM;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = n / TM, j = n % TM, at = SLOT * N + n, slot = (SLOT * TN + i) & 1;
      if (j == 0 && i + 1 < TN) read_w(now, i + 1, fw[slot ^ 1]);
      f32x16& mine = t[at & 1];
      mine = half_product(fw[slot][0], fa[j][0], f32x16{});
      mine = half_product(fw[slot][1], fa[j][1], mine);
      __builtin_amdgcn_sched_barrier(0);
      const f32x16& done = t[(at & 1) ^ 1];
      if (n) {
        scale_add((n - 1) / TM, (n - 1) % TM, done, s[(n - 1) % TM]);
      } else {  // the last product of the group before, by its own scale
        scale_add(TN - 1, TM - 1, done, s[TM - 1]);
#pragma unroll
        for (int k = 0; k < TM; ++k) s[k] = raw[SLOT][k] * sw;
      }
      __builtin_amdgcn_sched_barrier(0);
      if (n == N - TM) {
        meet();
        read_w(then, 0, fw[slot ^ 1]);
        read_scales(raw[SLOT], g + NB);
      }
      if (i == TN - 1) read_a(then, j);
      const int k = (n + TM) % N * kPerTile;  // the loads go on into the next group's first tiles
      if (k < kLoads) stage(i == TN - 1 ? now : last, i == TN - 1 ? g + NB : g + NB - 1, k, k + kPerTile);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The block meets when every wave has at most N loads on their way and its LDS
// operations are done.  (__syncthreads() would wait for every staging load.)
template <int N>
__device__ __forceinline__ void meet_with_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int BN, int BM, int WTN, int WTM, int NB, bool F32>
__global__ __launch_bounds__(64 * (BN / WTN) * (BM / WTM), 2) void fp8_tile_kernel(F8LinearArgs p, int tiles_n) {
  typedef Tile<BN, BM, WTN, WTM, NB, F32> T;
  static_assert((BN / 8) % T::kWaves == 0 && (BM / 8) % T::kWaves == 0 && T::kWaves % 2 == 0,
                "a wave's staging loads split evenly, 16 rows or a multiple apart");
  static_assert(NB == 2 || NB == 4, "an even number of buffers, as step() counts them");
  // separate arrays: the compiler sees that a read does not wait for the loads of another buffer
  __shared__ __attribute__((aligned(1024))) uint8_t buf0[T::kBufBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t buf1[T::kBufBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t buf2[NB == 4 ? T::kBufBytes : 1024];
  __shared__ __attribute__((aligned(1024))) uint8_t buf3[NB == 4 ? T::kBufBytes : 1024];
  // consecutive blocks go to the eight XCDs in turn: each XCD takes a contiguous
  // run of tiles, whose rows of w and a meet in its L2
  const int tiles = gridDim.x, per = (tiles + 7) / 8, rest = tiles % 8 ? tiles % 8 : 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int tile = xcd < rest ? xcd * per + at : rest * per + (xcd - rest) * (per - 1) + at;
  // ... and goes through it in bands of eight tiles of tokens: the 32 tiles that an
  // XCD works on at a time are 8 x 4, 12 tiles' rows for its L2 to fetch
  const int tiles_m = tiles / tiles_n, band = tile / (8 * tiles_n), in_band = tile - band * 8 * tiles_n;
  const int height = min(8, tiles_m - 8 * band);
  const int64_t m0 = (int64_t)(8 * band + in_band % height) * BM, n0 = (int64_t)(in_band / height) * BN;
  const int groups = p.K / kF8Group;
  const int last_n = (int)min((int64_t)BN, p.N - n0) - 1, last_m = (int)min((int64_t)BM, p.M - m0) - 1;

  T t;
  t.lane = threadIdx.x & 63;
  t.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  t.wn = t.wave % T::kWavesN;
  t.wm = t.wave / T::kWavesN;
  t.w = p.w + n0 * p.K;
  t.a = p.a + m0 * p.K;
  t.at_w = staged_at(t.wn * WTN + (t.lane & 31), t.lane >> 5);
  t.at_a = staged_at(t.wm * WTM + (t.lane & 31), t.lane >> 5);
  t.K = p.K;
  t.groups = groups;
  t.last_n = last_n;
  t.last_m = last_m;
#pragma unroll
  for (int i = 0; i < T::TN; ++i)
#pragma unroll
    for (int j = 0; j < T::TM; ++j) t.acc[i][j] = f32x16{};

  const __amdgpu_buffer_rsrc_t sa = buffer_of(p.a_scales + m0 * groups);
  // constant address space: the wave's scales of w come through scalar loads
  const auto sw = (const __attribute__((address_space(4))) float*)(p.w_scales +
                                                                   min(n0 + t.wn * WTN, p.N - 1) / kF8Group * groups);
  auto read_scales = [&](float (&to)[T::TM], int g) {
    const int token = t.wm * WTM + (opaque(threadIdx.x) & 31);
#pragma unroll
    for (int j = 0; j < T::TM; ++j)
      to[j] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(sa, 4 * __umul24(min(token + 32 * j, last_m), groups),
                                                      4 * min(g, groups - 1), 0));
  };
  // groups 0 .. NB - 1 begin; of the last one as much as step 0 does not go on with
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    read_scales(t.raw[i], i);
    t.stage(i == 0 ? buf0 : i == 1 ? buf1 : i == 2 ? buf2 : buf3, i, 0, i < NB - 1 ? T::kLoads : T::TM * T::kPerTile);
  }
  meet_with_loads<(NB - 2) * T::kLoads>();
#pragma unroll
  for (int j = 0; j < T::TM; ++j) {
    t.read_a(buf0, j);
    t.s[j] = 0.f;
  }
  t.read_w(buf0, 0, t.fw[0]);
  t.t[1] = f32x16{};  // no product is pending before the first
  // the loads of the NB - 2 groups after the next may go on
  auto meet = [&] { meet_with_loads<(NB - 2) * T::kLoads>(); };
  int g = 0;
  for (; g + NB <= groups; g += NB) {
    t.template step<0>(buf0, buf1, NB == 2 ? buf1 : buf3, g, sw[g], meet, read_scales);
    t.template step<1>(buf1, NB == 2 ? buf0 : buf2, buf0, g + 1, sw[g + 1], meet, read_scales);
    if (NB == 4) {
      t.template step<2 % NB>(buf2, buf3, buf1, g + 2, sw[g + 2], meet, read_scales);
      t.template step<3 % NB>(buf3, buf0, buf2, g + 3, sw[g + 3], meet, read_scales);
    }
  }
  if (g < groups) t.template step<0>(buf0, buf1, NB == 2 ? buf1 : buf3, g, sw[g], meet, read_scales);
  if (NB == 4 && g + 1 < groups) t.template step<1>(buf1, buf2, buf0, g + 1, sw[g + 1], meet, read_scales);
  if (NB == 4 && g + 2 < groups) t.template step<2 % NB>(buf2, buf3, buf1, g + 2, sw[g + 2], meet, read_scales);
  // the last product is pending in t[1], after an odd number of single-tile groups in t[0]
  if (T::TN * T::TM % 2 && groups % 2) t.scale_add(T::TN - 1, T::TM - 1, t.t[0], t.s[T::TM - 1]);
  else t.scale_add(T::TN - 1, T::TM - 1, t.t[1], t.s[T::TM - 1]);
  // no staging load is on its way any more: each wave turns its results round in
  // its share of the buffers and writes whole lines of y
  meet_with_loads<0>();
  t.store(p, t.wave < T::kWaves / 2 ? buf0 : buf1, m0 + t.wm * WTM, n0 + t.wn * WTN);
}

template <int BN, int BM, int WTN, int WTM, int NB, bool F32>
hipError_t launch_tiles(const F8LinearArgs& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + BN - 1) / BN, tiles = tiles_n * ((a.M + BM - 1) / BM);
  fp8_tile_kernel<BN, BM, WTN, WTM, NB, F32>
      <<<(unsigned)tiles, Tile<BN, BM, WTN, WTM, NB, F32>::kThreads, 0, stream>>>(a, (int)tiles_n);
  return hipGetLastError();
}

// ------------------------------------------------------------------ split kernel
// Few tokens and few rows of w: too few tiles to fill the card, and K the only
// axis left to share out.  A block takes 16 RT rows of w and 16 MT tokens, its
// eight waves the groups of K in turn.  Each wave stages its own groups in LDS
// (loads of whole lines: straight into registers a load would touch 16 rows, and
// ran at half the rate), two at a time, and waits for nobody; the waves' sums meet
// in LDS at the end and are added in wave order.  Bound by latency: 32 x 4096 x 2048
// takes 5.2 us, of which a launch with one trip to memory is half.
constexpr int kSplitWaves = 8;

template <int RT, int MT, bool F32>
__global__ __launch_bounds__(64 * kSplitWaves) void fp8_split_kernel(F8LinearArgs p) {
  constexpr int ROWS = 16 * (RT + MT), LOADS = ROWS / 8, BYTES = kSplitWaves * ROWS * kF8Group;
  typedef float Part[RT * MT][16][17];  // [tile][token][row], a row of 16 padded by one
  static_assert(sizeof(Part) * kSplitWaves <= BYTES, "the sums fit a buffer");
  __shared__ __attribute__((aligned(1024))) uint8_t buf0[BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t buf1[BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15,
            q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT), m0 = (int64_t)blockIdx.y * (16 * MT);
  const int groups = p.K / kF8Group;
  const int last_n = (int)min((int64_t)16 * RT, p.N - n0) - 1, last_m = (int)min((int64_t)16 * MT, p.M - m0) - 1;
  uint32_t off[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {  // rows past the matrix repeat its last row; their results are not stored
    const int row = 8 * i + (lane >> 3);
    off[i] = __umul24(i < 2 * RT ? min(row, last_n) : min(row - 16 * RT, last_m), p.K) +
             16 * ((lane & 7) ^ swizzle(row));
  }
  const __amdgpu_buffer_rsrc_t scales = buffer_of(p.a_scales + m0 * groups);
  const auto sw = (const __attribute__((address_space(4))) float*)(p.w_scales + n0 / kF8Group * groups);
  float s0[MT], s1[MT];
  auto load = [&](uint8_t* buf, float (&s)[MT], int g) {  // past the last group nothing is loaded
    const int at = min(g, groups - 1), bytes = __builtin_amdgcn_readfirstlane((g - groups) >> 31);
#pragma unroll
    for (int i = 0; i < MT; ++i)
      s[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                           scales, 4 * __umul24(min(16 * i + c, last_m), groups), 4 * at, 0));
    const __amdgpu_buffer_rsrc_t from_w = buffer_of(p.w + n0 * p.K, bytes), from_a = buffer_of(p.a + m0 * p.K, bytes);
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      load_to_lds(i < 2 * RT ? from_w : from_a, off[i], at * kF8Group, buf + (wave * ROWS + 8 * i) * kF8Group);
  };
  f32x4 acc[RT][MT] = {};
  auto multiply = [&](const uint8_t* buf, const float (&s)[MT], int g) {
    const float of_w = sw[g];
    // lane quarter q's 32 bytes of a row: pieces 2 q and the next
    const uint8_t* at = buf + wave * ROWS * kF8Group + c * kF8Group;
    const int first = 16 * ((2 * q) ^ swizzle(c));
    auto frag = [&](int tile) {
      const u32x4 lo = *(const u32x4*)(at + tile * 16 * kF8Group + first),
                  hi = *(const u32x4*)(at + tile * 16 * kF8Group + (first ^ 16));
      Frag<F32 ? kWide : kCodes> f;
      f.set(i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w});
      return f;
    };
    Frag<F32 ? kWide : kCodes> fw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) fw[r] = frag(r);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const Frag<F32 ? kWide : kCodes> fa = frag(RT + i);
      const float f = s[i] * of_w;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const f32x4 t = group_product(fw[r], fa);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[r][i][j] += t[j] * f;
      }
    }
  };
  // this wave's loads of one buffer have arrived (those of the other may go on);
  // its reads of a buffer are done before new loads write there
  auto arrived = [] { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory"); };
  auto read = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  load(buf0, s0, wave);
  load(buf1, s1, wave + kSplitWaves);
  for (int g = wave; g < groups; g += 2 * kSplitWaves) {
    arrived();
    multiply(buf0, s0, g);
    read();
    load(buf0, s0, g + 2 * kSplitWaves);
    arrived();
    if (g + kSplitWaves < groups) multiply(buf1, s1, g + kSplitWaves);
    read();
    load(buf1, s1, g + 3 * kSplitWaves);
  }
  meet_with_loads<0>();
  Part* part = (Part*)buf0;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[wave][r * MT + i][c][4 * q + j] = acc[r][i][j];
  __syncthreads();
  for (int k = threadIdx.x; k < MT * RT * 256; k += 64 * kSplitWaves) {
    const int tile = k >> 8, row = k & 15, col = (k >> 4) & 15;
    const int64_t t = m0 + 16 * (tile % MT) + col, n = n0 + 16 * (tile / MT) + row;
    float y = part[0][tile][col][row];
#pragma unroll
    for (int v = 1; v < kSplitWaves; ++v) y += part[v][tile][col][row];
    if (t < p.M && n < p.N) {
      if (F32) ((float*)p.y)[t * p.ldy + n] = y;
      else ((uint16_t*)p.y)[t * p.ldy + n] = (uint16_t)f32_to_bf16(y);
    }
  }
}

template <int RT, int MT, bool F32>
hipError_t launch_split(const F8LinearArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  fp8_split_kernel<RT, MT, F32><<<grid, 64 * kSplitWaves, 0, stream>>>(a);
  return hipGetLastError();
}

// The largest tile of which there are enough for three quarters of the 256 CUs,
// whose token side (above 32) is not half empty: a larger tile reads less per
// product, but each takes its time alone.  Microseconds for 4096 x 4096 x 4096, 1024 x 4096 x
// 4096, 512 x 4096 x 4096 and 333 x 2561 x 4096 tokens x rows x K to bf16:
//   256 x 256   73   -    -    -       (fp32 results do not fit the registers)
//   128 x 128   94   26   22   23
//   128 x 64    -    36   19   19
//    64 x 64    -    39   21   14
// Between one and two rounds of 256 x 256 tiles, 4096 x n x 4096 (another run):
//     n        4096 4352 5120 6144 7168 8192
//   256 x 256    78  113  113  117  126  137
//   128 x 128   104  109  113  130  157  187
// Four buffers where a CU has one block (1024 tokens: 26 us, two: 29), two where
// a second block fills the gaps (2048 x 4096 x 2048: 25.5 us, four: 28).  Where even
// the small tiles are too few, the split kernel with the largest block that there
// are 256 of (64 x 1024 x 8192: 6.9 us, 64 x 32 tiles 19; 64 x 8192 x 4096: 16, tiles 12).
template <bool F32>
hipError_t launch(const F8LinearArgs& a, hipStream_t stream) {
  constexpr int64_t CUS = 256;
  auto blocks = [&](int64_t n, int64_t m) { return ((a.N + n - 1) / n) * ((a.M + m - 1) / m); };
  auto fills = [&](int64_t n, int64_t m) { return (m == 32 || m < 2 * a.M) && 4 * blocks(n, m) >= 3 * CUS; };
  if (!F32 && fills(256, 256)) return launch_tiles<256, 256, 128, 64, 2, false>(a, stream);
  if (F32 && fills(128, 128) && blocks(128, 128) > CUS)  // larger wave tiles: fewer operands to widen
    return launch_tiles<128, 128, 64, 64, 2, true>(a, stream);
  if (fills(128, 128))
    return blocks(128, 128) <= CUS ? launch_tiles<128, 128, 64, 32, 4, F32>(a, stream)
                                   : launch_tiles<128, 128, 64, 32, 2, F32>(a, stream);
  if (fills(128, 64))
    return blocks(128, 64) <= CUS ? launch_tiles<128, 64, 32, 32, 4, F32>(a, stream)
                                  : launch_tiles<128, 64, 64, 32, 2, F32>(a, stream);
  if (fills(64, 64)) return launch_tiles<64, 64, 32, 32, 4, F32>(a, stream);
  if (fills(128, 32)) return launch_tiles<128, 32, 32, 32, 4, F32>(a, stream);
  if (fills(64, 32)) return launch_tiles<64, 32, 32, 32, 4, F32>(a, stream);
  if (a.M > 16 && blocks(32, 32) >= CUS) return launch_split<2, 2, F32>(a, stream);
  if (blocks(32, 16) >= CUS) return launch_split<2, 1, F32>(a, stream);
  return launch_split<1, 1, F32>(a, stream);
}

}  // namespace

hipError_t launch_fp8_linear(const F8LinearArgs& a, hipStream_t stream) {
  return a.f32 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace moe
