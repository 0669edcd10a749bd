// Attention over whole prompts for gfx950: packed sequences, grouped heads,
//   y_i = sum_j p_ij v_j,   p_ij = exp(s_ij - m_i) / sum_j exp(s_ij - m_i),   s_ij = scale q_i k_j
// over the keys j that query i sees: all of its sequence, or (causal) those up to
// i + lk - lq for lq queries that end where lk keys end.  One pass over the keys with
// the running maximum m and sum l of the softmax in fp32.
//
// A block takes 128 queries of one head, a wave 32 of them, and walks over tiles of
// keys and values in LDS.  Scores are formed transposed, S^T = K Q^T: a lane's results
// belong to one query, so the softmax needs one exchange between the wave's halves, and
// they stand as the second operand of y^T = V^T P^T wants them: the order of the keys
// inside a product is free, and the transposing reads of V follow the order in which
// the scores lie.  P is rounded to the values' type (nearest even) for the matrix cores;
// each p is off by half a step of itself, as y is by its own rounding, and l is summed
// before the rounding.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attention_device.h"
#include "attention_internal.h"

namespace moe {

namespace {

constexpr int kQRows = 128;  // queries of a block

// Keys of a tile: 64, of the widest heads 32, so that two tiles of keys and values take
// 64 KB of LDS and two blocks share a CU.
template <int D>
constexpr int kTileKeys = D == 256 ? 32 : 64;

// Piece p (16 bytes) of row r of a tile is kept at place p ^ f(r) of the row.  Sixteen
// rows read at one piece, and four consecutive rows read at four, spread over all banks.
template <int D>
__device__ __forceinline__ int swizzle(int r) {
  return D == 64 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3) : (r & 3) << 2 | ((r >> 2) & 3);
}

// The unit-th tile of queries: its sequence's first query and key, their numbers, and
// the tile's place, counted from the end (the last queries see the most keys).
struct Place {
  int q0, k0, lq, lk, tile;
  bool found;
};
__device__ __forceinline__ Place find_tile(const PrefillArgs& a, int64_t unit) {
  const int lane = threadIdx.x & 63;
  Place r{};
  for (int64_t c = 0; c < a.n; c += 64) {
    const int64_t i = c + lane;
    int from = 0, to = 0;
    if (i < a.n) {
      from = (int)min((int64_t)max(a.q_starts[i], 0), a.Tq);
      to = (int)min((int64_t)max(a.q_starts[i + 1], from), a.Tq);
    }
    const int tiles = (int)(((int64_t)to - from + kQRows - 1) / kQRows);
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int other = __shfl_up(upto, o, 64);
      if (lane >= o) upto += other;
    }
    const uint64_t past = __ballot(unit < upto);
    if (past) {
      const int l = __builtin_ctzll(past);
      r.q0 = __builtin_amdgcn_readlane(from, l);
      r.lq = __builtin_amdgcn_readlane(to, l) - r.q0;
      r.tile = __builtin_amdgcn_readlane(upto, l) - 1 - (int)unit;
      const int64_t s = c + l;
      const int k0 = (int)min((int64_t)max(a.k_starts[s], 0), a.Tk);
      r.k0 = __builtin_amdgcn_readfirstlane(k0);
      r.lk = __builtin_amdgcn_readfirstlane((int)min((int64_t)max(a.k_starts[s + 1], k0), a.Tk) - k0);
      r.found = true;
      return r;
    }
    unit -= __builtin_amdgcn_readlane(upto, 63);
  }
  return r;
}

template <bool F16, int D>
struct Prefill {
  using H = Half<F16>;
  static constexpr int BN = kTileKeys<D>, KT = BN / 32, DT = D / 32, KS = D / 16;
  static constexpr int kRow = 2 * D, kTile = BN * kRow;  // bytes of a row and of a tile
  static constexpr int kLoads = kTile / 1024 / 4;        // staging loads of a wave

  u32x4 q[KS];
  f32x16 o[DT];
  float m, l;
  int lane, wave, half, lim;  // lim: the last key that the lane's query sees

  // Tile `first` of the keys or values: a wave's load fills 1024 bytes, whole rows.  Rows
  // behind the last key repeat it; they are masked.
  __device__ __forceinline__ void stage(const uint16_t* base, int64_t stride, int first, int lk, uint8_t* dst) const {
    constexpr int PER = kRow / 16, ROWS = 64 / PER;  // pieces of a row, rows of a load
    const __amdgpu_buffer_rsrc_t src = rows_from(base + first * stride);
    const int last = lk - 1 - first;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (wave + 4 * i) * ROWS + lane / PER, piece = (lane % PER) ^ swizzle<D>(row);
      copy_to_lds(src, (uint32_t)min(row, last) * (uint32_t)(2 * stride) + 16 * piece, dst + (wave + 4 * i) * 1024);
    }
  }

  // One tile of keys and values.  masked: some query of the wave does not see all of it.
  __device__ __forceinline__ void tile(const uint8_t* ks, const uint8_t* vs, int first, float c, bool masked) {
    f32x16 s[KT];
    const int krow = lane & 31, kat = krow * kRow + ((half ^ swizzle<D>(krow)) << 4);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      s[t] = f32x16{};
#pragma unroll
      for (int k = 0; k < KS; ++k) s[t] = H::mfma32(*(const u32x4*)(ks + 32 * t * kRow + (kat ^ (k << 5))), q[k], s[t]);
    }
    if (masked) {
      const int seen = lim - first - 4 * half;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * t + 8 * (i / 4) + i % 4 > seen) s[t][i] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
    const f32x2_t tops = both_halves(top);
    top = fmaxf(tops.x, tops.y) * c;
    // The maximum that is subtracted may lag 2^8 behind the true one: the sums stay far
    // inside fp32, and y is scaled anew only when a query's maximum really moves.
    if (__any(top > m + 8.f)) {
      const float now = fmaxf(m, top), f = now == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    const float off = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(s[t][i] * c - off);
        sum += s[t][i];
      }
    l += sum;
    const int g = lane >> 4, i16 = lane & 15;
    int vat[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * r + 4 * half + (i16 >> 2), piece = 2 * (g & 1) + ((i16 & 3) >> 1);
      vat[r] = row * kRow + ((piece ^ swizzle<D>(row)) << 4) + 8 * (i16 & 1);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        u32x4 p;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = H::pack(s[t][8 * k + 2 * e], s[t][8 * k + 2 * e + 1]);
        const uint8_t* at = vs + (32 * t + 16 * k) * kRow;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const u32x2 lo = read_transposed(at + (vat[0] ^ (d << 6))), hi = read_transposed(at + (vat[1] ^ (d << 6)));
          o[d] = H::mfma32(u32x4{lo.x, lo.y, hi.x, hi.y}, p, o[d]);
        }
      }
  }

  // A weight of zero does not remove a value that is infinite or NaN.  Where a tile is
  // hidden in part and holds such values, they take part in the product as zeros and are
  // added here to the queries that see them.
  __device__ __forceinline__ void clear(uint8_t* vs) const {
    for (int i = threadIdx.x; i < kTile / 16; i += 256) {
      u32x4 v = *(const u32x4*)(vs + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((v[e] & H::kExponent) == H::kExponent) v[e] &= 0xFFFF0000u;
        if ((v[e] >> 16 & H::kExponent) == H::kExponent) v[e] &= 0xFFFFu;
      }
      *(u32x4*)(vs + 16 * i) = v;
    }
  }
  __device__ __forceinline__ void add_cleared(const uint16_t* v, int64_t stride, int first, int end) {
#pragma unroll 1
    for (int j = first; j < end; ++j) {
      const uint16_t* row = v + j * stride + 4 * half;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u32x2 x = *(const u32x2*)(row + 32 * d + 8 * e);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b = x[i / 2] >> (16 * (i & 1));
            if ((b & H::kExponent) == H::kExponent && j <= lim) o[d][4 * e + i] += H::widen(b & 0xFFFFu);
          }
        }
    }
  }
};

template <bool F16, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attention_prefill_kernel(PrefillArgs a, int64_t units) {
  using W = Prefill<F16, D>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * W::kTile];
  __shared__ int redo;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int head = (int)(block % a.heads);
  const Place at = find_tile(a, block / a.heads);
  if (!at.found) return;
  W w;
  w.lane = threadIdx.x & 63;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  w.half = w.lane >> 5;
  const int first_row = at.tile * kQRows + 32 * w.wave, row = first_row + (w.lane & 31);
  const int behind = a.causal ? at.lk - at.lq : 0;  // keys before the first query's own
  w.lim = a.causal ? min(row + behind, at.lk - 1) : at.lk - 1;
  const int64_t token = at.q0 + min(row, at.lq - 1);
  const uint16_t* qp = a.q.p + token * a.q.token + head * a.q.head + 8 * w.half;
#pragma unroll
  for (int k = 0; k < W::KS; ++k) w.q[k] = *(const u32x4*)(qp + 16 * k);
  const int kv = head / (a.heads / a.kv_heads);
  const uint16_t* kp = a.k.p + at.k0 * a.k.token + kv * a.k.head;
  const uint16_t* vp = a.v.p + at.k0 * a.v.token + kv * a.v.head;
  // keys that the block's and the wave's queries see, and those that all of the wave's see
  auto end = [&](int r) { return a.causal ? max(min(min(r, at.lq - 1) + behind + 1, at.lk), 0) : at.lk; };
  const int block_end = end(at.tile * kQRows + kQRows - 1);
  const int seen_by_all = a.causal ? end(at.tile * kQRows) : at.lk;
  const int wave_end = first_row < at.lq ? end(first_row + 31) : 0, all_end = a.causal ? end(first_row) : at.lk;
  const float c = a.scale * kLog2e;
  const int tiles = (block_end + W::BN - 1) / W::BN;
  for (int careful = 0;; ++careful) {
    w.m = -INFINITY;
    w.l = 0.f;
#pragma unroll
    for (int d = 0; d < W::DT; ++d) w.o[d] = f32x16{};
    if (tiles > 0) {
      w.stage(kp, a.k.token, 0, at.lk, lds);
      w.stage(vp, a.v.token, 0, at.lk, lds + W::kTile);
    }
    for (int t = 0; t < tiles; ++t) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      uint8_t* now = lds + (t & 1) * 2 * W::kTile;
      uint8_t* then = lds + (~t & 1) * 2 * W::kTile;
      const int first = t * W::BN;
      if (t + 1 < tiles) {
        w.stage(kp, a.k.token, first + W::BN, at.lk, then);
        w.stage(vp, a.v.token, first + W::BN, at.lk, then + W::kTile);
      }
      const bool cleared = careful && first + W::BN > seen_by_all;
      if (cleared) {
        w.clear(now + W::kTile);
        __syncthreads();
      }
      if (first >= wave_end) continue;
      w.tile(now, now + W::kTile, first, c, first + W::BN > all_end);
      if (cleared) w.add_cleared(vp, a.v.token, first, min(first + W::BN, at.lk));
    }
    // A result that is not finite: a value that a query must not see may have got in, so
    // the tiles that are hidden in part are gone through with care.
    if (careful) break;
    bool bad = false;
#pragma unroll
    for (int d = 0; d < W::DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) bad |= !(__builtin_fabsf(w.o[d][i]) < INFINITY);
    if (threadIdx.x == 0) redo = 0;
    __syncthreads();
    if (bad) redo = 1;
    __syncthreads();
    if (!redo) break;
  }
  const f32x2_t sums = both_halves(w.l);
  const float sum = sums.x + sums.y;
  if (row >= at.lq) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* y = a.y + (token * a.heads + head) * D + 4 * w.half;
#pragma unroll
  for (int d = 0; d < W::DT; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *(u32x2*)(y + 32 * d + 8 * e) = u32x2{W::H::pack(w.o[d][4 * e] * inv, w.o[d][4 * e + 1] * inv),
                                            W::H::pack(w.o[d][4 * e + 2] * inv, w.o[d][4 * e + 3] * inv)};
  if (a.lse && !w.half) a.lse[token * a.heads + head] = sum == 0.f ? -INFINITY : w.m * kLn2 + logf(sum);
}

}  // namespace

int64_t prefill_blocks(const PrefillArgs& a) {
  return (a.Tq / kQRows + std::min(a.n, a.Tq)) * a.heads;
}

hipError_t launch_attention_prefill(const PrefillArgs& a, hipStream_t stream) {
  const int64_t blocks = prefill_blocks(a), x = std::min<int64_t>(blocks, 1 << 20);
  const dim3 grid((unsigned)x, (unsigned)((blocks + x - 1) / x));
  auto kernel = a.f16 ? (a.D == 64 ? attention_prefill_kernel<true, 64> : a.D == 128 ? attention_prefill_kernel<true, 128>
                                                                                     : attention_prefill_kernel<true, 256>)
                      : (a.D == 64 ? attention_prefill_kernel<false, 64> : a.D == 128 ? attention_prefill_kernel<false, 128>
                                                                                      : attention_prefill_kernel<false, 256>);
  kernel<<<grid, 256, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace moe
