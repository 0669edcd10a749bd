// Attention over whole prompts for gfx950: packed sequences, grouped heads,
//   y_i = sum_j p_ij v_j,   p_ij = exp(s_ij - m_i) / sum_j exp(s_ij - m_i),   s_ij = scale q_i k_j
// over the keys j that query i sees: all of its sequence, or (causal) those up to
// i + lk - lq for lq queries that end where lk keys end.  One pass over the keys with
// the running maximum m and sum l of the softmax in fp32.
//
// A block takes 128 rows, a wave 32 of them: 128 queries of one head, or 64 of two or 32 of
// four heads that share their keys (then the waves see the same keys, and short or ragged
// sequences fill the rows better).  It walks over tiles of keys and values in LDS.  Scores
// are formed transposed, S^T = K Q^T: a lane's results belong to one query, so the softmax
// needs one exchange between the wave's halves, and they stand as the second operand of
// y^T = V^T P^T wants them: the order of the keys inside a product is free, and the
// transposing reads of V follow the order in which the scores lie.  Two blocks share a CU,
// and one's products run beside the other's softmax.  P is rounded to the values' type
// (nearest even) for the matrix cores; each p is off by half a step of itself, as y is by its
// own rounding (in fp16 by 2^-32 of the largest where that is more), and l is summed before
// the rounding.
//
// Where a launch has too few blocks for the card, several share the keys of a tile of
// queries, and a second launch joins what they leave in the workspace.
//
// The matrix cores bound long prompts, and the power that they may draw, which differs from card
// to card: 1 x 16384, 16 heads of 128, causal, takes 1012 to 1071 us (1.03 to 1.09 PFLOP/s; the
// library's largest products 1.35 to 1.39), 8 x 2048 of 16 heads, not causal, 471 to 490 us (0.98
// to 1.02), 1 x 8192, 16 heads of 256, 503 to 526 us (1.05 to 1.09), 1 x 4096, 32 heads of 64, 86
// to 98 us (0.70 to 0.80: the exponentials weigh twice as much, the vector units are busy 60% of
// the cycles and the matrix cores 35%).  In the first the matrix cores are busy 56% of the
// cycles, the vector units 54%, and LDS has no bank conflicts.  Times that stand for two choices
// below were taken in turn on one card.
// Ragged prompts are bound by the longest row's walk over its keys (4099 tokens in 11 sequences
// 52 us), and the smallest by a launch and three trips to memory (61 tokens 6.2 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attention_device.h"
#include "attention_internal.h"

namespace moe {

namespace {

constexpr int kRowBits = 7, kRows = 1 << kRowBits;  // rows (queries times heads) of a block
constexpr int kFill = 512;         // blocks that fill the card, two a CU
constexpr int kMaxSplits = 8;      // blocks that share the keys of a tile of queries
constexpr int kSplitTiles = 8;     // tiles of keys that make a share worth its joining

// Keys of a tile: 64, of the widest heads 32, so that two tiles of keys and values take
// 64 KB of LDS and two blocks share a CU.
constexpr int kTileKeysOf(int D) { return D == 256 ? 32 : 64; }
template <int D>
constexpr int kTileKeys = kTileKeysOf(D);

// Piece p (16 bytes) of row r of a tile is kept at place p ^ f(r) of the row.  Sixteen
// rows read at one piece, and four consecutive rows read at four, spread over all banks.
template <int D>
__device__ __forceinline__ int swizzle(int r) {
  return D == 64 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3) : (r & 3) << 2 | ((r >> 2) & 3);
}

// A number that the compiler no longer knows.  The widest heads leave no registers for the
// sixteen places in a tile that differ in a few address bits: they are made anew each time
// (1021 queries over 8191 keys 148 us, 185 with them kept and others spilled; at 128 and 64
// channels they fit, and keeping them is 1% faster).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

struct PrefillWork {
  int shift;        // 1 << shift query heads to a block: 1, 2 or 4
  int groups;       // blocks that share a tile of queries, one for each such set of heads
  int splits;       // blocks that may share the keys of a tile of queries
  int64_t units;    // tiles of queries, at most
  float* parts;     // [units x groups x splits] records: 128 x D sums, m and l
};

// The unit-th tile of queries: its sequence's first query and key, their numbers, and
// the tile's place, counted from the end (the last queries see the most keys).
struct Place {
  int q0, k0, lq, lk, tile;
  bool found;
};
__device__ __forceinline__ Place find_tile(const PrefillArgs& a, int shift, int64_t unit) {
  const int lane = threadIdx.x & 63;
  Place r{};
  for (int64_t c = 0; c < a.n; c += 64) {
    const int64_t i = c + lane;
    int from = 0, to = 0, k_from = 0, k_to = 0;
    if (i < a.n) {
      from = a.q_starts[i], to = a.q_starts[i + 1];
      k_from = a.k_starts[i], k_to = a.k_starts[i + 1];
      from = (int)min((int64_t)max(from, 0), a.Tq);
      to = (int)min((int64_t)max(to, from), a.Tq);
      k_from = (int)min((int64_t)max(k_from, 0), a.Tk);
      k_to = (int)min((int64_t)max(k_to, k_from), a.Tk);
    }
    const uint32_t upto = wave_scan(((uint32_t)(to - from) + ((kRows - 1) >> shift)) >> (kRowBits - shift));
    const uint64_t past = __ballot(unit < upto);
    if (past) {
      const int l = __builtin_ctzll(past);
      r.q0 = __builtin_amdgcn_readlane(from, l);
      r.lq = __builtin_amdgcn_readlane(to, l) - r.q0;
      r.tile = __builtin_amdgcn_readlane((int)upto, l) - 1 - (int)unit;
      r.k0 = __builtin_amdgcn_readlane(k_from, l);
      r.lk = __builtin_amdgcn_readlane(k_to, l) - r.k0;
      r.found = true;
      return r;
    }
    unit -= (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
  }
  return r;
}

// A block's place: which tile of queries, set of heads and share of the keys.
struct Share {
  Place at;
  int group, split;
  int64_t record;  // of split 0
};
__device__ __forceinline__ Share share_of(const PrefillArgs& a, const PrefillWork& w, int64_t block, int splits) {
  Share s;
  const int64_t rest = quotient(block, w.groups);
  s.group = (int)(block - rest * w.groups);  // neighbours on the card's eight parts take different heads
  // The last shares come first, and the first, which all tiles have, at the end: blocks that
  // have nothing to do stand together.  (Between the others they cost twice the time: blocks go
  // to the card's parts in turn, whatever there is to do.)
  const int from_end = (int)quotient(rest, w.units);
  s.split = splits - 1 - from_end;
  if (s.split < 0) {  // the last row of the grid may reach past the last block
    s.at.found = false;
    return s;
  }
  const int64_t unit = rest - from_end * w.units;
  s.at = find_tile(a, w.shift, unit);
  s.record = (unit * w.groups + s.group) * w.splits;
  return s;
}
// Keys that the queries up to r of the sequence see.
__device__ __forceinline__ int keys_seen(const PrefillArgs& a, const Place& at, int r) {
  return a.causal ? max(min(min(r, at.lq - 1) + at.lk - at.lq + 1, at.lk), 0) : at.lk;
}
// How many blocks share `tiles` tiles of keys.  (Divisions come from the vector unit, and the
// block's loop is to stay scalar.)
__device__ __forceinline__ int shares(const PrefillWork& w, int tiles) {
  return __builtin_amdgcn_readfirstlane(max(1, min(w.splits, tiles / kSplitTiles)));
}

template <bool F16, int D>
struct Prefill {
  using H = Half<F16>;
  static constexpr int BN = kTileKeys<D>, KT = BN / 32, DT = D / 32, KS = D / 16;
  static constexpr int kRow = 2 * D, kTile = BN * kRow;  // bytes of a row and of a tile
  static constexpr int kLoads = kTile / 1024 / 4;        // staging loads of a wave

  u32x4 q[KS];
  f32x16 o[DT], s[KT];
  u32x4 p[KT][2];  // the weights as the second operand wants them
  float m, l;
  int lane, wave, half, lim;  // lim: the last key that the lane's query sees

  // Tile `first` of the keys or values: a wave's load fills 1024 bytes, whole rows.  Rows
  // behind the last key repeat it; they are masked.  FIRST: before the loop, whose places the
  // widest heads would else keep in memory and wait for (1021 queries over 8191 keys 148 us, 153).
  template <bool FIRST = false>
  __device__ __forceinline__ void stage(const uint16_t* base, int64_t stride, int first, int lk, uint8_t* dst) const {
    constexpr int PER = kRow / 16, ROWS = 64 / PER;  // pieces of a row, rows of a load
    const __amdgpu_buffer_rsrc_t src = rows_from(base + first * stride);
    const int last = lk - 1 - first;
    const int lane = FIRST && D == 256 ? opaque(this->lane) : this->lane;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (wave + 4 * i) * ROWS + lane / PER, piece = (lane % PER) ^ swizzle<D>(row);
      copy_to_lds(src, (uint32_t)min(row, last) * (uint32_t)(2 * stride) + 16 * piece, dst + (wave + 4 * i) * 1024);
    }
  }

  __device__ __forceinline__ void load_queries(const uint16_t* from) {
#pragma unroll
    for (int k = 0; k < KS; ++k) q[k] = *(const u32x4*)(from + 16 * k);
  }
  // The queries are waited for here, and not where the compiler would wait for what was
  // asked for after them too.
  __device__ __forceinline__ void hold_queries() {
#pragma unroll
    for (int k = 0; k < KS; ++k) asm volatile("" : "+v"(q[k]));
  }

  // The softmax of the tile whose scores are in s: its weights in p.  masked: some query
  // of the wave does not see all of the tile.
  __device__ __forceinline__ void softmax(int first, float c, bool masked) {
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
    // inside fp32, and y is scaled anew only when a query's maximum really moves (1 x 16384
    // 1012 us, 1061 where it follows at once; 1 x 8192 of 256 channels 506 us, 573).
    if (__any(top > m + (H::kLift + H::kLag))) {
      const float now = fmaxf(m, top - H::kLift), f = now == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - now);
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
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[t][k][e] = H::pack(s[t][8 * k + 2 * e], s[t][8 * k + 2 * e + 1]);
  }

  // y^T += V^T P^T from the values at vs, then S^T = K Q^T from the keys at ks; without VALUES
  // the scores alone.  The operands are read from LDS kAhead products ahead, in an order that
  // the compiler is held to: a wave has one neighbour on its SIMD, which does not hide a read
  // that is waited for where it is used (1 x 16384, 16 heads of 128: 1012 us, 1040 in the
  // compiler's order, 1023 with 8 ahead; 1 x 8192, 16 heads of 256: 503 us, 540).
  template <bool VALUES>
  __device__ __forceinline__ void products(const uint8_t* vs, const uint8_t* ks) {
    constexpr int NV = VALUES ? 2 * KT * DT : 0, N = NV + KS * KT, kAhead = 4;
    const int i16 = lane & 15, g = lane >> 4, krow = lane & 31;
    int vat[2], kat = krow * kRow + ((half ^ swizzle<D>(krow)) << 4);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * r + 4 * half + (i16 >> 2), piece = 2 * (g & 1) + ((i16 & 3) >> 1);
      vat[r] = row * kRow + ((piece ^ swizzle<D>(row)) << 4) + 8 * (i16 & 1);
    }
    if (D == 256) vat[0] = opaque(vat[0]), vat[1] = opaque(vat[1]), kat = opaque(kat);
    u32x4 f[kAhead];
    auto read = [&](int j) {
      if (j >= N) return;
      if (j < NV) {
        const uint8_t* at = vs + 16 * (j / DT) * kRow;
        const int d = j % DT;
        const u32x2 lo = read_transposed(at + (vat[0] ^ (d << 6))), hi = read_transposed(at + (vat[1] ^ (d << 6)));
        f[j % kAhead] = u32x4{lo.x, lo.y, hi.x, hi.y};
      } else {
        const int k = (j - NV) / KT, t = (j - NV) % KT;
        f[j % kAhead] = *(const u32x4*)(ks + 32 * t * kRow + (kat ^ (k << 5)));
      }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) read(j);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      __builtin_amdgcn_sched_barrier(0);
      if (j < NV) {
        o[j % DT] = H::mfma32(f[j % kAhead], p[j / DT / 2][j / DT % 2], o[j % DT]);
      } else {
        const int k = (j - NV) / KT, t = (j - NV) % KT;
        if (k == 0) s[t] = f32x16{};
        s[t] = H::mfma32(f[j % kAhead], q[k], s[t]);
      }
      read(j + kAhead);
    }
    __builtin_amdgcn_sched_barrier(0);
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

  // The row's y from its sums, rounded once, and the logarithm of its sum.
  __device__ __forceinline__ void store(const PrefillArgs& a, int64_t token, int head, float sum) const {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* y = a.y + (token * a.heads + head) * D + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(u32x2*)(y + 32 * d + 8 * e) = u32x2{H::pack(o[d][4 * e] * inv, o[d][4 * e + 1] * inv),
                                              H::pack(o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv)};
    if (a.lse && !half) a.lse[token * a.heads + head] = H::log_of_sum(m, sum);
  }
};

__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// All loads have arrived but the last N.
template <int N = 0>
__device__ __forceinline__ void arrived() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <bool F16, int D>
__global__ __launch_bounds__(256, 2) void attention_prefill_kernel(PrefillArgs a, PrefillWork work) {
  using W = Prefill<F16, D>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * W::kTile];
  __shared__ int redo;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const Share share = share_of(a, work, block, work.splits);
  const Place& at = share.at;
  if (!at.found) return;
  W w;
  w.lane = threadIdx.x & 63;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  w.half = w.lane >> 5;
  const int queries = kRows >> work.shift, first_query = at.tile * queries;
  const int head = (share.group << work.shift) + (w.wave & ((1 << work.shift) - 1));
  const int first_row = first_query + 32 * (w.wave >> work.shift);
  const int row = first_row + (w.lane & 31);
  w.lim = a.causal ? min(row + at.lk - at.lq, at.lk - 1) : at.lk - 1;
  const int64_t token = at.q0 + min(row, at.lq - 1);
  const uint16_t* qp = a.q.p + token * a.q.token + head * a.q.head + 8 * w.half;
  // The widest heads' queries are asked for behind the first keys and waited for with them:
  // they have no registers to wait in (1 x 8192 506 us, 532 with the queries first; of 64 and 128
  // channels these go first, 1 x 4096 86 us and 91, 1 x 2048 54 and 60).
  constexpr bool kQueriesFirst = D < 256;
  if (kQueriesFirst) w.load_queries(qp);
  const int kv = head / (a.heads / a.kv_heads);
  const uint16_t* kp = a.k.p + at.k0 * a.k.token + kv * a.k.head;
  const uint16_t* vp = a.v.p + at.k0 * a.v.token + kv * a.v.head;
  // the block's tiles of keys; the keys that all its queries see, and that the wave's do
  const int tiles = (keys_seen(a, at, first_query + queries - 1) + W::BN - 1) / W::BN, n = shares(work, tiles);
  if (share.split >= n) return;
  const int each = __builtin_amdgcn_readfirstlane((uint32_t)tiles / (uint32_t)n), extra = tiles - each * n;
  const int from = each * share.split + min(share.split, extra), to = from + each + (share.split < extra);
  const int seen_by_all = a.causal ? keys_seen(a, at, first_query) : at.lk;
  const int wave_end = first_row < at.lq ? keys_seen(a, at, first_row + 31) : 0;
  const int all_end = a.causal ? keys_seen(a, at, first_row) : at.lk;
  const float c = a.scale * kLog2e;
  uint8_t* const kbuf = lds;
  uint8_t* const vbuf = lds + 2 * W::kTile;
  for (int careful = 0;; ++careful) {
    w.m = -INFINITY;
    w.l = 0.f;
#pragma unroll
    for (int d = 0; d < W::DT; ++d) w.o[d] = f32x16{};
    // Tile t's keys and values are in buffer t - from modulo 2.
    auto stage_next = [&](int t) {
      const int now = (t - from) & 1;
      if (t + 1 < to) w.stage(vp, a.v.token, (t + 1) * W::BN, at.lk, vbuf + (now ^ 1) * W::kTile);
      if (t + 2 < to) w.stage(kp, a.k.token, (t + 2) * W::BN, at.lk, kbuf + now * W::kTile);
    };
    if (from < to) {
      w.template stage<true>(kp, a.k.token, from * W::BN, at.lk, kbuf);
      if (!kQueriesFirst) {
        __builtin_amdgcn_sched_barrier(0);
        w.load_queries(qp);
        __builtin_amdgcn_sched_barrier(0);
      }
      w.template stage<true>(vp, a.v.token, from * W::BN, at.lk, vbuf);
      if (from + 1 < to) {
        w.template stage<true>(kp, a.k.token, (from + 1) * W::BN, at.lk, kbuf + W::kTile);
        arrived<2 * W::kLoads>();
        if (!kQueriesFirst) w.hold_queries();
      } else {
        arrived<W::kLoads>();
        if (!kQueriesFirst) w.hold_queries();
      }
      meet();
      if (from * W::BN < wave_end) w.template products<false>(nullptr, kbuf);
    }
    for (int t = from; t < to; ++t) {
      const int now = (t - from) & 1, first = t * W::BN;
      uint8_t* const vs = vbuf + now * W::kTile;
      if (first < wave_end) w.softmax(first, c, first + W::BN > all_end);
      arrived();
      meet();
      stage_next(t);
      const bool cleared = careful && first + W::BN > seen_by_all;
      if (cleared) {
        w.clear(vs);
        meet();
      }
      if (first < wave_end) {
        // Scores that no tile follows for are formed all the same and not looked at.
        w.template products<true>(vs, kbuf + (now ^ 1) * W::kTile);
        if (cleared) w.add_cleared(vp, a.v.token, first, min(first + W::BN, at.lk));
      }
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
  if (n > 1) {
    float* part = work.parts + (share.record + share.split) * (kRows * (D + 2));
    float* ml = part + kRows * D + 64 * w.wave;
    part += w.wave * (32 * D);
#pragma unroll
    for (int d = 0; d < W::DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(f32x4*)(part + 4 * (64 * (4 * d + e) + w.lane)) =
            f32x4{w.o[d][4 * e], w.o[d][4 * e + 1], w.o[d][4 * e + 2], w.o[d][4 * e + 3]};
    ml[w.lane] = w.half ? sum : w.m;
    return;
  }
  if (row < at.lq) w.store(a, token, head, sum);
}

// Rows whose keys several blocks shared: 32 of them and 64 channels a wave.
template <bool F16, int D>
__global__ __launch_bounds__(64) void attention_prefill_join_kernel(PrefillArgs a, PrefillWork work) {
  using W = Prefill<F16, D>;
  constexpr int PARTS = 4 * (D / 64), RECORD = kRows * (D + 2);
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int part = (int)(block % PARTS), wave = part % 4, d0 = 2 * (part / 4);
  const Share share = share_of(a, work, block / PARTS, 1);
  const Place& at = share.at;
  if (!at.found) return;
  const int lane = threadIdx.x, half = lane >> 5;
  const int queries = kRows >> work.shift, first_query = at.tile * queries;
  const int tiles = (keys_seen(a, at, first_query + queries - 1) + W::BN - 1) / W::BN, n = shares(work, tiles);
  if (n == 1) return;
  const int row = first_query + 32 * (wave >> work.shift) + (lane & 31);
  const float* base = work.parts + share.record * RECORD;
  const float* ml = base + kRows * D + 64 * wave + (lane & 31);
  float m[kMaxSplits], l[kMaxSplits], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) {
    m[i] = i < n ? ml[(int64_t)i * RECORD] : -INFINITY;
    l[i] = i < n ? ml[(int64_t)i * RECORD + 32] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) top = fmaxf(top, m[i]);
  f32x4 o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = f32x4{};
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) {
    if (i >= n) break;
    const float f = m[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[i] - top);
    sum += l[i] == 0.f ? 0.f : l[i] * f;
    const f32x4* r = (const f32x4*)(base + (int64_t)i * RECORD + wave * (32 * D)) + 256 * d0 + lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] += r[64 * e] * f;
  }
  if (row >= at.lq) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t out = (at.q0 + row) * (int64_t)a.heads + (share.group << work.shift) + (wave & ((1 << work.shift) - 1));
  uint16_t* y = a.y + out * D + 32 * d0 + 4 * half;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *(u32x2*)(y + 8 * e) = u32x2{W::H::pack(o[e].x * inv, o[e].y * inv), W::H::pack(o[e].z * inv, o[e].w * inv)};
  if (a.lse && part < 4 && !half) a.lse[out] = W::H::log_of_sum(top, sum);
}

PrefillWork work_of(const PrefillArgs& a) {
  PrefillWork w{};
  const int shared = a.heads / a.kv_heads;
  // As many heads to a block as share keys and divide it: fewer rows stay empty, and the waves
  // walk over the same keys (4099 tokens in 11 sequences 52 us, 58 with a head a block; 1 x 1000
  // 27.6 and 29.0).
  w.shift = shared % 4 == 0 ? 2 : shared % 2 == 0 ? 1 : 0;
  w.groups = a.heads >> w.shift;
  w.units = (a.Tq >> (kRowBits - w.shift)) + std::min(a.n, a.Tq);
  // Where there are fewer blocks than fill the card, several share the keys of one, if there
  // are enough of these (1021 queries over 8191 keys, 16 heads of 256: 148 us, 363 without;
  // shares of four tiles instead of eight: 1 x 1000, 32 us, 28 with eight).  The number is the
  // nearest, which starts up to a third more blocks than two a CU: rounded down it is slower
  // where a CU holds three (64 channels, 1100 queries over 8100 keys, 32 heads: 131 us, 111 so)
  // and faster where it holds two (128 channels, 700 over 8192: 121 us, 143 so; 1100 over 8192:
  // 185 and 196).
  // Not to even out ragged sequences: blocks that turn out to have nothing to do, and the
  // joining, cost more than that gains (1809 of 4099 tokens in one of 11 sequences: 67 us, 52
  // without).
  const int64_t blocks = w.units * w.groups, tiles = a.Tk / (kTileKeysOf(a.D) * kSplitTiles);
  w.splits = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, (kFill + blocks / 2) / blocks, tiles}));
  return w;
}

}  // namespace

int64_t prefill_blocks(const PrefillArgs& a) {
  const PrefillWork w = work_of(a);
  return w.units * w.groups * w.splits;
}

int64_t prefill_workspace_bytes(const PrefillArgs& a) {
  const PrefillWork w = work_of(a);
  return w.splits > 1 ? w.units * w.groups * w.splits * kRows * (a.D + 2) * 4 : 0;
}

hipError_t launch_attention_prefill(const PrefillArgs& a, void* ws, hipStream_t stream) {
  PrefillWork w = work_of(a);
  w.parts = (float*)ws;
  auto grid = [](int64_t blocks) {
    const int64_t x = std::min<int64_t>(blocks, 1 << 20);
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
  };
  auto by_dim = [&](auto f16, auto dim) {
    constexpr bool F = decltype(f16)::value;
    constexpr int D = decltype(dim)::value;
    attention_prefill_kernel<F, D><<<grid(w.units * w.groups * w.splits), 256, 0, stream>>>(a, w);
    if (w.splits > 1) attention_prefill_join_kernel<F, D><<<grid(w.units * w.groups * 4 * (D / 64)), 64, 0, stream>>>(a, w);
  };
  auto by_type = [&](auto f16) {
    if (a.D == 64) by_dim(f16, std::integral_constant<int, 64>{});
    else if (a.D == 128) by_dim(f16, std::integral_constant<int, 128>{});
    else by_dim(f16, std::integral_constant<int, 256>{});
  };
  if (a.f16) by_type(std::true_type{});
  else by_type(std::false_type{});
  return hipGetLastError();
}

}  // namespace moe
