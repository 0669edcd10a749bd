// The key-value cache for gfx950: new keys and values into its pages, and the pages'
// own bookkeeping.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attention_device.h"
#include "attention_internal.h"
#include "fp8_device.h"

namespace moe {

namespace {

// ------------------------------------------------------------------ append
// Of a rotated head, channels i and i + R / 2 (or 2 i and 2 i + 1) are one pair, turned by
// the angle position * inv_freq[i]:
//   (a, b) -> (a cos - b sin, b cos + a sin).
// The angle is formed and reduced to a fraction of a turn in fp64 (far positions keep
// their bits), its sine and cosine in fp32, once a token and for all its heads.
// A block has one token, or where there are few tokens a part of its heads.  A lane has two
// pieces of 16 bytes of a head row, a pair that is turned together where there is one, and a
// row's lanes are neighbours, so a row's largest magnitude, for e4m3, is a reduction among
// these; a row is read whole before any of it is written, so q and k may be written in place.
// The first rows are asked for before the angles and the page are known.
// HBM bounds long calls: 16381 tokens of 32 + 2 x 8 heads of 128, half of them turned, 84 us
// (5.2 TB/s; 92 us with two rows in a lane's hand, 105 with four); a step of 64 tokens into
// e4m3 is a launch, a trip to memory and the sines: 4.3 us.
constexpr int kAppendThreads = 256;

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int s = 1; s < LANES; s <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, s, 64));
  return v;
}

template <bool F16, bool F8, int D>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a, int blocks) {
  using H = Half<F16>;
  constexpr int PER = D / 8, LANES = PER / 2, ROWS = kAppendThreads / LANES;
  __shared__ __attribute__((aligned(16))) float turn[2][D / 2];
  const int64_t unit = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, t = unit / blocks;
  const int part = (int)(unit - t * blocks);
  if (t >= a.T) return;
  const int row = a.rows[t], position = a.positions[t];
  const int nq = a.q.p ? a.heads : 0, kvh = a.c.kv_heads, rows = nq + 2 * kvh;
  const int lane = threadIdx.x % LANES, half = a.rotary / 2;
  // The lane's two pieces: a pair that is turned together, or two that stay (interleaved
  // pairs lie in one piece).
  const int pairs = a.rotary / 16;
  const bool turned = lane < pairs;
  const int piece = turned ? lane : pairs + lane, other = turned ? lane + pairs : piece + LANES - pairs;

  u32x4 own[2];
  auto load = [&](int r) {
    const bool is_q = r < nq, is_k = !is_q && r < nq + kvh;
    const HeadRows& from = is_q ? a.q : is_k ? a.k : a.v;
    const uint16_t* x = from.p + t * from.token + (is_q ? r : is_k ? r - nq : r - nq - kvh) * from.head;
    own[0] = *(const u32x4*)(x + 8 * piece);
    own[1] = *(const u32x4*)(x + 8 * other);
  };
  int r = part * ROWS + threadIdx.x / LANES;
  if (row >= 0 && r < rows) load(r);

  int64_t page = -1;
  if (row >= 0 && row < a.c.rows && position >= 0 && (position >> a.c.shift) < a.c.width) {
    page = a.c.tables[row * (int64_t)a.c.width + (position >> a.c.shift)];
    if (page >= a.c.n_pages) page = -1;
  }
  const bool wrong = page < 0;
  if (threadIdx.x < half) {
    const double turns = (double)position * (double)a.inv_freq[threadIdx.x] * 0.15915494309189533577;
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    turn[0][threadIdx.x] = c;
    turn[1][threadIdx.x] = s;
  }
  __syncthreads();
  if (row < 0) return;  // padding: everything stays as it was
  while (r < rows) {
    const bool is_q = r < nq, is_k = !is_q && r < nq + kvh;
    const HeadRows& to = is_q ? a.q_out : a.k_out;
    const int h = is_q ? r : is_k ? r - nq : r - nq - kvh;
    float f[2][8];
    const bool turn_it = (is_q || is_k) && turned;
    u32x4 bits[2] = {own[0], own[1]};
    if (turn_it || F8) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = H::widen(own[i][e / 2] >> (16 * (e & 1)));
    }
    if (turn_it) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = 4 * (i ? other : piece);
          const f32x4 c = *(const f32x4*)(turn[0] + at), s = *(const f32x4*)(turn[1] + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = f[i][2 * e], hi = f[i][2 * e + 1];
            f[i][2 * e] = lo * c[e] - hi * s[e];
            f[i][2 * e + 1] = hi * c[e] + lo * s[e];
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const f32x4 c = *(const f32x4*)(turn[0] + 8 * piece + 4 * x), s = *(const f32x4*)(turn[1] + 8 * piece + 4 * x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = f[0][4 * x + e], hi = f[1][4 * x + e];
            f[0][4 * x + e] = lo * c[e] - hi * s[e];
            f[1][4 * x + e] = hi * c[e] + lo * s[e];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        bits[i] = u32x4{H::pack(f[i][0], f[i][1]), H::pack(f[i][2], f[i][3]), H::pack(f[i][4], f[i][5]), H::pack(f[i][6], f[i][7])};
    }
    if ((is_q || is_k) && to.p) {
      uint16_t* y = (uint16_t*)to.p + t * to.token + h * to.head;
      const uint32_t nan = 0x7FFF7FFFu;  // a NaN of either kind
      *(u32x4*)(y + 8 * piece) = wrong ? u32x4{nan, nan, nan, nan} : bits[0];
      *(u32x4*)(y + 8 * other) = wrong ? u32x4{nan, nan, nan, nan} : bits[1];
    }
    if (!is_q && !wrong) {
      const int64_t slot = (page * kvh + h) * a.c.P + (position & (a.c.P - 1));
      void* cache = (void*)(is_k ? a.c.k : a.c.v);
      if (F8) {
        const float m = floor_amax(lanes_max<LANES>(max(amax8(f[0]), amax8(f[1]))));
        ((u32x2*)cache)[slot * PER + piece] = codes8(f[0], kE4m3Max / m);
        ((u32x2*)cache)[slot * PER + other] = codes8(f[1], kE4m3Max / m);
        if (lane == 0) ((float*)(is_k ? a.c.k_scales : a.c.v_scales))[slot] = m / kE4m3Max;
      } else {
        ((u32x4*)cache)[slot * PER + piece] = bits[0];
        ((u32x4*)cache)[slot * PER + other] = bits[1];
      }
    }
    r += ROWS * blocks;
    if (r < rows) load(r);
  }
}

// ------------------------------------------------------------------ pages
// The free pages are those with no references.  A call that needs pages takes the lowest
// free ones, for the rows in rising order, so its result does not depend on how blocks
// and waves run.  One block makes the plan (what every row needs, running sums, the list
// of free pages); a second launch carries it out, rows and copies side by side.  The plan is a
// chain of a few trips to memory (5.5 us for 64 forks), the copies are bound by
// HBM (64 forks that copy 117 MB 24 us, with the pages in the Infinity Cache; 321 MB compacted
// 127 us, 5.0 TB/s).
constexpr int kPlanThreads = 1024, kPlanPer = 4;
enum Kind { kReserve, kFork };

// Sums of v over the threads before this one, this one included; all: over every thread.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int64_t other = __shfl_up(v, s, 64);
    if (lane >= s) v += other;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 64; ++i) {
    if (i < wave) v += sums[i];
    all += sums[i];
  }
  return v;
}

struct Plan {
  int64_t* count;   // [0]: pages given out or moved
  int64_t* upto;    // [rows]: pages needed by the rows up to this one
  int32_t *from, *to;  // [n_pages]: moves; to alone: the pages given out, in order
  int32_t* moved;   // [n_pages]: where a page goes (compact)
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) {
  return (tokens + ((int64_t)1 << shift) - 1) >> shift;
}
// Pages that a row holds: never more than its table has entries.
__device__ __forceinline__ int64_t held_by(const TableArgs& t, int64_t r) {
  return min(pages_of(max(t.lengths[r], 0), t.shift), (int64_t)t.width);
}
__device__ __forceinline__ bool is_page(const TableArgs& t, int p) { return p >= 0 && p < t.n_pages; }

// Whether row r asks for something that can be done, and how many pages it needs.
template <Kind KIND>
__device__ __forceinline__ bool wants(const TableArgs& t, const int32_t* ask, int64_t r, int64_t& need) {
  need = 0;
  const int v = ask[r];
  if (KIND == kReserve) {
    if (v < 0) return false;
    const int64_t len = max(t.lengths[r], 0), after = pages_of(len + v, t.shift);
    if (len + v > 0x7FFFFFFF || after > t.width) return false;
    need = after - pages_of(len, t.shift);
    return true;
  }
  if (v < 0 || v >= t.rows || t.lengths[r] > 0 || ask[v] >= 0) return false;
  const int64_t len = max(t.lengths[v], 0);
  if (pages_of(len, t.shift) > t.width) return false;
  need = (len & (t.P - 1)) != 0;
  return true;
}

// The first `needed` free pages into p.to; how many there are.
__device__ __forceinline__ int64_t list_free(const TableArgs& t, const Plan& p, int64_t needed, int64_t* sums) {
  int64_t found = 0, all;
  for (int64_t p0 = 0; p0 < t.n_pages && found < needed; p0 += kPlanThreads * kPlanPer) {
    const int64_t at = p0 + threadIdx.x * kPlanPer;
    int free = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) free |= (at + i < t.n_pages && t.refs[at + i] == 0) << i;
    int64_t k = found + block_scan(__builtin_popcount(free), sums, all) - __builtin_popcount(free);
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i)
      if (free >> i & 1) {
        if (k < needed) p.to[k] = (int)(at + i);
        ++k;
      }
    found += all;
  }
  return min(found, needed);
}

template <Kind KIND>
__global__ __launch_bounds__(kPlanThreads) void pages_plan_kernel(TableArgs t, const int32_t* ask, Plan p) {
  __shared__ int64_t sums[kPlanThreads / 64];
  int64_t needed = 0, all;
  for (int64_t r0 = 0; r0 < t.rows; r0 += kPlanThreads) {
    const int64_t r = r0 + threadIdx.x;
    int64_t need = 0;
    if (r < t.rows) wants<KIND>(t, ask, r, need);
    const int64_t upto = needed + block_scan(need, sums, all);
    if (r < t.rows) p.upto[r] = upto;
    needed += all;
  }
  const int64_t found = list_free(t, p, needed, sums);
  if (threadIdx.x == 0) *p.count = found;
  if (KIND == kFork) {
    for (int64_t r = threadIdx.x; r < t.rows; r += kPlanThreads) {
      int64_t need;
      if (!wants<KIND>(t, ask, r, need) || !need || p.upto[r] > found) continue;
      const int len = t.lengths[ask[r]];
      const int src = t.tables[(int64_t)ask[r] * t.width + (len >> t.shift)];
      p.from[p.upto[r] - 1] = is_page(t, src) ? src : -1;
    }
  }
}

// Row r as planned, by one wave.
template <Kind KIND>
__device__ __forceinline__ void carry_out(const TableArgs& t, const int32_t* ask, const Plan& p, int32_t* status,
                                          int64_t r) {
  const int lane = threadIdx.x & 63;
  int64_t need;
  const bool ok = wants<KIND>(t, ask, r, need);
  const bool served = ok && (!need || p.upto[r] <= *p.count);
  if (lane == 0) status[r] = served ? (int)need : ok ? -2 : KIND == kFork && ask[r] < 0 ? 0 : -1;
  if (!served) return;
  int32_t* row = t.tables + r * t.width;
  const int32_t* given = p.to + p.upto[r] - need;
  if (KIND == kReserve) {
    const int len = max(t.lengths[r], 0);
    const int64_t have = pages_of(len, t.shift);
    for (int64_t i = lane; i < need; i += 64) {
      row[have + i] = given[i];
      t.refs[given[i]] = 1;
    }
    __builtin_amdgcn_wave_barrier();
    if (lane == 0) t.lengths[r] = len + ask[r];
    return;
  }
  const int len = max(t.lengths[ask[r]], 0);
  const int32_t* parent = t.tables + (int64_t)ask[r] * t.width;
  const int64_t n = pages_of(len, t.shift);
  for (int64_t i = lane; i < n; i += 64) {
    const int page = need && i == n - 1 ? given[0] : parent[i];
    row[i] = page;
    if (is_page(t, page)) atomicAdd(t.refs + page, 1);
  }
  if (lane == 0) t.lengths[r] = len;
}

constexpr int64_t kCopyStep = 16 * 256 * 4;  // bytes of a block's step
constexpr int64_t kCopyBlocks = 16384;
// One plane's share of the moves: block x of `blocks`, 16 bytes a lane where pages allow.
__device__ __forceinline__ void copy_pages(const PoolArgs& pools, const int32_t* from, const int32_t* to, int64_t n,
                                           int64_t x, int64_t blocks, int64_t plane) {
  int which = 0;
  while (which < pools.n && plane >= pools.pool[which].planes) plane -= pools.pool[which++].planes;
  if (which >= pools.n) return;
  const int64_t bytes = pools.pool[which].page_bytes;
  char* base = pools.pool[which].base + plane * pools.n_pages * bytes;
  const bool wide = bytes % 16 == 0 && (uintptr_t)base % 16 == 0;
  constexpr int64_t CHUNK = kCopyStep;
  const int64_t chunks = (bytes + CHUNK - 1) / CHUNK;
  for (int64_t item = x; item < n * chunks; item += blocks) {
    const int64_t k = item / chunks, c = (item - k * chunks) * CHUNK;
    const int64_t src = from[k], dst = to[k];
    if (src < 0 || src >= pools.n_pages || dst < 0 || dst >= pools.n_pages || src == dst) continue;
    const char* s = base + src * bytes;
    char* d = base + dst * bytes;
    if (wide) {
      u32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = c + 16 * (int64_t)(threadIdx.x + 256 * i);
        if (at < bytes) v[i] = *(const u32x4*)(s + at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = c + 16 * (int64_t)(threadIdx.x + 256 * i);
        if (at < bytes) *(u32x4*)(d + at) = v[i];
      }
    } else {
      for (int64_t at = c + 4 * threadIdx.x; at < min(c + CHUNK, bytes); at += 4 * 256)
        *(uint32_t*)(d + at) = *(const uint32_t*)(s + at);
    }
  }
}

// The same in one launch, for up to a row a thread: each thread writes its row's new pages,
// or the wave does where a row gets many (a fork, a reserve and a free of 64 rows 39.5 us, 42.5
// with two launches for the reserve).
__global__ __launch_bounds__(kPlanThreads) void reserve_few_kernel(TableArgs t, const int32_t* grow, int32_t* status,
                                                                   Plan p) {
  __shared__ int64_t sums[kPlanThreads / 64];
  const int64_t r = threadIdx.x;
  const bool mine = r < t.rows;
  int64_t need = 0, needed, found;
  const bool ok = mine && wants<kReserve>(t, grow, r, need);
  const int len = ok ? max(t.lengths[r], 0) : 0;
  const int64_t upto = block_scan(need, sums, needed);
  found = list_free(t, p, needed, sums);
  __syncthreads();
  const bool served = ok && (!need || upto <= found);
  const int64_t have = pages_of(len, t.shift);
  if (mine) status[r] = served ? (int)need : ok ? -2 : -1;
  if (served) t.lengths[r] = len + grow[r];
  constexpr int FEW = 4;
  if (served && need <= FEW) {
    for (int64_t i = 0; i < need; ++i) {
      const int page = p.to[upto - need + i];
      t.tables[r * t.width + have + i] = page;
      t.refs[page] = 1;
    }
  }
  for (uint64_t many = __ballot(served && need > FEW); many; many &= many - 1) {
    const int l = __builtin_ctzll(many);
    const int64_t n = __shfl(need, l, 64), from = __shfl(upto, l, 64) - n;
    const int64_t to = __shfl(r, l, 64) * t.width + __shfl(have, l, 64);
    for (int64_t i = threadIdx.x & 63; i < n; i += 64) {
      const int page = p.to[from + i];
      t.tables[to + i] = page;
      t.refs[page] = 1;
    }
  }
}

// Rows as planned by the first blocks, four a block; copies by the others.
template <Kind KIND>
__global__ __launch_bounds__(256) void pages_do_kernel(TableArgs t, const int32_t* ask, Plan p, int32_t* status,
                                                       PoolArgs pools, int64_t row_blocks, int64_t per_plane) {
  const int64_t block = blockIdx.x;
  if (block < row_blocks) {
    const int64_t r = block * 4 + (threadIdx.x >> 6);
    if (r < t.rows) carry_out<KIND>(t, ask, p, status, r);
    return;
  }
  const int64_t x = block - row_blocks;
  copy_pages(pools, p.from, p.to, *p.count, x % per_plane, per_plane, x / per_plane);
}

__global__ __launch_bounds__(256) void kv_free_kernel(TableArgs t, const int32_t* drop) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= t.rows || !drop[r]) return;
  const int64_t n = held_by(t, r);
  for (int64_t i = threadIdx.x & 63; i < n; i += 64) {
    const int page = t.tables[r * t.width + i];
    if (is_page(t, page)) atomicSub(t.refs + page, 1);
  }
  __builtin_amdgcn_wave_barrier();
  if ((threadIdx.x & 63) == 0) t.lengths[r] = 0;
}

// Pages in use: n of them.  Those from n on move to the free ones below n, both in rising
// order, so the copies neither meet nor depend on each other.
__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(TableArgs t, Plan p, int32_t* new_refs, int32_t* live) {
  __shared__ int64_t sums[kPlanThreads / 64];
  int64_t used = 0, all;
  {
    int64_t mine = 0;
    for (int64_t at = threadIdx.x; at < t.n_pages; at += kPlanThreads) mine += t.refs[at] > 0;
    block_scan(mine, sums, used);
  }
  int64_t holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < t.n_pages; p0 += kPlanThreads * kPlanPer) {
    const int64_t at = p0 + threadIdx.x * kPlanPer;
    int hole = 0, mover = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i)
      if (at + i < t.n_pages) {
        const bool in_use = t.refs[at + i] > 0;
        hole += !in_use && at + i < used;
        mover += in_use && at + i >= used;
      }
    const int64_t both = block_scan((int64_t)hole << 32 | mover, sums, all) - ((int64_t)hole << 32 | mover);
    int64_t h = holes + (both >> 32), m = movers + (both & 0xFFFFFFFF);
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i)
      if (at + i < t.n_pages) {
        const bool in_use = t.refs[at + i] > 0;
        if (!in_use && at + i < used) p.to[h++] = (int)(at + i);
        if (in_use && at + i >= used) p.from[m++] = (int)(at + i);
        p.moved[at + i] = (int)(at + i);
      }
    holes += all >> 32;
    movers += all & 0xFFFFFFFF;
  }
  if (new_refs != t.refs)
    for (int64_t at = threadIdx.x; at < t.n_pages; at += kPlanThreads) new_refs[at] = t.refs[at];
  __syncthreads();
  for (int64_t k = threadIdx.x; k < movers; k += kPlanThreads) {
    const int src = p.from[k], dst = p.to[k];
    p.moved[src] = dst;
    new_refs[dst] = t.refs[src];
    new_refs[src] = 0;
  }
  if (threadIdx.x == 0) {
    *p.count = movers;
    *live = (int)used;
  }
}

__global__ __launch_bounds__(256) void compact_do_kernel(TableArgs t, Plan p, int32_t* new_tables, PoolArgs pools,
                                                         int64_t row_blocks, int64_t per_plane) {
  const int64_t block = blockIdx.x;
  if (block < row_blocks) {
    const int64_t r = block * 4 + (threadIdx.x >> 6);
    if (r >= t.rows) return;
    const int64_t n = held_by(t, r);
    for (int64_t i = threadIdx.x & 63; i < t.width; i += 64) {
      const int page = t.tables[r * t.width + i];
      new_tables[r * t.width + i] = i < n && is_page(t, page) ? p.moved[page] : page;
    }
    return;
  }
  const int64_t x = block - row_blocks;
  copy_pages(pools, p.from, p.to, *p.count, x % per_plane, per_plane, x / per_plane);
}

__global__ __launch_bounds__(256) void copy_pages_kernel(PoolArgs pools, const int32_t* from, const int32_t* to, int64_t n,
                                                         int64_t per_plane) {
  copy_pages(pools, from, to, n, blockIdx.x % per_plane, per_plane, blockIdx.x / per_plane);
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

Plan plan_in(void* ws, int64_t rows, int64_t n_pages) {
  char* at = (char*)ws;
  Plan p{};
  p.count = (int64_t*)at;
  at += 256;
  p.upto = (int64_t*)at;
  at += up256(8 * rows);
  p.from = (int32_t*)at;
  at += up256(4 * n_pages);
  p.to = (int32_t*)at;
  at += up256(4 * n_pages);
  p.moved = (int32_t*)at;
  return p;
}

int64_t planes_of(const PoolArgs& p) {
  int64_t n = 0;
  for (int i = 0; i < p.n; ++i) n += p.pool[i].planes;
  return n;
}
// Blocks that copy one plane's share of at most `moves` pages: a block for every two steps, up to
// enough over all planes to fill the card many times over (compacting 321 MB 132 us, 135 with
// 4096 blocks; 64 forks, a reserve and a free 39.5 us, 42 with 16384).
int64_t blocks_of_plane(const PoolArgs& p, int64_t moves) {
  const int64_t planes = planes_of(p);
  if (!planes) return 1;
  int64_t bytes = 0;
  for (int i = 0; i < p.n; ++i) bytes = std::max(bytes, p.pool[i].page_bytes);
  const int64_t steps = moves * ((bytes + kCopyStep - 1) / kCopyStep);
  return std::max<int64_t>(1, std::min<int64_t>((steps + 1) / 2, kCopyBlocks / planes));
}

}  // namespace

// (No rows take the space of one, which may stand in for them.)
int64_t pages_workspace_bytes(int64_t rows, int64_t n_pages) {
  return 256 + up256(8 * std::max<int64_t>(rows, 1)) + 3 * up256(4 * n_pages);
}

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream) {
  constexpr int PIECES = 2 * kAppendThreads;
  // 256 tokens fill the card with a block each; of fewer, a block a pass over the token's rows
  // (64 tokens of 32 + 2 x 8 heads of 128 into e4m3: 4.3 us, 5.3 with a block a token)
  const int pieces = ((a.q.p ? a.heads : 0) + 2 * a.c.kv_heads) * (a.c.D / 8);
  const int blocks = a.T < 256 ? std::max(1, std::min((pieces + PIECES - 1) / PIECES, 64)) : 1;
  const int64_t units = a.T * blocks, x = std::min<int64_t>(units, 1 << 20);
  const dim3 grid((unsigned)x, (unsigned)((units + x - 1) / x));
  auto by_dim = [&](auto f16, auto e4m3) {
    constexpr bool F = decltype(f16)::value, E = decltype(e4m3)::value;
    auto kernel = a.c.D == 64 ? kv_append_kernel<F, E, 64> : a.c.D == 128 ? kv_append_kernel<F, E, 128>
                                                                          : kv_append_kernel<F, E, 256>;
    kernel<<<grid, kAppendThreads, 0, stream>>>(a, blocks);
  };
  const bool f8 = a.c.k_scales != nullptr;
  if (a.f16) f8 ? by_dim(std::true_type{}, std::true_type{}) : by_dim(std::true_type{}, std::false_type{});
  else f8 ? by_dim(std::false_type{}, std::true_type{}) : by_dim(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const TableArgs& t, const int32_t* grow, int32_t* status, void* ws, hipStream_t stream) {
  const Plan p = plan_in(ws, t.rows, t.n_pages);
  if (t.rows <= kPlanThreads) {
    reserve_few_kernel<<<1, kPlanThreads, 0, stream>>>(t, grow, status, p);
    return hipGetLastError();
  }
  pages_plan_kernel<kReserve><<<1, kPlanThreads, 0, stream>>>(t, grow, p);
  const int64_t row_blocks = (t.rows + 3) / 4;
  pages_do_kernel<kReserve><<<(unsigned)row_blocks, 256, 0, stream>>>(t, grow, p, status, PoolArgs{}, row_blocks, 1);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const TableArgs& t, const int32_t* parents, const PoolArgs& pools, int32_t* status, void* ws,
                          hipStream_t stream) {
  const Plan p = plan_in(ws, t.rows, t.n_pages);
  pages_plan_kernel<kFork><<<1, kPlanThreads, 0, stream>>>(t, parents, p);
  const int64_t row_blocks = (t.rows + 3) / 4, planes = planes_of(pools), per = blocks_of_plane(pools, t.rows);
  pages_do_kernel<kFork><<<(unsigned)(row_blocks + planes * per), 256, 0, stream>>>(t, parents, p, status, pools, row_blocks,
                                                                                    per);
  return hipGetLastError();
}

hipError_t launch_kv_free(const TableArgs& t, const int32_t* drop, hipStream_t stream) {
  kv_free_kernel<<<(unsigned)((t.rows + 3) / 4), 256, 0, stream>>>(t, drop);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const TableArgs& t, const PoolArgs& pools, int32_t* new_tables, int32_t* new_refs,
                             int32_t* live, void* ws, hipStream_t stream) {
  const Plan p = plan_in(ws, t.rows, t.n_pages);
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(t, p, new_refs, live);
  const int64_t row_blocks = (t.rows + 3) / 4, planes = planes_of(pools), per = blocks_of_plane(pools, t.n_pages / 2);
  compact_do_kernel<<<(unsigned)(row_blocks + planes * per), 256, 0, stream>>>(t, p, new_tables, pools, row_blocks, per);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const PoolArgs& pools, const int32_t* src, const int32_t* dst, int64_t n,
                                hipStream_t stream) {
  const int64_t planes = planes_of(pools), per = blocks_of_plane(pools, n);
  copy_pages_kernel<<<(unsigned)(planes * per), 256, 0, stream>>>(pools, src, dst, n, per);
  return hipGetLastError();
}

}  // namespace moe
