// Internal interface of attention and its cache: prompts, one token over a paged
// cache, the write of new keys and values into the pages, and the pages themselves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int64_t kAttnMaxTokens = 0x7FFFFF00;          // int32, the end of a tile behind the last one included
constexpr int kAttnMaxHeads = 4096;
constexpr int64_t kAttnMaxStride = (int64_t)1 << 24;    // elements: a tile of 64 tokens stays inside 32 bits of bytes
constexpr int kMaxPage = 4096;
constexpr int64_t kAttnMaxBatch = 65535;                // sequences: one dimension of a launch

// A [tokens x heads x D] matrix of 16-bit values whose heads are contiguous.
struct HeadRows {
  const uint16_t* p;
  int64_t token, head;  // strides, elements
};

struct PrefillArgs {
  HeadRows q, k, v;
  int64_t Tq, Tk;
  int heads, kv_heads, D;
  const int32_t *q_starts, *k_starts;  // [n + 1] each
  int64_t n;
  bool causal, f16;
  float scale;
  uint16_t* y;  // [Tq x heads x D]
  float* lse;   // [Tq x heads] or NULL
};
int64_t prefill_blocks(const PrefillArgs& a);
int64_t prefill_workspace_bytes(const PrefillArgs& a);
hipError_t launch_attention_prefill(const PrefillArgs& a, void* ws, hipStream_t stream);

// One layer's cache: [n_pages x kv_heads x P x D] keys and values, 16-bit or e4m3 with
// fp32 scales [n_pages x kv_heads x P]; row r of the table lists a sequence's pages.
struct CacheArgs {
  const void *k, *v;  // written by the append
  const float *k_scales, *v_scales;  // NULL for 16-bit caches
  int64_t n_pages;
  int kv_heads, P, shift, D;  // P = 1 << shift
  const int32_t* tables;  // [rows x width]
  int64_t rows;
  int width;
};

struct DecodeArgs {
  HeadRows q;
  int64_t B;  // rows of the table that are used
  int heads;
  CacheArgs c;
  const int32_t* lengths;  // [B]
  bool f16;
  float scale;
  uint16_t* y;  // [B x heads x D]
  float* lse;   // [B x heads] or NULL
};
int64_t decode_workspace_bytes(int64_t B, int heads, int kv_heads, int D);
hipError_t launch_attention_decode(const DecodeArgs& a, void* ws, hipStream_t stream);

struct AppendArgs {
  HeadRows q, k, v;  // q may be NULL
  int64_t T;
  int heads;  // of q
  CacheArgs c;
  const int32_t *rows, *positions;  // [T]
  const float* inv_freq;            // [rotary / 2] or NULL
  int rotary;
  bool interleaved, f16;
  HeadRows q_out, k_out;  // p may be NULL
};
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream);

// Pages.  A pool is planes x n_pages pages; every plane of it moves with its page.
constexpr int kMaxPools = 8;
struct PoolArgs {
  struct { char* base; int64_t planes, page_bytes; } pool[kMaxPools];
  int n;
  int64_t n_pages;
};
struct TableArgs {
  int32_t* tables;  // [rows x width]
  int64_t rows;
  int width;
  int32_t *lengths, *refs;
  int64_t n_pages;
  int P, shift;
};
int64_t pages_workspace_bytes(int64_t rows, int64_t n_pages);
hipError_t launch_kv_reserve(const TableArgs& t, const int32_t* grow, int32_t* status, void* ws, hipStream_t stream);
hipError_t launch_kv_fork(const TableArgs& t, const int32_t* parents, const PoolArgs& p, int32_t* status, void* ws,
                          hipStream_t stream);
hipError_t launch_kv_free(const TableArgs& t, const int32_t* drop, hipStream_t stream);
hipError_t launch_kv_compact(const TableArgs& t, const PoolArgs& p, int32_t* new_tables, int32_t* new_refs, int32_t* live,
                             void* ws, hipStream_t stream);
hipError_t launch_kv_copy_pages(const PoolArgs& p, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream);

}  // namespace moe
