// Internal declarations of the full-attention operators: attention over
// prompts, the paged cache in 4 bits, attention over that cache.  The arguments
// are already checked by the entry points (kda_attention_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"
#include "kda_internal.h"
#include "kda_ops.h"

namespace kda {

// A unit of rows whose keys several blocks share (kda_attention.cu).
struct PartInfo {
  int32_t parts;            // fewer than 2: it is not shared
  int32_t q0, n_q, len, tok0, head0;
};

// ---- kda_attention_fwd (kda_attention.cu).  Leading dimensions in elements.
struct AttentionArgs {
  const Bf16* q;            // [Tq, heads, d], tokens ld_q apart
  const Bf16* k;            // [Tk, kv_heads, d]
  const Bf16* v;            // [Tk, kv_heads, d]
  Bf16* out;                // [Tq, heads, d]
  float* lse;               // [Tq, heads] or null
  const int32_t* cu_q;      // [N + 1], or null: N sequences of Tq / N queries
  const int32_t* cu_k;      // [N + 1], null with cu_q
  int64_t ld_q, ld_k, ld_v, ld_out, Tq, Tk;
  int32_t N, heads, kv_heads, d;
  float scale;
  bool causal;
  bool sectors;             // every row of out starts on a 32-byte boundary
  int sm_count;
  int* err;
  // Few units of rows: their keys shared by several blocks, up to `splits` of them
  // (kda_attention.cu); a part's sums [unit * splits + part][256][d], each row's
  // maximum and sum of p, and each unit's rows and how many parts it has.
  int32_t splits = 1, units = 0;
  float* part_out = nullptr;
  float2* part_ml = nullptr;
  PartInfo* parts = nullptr;
  // Units of many keys: what blocks move out of tensor memory (kda_attention.cu),
  // [sm_count][256][d + 4]; null where no unit can have as many.
  float* moved = nullptr;
};
// Allocates its workspace, if any: a status of its own if that fails, else `e`.
kda_status launch_attention(const AttentionArgs& a, cudaStream_t s, cudaError_t& e);

// ---- the paged cache of 4-bit codes (kda_kv4.cu)
constexpr int kKv4Group = 32;  // channels of a token and head that share a scale

struct Kv4Pages {
  uint8_t* k_codes;         // [n_pages, heads, page_size, d / 2]
  uint16_t* k_scales;       // bf16 [n_pages, heads, page_size, d / 32]
  uint8_t* v_codes;
  uint16_t* v_scales;
  int32_t n_pages, heads, d;
  int page_shift;           // log2 of page_size
  const int32_t* table;     // [N, width], rows ld_table apart: the page of each page_size positions
  int64_t ld_table;
  int32_t width;
};

// Writing and reading spans: token cu[n] + i of the rows is position start[n] + i
// of sequence n.
struct Kv4SpanArgs {
  Kv4Pages pages;
  Bf16* k;                  // [T, heads, d], tokens ld_k apart; only read by the write
  Bf16* v;
  const int32_t* start;     // [N] or null (zeros); negative: the sequence is left out
  const int32_t* cu;        // [N + 1] or null (N sequences of T / N tokens)
  int64_t ld_k, ld_v, T;
  int32_t N;
  int sm_count;
  int* err;
};
cudaError_t launch_kv4_write(const Kv4SpanArgs& a, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4SpanArgs& a, cudaStream_t s);

// ---- kda_kv4_attention (kda_kv4_attention.cu)
struct Kv4AttentionArgs {
  Kv4Pages pages;
  const Bf16* q;            // [N, tokens, heads, d], tokens ld_q apart
  Bf16* out;
  float* lse;               // [N, tokens, heads] or null
  const int32_t* seq_lens;  // [N], the queries' own positions among them
  int64_t ld_q, ld_out;
  int32_t N, tokens, heads;
  float scale;
  int sm_count;
  int* err;
};
// Allocates its workspace: a status of its own if that fails, else `e`.
kda_status launch_kv4_attention(const Kv4AttentionArgs& a, cudaStream_t s, cudaError_t& e);

// ---- device helpers
// The slot (page * page_size + place) of a position >= 0 of sequence n, or -1
// (recorded as an input error) where its table has no valid page for it.
__device__ __forceinline__ int64_t kv4_slot(const Kv4Pages& p, int32_t N, int32_t n, int64_t position,
                                            int* err) {
  const int64_t i = position >> p.page_shift, at = n * p.ld_table + i;
  int32_t page = -1;
  if (i < p.width && kda_guard(at, 1, (N - 1) * p.ld_table + p.width, err)) page = p.table[at];
  if (page < 0 || page >= p.n_pages) {
    atomicOr(err, kDevErrPage);
    return -1;
  }
  return (static_cast<int64_t>(page) << p.page_shift) + (position & ((1 << p.page_shift) - 1));
}
// The row of a slot and head in the cache's arrays (rows of d / 2 bytes, of d / 32 scales).
__device__ __forceinline__ int64_t kv4_row(const Kv4Pages& p, int64_t slot, int32_t head) {
  return (((slot >> p.page_shift) * p.heads + head) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}
__device__ __forceinline__ int64_t kv4_rows(const Kv4Pages& p) {
  return (static_cast<int64_t>(p.n_pages) * p.heads) << p.page_shift;
}

}  // namespace kda
