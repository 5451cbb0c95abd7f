// Entry points of the full-attention operators (include/kda.h): argument checks
// on the host, then the launches.
#include <cuda_runtime.h>

#include <cmath>

#include "kda.h"
#include "kda_attention.h"
#include "kda_checks.h"

using namespace kda;

namespace {

kda_status check_heads(int32_t heads, int32_t kv_heads, int32_t d) {
  if (heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "n_heads=%d is not a multiple of n_kv_heads=%d", heads, kv_heads);
  if (d != 64 && d != 128) return bad(KDA_ERR_UNSUPPORTED, "d=%d is not 64 or 128", d);
  if (heads > 65536) return bad(KDA_ERR_UNSUPPORTED, "n_heads=%d exceeds 65536", heads);
  return KDA_OK;
}

kda_status check_scale(float scale) {
  // (scale log2 e is a number of 32 bits too)
  if (!(scale > 0.0f) || std::isinf(scale * 1.5f))
    return bad(KDA_ERR_INVALID_ARGUMENT, "scale=%g is not positive and finite", scale);
  return KDA_OK;
}

// Rows of bf16 that are read or written 16 bytes at a time.
kda_status check_wide(const char* name, const void* p, int64_t rows, int64_t ld, int64_t cols) {
  KDA_TRY(check_rows(name, p, ld, cols, 2));
  if (p && (!aligned(p, 16) || (rows > 1 && ld % 8 != 0)))
    return bad(KDA_ERR_INVALID_ARGUMENT, "%s: every row must start on a 16-byte boundary", name);
  return KDA_OK;
}

// (a single row has no next one, whatever its distance: its own width does, which a tensor
// map takes, where distances end at 2^40 bytes)
int64_t pitch_of(int64_t rows, int64_t ld, int64_t cols) { return rows > 1 ? ld : cols; }

kda_status check_sequences(const char* what, int64_t T, int32_t N, const int32_t* cu) {
  if (T < 0 || N < 0) return bad(KDA_ERR_INVALID_ARGUMENT, "%s=%lld n_seqs=%d", what, (long long)T, N);
  if (T > 0x7fffffffLL) return bad(KDA_ERR_UNSUPPORTED, "%s=%lld", what, (long long)T);
  if (N == 0 && T > 0) return bad(KDA_ERR_INVALID_ARGUMENT, "tokens given but n_seqs = 0");
  if (!cu && N > 0 && T % N != 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens is NULL but %s=%lld is not a multiple of n_seqs=%d", what,
               (long long)T, N);
  return KDA_OK;
}

// The cache's arrays and the table; `parts` (6): what calls may not write over.
kda_status check_cache(const kda_kv4_cache* c, const int32_t* table, int64_t ld_table, int32_t width,
                       int32_t N, Kv4Pages& p, Rows* parts) {
  if (!c) return bad(KDA_ERR_INVALID_ARGUMENT, "cache is NULL");
  if (c->n_pages < 0 || width < 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "n_pages=%d max_pages=%d", c->n_pages, width);
  KDA_TRY(check_heads(c->n_kv_heads, c->n_kv_heads, c->d));
  const int32_t size = c->page_size;
  if (size < 16 || size > 65536 || (size & (size - 1)) != 0)
    return bad(KDA_ERR_UNSUPPORTED, "page_size=%d is not a power of two from 16 to 65536", size);
  if (static_cast<int64_t>(c->n_kv_heads) * size > 1 << 30 ||
      static_cast<int64_t>(c->n_pages) * c->n_kv_heads > (1LL << 48) / size)
    return bad(KDA_ERR_UNSUPPORTED, "n_pages=%d of n_kv_heads=%d and page_size=%d", c->n_pages, c->n_kv_heads, size);
  const struct { const void* p; const char* n; } arrays[] = {{c->k_codes, "k_codes"},
                                                             {c->k_scales, "k_scales"},
                                                             {c->v_codes, "v_codes"},
                                                             {c->v_scales, "v_scales"}};
  const int64_t rows = static_cast<int64_t>(c->n_pages) * c->n_kv_heads * size;
  for (int i = 0; i < 4; ++i) {
    if (!arrays[i].p && rows > 0) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", arrays[i].n);
    if (!aligned(arrays[i].p, 16))
      return bad(KDA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", arrays[i].n);
    const int64_t bytes = rows * (i % 2 ? c->d / 16 : c->d / 2);
    parts[i] = Rows{arrays[i].n, arrays[i].p, arrays[i].p ? 1 : 0, bytes, bytes};
  }
  if (!table && width > 0 && N > 0) return bad(KDA_ERR_INVALID_ARGUMENT, "block_table is NULL");
  if (N == 1) ld_table = width;
  KDA_TRY(check_rows("block_table", table, ld_table, width, 4));
  parts[4] = rows_of("block_table", table, N, ld_table, width, 4);
  p.k_codes = static_cast<uint8_t*>(c->k_codes);
  p.k_scales = static_cast<uint16_t*>(c->k_scales);
  p.v_codes = static_cast<uint8_t*>(c->v_codes);
  p.v_scales = static_cast<uint16_t*>(c->v_scales);
  p.n_pages = c->n_pages;
  p.heads = c->n_kv_heads;
  p.d = c->d;
  p.page_shift = 0;
  while ((1 << p.page_shift) < size) ++p.page_shift;
  p.table = table;
  p.ld_table = ld_table;
  p.width = width;
  return KDA_OK;
}

// What writing and reading share.
kda_status check_span(const void* k, int64_t ld_k, const void* v, int64_t ld_v, const kda_kv4_cache* cache,
                      const int32_t* table, int64_t ld_table, int32_t width, const int32_t* start,
                      const int32_t* cu, int64_t T, int32_t N, bool write, Kv4SpanArgs& a) {
  KDA_TRY(check_sequences("total_tokens", T, N, cu));
  Rows part[9];
  KDA_TRY(check_cache(cache, table, ld_table, width, N, a.pages, part));
  if (T > 0 && (!k || !v)) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", !k ? "k" : "v");
  const int64_t cols = static_cast<int64_t>(cache->n_kv_heads) * cache->d;
  KDA_TRY(check_wide("k", k, T, ld_k, cols));
  KDA_TRY(check_wide("v", v, T, ld_v, cols));
  KDA_TRY(check_rows("start", start, 1, 1, 4));
  KDA_TRY(check_rows("cu_seqlens", cu, 1, 1, 4));
  ld_k = pitch_of(T, ld_k, cols);
  ld_v = pitch_of(T, ld_v, cols);
  part[5] = rows_of("start", start, 1, N, N, 4);
  part[6] = rows_of("cu_seqlens", cu, 1, N + 1LL, N + 1LL, 4);
  part[7] = rows_of("k", k, T, ld_k, cols, 2);
  part[8] = rows_of("v", v, T, ld_v, cols, 2);
  if (write) {
    for (int i = 0; i < 4; ++i) {
      KDA_TRY(check_output(part[i], part + 4, 5, nullptr));
      KDA_TRY(check_output(part[i], part, i, nullptr));
    }
  } else {
    KDA_TRY(check_output(part[7], part, 7, nullptr));
    KDA_TRY(check_output(part[8], part, 8, nullptr));
  }
  a.k = static_cast<Bf16*>(const_cast<void*>(k));
  a.v = static_cast<Bf16*>(const_cast<void*>(v));
  a.start = start;
  a.cu = cu;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.T = T;
  a.N = N;
  if (N == 0) return KDA_OK;
  KDA_TRY(device_sm_count(&a.sm_count));
  return device_error_word(&a.err);
}

}  // namespace

extern "C" kda_status kda_attention_fwd(const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                                        const void* v, int64_t ld_v, const int32_t* cu_seqlens_q,
                                        const int32_t* cu_seqlens_k, void* out, int64_t ld_out, float* lse,
                                        int64_t total_q, int64_t total_k, int32_t n_seqs, int32_t n_heads,
                                        int32_t n_kv_heads, int32_t d, float scale, int32_t causal,
                                        void* stream) {
  NvtxRange nvtx_range("kda_attention_fwd");
  if (cu_seqlens_k && !cu_seqlens_q)
    return bad(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_k is given but cu_seqlens_q is NULL");
  KDA_TRY(check_sequences("total_q", total_q, n_seqs, cu_seqlens_q));
  KDA_TRY(check_sequences("total_k", total_k, n_seqs, cu_seqlens_q));
  KDA_TRY(check_heads(n_heads, n_kv_heads, d));
  KDA_TRY(check_scale(scale));
  if (cu_seqlens_q && !cu_seqlens_k) {
    if (total_k != total_q)
      return bad(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_k is NULL but total_k=%lld is not total_q=%lld",
                 (long long)total_k, (long long)total_q);
    cu_seqlens_k = cu_seqlens_q;
  }
  if (total_q * n_heads > (1LL << 37))
    return bad(KDA_ERR_UNSUPPORTED, "total_q=%lld of n_heads=%d", (long long)total_q, n_heads);
  if (total_q == 0) return KDA_OK;
  const struct { const void* p; const char* n; bool need; } req[] = {
      {q, "q", true}, {k, "k", total_k > 0}, {v, "v", total_k > 0}, {out, "out", true}};
  for (auto& r : req)
    if (r.need && !r.p) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", r.n);
  const int64_t wq = static_cast<int64_t>(n_heads) * d, wk = static_cast<int64_t>(n_kv_heads) * d;
  KDA_TRY(check_wide("q", q, total_q, ld_q, wq));
  KDA_TRY(check_wide("k", k, total_k, ld_k, wk));
  KDA_TRY(check_wide("v", v, total_k, ld_v, wk));
  KDA_TRY(check_wide("out", out, total_q, ld_out, wq));
  KDA_TRY(check_rows("lse", lse, n_heads, n_heads, 4));
  KDA_TRY(check_rows("cu_seqlens_q", cu_seqlens_q, 1, 1, 4));
  KDA_TRY(check_rows("cu_seqlens_k", cu_seqlens_k, 1, 1, 4));
  AttentionArgs a;
  a.ld_q = pitch_of(total_q, ld_q, wq);
  a.ld_k = pitch_of(total_k, ld_k, wk);
  a.ld_v = pitch_of(total_k, ld_v, wk);
  a.ld_out = pitch_of(total_q, ld_out, wq);
  const Rows in[] = {rows_of("q", q, total_q, a.ld_q, wq, 2), rows_of("k", k, total_k, a.ld_k, wk, 2),
                     rows_of("v", v, total_k, a.ld_v, wk, 2),
                     rows_of("cu_seqlens_q", cu_seqlens_q, 1, n_seqs + 1LL, n_seqs + 1LL, 4),
                     rows_of("cu_seqlens_k", cu_seqlens_k, 1, n_seqs + 1LL, n_seqs + 1LL, 4)};
  const Rows outs[] = {rows_of("out", out, total_q, a.ld_out, wq, 2),
                       rows_of("lse", lse, 1, total_q * n_heads, total_q * n_heads, 4)};
  KDA_TRY(check_output(outs[0], in, 5, nullptr));
  KDA_TRY(check_output(outs[1], in, 5, nullptr));
  KDA_TRY(check_output(outs[1], outs, 1, nullptr));
  a.q = static_cast<const Bf16*>(q);
  a.k = static_cast<const Bf16*>(k);
  a.v = static_cast<const Bf16*>(v);
  a.out = static_cast<Bf16*>(out);
  a.lse = lse;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.Tq = total_q;
  a.Tk = total_k;
  a.N = n_seqs;
  a.heads = n_heads;
  a.kv_heads = n_kv_heads;
  a.d = d;
  a.scale = scale;
  a.causal = causal != 0;
  a.sectors = aligned(out, 32) && a.ld_out % 16 == 0;
  KDA_TRY(device_sm_count(&a.sm_count));
  KDA_TRY(device_error_word(&a.err));
  cudaError_t e = cudaSuccess;
  KDA_TRY(launch_attention(a, static_cast<cudaStream_t>(stream), e));
  return launched(e, "attention launch");
}

extern "C" kda_status kda_kv4_write(const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                    const kda_kv4_cache* cache, const int32_t* block_table,
                                    int64_t ld_table, int32_t max_pages, const int32_t* start,
                                    const int32_t* cu_seqlens, int64_t total_tokens, int32_t n_seqs,
                                    void* stream) {
  NvtxRange nvtx_range("kda_kv4_write");
  Kv4SpanArgs a;
  KDA_TRY(check_span(k, ld_k, v, ld_v, cache, block_table, ld_table, max_pages, start, cu_seqlens,
                     total_tokens, n_seqs, true, a));
  if (n_seqs == 0) return KDA_OK;
  return launched(launch_kv4_write(a, static_cast<cudaStream_t>(stream)), "cache write launch");
}

extern "C" kda_status kda_kv4_read(void* k, int64_t ld_k, void* v, int64_t ld_v,
                                   const kda_kv4_cache* cache, const int32_t* block_table,
                                   int64_t ld_table, int32_t max_pages, const int32_t* start,
                                   const int32_t* cu_seqlens, int64_t total_tokens, int32_t n_seqs,
                                   void* stream) {
  NvtxRange nvtx_range("kda_kv4_read");
  Kv4SpanArgs a;
  KDA_TRY(check_span(k, ld_k, v, ld_v, cache, block_table, ld_table, max_pages, start, cu_seqlens,
                     total_tokens, n_seqs, false, a));
  if (n_seqs == 0) return KDA_OK;
  return launched(launch_kv4_read(a, static_cast<cudaStream_t>(stream)), "cache read launch");
}

extern "C" kda_status kda_kv4_attention(const void* q, int64_t ld_q, const kda_kv4_cache* cache,
                                        const int32_t* block_table, int64_t ld_table, int32_t max_pages,
                                        const int32_t* seq_lens, void* out, int64_t ld_out, float* lse,
                                        int32_t n_seqs, int32_t n_tokens, int32_t n_heads, float scale,
                                        void* stream) {
  NvtxRange nvtx_range("kda_kv4_attention");
  if (n_seqs < 0 || n_tokens < 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "n_seqs=%d n_tokens=%d", n_seqs, n_tokens);
  Kv4AttentionArgs a;
  Rows in[7];
  KDA_TRY(check_cache(cache, block_table, ld_table, max_pages, n_seqs, a.pages, in));
  KDA_TRY(check_heads(n_heads, cache->n_kv_heads, cache->d));
  KDA_TRY(check_scale(scale));
  const int64_t rows = static_cast<int64_t>(n_seqs) * n_tokens, cols = static_cast<int64_t>(n_heads) * cache->d;
  if (rows > 0x7fffffffLL || rows * n_heads > 0x7fffffffLL)
    return bad(KDA_ERR_UNSUPPORTED, "n_seqs=%d n_tokens=%d n_heads=%d", n_seqs, n_tokens, n_heads);
  if (rows == 0) return KDA_OK;
  const struct { const void* p; const char* n; } req[] = {{q, "q"}, {seq_lens, "seq_lens"}, {out, "out"}};
  for (auto& r : req)
    if (!r.p) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", r.n);
  KDA_TRY(check_wide("q", q, rows, ld_q, cols));
  KDA_TRY(check_wide("out", out, rows, ld_out, cols));
  KDA_TRY(check_rows("seq_lens", seq_lens, 1, 1, 4));
  KDA_TRY(check_rows("lse", lse, n_heads, n_heads, 4));
  a.ld_q = pitch_of(rows, ld_q, cols);
  a.ld_out = pitch_of(rows, ld_out, cols);
  in[5] = rows_of("seq_lens", seq_lens, 1, n_seqs, n_seqs, 4);
  in[6] = rows_of("q", q, rows, a.ld_q, cols, 2);
  const Rows outs[] = {rows_of("out", out, rows, a.ld_out, cols, 2),
                       rows_of("lse", lse, 1, rows * n_heads, rows * n_heads, 4)};
  KDA_TRY(check_output(outs[0], in, 7, nullptr));
  KDA_TRY(check_output(outs[1], in, 7, nullptr));
  KDA_TRY(check_output(outs[1], outs, 1, nullptr));
  a.q = static_cast<const Bf16*>(q);
  a.out = static_cast<Bf16*>(out);
  a.lse = lse;
  a.seq_lens = seq_lens;
  a.N = n_seqs;
  a.tokens = n_tokens;
  a.heads = n_heads;
  a.scale = scale;
  KDA_TRY(device_sm_count(&a.sm_count));
  KDA_TRY(device_error_word(&a.err));
  cudaError_t e = cudaSuccess;
  KDA_TRY(launch_kv4_attention(a, static_cast<cudaStream_t>(stream), e));
  return launched(e, "cache attention launch");
}
