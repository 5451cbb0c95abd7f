// Attention over prompts: grouped heads, packed sequences, causal or not.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j),  j < reach of i
//
// One warp takes a query and head: a key per lane, 32 at a time, with the
// running maximum and sum, and the values with a few channels per lane.
#include <cmath>

#include "kda_attention.h"

namespace kda {

namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attention_kernel(AttentionArgs a) {
  __shared__ float s_q[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.cu_q && blockIdx.x == 0) {
    check_cu_seqlens(a.cu_q, a.N, a.Tq, threadIdx.x, 32 * kWarps, a.err);
    check_cu_seqlens(a.cu_k, a.N, a.Tk, threadIdx.x, 32 * kWarps, a.err);
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (item >= a.Tq * a.heads) return;
  const int64_t t = item / a.heads;
  const int32_t head = static_cast<int32_t>(item - t * a.heads);
  const int32_t n = a.cu_q ? sequence_of(a.cu_q, a.N, t, a.err) : static_cast<int32_t>(t / (a.Tq / a.N));
  int64_t q0, q1, k0, k1;
  sequence_span(a.cu_q, a.N, a.Tq, n, q0, q1, a.err);
  sequence_span(a.cu_k, a.N, a.Tk, n, k0, k1, a.err);
  const int64_t len = k1 - k0;
  const int64_t reach = a.causal ? min(len, max(int64_t{0}, t - q0 + 1 + len - (q1 - q0))) : len;
  const Bf16* q = a.q + t * a.ld_q + head * D;
  for (int c = lane; c < D; c += 32) s_q[warp][c] = to_f32(q[c]) * (a.scale * kLog2e);
  __syncwarp();
  const int32_t kv = head / (a.heads / a.kv_heads);
  float top = -INFINITY, sum = 0.0f, o[D / 32] = {};
  for (int64_t j0 = 0; j0 < reach; j0 += 32) {
    const int64_t j = j0 + lane;
    float x = -INFINITY;
    if (j < reach) {
      const Bf16* k = a.k + (k0 + j) * a.ld_k + kv * D;
      x = 0.0f;
      for (int c = 0; c < D; c += 8) {
        float v[8];
        load8(k + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x = fmaf(v[i], s_q[warp][c + i], x);
      }
    }
    float next = max_nan(top, x);
#pragma unroll
    for (int w = 16; w; w /= 2) next = max_nan(next, __shfl_xor_sync(0xffffffffu, next, w));
    const float base = next == -INFINITY ? 0.0f : next, keep = ex2(top - base), p = ex2(x - base);
    top = next;
    sum = sum * keep + p;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= keep;
    const int count = static_cast<int>(min(int64_t{32}, reach - j0));
    for (int i = 0; i < count; ++i) {
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const Bf16* v = a.v + (k0 + j0 + i) * a.ld_v + kv * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[c] = fmaf(pi, to_f32(v[32 * c + lane]), o[c]);
    }
  }
#pragma unroll
  for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  const float r = reach > 0 ? 1.0f / sum : 0.0f;
  Bf16* out = a.out + t * a.ld_out + head * D;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) out[32 * c + lane] = from_f32<Bf16>(o[c] * r);
  if (a.lse && lane == 0) a.lse[item] = reach > 0 ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t s) {
  const int64_t blocks = (a.Tq * a.heads + kWarps - 1) / kWarps;
  prof_begin(s, "kda_attention_fwd");
  if (a.d == 128) attention_kernel<128><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, s>>>(a);
  else attention_kernel<64><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, s>>>(a);
  prof_end(s, "kda_attention_fwd");
  return cudaGetLastError();
}

}  // namespace kda
