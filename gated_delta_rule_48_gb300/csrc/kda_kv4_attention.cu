// A few query tokens of each sequence over the cache in 4 bits.
//
// One warp takes a query and head: a key per lane, 32 at a time, with the
// running maximum and sum, and the values with a few channels per lane.
#include <cmath>

#include "kda_attention.h"

namespace kda {

namespace {

constexpr int kWarps = 4;

template <int G>
__global__ void __launch_bounds__(32 * kWarps) kv4_attention_kernel(Kv4AttentionArgs a) {
  constexpr int D = 32 * G;
  __shared__ float s_q[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Kv4Pages& p = a.pages;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t rows = static_cast<int64_t>(a.N) * a.tokens;
  if (item >= rows * a.heads) return;
  const int64_t t = item / a.heads;
  const int32_t head = static_cast<int32_t>(item - t * a.heads), n = static_cast<int32_t>(t / a.tokens);
  const int32_t kv = head / (a.heads / p.heads);
  const int64_t reach = max(0, a.seq_lens[n] - a.tokens + 1 + static_cast<int32_t>(t % a.tokens));
  for (int c = lane; c < D; c += 32)
    s_q[warp][c] = to_f32(a.q[t * a.ld_q + head * D + c]) * (a.scale * kLog2e);
  __syncwarp();
  float top = -INFINITY, sum = 0.0f, o[G] = {};
  for (int64_t j0 = 0; j0 < reach; j0 += 32) {
    const int64_t j = j0 + lane;
    float x = -INFINITY;
    int64_t row = -1;
    if (j < reach) {
      const int64_t slot = kv4_slot(p, a.N, n, j, a.err);
      if (slot >= 0) row = kv4_row(p, slot, kv);
    }
    if (row >= 0) {
      x = 0.0f;
      for (int w = 0; w < 4 * G; ++w) {
        const int g = w % G, part = w / G;
        const uint32_t codes = reinterpret_cast<const uint32_t*>(p.k_codes + row * (16 * G))[w];
        float y = 0.0f;
        for (int i = 0; i < 8; ++i)
          y = fmaf(static_cast<float>(static_cast<int>(codes >> (4 * i) & 15u) - 8),
                   s_q[warp][32 * g + 8 * part + i], y);
        x = fmaf(y, bf16_to_f32(p.k_scales[row * G + g]), x);
      }
    }
    float next = max_nan(top, x);
#pragma unroll
    for (int w = 16; w; w /= 2) next = max_nan(next, __shfl_xor_sync(0xffffffffu, next, w));
    const float base = next == -INFINITY ? 0.0f : next, keep = ex2(top - base), e = ex2(x - base);
    top = next;
    sum = sum * keep + e;
#pragma unroll
    for (int i = 0; i < G; ++i) o[i] *= keep;
    for (int i = 0; i < 32; ++i) {
      const float pi = __shfl_sync(0xffffffffu, e, i);
      const int64_t r = __shfl_sync(0xffffffffu, row, i);
      if (r < 0) continue;
#pragma unroll
      for (int g = 0; g < G; ++g) {  // channel 32 g + lane
        const uint16_t h = reinterpret_cast<const uint16_t*>(p.v_codes + r * (16 * G))[(lane / 4) * G + g];
        const float v = static_cast<float>(static_cast<int>(h >> (4 * (lane % 4)) & 15) - 8);
        o[g] = fmaf(pi, v * bf16_to_f32(p.v_scales[r * G + g]), o[g]);
      }
    }
  }
#pragma unroll
  for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  const float r = reach > 0 ? 1.0f / sum : 0.0f;
  Bf16* out = a.out + t * a.ld_out + head * D;
#pragma unroll
  for (int g = 0; g < G; ++g) out[32 * g + lane] = from_f32<Bf16>(o[g] * r);
  if (a.lse && lane == 0) a.lse[item] = reach > 0 ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttentionArgs& a, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(a.N) * a.tokens * a.heads + kWarps - 1) / kWarps;
  prof_begin(s, "kda_kv4_attention");
  if (a.pages.d == 128) kv4_attention_kernel<4><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, s>>>(a);
  else kv4_attention_kernel<2><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, s>>>(a);
  prof_end(s, "kda_kv4_attention");
  return cudaGetLastError();
}

}  // namespace kda
