// Internal declarations of the operators around the recurrent layer (norm,
// 8-bit product, short convolution, selective scan): the arguments their
// kernels take, already checked by the entry points (kda_ops_api.cu), and the
// device helpers the kernels share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"
#include "kda_internal.h"

namespace kda {

constexpr int kScaleGroup = 128;         // columns (or rows and columns) that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 0x1p-64f;     // a group's largest magnitude counts as at least this
constexpr int kMaxNormDim = 65536;

// ---- kda_add_rms_norm (kda_norm.cu).  Leading dimensions in elements.
struct NormArgs {
  const void* x;
  const void* residual;   // null: h = x
  const void* weight;     // [dim]
  void* h;                // x + residual in x's type, or null
  void* y;                // x's type, or e4m3 with y_scale
  float* y_scale;         // [rows, ceil(dim / 128)] when y is e4m3
  int64_t ld_x, ld_res, ld_h, ld_y, ld_scale;
  int64_t rows;
  int32_t dim;
  float eps;
  bool bf16, w_bf16, quant;
  bool vec;               // every row starts on a 16-byte boundary and dim % 8 == 0
  int sm_count;
  int* err;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);

// ---- kda_short_conv_fwd, kda_short_conv_step (kda_conv.cu)
constexpr int kMaxConvWidth = 8;
struct ConvArgs {
  const void* x;          // [T, dim]; the step: [N, dim], one token of each sequence
  const void* weight;     // [dim, width]
  const void* bias;       // [dim] or null
  const void* state_in;   // [N, width - 1, dim] or null (zeros)
  void* state_out;        // [N, width - 1, dim] or null; the step: state_in itself
  const int32_t* cu;      // [N + 1] or null (N sequences of T / N tokens)
  void* y;                // [T, dim]
  int64_t ld_x, ld_y, T;
  int32_t N, dim, width;
  bool bf16, w_bf16, silu;
  int vec;                // channels that can be read and written at a time: 4, 2 or 1
  int sm_count;
  int* err;
};
cudaError_t launch_conv(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s);

// ---- kda_ssm_scan_fwd, kda_ssm_scan_step (kda_ssm.cu)
struct SsmArgs {
  const void* x;          // [T, dim]; the step: [N, dim], one token of each sequence
  const void* dt;         // [T, dim]
  const void* z;          // [T, dim] or null
  const void* B;          // [T, groups, state]
  const void* C;          // [T, groups, state]
  const float* A;         // [dim, state]
  const float* D;         // [dim] or null
  const float* dt_bias;   // [dim] or null
  const float* h0;        // [N, dim, state] or null; the step: h itself
  float* h_out;           // [N, dim, state] or null
  const int32_t* cu;      // [N + 1] or null (N sequences of T / N tokens)
  void* y;                // [T, dim]
  int64_t ld_x, ld_dt, ld_z, ld_b, ld_c, ld_y, T;
  int32_t N, dim, state, groups;
  bool bf16, softplus;
  bool vec;               // A, B and C can be read four values at a time
  bool pairs;             // so, and x, dt, z and y can be read and written two channels at a time
  int sm_count;
  int* err;
  // prompts cut into chunks: the summaries of the chunks (null without)
  int64_t chunk = 0, n_chunks = 1;
  float* chunk_h = nullptr;    // [n_chunks, dim, state]
  float* chunk_dt = nullptr;   // [n_chunks, dim]
};
// Tokens per chunk of a prompt's scan; `cut`: whether sequences may be cut by
// a chunk's end, so that summaries are needed.
void ssm_chunks(SsmArgs& a, bool& cut);
cudaError_t launch_ssm_scan(const SsmArgs& a, bool cut, cudaStream_t s);
cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t s);

// ---- kda_matmul_fp8 (kda_matmul_fp8.cu)
struct MatmulArgs {
  const void* a;          // e4m3 [M, K], rows on 16-byte boundaries
  const float* a_scale;   // [M, ceil(K / 128)]
  const void* b;          // e4m3 [N, K], rows on 16-byte boundaries
  const float* b_scale;   // [ceil(N / 128), ceil(K / 128)]
  void* out;              // bf16 or f32 [M, N]
  int64_t ld_a, ld_as, ld_b, ld_bs, ld_out;
  int32_t M, N, K;
  bool bf16;              // out's type
  int sm_count;
  int* err;
};
cudaError_t launch_matmul_fp8(const MatmulArgs& a, cudaStream_t s);

// ---- host-side state shared with the other entry points (kda_api.cu)
kda_status device_sm_count(int* out);
// Stream-ordered workspace from the library's pool (while `s` is being
// captured: from the device's default pool, as a graph memory node).
kda_status workspace_alloc(size_t bytes, cudaStream_t s, void** out);

// ---- device helpers
struct Bf16 { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Bf16 v) { return bf16_to_f32(v.bits); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float v) {
  Bf16 r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r.bits) : "f"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const Bf16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(Bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]),
                                            pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// N (1, 2 or 4) consecutive elements, aligned to their total size, in the
// registers they were loaded into: taking two bf16 values of one register
// apart, or widening one, would wait for the load.
template <typename T, int N>
struct RawVec;
template <>
struct RawVec<Bf16, 1> {
  Bf16 v;
  __device__ __forceinline__ void load(const Bf16* p) { v = *p; }
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
};
template <>
struct RawVec<Bf16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const Bf16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i ? v & 0xffff0000u : v << 16);
  }
};
template <>
struct RawVec<Bf16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const Bf16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct RawVec<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ float get(int) const { return v; }
};
template <>
struct RawVec<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ float get(int i) const { return i ? v.y : v.x; }
};
template <>
struct RawVec<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }
};
template <int N, typename T>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  RawVec<T, N> r;
  r.load(p);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = r.get(i);
}
template <int N>
__device__ __forceinline__ void store_n(Bf16* p, const float (&v)[N]) {
  if constexpr (N == 1) *p = from_f32<Bf16>(v[0]);
  else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = pack2_bf16(v[0], v[1]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&v)[N]) {
  if constexpr (N == 1) *p = v[0];
  else if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// The sequence of packed token t: the first n with cu[n + 1] > t (at most N - 1).
// Whatever cu holds, the result is in [0, N - 1].
__device__ __forceinline__ int32_t sequence_of(const int32_t* cu, int32_t N, int64_t t, int* err) {
  int32_t lo = 0, hi = N - 1;
  while (lo < hi) {
    const int32_t mid = lo + ((hi - lo) >> 1);
    if (!kda_guard(mid + 1, 1, static_cast<int64_t>(N) + 1, err)) break;
    if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// cu_seqlens checked by one block: cu[0] = 0, no decrease, cu[N] = T.
__device__ __forceinline__ void check_cu_seqlens(const int32_t* cu, int32_t N, int64_t T, int tid,
                                                 int n_threads, int* err) {
  bool ok = true;
  for (int64_t n = tid; n < N; n += n_threads) {
    if (!kda_guard(n, 2, static_cast<int64_t>(N) + 1, err)) break;
    ok = ok && cu[n + 1] >= cu[n];
    if (n == 0) ok = ok && cu[0] == 0;
    if (n == N - 1) ok = ok && cu[N] == T;
  }
  if (!ok) atomicOr(err, kDevErrCuSeqlens);
}

// Tokens [start, end) of sequence n: from cu, clamped to [0, T], or of T / N tokens.
__device__ __forceinline__ void sequence_span(const int32_t* cu, int32_t N, int64_t T, int32_t n,
                                              int64_t& start, int64_t& end, int* err) {
  if (cu) {
    start = end = 0;
    if (!kda_guard(n, 2, static_cast<int64_t>(N) + 1, err)) return;
    start = min(max(static_cast<int64_t>(cu[n]), int64_t{0}), T);
    end = min(max(static_cast<int64_t>(cu[n + 1]), start), T);
  } else {
    const int64_t len = T / N;
    start = len * n;
    end = start + len;
  }
}

// The larger of two values; NaN if either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two values to e4m3, round to nearest even, clamped to +-448 (NaN stays NaN).
__device__ __forceinline__ uint16_t pack2_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---- pairs of 32-bit values
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// v sigmoid(v).  Relative error: (1.25 |v| + 8) 2^-24, of which 1.25 |v| is the
// rounding of the exponent v log2 e and the rest the approximate exponential
// (2^-22.5) and reciprocal (2^-23) and two roundings.  Below v = -87.3 the
// reciprocal is smaller than 2^-126 and flushed: the result is -0, less than
// 88 * 2^-126 = 1.1e-36 off.  (The quotient in 32 bits, v / (1 + e^-v), is -0 from
// v = -88.8 on.  Scaled by powers of two so that the result fades out instead,
// the convolution was 2 to 3.5 % slower and the scan of 4 x 4096 tokens, 4096
// channels 10 %: 427 -> 471 us.)
__device__ __forceinline__ float silu(float v) { return v * rcp(1.0f + ex2(v * -kLog2e)); }

}  // namespace kda
