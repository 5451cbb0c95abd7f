// Selective state space scan over packed sequences, and its step for one token
// of each sequence.
//
// Per channel d with a state h of S values, decay rates A[d, :] and, per
// token, a step size dt, an input x and vectors B, C that the channels of a
// group share:
//
//   dt' = softplus(dt + dt_bias[d])                 (or dt + dt_bias[d])
//   h   = exp(dt' A[d, :]) h + dt' x B
//   y   = sum(h C) + D[d] x,   times z sigmoid(z) when there is a gate
//
// Everything is in 32 bits; exp(dt' A) is 2^(dt' (A log2 e)) by the hardware's
// approximate exponential.
//
// Bound: instruction issue and the exponentials (one per token, channel and
// state value, against 8 bytes per token and channel), then HBM.  Four lanes
// share a channel, a quarter of its state each, and take four tokens at a
// time: the work that a token needs once (softplus, gate, loads, the store)
// is done by the lane whose number is the token's, and handed round by
// shuffles, so nothing is computed four times.  The state's recurrence and the
// read-out run on pairs of 32-bit values in one instruction.  B and C come
// from shared memory, converted once per block; the next tile of tokens is
// fetched into registers while one is computed.
//
// Prompts are cut into chunks of the packed axis, whatever the sequences'
// lengths, so that blocks are equally long.  A sequence cut by a chunk's end
// maps its state affinely over the chunk, h -> exp(A sum(dt')) h + h_local: a
// first launch computes h_local and sum(dt') of such pieces, and in the second
// each block chains the pieces before its own to its entry state.  Where no
// sequence is cut there is one launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "kda_ops.h"

namespace kda {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kLanes = 4;            // lanes per channel, and tokens taken together
constexpr int kScanThreads = 128;
constexpr int kScanChannels = kScanThreads / kLanes;

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
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(ex2(lo), ex2(hi));
}

// log(1 + e^v)
__device__ __forceinline__ float softplus(float v) {
  return fmaxf(v, 0.0f) + log1pf(__expf(-fabsf(v)));
}

// Where state value s of a channel lives: lane (s / 4) % 4, its piece s / 16.
template <int S>
struct State {
  static constexpr int kQuads = S / (4 * kLanes);  // groups of four values per lane
  f32x2 h[2 * kQuads], a[2 * kQuads];              // the state, and A log2 e

  __device__ __forceinline__ static int64_t at(int lane4, int q) { return 16 * q + 4 * lane4; }

  // `live`: the channel exists
  __device__ __forceinline__ void load_rates(const float* A, int64_t c, int64_t dim, int lane4,
                                             bool live, int* err) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int64_t e = c * S + at(lane4, q);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live && kda_guard(e, 4, dim * S, err)) v = make_float4(A[e], A[e + 1], A[e + 2], A[e + 3]);
      a[2 * q] = pack2(v.x * kLog2e, v.y * kLog2e);
      a[2 * q + 1] = pack2(v.z * kLog2e, v.w * kLog2e);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 2 * kQuads; ++i) h[i] = 0;
  }
  // row: the channel's row of a [rows, S] buffer (dense, 16-byte aligned)
  __device__ __forceinline__ void load(const float* p, int64_t row, int64_t rows, int lane4,
                                       bool live, int* err) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int64_t e = row * S + at(lane4, q);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p && live && kda_guard(e, 4, rows * S, err)) v = *reinterpret_cast<const float4*>(p + e);
      h[2 * q] = pack2(v.x, v.y);
      h[2 * q + 1] = pack2(v.z, v.w);
    }
  }
  __device__ __forceinline__ void store(float* p, int64_t row, int64_t rows, int lane4, bool live,
                                        int* err) const {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int64_t e = row * S + at(lane4, q);
      float4 v;
      unpack2(h[2 * q], v.x, v.y);
      unpack2(h[2 * q + 1], v.z, v.w);
      if (live && kda_guard(e, 4, rows * S, err)) *reinterpret_cast<float4*>(p + e) = v;
    }
  }
  // h = exp(dt A) h + u B, B the token's row in shared memory
  __device__ __forceinline__ void step(float dt, float u, const float* B, int lane4) {
    const f32x2 dd = pack2(dt, dt), uu = pack2(u, u);
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(B + at(lane4, q));
      h[2 * q] = fma2(ex2_2(mul2(dd, a[2 * q])), h[2 * q], mul2(uu, b.x));
      h[2 * q + 1] = fma2(ex2_2(mul2(dd, a[2 * q + 1])), h[2 * q + 1], mul2(uu, b.y));
    }
  }
  // this lane's part of sum(h C)
  __device__ __forceinline__ float read(const float* C, int lane4) const {
    f32x2 acc = 0;
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(C + at(lane4, q));
      acc = fma2(h[2 * q], c.x, acc);
      acc = fma2(h[2 * q + 1], c.y, acc);
    }
    float lo, hi;
    unpack2(acc, lo, hi);
    return lo + hi;
  }
};

// One element of a [T, dim] tensor, or 0 past the end.
template <typename T>
__device__ __forceinline__ float element(const void* p, int64_t t, int64_t ld, int64_t c, bool live,
                                         const SsmArgs& a) {
  const int64_t e = t * ld + c;
  return live && kda_guard(e, 1, (a.T - 1) * ld + a.dim, a.err)
             ? to_f32(static_cast<const T*>(p)[e]) : 0.f;
}

// Sum over the four lanes of a channel, for four tokens at once: lane j ends
// with the sum of v[j].
__device__ __forceinline__ float sum_to_own(const float (&v)[4], int lane4) {
  const bool odd = lane4 & 1, high = lane4 & 2;
  float lo = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
  float hi = (odd ? v[3] : v[2]) + __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[3], 1);
  return (high ? hi : lo) + __shfl_xor_sync(0xffffffffu, high ? lo : hi, 2);
}

// SUMMARY: the piece's final state from zero (or the sequence's start) and its
// sum of step sizes; otherwise outputs and final states.
template <typename T, int S, bool SUMMARY>
struct Scan {
  static constexpr int kTile = S <= 32 ? 16 : 8;       // tokens per tile
  static constexpr int kBatches = kTile / kLanes;
  static constexpr int kRow = (SUMMARY ? 1 : 2) * S;   // B (and C) of a token in shared memory
  static constexpr int kLoads = kTile * kRow / kScanThreads;
  static_assert(kTile * kRow % kScanThreads == 0, "whole loads");

  const SsmArgs& a;
  float* smem;  // [2][kTile][kRow]
  int64_t c;    // channel
  int lane4, group;
  bool live;
  float bias, skip;
  State<S> st;
  float sum_dt = 0.f;
  float nx[kBatches], ndt[kBatches], nz[kBatches], nbc[kLoads];  // the next tile

  __device__ __forceinline__ void fetch(int64_t t, int64_t t1) {
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      const int64_t own = t + kLanes * b + lane4;
      const bool in = live && own < t1;
      nx[b] = element<T>(a.x, own, a.ld_x, c, in, a);
      ndt[b] = element<T>(a.dt, own, a.ld_dt, c, in, a);
      if (!SUMMARY) nz[b] = a.z ? element<T>(a.z, own, a.ld_z, c, in, a) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = i * kScanThreads + threadIdx.x, s = e % kRow;
      const int64_t own = t + e / kRow;
      const bool is_b = SUMMARY || s < S;
      const int64_t ld = is_b ? a.ld_b : a.ld_c;
      const int64_t at = own * ld + static_cast<int64_t>(group) * S + (is_b ? s : s - S);
      const T* p = static_cast<const T*>(is_b ? a.B : a.C);
      nbc[i] = own < t1 && kda_guard(at, 1, (a.T - 1) * ld + static_cast<int64_t>(a.groups) * S, a.err)
                   ? to_f32(p[at]) : 0.f;
    }
  }

  // Tokens [t, t1) of one sequence, st carried along.  Called by every thread
  // of the block with the same t, t1.
  __device__ __forceinline__ void run(int64_t t, int64_t t1) {
    fetch(t, t1);
    __syncthreads();  // the buffers' last readers (of an earlier piece) are done
    for (int buf = 0; t < t1; t += kTile, buf ^= 1) {
      float* rows = smem + buf * kTile * kRow;
      float x[kBatches], dt[kBatches], z[kBatches];
#pragma unroll
      for (int b = 0; b < kBatches; ++b) {
        x[b] = nx[b];
        dt[b] = ndt[b] + bias;
        if (!SUMMARY) z[b] = nz[b];
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) rows[i * kScanThreads + threadIdx.x] = nbc[i];
      // Two buffers: a tile's rows are overwritten two tiles later, after the
      // barrier between.
      __syncthreads();
      if (t + kTile < t1) fetch(t + kTile, t1);
      const int n = static_cast<int>(min(t1 - t, static_cast<int64_t>(kTile)));
#pragma unroll
      for (int b = 0; b < kBatches; ++b) {
        const int left = n - kLanes * b;  // tokens of this batch that exist
        if (left <= 0) break;
        if (a.softplus) dt[b] = softplus(dt[b]);
        const float u = dt[b] * x[b];
        if (SUMMARY && lane4 < left) sum_dt += dt[b];
        float part[kLanes];
#pragma unroll
        for (int j = 0; j < kLanes; ++j) {
          const float dj = __shfl_sync(0xffffffffu, dt[b], j, kLanes);
          const float uj = __shfl_sync(0xffffffffu, u, j, kLanes);
          part[j] = 0.f;
          if (j < left) {
            const float* row = rows + (kLanes * b + j) * kRow;
            st.step(dj, uj, row, lane4);
            if (!SUMMARY) part[j] = st.read(row + S, lane4);
          }
        }
        if (!SUMMARY) {
          float y = fmaf(skip, x[b], sum_to_own(part, lane4));
          if (a.z) y *= silu(z[b]);
          const int64_t own = t + kLanes * b + lane4, e = own * a.ld_y + c;
          if (live && lane4 < left && kda_guard(e, 1, (a.T - 1) * a.ld_y + a.dim, a.err))
            static_cast<T*>(a.y)[e] = from_f32<T>(y);
        }
      }
    }
  }
};

// Blocks, channel block fastest: each one chunk of the packed axis and up to 32
// channels of one group.
template <typename T, int S, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads) ssm_scan_kernel(SsmArgs a, int n_cb, int cb_per_group) {
  using K = Scan<T, S, SUMMARY>;
  __shared__ __align__(16) float smem[2 * K::kTile * K::kRow];
  const int cb = blockIdx.x % n_cb;
  const int64_t chunk = blockIdx.x / n_cb;
  if (!SUMMARY && blockIdx.x == 0 && a.cu)
    check_cu_seqlens(a.cu, a.N, a.T, threadIdx.x, kScanThreads, a.err);
  const int per_group = a.dim / a.groups;
  const int in_group = (cb % cb_per_group) * kScanChannels + threadIdx.x / kLanes;
  K k{a, smem};
  k.lane4 = threadIdx.x % kLanes;
  k.group = cb / cb_per_group;
  k.live = in_group < per_group;
  k.c = static_cast<int64_t>(k.group) * per_group + in_group;
  k.st.load_rates(a.A, k.c, a.dim, k.lane4, k.live, a.err);
  k.bias = a.dt_bias && k.live && kda_guard(k.c, 1, a.dim, a.err) ? a.dt_bias[k.c] : 0.f;
  k.skip = a.D && k.live && kda_guard(k.c, 1, a.dim, a.err) ? a.D[k.c] : 0.f;
  const int64_t rows = static_cast<int64_t>(a.N) * a.dim;     // of h0 and h_out
  const int64_t chunk_rows = a.n_chunks * a.dim;
  int64_t t = chunk * a.chunk;
  const int64_t t_end = min(t + a.chunk, a.T);
  int64_t start, end;

  if (SUMMARY) {
    // the sequence that goes on past this chunk, from its first token in here
    const int32_t n = a.cu ? sequence_of(a.cu, a.N, t_end, a.err)
                           : static_cast<int32_t>(t_end / (a.T / a.N));
    sequence_span(a.cu, a.N, a.T, n, start, end, a.err);
    if (start >= t_end) return;
    if (start >= t) k.st.load(a.h0, n * static_cast<int64_t>(a.dim) + k.c, rows, k.lane4, k.live, a.err);
    else k.st.zero();
    k.run(max(t, start), t_end);
    k.st.store(a.chunk_h, chunk * a.dim + k.c, chunk_rows, k.lane4, k.live, a.err);
    float sum = k.sum_dt + __shfl_xor_sync(0xffffffffu, k.sum_dt, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (k.live && k.lane4 == 0 && kda_guard(chunk * a.dim + k.c, 1, chunk_rows, a.err))
      a.chunk_dt[chunk * a.dim + k.c] = sum;
    return;
  }

  // sequences that end in (t, t_end] are finished here, the first chunk's also at 0
  int32_t n = 0;
  if (chunk > 0) n = a.cu ? sequence_of(a.cu, a.N, t, a.err) : static_cast<int32_t>(t / (a.T / a.N));
  sequence_span(a.cu, a.N, a.T, n, start, end, a.err);
  if (start < t && a.chunk_h) {
    // begun in an earlier chunk: that chunk's final state, carried over those between
    const int64_t first = start / a.chunk;
    k.st.load(a.chunk_h, first * a.dim + k.c, chunk_rows, k.lane4, k.live, a.err);
    for (int64_t i = first + 1; i < chunk; ++i) {
      State<S> local;
      local.load(a.chunk_h, i * a.dim + k.c, chunk_rows, k.lane4, k.live, a.err);
      const float sum = k.live && kda_guard(i * a.dim + k.c, 1, chunk_rows, a.err)
                            ? a.chunk_dt[i * a.dim + k.c] : 0.f;
      const f32x2 dd = pack2(sum, sum);
#pragma unroll
      for (int q = 0; q < 2 * State<S>::kQuads; ++q)
        k.st.h[q] = fma2(ex2_2(mul2(dd, k.st.a[q])), k.st.h[q], local.h[q]);
    }
  } else {
    k.st.load(a.h0, n * static_cast<int64_t>(a.dim) + k.c, rows, k.lane4, k.live, a.err);
  }
  while (true) {
    const int64_t stop = min(end, t_end);
    if (t < stop) {
      k.run(t, stop);
      t = stop;
    }
    if (end > t_end) return;  // goes on in the next chunk
    if (a.h_out)
      k.st.store(a.h_out, n * static_cast<int64_t>(a.dim) + k.c, rows, k.lane4, k.live, a.err);
    if (++n >= a.N) return;
    sequence_span(a.cu, a.N, a.T, n, start, end, a.err);
    if (start >= t_end && end > t_end) return;  // begins in the next chunk
    k.st.load(a.h0, n * static_cast<int64_t>(a.dim) + k.c, rows, k.lane4, k.live, a.err);
  }
}

// One token of each sequence, h in place.  S / 4 lanes per channel, four
// values each, so that the states are read and written in whole rows; bound by
// those bytes.
template <typename T, int S>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmArgs a) {
  constexpr int kPer = S / 4;  // lanes per channel
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t units = static_cast<int64_t>(a.N) * a.dim;
  const bool live = i / kPer < units;
  const int64_t unit = live ? i / kPer : units - 1;  // (sequence, channel)
  const int lane = static_cast<int>(i % kPer);
  const int64_t n = unit / a.dim, c = unit % a.dim;
  const int64_t g = c / (a.dim / a.groups);
  const int64_t states = units * S, at = unit * S + 4 * lane;
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
  if (kda_guard(at, 4, states, a.err)) h = *reinterpret_cast<const float4*>(a.h0 + at);
  float A[4], B[4], C[4];
  const int64_t gs = static_cast<int64_t>(a.groups) * S;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t s = 4 * lane + j;
    A[j] = kda_guard(c * S + s, 1, static_cast<int64_t>(a.dim) * S, a.err) ? a.A[c * S + s] : 0.f;
    B[j] = kda_guard(n * a.ld_b + g * S + s, 1, (a.N - 1) * a.ld_b + gs, a.err)
               ? to_f32(static_cast<const T*>(a.B)[n * a.ld_b + g * S + s]) : 0.f;
    C[j] = kda_guard(n * a.ld_c + g * S + s, 1, (a.N - 1) * a.ld_c + gs, a.err)
               ? to_f32(static_cast<const T*>(a.C)[n * a.ld_c + g * S + s]) : 0.f;
  }
  const float x = element<T>(a.x, n, a.ld_x, c, true, a);
  float dt = element<T>(a.dt, n, a.ld_dt, c, true, a);
  if (a.dt_bias && kda_guard(c, 1, a.dim, a.err)) dt += a.dt_bias[c];
  if (a.softplus) dt = softplus(dt);
  const float u = dt * x;
  h.x = fmaf(ex2(dt * (A[0] * kLog2e)), h.x, u * B[0]);
  h.y = fmaf(ex2(dt * (A[1] * kLog2e)), h.y, u * B[1]);
  h.z = fmaf(ex2(dt * (A[2] * kLog2e)), h.z, u * B[2]);
  h.w = fmaf(ex2(dt * (A[3] * kLog2e)), h.w, u * B[3]);
  if (live && kda_guard(at, 4, states, a.err)) *reinterpret_cast<float4*>(a.h_out + at) = h;
  float y = fmaf(h.x, C[0], h.y * C[1]) + fmaf(h.z, C[2], h.w * C[3]);
#pragma unroll
  for (int o = kPer / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (live && lane == 0) {
    if (a.D && kda_guard(c, 1, a.dim, a.err)) y = fmaf(a.D[c], x, y);
    if (a.z) y *= silu(element<T>(a.z, n, a.ld_z, c, true, a));
    const int64_t e = n * a.ld_y + c;
    if (kda_guard(e, 1, (a.N - 1) * a.ld_y + a.dim, a.err)) static_cast<T*>(a.y)[e] = from_f32<T>(y);
  }
}

struct Blocks {
  int per_group, n_cb;
};
Blocks channel_blocks(const SsmArgs& a) {
  const int per = (a.dim / a.groups + kScanChannels - 1) / kScanChannels;
  return Blocks{per, per * a.groups};
}

template <typename T, int S>
cudaError_t run_scan(const SsmArgs& a, bool cut, cudaStream_t s) {
  const Blocks b = channel_blocks(a);
  if (a.n_chunks * b.n_cb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (cut) {
    prof_begin(s, "kda_ssm_summary");
    ssm_scan_kernel<T, S, true><<<static_cast<unsigned>((a.n_chunks - 1) * b.n_cb), kScanThreads, 0, s>>>(
        a, b.n_cb, b.per_group);
    prof_end(s, "kda_ssm_summary");
  }
  prof_begin(s, "kda_ssm_scan");
  ssm_scan_kernel<T, S, false><<<static_cast<unsigned>(a.n_chunks * b.n_cb), kScanThreads, 0, s>>>(
      a, b.n_cb, b.per_group);
  prof_end(s, "kda_ssm_scan");
  return cudaGetLastError();
}

template <typename T, int S>
cudaError_t run_step(const SsmArgs& a, cudaStream_t s) {
  const int64_t threads = static_cast<int64_t>(a.N) * a.dim * (S / 4);
  const int64_t blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  ssm_step_kernel<T, S><<<static_cast<unsigned>(blocks), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_of(const SsmArgs& a, bool cut, cudaStream_t s) {
  switch (a.state) {
    case 16: return run_scan<T, 16>(a, cut, s);
    case 32: return run_scan<T, 32>(a, cut, s);
    case 64: return run_scan<T, 64>(a, cut, s);
    case 128: return run_scan<T, 128>(a, cut, s);
  }
  return cudaErrorInvalidValue;
}
template <typename T>
cudaError_t step_of(const SsmArgs& a, cudaStream_t s) {
  switch (a.state) {
    case 16: return run_step<T, 16>(a, s);
    case 32: return run_step<T, 32>(a, s);
    case 64: return run_step<T, 64>(a, s);
    case 128: return run_step<T, 128>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

void ssm_chunks(SsmArgs& a, bool& cut) {
  // A block of 4 warps walks its chunk's tokens one after another; about four
  // such blocks per SM keep its issue slots busy.  Cutting sequences costs the
  // first launch, about 3/4 of the second, for the cut pieces.
  const int64_t n_cb = channel_blocks(a).n_cb, slots = 4LL * a.sm_count;
  cut = false;
  a.n_chunks = 1;
  a.chunk = std::max<int64_t>(a.T, 1);
  if (a.T == 0) return;
  if (!a.cu) {
    // whole sequences: one launch, N n_cb blocks of T / N tokens
    const int64_t len = a.T / a.N;
    if (7 * a.N * n_cb >= 4 * slots || len <= 64) {
      a.chunk = len;
      a.n_chunks = a.N;
      return;
    }
  }
  const int64_t wanted = std::max<int64_t>(1, (slots + n_cb - 1) / n_cb);
  int64_t chunk = (a.T + wanted - 1) / wanted;
  chunk = std::max<int64_t>(64, (chunk + 15) / 16 * 16);
  if (chunk >= a.T) return;
  a.chunk = chunk;
  a.n_chunks = (a.T + chunk - 1) / chunk;
  cut = true;
}

cudaError_t launch_ssm_scan(const SsmArgs& a, bool cut, cudaStream_t s) {
  return a.bf16 ? scan_of<Bf16>(a, cut, s) : scan_of<float>(a, cut, s);
}

cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_ssm_scan_step");
  const cudaError_t e = a.bf16 ? step_of<Bf16>(a, s) : step_of<float>(a, s);
  prof_end(s, "kda_ssm_scan_step");
  return e;
}

}  // namespace kda
