// Short causal convolution per channel over packed sequences, and its step for
// one token of each sequence.
//
//   y[t, d] = act(bias[d] + sum_j w[d, j] x[t - W + 1 + j, d]),  act = SiLU or none
//
// Before a sequence's first token stand the W - 1 rows of its state (the last
// inputs of an earlier call), or zeros; its last W - 1 rows, those of the
// state among them when it is shorter, are its state afterwards.
//
// Bound: HBM, x read once and y written once.  A thread owns a vector of
// channels and walks down a strip of tokens with the last W - 1 rows in
// registers, so a row is loaded once per strip; only the W - 1 rows above a
// strip are read again (from L2).  The sums are in 32 bits.  The next batch of
// rows is loaded while one is computed, and kept as loaded until its turn;
// eight rows a batch keep enough bytes in flight (four: 16 % slower).
//
// 16384 x 12288 bf16, width 4, SiLU: 133 us, 6.1 TB/s.  Channels that can only
// be read two at a time (2050 of them) are bound by instructions: 20,011 rows
// 39 us, 4.2 TB/s.  The step for 256 x 12288: 9.2 us, 5.5 TB/s.
#include <cuda_runtime.h>

#include "kda_ops.h"

namespace kda {

namespace {

constexpr int kConvThreads = 128;
constexpr int kConvBatch = 8;  // rows whose loads are issued together, a batch ahead

template <typename T, int VEC, int W>
struct Taps {
  float w[VEC][W], bias[VEC];

  __device__ __forceinline__ void load(const ConvArgs& a, int c0) {
    const int64_t n = static_cast<int64_t>(a.dim) * W;
    auto any = [&](const void* p, int64_t i) {
      return a.w_bf16 ? to_f32(static_cast<const Bf16*>(p)[i]) : static_cast<const float*>(p)[i];
    };
    if (VEC > 1 && a.w_bf16 == (sizeof(T) == 2)) {  // W vectors of VEC weights
      const T* p = static_cast<const T*>(a.weight) + static_cast<int64_t>(c0) * W;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float v[VEC];
        if (kda_guard(static_cast<int64_t>(c0) * W + VEC * j, VEC, n, a.err)) load_n<VEC>(p + VEC * j, v);
        else for (int i = 0; i < VEC; ++i) v[i] = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[(VEC * j + i) / W][(VEC * j + i) % W] = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int64_t e = (static_cast<int64_t>(c0) + i) * W + j;
          w[i][j] = kda_guard(e, 1, n, a.err) ? any(a.weight, e) : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      bias[i] = a.bias && kda_guard(c0 + i, 1, a.dim, a.err) ? any(a.bias, c0 + i) : 0.f;
  }

  // rows: the W rows that end at the token, oldest first
  __device__ __forceinline__ float at(int i, const float (&rows)[W][VEC], bool act) const {
    float v = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) v = fmaf(w[i][j], rows[j][i], v);
    return act ? silu(v) : v;
  }
};

// The row `back` rows before the start of sequence n (back = 1 .. W - 1).
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_before(const ConvArgs& a, int32_t n, int back, int c0,
                                            float (&v)[VEC]) {
  const int64_t e = (static_cast<int64_t>(n) * (W - 1) + (W - 1 - back)) * a.dim + c0;
  if (a.state_in && kda_guard(e, VEC, static_cast<int64_t>(a.N) * (W - 1) * a.dim, a.err)) {
    load_n<VEC>(static_cast<const T*>(a.state_in) + e, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_x(const ConvArgs& a, int64_t t, int c0, float (&v)[VEC]) {
  const int64_t e = t * a.ld_x + c0;
  if (kda_guard(e, VEC, (a.T - 1) * a.ld_x + a.dim, a.err)) {
    load_n<VEC>(static_cast<const T*>(a.x) + e, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_y(const ConvArgs& a, int64_t t, int c0, const float (&v)[VEC]) {
  const int64_t e = t * a.ld_y + c0;
  if (kda_guard(e, VEC, (a.T - 1) * a.ld_y + a.dim, a.err)) store_n<VEC>(static_cast<T*>(a.y) + e, v);
}

// One strip of tokens, for this thread's channels.
template <typename T, int VEC, int W>
__device__ __forceinline__ void conv_strip(const ConvArgs& a, const int64_t t0, int64_t t_end, int c0) {
  int64_t t = t0;
  Taps<T, VEC, W> taps;
  taps.load(a, c0);
  int32_t n = a.cu ? sequence_of(a.cu, a.N, t, a.err) : static_cast<int32_t>(t / (a.T / a.N));
  int64_t start, end;
  sequence_span(a.cu, a.N, a.T, n, start, end, a.err);
  float rows[W][VEC];  // rows[0 .. W - 2]: the rows before token t
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t pos = t - (W - 1) + j;
    if (pos >= start) load_x<T, VEC>(a, pos, c0, rows[j]);
    else load_before<T, VEC, W>(a, n, static_cast<int>(min(start - pos, int64_t{W - 1})), c0, rows[j]);
  }
  auto token = [&](T* to, const float (&x)[VEC]) {
    float y[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      rows[W - 1][i] = x[i];
      y[i] = taps.at(i, rows, a.silu);
    }
    if (kda_guard(to - static_cast<T*>(a.y), VEC, (a.T - 1) * a.ld_y + a.dim, a.err)) store_n<VEC>(to, y);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) rows[j][i] = rows[j + 1][i];
  };
  while (true) {
    const int64_t stop = min(end, t_end);
    // Whole batches, a batch's loads ahead; their rows' places by addition.
    RawVec<T, VEC> next[kConvBatch];
    const T* px = static_cast<const T*>(a.x) + t * a.ld_x + c0;
    T* py = static_cast<T*>(a.y) + t * a.ld_y + c0;
    auto fetch = [&]() {
#pragma unroll
      for (int b = 0; b < kConvBatch; ++b, px += a.ld_x)
        if (kda_guard(px - static_cast<const T*>(a.x), VEC, (a.T - 1) * a.ld_x + a.dim, a.err))
          next[b].load(px);
    };
    if (t + kConvBatch <= stop) fetch();
    for (; t + kConvBatch <= stop; t += kConvBatch) {
      RawVec<T, VEC> now[kConvBatch];
#pragma unroll
      for (int b = 0; b < kConvBatch; ++b) now[b] = next[b];
      if (t + 2 * kConvBatch <= stop) fetch();
#pragma unroll
      for (int b = 0; b < kConvBatch; ++b, py += a.ld_y) {
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = now[b].get(i);
        token(py, x);
      }
    }
    for (; t < stop; ++t, px += a.ld_x, py += a.ld_y) {
      float x[VEC] = {};
      if (kda_guard(px - static_cast<const T*>(a.x), VEC, (a.T - 1) * a.ld_x + a.dim, a.err))
        load_n<VEC>(px, x);
      token(py, x);
    }
    if (stop >= t_end) return;
    t = max(stop, t0);
    do {  // the next sequence that has tokens
      if (++n >= a.N) return;
      sequence_span(a.cu, a.N, a.T, n, start, end, a.err);
    } while (end <= t);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_before<T, VEC, W>(a, n, W - 1 - j, c0, rows[j]);
  }
}

// The state of sequence n after its tokens.
template <typename T, int VEC, int W>
__device__ __forceinline__ void conv_state(const ConvArgs& a, int32_t n, int c0) {
  int64_t start, end;
  sequence_span(a.cu, a.N, a.T, n, start, end, a.err);
  float rows[W][VEC];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t pos = end - (W - 1) + j;
    if (pos >= start) load_x<T, VEC>(a, pos, c0, rows[j]);
    else load_before<T, VEC, W>(a, n, static_cast<int>(start - pos), c0, rows[j]);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t e = (static_cast<int64_t>(n) * (W - 1) + j) * a.dim + c0;
    if (kda_guard(e, VEC, static_cast<int64_t>(a.N) * (W - 1) * a.dim, a.err))
      store_n<VEC>(static_cast<T*>(a.state_out) + e, rows[j]);
  }
}

// Blocks, channel block fastest: first the strips, then one row of blocks per
// sequence for its state.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads)
conv_kernel(ConvArgs a, int strip, int64_t n_strips, int n_cb) {
  const int cb = blockIdx.x % n_cb;
  const int64_t unit = blockIdx.x / n_cb;
  if (blockIdx.x == 0 && a.cu)
    check_cu_seqlens(a.cu, a.N, a.T, threadIdx.x, blockDim.x, a.err);
  const int c0 = (cb * blockDim.x + threadIdx.x) * VEC;
  if (c0 >= a.dim) return;
  if (unit < n_strips) {
    const int64_t t = unit * strip;
    conv_strip<T, VEC, W>(a, t, min(t + strip, a.T), c0);
  } else {
    conv_state<T, VEC, W>(a, static_cast<int32_t>(unit - n_strips), c0);
  }
}

// One token of each sequence; the state moves up by a row, in place.  A thread
// keeps its channels' weights and goes over sequences.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs a, int n_cb, int n_groups) {
  const int cb = blockIdx.x % n_cb;
  const int c0 = (cb * blockDim.x + threadIdx.x) * VEC;
  if (c0 >= a.dim) return;
  Taps<T, VEC, W> taps;
  taps.load(a, c0);
  for (int64_t n = blockIdx.x / n_cb; n < a.N; n += n_groups) {
    float rows[W][VEC], y[VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_before<T, VEC, W>(a, static_cast<int32_t>(n), W - 1 - j, c0, rows[j]);
    load_x<T, VEC>(a, n, c0, rows[W - 1]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = taps.at(i, rows, a.silu);
    store_y<T, VEC>(a, n, c0, y);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t e = (n * (W - 1) + j) * a.dim + c0;
      if (kda_guard(e, VEC, static_cast<int64_t>(a.N) * (W - 1) * a.dim, a.err))
        store_n<VEC>(static_cast<T*>(a.state_out) + e, rows[j + 1]);
    }
  }
}

template <typename T, int VEC, int W>
cudaError_t run(const ConvArgs& a, bool step, cudaStream_t s) {
  const int vecs = (a.dim + VEC - 1) / VEC;
  const int threads = vecs >= kConvThreads ? kConvThreads : (vecs + 31) / 32 * 32;
  const int n_cb = (vecs + threads - 1) / threads;
  // blocks that keep every SM's loads in flight (8 of 128 threads at a time)
  const int64_t wanted = 8LL * a.sm_count * kConvThreads / threads;
  if (step) {
    const int64_t groups = a.N * static_cast<int64_t>(n_cb) <= wanted ? a.N : (wanted + n_cb - 1) / n_cb;
    if (groups * n_cb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    conv_step_kernel<T, VEC, W><<<static_cast<unsigned>(groups * n_cb), threads, 0, s>>>(
        a, n_cb, static_cast<int>(groups));
    return cudaGetLastError();
  }
  int strip = 64;  // shorter where the GPU would otherwise stand idle
  while (strip > 8 && (a.T + strip - 1) / strip * n_cb < wanted) strip /= 2;
  const int64_t n_strips = (a.T + strip - 1) / strip;
  const int64_t n_states = a.state_out ? a.N : 0;
  if ((n_strips + n_states) * n_cb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto launch = [&](const ConvArgs& b, int64_t strips, int64_t states) {
    const int64_t blocks = (strips + states) * n_cb;
    if (blocks > 0)
      conv_kernel<T, VEC, W><<<static_cast<unsigned>(blocks), threads, 0, s>>>(b, strip, strips, n_cb);
  };
  // In place, the state is written only after every strip has read it.
  if (a.state_out && a.state_out == a.state_in) {
    launch(a, n_strips, 0);
    launch(a, 0, n_states);
  } else {
    launch(a, n_strips, n_states);
  }
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t run_width(const ConvArgs& a, bool step, cudaStream_t s) {
  switch (a.width) {
    case 2: return run<T, VEC, 2>(a, step, s);
    case 3: return run<T, VEC, 3>(a, step, s);
    case 4: return run<T, VEC, 4>(a, step, s);
    case 5: return run<T, VEC, 5>(a, step, s);
    case 6: return run<T, VEC, 6>(a, step, s);
    case 7: return run<T, VEC, 7>(a, step, s);
    case 8: return run<T, VEC, 8>(a, step, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t run_types(const ConvArgs& a, bool step, cudaStream_t s) {
  switch (a.vec) {
    case 4: return a.bf16 ? run_width<Bf16, 4>(a, step, s) : run_width<float, 4>(a, step, s);
    case 2: return a.bf16 ? run_width<Bf16, 2>(a, step, s) : run_width<float, 2>(a, step, s);
  }
  return a.bf16 ? run_width<Bf16, 1>(a, step, s) : run_width<float, 1>(a, step, s);
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_short_conv_fwd");
  const cudaError_t e = run_types(a, false, s);
  prof_end(s, "kda_short_conv_fwd");
  return e;
}

cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_short_conv_step");
  const cudaError_t e = run_types(a, true, s);
  prof_end(s, "kda_short_conv_step");
  return e;
}

}  // namespace kda
