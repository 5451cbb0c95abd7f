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
// Floor: per token, channel and state value one exponential and four multiply-
// adds (against 8 bytes per token and channel).  What holds it above is that
// few warps hide each other's latencies: with 164 registers a thread a
// scheduler has two or three, and issues in 43 to 62 % of its cycles, no pipe
// above 66 %.  Where whole sequences make 256 blocks for 152 SMs, 104 of these
// have two and 48 one.
//
// Four lanes share two neighbouring channels, a quarter of their states each,
// and take a tile of tokens at a time.  What a token needs once (softplus,
// gate, loads, the store) is done by the lane whose number is the token's, and
// (dt', dt' x) handed round through shared memory, so nothing is computed four
// times; B and C are converted once per block, and a lane's read of them serves
// both channels (with one channel per lane the reads bound the kernel, and it
// was 15 % slower).  The recurrence runs on pairs of 32-bit values in one
// instruction (12 % faster than single ones), and a token's decays are computed
// three tokens ahead of its turn.  Three tiles are under way: one in the
// recurrence, one staged beside it, one in flight to registers.
//
// 16,384 tokens x 4096 channels x 16 states, bf16 with gate: 0.42 ms (1.3 TB/s
// of inputs and outputs); the tokens' own work is a third of the instructions.
//
// Prompts are cut into chunks of the packed axis, whatever the sequences'
// lengths, so that blocks are equally long.  A sequence cut by a chunk's end
// maps its state affinely over the chunk, h -> exp(A sum(dt')) h + h_local: a
// first launch computes h_local and sum(dt') of such pieces, and in the second
// each block chains the pieces before its own to its entry state, one after the
// other: in one sequence of 65,536 tokens that is 14 pieces at 2048 channels, but
// up to 454 at 64 (second launch 97 us, the first, the same without the readout,
// 21 us).  Where no sequence is cut there is one launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "kda_ops.h"

namespace kda {

namespace {

constexpr int kLanes = 4;            // lanes per channel, and tokens taken together
constexpr int kScanThreads = 128;
// Channels per lane: each value of B and C read from shared memory serves them
// all.  (At 128 states two channels' states do not fit in registers.)
constexpr int kChannelsOf(int state) { return state <= 64 ? 2 : 1; }
// Blocks per SM that the registers are divided among.
constexpr int scan_blocks_per_sm(int state) { return state <= 16 ? 3 : 2; }

__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(ex2(lo), ex2(hi));
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1].  With
// s = e / (2 + e) <= 1/3, log(1 + e) = 2 artanh(s) = 2 (s + s^3/3 + s^5/5 + ...)
// (Gregory's series); the first term left out, 2 s^15/15, is below 1e-8.
__device__ __forceinline__ float softplus(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  const float s = e * rcp(2.0f + e), q = s * s;
  float p = fmaf(q, 2.0f / 13.0f, 2.0f / 11.0f);
  p = fmaf(q, p, 2.0f / 9.0f);
  p = fmaf(q, p, 2.0f / 7.0f);
  p = fmaf(q, p, 2.0f / 5.0f);
  p = fmaf(q, p, 2.0f / 3.0f);
  return fmaxf(v, 0.0f) + fmaf(s * q, p, s + s);
}

// Four values of B (and of C behind them) from shared memory.
template <bool BOTH>
__device__ __forceinline__ void row_values(const float* p, f32x2* b, f32x2* c) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  b[0] = v.x;
  b[1] = v.y;
  if constexpr (BOTH) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(p + 4);
    c[0] = w.x;
    c[1] = w.y;
  }
}

// The states of a lane's NC channels (c, c + 1, ...).  Value s of a channel is
// in lane (s / 4) % 4, its piece s / 16.
template <int S, int NC>
struct State {
  static constexpr int kPairs = S / (2 * kLanes);  // pairs of values per lane and channel
  f32x2 h[NC][kPairs], a[NC][kPairs];              // the states, and A log2 e

  __device__ __forceinline__ static int64_t at(int lane4, int q) { return 16 * q + 4 * lane4; }

  // `live`: how many of the channels exist
  __device__ __forceinline__ void load_rates(const float* A, int64_t c, int64_t dim, int lane4,
                                             int live, int* err) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < kPairs / 2; ++q) {
        const int64_t e = (c + k) * S + at(lane4, q);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        // (A may be null where there are no tokens)
        if (A && k < live && kda_guard(e, 4, dim * S, err)) v = make_float4(A[e], A[e + 1], A[e + 2], A[e + 3]);
        a[k][2 * q] = pack2(v.x * kLog2e, v.y * kLog2e);
        a[k][2 * q + 1] = pack2(v.z * kLog2e, v.w * kLog2e);
      }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) h[k][i] = 0;
  }
  // row: the first channel's row of a [rows, S] buffer (dense, 16-byte aligned)
  __device__ __forceinline__ void load(const float* p, int64_t row, int64_t rows, int lane4, int live,
                                       int* err) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < kPairs / 2; ++q) {
        const int64_t e = (row + k) * S + at(lane4, q);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p && k < live && kda_guard(e, 4, rows * S, err)) v = *reinterpret_cast<const float4*>(p + e);
        h[k][2 * q] = pack2(v.x, v.y);
        h[k][2 * q + 1] = pack2(v.z, v.w);
      }
  }
  __device__ __forceinline__ void store(float* p, int64_t row, int64_t rows, int lane4, int live,
                                        int* err) const {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < kPairs / 2; ++q) {
        const int64_t e = (row + k) * S + at(lane4, q);
        float4 v;
        unpack2(h[k][2 * q], v.x, v.y);
        unpack2(h[k][2 * q + 1], v.z, v.w);
        if (k < live && kda_guard(e, 4, rows * S, err)) *reinterpret_cast<float4*>(p + e) = v;
      }
  }
  // h = exp(sum A) h + later's h: one chunk's map applied
  __device__ __forceinline__ void chain(const float (&sum)[NC], const State& later) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        h[k][i] = fma2(ex2_2(mul2(pack2(sum[k], sum[k]), a[k][i])), h[k][i], later.h[k][i]);
  }
  // What a token adds to the recurrence, all of it independent of the state:
  // exp(dt A), u B, and the token's C.
  struct Terms {
    f32x2 decay[NC][kPairs], add[NC][kPairs], c[kPairs];
  };
  // row: the token's B and C in shared memory, four of B then four of C for each
  // four state values (without READ, B alone); du: (dt, u) of the lane's channels
  template <typename T, bool READ>
  __device__ __forceinline__ void terms(const T* row, const float* du, int lane4, Terms& t) const {
    float d[NC], u[NC];
    if constexpr (NC == 2) {
      const float4 v = *reinterpret_cast<const float4*>(du);
      d[0] = v.x; u[0] = v.y; d[1] = v.z; u[1] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(du);
      d[0] = v.x; u[0] = v.y;
    }
#pragma unroll
    for (int q = 0; q < kPairs / 2; ++q) {
      f32x2 b[2];
      row_values<READ>(row + (READ ? 2 : 1) * at(lane4, q), b, t.c + 2 * q);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const f32x2 dd = pack2(d[k], d[k]), uu = pack2(u[k], u[k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          t.decay[k][2 * q + i] = ex2_2(mul2(dd, a[k][2 * q + i]));
          t.add[k][2 * q + i] = mul2(uu, b[i]);
        }
      }
    }
  }
  // h = exp(dt A) h + u B; part[k]: this lane's part of sum(h C)
  template <bool READ>
  __device__ __forceinline__ void advance(const Terms& t, float (&part)[NC]) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      f32x2 acc = 0;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        h[k][i] = fma2(t.decay[k][i], h[k][i], t.add[k][i]);
        if (READ) acc = i ? fma2(h[k][i], t.c[i], acc) : mul2(h[k][i], t.c[i]);
      }
      if (READ) {
        float lo, hi;
        unpack2(acc, lo, hi);
        part[k] = lo + hi;
      }
    }
  }
};

// NC consecutive elements in the registers they were loaded into.  Two bf16
// values that came in one load stay in one register until they are used:
// taking them apart would wait for the load.
template <typename T, int NC, bool WIDE>
struct Raw {
  T v[NC];
  __device__ __forceinline__ float get(int k) const { return to_f32(v[k]); }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < NC; ++k) v[k] = p[k];
  }
};
template <>
struct Raw<Bf16, 2, true> {
  uint32_t w;
  __device__ __forceinline__ float get(int k) const {
    return __uint_as_float(k ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ void load(const Bf16* p) { w = *reinterpret_cast<const uint32_t*>(p); }
};
template <>
struct Raw<float, 2, true> {
  float2 w;
  __device__ __forceinline__ float get(int k) const { return k ? w.y : w.x; }
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const float2*>(p); }
};
// N consecutive elements (1, or 4 aligned to their size) on their way from
// global to shared memory.
template <typename T, int N>
struct Four {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(float* p) const { *p = to_f32(v); }
};
template <>
struct Four<Bf16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const Bf16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) =
        make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                    __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
};
template <>
struct Four<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
};
__device__ __forceinline__ void store_pair(Bf16* p, float lo, float hi) {
  *reinterpret_cast<uint32_t*>(p) = pack2_bf16(lo, hi);
}
__device__ __forceinline__ void store_pair(float* p, float lo, float hi) {
  *reinterpret_cast<float2*>(p) = make_float2(lo, hi);
}

// One element of a [T, dim] tensor, or 0 past the end.
template <typename T>
__device__ __forceinline__ float element(const void* p, int64_t t, int64_t ld, int64_t c, bool live,
                                         const SsmArgs& a) {
  const int64_t e = t * ld + c;
  return live && kda_guard(e, 1, (a.T - 1) * ld + a.dim, a.err)
             ? to_f32(static_cast<const T*>(p)[e]) : 0.f;
}

// Sum over the four lanes of a channel, for four tokens at once: lane j ends
// with the sum of token j's parts.
__device__ __forceinline__ float sum_to_own(float v0, float v1, float v2, float v3, int lane4) {
  const bool odd = lane4 & 1, high = lane4 & 2;
  float lo = (odd ? v1 : v0) + __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
  float hi = (odd ? v3 : v2) + __shfl_xor_sync(0xffffffffu, odd ? v2 : v3, 1);
  return (high ? hi : lo) + __shfl_xor_sync(0xffffffffu, high ? lo : hi, 2);
}

// SUMMARY: the piece's final state from zero (or the sequence's start) and its
// sum of step sizes; otherwise outputs and final states.
// WIDE: a lane's channels come in one load.
template <typename T, int S, bool SUMMARY, bool WIDE>
struct Scan {
  static constexpr int NC = kChannelsOf(S);
  static constexpr int kTile = S <= 32 ? 16 : 8;       // tokens per tile
  static constexpr int kBatches = kTile / kLanes;
  static constexpr int kRow = (SUMMARY ? 1 : 2) * S;   // B (and C) of a token in shared memory
  // fetching B and C: `kUnit` values at a time (WIDE: four), units of a tile
  // dealt to the threads
  static constexpr int kUnit = WIDE ? 4 : 1;
  static constexpr int kUnits = kTile * kRow / kUnit;
  static constexpr int kLoads = (kUnits + kScanThreads - 1) / kScanThreads;
  using Unit = Four<T, kUnit>;
  // (dt, u) of the block's channels for a token, in floats; 32 bytes more, so
  // that the four tokens that a channel's lanes write fall in different banks
  static constexpr int kDuRow = 2 * NC * (kScanThreads / kLanes) + 8;
  static constexpr int kBcBytes = kTile * kRow * 4;
  static constexpr int kBufBytes = kBcBytes + kTile * kDuRow * 4;
  using Pair = Raw<T, NC, WIDE>;

  const SsmArgs& a;
  unsigned char* smem;  // two buffers of kTile rows of B and C, then kTile rows of (dt, u)
  int64_t c;    // first channel
  int lane4, group, live;  // live: how many of the lane's channels exist
  float bias[NC], skip[NC], sum_dt[NC];
  State<S, NC> st;
  // the next tile, as loaded (converting here would wait for the loads)
  Pair nx[kBatches], ndt[kBatches], nz[kBatches];
  Unit nbc[kLoads];
  float ny[kBatches][NC], ng[kBatches][NC];  // D x and the gate of the tile staged last
  T* py;                    // this lane's token of the tile
  const T *px, *pdt, *pz;   // of this lane's first token of the next tile
  int64_t t_bc;             // first token of the next tile

  __device__ __forceinline__ Pair get(const T* p, const void* base, int64_t ld, bool in) const {
    Pair r{};
    const int64_t e = p - static_cast<const T*>(base), extent = (a.T - 1) * ld + a.dim;
    if constexpr (WIDE || NC == 1) {
      if (in && live == NC && kda_guard(e, NC, extent, a.err)) r.load(p);
    } else {
#pragma unroll
      for (int k = 0; k < NC; ++k)
        if (in && k < live && kda_guard(e + k, 1, extent, a.err)) r.v[k] = p[k];
    }
    return r;
  }

  // The `n` tokens left from the pointers on, at most a tile of them.
  __device__ __forceinline__ void fetch(int64_t n) {
    const int left = static_cast<int>(min(n, static_cast<int64_t>(kTile)));
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      const bool in = kLanes * b + lane4 < left;
      nx[b] = get(px + b * kLanes * a.ld_x, a.x, a.ld_x, in);
      ndt[b] = get(pdt + b * kLanes * a.ld_dt, a.dt, a.ld_dt, in);
      if (!SUMMARY) nz[b] = get(pz + b * kLanes * a.ld_z, a.z, a.ld_z, in && a.z);
    }
    px += kTile * a.ld_x;
    pdt += kTile * a.ld_dt;
    pz += kTile * a.ld_z;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = (i * kScanThreads + static_cast<int>(threadIdx.x)) * kUnit, row = e / kRow;
      const int s = e % kRow;
      const bool is_b = SUMMARY || s < S;
      const int64_t ld = is_b ? a.ld_b : a.ld_c;
      const int64_t at = (t_bc + row) * ld + static_cast<int64_t>(group) * S + (is_b ? s : s - S);
      Unit v{};
      if (row < left &&
          kda_guard(at, kUnit, (a.T - 1) * ld + static_cast<int64_t>(a.groups) * S, a.err))
        v.load(static_cast<const T*>(is_b ? a.B : a.C) + at);
      nbc[i] = v;
    }
    t_bc += kTile;
  }

  __device__ __forceinline__ void point(int64_t t) {
    px = static_cast<const T*>(a.x) + (t + lane4) * a.ld_x + c;
    pdt = static_cast<const T*>(a.dt) + (t + lane4) * a.ld_dt + c;
    pz = static_cast<const T*>(a.z) + (t + lane4) * a.ld_z + c;
    py = static_cast<T*>(a.y) + (t + lane4) * a.ld_y + c;
    t_bc = t;
  }

  // What the fetched tile's `n` tokens need once: dt and u into shared memory,
  // D x and the gate into registers; B and C into shared memory.
  __device__ __forceinline__ void stage(unsigned char* buf, int n) {
    float* du = reinterpret_cast<float*>(buf + kBcBytes) + 2 * NC * (threadIdx.x / kLanes);
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      float d[NC], u[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        d[k] = ndt[b].get(k) + bias[k];
        if (a.softplus) d[k] = softplus(d[k]);
        const float x = nx[b].get(k);
        u[k] = d[k] * x;
        if (SUMMARY) {
          if (kLanes * b + lane4 < n) sum_dt[k] += d[k];
        } else {
          ny[b][k] = skip[k] * x;
          ng[b][k] = a.z ? silu(nz[b].get(k)) : 1.0f;
        }
      }
      float* to = du + (kLanes * b + lane4) * kDuRow;
      if constexpr (NC == 2) *reinterpret_cast<float4*>(to) = make_float4(d[0], u[0], d[1], u[1]);
      else *reinterpret_cast<float2*>(to) = make_float2(d[0], u[0]);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = (i * kScanThreads + static_cast<int>(threadIdx.x)) * kUnit, s = e % kRow;
      // B's value s at (s / 4) * 8 + s % 4, C's four places behind
      const int at = SUMMARY ? s : s < S ? s / 4 * 8 + s % 4 : (s - S) / 4 * 8 + 4 + s % 4;
      if (kUnits % kScanThreads == 0 || e < kTile * kRow)
        nbc[i].store(reinterpret_cast<float*>(buf) + e / kRow * kRow + at);
    }
  }

  // The recurrence over a staged tile; FULL: all of its tokens exist.
  template <bool FULL>
  __device__ __forceinline__ void tile(const unsigned char* buf, int n, float (&y)[kBatches][NC],
                                       const float (&g)[kBatches][NC]) {
    constexpr int kAhead = S == 16 ? 3 : 1;  // tokens whose decays are ready before their turn
    const float* bc = reinterpret_cast<const float*>(buf);
    const float* du = reinterpret_cast<const float*>(buf + kBcBytes) + 2 * NC * (threadIdx.x / kLanes);
    float part[kTile][NC];
    typename State<S, NC>::Terms terms[kAhead + 1];
    if (FULL) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        st.template terms<float, !SUMMARY>(bc + j * kRow, du + j * kDuRow, lane4, terms[j]);
#pragma unroll
      for (int j = 0; j < kTile; ++j) {
        if (j + kAhead < kTile)
          st.template terms<float, !SUMMARY>(bc + (j + kAhead) * kRow, du + (j + kAhead) * kDuRow, lane4,
                                         terms[(j + kAhead) % (kAhead + 1)]);
        st.template advance<!SUMMARY>(terms[j % (kAhead + 1)], part[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kTile; ++j) {
#pragma unroll
        for (int k = 0; k < NC; ++k) part[j][k] = 0.f;
        if (j < n) {
          st.template terms<float, !SUMMARY>(bc + j * kRow, du + j * kDuRow, lane4, terms[0]);
          st.template advance<!SUMMARY>(terms[0], part[j]);
        }
      }
    }
    if (SUMMARY) return;
#pragma unroll
    for (int b = 0; b < kBatches; ++b)
#pragma unroll
      for (int k = 0; k < NC; ++k)
        y[b][k] = (y[b][k] + sum_to_own(part[4 * b][k], part[4 * b + 1][k], part[4 * b + 2][k],
                                        part[4 * b + 3][k], lane4)) * g[b][k];
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      if (!FULL && kLanes * b + lane4 >= n) break;
      T* p = py + b * kLanes * a.ld_y;
      const int64_t e = p - static_cast<T*>(a.y), extent = (a.T - 1) * a.ld_y + a.dim;
      if constexpr (WIDE && NC == 2) {
        if (live == NC && kda_guard(e, NC, extent, a.err)) store_pair(p, y[b][0], y[b][1]);
      } else {
#pragma unroll
        for (int k = 0; k < NC; ++k)
          if (k < live && kda_guard(e + k, 1, extent, a.err)) p[k] = from_f32<T>(y[b][k]);
      }
    }
    py += kTile * a.ld_y;
  }

  // Tokens [t, t1) of one sequence, st carried along.  Called by every thread
  // of the block with the same t, t1.  Three tiles are under way: one in the
  // recurrence, the next one staged beside it, the one after in flight.
  __device__ __forceinline__ void run(int64_t t, int64_t t1) {
    auto left = [&](int64_t from) { return static_cast<int>(min(t1 - from, static_cast<int64_t>(kTile))); };
    point(t);
    fetch(t1 - t);
    __syncthreads();  // the buffers' last readers (of an earlier piece) are done
    stage(smem, left(t));
    if (t + kTile < t1) fetch(t1 - t - kTile);
    __syncthreads();
    for (int buf = 0; t < t1; t += kTile, buf ^= 1) {
      float y[kBatches][NC], g[kBatches][NC];
#pragma unroll
      for (int b = 0; b < kBatches; ++b)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          y[b][k] = ny[b][k];
          g[b][k] = ng[b][k];
        }
      if (t + kTile < t1) {
        tile<true>(smem + buf * kBufBytes, kTile, y, g);
        stage(smem + (buf ^ 1) * kBufBytes, left(t + kTile));
        if (t + 2 * kTile < t1) fetch(t1 - t - 2 * kTile);
      } else {
        tile<false>(smem + buf * kBufBytes, left(t), y, g);
      }
      __syncthreads();  // the staged buffer is written, the read one is free
    }
  }
};

// Blocks, channel block fastest: each one chunk of the packed axis and up to
// 32 NC channels of one group.
template <typename T, int S, bool SUMMARY, bool WIDE>
__global__ void __launch_bounds__(kScanThreads, scan_blocks_per_sm(S))
ssm_scan_kernel(SsmArgs a, int n_cb, int cb_per_group) {
  using K = Scan<T, S, SUMMARY, WIDE>;
  constexpr int NC = K::NC;
  __shared__ __align__(16) unsigned char smem[2 * K::kBufBytes];
  const int cb = blockIdx.x % n_cb;
  const int64_t chunk = blockIdx.x / n_cb;
  if (!SUMMARY && blockIdx.x == 0 && a.cu)
    check_cu_seqlens(a.cu, a.N, a.T, threadIdx.x, kScanThreads, a.err);
  const int per_group = a.dim / a.groups;
  const int in_group = NC * ((cb % cb_per_group) * (kScanThreads / kLanes) + threadIdx.x / kLanes);
  K k{a, smem};
  k.lane4 = threadIdx.x % kLanes;
  k.group = cb / cb_per_group;
  k.live = min(max(per_group - in_group, 0), NC);
  k.c = static_cast<int64_t>(k.group) * per_group + in_group;
  k.st.load_rates(a.A, k.c, a.dim, k.lane4, k.live, a.err);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const bool in = i < k.live && kda_guard(k.c + i, 1, a.dim, a.err);
    k.bias[i] = a.dt_bias && in ? a.dt_bias[k.c + i] : 0.f;
    k.skip[i] = a.D && in ? a.D[k.c + i] : 0.f;
    k.sum_dt[i] = 0.f;
  }
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
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float sum = k.sum_dt[i] + __shfl_xor_sync(0xffffffffu, k.sum_dt[i], 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int64_t e = chunk * a.dim + k.c + i;
      if (i < k.live && k.lane4 == 0 && kda_guard(e, 1, chunk_rows, a.err)) a.chunk_dt[e] = sum;
    }
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
      State<S, NC> local;
      local.load(a.chunk_h, i * a.dim + k.c, chunk_rows, k.lane4, k.live, a.err);
      float sum[NC];
#pragma unroll
      for (int m = 0; m < NC; ++m) {
        const int64_t e = i * a.dim + k.c + m;
        sum[m] = m < k.live && kda_guard(e, 1, chunk_rows, a.err) ? a.chunk_dt[e] : 0.f;
      }
      k.st.chain(sum, local);
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

// One token of each sequence, h in place.  S / 8 lanes per channel, two groups
// of four values each; bound by the states' bytes: 256 x 4096 x 16 takes 28 us,
// 5.2 TB/s.  (Four values a lane, less in flight and twice the work around
// them: 34 us; two or four sequences to a thread, fewer threads: 38 and 44 us.)
constexpr int kStepThreads = 256;
template <typename T, int S, bool VEC>
__global__ void __launch_bounds__(kStepThreads, 4) ssm_step_kernel(SsmArgs a, int per_group) {
  constexpr int kPer = S / 8;  // lanes per channel; value s is in lane (s / 4) % kPer
  const int lane = threadIdx.x % kPer;
  const int c_own = blockIdx.x * (kStepThreads / kPer) + threadIdx.x / kPer;
  const bool live = c_own < a.dim;
  const int c = live ? c_own : a.dim - 1;  // (whole warps take part in the sums)
  const int g = a.groups == 1 ? 0 : c / per_group;
  const int64_t n = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
  if (n >= a.N) return;  // (the whole block)
  const int64_t states = static_cast<int64_t>(a.N) * a.dim * S, gs = static_cast<int64_t>(a.groups) * S;
  auto load = [&](const auto* p, int64_t e, int64_t extent, float(&v)[4]) {
    if (VEC && kda_guard(e, 4, extent, a.err)) {
      load_n<4>(p + e, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = !VEC && kda_guard(e + j, 1, extent, a.err) ? to_f32(p[e + j]) : 0.f;
    }
  };
  const int64_t at = (n * a.dim + c) * S + 4 * lane;
  float4 h[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    h[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kda_guard(at + 4 * kPer * q, 4, states, a.err))
      h[q] = *reinterpret_cast<const float4*>(a.h0 + at + 4 * kPer * q);
  }
  const float x = element<T>(a.x, n, a.ld_x, c, true, a);
  float dt = element<T>(a.dt, n, a.ld_dt, c, true, a);
  float A[2][4], B[2][4], C[2][4];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int s = 4 * (lane + kPer * q);
    load(a.A, static_cast<int64_t>(c) * S + s, static_cast<int64_t>(a.dim) * S, A[q]);
    load(static_cast<const T*>(a.B), n * a.ld_b + g * S + s, (a.N - 1) * a.ld_b + gs, B[q]);
    load(static_cast<const T*>(a.C), n * a.ld_c + g * S + s, (a.N - 1) * a.ld_c + gs, C[q]);
  }
  const bool in = kda_guard(c, 1, a.dim, a.err);
  if (a.dt_bias && in) dt += a.dt_bias[c];
  if (a.softplus) dt = softplus(dt);
  const float u = dt * x, dl = dt * kLog2e;
  float y = 0.f;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float4& v = h[q];
    v.x = fmaf(ex2(dl * A[q][0]), v.x, u * B[q][0]);
    v.y = fmaf(ex2(dl * A[q][1]), v.y, u * B[q][1]);
    v.z = fmaf(ex2(dl * A[q][2]), v.z, u * B[q][2]);
    v.w = fmaf(ex2(dl * A[q][3]), v.w, u * B[q][3]);
    if (live && kda_guard(at + 4 * kPer * q, 4, states, a.err))
      *reinterpret_cast<float4*>(a.h_out + at + 4 * kPer * q) = v;
    y += fmaf(v.x, C[q][0], v.y * C[q][1]) + fmaf(v.z, C[q][2], v.w * C[q][3]);
  }
#pragma unroll
  for (int o = kPer / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (live && lane == 0) {
    if (a.D && in) y = fmaf(a.D[c], x, y);
    if (a.z) y *= silu(element<T>(a.z, n, a.ld_z, c, true, a));
    const int64_t e = n * a.ld_y + c;
    if (kda_guard(e, 1, (a.N - 1) * a.ld_y + a.dim, a.err)) static_cast<T*>(a.y)[e] = from_f32<T>(y);
  }
}

struct Blocks {
  int per_group, n_cb;
};
Blocks channel_blocks(const SsmArgs& a) {
  const int channels = kScanThreads / kLanes * kChannelsOf(a.state);  // of a block
  const int per = (a.dim / a.groups + channels - 1) / channels;
  return Blocks{per, per * a.groups};
}

template <typename T, int S, bool WIDE>
cudaError_t run_scan(const SsmArgs& a, bool cut, cudaStream_t s) {
  const Blocks b = channel_blocks(a);
  if (a.n_chunks * b.n_cb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (cut) {
    prof_begin(s, "kda_ssm_summary");
    ssm_scan_kernel<T, S, true, WIDE><<<static_cast<unsigned>((a.n_chunks - 1) * b.n_cb), kScanThreads, 0, s>>>(
        a, b.n_cb, b.per_group);
    prof_end(s, "kda_ssm_summary");
  }
  prof_begin(s, "kda_ssm_scan");
  ssm_scan_kernel<T, S, false, WIDE><<<static_cast<unsigned>(a.n_chunks * b.n_cb), kScanThreads, 0, s>>>(
      a, b.n_cb, b.per_group);
  prof_end(s, "kda_ssm_scan");
  return cudaGetLastError();
}

template <typename T, int S>
cudaError_t run_step(const SsmArgs& a, cudaStream_t s) {
  const int64_t blocks_x = (static_cast<int64_t>(a.dim) * (S / 8) + kStepThreads - 1) / kStepThreads;
  const int64_t blocks_y = std::min<int64_t>(a.N, 65535), blocks_z = (a.N + blocks_y - 1) / blocks_y;
  if (blocks_x > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks_x), static_cast<unsigned>(blocks_y),
                  static_cast<unsigned>(blocks_z));
  if (a.vec) ssm_step_kernel<T, S, true><<<grid, kStepThreads, 0, s>>>(a, a.dim / a.groups);
  else ssm_step_kernel<T, S, false><<<grid, kStepThreads, 0, s>>>(a, a.dim / a.groups);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_of(const SsmArgs& a, bool cut, cudaStream_t s) {
  switch (a.state) {
    case 16: return a.pairs ? run_scan<T, 16, true>(a, cut, s) : run_scan<T, 16, false>(a, cut, s);
    case 32: return a.pairs ? run_scan<T, 32, true>(a, cut, s) : run_scan<T, 32, false>(a, cut, s);
    case 64: return a.pairs ? run_scan<T, 64, true>(a, cut, s) : run_scan<T, 64, false>(a, cut, s);
    case 128: return a.pairs ? run_scan<T, 128, true>(a, cut, s) : run_scan<T, 128, false>(a, cut, s);
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
  // Whole sequences take one launch of N n_cb blocks.  Cutting them costs the
  // first launch, about 3/4 of the second, but fills the GPU: worth it below
  // about 1.35 blocks per SM (a second block on some SMs and none on the others
  // already takes as long as two on all).  At 256 blocks (4 sequences of 4096
  // tokens, 4096 channels) whole sequences take 0.42 ms, cut ones 0.57 ms.
  const int64_t n_cb = channel_blocks(a).n_cb;
  cut = false;
  a.n_chunks = 1;
  a.chunk = std::max<int64_t>(a.T, 1);
  if (a.T == 0) return;
  if (!a.cu) {
    const int64_t len = a.T / a.N;
    if (20 * a.N * n_cb >= 27LL * a.sm_count || len <= 64) {
      a.chunk = len;
      a.n_chunks = a.N;
      return;
    }
  }
  // One wave of resident blocks: more chunks only add a partial second wave
  // (65,536 tokens, 2048 channels: 3 blocks per SM 1.14 ms, 4 per SM 1.25 ms).
  const int64_t wanted = std::max<int64_t>(1, scan_blocks_per_sm(a.state) * a.sm_count / n_cb);
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
