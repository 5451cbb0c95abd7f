// The residual's addition and the root-mean-square norm of rows, with the
// output in the input's type or in 8 bits with scales.
//
//   h = x + residual                        (32 bits; stored in x's type)
//   y = h / sqrt(mean(h^2) + eps) * weight
//   8 bits: for each row and each 128 columns g, s_g = max(max |y_g|, 2^-64) / 448
//           and q = e4m3(y * (448 / max |y_g|))
//
// The norm is taken of the 32-bit sum, before h is rounded for storage.
//
// Bound: HBM.  Every element is read once and written once: a row stays in
// registers between its sum of squares and its scaling (above 16,384 columns, 64
// values a thread, partly in local memory).  A warp takes 256
// columns at a time, 8 to a lane, so a group of 128 columns lies in half a
// warp (16-byte loads of consecutive columns) or, where rows do not start on
// 16-byte boundaries, in four of each lane's eight elements (one element per
// lane and load, consecutive lanes on consecutive columns); either way the
// group's maximum needs only shuffles.
//
// 16384 x 4096 bf16 rows with a residual to e4m3: 83 us, 5.7 TB/s (94 us with a
// block for each row, whose loads then wait for nothing but its own end);
// 1777 x 2051 32-bit rows (no two of them aligned alike): 11 us, 4.3 TB/s; one
// row of 4096: 1.9 us.  Above 8192 columns no next row is fetched ahead: 4096 x
// 12288 and 4096 x 32768 bf16 rows with a residual to e4m3 take 92 and 330 us, 3.9
// and 2.9 TB/s.
//
// A value is multiplied by 448 / max rather than divided by the scale: one
// division a group.  Of bf16 rows 8 values in a million then come out one step of
// e4m3 beside the quotient's, those that lie within 1e-7 of the middle between
// two steps; either way the rows are equally far from the unrounded ones.
#include <cuda_runtime.h>

#include <algorithm>

#include "kda_ops.h"

namespace kda {

namespace {

// A lane's 8 columns of the 256 that start at `base`.
template <bool VEC>
__device__ __forceinline__ int column_of(int base, int lane, int i) {
  return VEC ? base + 8 * lane + i : base + 128 * (i >> 2) + 32 * (i & 3) + lane;
}

// A lane's 8 columns as loaded (widening them would wait for the loads).
template <bool VEC, typename T>
struct Cols {
  T v[8];
  __device__ __forceinline__ float get(int i) const { return to_f32(v[i]); }
};
template <>
struct Cols<true, Bf16> {
  uint4 v;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Cols<true, float> {
  float4 a, b;
  __device__ __forceinline__ float get(int i) const {
    const float4 q = i < 4 ? a : b;
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ Cols<VEC, T> load_cols(const T* row, int64_t row_off, int64_t extent,
                                                  int base, int lane, int dim, int* err) {
  Cols<VEC, T> r{};
  if constexpr (VEC) {
    const int c = base + 8 * lane;
    if (c < dim && kda_guard(row_off + c, 8, extent, err)) {
      if constexpr (sizeof(T) == 2) {
        r.v = *reinterpret_cast<const uint4*>(row + c);
      } else {
        r.a = reinterpret_cast<const float4*>(row + c)[0];
        r.b = reinterpret_cast<const float4*>(row + c)[1];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column_of<VEC>(base, lane, i);
      if (c < dim && kda_guard(row_off + c, 1, extent, err)) r.v[i] = row[c];
    }
  }
  return r;
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_cols(T* row, int64_t row_off, int64_t extent, int base,
                                           int lane, int dim, const float (&v)[8], int* err) {
  if (VEC) {
    const int c = base + 8 * lane;
    if (c < dim && kda_guard(row_off + c, 8, extent, err)) store8(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column_of<VEC>(base, lane, i);
      if (c < dim && kda_guard(row_off + c, 1, extent, err)) row[c] = from_f32<T>(v[i]);
    }
  }
}

// NV: 256-column pieces of the row per warp.  blockDim = (32 * warps per row,
// rows per block); several rows share a block only when a row is one warp.  A
// block goes over rows, the next row's loads in flight (with one piece a warp)
// while one is reduced and stored.
template <typename T, typename W, bool QUANT, bool VEC, int NV>
__global__ void __launch_bounds__(1024, 1)
norm_kernel(NormArgs a) {
  constexpr bool kAhead = NV == 1;
  __shared__ float s_part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int dim = a.dim;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  const W* w = static_cast<const W*>(a.weight);
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  auto piece = [&](const T* p, int64_t ld, int64_t row, int i) {
    return load_cols<VEC>(p + row * ld, row * ld, (a.rows - 1) * ld + dim,
                          256 * (i * n_warps + warp), lane, dim, a.err);
  };
  Cols<VEC, T> nx, nr;
  auto fetch = [&](int64_t row) {
    nx = piece(x, a.ld_x, row, 0);
    if (a.residual) nr = piece(res, a.ld_res, row, 0);
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (kAhead && row < a.rows) fetch(row);
  // (rows that share a block are a warp each, which need not stay together)
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    float h[NV][8];
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[0][j] = nx.get(j) + (a.residual ? nr.get(j) : 0.f);
      if (row + step < a.rows) fetch(row + step);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Cols<VEC, T> c = piece(x, a.ld_x, row, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = c.get(j);
      }
      if (a.residual) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const Cols<VEC, T> c = piece(res, a.ld_res, row, i);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += c.get(j);
        }
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    if (a.h) {
      T* ho = static_cast<T*>(a.h) + row * a.ld_h;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        store_cols<VEC>(ho, row * a.ld_h, (a.rows - 1) * a.ld_h + dim, 256 * (i * n_warps + warp),
                        lane, dim, h[i], a.err);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (n_warps > 1) {
      // (two sets of parts: one's readers may still be at it when the next row's
      // are written)
      if (lane == 0) s_part[turn][warp] = ss;
      __syncthreads();
      ss = lane < n_warps ? s_part[turn][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float inv = 1.0f / sqrtf(ss / static_cast<float>(dim) + a.eps);

#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int base = 256 * (i * n_warps + warp);
      if (base >= dim) break;
      const Cols<VEC, W> wv = load_cols<VEC>(w, 0, dim, base, lane, dim, a.err);
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[i][j] * inv * wv.get(j);
      if (!QUANT) {
        store_cols<VEC>(static_cast<T*>(a.y) + row * a.ld_y, row * a.ld_y,
                        (a.rows - 1) * a.ld_y + dim, base, lane, dim, y, a.err);
        continue;
      }
      // two groups of 128 columns: group 0 is lanes 0..15 (VEC) or elements 0..3
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 8; ++j) m[VEC ? 0 : j >> 2] = max_nan(m[VEC ? 0 : j >> 2], fabsf(y[j]));
#pragma unroll
      for (int o = VEC ? 8 : 16; o; o >>= 1) {
        m[0] = max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        if (!VEC) m[1] = max_nan(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
      }
      m[0] = max_nan(m[0], kAmaxMin);
      m[1] = max_nan(m[1], kAmaxMin);
      const int64_t n_groups = (dim + kScaleGroup - 1) / kScaleGroup;
      const int64_t s_off = row * a.ld_scale, s_ext = (a.rows - 1) * a.ld_scale + n_groups;
      const float f0 = kE4m3Max / m[0], f1 = VEC ? 0.f : kE4m3Max / m[1];
      const int g = base / kScaleGroup + (VEC ? lane >> 4 : lane);
      if ((VEC ? (lane & 15) == 0 : lane < 2) && g < n_groups &&
          kda_guard(s_off + g, 1, s_ext, a.err))
        a.y_scale[s_off + g] = ((VEC || lane == 0) ? m[0] : m[1]) / kE4m3Max;
      uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.ld_y;
      const int64_t q_off = row * a.ld_y, q_ext = (a.rows - 1) * a.ld_y + dim;
      if (VEC) {
        const int c = base + 8 * lane;
        uint32_t lo = pack2_e4m3(y[0] * f0, y[1] * f0) |
                      (static_cast<uint32_t>(pack2_e4m3(y[2] * f0, y[3] * f0)) << 16);
        uint32_t hi = pack2_e4m3(y[4] * f0, y[5] * f0) |
                      (static_cast<uint32_t>(pack2_e4m3(y[6] * f0, y[7] * f0)) << 16);
        if (c < dim && kda_guard(q_off + c, 8, q_ext, a.err))
          *reinterpret_cast<uint2*>(q + c) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = column_of<VEC>(base, lane, j);
          if (c < dim && kda_guard(q_off + c, 1, q_ext, a.err))
            q[c] = static_cast<uint8_t>(pack2_e4m3(y[j] * (j < 4 ? f0 : f1), 0.f) & 0xffu);
        }
      }
    }
  }
}

template <typename T, typename W, bool QUANT, bool VEC, int NV>
void launch_nv(const NormArgs& a, int warps, cudaStream_t s) {
  const int rows_per_block = warps == 1 ? 4 : 1;
  const dim3 block(32 * warps, rows_per_block);
  // 1024 threads to an SM: what its registers hold (a second, partial wave cost
  // a fifth)
  const int per_sm = std::max(1, 1024 / (32 * warps * rows_per_block));
  const int64_t blocks = std::min<int64_t>((a.rows + rows_per_block - 1) / rows_per_block,
                                           static_cast<int64_t>(per_sm) * a.sm_count);
  norm_kernel<T, W, QUANT, VEC, NV><<<static_cast<unsigned>(blocks), block, 0, s>>>(a);
}

template <typename T, typename W, bool QUANT, bool VEC>
void launch_vec(const NormArgs& a, cudaStream_t s) {
  // Pieces of 256 columns, shared out over the row's warps: one each while that
  // is at most 32 warps, so that a row's loads are all in flight at once (two
  // pieces a warp were 9 % slower at 1777 x 2051).
  const int pieces = (a.dim + 255) / 256;
  if (pieces <= 32) return launch_nv<T, W, QUANT, VEC, 1>(a, pieces, s);
  if (pieces <= 64) return launch_nv<T, W, QUANT, VEC, 2>(a, (pieces + 1) / 2, s);
  return launch_nv<T, W, QUANT, VEC, 8>(a, (pieces + 7) / 8, s);
}

template <typename T, typename W>
void launch_types(const NormArgs& a, cudaStream_t s) {
  if (a.quant)
    a.vec ? launch_vec<T, W, true, true>(a, s) : launch_vec<T, W, true, false>(a, s);
  else
    a.vec ? launch_vec<T, W, false, true>(a, s) : launch_vec<T, W, false, false>(a, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_add_rms_norm");
  if (a.bf16)
    a.w_bf16 ? launch_types<Bf16, Bf16>(a, s) : launch_types<Bf16, float>(a, s);
  else
    a.w_bf16 ? launch_types<float, Bf16>(a, s) : launch_types<float, float>(a, s);
  prof_end(s, "kda_add_rms_norm");
  return cudaGetLastError();
}

}  // namespace kda
