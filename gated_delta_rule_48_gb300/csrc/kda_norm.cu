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
// registers between its sum of squares and its scaling.  A warp takes 256
// columns at a time, 8 to a lane, so a group of 128 columns lies in half a
// warp (16-byte loads of consecutive columns) or, where rows do not start on
// 16-byte boundaries, in four of each lane's eight elements (one element per
// lane and load, consecutive lanes on consecutive columns); either way the
// group's maximum needs only shuffles.
//
// 16384 x 4096 bf16 rows with a residual to e4m3: 94 us, 5.0 TB/s; 1777 x 2051
// 32-bit rows (no two of them aligned alike): 12 us, 4.1 TB/s; one row of
// 4096: 2.1 us.
#include <cuda_runtime.h>

#include "kda_ops.h"

namespace kda {

namespace {

// A lane's 8 columns of the 256 that start at `base`.
template <bool VEC>
__device__ __forceinline__ int column_of(int base, int lane, int i) {
  return VEC ? base + 8 * lane + i : base + 128 * (i >> 2) + 32 * (i & 3) + lane;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_cols(const T* row, int64_t row_off, int64_t extent, int base,
                                          int lane, int dim, float (&v)[8], int* err) {
  if (VEC) {
    const int c = base + 8 * lane;
    if (c < dim && kda_guard(row_off + c, 8, extent, err)) {
      load8(row + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column_of<VEC>(base, lane, i);
      v[i] = c < dim && kda_guard(row_off + c, 1, extent, err) ? to_f32(row[c]) : 0.f;
    }
  }
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
// rows per block); several rows share a block only when a row is one warp.
template <typename T, typename W, bool QUANT, bool VEC, int NV>
__global__ void __launch_bounds__(1024)
norm_kernel(NormArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole rows leave: only blocks of one-warp rows have a remainder
  const int dim = a.dim;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* res = static_cast<const T*>(a.residual) + row * a.ld_res;
  const W* w = static_cast<const W*>(a.weight);

  float h[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    load_cols<VEC>(x, row * a.ld_x, (a.rows - 1) * a.ld_x + dim, 256 * (i * n_warps + warp), lane,
                   dim, h[i], a.err);
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[8];
      load_cols<VEC>(res, row * a.ld_res, (a.rows - 1) * a.ld_res + dim,
                     256 * (i * n_warps + warp), lane, dim, r, a.err);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += r[j];
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
    __shared__ float s_part[32];
    if (lane == 0) s_part[warp] = ss;
    __syncthreads();
    ss = lane < n_warps ? s_part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(dim) + a.eps);

#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int base = 256 * (i * n_warps + warp);
    if (base >= dim) break;
    float wv[8], y[8];
    load_cols<VEC>(w, 0, dim, base, lane, dim, wv, a.err);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[i][j] * inv * wv[j];
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

template <typename T, typename W, bool QUANT, bool VEC, int NV>
void launch_nv(const NormArgs& a, int warps, cudaStream_t s) {
  const int rows_per_block = warps == 1 ? 4 : 1;
  const dim3 block(32 * warps, rows_per_block);
  const int64_t blocks = (a.rows + rows_per_block - 1) / rows_per_block;
  norm_kernel<T, W, QUANT, VEC, NV><<<static_cast<unsigned>(blocks), block, 0, s>>>(a);
}

template <typename T, typename W, bool QUANT, bool VEC>
void launch_vec(const NormArgs& a, cudaStream_t s) {
  // Pieces of 256 columns, shared out over the row's warps: one each while that
  // is at most 32 warps, so that a row's loads are all in flight at once (two
  // pieces a warp: the same at 16384 x 4096, 9 % slower at 1777 x 2051).
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
