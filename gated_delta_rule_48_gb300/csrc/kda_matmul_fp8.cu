// Product of rows in 8 bits with weights in 8 bits, with a scale for each row
// and 128 columns of A and for each 128 x 128 block of B:
//
//   out[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in block b} A[m, k] B[n, k]
//
// Bound: the tensor cores when there are many rows, the weights' bytes when
// there are few.  A k-block of 128 e4m3 values is one 128-byte swizzled row, so
// it is one tensor copy per operand and four tcgen05 products of depth 32.  Its
// sum starts from zero in tensor memory and is then scaled and added to 32-bit
// sums in registers: the tensor core never adds across blocks of different
// scales.  One warp issues the copies, one the products, eight (or four) scale
// and add, with several buffers of tensor memory between, so that copies,
// products and additions overlap; a block goes over tiles until none is left.
//
// The 128 rows of a tile (tensor memory's lanes) are rows of A, or, with SWAP,
// rows of B, with the rows of A as columns: few rows of A then still fill the
// tensor core's 128 lanes, and a tile reads no more of A than there is.
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>

#include "kda_ops.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

using namespace sm100;

constexpr int kTileRows = 128;
constexpr int kBlockK = 128;

// D (+)= A B, 8-bit operands from shared memory; issued by one thread.
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int32_t c0, int32_t c1,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// Waits for this thread's tensor-memory loads; naming the registers keeps
// their uses behind the wait.
__device__ __forceinline__ void wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

template <int BN, bool SWAP>
struct Shape {
  static constexpr int kGroups = BN >= 32 ? 2 : 1;         // sets of four adding warps
  static constexpr int kCols = BN / kGroups;               // columns of a thread's row
  static constexpr int kWarps = 2 + 4 * kGroups;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kBufs = BN == 256 ? 2 : 4;          // of tensor memory
  static constexpr uint32_t kTmemCols = BN * kBufs < 32 ? 32 : BN * kBufs;
  static constexpr uint32_t kRowBytes = kTileRows * kBlockK, kColBytes = BN * kBlockK;
  static constexpr uint32_t kStageBytes = kRowBytes + kColBytes;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr uint32_t kSmem = kStages * kStageBytes + 1024;  // the tiles start on 1024 bytes
  static_assert(kCols % 16 == 0, "whole loads");
};

struct Maps {
  CUtensorMap rows, cols;  // the operand of a tile's 128 rows, and of its BN columns
};

template <int BN, bool SWAP, typename OutT>
__global__ void __launch_bounds__(Shape<BN, SWAP>::kThreads, 1)
matmul_kernel(const __grid_constant__ Maps maps, MatmulArgs a, int tiles_r, int tiles_c, int band) {
  using G = Shape<BN, SWAP>;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[G::kStages], empty[G::kStages], tfull[G::kBufs], tempty[G::kBufs];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                          ~uintptr_t{1023});
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kblocks = (a.K + kBlockK - 1) / kBlockK;
  const int64_t n_tiles = static_cast<int64_t>(tiles_r) * tiles_c;

  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < G::kBufs; ++i) { mbar_init(&tfull[i], 1); mbar_init(&tempty[i], 4 * G::kGroups); }
    mbar_fence_init();
    s_abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, G::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto timeout = [&]() {
    atomicOr(a.err, kDevErrTimeout);
    s_abort = 1;
  };
  // Tile order: bands of `band` row tiles, down a band's rows first, so that
  // the tiles in flight share few rows and columns (in L2).
  auto tile_at = [&](int64_t t, int& r, int& c) {
    const int64_t per_band = static_cast<int64_t>(band) * tiles_c;
    const int64_t first = t / per_band * band, in = t % per_band;
    const int64_t height = min(static_cast<int64_t>(band), tiles_r - first);
    r = static_cast<int>(first + in % height);
    c = static_cast<int>(in / height);
  };

  if (warp == 0) {
    if (lane == 0) {
      int64_t it = 0;
      for (int64_t t = blockIdx.x; t < n_tiles && !s_abort; t += gridDim.x) {
        int r, c;
        tile_at(t, r, c);
        for (int kb = 0; kb < kblocks && !s_abort; ++kb, ++it) {
          const int st = static_cast<int>(it % G::kStages);
          const uint32_t round = static_cast<uint32_t>(it / G::kStages);
          if (round > 0 && !mbar_wait(&empty[st], (round - 1) & 1)) { timeout(); break; }
          unsigned char* p = tiles + st * G::kStageBytes;
          mbar_arrive_expect_tx(&full[st], G::kStageBytes);
          tma_load_2d(p, &maps.rows, kb * kBlockK, r * kTileRows, &full[st]);
          tma_load_2d(p + G::kRowBytes, &maps.cols, kb * kBlockK, c * BN, &full[st]);
        }
      }
      // after an error: the copies in flight land before the block's memory goes
      if (s_abort)
        for (int64_t i = it < G::kStages ? 0 : it - G::kStages; i < it; ++i)
          mbar_wait(&full[i % G::kStages], static_cast<uint32_t>(i / G::kStages) & 1, 1u << 16);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc(0 /* e4m3 */, kTileRows, BN, false, false);
      int64_t it = 0;
      for (int64_t t = blockIdx.x; t < n_tiles && !s_abort; t += gridDim.x) {
        for (int kb = 0; kb < kblocks && !s_abort; ++kb, ++it) {
          const int st = static_cast<int>(it % G::kStages), buf = static_cast<int>(it % G::kBufs);
          const uint32_t turn = static_cast<uint32_t>(it / G::kBufs);
          if (turn > 0 && !mbar_wait(&tempty[buf], (turn - 1) & 1)) { timeout(); break; }
          if (!mbar_wait(&full[st], static_cast<uint32_t>(it / G::kStages) & 1)) { timeout(); break; }
          tc_fence_after();
          const uint32_t rows = smem_u32(tiles + st * G::kStageBytes), cols = rows + G::kRowBytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_e4m3_ss(tmem + buf * BN, smem_desc_sw128(rows + 32 * kk, 16, 1024),
                        smem_desc_sw128(cols + 32 * kk, 16, 1024), idesc, kk > 0);
          mma_commit(&empty[st]);
          mma_commit(&tfull[buf]);
        }
      }
      // the last products end before tensor memory is freed (the adding warps
      // have waited for them, unless there was an error)
      if (s_abort && it > 0)
        mbar_wait(&tfull[(it - 1) % G::kBufs], static_cast<uint32_t>((it - 1) / G::kBufs) & 1, 1u << 16);
    }
  } else {
    const int quad = warp & 3, group = (warp - 2) >> 2;
    int64_t it = 0;
    for (int64_t t = blockIdx.x; t < n_tiles && !s_abort; t += gridDim.x) {
      int r, c;
      tile_at(t, r, c);
      const int64_t row = static_cast<int64_t>(r) * kTileRows + 32 * quad + lane;
      const int64_t col0 = static_cast<int64_t>(c) * BN + G::kCols * group;
      float acc[G::kCols];
#pragma unroll
      for (int i = 0; i < G::kCols; ++i) acc[i] = 0.f;
      const int64_t n_as = (a.M - 1) * a.ld_as + kblocks;
      const int64_t n_bs = ((a.N + kScaleGroup - 1) / kScaleGroup - 1) * a.ld_bs + kblocks;
      auto scale_a = [&](int64_t m, int kb) {
        return m < a.M && kda_guard(m * a.ld_as + kb, 1, n_as, a.err) ? a.a_scale[m * a.ld_as + kb] : 0.f;
      };
      auto scale_b = [&](int64_t n, int kb) {
        const int64_t e = n / kScaleGroup * a.ld_bs + kb;
        return n < a.N && kda_guard(e, 1, n_bs, a.err) ? a.b_scale[e] : 0.f;
      };
      // the scale of this thread's row, times (not SWAP) that of its columns
      auto scale_of = [&](int kb) {
        return SWAP ? scale_b(static_cast<int64_t>(r) * kTileRows, kb) : scale_a(row, kb) * scale_b(col0, kb);
      };
      float next = scale_of(0);
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const int buf = static_cast<int>(it % G::kBufs);
        const float scale = next;
        if (kb + 1 < kblocks) next = scale_of(kb + 1);
        bool ok = mbar_wait(&tfull[buf], static_cast<uint32_t>(it / G::kBufs) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) timeout();
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem_addr(tmem, 32 * quad, buf * BN + G::kCols * group);
        uint32_t d[2][16];
        tmem_ld16(at, d[0]);
#pragma unroll
        for (int i = 0; i < G::kCols / 16; ++i) {
          wait_ld16(d[i & 1]);
          if (i + 1 < G::kCols / 16) tmem_ld16(at + 16 * (i + 1), d[(i + 1) & 1]);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float s = scale;
            if (SWAP) s *= scale_a(col0 + 16 * i + j, kb);
            acc[16 * i + j] = fmaf(__uint_as_float(d[i & 1][j]), s, acc[16 * i + j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
      }
      if (s_abort) break;
      OutT* out = static_cast<OutT*>(a.out);
      const int64_t extent = (a.M - 1) * a.ld_out + a.N;
      if (SWAP) {  // a thread holds one row of B for some rows of A
#pragma unroll
        for (int i = 0; i < G::kCols; ++i) {
          const int64_t m = col0 + i, e = m * a.ld_out + row;
          if (m < a.M && row < a.N && kda_guard(e, 1, extent, a.err)) out[e] = from_f32<OutT>(acc[i]);
        }
      } else if (row < a.M) {
        const int64_t e = row * a.ld_out + col0;
        const bool wide = (reinterpret_cast<uintptr_t>(out + e) & 15) == 0;
#pragma unroll
        for (int i = 0; i < G::kCols; i += 8) {
          if (wide && col0 + i + 8 <= a.N) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = acc[i + j];
            if (kda_guard(e + i, 8, extent, a.err)) store8(out + e + i, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col0 + i + j < a.N && kda_guard(e + i + j, 1, extent, a.err))
                out[e + i + j] = from_f32<OutT>(acc[i + j]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, G::kTmemCols);
}

// ---- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn find_encode() {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
          cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<EncodeTiledFn>(p);
  return nullptr;
}

// [rows, K] bytes; boxes of 128 bytes x `box` rows, 128-byte swizzle.  Past the
// last row and the last column, zeros (e4m3 0.0) are read.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int64_t ld, uint32_t box) {
  static const EncodeTiledFn fn = find_encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t boxes[2] = {kBlockK, box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool SWAP, typename OutT>
cudaError_t run(const MatmulArgs& a, cudaStream_t s) {
  using G = Shape<BN, SWAP>;
  constexpr auto kern = matmul_kernel<BN, SWAP, OutT>;
  const int64_t rows = SWAP ? a.N : a.M, cols = SWAP ? a.M : a.N;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!make_map(&maps.rows, SWAP ? a.b : a.a, rows, a.K, SWAP ? a.ld_b : a.ld_a, kTileRows) ||
      !make_map(&maps.cols, SWAP ? a.a : a.b, cols, a.K, SWAP ? a.ld_a : a.ld_b, BN))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(G::kSmem));
  if (e != cudaSuccess) return e;
  const int tiles_r = static_cast<int>((rows + kTileRows - 1) / kTileRows);
  const int tiles_c = static_cast<int>((cols + BN - 1) / BN);
  const int64_t n = static_cast<int64_t>(tiles_r) * tiles_c;
  const int band = 12;  // of 152 tiles in flight, 12 x 12.7
  kern<<<static_cast<unsigned>(std::min<int64_t>(n, a.sm_count)), G::kThreads, G::kSmem, s>>>(
      maps, a, tiles_r, tiles_c, band);
  return cudaGetLastError();
}

template <typename OutT>
cudaError_t choose(const MatmulArgs& a, cudaStream_t s) {
  if (a.M <= 16) return run<16, true, OutT>(a, s);
  if (a.M <= 32) return run<32, true, OutT>(a, s);
  if (a.M <= 64) return run<64, true, OutT>(a, s);
  const int64_t row_tiles = (a.M + kTileRows - 1) / kTileRows;
  // the widest tile of which there are enough for every SM
  if (row_tiles * ((a.N + 255) / 256) >= a.sm_count) return run<256, false, OutT>(a, s);
  if (row_tiles * ((a.N + 127) / 128) >= a.sm_count) return run<128, false, OutT>(a, s);
  return run<64, false, OutT>(a, s);
}

}  // namespace

cudaError_t launch_matmul_fp8(const MatmulArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_matmul_fp8");
  const cudaError_t e = a.bf16 ? choose<Bf16>(a, s) : choose<float>(a, s);
  prof_end(s, "kda_matmul_fp8");
  return e;
}

}  // namespace kda
