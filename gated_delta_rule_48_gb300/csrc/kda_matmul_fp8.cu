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

// 32 lanes x 32 consecutive columns of tensor memory: thread i gets lane i of
// its warp's quarter.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's tensor-memory loads; naming the registers keeps
// their uses behind the wait.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               ::"memory");
  // (at most 30 operands that are read and written: the last three in an empty
  // statement, which stays behind the wait)
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// A warp's rows of the output through its own piece of shared memory, 128
// bytes of each of 32 rows at a time, in the layout of a 128-byte-swizzled
// tensor copy.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t c0,
                                             int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
}

template <int BN, bool SWAP>
struct Shape {
  // sets of four adding warps; a thread's columns fill 128 bytes of bf16 (not SWAP)
  static constexpr int kGroups = BN >= (SWAP ? 32 : 128) ? 2 : 1;
  static constexpr int kCols = BN / kGroups;               // columns of a thread's row
  static constexpr int kWarps = 2 + 4 * kGroups;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kBufs = BN == 256 ? 2 : 4;          // of tensor memory
  static constexpr uint32_t kTmemCols = BN * kBufs < 32 ? 32 : BN * kBufs;
  static constexpr uint32_t kRowBytes = kTileRows * kBlockK, kColBytes = BN * kBlockK;
  static constexpr uint32_t kStageBytes = kRowBytes + kColBytes;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  // columns per tensor-memory load (at 128 sums a thread, 32 more do not fit)
  static constexpr int kLoad = kCols % 32 == 0 && kCols < 128 ? 32 : 16;
  static constexpr uint32_t kStoreBytes = SWAP ? 0 : 4 * kGroups * 4096;  // a piece per adding warp
  // the tiles start on 1024 bytes
  static constexpr uint32_t kSmem = kStages * kStageBytes + kStoreBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kCols % 16 == 0, "whole loads");
};

// A place in a ring of N barriers, and the parity of its present phase.
template <int N>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

struct Maps {
  CUtensorMap rows, cols;  // the operand of a tile's 128 rows, and of its BN columns
  CUtensorMap out;         // written 32 rows x 128 bytes at a time (where its rows allow it)
};

template <int BN, bool SWAP, typename OutT>
__global__ void __launch_bounds__(Shape<BN, SWAP>::kThreads, 1)
matmul_kernel(const __grid_constant__ Maps maps, MatmulArgs a, int tiles_r, int tiles_c, int band,
              bool tma_out) {
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

  // The copying and the multiplying thread are on every block's path, one
  // instruction after another: their loops hold little but the waits and the
  // issues (with 64-bit counters and descriptors built per product a block
  // took 0.5 us whatever its size).
  if (warp == 0) {
    if (lane == 0) {
      Ring<G::kStages> ring;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
        int r, c;
        tile_at(t, r, c);
        for (int kb = 0; kb < kblocks; ++kb) {
          // (a wait for the round before the first one passes at once)
          if (!(ok = mbar_wait(&empty[ring.at], ring.phase ^ 1))) break;
          unsigned char* p = tiles + ring.at * G::kStageBytes;
          mbar_arrive_expect_tx(&full[ring.at], G::kStageBytes);
          tma_load_2d(p, &maps.rows, kb * kBlockK, r * kTileRows, &full[ring.at]);
          tma_load_2d(p + G::kRowBytes, &maps.cols, kb * kBlockK, c * BN, &full[ring.at]);
          ring.next();
        }
      }
      if (!ok) {
        timeout();
        // the copies in flight land before the block's memory goes: each stage's
        // last one is in the phase before its next
        for (int i = 0; i < G::kStages; ++i) {
          mbar_wait(&full[ring.at], ring.phase ^ 1, 1u << 16);
          ring.next();
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc(0 /* e4m3 */, kTileRows, BN, false, false);
      const uint64_t rows0 = smem_desc_sw128(smem_u32(tiles), 16, 1024);
      Ring<G::kStages> ring;
      Ring<G::kBufs> bufs;
      const uint32_t n_blocks =
          static_cast<uint32_t>((n_tiles - blockIdx.x + gridDim.x - 1) / gridDim.x) * kblocks;
      bool ok = true;
      uint32_t i = 0;
      for (; i < n_blocks; ++i) {
        if (!(ok = mbar_wait(&tempty[bufs.at], bufs.phase ^ 1) &&
                   mbar_wait(&full[ring.at], ring.phase)))
          break;
        tc_fence_after();
        // descriptors count in 16 bytes
        const uint64_t rows = rows0 + ring.at * (G::kStageBytes >> 4), cols = rows + (G::kRowBytes >> 4);
        const uint32_t to = tmem + bufs.at * BN;
        mma_e4m3_ss(to, rows, cols, idesc, 0);
        mma_e4m3_ss(to, rows + 2, cols + 2, idesc, 1);
        mma_e4m3_ss(to, rows + 4, cols + 4, idesc, 1);
        mma_e4m3_ss(to, rows + 6, cols + 6, idesc, 1);
        mma_commit(&empty[ring.at]);
        mma_commit(&tfull[bufs.at]);
        ring.next();
        bufs.next();
      }
      if (!ok) {
        timeout();
        // the last products end before tensor memory is freed (otherwise the
        // adding warps have waited for them)
        if (i > 0) {
          const int last = (bufs.at + G::kBufs - 1) % G::kBufs;
          mbar_wait(&tfull[last], bufs.at ? bufs.phase : bufs.phase ^ 1, 1u << 16);
        }
      }
    }
  } else {
    const int quad = warp & 3, group = (warp - 2) >> 2;
    Ring<G::kBufs> bufs;
    for (int64_t t = blockIdx.x; t < n_tiles && !s_abort; t += gridDim.x) {
      int r, c;
      tile_at(t, r, c);
      const int64_t row = static_cast<int64_t>(r) * kTileRows + 32 * quad + lane;
      const int64_t col0 = static_cast<int64_t>(c) * BN + G::kCols * group;
      f32x2 acc[G::kCols / 2];
#pragma unroll
      for (int i = 0; i < G::kCols / 2; ++i) acc[i] = 0;
      // Scales, fetched four blocks ahead (a fetch takes longer than a block):
      // that of this thread's row (SWAP: of column `lane` of its columns), and,
      // one block in each lane, that of the 128 rows of B that they all share.
      const int64_t n_as = (a.M - 1) * a.ld_as + kblocks;
      const int64_t n_bs = ((a.N + kScaleGroup - 1) / kScaleGroup - 1) * a.ld_bs + kblocks;
      const int64_t m_scale = SWAP ? col0 + lane % G::kCols : row;
      const int64_t n_scale = (SWAP ? static_cast<int64_t>(r) * kTileRows : col0) / kScaleGroup;
      const bool m_in = m_scale < a.M, n_in = n_scale * kScaleGroup < a.N;
      const float* pa = a.a_scale + m_scale * a.ld_as;
      const float* pb = a.b_scale + n_scale * a.ld_bs;
      float sa[4], next[4], sb = 0.f, sb_next = 0.f;
      auto fetch_a = [&](int kb) {
        if (a.scale_vec && m_in && kb + 4 <= kblocks && kda_guard(pa - a.a_scale + kb, 4, n_as, a.err)) {
          const float4 v = *reinterpret_cast<const float4*>(pa + kb);
          next[0] = v.x; next[1] = v.y; next[2] = v.z; next[3] = v.w;
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            next[u] = m_in && kb + u < kblocks && kda_guard(pa - a.a_scale + kb + u, 1, n_as, a.err)
                          ? pa[kb + u] : 0.f;
        }
      };
      auto fetch_b = [&](int kb) {
        sb_next = n_in && kb + lane < kblocks && kda_guard(pb - a.b_scale + kb + lane, 1, n_bs, a.err)
                      ? pb[kb + lane] : 0.f;
      };
      fetch_a(0);
      fetch_b(0);
      for (int kb4 = 0; kb4 < kblocks && !s_abort; kb4 += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) sa[u] = next[u];
        if (kb4 + 4 < kblocks) fetch_a(kb4 + 4);
        if (kb4 % 32 == 0) {
          sb = sb_next;
          if (kb4 + 32 < kblocks) fetch_b(kb4 + 32);
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int kb = kb4 + u;
        if (kb >= kblocks) break;
        const float scale = sa[u] * __shfl_sync(0xffffffffu, sb, kb & 31);
        const bool ok = mbar_wait(&tfull[bufs.at], bufs.phase);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) timeout();
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem_addr(tmem, 32 * quad, bufs.at * BN + G::kCols * group);
#pragma unroll
        for (int i = 0; i < G::kCols / G::kLoad; ++i) {
          uint32_t d[G::kLoad];
          tmem_ld(at + G::kLoad * i, d);
          wait_ld(d);
#pragma unroll
          for (int j = 0; j < G::kLoad / 2; ++j) {
            f32x2 s;
            if (SWAP)  // lane j of the scales is column j's
              s = pack2(__shfl_sync(0xffffffffu, scale, G::kLoad * i + 2 * j, 32),
                        __shfl_sync(0xffffffffu, scale, G::kLoad * i + 2 * j + 1, 32));
            else
              s = pack2(scale, scale);
            f32x2& to = acc[G::kLoad / 2 * i + j];
            to = fma2(pack2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1])), s, to);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[bufs.at]);
        bufs.next();
      }
      }
      if (s_abort) break;
      OutT* out = static_cast<OutT*>(a.out);
      const int64_t extent = (a.M - 1) * a.ld_out + a.N;
      auto value = [&](int i) {
        float lo, hi;
        unpack2(acc[i / 2], lo, hi);
        return i & 1 ? hi : lo;
      };
      if constexpr (SWAP) {  // a thread holds one row of B for some rows of A
#pragma unroll
        for (int i = 0; i < G::kCols; ++i) {
          const int64_t m = col0 + i, e = m * a.ld_out + row;
          if (m < a.M && row < a.N && kda_guard(e, 1, extent, a.err)) out[e] = from_f32<OutT>(value(i));
        }
      } else {
        // 128 bytes of each of the warp's 32 rows at a time, turned in shared
        // memory: a tensor copy, which leaves out what lies past the last row
        // or column, or, where out's rows do not allow one, a row at a time
        constexpr int kPiece = 128 / sizeof(OutT);
        static_assert(G::kCols % kPiece == 0, "whole pieces");
        unsigned char* own = tiles + G::kStages * G::kStageBytes + 4096 * (warp - 2);
#pragma unroll
        for (int p = 0; p < G::kCols / kPiece; ++p) {
          if (tma_out && lane == 0) bulk_wait_read();  // the piece before has left
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {  // 16 bytes
            uint32_t w[4];
            constexpr int kPer = 4 / sizeof(OutT);  // values in 4 bytes
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = p * kPiece + (4 * q + k) * kPer;
              w[k] = kPer == 2 ? pack2_bf16(value(i), value(i + 1)) : __float_as_uint(value(i));
            }
            *reinterpret_cast<uint4*>(own + sw128_offset(32, lane, 16 * q)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          const int64_t c_at = col0 + p * kPiece, r_at = row - lane;
          if (tma_out) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (c_at < a.N && r_at < a.M)
                tma_store_2d(&maps.out, own, static_cast<int32_t>(c_at), static_cast<int32_t>(r_at));
              bulk_commit();
            }
          } else {
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < 32 && r_at + i < a.M; ++i)
#pragma unroll
              for (int k = 0; k < kPiece; k += 32) {
                const int64_t e = (r_at + i) * a.ld_out + c_at + k + lane;
                if (c_at + k + lane < a.N && kda_guard(e, 1, extent, a.err))
                  out[e] = *reinterpret_cast<const OutT*>(
                      own + sw128_offset(32, i, static_cast<uint32_t>(sizeof(OutT)) * (k + lane)));
              }
          }
        }
      }
    }
    if (!SWAP && tma_out && lane == 0) bulk_wait();  // the block's memory outlives its copies
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

// [rows, cols] elements of `size` bytes, rows `pitch` bytes apart, in boxes of 128 bytes x
// `box` rows with the 128-byte swizzle.  Past the last row and column zeros
// (e4m3 0.0) are read, and nothing is written.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int64_t size, const void* base, int64_t rows,
              int64_t cols, int64_t pitch, uint32_t box) {
  static const EncodeTiledFn fn = find_encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(128 / size), box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, boxes, estr,
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
  constexpr CUtensorMapDataType kBytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!make_map(&maps.rows, kBytes, 1, SWAP ? a.b : a.a, rows, a.K, SWAP ? a.ld_b : a.ld_a, kTileRows) ||
      !make_map(&maps.cols, kBytes, 1, SWAP ? a.a : a.b, cols, a.K, SWAP ? a.ld_a : a.ld_b, BN))
    return cudaErrorInvalidValue;
  constexpr int64_t kOut = sizeof(OutT);
  const bool tma_out = !SWAP && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                       a.ld_out * kOut % 16 == 0;
  if (tma_out && !make_map(&maps.out, kOut == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                           kOut, a.out, a.M, a.N, a.ld_out * kOut, 32))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(G::kSmem));
  if (e != cudaSuccess) return e;
  const int tiles_r = static_cast<int>((rows + kTileRows - 1) / kTileRows);
  const int tiles_c = static_cast<int>((cols + BN - 1) / BN);
  const int64_t n = static_cast<int64_t>(tiles_r) * tiles_c;
  const int band = 12;  // of 152 tiles in flight, 12 x 12.7
  kern<<<static_cast<unsigned>(std::min<int64_t>(n, a.sm_count)), G::kThreads, G::kSmem, s>>>(
      maps, a, tiles_r, tiles_c, band, tma_out);
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
