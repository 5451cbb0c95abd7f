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
// tensor core's 128 lanes, and a tile reads no more of A than there is.  Where
// there are few tiles a cluster of blocks shares each one's k-blocks.
//
// 16384 x 12288 x 4096: 0.66 to 0.74 ms (in a short and in a long run), 2.2 to
// 2.5 PFLOP/s.  What bounds it is the scaling: without the products it takes
// 0.63 ms, without the copies 0.67 ms, without reading and adding the sums 0.56
// ms.  32 x 12288 x 4096 (the weights' bytes, 50 MB): 12.6 us.  From K = 8192 to
// 16384 another 100 MB take 16.3 us, 6.2 TB/s: what is above the bytes is 4 us to
// launch, fill and write out.  32 x 4096 x 4096: 6.7 us; 128 x 12288 x 4096: 15 us.
// (Times of the kernel; from one call to the next 32 x 12288 x 4096 takes 14.4 us.)
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
constexpr int kMaxSplits = 8;  // blocks of a cluster, which share a tile's k-blocks

// D (+)= A B, 8-bit operands from shared memory; issued by one thread.
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// All threads of the cluster's blocks; shared memory written before is seen after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Four floats at this block's shared address `at`, but of block `rank` of the cluster.
__device__ __forceinline__ float4 load_of_block(uint32_t at, int rank) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 t;\n mapa.shared::cluster.u32 t, %4, %5;\n"
      " ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [t];\n}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}

// One lane of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 r;\n elect.sync r|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(is));
  return is != 0;
}

// 32 lanes x 16, 32 or 64 consecutive columns of tensor memory: thread i gets
// lane i of its warp's quarter.  Into 32-bit floats as they are used: a move to
// another kind of register would depend on the load alone, not on the wait
// behind it.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
      "}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]),
        "=f"(r[32]), "=f"(r[33]), "=f"(r[34]), "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]),
        "=f"(r[40]), "=f"(r[41]), "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]),
        "=f"(r[48]), "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]),
        "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]), "=f"(r[63])
      : "r"(taddr));
}
// Waits for this thread's tensor-memory loads and passes `v` on: what is
// computed with the result comes after the wait.  (Naming the loaded registers
// instead cost a move for each.)
__device__ __forceinline__ float wait_ld(float v) {
  float r;
  asm volatile("tcgen05.wait::ld.sync.aligned;\n mov.b32 %0, %1;" : "=f"(r) : "f"(v) : "memory");
  return r;
}
// lo += d0 s0, hi += d1 s1 in one instruction on a pair.  One statement that
// takes the loaded d0, d1 together with the scales that wait_ld passed on: a
// statement of its own to pair d0 and d1 would depend on nothing behind the wait
// and could be moved before it.
__device__ __forceinline__ void add_scaled_pair(float& lo, float& hi, float d0, float d1, float s0,
                                                float s1) {
  asm("{\n .reg .b64 d, s, sum;\n"
      " mov.b64 d, {%2, %3};\n mov.b64 s, {%4, %5};\n mov.b64 sum, {%0, %1};\n"
      " fma.rn.f32x2 sum, d, s, sum;\n mov.b64 {%0, %1}, sum;\n}"
      : "+f"(lo), "+f"(hi)
      : "f"(d0), "f"(d1), "f"(s0), "f"(s1));
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
  // the copying, the multiplying and the scale-fetching warp, one that only
  // fills up their set of four (register shares go by sets), then the adding warps
  static constexpr int kThreads = 128 + 128 * kGroups;
  // 128 sums a thread: the first set gives registers to the others (launched
  // with 168 each, 3 * 168 = 56 + 2 * 224)
  static constexpr bool kShares = kCols == 128;
  static constexpr int kLaunchRegs = 168, kAddRegs = 224, kRestRegs = 56;
  static_assert(!kShares || 128 * (kRestRegs + kGroups * kAddRegs) <= kThreads * kLaunchRegs,
                "register shares exceed the launch's");
  // k-blocks that are copied, multiplied and handed over together: one block's
  // products of a narrow tile take less time than the waits around them
  static constexpr int kUnit = BN == 256 ? 1 : 2;
  static constexpr int kBufs = BN >= 128 ? 2 : 4;           // of tensor memory, a unit each
  static constexpr uint32_t kTmemCols = BN * kUnit * kBufs;
  static constexpr uint32_t kRowBytes = kUnit * kTileRows * kBlockK, kColBytes = kUnit * BN * kBlockK;
  static constexpr uint32_t kStageBytes = kRowBytes + kColBytes;
  static constexpr int kStages = SWAP ? (BN == 64 ? 4 : 5) : BN == 128 ? 3 : 4;
  // columns per tensor-memory load: as many as there are registers for
  static constexpr int kLoad = kCols == 128 ? 64 : kCols % 32 == 0 && !SWAP ? 32 : 16;
  static constexpr int kOwn = SWAP ? BN : kTileRows;       // rows of A in a tile
  static constexpr uint32_t kStoreBytes = SWAP ? 0 : 4 * kGroups * 4096;  // a piece per adding warp
  static constexpr uint32_t kSmem = kStages * kStageBytes + kStoreBytes;
  // with the scales and barriers in front of it, up to the next 1024 bytes
  static constexpr uint32_t kFront = (4 * kOwn * 4 + 256 + 1023) / 1024 * 1024;
  static_assert(kSmem + kFront <= 227 * 1024 && kTmemCols <= 512, "memory of an SM");
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
              int cluster, bool whole, bool tma_out) {
  using G = Shape<BN, SWAP>;
  extern __shared__ __align__(1024) unsigned char tiles[];
  __shared__ uint64_t full[G::kStages], empty[G::kStages], tfull[G::kBufs], tempty[G::kBufs];
  // scales of A: two k-blocks of the tile's rows to a slot
  __shared__ uint64_t sfull[2], sempty[2];
  __shared__ float s_scale[2][2][G::kOwn];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kblocks = (a.K + kBlockK - 1) / kBlockK, units = (kblocks + G::kUnit - 1) / G::kUnit;
  const int64_t n_tiles = static_cast<int64_t>(tiles_r) * tiles_c;
  // a cluster of blocks shares a tile's k-blocks (SWAP), each its own units
  const int splits = SWAP ? cluster : 1, rank = blockIdx.x % splits;
  const int unit0 = SWAP ? static_cast<int>(static_cast<int64_t>(units) * rank / splits) : 0;
  const int unit1 = SWAP ? static_cast<int>(static_cast<int64_t>(units) * (rank + 1) / splits) : units;
  const int kb0 = unit0 * G::kUnit, kb1 = SWAP ? min(unit1 * G::kUnit, kblocks) : kblocks;
  const int64_t tile0 = blockIdx.x / splits, tile_step = gridDim.x / splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < G::kBufs; ++i) { mbar_init(&tfull[i], 1); mbar_init(&tempty[i], 4 * G::kGroups); }
    for (int i = 0; i < 2; ++i) { mbar_init(&sfull[i], 1); mbar_init(&sempty[i], 4 * G::kGroups); }
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

  // The copying and the multiplying warp are on every block's path, one
  // instruction after another: their loops hold little but the waits and the
  // issues, and whole warps run them, so that descriptors and addresses are
  // computed once per warp, where the issuing instructions take them from.
  // (With 64-bit counters, one thread and descriptors built per product, a
  // block of any size took 0.5 us.)
  if (warp < 4) {
    if constexpr (G::kShares) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kRestRegs));
    const bool issues = elect_one();
    if (warp == 0) {
      Ring<G::kStages> ring;
      bool ok = true;
      for (int64_t t = tile0; t < n_tiles && ok; t += tile_step) {
        int r, c;
        tile_at(t, r, c);
        for (int u = unit0; u < unit1; ++u) {
          // (a wait for the round before the first one passes at once)
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[ring.at], ring.phase ^ 1));
          if (!ok) break;
          if (issues) {
            unsigned char* p = tiles + ring.at * G::kStageBytes;
            mbar_arrive_expect_tx(&full[ring.at], G::kStageBytes);
            if (whole) {
              tma_load_3d(p, &maps.rows, 0, r * kTileRows, u * G::kUnit, &full[ring.at]);
              tma_load_3d(p + G::kRowBytes, &maps.cols, 0, c * BN, u * G::kUnit, &full[ring.at]);
            } else {
#pragma unroll
              for (int e = 0; e < G::kUnit; ++e) {
                const int k = (u * G::kUnit + e) * kBlockK;
                tma_load_3d(p + e * kTileRows * kBlockK, &maps.rows, k, r * kTileRows, 0, &full[ring.at]);
                tma_load_3d(p + G::kRowBytes + e * BN * kBlockK, &maps.cols, k, c * BN, 0,
                            &full[ring.at]);
              }
            }
          }
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
    } else if (warp == 1) {
      constexpr uint32_t idesc = make_idesc(0 /* e4m3 */, kTileRows, BN, false, false);
      const uint64_t rows0 = smem_desc_sw128(smem_u32(tiles), 16, 1024);
      Ring<G::kStages> ring;
      Ring<G::kBufs> bufs;
      const uint32_t n_units =
          static_cast<uint32_t>((n_tiles - tile0 + tile_step - 1) / tile_step) * (unit1 - unit0);
      bool ok = true;
      uint32_t i = 0;
      for (; i < n_units; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&tempty[bufs.at], bufs.phase ^ 1) &&
                                         mbar_wait(&full[ring.at], ring.phase));
        if (!ok) break;
        tc_fence_after();
        // descriptors count in 16 bytes
        const uint64_t rows = rows0 + ring.at * (G::kStageBytes >> 4), cols = rows + (G::kRowBytes >> 4);
        const uint32_t to = tmem + bufs.at * (G::kUnit * BN);
        if (issues) {
#pragma unroll
          for (int e = 0; e < G::kUnit; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_e4m3_ss(to + e * BN, rows + e * (kTileRows * kBlockK >> 4) + 2 * k,
                          cols + e * (BN * kBlockK >> 4) + 2 * k, idesc, k > 0);
          mma_commit(&empty[ring.at]);
          mma_commit(&tfull[bufs.at]);
        }
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
    } else if (warp == 2) {
      // The rows' scales lie a row apart, one cache line to each: fetched here
      // once for all the adding warps, up to four blocks ahead of them.
      const int64_t n_as = (a.M - 1) * a.ld_as + kblocks;
      Ring<2> slots;
      bool ok = true;
      for (int64_t t = tile0; t < n_tiles && ok; t += tile_step) {
        int r, c;
        tile_at(t, r, c);
        const int64_t m0 = static_cast<int64_t>(SWAP ? c : r) * G::kOwn;
        for (int kb = kb0; kb < kb1; kb += 2) {
          constexpr int kRows = (G::kOwn + 31) / 32;  // per lane
          float v[kRows][2];
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int64_t m = m0 + 32 * i + lane, e = m * a.ld_as + kb;
            const bool in = m < a.M && 32 * i + lane < G::kOwn;
            v[i][0] = v[i][1] = 0.f;  // (zeros past the last block)
            if (in && kda_guard(e, 1, n_as, a.err)) v[i][0] = a.a_scale[e];
            if (in && kb + 1 < kblocks && kda_guard(e + 1, 1, n_as, a.err)) v[i][1] = a.a_scale[e + 1];
          }
          ok = __all_sync(0xffffffffu, mbar_wait(&sempty[slots.at], slots.phase ^ 1));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (32 * i + lane < G::kOwn) {
              s_scale[slots.at][0][32 * i + lane] = v[i][0];
              s_scale[slots.at][1][32 * i + lane] = v[i][1];
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[slots.at]);
          slots.next();
        }
      }
      if (!ok) timeout();
    }
  } else {
    if constexpr (G::kShares) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kAddRegs));
    const int quad = warp & 3, group = (warp - 4) >> 2;
    Ring<G::kBufs> bufs;
    Ring<2> slots;
    for (int64_t t = tile0; t < n_tiles && !s_abort; t += tile_step) {
      int r, c;
      tile_at(t, r, c);
      const int64_t row = static_cast<int64_t>(r) * kTileRows + 32 * quad + lane;
      const int64_t col0 = static_cast<int64_t>(c) * BN + G::kCols * group;
      float acc[G::kCols];
#pragma unroll
      for (int i = 0; i < G::kCols; ++i) acc[i] = 0.f;
      // The scale of B's 128 rows that this thread's products share, one block
      // in each lane, fetched 32 blocks ahead; A's come through shared memory.
      const int64_t n_bs = ((a.N + kScaleGroup - 1) / kScaleGroup - 1) * a.ld_bs + kblocks;
      const int64_t n_scale = (SWAP ? static_cast<int64_t>(r) * kTileRows : col0) / kScaleGroup;
      const bool n_in = n_scale * kScaleGroup < a.N;
      const float* pb = a.b_scale + n_scale * a.ld_bs;
      float sb = 0.f, sb_next = 0.f;
      auto fetch_b = [&](int kb) {
        sb_next = 0.f;
        if (n_in && kb + lane < kblocks && kda_guard(pb - a.b_scale + kb + lane, 1, n_bs, a.err))
          sb_next = pb[kb + lane];
      };
      fetch_b(kb0);
      // this thread's row of A; SWAP: column `lane` of its columns
      const int own = SWAP ? G::kCols * group + lane % G::kCols : 32 * quad + lane;
      for (int kb = kb0; kb < kb1; kb += 2) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sfull[slots.at], slots.phase))) {
          if (lane == 0) timeout();
          break;
        }
        const float sa[2] = {s_scale[slots.at][0][own], s_scale[slots.at][1][own]};
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[slots.at]);
        slots.next();
        if ((kb - kb0) % 32 == 0) {
          sb = sb_next;
          if (kb + 32 < kblocks) fetch_b(kb + 32);
        }
        bool ok = true;
#pragma unroll
        for (int u = 0; u < 2; u += G::kUnit) {
          if (kb + u >= kb1) break;
          ok = __all_sync(0xffffffffu, mbar_wait(&tfull[bufs.at], bufs.phase));
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = tmem_addr(tmem, 32 * quad, bufs.at * (G::kUnit * BN) + G::kCols * group);
          // One set of registers for all the loads: with two, to load ahead of
          // the additions, the kernel was 20 % slower.
          constexpr int kPieces = G::kCols / G::kLoad;
          float d[G::kLoad];
          tmem_ld(at, d);
#pragma unroll
          for (int p = 0; p < G::kUnit * kPieces; ++p) {
            const int e = p / kPieces, i = p % kPieces;  // block of the unit, piece of its columns
            if (p > 0) tmem_ld(at + BN * e + G::kLoad * i, d);
            // (past the last block the scales and the products are zeros)
            const float scale =
                wait_ld(sa[u + e] * __shfl_sync(0xffffffffu, sb, (kb - kb0 + u + e) & 31));
#pragma unroll
            for (int j = 0; j < G::kLoad; j += 2) {
              // SWAP: lane j of the scales is column j's
              const float s0 = SWAP ? __shfl_sync(0xffffffffu, scale, G::kLoad * i + j, 32) : scale;
              const float s1 = SWAP ? __shfl_sync(0xffffffffu, scale, G::kLoad * i + j + 1, 32) : scale;
              float& lo = acc[G::kLoad * i + j];
              float& hi = acc[G::kLoad * i + j + 1];
              if constexpr (G::kCols == 128) {  // (single additions: 6 % faster here)
                lo = fmaf(d[j], s0, lo);
                hi = fmaf(d[j + 1], s1, hi);
              } else {
                add_scaled_pair(lo, hi, d[j], d[j + 1], s0, s1);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[bufs.at]);
          bufs.next();
        }
        if (!ok) {
          if (lane == 0) timeout();
          break;
        }
      }
      if (s_abort) break;
      OutT* out = static_cast<OutT*>(a.out);
      const int64_t extent = (a.M - 1) * a.ld_out + a.N;
      auto value = [&](int i) { return acc[i]; };
      if constexpr (SWAP) {  // a thread holds one row of B for some rows of A
        if (splits > 1) {  // (every copy and product of this block is done)
#pragma unroll
          for (int i = 0; i < G::kCols; ++i)
            reinterpret_cast<float*>(tiles)[(G::kCols * group + i) * kTileRows + 32 * quad + lane] = value(i);
          break;
        }
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
        unsigned char* own = tiles + G::kStages * G::kStageBytes + 4096 * (warp - 4);
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
#pragma unroll 4
            for (int i = 0; i < 32; ++i)
#pragma unroll
              for (int k = 0; k < kPiece; k += 32) {
                const int64_t e = (r_at + i) * a.ld_out + c_at + k + lane;
                if (r_at + i < a.M && c_at + k + lane < a.N && kda_guard(e, 1, extent, a.err))
                  out[e] = *reinterpret_cast<const OutT*>(
                      own + sw128_offset(32, i, static_cast<uint32_t>(sizeof(OutT)) * (k + lane)));
              }
          }
        }
      }
    }
    if (!SWAP && tma_out && lane == 0) bulk_wait();  // the block's memory outlives its copies
  }
  if constexpr (SWAP) {
    if (splits > 1) {
      // The blocks' sums lie in their shared memory; each block adds up some of
      // the columns, the blocks' parts in order.
      __syncwarp();
      cluster_sync();
      int r, c;
      tile_at(tile0, r, c);
      const int first = BN * rank / splits, last = BN * (rank + 1) / splits;
      const int64_t extent = (a.M - 1) * a.ld_out + a.N;
      // Four values of all blocks in flight at a time, added in the blocks' order:
      // one value and one block after the other, 64 x 1024 x 4096 took 13 us.
      for (int i = first * kTileRows + 4 * threadIdx.x; i < last * kTileRows; i += 4 * G::kThreads) {
        const int64_t m = static_cast<int64_t>(c) * BN + i / kTileRows;
        const int64_t n = static_cast<int64_t>(r) * kTileRows + i % kTileRows, e = m * a.ld_out + n;
        const uint32_t at = smem_u32(tiles) + 4 * i;
        float4 part[kMaxSplits];
#pragma unroll
        for (int q = 0; q < kMaxSplits; ++q)
          part[q] = q < splits ? load_of_block(at, q) : make_float4(0.f, 0.f, 0.f, 0.f);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kMaxSplits; ++q) {
          sum[0] += part[q].x;
          sum[1] += part[q].y;
          sum[2] += part[q].z;
          sum[3] += part[q].w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (m < a.M && n + k < a.N && kda_guard(e + k, 1, extent, a.err))
            static_cast<OutT*>(a.out)[e + k] = from_f32<OutT>(sum[k]);
      }
      __syncwarp();
      cluster_sync();  // no block's memory goes while another reads it
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

bool encode(CUtensorMap* m, CUtensorMapDataType type, uint32_t rank, const void* base,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  static const EncodeTiledFn fn = find_encode();
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn && fn(m, type, rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand's [rows, K] bytes, `box` rows of a k-block to a copy, 128-byte
// swizzle.  Where K is whole blocks, as (byte of a block, row, block), and one
// copy takes `unit` blocks; else as (byte of a row, row, 0): past the last row
// and the last byte zeros (e4m3 0.0) are read.
bool operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int64_t ld, uint32_t box,
                 uint32_t unit) {
  const bool whole = K % kBlockK == 0;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(whole ? kBlockK : K),
                              static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(whole ? K / kBlockK : 1)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld),
                                 static_cast<cuuint64_t>(whole ? kBlockK : 16)};
  const cuuint32_t boxes[3] = {kBlockK, box, whole ? unit : 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, boxes);
}

// Clusters of `splits` blocks that are resident at a time: fewer than the SMs
// would give, as a cluster stays within a group of SMs.  Asked for once.
template <int BN, bool SWAP, typename OutT>
int resident_clusters(int splits) {
  using G = Shape<BN, SWAP>;
  struct Counts {
    int of[kMaxSplits + 1];
  };
  static const Counts counts = [] {
    Counts c;
    memset(&c, 0, sizeof c);
    constexpr auto kern = matmul_kernel<BN, SWAP, OutT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(G::kSmem)) != cudaSuccess)
      return c;
    for (int n = 2; n <= kMaxSplits; n *= 2) {
      cudaLaunchConfig_t cfg;
      memset(&cfg, 0, sizeof cfg);
      cfg.gridDim = dim3(static_cast<unsigned>(n));
      cfg.blockDim = dim3(G::kThreads);
      cfg.dynamicSmemBytes = G::kSmem;
      cudaLaunchAttribute cluster;
      cluster.id = cudaLaunchAttributeClusterDimension;
      cluster.val.clusterDim.x = static_cast<unsigned>(n);
      cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
      cfg.attrs = &cluster;
      cfg.numAttrs = 1;
      int found = 0;
      if (cudaOccupancyMaxActiveClusters(&found, kern, &cfg) == cudaSuccess) c.of[n] = found;
    }
    return c;
  }();
  return counts.of[splits];
}

// How a product is cut into tiles, and into how many blocks its k-blocks.
struct Cut {
  int64_t tiles;
  int splits;
  double cost;  // estimated, in us
};

// Few tiles: a cluster of up to 8 blocks shares each one's k-blocks, as long as
// all are resident and a block has two copies to overlap.  (16 tiles of 64 x
// 128 with K = 4096: 8 blocks each, which are not all resident, 12.5 us.)
//
// The time goes by whole waves of tiles: a wave takes `block_us` per k-block
// and about 1.5 us to fill and to write out, a launch 3 us, a cluster's sum 1 us.
template <int BN, bool SWAP, typename OutT>
Cut cut(const MatmulArgs& a, double block_us) {
  using G = Shape<BN, SWAP>;
  const int64_t rows = SWAP ? a.N : a.M, cols = SWAP ? a.M : a.N;
  Cut c;
  c.tiles = ((rows + kTileRows - 1) / kTileRows) * ((cols + BN - 1) / BN);
  c.splits = 1;
  const int64_t kblocks = (a.K + kBlockK - 1) / kBlockK;
  const int64_t units = (kblocks + G::kUnit - 1) / G::kUnit;
  if (SWAP)
    while (c.splits < kMaxSplits && units >= 4 * c.splits &&
           c.tiles <= resident_clusters<BN, SWAP, OutT>(2 * c.splits))
      c.splits *= 2;
  const int64_t waves = c.splits > 1 ? 1 : (c.tiles + a.sm_count - 1) / a.sm_count;
  c.cost = waves * ((kblocks + c.splits - 1) / c.splits * block_us + 1.5) + 3 + (c.splits > 1 ? 1 : 0);
  return c;
}

template <int BN, bool SWAP, typename OutT>
cudaError_t run(const MatmulArgs& a, const Cut& how, cudaStream_t s) {
  using G = Shape<BN, SWAP>;
  constexpr auto kern = matmul_kernel<BN, SWAP, OutT>;
  const int64_t rows = SWAP ? a.N : a.M, cols = SWAP ? a.M : a.N;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  const bool whole = a.K % kBlockK == 0;
  if (!operand_map(&maps.rows, SWAP ? a.b : a.a, rows, a.K, SWAP ? a.ld_b : a.ld_a, kTileRows, G::kUnit) ||
      !operand_map(&maps.cols, SWAP ? a.a : a.b, cols, a.K, SWAP ? a.ld_a : a.ld_b, BN, G::kUnit))
    return cudaErrorInvalidValue;
  constexpr int64_t kOut = sizeof(OutT);
  const bool tma_out = !SWAP && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                       a.ld_out * kOut % 16 == 0;
  if (tma_out) {  // past the last row and column nothing is written
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ld_out * kOut)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / kOut), 32};
    if (!encode(&maps.out, kOut == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                2, a.out, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  if (G::kShares) {
    // a build that launches with fewer registers could never give the adding
    // warps their share: it is not launched
    static const int regs = [] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < G::kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(G::kSmem));
  if (e != cudaSuccess) return e;
  const int tiles_r = static_cast<int>((rows + kTileRows - 1) / kTileRows);
  const int tiles_c = static_cast<int>((cols + BN - 1) / BN);
  const int band = 12;  // of 152 tiles in flight, 12 x 12.7
  const int splits = how.splits;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(splits > 1 ? how.tiles * splits : std::min<int64_t>(how.tiles, a.sm_count)));
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = static_cast<unsigned>(splits);
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, a, tiles_r, tiles_c, band, splits, whole, tma_out);
}

template <typename OutT>
cudaError_t choose(const MatmulArgs& a, cudaStream_t s) {
  // Up to 32 rows one narrow tile holds them all, and the weights are read once:
  // no wider one was faster from 512 x 8192 to 12288 x 4096.
  if (a.M <= 16) return run<16, true, OutT>(a, cut<16, true, OutT>(a, 0.2), s);
  if (a.M <= 32) return run<32, true, OutT>(a, cut<32, true, OutT>(a, 0.2), s);
  // Above, the cheapest by whole waves, with the times per k-block that sweeps of
  // 33 to 4096 rows gave.  (Taking the widest tile of which there is one for
  // every SM, 128 x 12288 x 4096 took 25 us instead of 15, 384 x 4096 x 4096
  // 18.5 instead of 12.5, 1024 x 4096 x 12288 56 instead of 48.)
  const Cut s32 = cut<32, true, OutT>(a, 0.2), s64 = cut<64, true, OutT>(a, 0.31);
  const Cut n64 = cut<64, false, OutT>(a, 0.2), n128 = cut<128, false, OutT>(a, 0.255);
  const Cut n256 = cut<256, false, OutT>(a, 0.45);
  const double least = std::min({s32.cost, s64.cost, n64.cost, n128.cost, n256.cost});
  if (n256.cost <= least) return run<256, false, OutT>(a, n256, s);
  if (n128.cost <= least) return run<128, false, OutT>(a, n128, s);
  if (n64.cost <= least) return run<64, false, OutT>(a, n64, s);
  if (s64.cost <= least) return run<64, true, OutT>(a, s64, s);
  return run<32, true, OutT>(a, s32, s);
}

}  // namespace

cudaError_t launch_matmul_fp8(const MatmulArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_matmul_fp8");
  const cudaError_t e = a.bf16 ? choose<Bf16>(a, s) : choose<float>(a, s);
  prof_end(s, "kda_matmul_fp8");
  return e;
}

}  // namespace kda
