// Attention over prompts: grouped heads, packed sequences, causal or not.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j),  j < reach of i
//
// One pass over the keys with the running maximum m and sum l of a softmax:
// p = 2^(c s - c m) with c = scale log2 e, o = sum p v / l.  Where a tile's
// maximum passes m by more than 2^8 (in p), m moves up and o and l are scaled;
// below that p only grows, which costs bf16 and 32 bits no precision.
//
// A block takes 256 rows of queries, as two tiles of 128 (tensor memory's lanes),
// and goes over its keys 128 at a time.  Rows are tokens x query heads of one key
// head (as many as a power of two divides the group): heads of a group share the
// keys' tiles, and short sequences fill the rows.  Both products run on tcgen05:
// S = Q K^T into tensor memory; four warps per tile, a row to a thread, turn S
// into P in bf16 over it; O += P V with P read from tensor memory.  While one
// tile's softmax runs, the other's products do.  One warp issues the copies (TMA),
// one the products.
//
// P is rounded to bf16 because the tensor core multiplies bf16 by bf16 (V's
// type); the sum l is of the unrounded p, in 32 bits.
//
// Keys outside a query's reach get p = 0, and 0 times a value's infinity or NaN
// would be NaN: in tiles that reach past a row's last key two warps look through
// V's tile before it is used.  Where they find such values they put zeros there,
// and rows that do reach them get them added at the end.
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "kda_attention.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

using namespace sm100;

constexpr int kTile = 128;               // rows of queries, and keys, of a tile
constexpr int kRows = 2 * kTile;         // rows of a block
constexpr int kThreads = 128 + kRows;    // control warps, then a thread per row
constexpr int kLaunchRegs = 168, kRowRegs = 224, kRestRegs = 56;
static_assert(128 * kRestRegs + kRows * kRowRegs <= kThreads * kLaunchRegs,
              "register shares exceed the launch's");
constexpr int kParts = 2;                // of a tile's P, handed over one by one
constexpr float kSlack = 8.0f;           // log2 of how far p may pass 1

template <int D>
struct Shape {
  static constexpr int kBlocks = D / 64;                     // 128-byte column blocks of a row
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  // V's tile j and K's tile j + 1 are copied, used and given back together
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kSmem = (3 + 2 * kStages) * kTileBytes;  // Q's two, K's first, the pairs
  // tensor memory: S (and P over it) of both tiles, then O
  static constexpr uint32_t kColS = 0, kColO = 2 * kTile;
  static_assert(kSmem + 1024 + 512 <= 227 * 1024, "memory of an SM");
  static_assert(kSmem > 114 * 1024, "one block to an SM: each takes all of tensor memory");
};

struct Maps {
  CUtensorMap q, k, v;
};

// What a block works on.
struct Unit {
  int32_t seq, head0, kv_head;
  int64_t q0, q1;    // its sequence's queries
  int64_t k0, len;   // and keys
  int64_t tok0;      // the block's first query, in the sequence
};

// D (+)= A B with A (bf16 pairs in tensor memory's columns); issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 r;\n elect.sync r|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(is));
  return is != 0;
}

// A whole row of scores: this thread's lane, 128 columns.  One statement with its
// wait, so that nothing uses the registers before they are there.
__device__ __forceinline__ void tmem_row(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
      "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127"
      "}, [%128];\n tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]),
        "=f"(r[32]), "=f"(r[33]), "=f"(r[34]), "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]),
        "=f"(r[40]), "=f"(r[41]), "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]),
        "=f"(r[48]), "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]),
        "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]), "=f"(r[63]),
        "=f"(r[64]), "=f"(r[65]), "=f"(r[66]), "=f"(r[67]), "=f"(r[68]), "=f"(r[69]), "=f"(r[70]), "=f"(r[71]),
        "=f"(r[72]), "=f"(r[73]), "=f"(r[74]), "=f"(r[75]), "=f"(r[76]), "=f"(r[77]), "=f"(r[78]), "=f"(r[79]),
        "=f"(r[80]), "=f"(r[81]), "=f"(r[82]), "=f"(r[83]), "=f"(r[84]), "=f"(r[85]), "=f"(r[86]), "=f"(r[87]),
        "=f"(r[88]), "=f"(r[89]), "=f"(r[90]), "=f"(r[91]), "=f"(r[92]), "=f"(r[93]), "=f"(r[94]), "=f"(r[95]),
        "=f"(r[96]), "=f"(r[97]), "=f"(r[98]), "=f"(r[99]), "=f"(r[100]), "=f"(r[101]), "=f"(r[102]), "=f"(r[103]),
        "=f"(r[104]), "=f"(r[105]), "=f"(r[106]), "=f"(r[107]), "=f"(r[108]), "=f"(r[109]), "=f"(r[110]), "=f"(r[111]),
        "=f"(r[112]), "=f"(r[113]), "=f"(r[114]), "=f"(r[115]), "=f"(r[116]), "=f"(r[117]), "=f"(r[118]), "=f"(r[119]),
        "=f"(r[120]), "=f"(r[121]), "=f"(r[122]), "=f"(r[123]), "=f"(r[124]), "=f"(r[125]), "=f"(r[126]), "=f"(r[127])
      : "r"(taddr)
      : "memory");
}
// 32 columns of this thread's lane, with the wait.
__device__ __forceinline__ void tmem_part(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];\n tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "};" ::"f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]),
      "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]),
      "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31]),
      "r"(taddr)
      : "memory");
}

// 0 for finite pairs of bf16, NaN in a half whose value is not.
__device__ __forceinline__ uint32_t times_zero(uint32_t pair, uint32_t sum) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(pair), "r"(0u), "r"(sum));
  return r;
}
__device__ __forceinline__ bool finite_bf16(uint32_t bits) { return (bits & 0x7f80u) != 0x7f80u; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ Maps maps, AttentionArgs a, int pack) {
  using G = Shape<D>;
  extern __shared__ __align__(1024) unsigned char smem[];  // Q's tiles, then the ring
  __shared__ uint64_t q_full[2], k_full, kv_full[G::kStages], kv_empty[G::kStages], v_ok[G::kStages];
  __shared__ uint64_t s_full[2], p_full[2][kParts], o_full[2], drained[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_infinite;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (a.cu_q && blockIdx.x == 0) {
    check_cu_seqlens(a.cu_q, a.N, a.Tq, threadIdx.x, kThreads, a.err);
    check_cu_seqlens(a.cu_k, a.N, a.Tk, threadIdx.x, kThreads, a.err);
  }
  // ---- the block's queries.  Blocks with the most keys come first: a causal
  // sequence's last ones.
  const int tokens = kRows / pack;  // queries of a block
  const int head_blocks = a.heads / pack;
  Unit u;
  {
    int64_t block, slot = blockIdx.x / head_blocks;
    const int hb = static_cast<int>(blockIdx.x - slot * head_blocks);
    if (a.cu_q) {
      // sequence n's blocks lie in slots [cu[n] / tokens + n, cu[n + 1] / tokens + n + 1):
      // enough for its queries, wherever they start
      int32_t lo = 0, hi = a.N - 1;
      while (lo < hi) {
        const int32_t mid = lo + ((hi - lo + 1) >> 1);
        if (!kda_guard(mid, 1, static_cast<int64_t>(a.N) + 1, a.err)) break;
        if (a.cu_q[mid] / tokens + static_cast<int64_t>(mid) <= slot) lo = mid; else hi = mid - 1;
      }
      u.seq = lo;
      int32_t first = 0;
      if (kda_guard(lo, 1, static_cast<int64_t>(a.N) + 1, a.err)) first = a.cu_q[lo];
      block = slot - (first / tokens + static_cast<int64_t>(lo));
    } else {
      u.seq = static_cast<int32_t>(slot % a.N);
      block = slot / a.N;
    }
    sequence_span(a.cu_q, a.N, a.Tq, u.seq, u.q0, u.q1, a.err);
    int64_t k1;
    sequence_span(a.cu_k, a.N, a.Tk, u.seq, u.k0, k1, a.err);
    u.len = k1 - u.k0;
    const int64_t blocks = (u.q1 - u.q0 + tokens - 1) / tokens;
    if (block < 0 || block >= blocks) return;  // (no such block)
    u.tok0 = (blocks - 1 - block) * tokens;
    u.head0 = hb * pack;
    u.kv_head = u.head0 / (a.heads / a.kv_heads);
  }
  // how many keys the query at `tok` of the sequence reaches
  const int64_t n_q = u.q1 - u.q0;
  auto reach_of = [&](int64_t tok) {
    return a.causal ? min(u.len, max(int64_t{0}, tok + 1 + u.len - n_q)) : u.len;
  };
  int64_t n_tiles[2];  // of keys, for each tile of rows
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t first = u.tok0 + i * (tokens / 2), last = min(first + tokens / 2, n_q) - 1;
    n_tiles[i] = last >= first ? (reach_of(last) + kTile - 1) / kTile : 0;
  }
  const int64_t n_max = max(n_tiles[0], n_tiles[1]);
  const int64_t first_masked = reach_of(u.tok0) / kTile;  // tiles that some row does not reach all of

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      for (int h = 0; h < kParts; ++h) mbar_init(&p_full[i][h], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&drained[i], 1);
    }
    mbar_init(&k_full, 1);
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 3);  // both tiles' products and the look through V
      mbar_init(&v_ok[i], 1);
    }
    mbar_fence_init();
    s_infinite = 0;
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  unsigned char* const first_k = smem + 2 * G::kTileBytes;
  unsigned char* const ring = first_k + G::kTileBytes;  // V, K; V, K
  auto timeout = [&]() { atomicOr(a.err, kDevErrTimeout); };
  auto whole_warp = [](bool ok) { return __all_sync(0xffffffffu, ok); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == 0) {
      // ---- copies
      const bool issues = elect_one();
      auto copy = [&](unsigned char* to, const CUtensorMap* map, int32_t head, int64_t row, uint64_t* bar) {
#pragma unroll
        for (int b = 0; b < G::kBlocks; ++b)
          tma_load_3d(to + b * (kTile * 128), map, 64 * b, head, static_cast<int32_t>(row), bar);
      };
      if (issues && n_max > 0) {
        mbar_arrive_expect_tx(&k_full, G::kTileBytes);
        copy(first_k, &maps.k, u.kv_head, u.k0, &k_full);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (n_tiles[i] == 0) continue;
          mbar_arrive_expect_tx(&q_full[i], G::kTileBytes);
          copy(smem + i * G::kTileBytes, &maps.q, u.head0, u.q0 + u.tok0 + i * (tokens / 2), &q_full[i]);
        }
      }
      int at = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int64_t j = 0; j < n_max && ok; ++j) {
        ok = whole_warp(mbar_wait(&kv_empty[at], phase ^ 1));  // (the first round passes at once)
        if (!ok) break;
        if (issues) {
          unsigned char* const to = ring + at * (2 * G::kTileBytes);
          const bool more = j + 1 < n_max;
          mbar_arrive_expect_tx(&kv_full[at], more ? 2 * G::kTileBytes : G::kTileBytes);
          copy(to, &maps.v, u.kv_head, u.k0 + j * kTile, &kv_full[at]);
          if (more) copy(to + G::kTileBytes, &maps.k, u.kv_head, u.k0 + (j + 1) * kTile, &kv_full[at]);
        }
        if (++at == G::kStages) { at = 0; phase ^= 1; }
      }
      if (!ok) {
        timeout();
        // the copies in flight land before the block's memory goes
        for (int i = 0; i < G::kStages; ++i) {
          mbar_wait(&kv_full[at], phase ^ 1, 1u << 16);
          if (++at == G::kStages) { at = 0; phase ^= 1; }
        }
      }
    } else if (warp < 3) {
      // ---- products, a warp to a tile.  S_i of the next keys comes behind O_i of
      // these: P_i lies over S_i.
      const int i = warp - 1;
      const bool issues = elect_one();
      constexpr uint32_t id_s = make_idesc(kFmtBF16, kTile, kTile, false, false);
      constexpr uint32_t id_o = make_idesc(kFmtBF16, kTile, D, false, true);
      const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + i * G::kTileBytes), 16, 1024);
      const uint32_t t_s = tmem + G::kColS + i * kTile, t_o = tmem + G::kColO + i * D;
      auto scores = [&](uint64_t k) {  // S_i = Q_i K^T
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t step = (s / 4) * (kTile * 128 >> 4) + (s % 4) * 2;
          mma_f16_ss(t_s, q_desc + step, k + step, id_s, s > 0);
        }
        mma_commit(&s_full[i]);
      };
      const int64_t mine = n_tiles[i];
      int at = 0;
      uint32_t phase = 0;
      bool ok = true;
      if (mine > 0) {
        ok = mbar_wait(&k_full, 0) && mbar_wait(&q_full[i], 0);
        if (ok && issues) scores(smem_desc_sw128(smem_u32(first_k), 16, 1024));
      }
      for (int64_t j = 0; j < n_max && ok; ++j) {
        // (looked through, where some row does not reach all of V's tile)
        ok = mbar_wait(j >= first_masked ? &v_ok[at] : &kv_full[at], phase);
        if (j < mine) {
          const uint32_t pair = smem_u32(ring + at * (2 * G::kTileBytes));
          const uint64_t v = smem_desc_sw128(pair, kTile * 128, 1024);
#pragma unroll
          for (int part = 0; part < kParts; ++part) {  // O_i += P_i V
            ok = ok && mbar_wait(&p_full[i][part], static_cast<uint32_t>(j) & 1);
            if (ok && issues) {
              tc_fence_after();
#pragma unroll
              for (int s = part * (kTile / 16 / kParts); s < (part + 1) * (kTile / 16 / kParts); ++s)
                mma_f16_ts(t_o, t_s + 8 * s, v + s * (2048 >> 4), id_o, j > 0 || s > 0);
            }
          }
          if (ok && issues) {
            if (j + 1 < mine) scores(smem_desc_sw128(pair + G::kTileBytes, 16, 1024));
            else mma_commit(&o_full[i]);
          }
        }
        if (ok && issues) mma_commit(&kv_empty[at]);
        if (++at == G::kStages) { at = 0; phase ^= 1; }
      }
      if (!ok) {
        timeout();
        if (issues) {  // the products in flight end before their memory goes
          mma_commit(&drained[i]);
          mbar_wait(&drained[i], 0, 1u << 16);
        }
      }
      __syncwarp();
    } else {
      // ---- V's tiles that some row does not reach all of: no infinity or NaN
      bool ok = true;
      int at = 0;
      uint32_t phase = 0;
      for (int64_t j = 0; j < n_max && ok; ++j) {
        ok = whole_warp(mbar_wait(&kv_full[at], phase));
        if (!ok) break;
        if (j >= first_masked) {
          uint4* tile = reinterpret_cast<uint4*>(ring + at * (2 * G::kTileBytes));
          constexpr int kVecs = G::kTileBytes / 16;
          uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 8
          for (int e = lane; e < kVecs; e += 32) {
            const uint4 w = tile[e];
            sum[0] = times_zero(w.x, sum[0]);
            sum[1] = times_zero(w.y, sum[1]);
            sum[2] = times_zero(w.z, sum[2]);
            sum[3] = times_zero(w.w, sum[3]);
          }
          // (a sum of zeros is 0 or -0)
          if (((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0) {
            for (int e = lane; e < kVecs; e += 32) {
              uint4 w = tile[e];
              uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = (finite_bf16(x[k]) ? x[k] & 0xffffu : 0u) | (finite_bf16(x[k] >> 16) ? x[k] & 0xffff0000u : 0u);
              tile[e] = w;
            }
            s_infinite = 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(&v_ok[at]);
          mbar_arrive(&kv_empty[at]);
        }
        if (++at == G::kStages) { at = 0; phase ^= 1; }
      }
      if (!ok && lane == 0) timeout();
    }
  } else {
    // ---- softmax: a thread to a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const int i = (warp - 4) >> 2, quad = warp & 3;
    const int row = 32 * quad + lane;  // of the tile
    const int64_t tok = u.tok0 + i * (tokens / 2) + row / pack;
    const int32_t head = u.head0 + row % pack;
    const bool valid = tok < n_q;
    const int64_t reach = valid ? reach_of(tok) : 0;
    const int64_t tiles = n_tiles[i];
    // all of the tile's rows reach these tiles whole
    const int64_t whole = reach_of(u.tok0 + i * (tokens / 2)) / kTile;
    const uint32_t t_s = tmem_addr(tmem, 32 * quad, G::kColS + i * kTile);
    const uint32_t t_o = tmem_addr(tmem, 32 * quad, G::kColO + i * D);
    const float c = a.scale * kLog2e;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int64_t j = 0; j < tiles; ++j) {
      ok = whole_warp(mbar_wait(&s_full[i], static_cast<uint32_t>(j) & 1));
      if (!ok) break;
      tc_fence_after();
      float s[kTile];
      tmem_row(t_s, s);
      if (j >= whole) {
        const int limit = static_cast<int>(min(reach - j * kTile, int64_t{kTile}));
#pragma unroll
        for (int k = 0; k < kTile; ++k)
          if (k >= limit) s[k] = -INFINITY;
      }
      float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int k = 4; k < kTile; ++k) top[k % 4] = fmaxf(top[k % 4], s[k]);
      const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (j == 0) {
        m = most;
      } else if (__any_sync(0xffffffffu, (most - m) * c > kSlack)) {
        // (the products of the tile before are done: S came behind them)
        const float next = fmaxf(m, most);
        const float keep = next == -INFINITY ? 1.0f : ex2((m - next) * c);
        m = next;
        l *= keep;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          float o[32];
          tmem_part(t_o + k, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= keep;
          tmem_st32(t_o + k, o);
        }
        tmem_wait_st();
      }
      const float base = m == -INFINITY ? 0.0f : m * c;
      const f32x2 cc = pack2(c, c), less = pack2(-base, -base);
      f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float packed[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float lo, hi;
          unpack2(fma2(pack2(s[64 * k + 2 * e], s[64 * k + 2 * e + 1]), cc, less), lo, hi);
          lo = ex2(lo);
          hi = ex2(hi);
          sum[e % 2] = add2(sum[e % 2], pack2(lo, hi));
          packed[e] = __uint_as_float(pack2_bf16(lo, hi));
        }
        tmem_st32(t_s + 32 * k, packed);
        if (kParts == 2 || k == 1) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[i][kParts == 2 ? k : 0]);
        }
      }
      float lo, hi;
      unpack2(add2(sum[0], sum[1]), lo, hi);
      l += lo + hi;
    }
    // ---- output
    if (ok && tiles > 0) {
      ok = whole_warp(mbar_wait(&o_full[i], 0));
      tc_fence_after();
    }
    if (!ok) {
      if (lane == 0) timeout();
    } else {
      const float scale = reach > 0 ? 1.0f / l : 0.0f;
      const int64_t at = (u.q0 + tok) * a.ld_out + static_cast<int64_t>(head) * D;
      const int64_t extent = (a.Tq - 1) * a.ld_out + static_cast<int64_t>(a.heads) * D;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        if (tiles > 0) tmem_part(t_o + k, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = reach > 0 ? o[e] * scale : 0.0f;
        if (s_infinite) {  // values taken out of V's tiles, for rows that reach them
          for (int64_t t = first_masked * kTile; t < reach; ++t) {
            const int64_t from = (u.k0 + t) * a.ld_v + static_cast<int64_t>(u.kv_head) * D + k;
            if (!kda_guard(from, 32, (a.Tk - 1) * a.ld_v + static_cast<int64_t>(a.kv_heads) * D, a.err)) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t bits = a.v[from + e].bits;
              if (!finite_bf16(bits)) o[e] += bf16_to_f32(static_cast<uint16_t>(bits));
            }
          }
        }
        if (valid && kda_guard(at + k, 32, extent, a.err)) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4*>(a.out + at + k + e) =
                make_uint4(pack2_bf16(o[e], o[e + 1]), pack2_bf16(o[e + 2], o[e + 3]),
                           pack2_bf16(o[e + 4], o[e + 5]), pack2_bf16(o[e + 6], o[e + 7]));
        }
      }
      const int64_t e = (u.q0 + tok) * a.heads + head;
      if (a.lse && valid && kda_guard(e, 1, a.Tq * a.heads, a.err))
        a.lse[e] = reach > 0 ? (m == -INFINITY ? 0.0f : m) * a.scale + logf(l) : -INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
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

// [tokens, heads, d]: 64 channels x `heads_box` heads x `tokens_box` tokens to a copy.
// Past the last token zeros are read.
bool encode(CUtensorMap* m, const void* base, int d, int heads, int64_t tokens, int64_t ld,
            uint32_t heads_box, uint32_t tokens_box) {
  static const EncodeTiledFn fn = find_encode();
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, heads_box, tokens_box}, one[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t run(const AttentionArgs& a, cudaStream_t s) {
  using G = Shape<D>;
  // heads of a group side by side in a tile: the largest power of two in the group
  const int group = a.heads / a.kv_heads, pack = std::min(group & -group, kTile);
  Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!encode(&maps.q, a.q, D, a.heads, a.Tq, a.ld_q, static_cast<uint32_t>(pack),
              static_cast<uint32_t>(kTile / pack)))
    return cudaErrorInvalidValue;
  // (without keys no tile of them is copied)
  if (a.Tk > 0 && (!encode(&maps.k, a.k, D, a.kv_heads, a.Tk, a.ld_k, 1, kTile) ||
                   !encode(&maps.v, a.v, D, a.kv_heads, a.Tk, a.ld_v, 1, kTile)))
    return cudaErrorInvalidValue;
  constexpr auto kern = attention_kernel<D>;
  // a build that launches with fewer registers could never give the rows' warps
  // their share: it is not launched
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(G::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t tokens = kRows / pack;
  const int64_t slots = a.cu_q ? a.Tq / tokens + a.N : (a.Tq / a.N + tokens - 1) / tokens * a.N;
  const int64_t grid = slots * (a.heads / pack);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<static_cast<unsigned>(grid), kThreads, G::kSmem, s>>>(maps, a, pack);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t s) {
  prof_begin(s, "kda_attention_fwd");
  const cudaError_t e = a.d == 128 ? run<128>(a, s) : run<64>(a, s);
  prof_end(s, "kda_attention_fwd");
  return e;
}

}  // namespace kda
