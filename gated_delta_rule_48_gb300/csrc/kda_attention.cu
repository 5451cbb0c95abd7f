// Attention over prompts: grouped heads, packed sequences, causal or not.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j),  j < reach of i
//
// One pass over the keys with the running maximum m and sum l of a softmax:
// p = 2^(c s - c m - 8) with c = scale log2 e, o = sum p v / l.  Where a tile's
// maximum passes m by more than 2^8 (in p), m moves up and o and l are scaled;
// below that p only grows, up to 1, which costs bf16 and 32 bits no precision.  (Without
// the 8 p grew up to 2^8, and sums over values of 2^120 passed what 32 bits hold.)
//
// A unit of work is 256 rows of queries, as two tiles of 128 (tensor memory's lanes),
// over their keys, 128 at a time.  Rows are tokens x query heads of one key head (as
// many as a power of two divides the group): heads of a group share the keys' tiles,
// and short sequences fill the rows.  Both products run on tcgen05: S = Q K^T into
// tensor memory; four warps per tile, a row to a thread, turn S into P in bf16 over it;
// O += P V with P read from tensor memory.  One warp finds units and issues the copies
// (TMA), one per tile its products (a single one for both had to wait for each tile's
// softmax before it could look after the other: 199 us instead of 177 for 128 tiles of
// keys on every SM), one looks through V (below).
//
// A block stays on its SM and asks for further units (cluster launch control), so that
// one unit's first copies run beside the last one's output.  Units go out with the most
// keys first.  Few units are cut along the keys, up to eight blocks for each SM, and a
// second launch joins the parts (32 queries of 8 heads over 65,536 keys of one, 128
// channels: 0.7 ms whole, 32 us cut).  The parts of a unit are equal, so sizes just above
// a full wave of units do badly (2500 queries below).
//
// Bound: for long sequences the products and the softmax beside them.  Two tiles by
// 128 keys are 2048 cycles of products (d = 128); a full wave (2432 queries over 16,384
// keys, 16 heads, not causal) takes 179 us, 1.82 PFLOP/s of 1.9, but 2500 queries over
// 16,452 282 us: 158 units in halves, three rounds.  32,768 causal tokens of 16 heads take
// 2.35 to 2.8 ms, 1.56 to 1.87 PFLOP/s, by how long the power limit has held.  With d = 64
// the floor is the exponentials: 16 a cycle and SM, 128 x 256 of them to 1024 cycles of
// products.  For short ones it is the units' ends: 4 x 4096 tokens of 32 heads 375 to 415 us
// (1.33 to 1.47 PFLOP/s), 2 x 4096 with d = 64 155 us (both pipes 40 % busy), 100 tokens
// 10.6 us, most of it the way from the launch to the first product and from the last one to
// the output, 1024 tokens 36 us, of which the halves' output and the join are a good part
// (2048, whole: 36 us).
//
// P is rounded to bf16 because the tensor core multiplies bf16 by bf16 (V's
// type); the sum l is of the unrounded p, in 32 bits.
//
// The tensor core adds to O with what lies some 2^-25 below it cut off: of 2^20 keys of
// like weights the sum came out 0.5 % too small, of 2^22 2.3 %.  So after every 2^18 keys
// of a unit O (and l) is moved to a sum in the block's own memory, and begins again at 0
// (2^22 keys: within 0.03 %).  That is a kernel of its own (MOVES), for calls with that many
// keys: with the move in it the softmax's loop is slower (32,768 tokens 2.60 ms instead of
// 2.43, 164,000 keys of 40 packed sequences 278 us instead of 270).
//
// Keys outside a query's reach get p = 0, and 0 times a value's infinity or NaN
// would be NaN: in tiles that reach past a row's last key a warp looks through
// V's tile before it is used.  Where it finds such values it puts zeros there,
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
constexpr int kPartTiles = 4;            // the least of a unit's part of the keys
constexpr int kMoveTiles = 2048;         // of keys, after which O is moved
constexpr int kMaxPlaces = 1024;         // for it: as many as SMs, a block to each
// The wait for a block's next unit lasts as long as this one where a tile has no rows of
// it, and a unit may have 2^24 tiles of keys, some 25 s.  Others last a few tiles.
constexpr uint32_t kUnitPolls = 24u << 20;  // of 2 us, as mbar_wait's
constexpr int kHandOver = 4;             // pairs of p between a part's store and its handing over
constexpr float kSlack = 8.0f;           // log2 of how far p may grow: from 2^-8 to 1
constexpr float kLn2 = 0.6931471805599453f;
// Up to here p = 2^(c s - b) with b = c m + 8 rounded once: all of a row's p, and its l and o,
// have the same factor 2^(c m + 8 - b), at most 2^(1/32), which o / l and log l + b take
// off again.  From here on that factor grows (from 2^31 on p would be 0 or infinite): m is
// taken off the scores before c is multiplied in.
constexpr float kLarge = 1048576.0f;

template <int D>
struct Shape {
  static constexpr int kBlocks = D / 64;                     // 128-byte column blocks of a row
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  // V's tile j and K's tile j + 1 are copied, used and given back together
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kSmem = (3 + 2 * kStages) * kTileBytes;  // Q's two, K's first, the pairs
  // tensor memory: S of both tiles, then O.  P lies over S, or behind O where there is
  // room for it.
  static constexpr bool kApart = D == 64;
  static constexpr uint32_t kColS = 0, kColO = 2 * kTile, kColP = kApart ? kColO + 2 * D : 0;
  static constexpr uint32_t kStepP = kApart ? kTile / 2 : kTile;  // from one tile's P to the other's
  static_assert(!kApart || kColP + 2 * kStepP <= 512, "tensor memory");
  static_assert(kSmem + 1024 <= 227 * 1024, "memory of an SM");
  static_assert(kSmem > 114 * 1024, "one block to an SM: each takes all of tensor memory");
};

struct Maps {
  CUtensorMap q, k, v;
};

// What a row's p lack: p = 2^(c (s - less) - base), for the maximum m of its scores so far
// (or, where the slack has let p grow, an earlier one).
struct Base {
  float less, base;
};
__device__ __forceinline__ Base base_of(float m, float c) {
  const float b = m == -INFINITY ? 0.0f : fmaf(m, c, kSlack);
  const bool large = fabsf(b) > kLarge;
  return Base{large ? m : 0.0f, large ? kSlack : b};
}
// The factor from p's of maximum `from` to those of `to`, `to` not below: by what was taken
// off them, with its roundings (by c m itself keys behind a move of m, or of another part,
// would weigh up to 4 % more or less than those before).  0 without a score so far.
__device__ __forceinline__ float rescale(float from, float to, float c) {
  const Base a = base_of(from, c), b = base_of(to, c);
  return from == -INFINITY ? 0.0f : ex2(fmaf(a.less - b.less, c, a.base - b.base));
}

// (l as it would be without the slack: near 1 the logarithm is at its most exact.)
__device__ __forceinline__ float log_of_sum(float m, float l, float scale) {
  const Base off = base_of(m, scale * kLog2e);
  return off.less * scale + fmaf(off.base - kSlack, kLn2, logf(l * 256.0f));
}

// What a block works on: 256 rows of a sequence.
struct Unit {
  int32_t live;        // 0: no more; from 2 on: O is moved to place live - 2 (48 bytes in all)
  int32_t q0, n_q;     // the sequence's queries
  int32_t k0, len;     // and keys
  int32_t tok0;        // the unit's first query, in the sequence
  int32_t head0, kv_head;
  int32_t tiles[2];    // of keys, for each tile of rows
  int32_t masked;      // from this one on some row does not reach a tile's keys all
  int32_t record;      // where a part of the keys is kept; -1: the unit has all of them

  // how many keys query `tok` of the sequence reaches
  __device__ __forceinline__ int32_t reach(int32_t tok, bool causal) const {
    return max(0, causal ? len + min(0, tok + 1 - n_q) : len);
  }
  __device__ __forceinline__ int32_t most() const { return max(tiles[0], tiles[1]); }
};

// The sequences of a packed batch, up to 64 of them, two to a lane: where they lie,
// and the first of their units, longest sequences (by keys) first.  Held by the warp
// that hands out units: looked up in memory, one load behind the other, a unit took
// some 3 us to find, and in the sequences' own order the longest came when it came.
struct Line {
  int32_t q0[2], n_q[2], k0[2], len[2], first[2];
};
constexpr int kLine = 64;

__device__ __forceinline__ int32_t units_of(int32_t n_q, int shift) { return (n_q >> shift) + ((n_q & ((1 << shift) - 1)) != 0); }

// `shift`: log2 of a unit's queries.  Also the tiles of keys that there are for an SM,
// about, where units may be cut (a.splits > 1): the same for all lanes.
__device__ void make_line(const AttentionArgs& a, int pack, int shift, int lane, Line& line, int32_t& per_sm) {
  float sum = 0.0f;
  for (int32_t n = lane; n < a.N && (a.splits > 1 || n < kLine); n += 32) {
    int64_t q0, q1, k0, k1;
    sequence_span(a.cu_q, a.N, a.Tq, n, q0, q1, a.err);
    sequence_span(a.cu_k, a.N, a.Tk, n, k0, k1, a.err);
    sum += static_cast<float>((q1 - q0 + (1 << shift) - 1) >> shift) * static_cast<float>((k1 - k0 + kTile - 1) / kTile);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (n >> 5 == e) {
        line.q0[e] = static_cast<int32_t>(q0);
        line.n_q[e] = static_cast<int32_t>(q1 - q0);
        line.k0[e] = static_cast<int32_t>(k0);
        line.len[e] = static_cast<int32_t>(k1 - k0);
      }
  }
#pragma unroll
  for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  per_sm = static_cast<int32_t>(fminf(sum * (a.heads / pack) / a.sm_count, 1e9f));
  if (!a.cu_q || a.N > kLine) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    line.first[e] = 0;
    if (lane + 32 * e >= a.N) line.n_q[e] = line.len[e] = line.q0[e] = line.k0[e] = 0;
  }
  for (int n = 0; n < a.N; ++n) {
    const int32_t len = __shfl_sync(0xffffffffu, n < 32 ? line.len[0] : line.len[1], n & 31);
    const int32_t units = units_of(__shfl_sync(0xffffffffu, n < 32 ? line.n_q[0] : line.n_q[1], n & 31), shift);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int32_t own = lane + 32 * e;
      if (len > line.len[e] || (len == line.len[e] && n < own)) line.first[e] += units;
    }
  }
}

// The unit of block `index`, for a whole warp; false: there is none.  Those with the
// most keys come first: the longest sequences, of a causal one its last queries.  With
// `splits`, one of a unit's parts: of at least kPartTiles tiles of keys and three
// quarters of what an SM has to do; `parts` is how many there are.  Of packed sequences
// all parts of a unit come side by side, longest units first (8 parts of prompts behind
// their keys: 103 us, 119 with all first parts first); of a uniform batch all first parts
// come first (512 queries behind 7000 keys: 65 us, 85 side by side, where blocks that had
// no part went from one to the next while the last units waited).
__device__ bool find_unit(const AttentionArgs& a, int pack, int shift, int32_t index, const Line& line,
                          int32_t per_sm, int lane, Unit& u, int32_t& parts) {
  int32_t part = 0;
  if (a.splits > 1) {
    part = a.cu_q ? index % a.splits : index / a.units;
    index = a.cu_q ? index / a.splits : index % a.units;
  }
  parts = 1;
  u.record = -1;
  const int head_blocks = a.heads / pack;
  const int32_t slot = index / head_blocks, hb = index - slot * head_blocks;
  int32_t block;
  if (a.cu_q && a.N <= kLine) {
    bool is[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      is[e] = slot >= line.first[e] && slot - line.first[e] < units_of(line.n_q[e], shift);
    const uint32_t in0 = __ballot_sync(0xffffffffu, is[0]), in1 = __ballot_sync(0xffffffffu, is[1]);
    if (!in0 && !in1) return false;
    const int from = __ffs(in0 ? in0 : in1) - 1;
    auto get = [&](const int32_t (&v)[2]) { return __shfl_sync(0xffffffffu, in0 ? v[0] : v[1], from); };
    block = slot - get(line.first);
    u.q0 = get(line.q0);
    u.n_q = get(line.n_q);
    u.k0 = get(line.k0);
    u.len = get(line.len);
  } else {
    int32_t seq;
    if (a.cu_q) {
      // sequence n's units lie in slots [cu[n] / queries + n, cu[n + 1] / queries + n + 1):
      // enough for its queries, wherever they start
      int32_t lo = 0, hi = a.N - 1;
      while (lo < hi) {
        const int32_t mid = lo + ((hi - lo + 1) >> 1);
        if (!kda_guard(mid, 1, static_cast<int64_t>(a.N) + 1, a.err)) break;
        if (static_cast<int64_t>(a.cu_q[mid] >> shift) + mid <= slot) lo = mid; else hi = mid - 1;
      }
      seq = lo;
      int32_t first = 0;
      if (kda_guard(lo, 1, static_cast<int64_t>(a.N) + 1, a.err)) first = a.cu_q[lo];
      const int64_t at = slot - (static_cast<int64_t>(first >> shift) + lo);
      block = at < 0 || at > 0x7fffff ? -1 : static_cast<int32_t>(at);
    } else {
      seq = slot % a.N;
      block = slot / a.N;
    }
    int64_t q0, q1, k0, k1;
    sequence_span(a.cu_q, a.N, a.Tq, seq, q0, q1, a.err);
    sequence_span(a.cu_k, a.N, a.Tk, seq, k0, k1, a.err);
    u.q0 = static_cast<int32_t>(q0);
    u.n_q = static_cast<int32_t>(q1 - q0);
    u.k0 = static_cast<int32_t>(k0);
    u.len = static_cast<int32_t>(k1 - k0);
  }
  const int32_t blocks = units_of(u.n_q, shift);
  if (block < 0 || block >= blocks) return false;
  u.live = 1;
  u.tok0 = (blocks - 1 - block) << shift;
  u.head0 = hb * pack;
  u.kv_head = u.head0 / (a.heads / a.kv_heads);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t first = u.tok0 + (i << (shift - 1)), last = min(first + (1 << (shift - 1)), u.n_q) - 1;
    const int32_t keys = last >= first ? u.reach(last, a.causal) : 0;
    u.tiles[i] = keys / kTile + (keys % kTile != 0);
  }
  if (a.splits > 1) {
    const int32_t most = u.most(), length = max(kPartTiles, static_cast<int32_t>(int64_t{3} * per_sm / 4));
    parts = max(1, min(a.splits, (most + length - 1) / length));
    if (part == 0 && lane == 0) a.parts[index] = PartInfo{parts, u.q0, u.n_q, u.len, u.tok0, u.head0};
    if (part >= parts) return false;
    if (parts > 1) {
      const int32_t count = (most + parts - 1) / parts, first = min(part * count, most);
      u.record = index * a.splits + part;
      u.k0 += first * kTile;
      u.len -= first * kTile;
#pragma unroll
      for (int i = 0; i < 2; ++i) u.tiles[i] = max(0, min(u.tiles[i] - first, count));
    }
  }
  u.masked = u.reach(u.tok0, a.causal) / kTile;
  return true;
}

// Places for what is moved out of tensor memory, taken by blocks of any call for as long
// as they run: there are no more blocks at a time than SMs, whatever the calls.
__device__ int g_places[kMaxPlaces];

__device__ __forceinline__ int take_place(int count) {
  for (uint32_t t = 0; t < 1u << 20; ++t) {
    const int at = static_cast<int>((blockIdx.x + t) % static_cast<uint32_t>(count));
    if (atomicCAS(&g_places[at], 0, 1) == 0) {
      __threadfence();  // (what a block before wrote there is behind it)
      return at;
    }
  }
  return -1;
}
__device__ __forceinline__ void give_place_back(int at) {
  __threadfence();
  atomicExch(&g_places[at], 0);
}

// Asks for a block of this grid that has not begun, to work on it in this one: 16
// bytes at `to`, counted on `bar`.
__device__ __forceinline__ void ask_for_block(uint4* to, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(to)),
               "r"(smem_u32(bar))
               : "memory");
}
// The answer: whether there was one, and its index.
__device__ __forceinline__ bool block_given(const uint4* from, int32_t& index) {
  uint32_t is, x;
  asm volatile(
      "{\n .reg .b128 a;\n .reg .pred p;\n .reg .b32 y, z, w;\n"
      " ld.shared.b128 a, [%2];\n mov.b32 %1, 0;\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n selp.u32 %0, 1, 0, p;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, a;\n}"
      : "=r"(is), "=r"(x)
      : "r"(smem_u32(from))
      : "memory");
  index = static_cast<int32_t>(x);
  return is != 0;
}

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

// This thread's row of O, with what was moved before added to it: moved to `sums` and set
// to 0, or kept.  (Eight columns at a time: seldom done, and code beside the softmax's loop.)
template <int D>
__device__ __forceinline__ void move_sums(uint32_t t_o, float* sums, float keep, bool add, bool move) {
#pragma unroll 1
  for (int k = 0; k < D; k += 8) {
    float o[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
        : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
        : "r"(t_o + k)
        : "memory");
    float4* const at = reinterpret_cast<float4*>(sums + k);
    if (add) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 x = __ldcg(at + e);
        o[4 * e] = fmaf(x.x, keep, o[4 * e]);
        o[4 * e + 1] = fmaf(x.y, keep, o[4 * e + 1]);
        o[4 * e + 2] = fmaf(x.z, keep, o[4 * e + 2]);
        o[4 * e + 3] = fmaf(x.w, keep, o[4 * e + 3]);
      }
    }
    if (move) {
#pragma unroll
      for (int e = 0; e < 2; ++e) __stcg(at + e, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.0f;
    }
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(o[0]), "f"(o[1]),
                 "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7]), "r"(t_o + k)
                 : "memory");
  }
  tmem_wait_st();
}

// 32 bytes, a whole sector, at a multiple of 32.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 0 for finite pairs of bf16, NaN in a half whose value is not.
__device__ __forceinline__ uint32_t times_zero(uint32_t pair, uint32_t sum) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(pair), "r"(0u), "r"(sum));
  return r;
}
__device__ __forceinline__ bool finite_bf16(uint32_t bits) { return (bits & 0x7f80u) != 0x7f80u; }

template <int D, bool MOVES>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ Maps maps, AttentionArgs a, int pack) {
  using G = Shape<D>;
  extern __shared__ __align__(1024) unsigned char smem[];  // Q's tiles, K's first, the ring
  __shared__ uint64_t q_full[2], q_empty[2], k_full, k_empty;
  __shared__ uint64_t kv_full[G::kStages], kv_empty[G::kStages], v_ok[G::kStages];
  __shared__ uint64_t s_full[2], s_empty[2], p_full[2][2], p_empty[2], o_full[2], o_empty[2], turn[2], drained[2];
  __shared__ uint64_t unit_full[2], unit_empty[2], given_full;
  __shared__ Unit units[2];
  __shared__ __align__(16) uint4 given;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_infinite;
  __shared__ int s_place;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = kRows / pack;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
      for (int h = 0; h < 2; ++h) mbar_init(&p_full[i][h], 4);
      mbar_init(&p_empty[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 4);
      mbar_init(&turn[i], 1);
      mbar_init(&drained[i], 1);
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], 11);  // the warps but the copying one
    }
    mbar_init(&k_full, 1);
    mbar_init(&k_empty, 2);
    mbar_init(&given_full, 1);
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 3);  // both tiles' products and the look through V
      mbar_init(&v_ok[i], 1);
    }
    mbar_fence_init();
    s_infinite = 0;
    s_place = -1;
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
  // The block's unit number n, for all warps but the copying one.
  auto get_unit = [&](uint32_t n, Unit& u) {
    if (!whole_warp(mbar_wait(&unit_full[n & 1], (n >> 1) & 1, kUnitPolls))) return false;
    u = units[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&unit_empty[n & 1]);
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == 0) {
      // ---- units and copies
      const bool issues = elect_one();
      auto copy = [&](unsigned char* to, const CUtensorMap* map, int32_t head, int32_t row, uint64_t* bar) {
#pragma unroll
        for (int b = 0; b < G::kBlocks; ++b) tma_load_3d(to + b * (kTile * 128), map, 64 * b, head, row, bar);
      };
      auto ask = [&]() {
        if (!issues) return;
        fence_proxy_async_smem();  // (the answer before has been read)
        ask_for_block(&given, &given_full);
      };
      int at = 0;
      uint32_t phase = 0, n = 0, asked = 0, k_uses = 0, q_uses[2] = {0, 0};
      bool ok = true, more = true;
      int32_t index = blockIdx.x, parts;
      const int shift = 31 - __clz(tokens);
      Line line;
      int32_t per_sm;
      make_line(a, pack, shift, lane, line, per_sm);
      while (more && ok) {
        if (index == 0 && a.cu_q) {
          check_cu_seqlens(a.cu_q, a.N, a.Tq, lane, 32, a.err);
          check_cu_seqlens(a.cu_k, a.N, a.Tk, lane, 32, a.err);
        }
        Unit u;
        const bool there = find_unit(a, pack, shift, index, line, per_sm, lane, u, parts);
        if (!there && a.splits > 1 && a.cu_q && index % a.splits == 0 && lane == 0) a.parts[index / a.splits].parts = 0;
        if (there) {
          if (MOVES && u.most() > kMoveTiles) {
            if (lane == 0 && s_place < 0) {
              s_place = take_place(a.sm_count);
              if (s_place < 0) timeout();
            }
            __syncwarp();
            u.live = 2 + s_place;
          }
          ok = whole_warp(mbar_wait(&unit_empty[n & 1], ((n >> 1) & 1) ^ 1));  // (the first round passes at once)
          if (!ok) break;
          if (lane == 0) {
            units[n & 1] = u;
            mbar_arrive(&unit_full[n & 1]);
          }
          ++n;
          const int32_t most = u.most();
          if (most > 0) {
            ok = whole_warp(mbar_wait(&k_empty, (k_uses++ & 1) ^ 1));
            if (!ok) break;
            if (issues) {
              mbar_arrive_expect_tx(&k_full, G::kTileBytes);
              copy(first_k, &maps.k, u.kv_head, u.k0, &k_full);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (u.tiles[i] == 0 || !ok) continue;
              ok = whole_warp(mbar_wait(&q_empty[i], (q_uses[i]++ & 1) ^ 1));
              if (ok && issues) {
                mbar_arrive_expect_tx(&q_full[i], G::kTileBytes);
                copy(smem + i * G::kTileBytes, &maps.q, u.head0, u.q0 + u.tok0 + i * (tokens / 2), &q_full[i]);
              }
            }
            if (!ok) break;
          }
          // The next unit is asked for when this one's copies come to an end: a block
          // that asked at its start would take units that other SMs are free for.
          // (4 x 263 queries of 8 heads behind 4000 keys each: 236 us instead of 121.)
          const int32_t ask_at = max(0, most - 1 - G::kStages);
          for (int32_t j = 0; j < most; ++j) {
            ok = whole_warp(mbar_wait(&kv_empty[at], phase ^ 1));
            if (!ok) break;
            if (j == ask_at) ask();
            if (issues) {
              unsigned char* const to = ring + at * (2 * G::kTileBytes);
              const bool next = j + 1 < most;
              mbar_arrive_expect_tx(&kv_full[at], next ? 2 * G::kTileBytes : G::kTileBytes);
              copy(to, &maps.v, u.kv_head, u.k0 + j * kTile, &kv_full[at]);
              if (next) copy(to + G::kTileBytes, &maps.k, u.kv_head, u.k0 + (j + 1) * kTile, &kv_full[at]);
            }
            if (++at == G::kStages) { at = 0; phase ^= 1; }
          }
          if (!ok) break;
          if (most == 0) ask();
        } else {
          ask();
        }
        ok = whole_warp(mbar_wait(&given_full, asked++ & 1));
        if (!ok) break;
        more = block_given(&given, index);
        __syncwarp();
      }
      if (ok) ok = whole_warp(mbar_wait(&unit_empty[n & 1], ((n >> 1) & 1) ^ 1));
      if (ok) {
        if (lane == 0) {
          units[n & 1].live = 0;
          mbar_arrive(&unit_full[n & 1]);
        }
        // the ring's last stages are given back (by commits behind the one that the output
        // waits for) before the block's memory goes
        for (int i = 0; i < G::kStages && ok; ++i) {
          ok = whole_warp(mbar_wait(&kv_empty[at], phase ^ 1));
          if (++at == G::kStages) { at = 0; phase ^= 1; }
        }
        if (!ok) timeout();
      } else {
        timeout();
        if (lane == 0) {  // (who waits for a unit need not wait on)
          units[n & 1].live = 0;
          mbar_arrive(&unit_full[n & 1]);
        }
        // the copies in flight land before the block's memory goes
        for (int i = 0; i < G::kStages; ++i) {
          mbar_wait(&kv_full[at], phase ^ 1, 1u << 16);
          if (++at == G::kStages) { at = 0; phase ^= 1; }
        }
        mbar_wait(&k_full, (k_uses & 1) ^ 1, 1u << 16);
        for (int i = 0; i < 2; ++i) mbar_wait(&q_full[i], (q_uses[i] & 1) ^ 1, 1u << 16);
        mbar_wait(&given_full, asked & 1, 1u << 16);  // (whether or not one is under way)
      }
    } else if (warp < 3) {
      // ---- products, a warp to a tile: O_i += P_i V and S_i of the next keys.
      // Where P_i lies over S_i, S_i comes behind O_i, and the warps take turns, so that
      // one tile's products run while the other's softmax does: left to themselves they
      // fall into step, both tiles' products at once and then both softmaxes (a block of
      // 128 tiles of keys took 177 us or 270, by chance; in turns 177).  Else S_i comes
      // first, while the softmax of the keys before is under way.
      const int i = warp - 1;
      const bool issues = elect_one();
      constexpr uint32_t id_s = make_idesc(kFmtBF16, kTile, kTile, false, false);
      constexpr uint32_t id_o = make_idesc(kFmtBF16, kTile, D, false, true);
      const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + i * G::kTileBytes), 16, 1024);
      const uint32_t t_s = tmem + G::kColS + i * kTile, t_o = tmem + G::kColO + i * D;
      const uint32_t t_p = tmem + G::kColP + i * G::kStepP;
      auto scores = [&](uint64_t k) {  // S_i = Q_i K^T
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t step = (s / 4) * (kTile * 128 >> 4) + (s % 4) * 2;
          mma_f16_ss(t_s, q_desc + step, k + step, id_s, s > 0);
        }
        mma_commit(&s_full[i]);
      };
      int at = 0;
      // (units with keys; with rows; tiles of keys, by S and by P; turns)
      uint32_t phase = 0, k_uses = 0, uses = 0, s_tile = 0, p_tile = 0, turns = 0;
      bool ok = true;
      Unit u;
      for (uint32_t n = 0;; ++n) {
        ok = get_unit(n, u);
        if (!ok || !u.live) break;
        const int32_t mine = i ? u.tiles[1] : u.tiles[0], most = u.most();
        if (most == 0) continue;
        // (waited for without rows too: no warp gives a tile back twice)
        ok = mbar_wait(&k_full, k_uses & 1);
        if (mine > 0) {
          ok = ok && mbar_wait(&q_full[i], uses & 1);
          if (G::kApart) ok = ok && mbar_wait(&s_empty[i], (s_tile & 1) ^ 1);
          if (ok && issues) {
            tc_fence_after();
            scores(smem_desc_sw128(smem_u32(first_k), 16, 1024));
            mma_commit(&k_empty);
            if (mine == 1) mma_commit(&q_empty[i]);
          }
          ++s_tile;
        } else if (ok && issues) {
          mbar_arrive(&k_empty);
        }
        ++k_uses;
        for (int32_t j = 0; j < most && ok; ++j) {
          // (looked through, where some row does not reach all of V's tile)
          ok = mbar_wait(j >= u.masked ? &v_ok[at] : &kv_full[at], phase);
          const uint32_t pair = smem_u32(ring + at * (2 * G::kTileBytes));
          const uint64_t v = smem_desc_sw128(pair, kTile * 128, 1024);
          auto next_scores = [&]() {
            if (j + 1 >= mine) return;
            if (G::kApart) ok = ok && mbar_wait(&s_empty[i], (s_tile & 1) ^ 1);
            if (ok && issues) {
              tc_fence_after();
              scores(smem_desc_sw128(pair + G::kTileBytes, 16, 1024));
              if (j + 2 == mine) mma_commit(&q_empty[i]);
            }
            ++s_tile;
          };
          if (G::kApart) next_scores();
          if (!G::kApart && j >= mine) ok = ok && mbar_wait(&turn[i], (turns & 1) ^ (i == 0));
          if (j < mine) {
            if (j == 0) ok = ok && mbar_wait(&o_empty[i], (uses & 1) ^ 1);  // the unit before has been read
#pragma unroll
            for (int part = 0; part < 2; ++part) {  // O_i += P_i V
              ok = ok && mbar_wait(&p_full[i][part], p_tile & 1);
              if (!G::kApart && part == 1) ok = ok && mbar_wait(&turn[i], (turns & 1) ^ (i == 0));
              if (ok && issues) {
                tc_fence_after();
#pragma unroll
                for (int s = part * 4; s < part * 4 + 4; ++s)
                  mma_f16_ts(t_o, t_p + 8 * s, v + s * (2048 >> 4), id_o, j > 0 || s > 0);
              }
            }
            ++p_tile;
            if (ok && issues) {
              if (G::kApart) mma_commit(&p_empty[i]);
              if (j + 1 == mine) mma_commit(&o_full[i]);
            }
            if (!G::kApart) next_scores();
          }
          if (ok && issues) {
            if (!G::kApart) mbar_arrive(&turn[1 - i]);
            mma_commit(&kv_empty[at]);
          }
          ++turns;
          if (++at == G::kStages) { at = 0; phase ^= 1; }
        }
        if (mine > 0) ++uses;
        ok = whole_warp(ok);
        if (!ok) break;
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
      Unit u;
      for (uint32_t n = 0; ok; ++n) {
        ok = get_unit(n, u);
        if (!ok || !u.live) break;
        const int32_t most = u.most();
        for (int32_t j = 0; j < most; ++j) {
          ok = whole_warp(mbar_wait(&kv_full[at], phase));
          if (!ok) break;
          if (j >= u.masked) {
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
              s_infinite = 1;  // (from now on; rows without such values are not changed by it)
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
      }
      if (!ok && lane == 0) timeout();
    }
  } else {
    // ---- softmax: a thread to a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const int i = (warp - 4) >> 2, quad = warp & 3;
    const int row = 32 * quad + lane;  // of the tile
    const uint32_t t_s = tmem_addr(tmem, 32 * quad, G::kColS + i * kTile);
    const uint32_t t_o = tmem_addr(tmem, 32 * quad, G::kColO + i * D);
    const uint32_t t_p = tmem_addr(tmem, 32 * quad, G::kColP + i * G::kStepP);
    const float c = a.scale * kLog2e;
    // this row's sums moved out of tensor memory, then the maximum they were taken with and l
    auto sums_of = [&](int32_t place) { return a.moved + (static_cast<int64_t>(place) * kRows + i * kTile + row) * (D + 4); };
    uint32_t uses = 0, tile = 0;
    bool ok = true;
    Unit u;
    for (uint32_t n = 0;; ++n) {
      ok = get_unit(n, u);
      if (!ok || !u.live) break;
      const int32_t tok = u.tok0 + i * (tokens / 2) + row / pack;
      const int32_t head = u.head0 + row % pack;
      const bool valid = tok < u.n_q;
      const int32_t reach = valid ? u.reach(tok, a.causal) : 0;
      const int32_t tiles = i ? u.tiles[1] : u.tiles[0];
      // all of the tile's rows reach these tiles whole
      const int32_t whole = u.reach(u.tok0 + i * (tokens / 2), a.causal) / kTile;
      float m = -INFINITY, l = 0.0f;
      for (int32_t j = 0; j < tiles; ++j) {
        ok = whole_warp(mbar_wait(&s_full[i], tile & 1));
        if (!ok) break;
        tc_fence_after();
        float s[kTile];
        tmem_row(t_s, s);
        if (G::kApart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[i]);
        }
        if (j >= whole) {
          const int32_t limit = reach - j * kTile;
#pragma unroll
          for (int k = 0; k < kTile; ++k)
            if (k >= limit) s[k] = -INFINITY;
        }
        float top[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) top[k] = fmaxf(s[2 * k], s[2 * k + 1]);
#pragma unroll
        for (int k = 16; k < kTile; k += 2) top[k / 2 % 8] = fmaxf(fmaxf(top[k / 2 % 8], s[k]), s[k + 1]);
        const float most = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])),
                                 fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
        // The products of the tile before are done: S came behind them, or is waited for here.
        if (G::kApart) {
          ok = whole_warp(mbar_wait(&p_empty[i], (tile & 1) ^ 1));
          if (!ok) break;
          tc_fence_after();
        }
        if (j == 0) m = most;
        float base = m == -INFINITY ? 0.0f : fmaf(m, c, kSlack);
        const bool full = MOVES && j > 0 && j % kMoveTiles == 0 && u.live >= 2;  // (the same for all)
        if (__any_sync(0xffffffffu, (most - m) * c > kSlack || fabsf(base) > kLarge || full)) {
          if (full) {
            float* const sums = sums_of(u.live - 2);
            float2 ml = make_float2(-INFINITY, 0.0f);
            if (j > kMoveTiles) ml = __ldcg(reinterpret_cast<const float2*>(sums + D));
            const float keep = rescale(ml.x, m, c);
            move_sums<D>(t_o, sums, keep, j > kMoveTiles, true);
            __stcg(reinterpret_cast<float2*>(sums + D), make_float2(m, fmaf(ml.y, keep, l)));
            l = 0.0f;
          }
          const float next = fmaxf(m, most);
          if (j > 0 && __any_sync(0xffffffffu, next != m)) {
            const float keep = next == -INFINITY ? 1.0f : rescale(m, next, c);
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
          m = next;
          const Base off = base_of(m, c);
          base = off.base;
          if (__any_sync(0xffffffffu, off.less != 0.0f)) {
#pragma unroll
            for (int k = 0; k < kTile; ++k) s[k] -= off.less;
          }
        }
        ++tile;
        const f32x2 cc = pack2(c, c), less = pack2(-base, -base);
        f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
        auto hand_over = [&](int part) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[i][part]);
        };
#pragma unroll
        for (int e = 0; e < kTile / 2; ++e) {
          float lo, hi;
          unpack2(fma2(pack2(s[2 * e], s[2 * e + 1]), cc, less), lo, hi);
          lo = ex2(lo);
          hi = ex2(hi);
          sum[e % 2] = add2(sum[e % 2], pack2(lo, hi));
          s[e] = __uint_as_float(pack2_bf16(lo, hi));
          // P in two parts.  The first is handed over once its store has had some time
          // (at once: 195 us instead of 177 for 128 tiles).
          if (e == 31) tmem_st32(t_p, s);
          if (e == 31 + kHandOver) hand_over(0);
          if (e == 63) tmem_st32(t_p + 32, s + 32);
        }
        hand_over(1);
        float lo, hi;
        unpack2(add2(sum[0], sum[1]), lo, hi);
        l += lo + hi;
      }
      if (!ok) break;
      // ---- output
      if (tiles > 0) {
        ok = whole_warp(mbar_wait(&o_full[i], uses++ & 1));
        if (!ok) break;
        tc_fence_after();
      }
      if (MOVES && u.live >= 2 && tiles > kMoveTiles) {
        float* const sums = sums_of(u.live - 2);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(sums + D));
        const float keep = rescale(ml.x, m, c);
        move_sums<D>(t_o, sums, keep, true, false);
        l = fmaf(ml.y, keep, l);
      }
      const bool part = u.record >= 0;
      const float scale = part ? 1.0f : reach > 0 ? 1.0f / l : 0.0f;
      const int64_t at = (static_cast<int64_t>(u.q0) + tok) * a.ld_out + static_cast<int64_t>(head) * D;
      const int64_t extent = (a.Tq - 1) * a.ld_out + static_cast<int64_t>(a.heads) * D;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        if (tiles > 0) {
          tmem_part(t_o + k, o);
          if (k + 32 == D) {  // the next unit's products may write
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[i]);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = reach > 0 ? o[e] * scale : 0.0f;
        if (s_infinite) {  // values taken out of V's tiles, for rows that reach them
          for (int32_t t = u.masked * kTile; t < min(reach, tiles * kTile); ++t) {
            const int64_t from = (static_cast<int64_t>(u.k0) + t) * a.ld_v + static_cast<int64_t>(u.kv_head) * D + k;
            if (!kda_guard(from, 32, (a.Tk - 1) * a.ld_v + static_cast<int64_t>(a.kv_heads) * D, a.err)) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t bits = a.v[from + e].bits;
              if (!finite_bf16(bits)) o[e] += bf16_to_f32(static_cast<uint16_t>(bits));
            }
          }
        }
        if (part) {
          float* to = a.part_out + (static_cast<int64_t>(u.record) * kRows + i * kTile + row) * D + k;
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) w[x] = __float_as_uint(o[e + x]);
              store32(to + e, w);
            }
          }
        } else if (valid && kda_guard(at + k, 32, extent, a.err)) {
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = pack2_bf16(o[e + 2 * x], o[e + 2 * x + 1]);
            if (a.sectors) {
              store32(a.out + at + k + e, w);
            } else {
              *reinterpret_cast<uint4*>(a.out + at + k + e) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(a.out + at + k + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      const int64_t e = (static_cast<int64_t>(u.q0) + tok) * a.heads + head;
      if (part) {
        if (valid) a.part_ml[static_cast<int64_t>(u.record) * kRows + i * kTile + row] = make_float2(m, l);
      } else if (a.lse && valid && kda_guard(e, 1, a.Tq * a.heads, a.err))
        a.lse[e] = reach > 0 ? log_of_sum(m, l, a.scale) : -INFINITY;
    }
    if (!ok && lane == 0) timeout();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (MOVES && threadIdx.x == 0 && s_place >= 0) give_place_back(s_place);
}

// The parts of units whose keys several blocks shared: kJoinRows rows of a unit to a
// block, four channels (or two) of a row to a lane.  The parts go to the block's warps
// in turn (SHARED), or, where there are few, all to the warp of a row.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinRows = 8;

template <int D, bool SHARED>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttentionArgs a, int pack) {
  constexpr int kPer = D / 32, kMine = SHARED ? kJoinRows : kJoinRows / kJoinWarps;  // rows of a warp
  __shared__ float s_o[SHARED ? kJoinWarps : 1][kJoinRows][D];
  __shared__ float2 s_ml[SHARED ? kJoinWarps : 1][kJoinRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t unit = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the first kernel's end
  const PartInfo u = a.parts[unit];
  const int32_t parts = u.parts;
  if (parts < 2) return;
  // (a unit that was not reached because a wait ran out has anything here)
  if (parts > a.splits || u.q0 < 0 || u.n_q > a.Tq - u.q0 || u.tok0 < 0 || u.head0 < 0 || u.head0 > a.heads - pack) return;
  if (u.tok0 >= u.n_q) return;
  const int32_t queries = u.n_q - u.tok0;  // from the unit's first one on
  if (static_cast<int32_t>(blockIdx.y) * kJoinRows / pack >= queries) return;
  const int row0 = blockIdx.y * kJoinRows + (SHARED ? 0 : warp * kMine);
  const int64_t first = static_cast<int64_t>(unit) * a.splits * kRows + row0;
  const float c = a.scale * kLog2e;
  // (rows behind a sequence's last query hold anything, and go nowhere)
  float m[kMine], l[kMine], o[kMine][kPer];
#pragma unroll
  for (int r = 0; r < kMine; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[r][e] = 0.0f;
  }
  if constexpr (SHARED) {
    if (parts <= kJoinWarps) {  // a part to a warp: as it is
      const int64_t at = first + static_cast<int64_t>(warp) * kRows;
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        if (warp >= parts) break;
        load_n<kPer>(a.part_out + (at + r) * D + kPer * lane, o[r]);
        const float2 ml = a.part_ml[at + r];
        m[r] = ml.x;
        l[r] = ml.y;
      }
    } else {
      // This warp's parts: the maximum and the weight of a part by a lane, its sums by all
      // lanes.  (A weight computed by all lanes for each part and row, and sums rescaled from
      // part to part: 32 queries of 8 heads over 65,536 keys took 47 us instead of 32.  For few
      // parts that is the faster way, 9.1 us instead of 9.6 for 128 units of two.)
      auto part_ml = [&](int32_t p, int r) {
        return p < parts ? a.part_ml[first + static_cast<int64_t>(p) * kRows + r] : make_float2(-INFINITY, 0.0f);
      };
      float2 ml[kMine];
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        ml[r] = part_ml(warp + kJoinWarps * lane, r);
        m[r] = ml[r].x;
      }
      for (int32_t p = warp + kJoinWarps * (lane + 32); p < parts; p += 32 * kJoinWarps) {
#pragma unroll
        for (int r = 0; r < kMine; ++r) m[r] = fmaxf(m[r], part_ml(p, r).x);
      }
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
#pragma unroll
        for (int w = 16; w; w /= 2) m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], w));
      }
      for (int32_t p0 = warp; p0 < parts; p0 += 32 * kJoinWarps) {
        float weight[kMine];
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
          if (p0 != warp) ml[r] = part_ml(p0 + kJoinWarps * lane, r);
          weight[r] = rescale(ml[r].x, m[r], c);
          l[r] = fmaf(ml[r].y, weight[r], l[r]);
        }
        const int32_t count = min(32, (parts - p0 + kJoinWarps - 1) / kJoinWarps);
#pragma unroll 2
        for (int32_t i = 0; i < count; ++i) {
          const int64_t at = first + static_cast<int64_t>(p0 + kJoinWarps * i) * kRows;
#pragma unroll
          for (int r = 0; r < kMine; ++r) {
            float v[kPer];
            load_n<kPer>(a.part_out + (at + r) * D + kPer * lane, v);
            const float w = __shfl_sync(0xffffffffu, weight[r], i);
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[r][e] = fmaf(v[e], w, o[r][e]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
#pragma unroll
        for (int w = 16; w; w /= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
      }
    }
  } else {
#pragma unroll 2
    for (int32_t p = 0; p < parts; ++p) {
      const int64_t at = first + static_cast<int64_t>(p) * kRows;
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        float v[kPer];
        load_n<kPer>(a.part_out + (at + r) * D + kPer * lane, v);
        const float2 ml = a.part_ml[at + r];
        const float next = fmaxf(m[r], ml.x), keep = rescale(m[r], next, c), w = rescale(ml.x, next, c);
        m[r] = next;
        l[r] = fmaf(ml.y, w, l[r] * keep);
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[r][e] = fmaf(v[e], w, o[r][e] * keep);
      }
    }
  }
  auto put = [&](int row, int r) {
    if (row / pack >= queries) return;
    const int32_t tok = u.tok0 + row / pack, head = u.head0 + row % pack;
    const bool any = (a.causal ? u.len + min(0, tok + 1 - u.n_q) : u.len) > 0;
    const float scale = 1.0f / l[r];
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[r][e] = any ? o[r][e] * scale : 0.0f;
    const int64_t at = (static_cast<int64_t>(u.q0) + tok) * a.ld_out + static_cast<int64_t>(head) * D + kPer * lane;
    if (kda_guard(at, kPer, (a.Tq - 1) * a.ld_out + static_cast<int64_t>(a.heads) * D, a.err))
      store_n<kPer>(a.out + at, o[r]);
    const int64_t e = (static_cast<int64_t>(u.q0) + tok) * a.heads + head;
    if (a.lse && lane == 0 && kda_guard(e, 1, a.Tq * a.heads, a.err))
      a.lse[e] = any ? log_of_sum(m[r], l[r], a.scale) : -INFINITY;
  };
  if constexpr (SHARED) {
#pragma unroll
    for (int r = 0; r < kMine; ++r) {
      store_n<kPer>(&s_o[warp][r][kPer * lane], o[r]);
      if (lane == 0) s_ml[warp][r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    // a row to a warp, in the parts' order of warps, a warp's weight by a lane
    const float2 of = s_ml[lane % kJoinWarps][warp];
    m[0] = of.x;
#pragma unroll
    for (int w = kJoinWarps / 2; w; w /= 2) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], w));
    const float weight = rescale(of.x, m[0], c), part_l = of.y * weight;
    l[0] = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[0][e] = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      float v[kPer];
      load_n<kPer>(&s_o[w][warp][kPer * lane], v);
      l[0] += __shfl_sync(0xffffffffu, part_l, w);
      const float by = __shfl_sync(0xffffffffu, weight, w);
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[0][e] = fmaf(v[e], by, o[0][e]);
    }
    put(row0 + warp, 0);
  } else {
#pragma unroll
    for (int r = 0; r < kMine; ++r) put(row0 + r, r);
  }
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

// Tiles of keys that a sequence may have (a packed one: all there are).
int64_t most_tiles(const AttentionArgs& a) { return ((a.cu_k ? a.Tk : a.Tk / a.N) + kTile - 1) / kTile; }

template <int D, bool MOVES>
kda_status run(AttentionArgs a, cudaStream_t s, cudaError_t& e) {
  using G = Shape<D>;
  // heads of a group side by side in a tile: the largest power of two in the group
  const int group = a.heads / a.kv_heads, pack = std::min(group & -group, kTile);
  Maps maps;
  memset(&maps, 0, sizeof maps);
  e = cudaErrorInvalidValue;
  if (!encode(&maps.q, a.q, D, a.heads, a.Tq, a.ld_q, static_cast<uint32_t>(pack),
              static_cast<uint32_t>(kTile / pack)))
    return KDA_OK;
  // (without keys no tile of them is copied)
  if (a.Tk > 0 && (!encode(&maps.k, a.k, D, a.kv_heads, a.Tk, a.ld_k, 1, kTile) ||
                   !encode(&maps.v, a.v, D, a.kv_heads, a.Tk, a.ld_v, 1, kTile)))
    return KDA_OK;
  constexpr auto kern = attention_kernel<D, MOVES>;
  // a build that launches with fewer registers could never give the rows' warps
  // their share: it is not launched
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  e = cudaErrorInvalidConfiguration;
  if (regs < kLaunchRegs) return KDA_OK;
  const int64_t tokens = kRows / pack;
  const int64_t slots = a.cu_q ? a.Tq / tokens + a.N : (a.Tq / a.N + tokens - 1) / tokens * a.N;
  const int64_t units = slots * (a.heads / pack);
  if (units > 0x7fffffffLL) return KDA_OK;
  // With fewer units than two for each SM, the longest one's keys may keep its SM busy
  // when the others are done: units may be cut into parts then, as many blocks as eight
  // for each SM, no more parts than a sequence can have.  (8 x 263 queries of 32 heads
  // behind 3900 keys on average, 280 units: 120 us whole.)
  const int64_t longest = most_tiles(a);
  if (units < 2 * a.sm_count) {
    int64_t splits = std::min(8 * a.sm_count / units, longest / kPartTiles);
    if (!a.cu_q) {
      // No more than find_unit will make of these lengths; none where each unit has an SM
      // and about the mean's length.  (152 units of 128 tiles of keys: 183 us whole, 227 in
      // halves.)
      const int64_t n_q = a.Tq / a.N, len = a.Tk / a.N, work = units * longest / a.sm_count;
      const int64_t length = std::max<int64_t>(kPartTiles, 3 * work / 4);
      const double mean = !a.causal ? len : n_q <= len ? len - 0.5 * n_q : 0.5 * len * len / n_q;
      splits = std::min(splits, (longest + length - 1) / length);
      if (units <= a.sm_count && len <= 1.25 * mean * units / a.sm_count) splits = 1;
    }
    a.splits = static_cast<int32_t>(std::max<int64_t>(1, splits));
    a.units = static_cast<int32_t>(units);
  }
  void* ws = nullptr;
  if (MOVES && a.sm_count > kMaxPlaces) return KDA_OK;
  if (a.splits > 1 || MOVES) {
    const size_t rows = a.splits > 1 ? static_cast<size_t>(units) * a.splits * kRows : 0;
    const size_t places = MOVES ? static_cast<size_t>(a.sm_count) * kRows * (D + 4) : 0;
    const kda_status st = workspace_alloc((places + rows * D) * sizeof(float) + rows * sizeof(float2) +
                                              (rows ? units * sizeof(PartInfo) : 0), s, &ws);
    if (st != KDA_OK) return st;
    float* const at = static_cast<float*>(ws);
    if (MOVES) a.moved = at;
    if (a.splits > 1) {
      a.part_out = at + places;
      a.part_ml = reinterpret_cast<float2*>(a.part_out + rows * D);
      a.parts = reinterpret_cast<PartInfo*>(a.part_ml + rows);
    }
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(G::kSmem));
  if (e == cudaSuccess) {
    kern<<<static_cast<unsigned>(units * a.splits), kThreads, G::kSmem, s>>>(maps, a, pack);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.splits > 1) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(units), kRows / kJoinRows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    e = a.splits > kJoinWarps ? cudaLaunchKernelEx(&cfg, join_kernel<D, true>, a, pack)
                              : cudaLaunchKernelEx(&cfg, join_kernel<D, false>, a, pack);
  }
  if (ws) {
    const cudaError_t ef = cudaFreeAsync(ws, s);
    if (e == cudaSuccess) e = ef;
  }
  return KDA_OK;
}

}  // namespace

kda_status launch_attention(const AttentionArgs& a, cudaStream_t s, cudaError_t& e) {
  prof_begin(s, "kda_attention_fwd");
  const bool moves = most_tiles(a) > kMoveTiles;
  const kda_status st = a.d == 128 ? (moves ? run<128, true>(a, s, e) : run<128, false>(a, s, e))
                                   : (moves ? run<64, true>(a, s, e) : run<64, false>(a, s, e));
  prof_end(s, "kda_attention_fwd");
  return st;
}

}  // namespace kda
