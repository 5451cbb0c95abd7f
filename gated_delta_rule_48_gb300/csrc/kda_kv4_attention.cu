// A few query tokens of each sequence over the cache in 4 bits.
//
//   x = c sum_g s_tg sum_{c in g} q_c n_tc,   p = 2^(x - m - 8),   o_c = sum_t p_t s'_tg n'_tc / sum_t p_t
//
// with c = scale log2 e, a key's scales s and codes n, a value's s' and n', per
// group g of 32 channels.
//
// Bound: the cache's bytes (1.125 per channel of a token and head), and beside
// them the latency of taking codes apart.  A step is a token or a few, so
// that there are 1 to 16 query rows (tokens x heads of a group) for each key: too
// few for tensor memory's 128 lanes, and codes would have to go through shared
// memory as bf16 first.  So the products are warp-wide ones (m16n8k16) with the
// cache as the 16-row operand, straight from the registers it was unpacked into:
// S^T = K Q^T (16 tokens x 8 query rows), O^T += V^T P^T (16 channels x 8 query
// rows).
//   - A key's code n + 8 in the low bits of a 16-bit half is the f16 number
//     (n + 8) 2^-24 as it stands (a subnormal one), in bits 4..7 16 times that: two
//     codes to an AND, and four bits' shift less.  The queries' bf16 values are f16
//     ones after a power of two for each row (what is 2^28 times smaller than a row's
//     largest value may round: odd channels are read 16 times as large).  The 8 goes away with the accumulator's first
//     value, one product of the groups' scales with -8 2^-24 sum_{c in g} q_c in four
//     bf16 parts.  (So a score's rounding goes by the sums of |q| (|n| + 16), not of
//     |q n|: 2^-23 of them a step.)
//   - A value's code is, as it stands, the bf16 number (n + 8) 2^-133 or 16 times
//     that; one multiply-add makes it n 2^-6 exactly.  p, which it is multiplied by,
//     needs the range of bf16.  (Leaving the 8 in and taking it off by a product with
//     a constant was slower, 342 instead of 325 us, and not exact where p n is small.)
//   - Scales never touch the codes: a group's part of a score is scaled in 32
//     bits, and a value's scale is multiplied into p, which is rounded to bf16
//     then (as in kda_attention_fwd; the rounding of p itself is left out).
//   - The order of codes in a row is that in which a lane needs them: 16 bytes of
//     a key, 8 of a value, each with channels of all groups.
//
// Work: the slices of 32 positions of all (sequence, key head, 16 query rows)
// form one line that is cut into equal parts, one per block, whatever the
// sequences' lengths.  A block goes through its part unit by unit, its warps a
// slice each in turn, with copies a few slices ahead; units that lie in one block
// are written out, the parts of others combined by a second launch.  Where units are
// short its warps have parts of their own instead (1000 sequences of 64 positions:
// 124 us shared, 69 apart).
//
// The tensor core adds to a sum with what lies some 2^-25 below it cut off: of 2^20
// positions of like weights to a warp the sum came out 0.5 % too small.  So every 2^17
// positions a warp moves its sums to memory, adds them there, and begins again at 0.  That
// is a kernel of its own (MOVES), for tables of so many positions: others lost 1 to 3 % by
// the code (64 x 4096 with drafts of 4: 111 us instead of 108).
//
// Measured, 8 key heads of 128 channels: 256 sequences of 4096 positions on average
// and 32 query heads 244 us, 5.0 TB/s (73 % of a copy; issue slots 57 %, the ALU pipe
// 50 %: about 300 instructions for 16 positions, three warps to a scheduler and no pipe
// saturated: latency); one of 131,072 45 us, 3.4 TB/s, of
// which some 15 are launches, first copies and the combination; 16 columns instead
// of 8 107 us instead of 75 (64 x 4096): the products, the softmax and their registers,
// two blocks an SM for three.
// The next slice's scores before this one's values, so that one chain covers the
// other, were slower (253 us instead of 243): its copies have a slice less of time.
#include <string.h>

#include <cmath>

#include <algorithm>
#include <type_traits>

#include "kda_attention.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

using sm100::smem_u32;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlice = 32;        // positions of a slice: two halves, for a page may end between them
constexpr int kHalf = 16;
constexpr int kDepth = 3;         // slices of a warp in flight
constexpr int kSoloSlices = 16;   // of a unit, on average: up to as many, a warp to a unit
constexpr int kMoveSlices = 4096; // of a warp in a unit, after which its sums are moved
constexpr float kLowest = -3e38f; // a maximum of nothing (-infinity less itself is NaN)
constexpr float kSlack = 8.0f;    // log2 of how far p may grow, from 2^-8 to 1 (p s' is never above s')
constexpr float kLn2 = 0.6931471805599453f;

// Where a block's part of a unit lies that is not whole.
struct Meta {
  int32_t last;       // the last block that has a part (-1: nothing to combine)
  int32_t slot;       // of the first block's part
  int32_t seq, head, col0;
  int32_t visible;    // positions the first query reaches
  int32_t solo;       // parts are of warps, not of blocks
  int32_t pad;
};

template <int G, int NT>
struct Shape {
  static constexpr int D = 32 * G, kCols = 8 * NT;
  static constexpr int kRow = 16 * G;                           // bytes of a row of codes
  static constexpr int kPitchV = kRow + 16;                     // so that a warp's reads meet no bank twice
  static constexpr int kScaleBytes = kSlice * 2 * G;            // of keys, of values
  static constexpr int kStage = kSlice * (kRow + kPitchV) + 2 * kScaleBytes;
  static constexpr int kRing = kWarps * kDepth * kStage;
  static constexpr int kParts = kWarps * kCols * (D + 4) * 4;   // the warps' results, over the ring
  static constexpr int kSmem = kRing > kParts ? kRing : kParts;
  static constexpr int kRecord = kCols * (D + 3);               // floats of a part: o, then m and l, then cc
};

// d += A B (or d = A B), bf16 operands.
template <bool ADD = true>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (ADD)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// 8 x 8 values of 16 bits, turned.
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// d = A B (or d += A B), f16 operands.
template <bool ADD>
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (ADD)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Codes n + 8 of both halves (bits 0..3, or 4..7 with HIGH) as n 2^-6 in bf16, exactly:
// bits 0..7 of a bf16 number without the others are a whole number of 2^-133, also
// where bit 7 makes it a normal one.
template <bool HIGH>
__device__ __forceinline__ uint32_t whole_numbers(uint32_t w) {
  uint32_t r;
  // (times 2^127 or 2^123, less 8 2^-6)
  asm("fma.rn.bf16x2 %0, %1, %2, %3;"
      : "=r"(r)
      : "r"(w & (HIGH ? 0x00f000f0u : 0x000f000fu)), "r"(HIGH ? 0x7d007d00u : 0x7f007f00u), "r"(0xbe00be00u));
  return r;
}
template <int N>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ float half_of(uint32_t pair, int i) {
  return __uint_as_float(i ? pair & 0xffff0000u : pair << 16);
}

// (16 columns at three blocks an SM spill 0.6 KB a thread: 64 x 4096 with a draft of 4 took
// 122 us instead of 107.)
template <int G, int NT, bool MOVES>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
kv4_attention_kernel(Kv4AttentionArgs a, float* records, Meta* metas) {
  using S = Shape<G, NT>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_start[kWarps][2];  // of a part's first slice: the sequence, slices before it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, j = lane & 3;
  const Kv4Pages& p = a.pages;
  const int group = a.heads / p.heads, cols = a.tokens * group;
  const int blocks_c = (cols + S::kCols - 1) / S::kCols;
  const int64_t per_seq = static_cast<int64_t>(p.heads) * blocks_c;  // units of a sequence
  const int64_t n_rows = static_cast<int64_t>(a.N) * a.tokens;
  // No more positions than the table has pages for (what is beyond is an error), and
  // none whose number could pass 32 bits a few slices ahead.
  const int64_t capacity = min(static_cast<int64_t>(p.width) << p.page_shift, int64_t{0x7ffff000});
  auto len_of = [&](int64_t n) -> int64_t {
    return kda_guard(n, 1, a.N, a.err) ? min(static_cast<int64_t>(max(a.seq_lens[n], 0)), capacity) : 0;
  };
  auto slices_of = [&](int64_t n) { return (len_of(n) + kSlice - 1) / kSlice; };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // sequences of no positions: zeros
  auto write_zeros = [&]() {
    const int width = a.heads * (S::D / 8);  // pieces of 16 bytes of a token
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
      if (len_of(n) > 0) continue;
      for (int64_t row = n * a.tokens; row < (n + 1) * a.tokens; ++row)
        for (int e = threadIdx.x; e < width; e += kThreads)
          if (kda_guard(row * a.ld_out + 8 * e, 8, (n_rows - 1) * a.ld_out + a.heads * S::D, a.err))
            *reinterpret_cast<uint4*>(a.out + row * a.ld_out + 8 * e) = make_uint4(0, 0, 0, 0);
      if (!a.lse) continue;
      for (int64_t e = n * a.tokens * a.heads + threadIdx.x; e < (n + 1) * a.tokens * a.heads; e += kThreads)
        if (kda_guard(e, 1, n_rows * a.heads, a.err)) a.lse[e] = -INFINITY;
    }
  };

  // ---- this block's part of the line (or the parts of its warps)
  const int64_t chunk = (a.N + kThreads - 1) / kThreads;
  const int64_t c0 = min(chunk * threadIdx.x, static_cast<int64_t>(a.N)), c1 = min(c0 + chunk, static_cast<int64_t>(a.N));
  int64_t own = 0;
  for (int64_t n = c0; n < c1; ++n) {
    own += slices_of(n);
    if (blockIdx.x == 0 && kda_guard(n, 1, a.N, a.err) && a.seq_lens[n] > capacity) atomicOr(a.err, kDevErrPage);
  }
  int64_t scan = own;
#pragma unroll
  for (int w = 1; w < 32; w *= 2) {
    const int64_t up = __shfl_up_sync(0xffffffffu, scan, w);
    if (lane >= w) scan += up;
  }
  if (lane == 31) s_sum[warp] = scan;
  __syncthreads();
  int64_t before = scan - own, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  const int64_t all = total * per_seq;
  // Short units (up to kSoloSlices slices on average) go to single warps, each with a
  // part of the line of its own: shared by a block's warps, most of a unit's time is
  // spent before its first slice and behind its last.
  // (Never with so many slices to a warp that its sums would have to be moved.)
  const bool solo = all <= kSoloSlices * (per_seq * a.N) && all <= int64_t{kMoveSlices} * kWarps * gridDim.x;
  const int workers = solo ? kWarps : 1, me = solo ? warp : 0;
  const int64_t all_workers = static_cast<int64_t>(gridDim.x) * workers;
  // no more parts than have two slices for each warp
  const int64_t used = max(int64_t{1}, min(all_workers, all >> (solo ? 1 : 3)));
  static_assert(kWarps == 4, "two slices for each warp");
  // part n begins at all * n / used
  const bool small = all >> 32 == 0;  // (a division of 64 bits takes some hundred instructions)
  const int64_t share = small ? static_cast<uint32_t>(all) / static_cast<uint32_t>(used) : all / used;
  const uint32_t over = static_cast<uint32_t>(all - share * used);
  auto part_at = [&](int64_t n) {
    return n < used ? share * n + over * static_cast<uint32_t>(n) / static_cast<uint32_t>(used) : all;
  };
  const int64_t b = static_cast<int64_t>(blockIdx.x) * workers + me;
  const int64_t part0 = part_at(b), part1 = part_at(b + 1);
  if (threadIdx.x < kWarps) {
    Meta none;
    none.last = -1;
    none.solo = solo;
    metas[blockIdx.x * kWarps + threadIdx.x] = none;
  }
  for (int w = 0; w < workers; ++w) {
    const int64_t from = workers == 1 ? part0 : part_at(static_cast<int64_t>(blockIdx.x) * workers + w);
    if (from >= before * per_seq && from < (before + own) * per_seq) {
      int64_t n = c0, at = before, count = slices_of(n);
      while ((at + count) * per_seq <= from) {
        at += count;
        count = slices_of(++n);
      }
      s_start[w][0] = n;
      s_start[w][1] = at;
    }
  }
  __syncthreads();
  if (part0 >= part1) {
    write_zeros();
    return;
  }
  int64_t seq = s_start[me][0], seq_first = s_start[me][1] * per_seq;  // the sequence's first slice of the line

  auto work = [&](auto SOLO_c) {
  constexpr bool SOLO = decltype(SOLO_c)::value;
  constexpr int32_t stride = (SOLO ? 1 : kWarps) * kSlice;  // this warp's slices of a unit: first + mine0, and so on
  const int mine0 = SOLO ? 0 : warp;
  unsigned char* const ring = smem + warp * (kDepth * S::kStage);
  const float c = a.scale * kLog2e;
  for (int64_t at = part0; at < part1;) {
    int64_t slices = slices_of(seq);
    while (at >= seq_first + slices * per_seq) {
      seq_first += slices * per_seq;
      slices = slices_of(++seq);
    }
    const int64_t in_seq = at - seq_first;
    const int64_t unit = ((in_seq | slices) >> 32) == 0  // of the sequence
                             ? static_cast<uint32_t>(in_seq) / static_cast<uint32_t>(slices) : in_seq / slices;
    const int64_t unit_first = seq_first + unit * slices;
    const int32_t head = static_cast<int32_t>(unit) / blocks_c, col0 = (static_cast<int32_t>(unit) - head * blocks_c) * S::kCols;
    const int64_t first = at - unit_first, last = min(part1 - unit_first, slices);  // slices [first, last)
    const int64_t len = len_of(seq);
    const int32_t visible = static_cast<int32_t>(len) - a.tokens + 1;  // positions the first query reaches

    // ---- queries: fragments of Q^T in f16, and -8 times the groups' sums
    uint32_t q[G][2][NT][2];   // [group][k 16]: channels 8 j + (0, 4), (1, 5), then (2, 6), (3, 7)
    uint32_t offset[NT][2];    // their parts in bf16: of groups (0, 1), (2, 3), lane j the part j
    float cc[NT][2];
    int32_t reach[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int col = col0 + 8 * t + r;
      const int64_t row = seq * a.tokens + col / group;
      const int64_t from = row * a.ld_q + static_cast<int64_t>(head * group + col % group) * S::D;
      uint4 w[G];
      uint32_t top = 0;  // of the magnitudes' bits
#pragma unroll
      for (int g = 0; g < G; ++g) {
        w[g] = make_uint4(0, 0, 0, 0);
        if (col < cols && kda_guard(from + 32 * g + 8 * j, 8, (n_rows - 1) * a.ld_q + a.heads * S::D, a.err))
          w[g] = *reinterpret_cast<const uint4*>(a.q + from + 32 * g + 8 * j);
        const uint32_t u = __vmaxu2(__vmaxu2(w[g].x & 0x7fff7fffu, w[g].y & 0x7fff7fffu),
                                    __vmaxu2(w[g].z & 0x7fff7fffu, w[g].w & 0x7fff7fffu));
        top = max(top, max(u >> 16, u & 0xffffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^k brings the largest magnitude into [2^14, 2^15); an infinity or NaN makes the row NaN
      const int k = min(141 - static_cast<int>(top >> 7), 126);
      const float up = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
      // 2^-k, the 2^24 of codes read as f16, and c: never 0, which times a hidden score's
      // infinity would be NaN (queries of zeros and a tiny scale come to it)
      const float down = fmaxf(c * (__uint_as_float(static_cast<uint32_t>(127 - k) << 23) * 0x1p24f), 0x1p-126f);
      cc[t][0] = __shfl_sync(0xffffffffu, down, 8 * j);
      cc[t][1] = __shfl_sync(0xffffffffu, down, 8 * j + 4);
      offset[t][0] = offset[t][1] = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t x[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // channels 8 j + i, 8 j + i + 4: nibbles i and i + 4
          const float v0 = half_of(x[i / 2], i % 2) * up, v1 = half_of(x[2 + i / 2], i % 2) * up;
          // (codes in bits 4..7 of a half are read 16 times as large)
          q[g][i / 2][t][i % 2] = pack2_f16(v0 * (i % 2 ? 0.0625f : 1.0f), v1 * (i % 2 ? 0.0625f : 1.0f));
          sum += v0 + v1;
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.0f * 0x1p-24f;
        uint32_t part = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t bits = from_f32<Bf16>(sum).bits;
          if (i == j) part = bits;
          sum -= __uint_as_float(bits << 16);
        }
        offset[t][g / 2] |= part << (16 * (g % 2));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)  // of this lane's columns 2 j + e, from its first position r on
        reach[t][e] = visible + (col0 + 8 * t + 2 * j + e) / group - r;
    }
    float o[2 * G][NT][4], m[NT][2], l[NT][2], limit[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int g = 0; g < 2 * G; ++g) o[g][t][0] = o[g][t][1] = o[g][t][2] = o[g][t][3] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = limit[t][e] = kLowest;
        l[t][e] = 0.0f;
      }
    }

    // ---- this warp's slices: first + warp, + 4, ... (or all of them)
    const int32_t left = static_cast<int32_t>(last - first) - mine0;
    const int32_t mine = left <= 0 ? 0 : SOLO ? left : (left + kWarps - 1) / kWarps;
    const int32_t pos0 = static_cast<int32_t>(first + mine0) * kSlice;  // of the first one
    const int32_t* const pages = p.table + seq * p.ld_table;
    const int32_t place = (1 << p.page_shift) - 1;  // a position's bits in its page
    const int32_t head_rows = head << p.page_shift, page_rows = p.heads << p.page_shift;
    // 16 lanes copy a half, each from its half's page
    const int half = lane >> 4, of_half = lane & 15;
    const uint8_t* const from_k = p.k_codes + 16 * of_half;
    const uint8_t* const from_v = p.v_codes + 16 * of_half;
    constexpr int kS = kHalf * 2 * G / 16;  // pieces of 16 bytes of a half's scales
    const uint8_t* const from_s =
        reinterpret_cast<const uint8_t*>(of_half < kS ? p.k_scales : p.v_scales) + 16 * (of_half % kS);
    constexpr int kChunks = S::kRow / 16;  // of a row
    const uint32_t to_k = smem_u32(ring) + half * (kHalf * S::kRow) + 16 * of_half;
    const uint32_t to_v = smem_u32(ring) + kSlice * S::kRow + (half * kHalf + of_half / kChunks) * S::kPitchV +
                          of_half % kChunks * 16;
    const uint32_t to_s = smem_u32(ring) + kSlice * (S::kRow + S::kPitchV) + (of_half < kS ? 0 : S::kScaleBytes) +
                          half * (16 * kS) + 16 * (of_half % kS);
    const int32_t stop = pos0 + mine * stride;
    // (the last slice's second half may lie behind the sequence's last position)
    const int32_t held = static_cast<int32_t>(len);
    auto page_of = [&](int32_t pos) -> int32_t {  // of this lane's half of a slice
      const int32_t at_page = (pos + half * kHalf) >> p.page_shift;
      int32_t page = -1;
      if (pos < stop && pos + half * kHalf < held &&
          kda_guard(seq * p.ld_table + at_page, 1, (a.N - 1) * p.ld_table + p.width, a.err))
        page = pages[at_page];
      return page;
    };
    auto fetch = [&](int32_t pos, int32_t page, uint32_t at_stage) {
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.n_pages)) {
        const int64_t row = static_cast<int64_t>(page) * page_rows + (head_rows + ((pos + half * kHalf) & place));
        if (kda_guard(row, kHalf, kv4_rows(p), a.err)) {
          const uint8_t* k = from_k + row * S::kRow;
          const uint8_t* v = from_v + row * S::kRow;
#pragma unroll
          for (int e = 0; e < kHalf * kChunks; e += 16) {
            copy16(to_k + at_stage + 16 * e, k + 16 * e);
            copy16(to_v + at_stage + e / kChunks * S::kPitchV, v + 16 * e);
          }
          if (of_half < 2 * kS) copy16(to_s + at_stage, from_s + row * (2 * G));
        }
      } else if (pos < stop && pos + half * kHalf < held) {
        atomicOr(a.err, kDevErrPage);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // One slice; MASKED: some column does not reach all of its positions.
    auto process = [&](const unsigned char* stage, int32_t pos, auto masked_c) {
      constexpr bool MASKED = decltype(masked_c)::value;
      // ---- scores of positions r and r + 8 of both halves
      float x[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t k0[G], k1[G], s0[G / 2], s1[G / 2];
        const unsigned char* keys = stage + h * (kHalf * S::kRow) + 4 * G * j;
        const unsigned char* key_scales = stage + kSlice * (S::kRow + S::kPitchV) + h * (kHalf * 2 * G);
        load_words<G>(keys + r * S::kRow, k0);
        load_words<G>(keys + (r + 8) * S::kRow, k1);
        load_words<G / 2>(key_scales + 2 * G * r, s0);
        load_words<G / 2>(key_scales + 2 * G * (r + 8), s1);
        // what the 8 in n + 8 adds: the groups' scales times the offsets' four parts
        const uint32_t scales[4] = {s0[0], s1[0], G == 4 ? s0[G / 2 - 1] : 0u, G == 4 ? s1[G / 2 - 1] : 0u};
#pragma unroll
        for (int t = 0; t < NT; ++t) mma<false>(x[h][t], scales, offset[t][0], offset[t][1]);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t h0 = k0[g] >> 8, h1 = k1[g] >> 8;
          const uint32_t f0[4] = {k0[g] & 0x000f000fu, k1[g] & 0x000f000fu, k0[g] & 0x00f000f0u, k1[g] & 0x00f000f0u};
          const uint32_t f1[4] = {h0 & 0x000f000fu, h1 & 0x000f000fu, h0 & 0x00f000f0u, h1 & 0x00f000f0u};
          const float lo = half_of(s0[g / 2], g % 2), hi = half_of(s1[g / 2], g % 2);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float d[4];
            mma_f16<false>(d, f0, q[g][0][t]);
            mma_f16<true>(d, f1, q[g][1][t]);
            x[h][t][0] = fmaf(d[0], lo, x[h][t][0]);
            x[h][t][1] = fmaf(d[1], lo, x[h][t][1]);
            x[h][t][2] = fmaf(d[2], hi, x[h][t][2]);
            x[h][t][3] = fmaf(d[3], hi, x[h][t][3]);
          }
        }
      }
      // ---- softmax
      auto hidden = [&](int h, int t, int e) { return pos + h * kHalf + (e >> 1) * 8 >= reach[t][e & 1]; };
      bool up = false;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (MASKED && hidden(h, t, e)) x[h][t][e] = -INFINITY;
            up = up || x[h][t][e] > limit[t][e & 1];
          }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaxf(x[0][t][e], x[0][t][e + 2]), fmaxf(x[1][t][e], x[1][t][e + 2]));
#pragma unroll
            for (int w = 4; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            top = fmaxf(m[t][e], top);
            const float keep = ex2((m[t][e] - top) * cc[t][e]);
            m[t][e] = top;
            limit[t][e] = top + kSlack / cc[t][e];
            l[t][e] *= keep;
#pragma unroll
            for (int g = 0; g < 2 * G; ++g) {
              o[g][t][e] *= keep;
              o[g][t][e + 2] *= keep;
            }
          }
      }
      // (m off before cc is multiplied in: of scores of 2^24 and more the product's rounding
      // would be whole numbers)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[h][t][e] = ex2(fmaf(x[h][t][e] - m[t][e & 1], cc[t][e & 1], -kSlack));
            l[t][e & 1] += x[h][t][e];
          }
      // ---- values
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t s0[G / 2], s1[G / 2], w[4][G / 2];
        const unsigned char* scales = stage + kSlice * (S::kRow + S::kPitchV) + S::kScaleBytes + h * (kHalf * 2 * G);
        load_words<G / 2>(scales + 2 * G * r, s0);
        load_words<G / 2>(scales + 2 * G * (r + 8), s1);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // positions 2 j, 2 j + 1, 2 j + 8, 2 j + 9
          load_words<G / 2>(stage + kSlice * S::kRow + (h * kHalf + 2 * j + k / 2 * 8 + k % 2) * S::kPitchV + 2 * G * r, w[k]);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float lo = half_of(s0[g / 2], g % 2), hi = half_of(s1[g / 2], g % 2);
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float f[4] = {x[h][t][0] * lo, x[h][t][1] * lo, x[h][t][2] * hi, x[h][t][3] * hi};
            if constexpr (MASKED) {  // (what is not reached may have any scale)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hidden(h, t, e)) f[e] = 0.0f;
            }
            b0[t] = turned(pack2_bf16(f[0], f[1]));
            b1[t] = turned(pack2_bf16(f[2], f[3]));
          }
          // channels 4 r + i of the group, positions in pairs
          const uint32_t sel = g % 2 ? 0x7632 : 0x5410;
          const uint32_t y0 = __byte_perm(w[0][g / 2], w[1][g / 2], sel), y1 = __byte_perm(w[2][g / 2], w[3][g / 2], sel);
          const uint32_t z0 = y0 >> 8, z1 = y1 >> 8;
          const uint32_t f0[4] = {whole_numbers<false>(y0), whole_numbers<true>(y0), whole_numbers<false>(y1),
                                  whole_numbers<true>(y1)};
          const uint32_t f1[4] = {whole_numbers<false>(z0), whole_numbers<true>(z0), whole_numbers<false>(z1),
                                  whole_numbers<true>(z1)};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma(o[2 * g][t], f0, b0[t], b1[t]);
            mma(o[2 * g + 1][t], f1, b0[t], b1[t]);
          }
        }
      }
    };

#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(pos0 + i * stride, page_of(pos0 + i * stride), i * S::kStage);
    int32_t ahead = pos0 + (kDepth - 1) * stride, next_page = page_of(ahead);
    uint32_t here = 0;  // the stage of the slice at hand
    // Where this warp moves its sums, o and l: [sum][lane], then the columns' maxima that
    // they were taken with.  (Of its eight records a block uses two otherwise.)
    constexpr int kSums = 8 * G * NT, kMoved = S::kRecord * 6 / kWarps;
    static_assert(32 * (kSums + 2 * NT) + S::kCols <= kMoved, "sums moved");
    float* const moved = records + static_cast<int64_t>(gridDim.x) * 2 * S::kRecord +
                         (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kMoved;
    float* const moved_m = moved + 32 * (kSums + 2 * NT);
    // what was moved added, by the maxima of now
    auto add_moved = [&]() {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float keep = ex2((moved_m[8 * t + 2 * j + e] - m[t][e]) * cc[t][e]);
          l[t][e] = fmaf(moved[(kSums + 2 * t + e) * 32 + lane], keep, l[t][e]);
#pragma unroll
          for (int g = 0; g < 2 * G; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& sum = o[g][t][e + 2 * h];
              sum = fmaf(moved[((g * NT + t) * 4 + e + 2 * h) * 32 + lane], keep, sum);
            }
        }
    };
    int32_t move_at = SOLO || !MOVES ? stop : pos0 + min(mine, kMoveSlices) * stride;
    for (int32_t pos = pos0; pos < stop; pos += stride) {
      if (MOVES && !SOLO && pos == move_at) {
        if (move_at - pos0 > kMoveSlices * stride) add_moved();
        __syncwarp();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int g = 0; g < 2 * G; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              moved[((g * NT + t) * 4 + e) * 32 + lane] = o[g][t][e];
              o[g][t][e] = 0.0f;
            }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            moved[(kSums + 2 * t + e) * 32 + lane] = l[t][e];
            l[t][e] = 0.0f;
            if (r == 0) moved_m[8 * t + 2 * j + e] = m[t][e];
          }
        }
        __syncwarp();
        move_at += min((stop - move_at) / stride, kMoveSlices) * stride;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
      __syncwarp();  // this slice has come, and the one before has been read
      fetch(ahead, next_page, here == 0 ? (kDepth - 1) * S::kStage : here - S::kStage);
      ahead += stride;
      next_page = page_of(ahead);
      if (pos + kSlice > visible) process(ring + here, pos, std::true_type{});
      else process(ring + here, pos, std::false_type{});
      here = here == (kDepth - 1) * S::kStage ? 0 : here + S::kStage;
    }
    if (MOVES && !SOLO && mine > kMoveSlices) add_moved();

    const bool complete = first == 0 && last == slices;
    const int slot = at == part0 ? 0 : 1;
    float* const record = records + (b * 2 + slot) * S::kRecord;
    // four channels of a column: to the output, or to the part's record
    auto put = [&](int col, int ch, const float4& v, float top, float sum, float cc_of) {
      if (complete) {
        const int g_col = col0 + col;
        if (g_col < cols) {
          const bool any = visible + g_col / group > 0;
          const float scale = 64.0f / sum;  // (codes were read as n 2^-6)
          const int64_t row = seq * a.tokens + g_col / group;
          const int32_t h = head * group + g_col % group;
          const int64_t to = row * a.ld_out + static_cast<int64_t>(h) * S::D + ch;
          if (kda_guard(to, 4, (n_rows - 1) * a.ld_out + a.heads * S::D, a.err))
            *reinterpret_cast<uint2*>(a.out + to) =
                any ? make_uint2(pack2_bf16(v.x * scale, v.y * scale), pack2_bf16(v.z * scale, v.w * scale))
                    : make_uint2(0, 0);
          if (a.lse && ch == 0 && kda_guard(row * a.heads + h, 1, n_rows * a.heads, a.err))
            a.lse[row * a.heads + h] = any ? fmaf(top * cc_of, kLn2, logf(sum * 256.0f)) : -INFINITY;
        }
      } else {
        *reinterpret_cast<float4*>(record + col * S::D + ch) = v;
        if (ch == 0) {
          record[S::kCols * S::D + 2 * col] = top;
          record[S::kCols * S::D + 2 * col + 1] = sum;
          record[S::kCols * (S::D + 2) + col] = cc_of;
        }
      }
    };
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 4; w < 32; w *= 2) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], w);
    // (Parts are joined by differences of maxima, and cc then multiplied in, as above:
    // between maxima that were multiplied first the weights of large scores were up to 4 %
    // off at 2^20.)
    if constexpr (SOLO) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < G; ++g)  // channels 32 g + 4 r + 0..3
            put(8 * t + 2 * j + e, 32 * g + 4 * r,
                make_float4(o[2 * g][t][e], o[2 * g][t][e + 2], o[2 * g + 1][t][e], o[2 * g + 1][t][e + 2]), m[t][e],
                l[t][e], cc[t][e]);
    } else {
    // ---- the warps' results together
    __syncthreads();
    float* const parts = reinterpret_cast<float*>(smem);  // [warp][column][D + 4]: o, m, l, cc
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* to = parts + (warp * S::kCols + 8 * t + 2 * j + e) * (S::D + 4);
#pragma unroll
        for (int g = 0; g < G; ++g)
          *reinterpret_cast<float4*>(to + 32 * g + 4 * r) =
              make_float4(o[2 * g][t][e], o[2 * g][t][e + 2], o[2 * g + 1][t][e], o[2 * g + 1][t][e + 2]);
        if (r == 0) {
          to[S::D] = m[t][e];
          to[S::D + 1] = l[t][e];
          to[S::D + 2] = cc[t][e];
        }
      }
    __syncthreads();
    for (int e = threadIdx.x; e < S::kCols * (S::D / 4); e += kThreads) {
      const int col = e / (S::D / 4), ch = e % (S::D / 4) * 4;
      const float cc_of = parts[col * (S::D + 4) + S::D + 2];  // (of the column: the same in all warps)
      float top = kLowest, sum = 0.0f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, parts[(w * S::kCols + col) * (S::D + 4) + S::D]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* from = parts + (w * S::kCols + col) * (S::D + 4);
        const float keep = ex2((from[S::D] - top) * cc_of);
        const float4 x = *reinterpret_cast<const float4*>(from + ch);
        sum = fmaf(from[S::D + 1], keep, sum);
        v.x = fmaf(x.x, keep, v.x);
        v.y = fmaf(x.y, keep, v.y);
        v.z = fmaf(x.z, keep, v.z);
        v.w = fmaf(x.w, keep, v.w);
      }
      put(col, ch, v, top, sum, cc_of);
    }
    }
    if (!complete && first == 0 && (SOLO ? lane : static_cast<int>(threadIdx.x)) == 0) {  // the unit's first part
      Meta mt;
      mt.last = static_cast<int32_t>(((unit_first + slices) * used - 1) / all);
      mt.slot = slot;
      mt.seq = static_cast<int32_t>(seq);
      mt.head = head;
      mt.col0 = col0;
      mt.visible = visible;
      mt.solo = SOLO;
      metas[SOLO ? b : b * kWarps] = mt;
    }
    if (SOLO) __syncwarp();
    else __syncthreads();  // the ring is filled again
    at = unit_first + last;
  }
  };
  if (solo) work(std::true_type{});
  else work(std::false_type{});
  write_zeros();
}

// The parts of units that several blocks (or warps) worked on: block b those of the
// unit that begins in block b's part of the line (or in those of its warps) and goes
// on behind it.  Four channels of a column to a thread.
constexpr int kCombineThreads = 1024;

template <int G, int NT>
__global__ void __launch_bounds__(kCombineThreads, 2) combine_kernel(Kv4AttentionArgs a, const float* records, const Meta* metas) {
  using S = Shape<G, NT>;
  constexpr int kItems = S::kCols * (S::D / 4), kSets = kCombineThreads / kItems;
  __shared__ float4 s_v[kSets - 1][kItems];
  __shared__ float2 s_ml[kSets - 1][kItems];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the first kernel's end
  const int group = a.heads / a.pages.heads, cols = a.tokens * group;
  const int item = threadIdx.x % kItems, set = threadIdx.x / kItems;
  const int col = item / (S::D / 4), ch = item % (S::D / 4) * 4;
  float top = kLowest, sum = 0.0f, cc = 1.0f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m2, float l2, const float4& x) {
    const float next = fmaxf(top, m2), k0 = ex2((top - next) * cc), k1 = ex2((m2 - next) * cc);
    top = next;
    sum = fmaf(l2, k1, sum * k0);
    v.x = fmaf(x.x, k1, v.x * k0);
    v.y = fmaf(x.y, k1, v.y * k0);
    v.z = fmaf(x.z, k1, v.z * k0);
    v.w = fmaf(x.w, k1, v.w * k0);
  };
  auto add_parts = [&](const Meta& mt, int b0, int from, int by) {
    // (a column's, the same in all parts)
    cc = records[(static_cast<int64_t>(b0) * 2 + mt.slot) * S::kRecord + S::kCols * (S::D + 2) + col];
    top = kLowest;
    sum = 0.0f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int b = b0 + from; b <= mt.last; b += by) {
      const float* record = records + (static_cast<int64_t>(b) * 2 + (b == b0 ? mt.slot : 0)) * S::kRecord;
      const float2 ml = *reinterpret_cast<const float2*>(record + S::kCols * S::D + 2 * col);
      add(ml.x, ml.y, *reinterpret_cast<const float4*>(record + col * S::D + ch));
    }
  };
  auto put = [&](const Meta& mt) {
    const int g_col = mt.col0 + col;
    if (g_col >= cols) return;
    const int64_t n_rows = static_cast<int64_t>(a.N) * a.tokens;
    const int64_t row = static_cast<int64_t>(mt.seq) * a.tokens + g_col / group;
    const int32_t h = mt.head * group + g_col % group;
    const bool any = mt.visible + g_col / group > 0;
    const float scale = 64.0f / sum;  // (codes were read as n 2^-6)
    const int64_t to = row * a.ld_out + static_cast<int64_t>(h) * S::D + ch;
    if (kda_guard(to, 4, (n_rows - 1) * a.ld_out + a.heads * S::D, a.err))
      *reinterpret_cast<uint2*>(a.out + to) =
          any ? make_uint2(pack2_bf16(v.x * scale, v.y * scale), pack2_bf16(v.z * scale, v.w * scale)) : make_uint2(0, 0);
    if (a.lse && ch == 0 && kda_guard(row * a.heads + h, 1, n_rows * a.heads, a.err))
      a.lse[row * a.heads + h] = any ? fmaf(top * cc, kLn2, logf(sum * 256.0f)) : -INFINITY;
  };
  const Meta first = metas[blockIdx.x * kWarps];
  if (!first.solo) {  // (of a block: all sets of threads share the parts)
    if (first.last < 0) return;
    add_parts(first, blockIdx.x, set, kSets);
    if (set > 0) {
      s_v[set - 1][item] = v;
      s_ml[set - 1][item] = make_float2(top, sum);
    }
    __syncthreads();
    if (set != 0) return;
#pragma unroll
    for (int i = 0; i < kSets - 1; ++i) add(s_ml[i][item].x, s_ml[i][item].y, s_v[i][item]);
    put(first);
    return;
  }
  for (int w = set; w < kWarps; w += kSets) {  // (of its warps: one to a set)
    const Meta mt = metas[blockIdx.x * kWarps + w];
    if (mt.last < 0) continue;
    add_parts(mt, blockIdx.x * kWarps + w, 0, 1);
    put(mt);
  }
}

template <int G, int NT, bool MOVES>
kda_status run(const Kv4AttentionArgs& a, cudaStream_t s, cudaError_t& e) {
  using S = Shape<G, NT>;
  constexpr auto kern = kv4_attention_kernel<G, NT, MOVES>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return KDA_OK;
  static const int resident = [] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, S::kSmem) == cudaSuccess ? n : 0;
  }();
  const int blocks = a.sm_count * std::max(resident, 1);
  void* ws = nullptr;
  const size_t records = sizeof(float) * 2 * blocks * kWarps * S::kRecord;
  const kda_status st = workspace_alloc(records + sizeof(Meta) * blocks * kWarps, s, &ws);
  if (st != KDA_OK) return st;
  float* rec = static_cast<float*>(ws);
  Meta* metas = reinterpret_cast<Meta*>(static_cast<unsigned char*>(ws) + records);
  kern<<<blocks, kThreads, S::kSmem, s>>>(a, rec, metas);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    // its blocks may come while the first kernel's last ones work, and wait for its end
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = s;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, combine_kernel<G, NT>, a, static_cast<const float*>(rec),
                           static_cast<const Meta*>(metas));
  }
  const cudaError_t ef = cudaFreeAsync(ws, s);
  if (e == cudaSuccess) e = ef;
  return KDA_OK;
}

// (a warp of a block sees a quarter of a sequence's slices)
template <int G, int NT>
kda_status pick(const Kv4AttentionArgs& a, cudaStream_t s, cudaError_t& e) {
  const int64_t positions = static_cast<int64_t>(a.pages.width) << a.pages.page_shift;
  return positions > int64_t{kMoveSlices} * kWarps * kSlice ? run<G, NT, true>(a, s, e) : run<G, NT, false>(a, s, e);
}

}  // namespace

kda_status launch_kv4_attention(const Kv4AttentionArgs& a, cudaStream_t s, cudaError_t& e) {
  const int cols = a.tokens * (a.heads / a.pages.heads);
  prof_begin(s, "kda_kv4_attention");
  const kda_status st = a.pages.d == 128 ? (cols <= 8 ? pick<4, 1>(a, s, e) : pick<4, 2>(a, s, e))
                                         : (cols <= 8 ? pick<2, 1>(a, s, e) : pick<2, 2>(a, s, e));
  prof_end(s, "kda_kv4_attention");
  return st;
}

}  // namespace kda
