// The cache in 4 bits: keys and values quantised as they are written into its
// pages, and spans of it read back.
//
//   s = bf16(max(max |x|, 2^-64) / 7) over 32 channels,  n = x / s rounded half
//   to even, stored as n + 8;  read back: bf16(n s)
//
// Bound: bytes (2 read and 0.5625 written per value, or the reverse): 65,536 tokens
// of 8 x 128 keys and values are read back in 57 us, 6.0 TB/s; 16,384
// are written and read back in 39 us, 4.4 TB/s (partly from L2; the write 44 % of HBM's
// rate: a block does one pass over 8 tokens behind a chain of lookups); 256 in 2.6 and
// 2.8, latencies.  (Written with a division per value: twice the time.)  Four
// lanes take a token and head: lane j reads channels 8 j .. 8 j + 7 of every
// group, 16 bytes at a time, and ends up with 16 bytes of codes that lie side by
// side; a group's maximum is that of its four lanes.
//
// The order of a row's codes is the one in which kda_kv4_attention's lanes need
// them.  Keys: 32-bit word j G + g holds channels 32 g + 8 j + 0..7 (G = d / 32
// groups, nibble i the channel + i).  Values: 16-bit word r G + g holds channels
// 32 g + 4 r + 0..3.
#include <algorithm>

#include "kda_attention.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

// The scale's bits from those of the largest magnitude (bf16; a NaN or an infinity
// is larger than any number).  top * fl(1/7) rounds to the bf16 number that top / 7
// does: of T / 7 with T of 8 bits no multiple of half a unit is nearer than 2^-12.
__device__ __forceinline__ uint32_t scale_bits(uint32_t top) {
  const float v = __uint_as_float(top << 16);
  return from_f32<Bf16>(max_nan(v, kAmaxMin) * (1.0f / 7.0f)).bits;
}

// Eight values' codes n + 8, n = x / s rounded half to even, for a finite scale s.
//
// x r, r = 1 / s as the hardware gives it, is x / s but for 2^-21.  x and s have 8
// bits, so where x / s is not a half, it is 2^-11 or more away from one (for quotients
// from 1/4 on; smaller ones are 0 anyway).  So x r is first rounded to multiples of
// 2^-12, which makes halves exact, and then to a whole number: each time by adding a
// number whose last bit has that value.  The whole number then is the low bits of the
// sum's significand, and a product and sum puts it in its place.
__device__ __forceinline__ uint32_t codes_of(const uint4& raw, uint32_t scale) {
  constexpr float kFine = 1.5f * 2048.0f, kWhole = 1.5f * 8388608.0f + 8.0f;  // last bits 2^-12, 1
  const float r = rcp(__uint_as_float(scale << 16));
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const f32x2 rr = pack2(r, r), fine = pack2(kFine, kFine), less = pack2(-kFine, -kFine), whole = pack2(kWhole, kWhole);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 x = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    const f32x2 n = add2(add2(fma2(x, rr, fine), less), whole);
    float lo, hi;
    unpack2(n, lo, hi);
    // (the bits above the lowest four, the same for all n, go away below)
    word += (__float_as_uint(lo) << (8 * i)) + (__float_as_uint(hi) << (8 * i + 4));
  }
  constexpr uint32_t kHigh = 0x4b400008u;  // of kWhole, and so of every sum less n
  constexpr uint32_t kAll = (kHigh << 0) + (kHigh << 4) + (kHigh << 8) + (kHigh << 12) + (kHigh << 16) +
                            (kHigh << 20) + (kHigh << 24) + (kHigh << 28);
  word = word - kAll + 0x88888888u;
  return (scale & 0x7f80u) == 0x7f80u ? 0x88888888u : word;  // (a group with a NaN or an infinity)
}

// Words of codes of 8 channels each, one of every group: as they lie in a row of
// keys (KEYS), or in a row of values (2 x 4 channels, the groups' halves side by
// side).  Turns one into the other; its own inverse where G = 2.
template <int G>
__device__ __forceinline__ void to_values(const uint32_t (&w)[G], uint32_t (&out)[G]) {
#pragma unroll
  for (int i = 0; i < G / 2; ++i) {
    out[i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
    out[G / 2 + i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
  }
}
template <int G>
__device__ __forceinline__ void from_values(const uint32_t (&w)[G], uint32_t (&out)[G]) {
#pragma unroll
  for (int i = 0; i < G / 2; ++i) {
    out[2 * i] = __byte_perm(w[i], w[G / 2 + i], 0x5410);
    out[2 * i + 1] = __byte_perm(w[i], w[G / 2 + i], 0x7632);
  }
}

template <int G>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[G]) {
  if constexpr (G == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int G>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[G]) {
  if constexpr (G == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  }
}

// A row's part of one lane: values to codes, scales by the first lane.  (All lanes come
// here, `valid` or not: a group's maximum goes over four.)
template <int G, bool KEYS>
__device__ __forceinline__ void quantise(const Kv4Pages& p, const uint4 (&raw)[G], bool valid, int64_t row, int j,
                                         int* err) {
  uint32_t words[G], scales[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t u = __vmaxu2(__vmaxu2(raw[g].x & 0x7fff7fffu, raw[g].y & 0x7fff7fffu),
                                __vmaxu2(raw[g].z & 0x7fff7fffu, raw[g].w & 0x7fff7fffu));
    uint32_t top = max(u >> 16, u & 0xffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    scales[g] = scale_bits(top);
    words[g] = codes_of(raw[g], scales[g]);
  }
  if (!valid || !kda_guard(row, 1, kv4_rows(p), err)) return;
  uint8_t* codes = (KEYS ? p.k_codes : p.v_codes) + row * (16 * G) + 4 * G * j;
  if constexpr (KEYS) {
    store_words<G>(codes, words);
  } else {
    uint32_t turned[G];
    to_values<G>(words, turned);
    store_words<G>(codes, turned);
  }
  if (j == 0) {
    uint32_t* to = reinterpret_cast<uint32_t*>((KEYS ? p.k_scales : p.v_scales) + row * G);
    if constexpr (G == 4)
      *reinterpret_cast<uint2*>(to) = make_uint2(scales[0] | scales[1] << 16, scales[2] | scales[3] << 16);
    else
      *to = scales[0] | scales[1] << 16;
  }
}

template <int G, bool KEYS>
__device__ __forceinline__ void restore(const Kv4Pages& p, Bf16* x, int64_t row, int j, int* err) {
  if (!kda_guard(row, 1, kv4_rows(p), err)) return;
  uint32_t words[G];
  const uint8_t* codes = (KEYS ? p.k_codes : p.v_codes) + row * (16 * G) + 4 * G * j;
  if constexpr (KEYS) {
    load_words<G>(codes, words);
  } else {
    uint32_t turned[G];
    load_words<G>(codes, turned);
    from_values<G>(turned, words);
  }
  const uint16_t* scales = (KEYS ? p.k_scales : p.v_scales) + row * G;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float scale = bf16_to_f32(scales[g]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = static_cast<float>(static_cast<int>(words[g] >> (4 * i) & 15u) - 8) * scale;
    store8(x + 32 * g + 8 * j, v);
  }
}

// The heads of a few tokens to a block.  The tokens' places are looked up once for the
// block, a token to a thread, while the rows to be written are already on their way.
// Where there are few tokens (gridDim.y = 2) keys and values go to different blocks:
// twice as many threads finish sooner.
template <int G, bool WRITE>
__global__ void __launch_bounds__(kThreads) span_kernel(Kv4SpanArgs a, int32_t block_tokens) {
  constexpr int D = 32 * G;
  __shared__ int64_t s_slot[kThreads / 4];
  if (a.cu && blockIdx.x == 0 && blockIdx.y == 0) check_cu_seqlens(a.cu, a.N, a.T, threadIdx.x, kThreads, a.err);
  const int j = threadIdx.x & 3;
  const int32_t heads = a.pages.heads;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * block_tokens;
  const int64_t width = static_cast<int64_t>(heads) * D;
  const int64_t extent_k = (a.T - 1) * a.ld_k + width, extent_v = (a.T - 1) * a.ld_v + width;
  const bool keys = gridDim.y == 1 || blockIdx.y == 0, values = gridDim.y == 1 || blockIdx.y == 1;
  const int32_t here = static_cast<int32_t>(min(static_cast<int64_t>(block_tokens), a.T - t0));
  const uint32_t rows = static_cast<uint32_t>(max(here, 0)) * heads;
  for (uint32_t base = 0; base < rows; base += kThreads / 4) {
    const uint32_t item = base + (threadIdx.x >> 2), token = item / static_cast<uint32_t>(heads);
    const int32_t head = static_cast<int32_t>(item - token * heads);
    const int64_t t = t0 + token;
    Bf16* const k = a.k + t * a.ld_k + static_cast<int64_t>(head) * D;
    Bf16* const v = a.v + t * a.ld_v + static_cast<int64_t>(head) * D;
    bool valid = item < rows && kda_guard(k - a.k, D, extent_k, a.err) && kda_guard(v - a.v, D, extent_v, a.err);
    uint4 raw_k[G], raw_v[G];
    if constexpr (WRITE) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        raw_k[g] = raw_v[g] = make_uint4(0, 0, 0, 0);
        if (valid && keys) raw_k[g] = *reinterpret_cast<const uint4*>(k + 32 * g + 8 * j);
        if (valid && values) raw_v[g] = *reinterpret_cast<const uint4*>(v + 32 * g + 8 * j);
      }
    }
    if (base == 0) {
      if (static_cast<int32_t>(threadIdx.x) < here) {
        const int64_t mine = t0 + threadIdx.x;
        int32_t n;
        int64_t first, end;
        if (a.cu) n = sequence_of(a.cu, a.N, mine, a.err);
        else n = static_cast<int32_t>(static_cast<uint32_t>(mine) / static_cast<uint32_t>(a.T / a.N));
        sequence_span(a.cu, a.N, a.T, n, first, end, a.err);
        int32_t start = 0;
        if (a.start && kda_guard(n, 1, a.N, a.err)) start = a.start[n];
        s_slot[threadIdx.x] = start >= 0 && mine >= first && mine < end
                                  ? kv4_slot(a.pages, a.N, n, start + (mine - first), a.err) : -1;
      }
      __syncthreads();
    }
    const int64_t slot = valid ? s_slot[token] : -1;
    valid = slot >= 0;
    const int64_t row = valid ? kv4_row(a.pages, slot, head) : 0;
    if constexpr (WRITE) {
      if (keys) quantise<G, true>(a.pages, raw_k, valid, row, j, a.err);
      if (values) quantise<G, false>(a.pages, raw_v, valid, row, j, a.err);
    } else if (valid) {
      if (keys) restore<G, true>(a.pages, k, row, j, a.err);
      if (values) restore<G, false>(a.pages, v, row, j, a.err);
    }
  }
}

template <bool WRITE>
cudaError_t launch(const Kv4SpanArgs& a, const char* name, cudaStream_t s) {
  // a block's threads once around, or all the heads of a token
  const int32_t block_tokens = std::max(1, kThreads / 4 / a.pages.heads);
  const int64_t blocks = std::max<int64_t>(1, (a.T + block_tokens - 1) / block_tokens);
  // (256 tokens of 8 heads, 32 blocks: 3.7 us together, 2.6 apart; 65,536 tokens: 54 and 61)
  const dim3 grid(static_cast<unsigned>(blocks), blocks < 2 * a.sm_count ? 2 : 1);
  prof_begin(s, name);
  if (a.pages.d == 128) span_kernel<4, WRITE><<<grid, kThreads, 0, s>>>(a, block_tokens);
  else span_kernel<2, WRITE><<<grid, kThreads, 0, s>>>(a, block_tokens);
  prof_end(s, name);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4SpanArgs& a, cudaStream_t s) { return launch<true>(a, "kda_kv4_write", s); }
cudaError_t launch_kv4_read(const Kv4SpanArgs& a, cudaStream_t s) { return launch<false>(a, "kda_kv4_read", s); }

}  // namespace kda
