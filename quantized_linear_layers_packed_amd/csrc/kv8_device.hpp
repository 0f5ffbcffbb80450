// Device helpers that the 8-bit cache's attention kernels share.
#pragma once

#include "common.hpp"
#include "device.hpp"
#include "kv8.hpp"

namespace qlin {

constexpr int kTile = 64;                      // positions per step of a wave or workgroup
// A row's reference is set kHead below its largest score and moves when a score
// exceeds it by more than kSlack.  The weights 2^(score - reference) are rounded to
// fp16: the largest is then 2^7 at least and no weight passes 2^15 (of 65504), so
// that weights down to 2^-21 of the largest keep 11 bits and those below lose 2^-32
// of it at most.  The tail of a long sequence lives there: 131003 tokens of
// 2^-20.6 each beside one large weight came out 2 % off with weights of up to 1.
constexpr float kHead = 7.0f;
constexpr float kSlack = kHead + 8.0f;
// References of rows that have seen nothing, and nothing but scores below all that
// fp32 holds: any finite score moves both.
constexpr float kNone = -3.40282347e38f;
constexpr float kLowest = -3.4e38f;

// 8 codes (two words) as 8 fp16 integers, in order: byte + 128 into the low
// mantissa of 1024, minus 1152.
__device__ __forceinline__ h8_t codes_f16(uint32_t w0, uint32_t w1) {
  const uint32_t x0 = w0 ^ 0x80808080u, x1 = w1 ^ 0x80808080u;
  const uint32_t p[4] = {__builtin_amdgcn_perm(0x64646464u, x0, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, x0, 0x04030402u),
                         __builtin_amdgcn_perm(0x64646464u, x1, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, x1, 0x04030402u)};
  const h2_t off = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
  h8_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const h2_t v = bitcast<h2_t>(p[j]) - off;
    r[2 * j] = v[0];
    r[2 * j + 1] = v[1];
  }
  return r;
}

// Exchanges between lanes 32 (or 16 and 32) apart on the VALU: both operands of a
// swap hold v, so that afterwards one holds the lower partner's value in both
// lanes and the other the upper partner's.
__device__ __forceinline__ float2 pair_over_32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(v), bitcast<uint32_t>(v), false, false);
  return make_float2(bitcast<float>(static_cast<uint32_t>(r[0])), bitcast<float>(static_cast<uint32_t>(r[1])));
}
__device__ __forceinline__ float2 pair_over_16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(bitcast<uint32_t>(v), bitcast<uint32_t>(v), false, false);
  return make_float2(bitcast<float>(static_cast<uint32_t>(r[0])), bitcast<float>(static_cast<uint32_t>(r[1])));
}
__device__ __forceinline__ float max_over_32(float v) {
  const float2 p = pair_over_32(v);
  return fmaxf(p.x, p.y);
}
__device__ __forceinline__ float sum_over_32(float v) {
  const float2 p = pair_over_32(v);
  return p.x + p.y;
}
__device__ __forceinline__ uint32_t most_over_32(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(static_cast<uint32_t>(r[0]), static_cast<uint32_t>(r[1]));
}
// Over the four lanes q, q + 16, q + 32, q + 48.
__device__ __forceinline__ float max_over_g(float v) {
  const float2 p = pair_over_16(v);
  return max_over_32(fmaxf(p.x, p.y));
}
__device__ __forceinline__ float sum_over_g(float v) {
  const float2 p = pair_over_16(v);
  return sum_over_32(p.x + p.y);
}
__device__ __forceinline__ uint32_t most_over_g(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return most_over_32(max(static_cast<uint32_t>(r[0]), static_cast<uint32_t>(r[1])));
}

// The tiles of 64 positions that the rows at positions p0 .. p1 see: those of the
// first tokens and those from the start of the window of p0.
struct Kv8Tiles {
  int sinks, first, count;
  __device__ __forceinline__ Kv8Tiles(int p0, int p1, int window, int sink_tokens) {
    if (p1 < 0) {
      sinks = first = count = 0;
      return;
    }
    first = window > 0 ? max(0, max(p0, 0) - window + 1) / kTile : 0;
    sinks = min(sink_tokens > 0 ? (sink_tokens - 1) / kTile + 1 : 0, first);
    count = sinks + p1 / kTile - first + 1;
  }
  __device__ __forceinline__ int operator[](int x) const { return x < sinks ? x : first + x - sinks; }
};

// The sequence with the n-th most tiles (n from 0, ties to the lower index), found
// by every wave for itself: a search down the bits of (tiles, 255 - index), a few
// scalar instructions a bit.  Workgroups that start in this order end together:
// 64 ragged sequences of up to 8192 tokens 99 -> 88 us.
constexpr int kSortedSeqs = 256;
template <int CHUNKS>
__device__ __forceinline__ int nth_longest(const Kv8View& c, int n) {
  const int lane = threadIdx.x & 63;
  uint32_t key[CHUNKS];
  uint64_t in[CHUNKS];
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int j = lane + 64 * i;
    const int tiles = min(max(c.kv_lens[min(j, c.seqs - 1)], 0) / kTile, 0xFFFF);
    key[i] = static_cast<uint32_t>(tiles) << 8 | static_cast<uint32_t>(255 - (j & 255));
    in[i] = __ballot(j < c.seqs);
  }
  for (int bit = 23; bit >= 0; --bit) {
    uint64_t set[CHUNKS];
    int count = 0;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      set[i] = in[i] & __ballot((key[i] >> bit) & 1u);
      count += __popcll(set[i]);
    }
    const bool up = n < count;
    n -= up ? 0 : count;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) in[i] = up ? set[i] : in[i] & ~set[i];
  }
  int found = 0;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i)
    if (in[i]) found = 64 * i + __ffsll(static_cast<unsigned long long>(in[i])) - 1;
  return __builtin_amdgcn_readfirstlane(found);
}

// Which of the N consecutive positions from j0 the row at `pos` sees, as bits
// (low: first position of its window).
template <int N>
__device__ __forceinline__ uint32_t visible_bits(int j0, int pos, int low, int sinks, bool held) {
  const auto below = [&](int end) { return (1u << min(max(end - j0, 0), N)) - 1u; };   // positions before `end`
  const uint32_t seen = below(pos + 1) & (~below(low) | below(sinks));
  return held ? seen : 0u;
}

// Power of two that brings a row of bf16 values with largest magnitude bits
// `most` into fp16's range: the row maximum into [2^14, 2^15).  Rows of zeros,
// subnormals or with a value that is not finite stay as they are.
__device__ __forceinline__ int row_exponent(uint32_t most) {
  const int E = static_cast<int>(most >> 7);
  return E == 0 || E == 255 ? 0 : E - 127 - 14;
}
__device__ __forceinline__ uint32_t chunk_most(const uint4& w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) most = max(most, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
  return most;
}
__device__ __forceinline__ h8_t chunk_f16(const uint4& w, int e) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  h8_t q;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    q[j] = static_cast<_Float16>(ldexpf(bf16_bits_to_f32(static_cast<uint16_t>(x[j >> 1] >> (16 * (j & 1)))), -e));
  return q;
}

// What sums of weighted codes are multiplied by, from the sum of weights and the
// row's reference: rows that see nothing give zeros, rows that see scores of -inf
// alone NaN.
__device__ __forceinline__ float by_weights(float total, float ref) {
  return total == 0.0f ? (ref > kNone ? __builtin_nanf("") : 0.0f) : 1.0f / total;
}

// Values rounded to the output type, two to a word.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16)
    return bitcast<uint16_t>(static_cast<__bf16>(a)) | (static_cast<uint32_t>(bitcast<uint16_t>(static_cast<__bf16>(b))) << 16);
  else
    return bitcast<uint16_t>(static_cast<_Float16>(a)) | (static_cast<uint32_t>(bitcast<uint16_t>(static_cast<_Float16>(b))) << 16);
}

}  // namespace qlin
