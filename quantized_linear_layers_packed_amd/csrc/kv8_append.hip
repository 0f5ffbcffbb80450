// Appending to the 8-bit paged key/value cache with the position rotation on the
// way, and reading cached values back, gfx950.
//
// Per page and head, K and V apart, in fp32:
//   x = the new tokens' values (keys rotated: (a, b) -> (a cos - b sin,
//       b cos + a sin), products and sums rounded one by one),
//   s = max(s_old if the page holds earlier tokens, max |x| / 127),
//   codes clamp(rint(x / s), -127, 127); earlier codes become rint(q s_old / s)
//   where the scale grew.
// A page's scale only grows while it fills, and for independent tokens a new
// maximum comes about ln(page) times, so an old code is rounded again a few
// times at most, each time by half a step of a scale below the final one.
//
// Everything here is bound by memory: 16-bit values in, 8-bit codes (and rotated
// queries) out, a handful of operations per value.  One workgroup owns one page
// of one sequence and one key/value head (all of a page's new tokens, hence its
// maximum and its scale without atomics), and its values stay in registers
// between the maximum and the codes.  A work item is one token's 16 dimensions as
// two 8-value chunks that the rotation pairs, so a rotation never crosses lanes.
// V is stored with tokens contiguous (the order in which the attention feeds
// the matrix instructions): its codes are transposed through LDS and written in
// 16-byte pieces, merged with the earlier tokens' bytes where a piece holds both.
// Workgroups of the query heads come after those of the key/value heads.
//
// Measured: ragged prompts of 8.8 thousand tokens, 64 / 8 heads of 128, pages of 32:
// 84 us for 337 MB, 4.0 TB/s (a large copy: 4.8), of which the queries' part is 70;
// reading the touched pages back 15 us.  One token of one sequence: 5.6 and 4.8 us, a
// chain of launch, lengths, page number, scale and store.  Tried without gain:
// queries read past the caches (+5 %), written past them (faster for long pages,
// 22 % slower here), the page's scale and boundary piece fetched before the new
// values have come (more registers: 64 single tokens 7 -> 10 us).

#include <algorithm>

#include "common.hpp"
#include "device.hpp"
#include "kv8.hpp"

namespace qlin {

namespace {

template <bool BF16>
__device__ __forceinline__ float load16(uint32_t h) {
  return BF16 ? bf16_bits_to_f32(static_cast<uint16_t>(h)) : f16_bits_to_f32(static_cast<uint16_t>(h));
}
template <bool BF16>
__device__ __forceinline__ uint32_t round16(float v) {
  if constexpr (BF16) return bitcast<uint16_t>(static_cast<__bf16>(v));
  else return bitcast<uint16_t>(static_cast<_Float16>(v));
}

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = load16<BF16>((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = round16<BF16>(x[2 * j]) | (round16<BF16>(x[2 * j + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The two chunks (8 dimensions each) of work item p of a head: with the rotation
// in halves, chunk p and its partner half a rotation further; the others and
// pairs of neighbours, chunks 2p and 2p + 1.  Either way an item that turns uses
// table columns 8p .. 8p + 7.
__device__ __forceinline__ void item_chunks(int p, int rot, int pairs, int* c0, int* c1) {
  const bool halves = !pairs && 16 * p < rot;
  *c0 = halves ? p : 2 * p;
  *c1 = halves ? p + rot / 16 : 2 * p + 1;
}

// Cosines and sines of an item that turns, at a position.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ Turn load_turn(int p, int pos, const Kv8AppendArgs& a) {
  Turn t;
  const size_t at = static_cast<size_t>(min(pos, a.max_pos - 1)) * (a.rot / 2) + 8 * p;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    *reinterpret_cast<float4*>(t.c + 4 * j) = reinterpret_cast<const float4*>(a.cos + at)[j];
    *reinterpret_cast<float4*>(t.s + 4 * j) = reinterpret_cast<const float4*>(a.sin + at)[j];
  }
  return t;
}

// x[0..7], x[8..15]: the item's two chunks, turned in place.
__device__ __forceinline__ void turn_item(float* x, const Turn& t, int pairs) {
  if (pairs) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = x[2 * j], v = x[2 * j + 1];
      x[2 * j] = u * t.c[j] - v * t.s[j];
      x[2 * j + 1] = v * t.c[j] + u * t.s[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = x[j], v = x[8 + j];
      x[j] = u * t.c[j] - v * t.s[j];
      x[8 + j] = v * t.c[j] + u * t.s[j];
    }
  }
}

__device__ __forceinline__ uint32_t code_of(float x, float inv) {
  return static_cast<uint32_t>(static_cast<int32_t>(fminf(fmaxf(rintf(x * inv), -127.0f), 127.0f))) & 0xFFu;
}
__device__ __forceinline__ uint32_t pack_codes4(const float* x, float inv) {
  return code_of(x[0], inv) | (code_of(x[1], inv) << 8) | (code_of(x[2], inv) << 16) | (code_of(x[3], inv) << 24);
}
// Four earlier codes under the grown scale (r = s_old / s).
__device__ __forceinline__ uint32_t recode4(uint32_t w, float r) {
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) o |= code_of(static_cast<float>(static_cast<int8_t>(w >> (8 * j))), r) << (8 * j);
  return o;
}

// Mask of the first n bytes of a word (n may be negative or past 4).
__device__ __forceinline__ uint32_t low_bytes(int n) {
  return n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
}

// The scale of a page after the call, its reciprocal for new values and the
// factor for earlier codes.  most: the largest magnitude bits of the new values
// (they order like the magnitudes, infinities and NaN last).  least: smaller scales
// are 0.
struct PageScale {
  float s, inv, r;
  bool grew;
};
__device__ __forceinline__ PageScale page_scale(uint32_t most, bool earlier, float s_old, float least) {
  PageScale p;
  const float fresh = __fdiv_rn(bitcast<float>(most), 127.0f);
  p.s = earlier ? fmaxf(fresh, s_old) : fresh;
  if (p.s < least) p.s = 0.0f;
  if (most >= 0x7F800000u || (earlier && s_old != s_old)) p.s = __builtin_nanf("");
  p.inv = p.s > 0.0f ? __fdiv_rn(1.0f, p.s) : 0.0f;
  p.r = s_old * p.inv;
  p.grew = earlier && !(p.s == s_old);
  return p;
}

// Keys and values of one page and head; rows lo .. hi-1 of the sequence's
// positions are new.  NP: work items per thread that a page can hold.
template <bool BF16, int NP>
__device__ __forceinline__ void store_page(const Kv8AppendArgs& a, const Kv8Seq& q, int head, int page, int lo, int hi,
                                           uint8_t* turn, uint32_t (*red)[8]) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int D = a.c.dim, P = 1 << a.c.log_page, log_dp = __ffs(D) - 5, DP = 1 << log_dp;   // DP work items a token
  const int base = lo & ~(P - 1), olds = lo - base, fresh = hi - lo;
  const size_t at = (static_cast<size_t>(page) * a.c.heads + head) * P * D;
  int8_t* kp = a.c.k + at;
  int8_t* vp = a.c.v + at;
  float2* sp = reinterpret_cast<float2*>(a.c.scales) + static_cast<size_t>(page) * a.c.heads + head;
  const float2 s_old = olds > 0 ? *sp : make_float2(0.0f, 0.0f);

  float kx[NP][16], vx[NP][16];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const int i = tid + n * nt, t = i >> log_dp, p = i & (DP - 1);
    if (t < fresh) {
      const size_t row = static_cast<size_t>(q.row + (lo - q.start) + t);
      int c0, c1;
      item_chunks(p, a.rot, a.pairs, &c0, &c1);
      const uint4* kr = reinterpret_cast<const uint4*>(a.K + row * a.k_stride + static_cast<size_t>(head) * D);
      const uint4* vr = reinterpret_cast<const uint4*>(a.V + row * a.v_stride + static_cast<size_t>(head) * D);
      widen8<BF16>(kr[c0], kx[n]);
      widen8<BF16>(kr[c1], kx[n] + 8);
      widen8<BF16>(vr[2 * p], vx[n]);
      widen8<BF16>(vr[2 * p + 1], vx[n] + 8);
      if (16 * p < a.rot) turn_item(kx[n], load_turn(p, lo + t, a), a.pairs);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        mk = max(mk, bitcast<uint32_t>(kx[n][j]) & 0x7FFFFFFFu);
        mv = max(mv, bitcast<uint32_t>(vx[n][j]) & 0x7FFFFFFFu);
      }
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    mk = max(mk, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mk), off, 64)));
    mv = max(mv, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mv), off, 64)));
  }
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = mk;
    red[1][tid >> 6] = mv;
  }
  __syncthreads();
  for (int w = 0; w < nt / 64; ++w) {
    mk = max(mk, red[0][w]);
    mv = max(mv, red[1][w]);
  }
  const PageScale sk = page_scale(mk, olds > 0, s_old.x, 1.17549435e-38f), sv = page_scale(mv, olds > 0, s_old.y, kLeastScale);
  if (tid == 0) *sp = make_float2(sk.s, sv.s);

  // keys, and the values' codes into the transposed page in LDS
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const int i = tid + n * nt, t = i >> log_dp, p = i & (DP - 1);
    if (t < fresh) {
      int c0, c1;
      item_chunks(p, a.rot, a.pairs, &c0, &c1);
      uint2* kr = reinterpret_cast<uint2*>(kp + static_cast<size_t>(olds + t) * D);
      kr[c0] = make_uint2(pack_codes4(kx[n], sk.inv), pack_codes4(kx[n] + 4, sk.inv));
      kr[c1] = make_uint2(pack_codes4(kx[n] + 8, sk.inv), pack_codes4(kx[n] + 12, sk.inv));
#pragma unroll
      for (int j = 0; j < 16; ++j) turn[(16 * p + j) * P + olds + t] = static_cast<uint8_t>(code_of(vx[n][j], sv.inv));
    }
  }
  if (sk.grew) {                                           // earlier keys: rows 0 .. olds-1, contiguous
    uint4* kr = reinterpret_cast<uint4*>(kp);
    for (int i = tid; i < olds * D / 16; i += nt) {
      const uint4 w = kr[i];
      kr[i] = make_uint4(recode4(w.x, sk.r), recode4(w.y, sk.r), recode4(w.z, sk.r), recode4(w.w, sk.r));
    }
  }
  __syncthreads();
  // values: 16-byte pieces of 16 tokens of one dimension, from the first that
  // changes to the last one with a new token
  const int first = sv.grew ? 0 : olds >> 4, pieces = ((olds + fresh + 15) >> 4) - first;
  for (int i = tid; i < pieces * D; i += nt) {
    const int d = i / pieces, c = first + (i - d * pieces);
    uint4* vr = reinterpret_cast<uint4*>(vp + static_cast<size_t>(d) * P) + c;
    const uint4 fresh16 = *reinterpret_cast<const uint4*>(turn + d * P + 16 * c);
    const int before = olds - 16 * c, upto = before + fresh;   // of this piece: earlier tokens, and tokens in all
    const uint4 was = before > 0 ? *vr : make_uint4(0, 0, 0, 0);
    const uint32_t o[4] = {was.x, was.y, was.z, was.w}, f[4] = {fresh16.x, fresh16.y, fresh16.z, fresh16.w};
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t kept = sv.grew ? recode4(o[j], sv.r) : o[j], olds4 = low_bytes(before - 4 * j);
      w[j] = (kept & olds4) | (f[j] & low_bytes(upto - 4 * j) & ~olds4);   // slots past the last token: 0
    }
    *vr = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncthreads();                                         // red and turn may be used for the next page
}

// Grid: x pages from the sequence's first touched one, y key/value heads (stores)
// and then as many groups of query heads, z sequences.  A page index past the
// grid is taken up by the workgroups in turn.
template <bool BF16, int NP>
__global__ __launch_bounds__(512) void kv8_append_kernel(const Kv8AppendArgs a) {
  extern __shared__ __align__(16) uint8_t turn[];
  __shared__ uint32_t red[2][8];
  const int P = 1 << a.c.log_page;
  const Kv8Seq q = kv8_seq(a.c, blockIdx.z);
  if (q.count == 0) return;
  const bool keys = blockIdx.y < static_cast<unsigned>(a.c.heads);
  const int head = keys ? blockIdx.y : blockIdx.y - a.c.heads;
  const int first = max(q.start, 0) >> a.c.log_page, last = (q.len - 1) >> a.c.log_page;
  if (keys) {
    for (int x = first + blockIdx.x; x <= last; x += gridDim.x) {
      const int page = a.c.table[static_cast<size_t>(blockIdx.z) * a.c.table_stride + x];
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.pages)) continue;
      store_page<BF16, NP>(a, q, head, page, max(q.start, x << a.c.log_page), min(q.len, (x + 1) << a.c.log_page), turn,
                           red);
    }
    return;
  }
  // queries: P tokens at a time; an item's cosines and sines serve the heads of the
  // group, which are dealt out over the threads that few tokens leave idle
  const int D = a.c.dim, log_dp = __ffs(D) - 5, G = a.group;
  const size_t stride = static_cast<size_t>(D) / 8;         // between heads, in chunks
  for (long long t0 = static_cast<long long>(blockIdx.x) << a.c.log_page; t0 < q.count;
       t0 += static_cast<long long>(gridDim.x) << a.c.log_page) {
    const int n = min(P, q.count - static_cast<int>(t0)) << log_dp;
    const int deals = min(max(static_cast<int>(blockDim.x) / n, 1), G);
    for (int k = threadIdx.x; k < n * deals; k += blockDim.x) {
      const int deal = deals > 1 ? k / n : 0, i = k - deal * n;
      const int t = i >> log_dp, p = i & ((1 << log_dp) - 1);
      const size_t row = static_cast<size_t>(q.row + t0 + t);
      int c0, c1;
      item_chunks(p, a.rot, a.pairs, &c0, &c1);
      const uint4* src = reinterpret_cast<const uint4*>(a.Q + row * a.q_stride + static_cast<size_t>(head) * G * D);
      uint4* dst = reinterpret_cast<uint4*>(a.Q_out + (row * a.q_heads + static_cast<size_t>(head) * G) * D);
      const bool turns = 16 * p < a.rot;
      Turn turn;
      if (turns) turn = load_turn(p, max(q.start + static_cast<int>(t0) + t, 0), a);
      constexpr int AHEAD = 4;                              // heads on their way
      for (int h0 = deal; h0 < G; h0 += AHEAD * deals) {
        uint4 w[AHEAD][2];
#pragma unroll
        for (int h = 0; h < AHEAD; ++h) {
          const uint4* s = src + min(h0 + h * deals, G - 1) * stride;
          w[h][0] = s[c0];
          w[h][1] = s[c1];
        }
#pragma unroll
        for (int h = 0; h < AHEAD; ++h) {
          if (h0 + h * deals >= G) break;
          if (turns) {
            float x[16];
            widen8<BF16>(w[h][0], x);
            widen8<BF16>(w[h][1], x + 8);
            turn_item(x, turn, a.pairs);
            w[h][0] = narrow8<BF16>(x);
            w[h][1] = narrow8<BF16>(x + 8);
          }
          uint4* d = dst + (h0 + h * deals) * stride;
          d[c0] = w[h][0];
          d[c1] = w[h][1];
        }
      }
    }
  }
}

// Values of the batch's tokens: one workgroup per page and head; the page's V
// codes go through LDS (read along tokens, needed along dimensions).
template <bool BF16>
__global__ __launch_bounds__(256) void kv8_gather_kernel(const Kv8View c, uint16_t* __restrict__ K,
                                                         uint16_t* __restrict__ V) {
  extern __shared__ __align__(16) uint8_t turn[];
  const int tid = threadIdx.x, D = c.dim, P = 1 << c.log_page, log_dp = __ffs(D) - 5, DP = 1 << log_dp, head = blockIdx.y;
  const int stride = P + 4;                                // bytes per dimension: neighbours in other banks
  const Kv8Seq q = kv8_seq(c, blockIdx.z);
  if (q.count == 0) return;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0) {                                   // positions below 0: nothing stored
    for (int i = tid; i < min(q.count, max(-q.start, 0)) * DP; i += blockDim.x) {
      const int t = i >> log_dp, p = i & (DP - 1);
      const size_t o = ((static_cast<size_t>(q.row + t) * c.heads + head) * D + 16 * p) / 8;
      reinterpret_cast<uint4*>(K)[o] = reinterpret_cast<uint4*>(K)[o + 1] = zero;
      reinterpret_cast<uint4*>(V)[o] = reinterpret_cast<uint4*>(V)[o + 1] = zero;
    }
  }
  const int first = max(q.start, 0) >> c.log_page, last = (q.len - 1) >> c.log_page;
  for (int x = first + blockIdx.x; x <= last; x += gridDim.x) {
    const int page = c.table[static_cast<size_t>(blockIdx.z) * c.table_stride + x];
    const bool held = static_cast<unsigned>(page) < static_cast<unsigned>(c.pages);
    const int lo = max(q.start, x << c.log_page), hi = min(q.len, (x + 1) << c.log_page), s0 = lo & (P - 1);
    const size_t block = static_cast<size_t>(held ? page : 0) * c.heads + head;
    const float2 s = reinterpret_cast<const float2*>(c.scales)[block];
    const int8_t* kp = c.k + block * P * D;
    const uint4* vp = reinterpret_cast<const uint4*>(c.v + block * P * D);
    const auto key = [&](int i) {                            // 16 key codes of item i
      return *reinterpret_cast<const uint4*>(kp + static_cast<size_t>(s0 + (i >> log_dp)) * D + 16 * (i & (DP - 1)));
    };
    const int n = (hi - lo) << log_dp;
    const uint4 first_key = key(min(tid, n - 1));            // on its way beside the values
    const int c0 = s0 >> 4, pieces = ((s0 + hi - lo + 15) >> 4) - c0;
    for (int i = tid; i < D * pieces; i += blockDim.x) {
      const int d = i / pieces, piece = c0 + i - d * pieces;
      const uint4 w = vp[(d << (c.log_page - 4)) + piece];
      uint32_t* o = reinterpret_cast<uint32_t*>(turn + d * stride + 16 * piece);
      o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
    }
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x) {
      const int t = i >> log_dp, p = i & (DP - 1);
      const size_t row = static_cast<size_t>(q.row + (lo - q.start) + t);
      const uint4 w = i == tid ? first_key : key(i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      float kx[16], vx[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        kx[j] = s.x * static_cast<float>(static_cast<int8_t>(u[j >> 2] >> (8 * (j & 3))));
        vx[j] = s.y * static_cast<float>(static_cast<int8_t>(turn[(16 * p + j) * stride + s0 + t]));
      }
      const size_t o = ((row * c.heads + head) * D + 16 * p) / 8;
      reinterpret_cast<uint4*>(K)[o] = held ? narrow8<BF16>(kx) : zero;
      reinterpret_cast<uint4*>(K)[o + 1] = held ? narrow8<BF16>(kx + 8) : zero;
      reinterpret_cast<uint4*>(V)[o] = held ? narrow8<BF16>(vx) : zero;
      reinterpret_cast<uint4*>(V)[o + 1] = held ? narrow8<BF16>(vx + 8) : zero;
    }
    __syncthreads();
  }
}

// Pages that max_new consecutive tokens can touch.
int touched_pages(const Kv8View& c) {
  const long long P = 1LL << c.log_page;
  return static_cast<int>(std::min<long long>((c.max_new + 2 * P - 2) / P, 1 << 20));
}

template <bool BF16>
void append_launch(const Kv8AppendArgs& a, hipStream_t stream) {
  const int items = (a.c.dim / 16) << a.c.log_page;                    // of a full page: 64 .. 2048
  const dim3 grid(touched_pages(a.c), a.Q ? 2 * a.c.heads : a.c.heads, a.c.seqs);
  const size_t lds = static_cast<size_t>(a.c.dim) << a.c.log_page;
  const int threads = items >= 2048 ? 512 : std::min(items, 256);
  switch (items / threads) {
    case 1: hipLaunchKernelGGL((kv8_append_kernel<BF16, 1>), grid, dim3(threads), lds, stream, a); break;
    case 2: hipLaunchKernelGGL((kv8_append_kernel<BF16, 2>), grid, dim3(threads), lds, stream, a); break;
    default: hipLaunchKernelGGL((kv8_append_kernel<BF16, 4>), grid, dim3(threads), lds, stream, a); break;
  }
}

}  // namespace

void kv8_append_launch(const Kv8AppendArgs& a, int dtype, hipStream_t stream) {
  if (dtype == QLIN_BF16) append_launch<true>(a, stream);
  else append_launch<false>(a, stream);
}

void kv8_gather_launch(const Kv8View& c, uint16_t* K, uint16_t* V, int dtype, hipStream_t stream) {
  const dim3 grid(touched_pages(c), c.heads, c.seqs);
  const size_t lds = static_cast<size_t>(c.dim) * ((1 << c.log_page) + 4);
  if (dtype == QLIN_BF16) hipLaunchKernelGGL(kv8_gather_kernel<true>, grid, dim3(256), lds, stream, c, K, V);
  else hipLaunchKernelGGL(kv8_gather_kernel<false>, grid, dim3(256), lds, stream, c, K, V);
}

}  // namespace qlin
