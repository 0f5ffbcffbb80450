// Attention over the 8-bit paged key/value cache, gfx950: the kernel for many query
// rows per key/value head (prompts and chunks of prompts).
//
// The mathematics and the transposed products are those of the kernel for few
// rows (kv8_attn.hip), on the 32x32x16 matrix instruction: a workgroup of W waves
// holds 32 W rows (token by token, the query heads that share a key/value head
// next to each other), walks the tiles of 64 positions that any of them sees and
// shares each tile through LDS: every thread converts its part of the next
// tile's codes to fp16 once, while the waves multiply the present one.
//   S^T = K Q^T  lane (q, h) (q = lane % 32, h = lane / 32) gets, of each run of 16
//   O^T += V^T P tokens, the weights of tokens 8 h .. 8 h + 7 for row q: the B
//                operand of the second product as it stands, because K's rows are
//                fed in the order that makes it so.
// A run of 16 tokens lies in one page: its two scales are the same for every lane.
//
// Bound by the matrix and vector units together, under the power limit: a prompt
// of 8192 with 64 / 8 heads of 128 runs at 0.96 PFLOP/s (a large fp16 product of
// the library at 1.17), 1.1 on operands of zeros; the matrix units are busy 45 %
// of the cycles, the vector units (an exponential, a multiply-add, a sum, half a
// maximum and half a conversion for each score) about 55 %.  Taking the
// exponentials, the conversions or the LDS reads out one at a time gains 0-11 %
// each.  Tried without gain: the next tile's scores beside this tile's weights
// (30 more registers; 7 % for heads of 256 only, since overtaken by the look-ahead),
// vector work dealt out between the products by hand, 4 waves instead of 8.

#include <algorithm>

#include "common.hpp"
#include "device.hpp"
#include "kv8.hpp"
#include "kv8_device.hpp"

namespace qlin {

namespace {

// Waves of a workgroup, and of a SIMD.  A code is converted once per workgroup, so
// more waves convert less (prompt of 8192 with heads of 128: 8 waves 1.24, 4 waves
// 1.31 ms); heads of 256 dimensions fill the registers with one wave per SIMD.  A
// third wave for heads of 64 changes nothing.
template <int D>
constexpr int kPromptWaves = D == 128 ? 8 : 4;
template <int D>
constexpr int kPromptOccupancy = D > 128 ? 1 : 2;

// A run of 16 tokens of a tile: its key scale, log2 and reciprocal of its value
// scale.
struct alignas(16) Run {
  float key, lv, iv;
};

// fp16 tiles in LDS, rows padded by 16 bytes so that 16 lanes reading 16 bytes
// each of consecutive rows hit every bank once.
template <int D>
struct alignas(16) Tile16 {
  _Float16 k[kTile][D + 8];
  _Float16 v[D][kTile + 8];
  Run run[4];
  uint32_t held;                                            // bit s: run s has a page
};

// Schedules the N products of this block, whose A operands come from LDS, so that a
// product's operand is on its way six products ahead, and ends the scheduling
// region.  The compiler alone asks for it one product ahead and waits each time:
// heads of 256, one wave to a SIMD: a prompt of 4096 with 16 heads 230 -> 202 us; heads of
// 128: 1046 -> 1001 us on operands of zeros, where the clock does not sink.
template <int N>
__device__ __forceinline__ void lookahead() {
  constexpr int AHEAD = 6;
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);     // LDS reads
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);         // a matrix product
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// A row tile: rows r0 .. r0 + nrows - 1 of a sequence, the tiles they see and how
// many of them a split takes.  Row tiles beyond those planned for are not split:
// their partial results would share workspace with the first ones'.
template <int D>
struct RowTile {
  static constexpr int ROWS = 32 * kPromptWaves<D>;
  int nrows, p0, p1;
  Kv8Tiles tiles;
  int per, used;
  __device__ __forceinline__ RowTile(const Kv8AttnArgs& a, const Kv8Seq& seq, int rows, int r0)
      : nrows(min(rows - r0, ROWS)), p0(seq.start + a.by_group(r0)), p1(seq.start + a.by_group(r0 + nrows - 1)),
        tiles(p0, p1, a.window, a.sinks) {
    const bool planned = r0 < a.row_tiles * ROWS;
    per = planned ? max(a.chunk, a.by_splits(tiles.count + a.splits - 1)) : max(tiles.count, 1);
    used = per >= tiles.count ? 1 : (tiles.count + per - 1) / per;
  }
};

// Floats of a split's partial result: per wave and lane its 16 DT sums, the
// reference and the sum of weights.
template <int D>
constexpr int kPromptSlot = kPromptWaves<D> * 64 * (D / 2 + 2);

// Threads of a workgroup that joins splits, SHARE waves to a task.
template <int SHARE>
constexpr int kJoinThreads = SHARE > 4 ? 64 * SHARE : 256;

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kPromptWaves<D>, kPromptOccupancy<D>) void kv8_prompt_kernel(const Kv8AttnArgs a) {
  constexpr int W = kPromptWaves<D>, NT = 64 * W, ROWS = 32 * W, DT = D / 32, KS = D / 16;
  constexpr int NL = D * kTile / 16 / NT;                  // 16-byte pieces of K (and of V) per thread and tile
  extern __shared__ __align__(16) char smem[];
  Tile16<D>* tile = reinterpret_cast<Tile16<D>*>(smem);    // two of them
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, h = lane >> 5, ql = lane & 31;
  const int unit = a.by_heads(blockIdx.x), head = blockIdx.x - unit * a.c.heads;
  const int b = a.by_row_tiles(unit), split = blockIdx.y;
  const Kv8Seq seq = kv8_seq(a.c, b);
  const int P = 1 << a.c.log_page, G = a.group;
  const int rows = seq.count * G;                             // below 2^30
  if (rows < a.least_rows || rows > a.most_rows) return;
  const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.table_stride;
  const int last_entry = (seq.len - 1) >> a.c.log_page;    // entries past it are not read

  // Row tiles from the last, which sees the most, to the first; row tiles past
  // the grid are taken up in turn.
  for (int r0 = (a.row_tiles - 1 - (unit - b * a.row_tiles)) * ROWS; r0 < rows; r0 += a.row_tiles * ROWS) {
    const RowTile<D> rt(a, seq, rows, r0);
    const int nrows = rt.nrows, p0 = rt.p0, p1 = rt.p1;
    const Kv8Tiles& tiles = rt.tiles;
    if (split >= rt.used) continue;
    const int x0 = split * rt.per, x1 = min(x0 + rt.per, tiles.count);

    // this lane's row
    const int r = r0 + min(32 * wv + ql, nrows - 1), t = a.by_group(r), hq = head * G + r - t * G;
    const bool mine = 32 * wv + ql < nrows;
    const int pos = seq.start + t, low = a.window > 0 ? max(pos, 0) - a.window + 1 : 0;
    const int low_most = a.window > 0 ? max(p1, 0) - a.window + 1 : 0;
    h8_t qf[KS];                                            // slice s: dimensions 16 s + 8 h .. + 7
    float cq = a.scale;
    {
      int again = tid;
      asm volatile("" : "+v"(again));                       // (nothing of the address to be held for the next rows)
      const uint16_t* row = a.Q + static_cast<size_t>(seq.row + t) * a.q_stride + static_cast<size_t>(hq) * D + ((again & 32) >> 2);
      if constexpr (BF16) {
        uint32_t most = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) most = max(most, chunk_most(*reinterpret_cast<const uint4*>(row + 16 * s)));
        const int e = row_exponent(most_over_32(most));
        cq *= ldexpf(1.0f, e);
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = chunk_f16(*reinterpret_cast<const uint4*>(row + 16 * s), e);
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const h8_t*>(row + 16 * s);
      }
    }
    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    float m = kNone, l = 0.0f;

    // Loads of a tile.  A thread's place in the tile's pages is fixed (but for where
    // the tile lies in pages longer than it): its K row `token` and its V piece (16
    // tokens, number tid % 4) each have one page entry, the latter also that of the
    // run of tokens whose scales the thread takes.  Its n-th pieces lie STEP tokens
    // (a multiple of 16, so `token` stays in the same place of a page) and NT / 4
    // dimensions further.
    constexpr int STEP = NT / (D / 16);
    const size_t block_bytes = static_cast<size_t>(D) << a.c.log_page;
    const int token = tid / (D / 16);
    const uint32_t kplace = (token & (P - 1)) * D + 16 * (tid % (D / 16));
    const uint32_t vplace = ((tid / 4) << a.c.log_page) + ((16 * (tid % 4)) & (P - 1));
    const int kentry = token >> a.c.log_page, ventry = (16 * (tid % 4)) >> a.c.log_page;
    uint4 kw[NL], vw[NL];
    int kpage[NL], vpage;
    float2 scale2;
    bool held_next;
    auto block_of = [&](int page) {                         // pages that are not there: any other
      return static_cast<uint32_t>(static_cast<unsigned>(page) < static_cast<unsigned>(a.c.pages) ? page : 0) * a.c.heads + head;
    };
    auto load_pages = [&](int x) {
      const int entry = (tiles[min(x, x1 - 1)] * kTile) >> a.c.log_page;
#pragma unroll
      for (int n = 0; n < NL; ++n) kpage[n] = table[static_cast<unsigned>(min(entry + kentry + ((n * STEP) >> a.c.log_page), last_entry))];
      vpage = table[static_cast<unsigned>(min(entry + ventry, last_entry))];
    };
    auto load_codes = [&](int x) {
      const int within = (tiles[min(x, x1 - 1)] * kTile) & (P - 1);
#pragma unroll
      for (int n = 0; n < NL; ++n)
        kw[n] = *reinterpret_cast<const uint4*>(a.c.k + (block_of(kpage[n]) * block_bytes + (kplace + (within + ((n * STEP) & (P - 1))) * D)));
      const uint32_t block = block_of(vpage);
#pragma unroll
      for (int n = 0; n < NL; ++n)
        vw[n] = *reinterpret_cast<const uint4*>(a.c.v + (block * block_bytes + (vplace + within + ((n * (NT / 4)) << a.c.log_page))));
      scale2 = reinterpret_cast<const float2*>(a.c.scales)[block];
      held_next = static_cast<unsigned>(vpage) < static_cast<unsigned>(a.c.pages);
    };
    auto put_codes = [&](Tile16<D>& to) __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const int i = tid + n * NT, token = i / (D / 16), c = i % (D / 16);
        *reinterpret_cast<h8_t*>(&to.k[token][16 * c]) = codes_f16(kw[n].x, kw[n].y);
        *reinterpret_cast<h8_t*>(&to.k[token][16 * c + 8]) = codes_f16(kw[n].z, kw[n].w);
        *reinterpret_cast<h8_t*>(&to.v[i / 4][16 * (i % 4)]) = codes_f16(vw[n].x, vw[n].y);
        *reinterpret_cast<h8_t*>(&to.v[i / 4][16 * (i % 4) + 8]) = codes_f16(vw[n].z, vw[n].w);
      }
    };
    auto put_runs = [&](Tile16<D>& to) {
      if (tid < 4) {
        const float vs = scale2.y < kLeastScale ? kLeastScale : scale2.y;     // NaN stays
        to.run[tid] = Run{scale2.x, __log2f(vs), __builtin_amdgcn_rcpf(vs)};
      }
      const uint32_t held = static_cast<uint32_t>(__ballot(held_next)) & 15u;  // lanes 0 .. 3 of wave 0: the four runs
      if (tid == 0) to.held = held;
    };

    if (x0 < x1) {
      load_pages(x0);
      load_codes(x0);
      load_pages(x0 + 1);
      put_codes(tile[0]);
      put_runs(tile[0]);
      // (the loop inside this block, so that its waits know that the queries are there)
      // K row that this lane feeds to row `lane % 32` of a 32-token product
      const int krow = 16 * (ql >> 4) + 8 * ((ql >> 2) & 1) + 4 * ((ql >> 3) & 1) + (ql & 3);
      for (int x = x0; x < x1; ++x) {
        const Tile16<D>& now = tile[(x - x0) & 1];
        const int base = tiles[x] * kTile;
        load_codes(x + 1);
        load_pages(x + 2);
        __syncthreads();                                      // the tile is complete, and the other one is free
        f32x16_t st[2];
#pragma unroll
        for (int T = 0; T < 2; ++T) {
#pragma unroll
          for (int i = 0; i < 16; ++i) st[T][i] = 0.0f;
#pragma unroll
          for (int s = 0; s < KS; ++s)
            st[T] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const h8_t*>(&now.k[32 * T + krow][16 * s + 8 * h]), qf[s],
                                                           st[T], 0, 0, 0);
        }
        lookahead<2 * KS>();
        float c[4], lv[4], iv[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const Run run = now.run[s];
          c[s] = run.key * cq;
          lv[s] = run.lv;
          iv[s] = run.iv;
        }
        const uint32_t held = __builtin_amdgcn_readfirstlane(now.held);
        const bool full = base + kTile - 1 <= p0 && (base >= low_most || base + kTile <= a.sinks) && held == 15u;
        uint32_t seen[4];                                     // bit i of run s: this lane's token i
        float top = kLowest;
        if (!full) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            seen[s] = visible_bits<8>(base + 16 * s + 8 * h, pos, low, a.sinks, (held >> s) & 1u);
            c[s] = seen[s] != 0 ? c[s] : 0.0f;                // (a hidden page's scale may be below 0: -inf must not turn)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st[s >> 1][8 * (s & 1) + i] = (seen[s] >> i) & 1u ? st[s >> 1][8 * (s & 1) + i] : -INFINITY;
          }
          top = (seen[0] | seen[1] | seen[2] | seen[3]) != 0 ? kLowest : kNone;
        }
        // run s: values st[s / 2][8 (s % 2) .. + 7]
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          float mx = st[s >> 1][8 * (s & 1)];
#pragma unroll
          for (int i = 1; i < 8; ++i) mx = fmaxf(mx, st[s >> 1][8 * (s & 1) + i]);
          top = fmaxf(top, fmaf(mx, c[s], lv[s]));
        }
        if (__any(top > m + kSlack)) {
          const float high = max_over_32(top), was = m;
          m = high > was + kSlack ? high - kHead : was;               // by the row's own scores alone
          const float f = __builtin_amdgcn_exp2f(was - m);
          l *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] *= f;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float shift = lv[s] - m;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = 8 * (s & 1) + i;
            st[s >> 1][k] = __builtin_amdgcn_exp2f(fmaf(st[s >> 1][k], c[s], shift));
          }
        }
        if (!full) {                                          // scales of hidden pages may be anything, NaN among it
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            iv[s] = seen[s] != 0 ? iv[s] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st[s >> 1][8 * (s & 1) + i] = (seen[s] >> i) & 1u ? st[s >> 1][8 * (s & 1) + i] : 0.0f;
          }
        }
        h8_t pf[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          float part = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float p = st[s >> 1][8 * (s & 1) + i];
            part += p;
            pf[s][i] = static_cast<_Float16>(p);
          }
          l = fmaf(part, iv[s], l);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int d = 0; d < DT; ++d)
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const h8_t*>(&now.v[32 * d + ql][16 * s + 8 * h]), pf[s],
                                                          o[d], 0, 0, 0);
        put_codes(tile[(x - x0 + 1) & 1]);
        lookahead<4 * DT>();
        put_runs(tile[(x - x0 + 1) & 1]);
      }
    }
    l = sum_over_32(l);

    if (rt.used > 1) {
      // every value at its register's and lane's own place, for the joining kernel
      int place = wv * 64 * (16 * DT + 2) + lane;
      asm volatile("" : "+v"(place));                       // its 16 DT addresses are not to be held through the loop
      float* part = a.partials + (static_cast<size_t>(blockIdx.x) * a.splits + split) * kPromptSlot<D> + place;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) part[64 * (16 * d + i)] = o[d][i];
      part[64 * 16 * DT] = m;
      part[64 * 16 * DT + 64] = l;
    } else if (mine) {
      const float inv = by_weights(l, m);
      int again = tid;
      asm volatile("" : "+v"(again));                       // (nothing of the address to be held through the loop)
      uint16_t* y = a.Y + (static_cast<size_t>(seq.row + t) * a.q_heads + hq) * D + ((again & 32) >> 3);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<uint2*>(y + 32 * d + 2 * i) =
              make_uint2(pack2<BF16>(o[d][i] * inv, o[d][i + 1] * inv), pack2<BF16>(o[d][i + 2] * inv, o[d][i + 3] * inv));
    }
    __syncthreads();                                        // the tiles may be used for the next rows
  }
}

// Joins the splits of row tiles, in their order, spread over the whole device (one
// workgroup joining 64 splits of 256 rows would read 9 MB by itself): a row tile's
// wave and a group of four of its sums are a task, of SHARE waves that take
// consecutive splits each.  What bounds it is the latency of its loads: with one
// wave to a task 64 splits took 24.5 us, with sixteen, whose loads all leave at
// once, 5 us.
template <int D, int SHARE, bool BF16>
__global__ __launch_bounds__(kJoinThreads<SHARE>) void kv8_prompt_join_kernel(const Kv8AttnArgs a) {
  constexpr int GROUPS = D / 8, AHEAD = 8;
  const int lane = threadIdx.x & 63, h = lane >> 5, ql = lane & 31, wave = threadIdx.x >> 6, member = wave % SHARE;
  const int task = blockIdx.y * (kJoinThreads<SHARE> / 64 / SHARE) + wave / SHARE, wv = task / GROUPS, group = task % GROUPS;
  const int unit = a.by_heads(blockIdx.x), head = blockIdx.x - unit * a.c.heads, b = a.by_row_tiles(unit);
  const Kv8Seq seq = kv8_seq(a.c, b);
  const int rows = seq.count * a.group, r0 = (a.row_tiles - 1 - (unit - b * a.row_tiles)) * RowTile<D>::ROWS;
  if (r0 >= rows || rows < a.least_rows || rows > a.most_rows) return;
  const RowTile<D> rt(a, seq, rows, r0);
  if (rt.used == 1 || 32 * wv >= rt.nrows) return;          // (the same for all of a task)
  const float* part = a.partials + static_cast<size_t>(blockIdx.x) * a.splits * kPromptSlot<D> + wv * 64 * (D / 2 + 2) + lane;
  const int each = (rt.used + SHARE - 1) / SHARE, k1 = min(rt.used, (member + 1) * each);
  float m = kNone, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = member * each; k < k1; k += AHEAD) {
    float ref[AHEAD], sum[AHEAD], v[AHEAD][4];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const float* at = part + static_cast<size_t>(min(k + j, k1 - 1)) * kPromptSlot<D>;
      ref[j] = at[64 * (D / 2)];
      sum[j] = at[64 * (D / 2 + 1)];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = at[64 * (4 * group + i)];
    }
    float next = m;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) next = fmaxf(next, ref[j]);
    const float f = __builtin_amdgcn_exp2f(m - next);
    m = next;
    l *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= f;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (k + j >= k1) break;
      const float g = __builtin_amdgcn_exp2f(ref[j] - m);
      l = fmaf(sum[j], g, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(v[j][i], g, o[i]);
    }
  }
  if constexpr (SHARE > 1) {
    __shared__ float held[SHARE][6][64];
    held[member][0][lane] = m;
    held[member][1][lane] = l;
#pragma unroll
    for (int i = 0; i < 4; ++i) held[member][2 + i][lane] = o[i];
    __syncthreads();
    if (member) return;
#pragma unroll
    for (int k = 1; k < SHARE; ++k) m = fmaxf(m, held[k][0][lane]);
    l = o[0] = o[1] = o[2] = o[3] = 0.0f;
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
      const float g = __builtin_amdgcn_exp2f(held[k][0][lane] - m);
      l = fmaf(held[k][1][lane], g, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(held[k][2 + i][lane], g, o[i]);
    }
  }
  if (32 * wv + ql >= rt.nrows) return;
  const int r = r0 + 32 * wv + ql, t = a.by_group(r), hq = head * a.group + r - t * a.group;
  const float inv = by_weights(l, m);
  uint16_t* y = a.Y + (static_cast<size_t>(seq.row + t) * a.q_heads + hq) * D + 32 * (group >> 2) + 8 * (group & 3) + 4 * h;
  *reinterpret_cast<uint2*>(y) = make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
}

template <int D, int SHARE>
void join_launch(const Kv8AttnArgs& a, int dtype, unsigned units, hipStream_t stream) {
  constexpr int kTasks = kPromptWaves<D> * (D / 8);
  const dim3 grid(units, kTasks / (kJoinThreads<SHARE> / 64 / SHARE)), block(kJoinThreads<SHARE>);
  const auto fn = dtype == QLIN_BF16 ? kv8_prompt_join_kernel<D, SHARE, true> : kv8_prompt_join_kernel<D, SHARE, false>;
  hipLaunchKernelGGL(fn, grid, block, 0, stream, a);
}

template <int D>
void prompt_launch(const Kv8AttnArgs& a, int dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.c.seqs) * a.row_tiles * a.c.heads, a.splits), block(64 * kPromptWaves<D>);
  const size_t lds = 2 * sizeof(Tile16<D>);
  const auto fn = dtype == QLIN_BF16 ? kv8_prompt_kernel<D, true> : kv8_prompt_kernel<D, false>;
  hipLaunchKernelGGL(fn, grid, block, lds, stream, a);
  if (a.splits > 32) join_launch<D, 16>(a, dtype, grid.x, stream);
  else if (a.splits > 8) join_launch<D, 4>(a, dtype, grid.x, stream);
  else if (a.splits > 1) join_launch<D, 1>(a, dtype, grid.x, stream);
}

}  // namespace

int kv8_prompt_rows(int dim) { return 32 * (dim == 64 ? kPromptWaves<64> : dim == 128 ? kPromptWaves<128> : kPromptWaves<256>); }

int kv8_prompt_resident(int dim) {
  return dim == 64 ? 4 * kPromptOccupancy<64> / kPromptWaves<64>
                   : dim == 128 ? 4 * kPromptOccupancy<128> / kPromptWaves<128> : 4 * kPromptOccupancy<256> / kPromptWaves<256>;
}

size_t kv8_prompt_partial(int dim) {
  return sizeof(float) * (dim == 64 ? kPromptSlot<64> : dim == 128 ? kPromptSlot<128> : kPromptSlot<256>);
}

void kv8_prompt_launch(const Kv8AttnArgs& a, int dtype, hipStream_t stream) {
  switch (a.c.dim) {
    case 64: prompt_launch<64>(a, dtype, stream); break;
    case 128: prompt_launch<128>(a, dtype, stream); break;
    default: prompt_launch<256>(a, dtype, stream); break;
  }
}

}  // namespace qlin
