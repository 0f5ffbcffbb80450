// Attention over the 8-bit paged key/value cache, gfx950: the kernel for few query
// rows per key/value head (single tokens, draft verification, short prompts).
//
//   O[q] = sum_j p_qj t_j v_j / sum_j p_qj,   p_qj = exp2(c_q s_j (q . k_j))
// with the codes k_j, v_j, the page scales s_j (keys) and t_j (values) and
// c_q = scale log2(e).  One pass with a running reference m_q (below).
//
// A row is one (token, query head) pair; the rows of the query heads that share
// a key/value head and of all the call's tokens of a sequence are numbered token
// by token, so one read of the cache serves 16 NT of them.  Each wave walks
// tiles of 64 positions on its own, with nothing shared and no barrier:
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16, A = K codes, B = Q (in registers)
//   O^T += V^T P  A = V^T codes, B = P
// The transposed products leave, in lane (q, g) (q = lane % 16, g = lane / 16),
// the weights of one row and 16 consecutive tokens 16 g .. 16 g + 15: exactly
// the B operand of the second product when its contraction index is permuted the
// same way, so P never leaves the registers, and as pages hold whole runs of 16
// tokens a lane needs one page scale whatever the page size.  K rows are read in
// the order that makes this so; V^T is stored with tokens contiguous, so both
// operands come from memory in 16-byte pieces, without LDS, one tile ahead of
// their use.
//
// Codes become exact fp16 integers (one v_perm for two codes and one packed
// subtraction).  The key scale multiplies the fp32 scores.  The value scale t_j
// goes into the weights, in the exponent: p'_qj = p_qj t_j 2^-m_q, with the
// reference m_q somewhat below the row's maximum of score + log2 t_j, so the largest
// p' are 2^7 to 2^15: p' down to 2^-14 round to fp16 with 11 bits, smaller ones to
// a multiple of 2^-24.  O[q] = sum p' (codes of v) / sum p' / t, the sum of weights
// in fp32.
//
// The reference only has to be near the maximum: it moves (and the sums are
// rescaled) when a score exceeds it by more than kSlack, which spares the
// cross-lane maximum and the rescaling in most tiles.
//
// Bound by memory: 2 D bytes a token against 4 D 16 NT matrix flops.  64 ragged
// sequences of up to 8192 tokens (8 heads of 128, 499 MB) run at 6.0 TB/s, one of
// 131072 (269 MB) at 5.5, where a bare streaming read of the same sizes makes 7.0
// and 6.7.  The vector units are busy 45 % of the time (conversion of the codes
// two thirds of it); what is left is the beginning and the end of a workgroup:
// the chain lengths -> page -> codes, and joining the waves and the splits (2, 2
// and 4 us of the 49 us of 131072 tokens).  Tried without gain: 32 positions to a step
// with twice the waves (64 sequences 103 -> 117 us at the time), 128 registers for
// four waves per SIMD (103 -> 141).

#include <algorithm>

#include "common.hpp"
#include "device.hpp"
#include "kv8.hpp"
#include "kv8_device.hpp"
#include "splitk.hpp"

namespace qlin {

namespace {

// Waves of a SIMD that the registers allow.
constexpr int row_occupancy(int dim, int nt) { return dim * nt <= 128 ? 2 : 1; }
constexpr int kMostSplits = 64;           // a lane each when they are joined
constexpr int kMostManySplits = 256;      // of the kernel for many rows: joined by a kernel of its own
// 16 NT query rows as B operands: lane (q, g), slice (u, e) holds dimensions
// 64 u + 16 g + 8 e .. + 7 of row q.  bf16 rows are scaled by a power of two into
// fp16's range; *mul is what undoes it.
template <int D, bool BF16>
__device__ __forceinline__ void load_rows(const uint16_t* row, int g, h8_t (&q)[D / 64][2], float* mul) {
  uint4 w[D / 64][2];
#pragma unroll
  for (int u = 0; u < D / 64; ++u)
#pragma unroll
    for (int e = 0; e < 2; ++e) w[u][e] = *reinterpret_cast<const uint4*>(row + 64 * u + 16 * g + 8 * e);
  if constexpr (!BF16) {
    *mul = 1.0f;
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) q[u][e] = bitcast<h8_t>(w[u][e]);
  } else {
    uint32_t most = 0;
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) most = max(most, chunk_most(w[u][e]));
    const int e14 = row_exponent(most_over_g(most));
    *mul = ldexpf(1.0f, e14);
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) q[u][e] = chunk_f16(w[u][e], e14);
  }
}

// Partial result of a split: [16 NT][D] sums, then [16 NT] (reference, sum of weights).
template <int D, int NT>
constexpr size_t kPartial = 16 * NT * (D + 2);

// Grid: splits x (sequence, row tile) x key/value heads, heads fastest.
// STREAM: V is read past the caches, which pays where a load covers whole 128-byte
// lines (of pages of 128 tokens it takes every other half line): 131072 tokens of
// 8 heads 54 -> 50 us, but 32 x 8192 tokens in pages of 128 99 -> 111 us.  K's
// lines are shared by two loads each and stay cached.
template <int D, int NT, int W, bool BF16, bool STREAM>
__global__ __launch_bounds__(64 * W, row_occupancy(D, NT)) void kv8_rows_kernel(const Kv8AttnArgs a) {
  constexpr int KU = D / 64, DT = D / 16;
  __shared__ __align__(16) float sums[W][16][D + 4];
  __shared__ float refs[W][16 * NT], weights[W][16 * NT];
  __shared__ int flag;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, g = lane >> 4, ql = lane & 15;
  const int unit = a.by_heads(blockIdx.x), head = blockIdx.x - unit * a.c.heads;
  const int rank = a.by_row_tiles(unit), split = blockIdx.y;
  const int b = !a.sorted ? rank : a.c.seqs <= 64 ? nth_longest<1>(a.c, rank) : nth_longest<kSortedSeqs / 64>(a.c, rank);
  const Kv8Seq seq = kv8_seq(a.c, b);
  const int P = 1 << a.c.log_page, G = a.group;
  const int rows = seq.count * G;                             // below 2^30
  if (rows < a.least_rows || rows > a.most_rows) return;
  // row tiles past the grid are taken up in turn
  for (int r0 = (unit - rank * a.row_tiles) * (16 * NT); r0 < rows; r0 += a.row_tiles * (16 * NT)) {
    const int nrows = min(rows - r0, 16 * NT);
    const int p0 = seq.start + a.by_group(r0), p1 = seq.start + a.by_group(r0 + nrows - 1);
    const Kv8Tiles tiles(p0, p1, a.window, a.sinks);
    // row tiles beyond those planned for are not split: their partial results
    // would share workspace with the first ones'
    const bool planned = r0 < a.row_tiles * (16 * NT);
    const int per = planned ? max(a.chunk, a.by_splits(tiles.count + a.splits - 1)) : max(tiles.count, 1);
    if (split > 0 && split * per >= tiles.count) continue;
    const int used = per >= tiles.count ? 1 : (tiles.count + per - 1) / per;
    const int x0 = split * per + wv, x1 = min(split * per + per, tiles.count);

    h8_t qf[NT][KU][2];
    float cq[NT], m[NT], l[NT];
    int pos[NT], low[NT];                    // visible: j <= pos and (j >= low or j < sinks)
    f32x4_t o[NT][DT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = r0 + min(16 * n + ql, nrows - 1), t = a.by_group(r), h = head * G + r - t * G;
      load_rows<D, BF16>(a.Q + static_cast<size_t>(seq.row + t) * a.q_stride + static_cast<size_t>(h) * D, g, qf[n], &cq[n]);
      cq[n] *= a.scale;
      pos[n] = seq.start + t;
      low[n] = a.window > 0 ? max(pos[n], 0) - a.window + 1 : 0;
      m[n] = kNone;
      l[n] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[n][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int low_most = a.window > 0 ? max(p1, 0) - a.window + 1 : 0;

    // Loads of a tile: the pages of this lane's K rows (tokens 16 ((lane / 4) % 4) + ..)
    // and V rows (tokens 16 g ..).
    const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.table_stride;
    const int last_entry = (seq.len - 1) >> a.c.log_page;       // entries past it are not read
    const int gk = (ql >> 2);
    const int xl = x0 + (max(x1 - x0, 1) - 1) / W * W;   // this wave's last tile
    struct Pages { int k, v; };
    auto load_pages = [&](int x) {
      const int base = tiles[min(x, xl)] * kTile;
      return Pages{table[min((base + 16 * gk) >> a.c.log_page, last_entry)], table[min((base + 16 * g) >> a.c.log_page, last_entry)]};
    };
    auto valid = [&](int page) { return static_cast<unsigned>(page) < static_cast<unsigned>(a.c.pages); };
    uint4 kw[4][KU], vw[DT];
    float2 sc;
    bool held;
    // Past the wave's last tile the loads are still issued (a branch around them
    // would make the waits for the present tile wait for everything), all lanes at
    // the pool's first bytes.
    auto load_k = [&](int x, const Pages& p) {
      const int base = tiles[min(x, xl)] * kTile;
      const size_t pk = valid(p.k) ? p.k : 0, pv = valid(p.v) ? p.v : 0;
      held = valid(p.v);
      sc = reinterpret_cast<const float2*>(a.c.scales)[pv * a.c.heads + head];   // not looked at unless held
      const size_t at = (((pk * a.c.heads + head) << a.c.log_page) + ((base + 16 * gk) & (P - 1)) + (ql & 3)) * D + 16 * g;
      const int8_t* src = a.c.k + (x <= xl ? at : 0);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < KU; ++u) kw[t][u] = *reinterpret_cast<const uint4*>(src + 4 * t * D + 64 * u);
    };
    auto load_v = [&](int x, const Pages& p) {
      const int base = tiles[min(x, xl)] * kTile;
      const size_t pv = valid(p.v) ? p.v : 0;
      const size_t at = (((pv * a.c.heads + head) * D + ql) << a.c.log_page) + ((base + 16 * g) & (P - 1));
      const int8_t* src = a.c.v + (x <= xl ? at : 0);
      if constexpr (STREAM) {
#pragma unroll
        for (int d = 0; d < DT; ++d) vw[d] = load_stream16(src + (static_cast<size_t>(16 * d) << a.c.log_page));
      } else {
#pragma unroll
        for (int d = 0; d < DT; ++d) vw[d] = *reinterpret_cast<const uint4*>(src + (static_cast<size_t>(16 * d) << a.c.log_page));
      }
    };

    if (x0 < x1) {
      Pages now = load_pages(x0), next = load_pages(x0 + W);
      load_k(x0, now);
      load_v(x0, now);
      for (int x = x0; x < x1; x += W) {
        const int base = tiles[x] * kTile, j0 = base + 16 * g;
        const bool here = held;
        const float2 s = sc;
        f32x4_t st[NT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int n = 0; n < NT; ++n) st[n][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 0; u < KU; ++u) {
            const h8_t k0 = codes_f16(kw[t][u].x, kw[t][u].y), k1 = codes_f16(kw[t][u].z, kw[t][u].w);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              st[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][u][0], st[n][t], 0, 0, 0);
              st[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[n][u][1], st[n][t], 0, 0, 0);
            }
          }
        }
        const Pages coming = next;
        next = load_pages(x + 2 * W);
        load_k(x + W, coming);

        // every position of the tile visible to every row, and every page there
        const bool full = base + kTile - 1 <= p0 && (base >= low_most || base + kTile <= a.sinks) && !__any(!here);
        const float vs = s.y < kLeastScale ? kLeastScale : s.y;                // NaN stays
        const float lv = __log2f(vs), iv = 1.0f / vs;
        h8_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float c = s.x * cq[n];
          const uint32_t seen = full ? 0xFFFFu : visible_bits<16>(j0, pos[n], low[n], a.sinks, here);
          float top = seen != 0 ? kLowest : kNone;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) st[n][t][i] = fmaf(st[n][t][i], c, lv);
          if (!full) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) st[n][t][i] = (seen >> (4 * t + i)) & 1u ? st[n][t][i] : -INFINITY;
          }
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, st[n][t][i]);
          if (__any(top > m[n] + kSlack)) {
            const float was = m[n];
            const float high = max_over_g(top);
            m[n] = high > was + kSlack ? high - kHead : was;           // by the row's own scores alone
            const float f = __builtin_amdgcn_exp2f(was - m[n]);
            l[n] *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[n][d] *= f;
          }
          float part = 0.0f;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = __builtin_amdgcn_exp2f(st[n][t][i] - m[n]);   // hidden: exp2(-inf) = 0
              part += p;
              pf[n][t >> 1][4 * (t & 1) + i] = static_cast<_Float16>(p);
            }
          l[n] = fmaf(part, seen != 0 ? iv : 0.0f, l[n]);          // a hidden page's scale may be NaN
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const h8_t v0 = codes_f16(vw[d].x, vw[d].y), v1 = codes_f16(vw[d].z, vw[d].w);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[n][0], o[n][d], 0, 0, 0);
            o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[n][1], o[n][d], 0, 0, 0);
          }
        }
        load_v(x + W, coming);
      }
    }

    // Join the waves: references and sums of weights first, then the sums, 16
    // rows at a time through LDS.
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float all = sum_over_g(l[n]);
      if (g == 0) {
        refs[wv][16 * n + ql] = m[n];
        weights[wv][16 * n + ql] = all;
      }
    }
    __syncthreads();
    const int tile_unit = blockIdx.x;
    float* part = a.partials + (static_cast<size_t>(tile_unit) * a.splits + split) * kPartial<D, NT>;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = refs[0][16 * n + ql];
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, refs[w][16 * n + ql]);
      const float f = exp2f(m[n] - top);
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4_t*>(&sums[wv][ql][16 * d + 4 * g]) = o[n][d] * f;
      __syncthreads();
      for (int i = tid; i < 16 * D / 2; i += 64 * W) {
        const int rr = i / (D / 2), d = 2 * (i - rr * (D / 2)), r = 16 * n + rr;
        if (r >= nrows) break;
        float ref = refs[0][r];
#pragma unroll
        for (int w = 1; w < W; ++w) ref = fmaxf(ref, refs[w][r]);
        float total = 0.0f, y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          total = fmaf(weights[w][r], exp2f(refs[w][r] - ref), total);
          y0 += sums[w][rr][d];
          y1 += sums[w][rr][d + 1];
        }
        if (used == 1) {
          const float inv = by_weights(total, ref);
          const int row = r0 + r, t = a.by_group(row), h = head * G + row - t * G;
          *reinterpret_cast<uint32_t*>(a.Y + (static_cast<size_t>(seq.row + t) * a.q_heads + h) * D + d) = pack2<BF16>(y0 * inv, y1 * inv);
        } else {
          sk_store2(part + r * D + d, y0, y1);
          if (d == 0) sk_store2(part + 16 * NT * D + 2 * r, ref, total);
        }
      }
      __syncthreads();
    }
    if (used == 1) continue;

    // The split that arrives last joins them all, in their order: a wave per row
    // weighs the splits (one per lane), then every thread sums a pair of values.
    if (!sk_arrive_last(a.counters + tile_unit, used - 1, &flag)) continue;
    const float* first = a.partials + static_cast<size_t>(tile_unit) * a.splits * kPartial<D, NT>;
    float* weigh = &sums[0][0][0];                            // [row][split], the rows' factors after them
    float* factor = weigh + 16 * NT * kMostSplits;
    for (int r = wv; r < nrows; r += W) {
      const float2 mine = lane < used ? sk_load2(first + lane * kPartial<D, NT> + 16 * NT * D + 2 * r) : make_float2(kNone, 0.0f);
      const float ref = wave_max(mine.x), f = __builtin_amdgcn_exp2f(mine.x - ref);
      weigh[r * kMostSplits + lane] = f;
      const float total = wave_sum(mine.y * f);
      if (lane == 0) factor[r] = by_weights(total, ref);
    }
    __syncthreads();
    for (int i = tid; i < nrows * (D / 2); i += 64 * W) {
      const int r = i / (D / 2), d = 2 * (i - r * (D / 2));
      const float* src = first + r * D + d;
      const float* f = weigh + r * kMostSplits;
      float y0 = 0.0f, y1 = 0.0f;
      constexpr int AHEAD = 16;                               // loads in flight
      for (int k = 0; k < used; k += AHEAD) {
        float2 v[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) v[j] = sk_load2(src + min(k + j, used - 1) * kPartial<D, NT>);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const float g = k + j < used ? f[k + j] : 0.0f;
          y0 = fmaf(v[j].x, g, y0);
          y1 = fmaf(v[j].y, g, y1);
        }
      }
      const int row = r0 + r, t = a.by_group(row), h = head * G + row - t * G;
      *reinterpret_cast<uint32_t*>(a.Y + (static_cast<size_t>(seq.row + t) * a.q_heads + h) * D + d) = pack2<BF16>(y0 * factor[r], y1 * factor[r]);
    }
    if (tid == 0) sk_reset(a.counters + tile_unit);
    __syncthreads();
  }
}

template <int D, int NT, int W>
void rows_launch(const Kv8AttnArgs& a, int dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.c.seqs) * a.row_tiles * a.c.heads, a.splits), block(64 * W);
  const bool bf16 = dtype == QLIN_BF16, stream_v = a.c.log_page < 7;
  const auto fn = bf16 ? (stream_v ? kv8_rows_kernel<D, NT, W, true, true> : kv8_rows_kernel<D, NT, W, true, false>)
                       : (stream_v ? kv8_rows_kernel<D, NT, W, false, true> : kv8_rows_kernel<D, NT, W, false, false>);
  hipLaunchKernelGGL(fn, grid, block, 0, stream, a);
}

// 16-row column tiles per wave of the kernel for few rows, 0 for the kernel for
// many rows.  One column tile with a workgroup for each 16 rows reads the cache
// once for each of them, and is fastest while these do not fill the device (one,
// two column tiles, many rows; heads of 128: 64 rows over 32768 tokens of 4 heads
// 28, 36 and 32 us, 32 rows over 16 sequences of 2048 of 8 heads 19, 28 and 49);
// then two column tiles (64 sequences of 2048, 64 rows each: 119, 99 and 151 us),
// for up to 32 rows over long sequences already where a quarter is full (32 of
// 8192 of 2 heads: 47, 35 and 35 us at half).  From 65 rows the kernel for many is
// as good or better (128 rows over 32768 tokens of 8 heads: 58, 51 and 49 us).
// Heads of 256 dimensions have registers for one column tile, which pays for up to
// 32 rows (64 sequences of 4096 of 2 heads: 87 against 110 us, 33 to 48 rows 144
// against 112) from eight key/value heads of sequences on (one sequence of 32768
// with 8 heads 47 against 62, with 2 heads 44 against 29).
int rows_nt(const Kv8AttnArgs& a, int cus) {
  const long long rows = static_cast<long long>(a.c.max_new) * a.group, per_tile = static_cast<long long>(a.c.seqs) * a.c.heads;
  const long long units = per_tile * ((rows + 15) / 16);
  if (rows <= 16) return 1;
  if (a.c.dim > 128) return rows <= 32 && per_tile >= 8 ? 1 : 0;
  if (rows <= 64) return units <= (rows <= 32 && a.c.max_kv > 4096 ? cus / 4 : cus) ? 1 : 2;
  return 0;
}

// Waves of a workgroup.  With 4, two workgroups share a compute unit and one's
// beginning and end hide behind the other's tiles: many short sequences are
// faster (200 x 512 tokens of 8 heads 78 -> 52 us, one of 1024 11.5 -> 9.5 us).
// With 8, long sequences that leave at most two workgroups to a compute unit end
// together more nearly (64 ragged ones of up to 8192: 99 -> 86 us) and fewer
// splits have to be joined.  Two column tiles of narrow heads (draft
// verification) have no short form that pays: 27 against 23 us for 32 windows of
// 4096.
int rows_waves(const Kv8AttnArgs& a, int nt, long long units, long long tiles, int cus) {
  if (row_occupancy(a.c.dim, nt) == 1) return 4;
  return nt == 2 || (tiles >= 64 && units * tiles >= 64LL * cus && units <= 2LL * cus) ? 8 : 4;
}

// The launch of one kernel for sequences of up to `rows` rows (nt as above): its
// grid and splits; returns the bytes of its partial results.
size_t plan_launch(Kv8AttnArgs* a, int nt, long long rows, int cus) {
  a->row_columns = nt;
  const long long tile_rows = nt ? 16 * nt : kv8_prompt_rows(a->c.dim);
  const long long most = std::min(std::max<long long>(1, (1LL << 22) / (static_cast<long long>(a->c.seqs) * a->c.heads)), 65535LL);
  a->row_tiles = static_cast<int>(std::min((rows + tile_rows - 1) / tile_rows, most));
  long long tiles = (static_cast<long long>(a->c.max_kv) + kTile - 1) / kTile;
  if (a->window > 0)
    tiles = std::min(tiles, (a->window + tile_rows / a->group) / kTile + 2 + (static_cast<long long>(a->sinks) + kTile - 1) / kTile);
  const long long units = static_cast<long long>(a->c.seqs) * a->row_tiles * a->c.heads;
  a->by_group = FastDiv(a->group);
  a->by_heads = FastDiv(a->c.heads);
  a->by_row_tiles = FastDiv(a->row_tiles);
  a->waves = nt ? rows_waves(*a, nt, units, tiles, cus) : 0;
  // more workgroups than run at once: the longest first
  a->sorted = nt && a->c.seqs > 1 && a->c.seqs <= kSortedSeqs && units > cus;
  a->splits = 1;
  a->by_splits = FastDiv(1);
  a->chunk = static_cast<int>(tiles);
  if (units > kCounterSlots) return 0;
  // Splits: the rounds of the workgroups over the device, times a workgroup's steps
  // (of W tiles; the kernel for many rows takes one at a time) and what its
  // beginning and end, and joining splits, cost in steps.  One workgroup to a
  // compute unit, also where two would fit: twice the splits cost more than they
  // hide (131072 tokens 50 -> 59 us).  Row tiles of a prompt differ in length and
  // are not split once there is one for every workgroup that fits.  Up to 256 splits
  // for many rows (256 rows of one head over 131072 tokens 70 us with 64, 39 with 256).
  const long long slots = static_cast<long long>(cus) * (nt ? 1 : kv8_prompt_resident(a->c.dim));
  const long long steps = nt ? a->waves : 1, alone = 3, split = 5;
  const long long most_splits = nt ? kMostSplits : kMostManySplits;
  long long splits = 1, best = -1;
  for (long long n = 1; (nt || units < slots) && n <= most_splits && n <= std::max<long long>(tiles / 2, 1); ++n) {
    const long long each = ((tiles + n - 1) / n + steps - 1) / steps;
    const long long cost = ((units * n + slots - 1) / slots) * (each + (n > 1 ? split : alone));
    if (best < 0 || cost < best) best = cost, splits = n;
  }
  a->splits = static_cast<int>(splits);
  a->by_splits = FastDiv(a->splits);
  a->chunk = static_cast<int>((tiles + splits - 1) / splits);
  if (a->splits == 1) return 0;
  const size_t partial = nt ? static_cast<size_t>(tile_rows) * (a->c.dim + 2) * sizeof(float) : kv8_prompt_partial(a->c.dim);
  return static_cast<size_t>(units) * splits * partial;
}

void few_launch(const Kv8AttnArgs& a, int dtype, hipStream_t stream) {
  const int nt = a.row_columns;
  const bool wide = a.waves == 8;
  switch (a.c.dim) {
    case 64:
      if (nt == 2) rows_launch<64, 2, 8>(a, dtype, stream);
      else wide ? rows_launch<64, 1, 8>(a, dtype, stream) : rows_launch<64, 1, 4>(a, dtype, stream);
      break;
    case 128:
      if (nt == 2) rows_launch<128, 2, 4>(a, dtype, stream);
      else wide ? rows_launch<128, 1, 8>(a, dtype, stream) : rows_launch<128, 1, 4>(a, dtype, stream);
      break;
    default: rows_launch<256, 1, 4>(a, dtype, stream); break;
  }
}

constexpr int kFewRows = 16;              // one column tile
constexpr int kMixedSeqs = 8;

}  // namespace

// Where the longest sequence wants the kernel for many rows, batches of eight and
// more sequences may well hold single tokens too (prompts that join a running
// batch): those then have a launch of the kernel for few rows of their own, which
// costs 4 us when there are none.
Kv8AttnPlan kv8_attn_plan(const Kv8AttnArgs& a) {
  Kv8AttnPlan p{};
  const int cus = device_cus();
  const long long rows = static_cast<long long>(a.c.max_new) * a.group;
  p.few = p.many = a;
  p.few.least_rows = p.many.least_rows = 0;
  p.few.most_rows = p.many.most_rows = INT32_MAX;
  const int nt = rows_nt(a, cus);
  p.has_many = nt == 0;
  p.has_few = nt != 0 || a.c.seqs >= kMixedSeqs;
  if (p.has_few) p.few_bytes = ws_round(plan_launch(&p.few, nt ? nt : 1, nt ? rows : kFewRows, cus));
  if (p.has_many) p.many_bytes = ws_round(plan_launch(&p.many, 0, rows, cus));
  if (p.has_few && p.has_many) {
    p.few.most_rows = kFewRows;
    p.many.least_rows = kFewRows + 1;
  }
  return p;
}

void kv8_attn_launch(Kv8AttnPlan p, int* counters, char* partials, int dtype, hipStream_t stream) {
  if (p.has_many) {
    p.many.partials = reinterpret_cast<float*>(partials + p.few_bytes);
    kv8_prompt_launch(p.many, dtype, stream);
  }
  if (p.has_few) {
    p.few.counters = counters;
    p.few.partials = reinterpret_cast<float*>(partials);
    few_launch(p.few, dtype, stream);
  }
}

}  // namespace qlin
