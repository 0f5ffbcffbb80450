// The book of the 8-bit cache's pages (who holds which page) and the copies of
// pages that its changes call for, gfx950.
//
// refs[p] counts the table entries that hold page p (0: free).  Every choice is a
// function of the book alone: free pages go out from the lowest, wanted places are
// served in (row, entry) order, counts change by integer atomics, whose order does
// not matter.  So a captured step gives the same pages whenever it is replayed on
// the same book.
//
// A choice over the whole pool (the r-th free page) is a prefix sum over refs.  One
// workgroup of 1024 threads makes it, 16 pages to a thread and 16384 to a step, and
// stops at the last page that it needs: a pool that fills the card's memory has some
// ten thousand pages, so its counts are a few hundred KB, and what bounds these
// kernels is the latency of dependent loads and barriers, which a second launch
// would only add to.  What touches a whole table is spread over the device.

#include <algorithm>

#include "common.hpp"
#include "device.hpp"
#include "kv8.hpp"

namespace qlin {

namespace {

constexpr int kThreads = 1024;
constexpr int kEach = 16;                     // pages of a thread in a step
constexpr int kStep = kThreads * kEach;

__device__ __forceinline__ bool is_page(int page, int pages) { return static_cast<unsigned>(page) < static_cast<unsigned>(pages); }

// Sum of v over the threads before this one, and over all in *total.
// part: 17 ints in LDS, free again when the call returns.
__device__ __forceinline__ int sum_before(int v, int* part, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int up = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int other = __shfl_up(up, off, 64);
    if (lane >= off) up += other;
  }
  if (lane == 63) part[wave] = up;
  __syncthreads();
  int before = up - v, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    const int p = part[w];
    before += w < wave ? p : 0;
    all += p;
  }
  *total = all;
  __syncthreads();
  return before;
}

// Which of the 16 pages from `first` on (a multiple of 16; it may lie past the pool's end) are free, as bits.
__device__ __forceinline__ uint32_t free_bits(const int32_t* refs, int pages, int first) {
  uint32_t bits = 0;
  if (first + kEach <= pages) {
    int4 r[kEach / 4];
#pragma unroll
    for (int i = 0; i < kEach / 4; ++i) r[i] = reinterpret_cast<const int4*>(refs + first)[i];
#pragma unroll
    for (int i = 0; i < kEach / 4; ++i) {
      bits |= static_cast<uint32_t>(r[i].x <= 0) << (4 * i) | static_cast<uint32_t>(r[i].y <= 0) << (4 * i + 1) |
              static_cast<uint32_t>(r[i].z <= 0) << (4 * i + 2) | static_cast<uint32_t>(r[i].w <= 0) << (4 * i + 3);
    }
  } else {
    for (int i = 0; i < pages - first; ++i) bits |= static_cast<uint32_t>(refs[first + i] <= 0) << i;
  }
  return bits;
}
__device__ __forceinline__ int pages_of(int pages, int first) { return min(max(pages - first, 0), kEach); }

// give(rank, page) for the `wanted` lowest free pages in turn, if there are as many;
// returns how many are missing (the same in every thread).  Nothing is given then.
template <class Give>
__device__ __forceinline__ int take_free(const int32_t* refs, int pages, int wanted, int* part, Give give) {
  int found = 0, steps = 0;
  uint32_t bits = 0;
  int before = 0;
  for (int at = 0; at < pages && found < wanted; at += kStep, ++steps) {
    bits = free_bits(refs, pages, at + static_cast<int>(threadIdx.x) * kEach);
    int total;
    before = found + sum_before(__popc(bits), part, &total);
    found += total;
  }
  if (found < wanted) return wanted - found;
  // every count has been read: what follows may change them
  for (int s = 0, have = 0; s < steps; ++s) {
    const int first = s * kStep + static_cast<int>(threadIdx.x) * kEach;
    if (steps > 1) {
      bits = free_bits(refs, pages, first);
      int total;
      before = have + sum_before(__popc(bits), part, &total);
      have += total;
    }
    for (int rank = before; bits != 0 && rank < wanted; ++rank) {
      const int i = __ffs(bits) - 1;
      bits &= bits - 1;
      give(rank, first + i);
    }
  }
  return 0;
}

// Entries that a row's tokens need, -1 if the table has no room for them.
__device__ __forceinline__ int entries_of(int len, const Kv8Book& k) {
  if (len <= 0) return 0;
  const int n = ((len - 1) >> k.log_page) + 1;
  return n <= k.stride ? n : -1;
}

// Pages for the entries behind each row's last held one, up to the row's tokens.
// A row's need is known at once where its last entry, or the one before, is held (a
// growing sequence); rows with more to find (prompts) are searched back from the end
// by a wave each, 512 entries at a time.
__global__ __launch_bounds__(kThreads) void kv8_grow_kernel(const Kv8Book k, const int32_t* __restrict__ lens,
                                                            int2* __restrict__ moves) {
  extern __shared__ int start[];               // [rows + 1]: wanted pages before each row; before that the needs
  __shared__ int part[17];
  __shared__ int bad, searched;
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid == 0) bad = searched = 0;
  __syncthreads();
  for (int b = tid; b < k.rows; b += kThreads) {
    const int want = entries_of(lens[b], k);
    const int32_t* row = k.table + static_cast<size_t>(b) * k.stride;
    int need = 0;
    if (want < 0) bad = 1;
    if (want > 0) {
      const int last = row[want - 1], before = row[max(want - 2, 0)];
      need = is_page(last, k.pages) ? 0 : want == 1 || is_page(before, k.pages) ? 1 : -1;
    }
    if (need < 0) searched = 1;
    start[b] = need;
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) moves[0] = make_int2(0, -1);
    return;
  }
  if (searched) {
    for (int b = tid >> 6; b < k.rows; b += kThreads / 64) {
      if (start[b] >= 0) continue;             // (the wave's own rows: nobody else writes them)
      const int want = entries_of(lens[b], k);
      const int32_t* row = k.table + static_cast<size_t>(b) * k.stride;
      constexpr int AHEAD = 8;
      int last = -1;
      for (int end = want; end > 0 && last < 0; end -= 64 * AHEAD) {
        int page[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) page[i] = row[max(end - 1 - 64 * i - lane, 0)];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const uint64_t held = __ballot(end - 1 - 64 * i - lane >= 0 && is_page(page[i], k.pages));
          if (held != 0 && last < 0) last = end - 1 - 64 * i - (__ffsll(static_cast<unsigned long long>(held)) - 1);
        }
      }
      if (lane == 0) start[b] = want - 1 - last;
    }
    __syncthreads();
  }
  // needs to places, in runs of consecutive rows to a thread
  const int per = (k.rows + kThreads - 1) / kThreads, b0 = min(tid * per, k.rows), b1 = min(b0 + per, k.rows);
  int mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += start[b];
  int at = sum_before(mine, part, &total);
  for (int b = b0; b < b1; ++b) {
    const int need = start[b];
    start[b] = at;
    at += need;
  }
  if (tid == 0) start[k.rows] = total;
  __syncthreads();
  const int missing = total == 0 ? 0 : take_free(k.refs, k.pages, total, part, [&](int rank, int page) {
    int lo = 0, hi = k.rows;                   // the row whose places hold the rank: start[lo] <= rank < start[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= rank) lo = mid;
      else hi = mid;
    }
    const int want = entries_of(lens[lo], k);
    k.table[static_cast<size_t>(lo) * k.stride + want - (start[lo + 1] - rank)] = page;
    k.refs[page] = 1;
  });
  if (tid == 0) moves[0] = make_int2(missing ? 0 : total, missing);
}

// The plan of a fork: what is wrong with it, and a fresh page for each child whose
// prefix ends inside a page.  n <= 16384 children.
__global__ __launch_bounds__(kThreads) void kv8_fork_plan_kernel(const Kv8Book k, const int32_t* __restrict__ parents,
                                                                 const int32_t* __restrict__ children,
                                                                 const int32_t* __restrict__ lens, int n,
                                                                 int2* __restrict__ moves) {
  extern __shared__ int held[];                // fresh pages by rank [n], then rows that are children, and parents, as bits
  __shared__ int part[17];
  __shared__ int bad;
  const int tid = threadIdx.x, words = (k.rows + 31) / 32;
  int* is_child = held + n;
  int* is_parent = is_child + words;
  for (int i = tid; i < 2 * words; i += kThreads) is_child[i] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int p = parents[i], c = children[i];
    if (p < 0 || c < 0) continue;              // padding
    if (p >= k.rows || c >= k.rows || lens[i] < 0 || entries_of(lens[i], k) < 0) {
      bad = 1;
      continue;
    }
    atomicOr(&is_parent[p >> 5], 1 << (p & 31));
    if ((atomicOr(&is_child[c >> 5], 1 << (c & 31)) >> (c & 31)) & 1) bad = 1;
  }
  __syncthreads();
  for (int i = tid; i < words; i += kThreads)
    if (is_child[i] & is_parent[i]) bad = 1;
  __syncthreads();
  if (bad) {
    for (int i = tid; i <= n; i += kThreads) moves[i] = i ? make_int2(-1, -1) : make_int2(0, -1);
    return;
  }
  // children of consecutive numbers to a thread, as in the sums before them
  const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  const auto source = [&](int i) {             // the parent's page that is to be copied, or -1
    const int p = parents[i], len = lens[i];
    if (p < 0 || children[i] < 0 || (len & ((1 << k.log_page) - 1)) == 0) return -1;
    const int page = k.table[static_cast<size_t>(p) * k.stride + (len >> k.log_page)];
    return is_page(page, k.pages) ? page : -1;
  };
  int mine = 0, total;
  for (int i = i0; i < i1; ++i) mine += source(i) >= 0;
  int rank = sum_before(mine, part, &total);
  const int missing = total == 0 ? 0 : take_free(k.refs, k.pages, total, part, [&](int r, int page) {
    held[r] = page;
    k.refs[page] = 1;
  });
  __syncthreads();
  for (int i = i0; i < i1; ++i) {
    const int src = missing ? -1 : source(i);
    moves[1 + i] = src >= 0 ? make_int2(src, held[rank++]) : make_int2(-1, -1);
  }
  if (tid == 0) moves[0] = make_int2(missing ? 0 : n, missing);
}

// The children's rows: shared pages, the fresh one, nothing behind; what they held
// before goes back.  Grid: entries x children.
__global__ __launch_bounds__(256) void kv8_fork_rows_kernel(const Kv8Book k, const int32_t* __restrict__ parents,
                                                            const int32_t* __restrict__ children,
                                                            const int32_t* __restrict__ lens,
                                                            const int2* __restrict__ moves) {
  const int i = blockIdx.y, p = parents[i], c = children[i];
  const int2 head = moves[0], move = moves[1 + i];
  if (head.y != 0 || p < 0 || c < 0) return;
  const int len = lens[i], full = len >> k.log_page;
  const int32_t* from = k.table + static_cast<size_t>(p) * k.stride;
  int32_t* to = k.table + static_cast<size_t>(c) * k.stride;
  for (int e = blockIdx.x * 256 + threadIdx.x; e < k.stride; e += gridDim.x * 256) {
    const int was = to[e], theirs = e < full ? from[e] : -1;
    const int shared = is_page(theirs, k.pages) ? theirs : -1, now = e == full ? move.y : shared;
    if (now == was) continue;                  // (never the fresh page: that one was free)
    if (shared >= 0) atomicAdd(k.refs + shared, 1);
    if (is_page(was, k.pages)) atomicSub(k.refs + was, 1);
    to[e] = now;
  }
}

// Gives back the entries whose tokens all lie in begin .. end-1.  An entry is taken
// by an exchange, so that rows named twice give their pages back once.
__global__ __launch_bounds__(256) void kv8_free_kernel(const Kv8Book k, const int32_t* __restrict__ rows,
                                                       const int32_t* __restrict__ begin, const int32_t* __restrict__ end) {
  const int i = blockIdx.y, b = rows[i], P = 1 << k.log_page;
  if (!is_page(b, k.rows)) return;             // padding
  int e0 = 0, e1 = k.stride;
  if (begin) {
    const int t = max(begin[i], 0);
    e0 = (t >> k.log_page) + ((t & (P - 1)) != 0);
  }
  if (end) e1 = min(max(end[i], 0) >> k.log_page, k.stride);
  int32_t* row = k.table + static_cast<size_t>(b) * k.stride;
  for (int e = e0 + blockIdx.x * 256 + threadIdx.x; e < e1; e += gridDim.x * 256) {
    if (row[e] == -1) continue;
    const int was = atomicExch(row + e, -1);
    if (is_page(was, k.pages)) atomicSub(k.refs + was, 1);
  }
}

// The moves of a compaction: with U pages in use, every free page below U gets one of
// the used pages from U on, the lowest the highest; at most `most` of them.
__global__ __launch_bounds__(kThreads) void kv8_compact_plan_kernel(const Kv8Book k, int most, int2* __restrict__ moves) {
  __shared__ int part[17];
  const int tid = threadIdx.x;
  int total;
  int unused = 0;
  for (int at = 0; at < k.pages; at += kStep) unused += __popc(free_bits(k.refs, k.pages, at + tid * kEach));
  sum_before(unused, part, &total);
  const int used = k.pages - total;
  int low = 0;                                 // free pages below `used`: as many as there are used ones from there on
  for (int at = 0; at < used; at += kStep) {
    const int first = at + tid * kEach;
    uint32_t bits = free_bits(k.refs, k.pages, first) & ((1u << pages_of(used, first)) - 1u);
    int rank = low + sum_before(__popc(bits), part, &total);
    low += total;
    for (; bits != 0 && rank < most; ++rank) {
      const int i = __ffs(bits) - 1;
      bits &= bits - 1;
      moves[1 + rank].y = first + i;
    }
  }
  for (int at = used, have = 0; at < k.pages && have < low; at += kStep) {
    // (from a page that need not be a multiple of four: word by word)
    const int first = at + tid * kEach, n = pages_of(k.pages, first);
    uint32_t bits = 0;
    for (int i = 0; i < n; ++i) bits |= static_cast<uint32_t>(k.refs[first + i] > 0) << i;
    int rank = low - 1 - (have + sum_before(__popc(bits), part, &total));
    have += total;
    for (; bits != 0; --rank) {
      const int i = __ffs(bits) - 1;
      bits &= bits - 1;
      if (rank < most) moves[1 + rank].x = first + i;
    }
  }
  const int count = min(low, most);
  for (int i = count + tid; i < most; i += kThreads) moves[1 + i] = make_int2(-1, -1);
  if (tid == 0) moves[0] = make_int2(count, 0);
  __syncthreads();                             // every count has been read, every move is there
  for (int i = tid; i < count; i += kThreads) {
    const int2 m = moves[1 + i];
    k.refs[m.y] = k.refs[m.x];
    k.refs[m.x] = 0;
  }
}

// The table after the moves: an entry from the lowest moved page on is looked up
// among them (their sources descend).
__global__ __launch_bounds__(256) void kv8_compact_rows_kernel(const Kv8Book k, const int2* __restrict__ moves) {
  const int count = moves[0].x;
  if (count == 0) return;
  const int lowest = moves[count].x;
  const long long entries = static_cast<long long>(k.rows) * k.stride;
  for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < entries; e += static_cast<long long>(gridDim.x) * 256) {
    const int page = k.table[e];
    if (page < lowest || !is_page(page, k.pages)) continue;
    int lo = 1, hi = count;                    // the last move whose source is at least the page
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (moves[mid].x >= page) lo = mid;
      else hi = mid - 1;
    }
    const int2 m = moves[lo];
    if (m.x == page) k.table[e] = m.y;
  }
}

// Pages listed in moves, of every layer: 16 bytes a lane, four loads in flight.
// Grid: pieces of 1024 chunks of a page's K and V x moves (taken up in turn) x layers.
constexpr int kCopyEach = 4;
__global__ __launch_bounds__(256) void kv8_copy_kernel(const Kv8CopyArgs a) {
  const Kv8CopyLayer l = a.layers[blockIdx.z];
  const int count = min(a.moves[0].x, a.most);
  const int half = a.chunks, first = blockIdx.x * (256 * kCopyEach) + threadIdx.x;
  for (int m = blockIdx.y; m < count; m += gridDim.y) {
    const int2 move = a.moves[1 + m];
    if (!is_page(move.x, a.from_pages) || !is_page(move.y, a.to_pages)) continue;
    const uint4* k = reinterpret_cast<const uint4*>(l.from_k) + static_cast<size_t>(move.x) * half;
    const uint4* v = reinterpret_cast<const uint4*>(l.from_v) + static_cast<size_t>(move.x) * half;
    uint4* k_to = reinterpret_cast<uint4*>(l.to_k) + static_cast<size_t>(move.y) * half;
    uint4* v_to = reinterpret_cast<uint4*>(l.to_v) + static_cast<size_t>(move.y) * half;
    uint4 w[kCopyEach];                        // (chunks past the end: the last one, not stored)
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i) {
      const int c = min(first + 256 * i, 2 * half - 1);
      w[i] = *(c < half ? k + c : v + (c - half));
    }
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i) {
      const int c = first + 256 * i;
      if (c < half) k_to[c] = w[i];
      else if (c < 2 * half) v_to[c - half] = w[i];
    }
    if (blockIdx.x == 0)
      for (int h = threadIdx.x; h < a.heads; h += 256)
        l.to_scales[static_cast<size_t>(move.y) * a.heads + h] = l.from_scales[static_cast<size_t>(move.x) * a.heads + h];
  }
}

unsigned chunks_of(int n, int by, int most) { return static_cast<unsigned>(std::min((n + by - 1) / by, most)); }

}  // namespace

void kv8_grow_launch(const Kv8Book& k, const int32_t* lens, int32_t* moves, hipStream_t stream) {
  hipLaunchKernelGGL(kv8_grow_kernel, dim3(1), dim3(kThreads), sizeof(int) * (k.rows + 1), stream, k, lens,
                     reinterpret_cast<int2*>(moves));
}

void kv8_fork_launch(const Kv8Book& k, const int32_t* parents, const int32_t* children, const int32_t* lens, int n,
                     int32_t* moves, hipStream_t stream) {
  int2* m = reinterpret_cast<int2*>(moves);
  const size_t lds = sizeof(int) * (n + 2 * ((k.rows + 31) / 32));
  hipLaunchKernelGGL(kv8_fork_plan_kernel, dim3(1), dim3(kThreads), lds, stream, k, parents, children, lens, n, m);
  hipLaunchKernelGGL(kv8_fork_rows_kernel, dim3(chunks_of(k.stride, 256, 64), n), dim3(256), 0, stream, k, parents, children,
                     lens, static_cast<const int2*>(m));
}

void kv8_free_launch(const Kv8Book& k, const int32_t* rows, const int32_t* begin, const int32_t* end, int n, hipStream_t stream) {
  hipLaunchKernelGGL(kv8_free_kernel, dim3(chunks_of(k.stride, 1024, 64), n), dim3(256), 0, stream, k, rows, begin, end);
}

void kv8_compact_launch(const Kv8Book& k, int most, int32_t* moves, hipStream_t stream) {
  int2* m = reinterpret_cast<int2*>(moves);
  hipLaunchKernelGGL(kv8_compact_plan_kernel, dim3(1), dim3(kThreads), 0, stream, k, most, m);
  const long long entries = static_cast<long long>(k.rows) * k.stride;
  hipLaunchKernelGGL(kv8_compact_rows_kernel, dim3(static_cast<unsigned>(std::min<long long>((entries + 255) / 256, 4096))),
                     dim3(256), 0, stream, k, static_cast<const int2*>(m));
}

void kv8_copy_launch(Kv8CopyArgs a, int layers, hipStream_t stream) {
  // Moves beyond those of the grid are taken up in turn: enough workgroups to fill
  // the device, not one for every move that might be listed.
  constexpr int kGroups = 8192;
  const unsigned pieces = (2u * a.chunks + 256 * kCopyEach - 1) / (256 * kCopyEach);
  const int at_once = std::max(1, static_cast<int>(kGroups / (static_cast<long long>(pieces) * layers)));
  hipLaunchKernelGGL(kv8_copy_kernel, dim3(pieces, std::min(std::min(a.most, at_once), 65535), layers), dim3(256), 0, stream, a);
}

}  // namespace qlin
