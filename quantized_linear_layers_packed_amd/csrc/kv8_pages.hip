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
// stops at the last page that it needs.  A pool that fills the card's memory has from
// some ten thousand pages on (of 128 tokens in many layers) to a few hundred thousand:
// 40 KB to a few MB of counts, and what bounds these kernels is the latency of
// dependent loads and barriers, which a second launch would only add to.  What touches
// a whole table is spread over the device.
//
// Measured, calls and all: a token for each of 256 sequences (131072 pages; two
// releases and the grow) 15.6 us, of which the host's three calls are 14; 32768 pages
// for 16 prompts 29.5 us (the grow 24: one workgroup's 65536 stores, and the search for
// the rows' ends), 16168 for 512 prompts of 32 pages 59; 128 forks of two prompts with a
// page of 131 KB each to copy in 4 layers 39 us, the copies 17; a pool of 6082 pages half
// in use, 1520 of 262 KB moved in 2 layers, 168 us, 4.74 TB/s (a large copy: 4.73).
// The grow of a token for each of 256 sequences takes 7 us where free pages lie among the
// first 16384 of the pool and 24 behind 98204 pages in use, whose counts are read twice.

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
// An entry that grow looks for pages behind: held, or its tokens came with a fork and their
// page was gone by then.  Pages dealt out for such tokens would show what others left there.
// (A selection: as two comparisons or-ed the searches spill scalar registers, and the grow of
// 32768 pages takes 25.2 instead of 24.2 us.)
__device__ __forceinline__ bool is_past(int page, int pages) { return is_page(page == kKv8Gone ? 0 : page, pages); }

// Sum of v over the threads before this one, and over all in *total.
// part: 16 ints in LDS, free again when the call returns.
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

// The pages of a step are dealt out 1024 to a wave, in 16 rows of 64: lane l's i-th is
// first + 64 i + l, so that loads, and what is written for pages in turn, are
// consecutive over the lanes.  A row is a mask over the lanes, in scalar registers.
struct Rows16 {
  uint64_t row[kEach];
  __device__ __forceinline__ int count() const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) n += __popcll(row[i]);
    return n;
  }
};
// Of the step's pages before `end` (which is above 0): which are free, or (USED) are not.
template <bool USED = false>
__device__ __forceinline__ Rows16 free_pages(const int32_t* refs, int at, int end) {
  const int wave = __builtin_amdgcn_readfirstlane(at + (threadIdx.x & ~63) * kEach), first = wave + (threadIdx.x & 63);
  Rows16 f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) f.row[i] = 0;
  if (wave >= end) return f;
  int r[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) r[i] = refs[min(first + 64 * i, end - 1)];
#pragma unroll
  for (int i = 0; i < kEach; ++i) f.row[i] = __ballot((r[i] <= 0) != USED && first + 64 * i < end);
  return f;
}
// Sum over the waves before this one of a number that is the same in all of a wave's
// lanes, and over all waves in *total.
__device__ __forceinline__ int waves_before(int n, int* part, int* total) {
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) part[wave] = n;
  __syncthreads();
  int before = 0, all = 0;
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
// give(rank, page) for the pages of a step, `rank` being that of the wave's first,
// until `limit`.
template <class Give>
__device__ __forceinline__ void each_page(const Rows16& f, int at, int rank, int limit, Give give) {
  const int lane = threadIdx.x & 63, first = at + (threadIdx.x & ~63) * kEach + lane;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint64_t all = f.row[i];
    if (all == 0) continue;
    const int mine = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                               __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), static_cast<uint32_t>(rank)));
    if (__builtin_amdgcn_inverse_ballot_w64(all) && mine < limit) give(mine, first + 64 * i);
    rank += __popcll(all);
  }
}

// give(rank, page) for the `wanted` lowest free pages in turn, if there are as many;
// returns how many are missing (the same in every thread).  Nothing is given then.
// ahead: free_pages of the first step, asked for before it was known how many are
// wanted.
template <class Give>
__device__ __forceinline__ int take_free(const int32_t* refs, int pages, int wanted, const Rows16& ahead, int* part, Give give) {
  int found = 0, steps = 0, before = 0;
  for (int at = 0; at < pages && found < wanted; at += kStep, ++steps) {
    int total;
    before = found + waves_before(at == 0 ? ahead.count() : free_pages(refs, at, pages).count(), part, &total);
    found += total;
  }
  if (found < wanted) return wanted - found;
  // every count has been read: what follows may change them
  if (steps == 1) {
    if (before < wanted) each_page(ahead, 0, before, wanted, give);
    return 0;
  }
  for (int s = 0, have = 0; s < steps; ++s) {
    const Rows16 f = free_pages(refs, s * kStep, pages);
    int total;
    before = have + waves_before(f.count(), part, &total);
    have += total;
    if (before < wanted) each_page(f, s * kStep, before, wanted, give);
  }
  return 0;
}

// Entries that a row's tokens need, -1 if the table has no room for them.
__device__ __forceinline__ int entries_of(int len, const Kv8Book& k) {
  if (len <= 0) return 0;
  const int n = ((len - 1) >> k.log_page) + 1;
  return n <= k.stride ? n : -1;
}

// Needs of the rows that have more to find: searched back from the end for the last
// held (or gone) entry, ROWS rows of a wave and 1024 / ROWS entries of each at a time.  With one, few
// long rows are found soonest (16 of 2500 entries: 4 reads in turn), with four, many short
// ones (512 prompts of 32 pages, releases and all, 103 -> 59 us; 16 of 2500 30.6 with either).
constexpr int kAFew = 2 * kThreads / 64;
template <int ROWS>
__device__ __forceinline__ void search_rows(const Kv8Book& k, const int32_t* lens, int* need) {
  constexpr int AHEAD = 16 / ROWS;
  const int lane = threadIdx.x & 63;
  for (int b = (threadIdx.x >> 6) * ROWS; b < k.rows; b += kThreads / 64 * ROWS) {
    int want[ROWS], end[ROWS], last[ROWS];
    bool more = false;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {           // (the wave's own rows: nobody else writes them)
      want[j] = end[j] = b + j < k.rows && need[b + j] < 0 ? entries_of(lens[b + j], k) : 0;
      last[j] = -1;
      more |= end[j] > 0;
    }
    while (more) {
      int page[ROWS][AHEAD];
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          page[j][i] = k.table[static_cast<size_t>(min(b + j, k.rows - 1)) * k.stride + max(end[j] - 1 - 64 * i - lane, 0)];
      more = false;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const uint64_t held = __ballot(end[j] - 1 - 64 * i - lane >= 0 && is_past(page[j][i], k.pages));
          if (held != 0 && last[j] < 0) last[j] = end[j] - 1 - 64 * i - (__ffsll(static_cast<unsigned long long>(held)) - 1);
        }
        end[j] = last[j] >= 0 ? 0 : end[j] - 64 * AHEAD;
        more |= end[j] > 0;
      }
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
      if (lane == 0 && want[j] > 0) need[b + j] = want[j] - 1 - last[j];
  }
}

// Pages for the entries behind each row's last held (or gone) one, up to the row's tokens.
// A row's need is known at once where one of its last four entries is held (a growing
// sequence) or it has no more; rows with more to find (prompts) are searched.
constexpr int kLook = 4;
__global__ __launch_bounds__(kThreads) void kv8_grow_kernel(const Kv8Book k, const int32_t* __restrict__ lens,
                                                            int2* __restrict__ moves) {
  extern __shared__ int start[];               // [rows + 1]: wanted pages before each row; before that the needs
  __shared__ int part[kThreads / 64];
  __shared__ int bad, searched;
  const int tid = threadIdx.x;
  if (tid == 0) bad = searched = 0;
  __syncthreads();
  const Rows16 ahead = free_pages(k.refs, 0, k.pages);
  for (int b = tid; b < k.rows; b += kThreads) {
    const int want = entries_of(lens[b], k);
    const int32_t* row = k.table + static_cast<size_t>(b) * k.stride;
    int need = 0;
    if (want < 0) bad = 1;
    if (want > 0) {
      int page[kLook];
#pragma unroll
      for (int i = 0; i < kLook; ++i) page[i] = row[max(want - 1 - i, 0)];
      need = want <= kLook ? want : -1;        // unless one of them is held
#pragma unroll
      for (int i = kLook - 1; i >= 0; --i) need = want > i && is_past(page[i], k.pages) ? i : need;
    }
    if (need < 0) atomicAdd(&searched, 1);
    start[b] = need;
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) moves[0] = make_int2(0, -1);
    return;
  }
  if (searched > kAFew) search_rows<4>(k, lens, start);
  else if (searched > 0) search_rows<1>(k, lens, start);
  if (searched > 0) __syncthreads();
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
  // the row whose places hold a rank, start[row] <= rank < start[row + 1], and where its
  // entries end: a thread's ranks ascend, and often stay in the row
  int row = -1, row_end = 0;
  long long place = 0;                         // of rank 0 as the row would have it
  const int missing = total == 0 ? 0 : take_free(k.refs, k.pages, total, ahead, part, [&](int rank, int page) {
    if (rank >= row_end) {
      int lo = row + 1, hi = k.rows;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= rank) lo = mid;
        else hi = mid;
      }
      row = lo;
      row_end = start[row + 1];
      place = static_cast<long long>(row) * k.stride + entries_of(lens[row], k) - row_end;
    }
    k.table[place + rank] = page;
    k.refs[page] = 1;
  });
  if (tid == 0) moves[0] = make_int2(missing ? 0 : total, missing);
}

// Adds to the counts of pages, summed while the page stays the same: neighbours in a
// list often share theirs (forks of one prefix: 64 children of 2 parents each way took
// 8.6 us with an addition for every child).
struct Counts {
  int32_t* refs;
  int page = -1, by = 0;
  __device__ __forceinline__ void add(int p, int n) {
    if (p != page) {
      flush();
      page = p;
      by = 0;
    }
    by += n;
  }
  __device__ __forceinline__ void flush() {
    if (page >= 0 && by != 0) atomicAdd(refs + page, by);
  }
};
constexpr int kListEach = 8;                  // of a list, to a workgroup

// Entries from e0 on, `step` apart, of the rows of children i0 .. i0 + 7: shared pages, the
// fresh one, nothing behind; what they held before goes back.  The prefix's last entry says
// so if the parent's page is gone: else the row would look like one with tokens to come.
__device__ __forceinline__ void fork_rows(const Kv8Book& k, const int32_t* parents, const int32_t* children, const int32_t* lens,
                                          int n, const int2* moves, int i0, unsigned e0, unsigned step) {
  const int short_by = moves[0].y;
  int p[kListEach], c[kListEach], len[kListEach], fresh[kListEach];
#pragma unroll
  for (int j = 0; j < kListEach; ++j) {
    const int i = min(i0 + j, n - 1);
    p[j] = parents[i];
    c[j] = i0 + j < n ? children[i] : -1;
    len[j] = lens[i];
    fresh[j] = moves[1 + i].y;
  }
  if (short_by != 0) return;                   // (lists that do not fit the table among it)
  for (unsigned at = e0; at < static_cast<unsigned>(k.stride); at += step) {   // (past the end it may leave int's range)
    const int e = static_cast<int>(at);
    int was[kListEach], theirs[kListEach];
#pragma unroll
    for (int j = 0; j < kListEach; ++j) {
      was[j] = theirs[j] = -1;
      if (p[j] < 0 || c[j] < 0) continue;      // padding
      was[j] = k.table[static_cast<size_t>(c[j]) * k.stride + e];
      if (e < len[j] >> k.log_page) theirs[j] = k.table[static_cast<size_t>(p[j]) * k.stride + e];
    }
    Counts more{k.refs}, fewer{k.refs};
#pragma unroll
    for (int j = 0; j < kListEach; ++j) {
      if (p[j] < 0 || c[j] < 0) continue;
      const int shared = is_page(theirs[j], k.pages) ? theirs[j] : -1;
      int now = e == len[j] >> k.log_page ? fresh[j] : shared;
      if (now < 0 && e == (len[j] - 1) >> k.log_page) now = kKv8Gone;
      if (now == was[j]) continue;             // (never the fresh page: that one was free)
      if (shared >= 0) more.add(shared, 1);
      if (is_page(was[j], k.pages)) fewer.add(was[j], -1);
      k.table[static_cast<size_t>(c[j]) * k.stride + e] = now;
    }
    more.flush();
    fewer.flush();
  }
}

// The plan of a fork: what is wrong with it, and a fresh page for each child whose
// prefix ends inside a page.  n <= 16384 children.  ROWS: the children's rows, too.
template <bool ROWS>
__global__ __launch_bounds__(kThreads) void kv8_fork_plan_kernel(const Kv8Book k, const int32_t* __restrict__ parents,
                                                                 const int32_t* __restrict__ children,
                                                                 const int32_t* __restrict__ lens, int n,
                                                                 int2* __restrict__ moves) {
  extern __shared__ int held[];                // fresh pages by rank [n], then rows that are children, and parents, as bits
  __shared__ int part[kThreads / 64];
  __shared__ int bad;
  const int tid = threadIdx.x, words = (k.rows + 31) / 32;
  int* is_child = held + n;
  int* is_parent = is_child + words;
  const Rows16 ahead = free_pages(k.refs, 0, k.pages);
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
  const int missing = total == 0 ? 0 : take_free(k.refs, k.pages, total, ahead, part, [&](int r, int page) {
    held[r] = page;
    k.refs[page] = 1;
  });
  __syncthreads();
  for (int i = i0; i < i1; ++i) {
    const int src = missing ? -1 : source(i);
    moves[1 + i] = src >= 0 ? make_int2(src, held[rank++]) : make_int2(-1, -1);
  }
  if (tid == 0) moves[0] = make_int2(missing ? 0 : n, missing);
  if constexpr (ROWS) {
    __syncthreads();                           // every move is there, no fresh page is counted any more
    const int groups = (n + kListEach - 1) / kListEach;
    for (int at = tid; at < groups * k.stride; at += kThreads)
      fork_rows(k, parents, children, lens, n, moves, at / k.stride * kListEach, at % k.stride, k.stride);
  }
}

// Grid: entries x children.
__global__ __launch_bounds__(256) void kv8_fork_rows_kernel(const Kv8Book k, const int32_t* __restrict__ parents,
                                                            const int32_t* __restrict__ children,
                                                            const int32_t* __restrict__ lens, int n,
                                                            const int2* __restrict__ moves) {
  fork_rows(k, parents, children, lens, n, moves, blockIdx.y * kListEach, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// Gives back the entries whose tokens all lie in begin .. end-1.  An entry is taken
// by an exchange, so that rows named twice give their pages back once.
__global__ __launch_bounds__(256) void kv8_free_kernel(const Kv8Book k, const int32_t* __restrict__ rows,
                                                       const int32_t* __restrict__ begin, const int32_t* __restrict__ end, int n) {
  const int i0 = blockIdx.y * kListEach, P = 1 << k.log_page;
  int b[kListEach], e0[kListEach], e1[kListEach];
#pragma unroll
  for (int j = 0; j < kListEach; ++j) {
    const int i = min(i0 + j, n - 1), t = begin ? max(begin[i], 0) : 0;
    b[j] = rows[i];
    e0[j] = (t >> k.log_page) + ((t & (P - 1)) != 0);
    e1[j] = end ? min(max(end[i], 0) >> k.log_page, k.stride) : k.stride;
    if (i0 + j >= n || !is_page(b[j], k.rows)) e1[j] = 0;      // past the list, or padding
  }
  int first = e0[0], last = e1[0];
#pragma unroll
  for (int j = 1; j < kListEach; ++j) {
    first = min(first, e0[j]);
    last = max(last, e1[j]);
  }
  for (unsigned at = first + blockIdx.x * 256 + threadIdx.x; at < static_cast<unsigned>(last); at += gridDim.x * 256) {
    const int e = static_cast<int>(at);        // (past the end `at` may leave int's range)
    int was[kListEach];
#pragma unroll
    for (int j = 0; j < kListEach; ++j)
      was[j] = e >= e0[j] && e < e1[j] ? k.table[static_cast<size_t>(b[j]) * k.stride + e] : -1;
#pragma unroll
    for (int j = 0; j < kListEach; ++j)
      if (was[j] != -1) was[j] = atomicExch(k.table + static_cast<size_t>(b[j]) * k.stride + e, -1);
    Counts fewer{k.refs};
#pragma unroll
    for (int j = 0; j < kListEach; ++j)
      if (is_page(was[j], k.pages)) fewer.add(was[j], -1);
    fewer.flush();
  }
}

// The table after the moves: entries `step` apart are looked up among them (their
// sources descend) where they are from the lowest moved page on, in a copy in LDS of
// all of them or of every 2^s-th, and from there in the list itself.
constexpr int kSamples = 4096;
template <int NT>
__device__ __forceinline__ void compact_rows(const Kv8Book& k, const int2* moves, int* sample, long long e0, long long step) {
  const int count = moves[0].x;
  if (count == 0) return;
  int shift = 0;
  while ((count - 1) >> shift >= kSamples) ++shift;
  const int samples = ((count - 1) >> shift) + 1;
  constexpr int AHEAD = 4;
  for (int i = threadIdx.x; i < samples; i += AHEAD * NT) {
    int x[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) x[j] = moves[1 + (min(i + j * NT, samples - 1) << shift)].x;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) sample[min(i + j * NT, samples - 1)] = x[j];
  }
  const int lowest = moves[count].x;
  __syncthreads();
  const long long entries = static_cast<long long>(k.rows) * k.stride;
  for (long long e = e0; e < entries; e += step) {
    const int page = k.table[e];
    if (page < lowest || !is_page(page, k.pages)) continue;
    int lo = 0, hi = samples - 1;              // the last of them whose source is at least the page
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sample[mid] >= page) lo = mid;
      else hi = mid - 1;
    }
    lo <<= shift;
    hi = min(lo + (1 << shift), count) - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (moves[1 + mid].x >= page) lo = mid;
      else hi = mid - 1;
    }
    const int2 m = moves[1 + lo];
    if (m.x == page) k.table[e] = m.y;
  }
}
// The moves of a compaction: with U pages in use, every free page below U gets one of
// the used pages from U on, the lowest the highest; at most `most` of them.
// ROWS: the table, too.
template <bool ROWS>
__global__ __launch_bounds__(kThreads) void kv8_compact_plan_kernel(const Kv8Book k, int most, int2* __restrict__ moves) {
  __shared__ int part[kThreads / 64];
  const int tid = threadIdx.x;
  int total, unused = 0;
  for (int at = 0; at < k.pages; at += kStep) unused += free_pages(k.refs, at, k.pages).count();
  waves_before(unused, part, &total);
  const int used = k.pages - total;
  int low = 0;                                 // free pages below `used`: as many as there are used ones from there on
  for (int at = 0; at < used; at += kStep) {
    const Rows16 f = free_pages(k.refs, at, used);
    const int rank = low + waves_before(f.count(), part, &total);
    low += total;
    each_page(f, at, rank, most, [&](int r, int page) { moves[1 + r].y = page; });
  }
  for (int at = used, have = 0; at < k.pages && have < low; at += kStep) {
    const Rows16 f = free_pages<true>(k.refs, at, k.pages);
    const int rank = have + waves_before(f.count(), part, &total);
    have += total;
    each_page(f, at, rank, low, [&](int r, int page) {
      if (low - 1 - r < most) moves[1 + low - 1 - r].x = page;
    });
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
  if constexpr (ROWS) {
    __shared__ int sample[kSamples];
    compact_rows<kThreads>(k, moves, sample, tid, kThreads);
  }
}

__global__ __launch_bounds__(256) void kv8_compact_rows_kernel(const Kv8Book k, const int2* __restrict__ moves) {
  __shared__ int sample[kSamples];
  compact_rows<256>(k, moves, sample, static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, static_cast<long long>(gridDim.x) * 256);
}

// Pages listed in moves, of every layer: 16 bytes a lane, four loads in flight.
// Grid: pieces of 1024 chunks of a page's K and V x moves (taken up in turn) x layers.
constexpr int kCopyEach = 4;
__global__ __launch_bounds__(256) void kv8_copy_kernel(const Kv8CopyArgs a) {
  const Kv8CopyLayer l = a.layers[blockIdx.z];
  const int half = a.chunks, first = blockIdx.x * (256 * kCopyEach) + threadIdx.x;
  int2 move = a.moves[1 + blockIdx.y];         // (there, also where it is not counted)
  const int count = min(a.moves[0].x, a.most);
  for (int m = blockIdx.y; m < count;) {
    if (is_page(move.x, a.from_pages) && is_page(move.y, a.to_pages)) {
      const u32x4_t* k = reinterpret_cast<const u32x4_t*>(l.from_k) + static_cast<size_t>(move.x) * half;
      const u32x4_t* v = reinterpret_cast<const u32x4_t*>(l.from_v) + static_cast<size_t>(move.x) * half;
      u32x4_t* k_to = reinterpret_cast<u32x4_t*>(l.to_k) + static_cast<size_t>(move.y) * half;
      u32x4_t* v_to = reinterpret_cast<u32x4_t*>(l.to_v) + static_cast<size_t>(move.y) * half;
      const float2* s = l.from_scales + static_cast<size_t>(move.x) * a.heads;
      float2* s_to = l.to_scales + static_cast<size_t>(move.y) * a.heads;
      u32x4_t w[kCopyEach];                    // (chunks past the end: the last one, not stored)
#pragma unroll
      for (int i = 0; i < kCopyEach; ++i) {
        const int c = min(first + 256 * i, 2 * half - 1);
        w[i] = *(c < half ? k + c : v + (c - half));
      }
      if (blockIdx.x == 0)
        for (int h = threadIdx.x; h < a.heads; h += 256) s_to[h] = s[h];
#pragma unroll
      for (int i = 0; i < kCopyEach; ++i) {
        const int c = first + 256 * i;
        if (c < 2 * half) *(c < half ? k_to + c : v_to + (c - half)) = w[i];
      }
    }
    m += gridDim.y;
    if (m < count) move = a.moves[1 + m];
  }
}

// Up to so many table entries (of groups of children, of a whole table) the workgroup
// that makes the plan writes them itself, which spares a launch.
constexpr int kAlone = 1024;

constexpr unsigned chunks_of(int64_t n, int by, int most) { return static_cast<unsigned>(std::min<int64_t>((n + by - 1) / by, most)); }
static_assert(chunks_of(INT32_MAX, 256, 64) == 64, "a table's longest row");

}  // namespace

void kv8_grow_launch(const Kv8Book& k, const int32_t* lens, int32_t* moves, hipStream_t stream) {
  hipLaunchKernelGGL(kv8_grow_kernel, dim3(1), dim3(kThreads), sizeof(int) * (k.rows + 1), stream, k, lens,
                     reinterpret_cast<int2*>(moves));
}

void kv8_fork_launch(const Kv8Book& k, const int32_t* parents, const int32_t* children, const int32_t* lens, int n,
                     int32_t* moves, hipStream_t stream) {
  int2* m = reinterpret_cast<int2*>(moves);
  const size_t lds = sizeof(int) * (n + 2 * ((k.rows + 31) / 32));
  if (static_cast<int64_t>((n + kListEach - 1) / kListEach) * k.stride <= kAlone) {
    hipLaunchKernelGGL(kv8_fork_plan_kernel<true>, dim3(1), dim3(kThreads), lds, stream, k, parents, children, lens, n, m);
    return;
  }
  hipLaunchKernelGGL(kv8_fork_plan_kernel<false>, dim3(1), dim3(kThreads), lds, stream, k, parents, children, lens, n, m);
  hipLaunchKernelGGL(kv8_fork_rows_kernel, dim3(chunks_of(k.stride, 256, 64), chunks_of(n, kListEach, n)), dim3(256), 0, stream,
                     k, parents, children, lens, n, static_cast<const int2*>(m));
}

void kv8_free_launch(const Kv8Book& k, const int32_t* rows, const int32_t* begin, const int32_t* end, int n, hipStream_t stream) {
  hipLaunchKernelGGL(kv8_free_kernel, dim3(chunks_of(k.stride, 256, 64), chunks_of(n, kListEach, n)), dim3(256), 0, stream, k, rows,
                     begin, end, n);
}

void kv8_compact_launch(const Kv8Book& k, int most, int32_t* moves, hipStream_t stream) {
  int2* m = reinterpret_cast<int2*>(moves);
  const long long entries = static_cast<long long>(k.rows) * k.stride;
  if (entries <= kAlone) {
    hipLaunchKernelGGL(kv8_compact_plan_kernel<true>, dim3(1), dim3(kThreads), 0, stream, k, most, m);
    return;
  }
  hipLaunchKernelGGL(kv8_compact_plan_kernel<false>, dim3(1), dim3(kThreads), 0, stream, k, most, m);
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
