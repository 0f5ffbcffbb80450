// The 8-bit paged key/value cache as the kernels see it, and the launchers of
// its operators.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/qlin.h"
#include "workspace.hpp"

namespace qlin {

// 2^-80.  Append stores pages whose values would need a smaller scale as zeros, and
// the attention takes a value scale below it (0 among them) as that: with zero codes
// any will do that keeps the weights of such a page, 2^(score - reference) times the
// scale, and their sum without the scale in fp32's range: it is below 2^(15 + 80 +
// 31) for any number of tokens, and beside values with scales of up to 2^20 weights
// of 2^-26 of the row's largest still count, also where splits are joined.
constexpr float kLeastScale = 8.2718061e-25f;

// Cache and batch with the sizes that the host has checked.
struct Kv8View {
  int8_t* k;
  int8_t* v;
  float* scales;
  const int32_t* offsets;
  const int32_t* kv_lens;
  const int32_t* table;
  int pages, heads, dim, log_page;
  int seqs, tokens, table_stride, max_new, max_kv;
};

// One sequence of the batch: its first token row, its new tokens, the position
// of the first of them (negative if there are more of them than the sequence
// is long) and its length.  Everything clamped, so that whatever the device
// arrays hold, rows stay in 0 .. tokens and positions below the table's end.
struct Kv8Seq {
  int row, count, start, len;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8View& c, int b) {
  Kv8Seq s;
  s.row = min(max(c.offsets[b], 0), c.tokens);
  s.count = min(max(c.offsets[b + 1], s.row), c.tokens) - s.row;
  const long long most = static_cast<long long>(c.table_stride) << c.log_page;
  s.len = static_cast<int>(min(static_cast<long long>(max(c.kv_lens[b], 0)), min(most, 0x7FFF0000LL)));
  s.start = s.len - s.count;
  return s;
}

struct Kv8AppendArgs {
  Kv8View c;
  const uint16_t* Q;
  const uint16_t* K;
  const uint16_t* V;
  long long q_stride, k_stride, v_stride;
  int q_heads, group;   // group: query heads that share a key/value head
  const float* cos;
  const float* sin;
  int max_pos, rot, pairs;
  uint16_t* Q_out;
};

// Division by a number known on the host: n / d for 0 <= n < 2^31, exactly
// (d <= 65535: mul = ceil(2^(32 + shift) / d) with 2^(shift + 1) >= d fits 32
// bits, and its error times n stays below 2^(32 + shift) / d).
struct FastDiv {
  uint32_t d = 1, mul = 0;
  int shift = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t by) : d(by) {
    while ((2u << shift) < by) ++shift;
    mul = static_cast<uint32_t>(((uint64_t{1} << (32 + shift)) + by - 1) / by);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
  }
};

struct Kv8AttnArgs {
  Kv8View c;
  const uint16_t* Q;
  long long q_stride;
  int q_heads, group;   // group: query heads that share a key/value head
  float scale;          // times log2(e)
  int window, sinks;    // window 0: none (sinks then 0)
  uint16_t* Y;
  int least_rows, most_rows;   // of a sequence that this launch computes
  // the split of long sequences (see kv8_attn.hip)
  int row_columns, row_tiles, splits, chunk, waves;
  bool sorted;          // few rows: sequences in the order of their lengths; many: a sequence's row tiles in that of theirs
  FastDiv by_group, by_heads, by_row_tiles, by_splits;
  int* counters;
  float* partials;
  // other scores and masks (the kernels' SCORED form)
  bool scored;
  float cap;                    // times log2(e); 0: none.  `scale` is then 2 log2(e) scale / cap
  const float* slopes;          // of the query heads; NULL: none
  const int32_t* prefix_lens;   // of the sequences
  const int32_t* starts;        // of the tokens
};

// The book of a cache's pages with the sizes that the host has checked.
struct Kv8Book {
  int32_t* refs;
  int32_t* table;
  int pages, log_page, rows, stride;
};

// A table entry of tokens that a forked row counts but whose page its parent had given back.
constexpr int kKv8Gone = -2;

// Copies of listed pages, layer by layer.
constexpr int kCopyLayers = 32;           // of a launch
struct Kv8CopyLayer {
  const int8_t* from_k;
  const int8_t* from_v;
  const float2* from_scales;
  int8_t* to_k;
  int8_t* to_v;
  float2* to_scales;
};
struct Kv8CopyArgs {
  const int2* moves;
  int most, chunks, heads, from_pages, to_pages;   // chunks: 16-byte ones of a page's K
  Kv8CopyLayer layers[kCopyLayers];
};

constexpr int kMostRows = 32767;          // of a book: a workgroup holds an integer for each
constexpr int kMostForks = 16384;

void kv8_grow_launch(const Kv8Book& k, const int32_t* lens, int32_t* moves, hipStream_t stream);
void kv8_fork_launch(const Kv8Book& k, const int32_t* parents, const int32_t* children, const int32_t* lens, int n,
                     int32_t* moves, hipStream_t stream);
void kv8_free_launch(const Kv8Book& k, const int32_t* rows, const int32_t* begin, const int32_t* end, int n, hipStream_t stream);
void kv8_compact_launch(const Kv8Book& k, int most, int32_t* moves, hipStream_t stream);
void kv8_copy_launch(Kv8CopyArgs a, int layers, hipStream_t stream);

void kv8_append_launch(const Kv8AppendArgs& a, int dtype, hipStream_t stream);
void kv8_gather_launch(const Kv8View& c, uint16_t* K, uint16_t* V, int dtype, hipStream_t stream);

// The launches of a call, each for the sequences whose number of rows suits it,
// and the workspace bytes beyond the counters (0: the call needs no workspace).
struct Kv8AttnPlan {
  Kv8AttnArgs few, many;
  bool has_few, has_many;
  size_t few_bytes, many_bytes;
};
Kv8AttnPlan kv8_attn_plan(const Kv8AttnArgs& a);
// With the workspace's counters and the memory after them.
void kv8_attn_launch(Kv8AttnPlan p, int* counters, char* partials, int dtype, hipStream_t stream);
// The kernel for many rows: rows of a workgroup, workgroups that share a compute
// unit, bytes of a split's partial result; and for documents, where row tiles are not
// split, waves of a workgroup (of 32 rows each).
int kv8_prompt_document_waves();
int kv8_prompt_rows(int dim);
int kv8_prompt_resident(int dim);
size_t kv8_prompt_partial(int dim);
void kv8_prompt_launch(const Kv8AttnArgs& a, int dtype, hipStream_t stream);

}  // namespace qlin
