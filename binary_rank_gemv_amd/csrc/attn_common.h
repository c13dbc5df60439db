// Shared device helpers of the operators between the projections.
#pragma once

#include "attn_launch.h"
#include "head_common.h"

namespace lbh {

// The sequence that a row belongs to: the last one that starts at or before it, -1 if
// none does.  64 starts a step, one a lane, so up to 64 sequences take one load and up
// to 4096 two.  All lanes of the wave are active and get the same answer.
__device__ __forceinline__ int sequence_of(const LbPages& P, int row) {
  const int lane = threadIdx.x & 63;
  int first = 0, count = P.seqs;
  while (true) {
    const int step = (count + 63) >> 6;
    const int at = lane * step;
    const bool before = at < count && P.starts[first + min(at, count - 1)] <= row;
    const uint64_t b = __ballot(before);
    if (b == 0) return -1;   // in later steps the first one is before the row: the step before found it so
    const int last = 63 - __builtin_clzll(b);
    first += last * step;
    count = min(step, count - last * step);
    if (step == 1) return first;
  }
}

// What a sequence has in a call.
struct Span {
  int start;   // its first row
  int rows;    // rows of it that the call has
  int keys;    // keys of it that its columns can hold
  int base;    // keys before its rows (less than 0 where lens is wrong: those do not exist)
};
__device__ __forceinline__ Span span_of(const LbPages& P, int start, int end, int len, int tokens) {
  Span s;
  s.start = start;
  const bool fine = start >= 0 && start < tokens && end > start && len >= 0;
  const int rows = fine ? end - start : 0;
  s.base = fine ? len - rows : 0;
  s.rows = fine ? min(rows, tokens - start) : 0;
  s.keys = fine ? min(len, P.columns << P.shift) : 0;
  return s;
}
__device__ __forceinline__ Span span_of(const LbPages& P, int seq, int tokens) {
  return span_of(P, P.starts[seq], P.starts[seq + 1], P.lens[seq], tokens);
}

// Where the page of a key begins, in pages; less than 0 where it has none.
__device__ __forceinline__ int page_of(const LbPages& P, int seq, int key) {
  const int column = key >> P.shift;
  if (key < 0 || column >= P.columns) return -1;
  const int page = P.table[seq * P.table_stride + column];
  return page < P.pages ? page : -1;
}

}  // namespace lbh
