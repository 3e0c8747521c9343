// What the window and paged attention kernels share: which keys a query sees,
// which key blocks a tile of queries visits, and where the tokens of a paged
// batch lie.
#pragma once

#include "common.cuh"
#include "layer.h"

namespace elsaa {

// Key j of the query at position i (window INT32_MAX: every earlier key).
ELSAA_DEV bool sees(int i, int j, int window, int sinks) {
  return j <= i && (i - j < window || j < sinks);
}

// How many keys the query at position i sees, and the x-th of them.
ELSAA_DEV int seen_keys(int i, int window, int sinks) {
  const int lo = max(i - window + 1, 0);
  return i - lo + 1 + min(sinks, lo);
}
ELSAA_DEV int seen_key(int x, int i, int window, int sinks) {
  const int lo = max(i - window + 1, 0), s = min(sinks, lo);
  return x < s ? x : lo + x - s;
}

// The backward's delta_i = y_i . dy_i takes y as it was stored.  For rows that see few
// keys that is a large part of dS = p (dy v - delta), a difference of like numbers: at
// bf16 and two keys dq and dk were off by 0.004 to 0.007 of their norm, at 32 keys by no
// more than the other roundings (0.0025).  So rows with up to this many keys take delta
// from its other form, sum_j p_ij dy_i . v_j, in fp32 (0.0024 to 0.0030): all rows of
// windows that short (2 x 12 heads of d = 64, 32768 tokens: the backward at window 16 893
// us, at 17 542), else the first of each sequence.
constexpr int kFewKeys = 16;

// The key blocks (of `size` keys) of a tile whose rows lie at positions
// p_lo .. p_hi: the sinks' blocks before the window, then the window's.
struct KeyBlocks {
  int sink_blocks, first, last;
  __host__ __device__ int count() const { return sink_blocks + (last - first + 1); }
  __host__ __device__ int block(int n) const { return n < sink_blocks ? n : first + n - sink_blocks; }
};
__host__ __device__ inline KeyBlocks key_blocks(int p_lo, int p_hi, int window, int sinks, int size) {
  KeyBlocks k{0, 0, -1};
  if (p_hi < p_lo) return k;   // a tile without positions
  const int lo = p_lo - window + 1;   // (window >= 1, p_lo >= 0: no overflow)
  k.first = lo > 0 ? lo / size : 0;
  k.last = p_hi / size;
  const int64_t sb = ((int64_t)sinks + size - 1) / size;
  k.sink_blocks = (int)(sb < k.first ? sb : k.first);
  return k;
}

// x / y of values below 2^63, in 32 bits where they fit (four times as fast).
ELSAA_DEV int64_t div64(int64_t x, int64_t y) {
  if (((uint64_t)x | (uint64_t)y) >> 32 == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}

// ---- pages -----------------------------------------------------------------

// Whether a sequence's new tokens, rows s0 .. s1 - 1 of q, lie in q's rows and its length holds
// them and fits its page table.  A sequence that does not fit is recorded and left out whole, by
// the write as by the attention: following part of it would put tokens into other tokens' slots.
ELSAA_DEV bool tokens_fit(int s0, int s1, int len, int rows, int64_t context) {
  return s0 >= 0 && s1 >= s0 && s1 <= rows && len >= s1 - s0 && len <= context;
}

// New tokens of sequence b; none (recorded) where they do not fit.
ELSAA_DEV int new_tokens(const AttendArgs& a, int b, int* start, int* len, bool lead) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1], l = a.lengths[b];
  *start = s0;
  *len = l;
  if (tokens_fit(s0, s1, l, a.rows, (int64_t)a.page_size * a.table_width)) return s1 - s0;
  if (lead) raise_error(a.err, ERR_CHECK);
  return 0;
}

// The page of token j of sequence b; -1 (recorded) where the entry is no page.
ELSAA_DEV int page_of(const AttendArgs& a, int b, int j) {
  const int page = a.page_table[(int64_t)b * a.table_width + j / a.page_size];
  if (page >= 0 && page < a.pages) return page;
  raise_error(a.err, ERR_CHECK);
  return -1;
}

}  // namespace elsaa
