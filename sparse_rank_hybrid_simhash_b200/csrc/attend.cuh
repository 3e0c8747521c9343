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

// ---- pages -----------------------------------------------------------------

// Most row tiles of a paged call: rows (token, head of the group) of each
// sequence fill tiles of their own.
inline int64_t paged_tiles(const AttendArgs& a, int tile) {
  return ((int64_t)a.rows * a.g + tile - 1) / tile + a.seqs;
}

struct PagedTile {
  int seq;     // -1: no such tile
  int tile;    // of the sequence
  int rows;    // (token, head) rows of the sequence
  int start;   // its first row of q
  int pos0;    // position of its first new token
  int len;     // context length with the new tokens
};

// New tokens of sequence b: clamped to what q holds and the context has
// (anything else is recorded and left out).
ELSAA_DEV int new_tokens(const AttendArgs& a, int b, int* start, int* len, bool lead) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1], l = a.lengths[b];
  *start = s0;
  *len = l;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.rows && l >= s1 - s0 &&
                  l <= (int64_t)a.page_size * a.table_width;
  if (ok) return s1 - s0;
  if (lead) raise_error(a.err, ERR_CHECK);
  return 0;
}

// Tile `t` of the whole batch, by one warp: sequences in order, each with
// ceil(tokens g / size) tiles.
ELSAA_DEV PagedTile find_paged_tile(const AttendArgs& a, int t, int size) {
  const int lane = threadIdx.x & 31;
  PagedTile f{-1, 0, 0, 0, 0, 0};
  for (int b0 = 0; b0 < a.seqs; b0 += 32) {
    int start = 0, len = 0, n = 0;
    if (b0 + lane < a.seqs) n = new_tokens(a, b0 + lane, &start, &len, true);
    const int rows = n * a.g, tiles = (rows + size - 1) / size;
    int upto = tiles;   // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, t < upto);
    if (hit) {
      const int w = __ffs(hit) - 1;
      f.seq = b0 + w;
      f.tile = t - __shfl_sync(0xffffffffu, upto - tiles, w);
      f.rows = __shfl_sync(0xffffffffu, rows, w);
      f.start = __shfl_sync(0xffffffffu, start, w);
      f.len = __shfl_sync(0xffffffffu, len, w);
      f.pos0 = f.len - __shfl_sync(0xffffffffu, n, w);
      return f;
    }
    t -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return f;
}

// The page of token j of sequence b; -1 (recorded) where the entry is no page.
ELSAA_DEV int page_of(const AttendArgs& a, int b, int j) {
  const int page = a.page_table[(int64_t)b * a.table_width + j / a.page_size];
  if (page >= 0 && page < a.pages) return page;
  raise_error(a.err, ERR_CHECK);
  return -1;
}

}  // namespace elsaa
