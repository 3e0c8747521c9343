// Work of a paged call for the kernels with 64-key blocks: one list of (row tile, key
// head, key block) units, in the order of the sequences, cut into equal runs, one per
// CTA.  The cuts follow the lengths on the device, so a captured launch does too.
#pragma once

#include "attend.cuh"

namespace elsaa {

constexpr int kBlk = 64;         // keys of a block
constexpr int kRuns = 444;       // most CTAs of a paged call (3 x 148)
constexpr int kMinUnits = 2;     // a run shorter than this is not worth a CTA

// Rows of a tile: 16 where a sequence's new (token, head of the group) rows fill no
// more on average (and the group fits), else 64.
inline int paged_tile_rows(int64_t rows, int seqs, int g) {
  return g <= 16 && (rows + seqs - 1) / seqs * g <= 16 ? 16 : 64;
}
inline size_t paged_runs_bytes(int d, int tile_rows) {
  return (size_t)2 * kRuns * tile_rows * (d + 2) * sizeof(float);
}

// A row tile: tt tokens of sequence b.
struct PagedItem {
  int p_lo, p_hi;          // positions of the tile's rows
  KeyBlocks kb;
};
ELSAA_DEV PagedItem paged_item(const AttendArgs& a, int tt, int tile, int tokens, int len) {
  PagedItem it;
  it.p_lo = len - tokens + tile * tt;
  it.p_hi = len - tokens + min(tokens, (tile + 1) * tt) - 1;
  it.kb = key_blocks(it.p_lo, it.p_hi, a.window, a.sinks, kBlk);
  return it;
}
ELSAA_DEV int64_t seq_units(const AttendArgs& a, int tt, int tokens, int len) {
  int64_t u = 0;
  for (int t = 0; t * tt < tokens; ++t) u += paged_item(a, tt, t, tokens, len).kb.count();
  return u * a.Hkv;
}

struct Run {
  int b, tile, hk, off, units;   // where it begins, and its length (0: no work)
  int start, tokens, len;        // of sequence b
  int64_t per;                   // units of a run
};
// The run of CTA `cta` of `ctas`, by one warp.
ELSAA_DEV Run find_run(const AttendArgs& a, int tt, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0, mine = 0;
  int start = 0, len = 0, n = 0;
  for (int b = lane; b < a.seqs; b += 32) {
    n = new_tokens(a, b, &start, &len, cta == 0);
    total += mine = seq_units(a, tt, n, len);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  int64_t per = div64(total + ctas - 1, ctas);
  if (per < kMinUnits) per = kMinUnits;
  Run c{0, 0, 0, 0, 0, 0, 0, 0, per};
  int64_t w = per * cta;
  if (w >= total) return c;
  c.units = (int)(per < total - w ? per : total - w);
  for (int b0 = 0; b0 < a.seqs; b0 += 32) {
    if (a.seqs > 32) {
      mine = n = 0;
      if (b0 + lane < a.seqs) {
        n = new_tokens(a, b0 + lane, &start, &len, false);
        mine = seq_units(a, tt, n, len);
      }
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w < upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      int64_t rest = w - __shfl_sync(0xffffffffu, upto - mine, l);
      c.b = b0 + l;
      c.start = __shfl_sync(0xffffffffu, start, l);
      c.tokens = __shfl_sync(0xffffffffu, n, l);
      c.len = __shfl_sync(0xffffffffu, len, l);
      for (; c.tile * tt < c.tokens; ++c.tile) {
        const int blk = paged_item(a, tt, c.tile, c.tokens, c.len).kb.count();
        if (rest < (int64_t)blk * a.Hkv) {
          c.hk = (int)div64(rest, blk);
          c.off = (int)(rest - (int64_t)c.hk * blk);
          break;
        }
        rest -= (int64_t)blk * a.Hkv;
      }
      return c;
    }
    w -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return c;
}

// The CTAs of an item of nblk units that begins with unit `begin`, and whether it is
// not the first item of its first CTA's run.
struct Ctas {
  int first, last, slot0;
};
ELSAA_DEV Ctas ctas_of(int64_t begin, int nblk, int64_t per) {
  Ctas c;
  c.first = (int)div64(begin, per);
  c.last = (int)div64(begin + nblk - 1, per);
  c.slot0 = begin == c.first * per ? 0 : 1;
  return c;
}

// Partial rows of items cut between CTAs: [slot][row][d] and (m, l) [slot][row], slot =
// 2 cta + (not the run's first item).
template <int ROWS>
ELSAA_DEV float* partial_o(const AttendArgs& a, int d, int slot, int row) {
  return reinterpret_cast<float*>(a.scratch) + ((int64_t)slot * ROWS + row) * d;
}
template <int ROWS>
ELSAA_DEV float2* partial_ml(const AttendArgs& a, int d, int slot, int row) {
  return reinterpret_cast<float2*>(partial_o<ROWS>(a, d, 2 * kRuns, 0)) + (int64_t)slot * ROWS + row;
}

}  // namespace elsaa
