// Causal attention over a sliding window with sinks, and over a paged cache, on
// the tensor cores (bf16, d = 64 or 128): a persistent warp-specialized tcgen05
// pipeline, one pass over the keys with the running maximum and sum.
//
// Two streams of 128 query rows share every 128-key block of K and V: S = Q K^T
// (TMEM), P = 2^(scale log2e S - m) written over S as bf16, O += P V (TMEM).  A stream
// works on 64-key halves in turn: while its softmax reads one, the tensor cores put
// the other's P into O and the next S in its place, and a half that no row of the
// stream sees is skipped.  (With whole blocks the softmax waited for both products; a
// padded batch at d = 128 171 -> 159 us, prompt chunks 172 -> 154 us, long windows
// unchanged within 4 %.)  A row belongs to one thread, so maximum, sum and rescaling stay in its registers.  O is
// rescaled only when a row's maximum has grown by more than 2^8 over the one it
// used so far (P <= 2^8 otherwise; bf16 keeps the same relative precision there,
// and the final division cancels the reference): a rare event after the first
// blocks, where a rescaling of every block costs a pass over O.  P is rounded to bf16,
// the type of V and so of both operands of P V: half a step (2^-8) of every probability,
// in both directions, takes the error of y against 64 bits from its own rounding's
// 0.0016 of its norm to 0.0021 .. 0.0023.  P as two bf16 parts (P V twice; they fit over
// S) would leave y's own rounding, at 1035 -> 1365 us for a 16k prefill (32 and 8 heads
// of d = 128, window 4096), 168 -> 207 for prompt chunks and 1781 -> 1880 for text-32k
// with its backward: not taken.  Sums and maxima are fp32.
//
// Streams of an item:
//   window, g even    two query heads of one key head at the same 128 tokens
//   window, g odd     two successive 128-token tiles of one head
//   pages             two successive tiles of (token, head of the group) rows; where
//                     a sequence's rows fill one tile, the streams take alternate key
//                     blocks of it and are merged at the end.  (Calls with up to 16 rows
//                     a sequence on average go to paged_decode.cu.)
// Paged work is one list of (tile pair, key head, key block) units cut into equal
// runs, one per CTA (the cuts are found from the lengths on the device, so a
// captured launch follows them); an item cut between CTAs leaves unnormalised
// partial rows in the workspace, and the last CTA to get there adds them up, in the
// CTAs' order whichever it is (a counter a warp: a row's partials come from the same
// warp of every CTA).  A second kernel for that cost 12 us a call.
//
// Roles (384 threads, one CTA per SM): warps 0..3 and 4..7 softmax and output of
// the two streams, warp 8 copies Q and K, warps 9 and 10 issue the streams' products,
// warp 11 copies V and hands out the items through a ring in shared memory (registers move
// between whole warpgroups: a softmax thread holds its row of S).  With pages of 16
// tokens a block is 16 copies each of K and V, at about 70 cycles a copy a warp: two
// copying warps keep up with the pages' bytes.  K and V blocks pass
// through one ring of slots (K0 V0 K1 V1 ...).  Keys behind a length may hold
// anything: their scores are replaced, and the MMA warps zero their value rows
// in shared memory (0 times a stray infinity is not 0).
//
// Bound: at d = 128 a block costs 1024 cycles of products and 1024 of
// exponentials (16 a cycle an SM) a stream, at d = 64 512 and 1024; one pair of
// exponentials in four goes to the FMA pipe (attend_tc.cuh).  What is left over is the
// chain of a half block: S read from TMEM, maximum, exponentials, P written, handed over.
// Measured: 8192 tokens, 32 query and 8 key heads, window 4096: d = 128 402 us (1026
// TFLOP/s), d = 64 360 us (572); text-32k (2 x 12 heads of d = 64, 32768 tokens) at window
// 1024 431 us (480).
//
// Every wait is bounded; one that gives up records ERR_TIMEOUT, every role leaves
// its loop, and copies and products in flight end before TMEM is freed.
#include <math.h>

#include "attend_tc.cuh"
#include "internal.h"
#include "ring_drain.h"

namespace elsaa {
namespace {

using namespace tc;

constexpr int kThreads = 384;
// registers a thread: 384 x 168 at launch = 256 x 216 + 128 x 72
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 11;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTO = 256;            // O of stream s at kTO + 128 s; S (and P) at 128 s
constexpr float kGrow = 8.0f;            // log2 of the growth that rescales O
constexpr int kMinUnits = 2;             // a run shorter than this is not worth a CTA

template <int D>
struct Lay {
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kBars = kRing + kSlots * kTile;
  static constexpr uint32_t kMl = kBars + 1024;                // m, l of stream 1 [2][128]
  static constexpr uint32_t kDyn = kMl + 1024;
};
static_assert(Lay<128>::kDyn <= 232448, "shared memory at d = 128");

struct Maps {
  CUtensorMap q, k, v;
};

struct Shape {
  int tiles;        // window: 128-token tiles (g even) or pairs of them (g odd)
  int pair_heads;   // window: the streams are two heads
  int tt;           // pages: tokens of a row tile, 128 / g
  int sub;          // pages: rows of a page box
  float scale_log2;
  int slot_rows;    // pages: rows of a partial slot
};

// One CTA's piece of work: rows of both streams against the blocks n0 .. n1 - 1
// of the item's block list.
struct Item {
  int b, hk, len;
  int h[2], r0[2];          // window: head and first token; pages: - and first new token
  int p_first[2], p_last[2];   // positions of a stream's rows (p_last < 0: no rows)
  int start, tokens;        // pages: first row of q, new tokens
  bool split;               // one tile, alternate blocks
  int sink_blocks, first, nblk, n0, n1;
  int f64[2], l64[2], s64;  // a stream's window in 64-key halves of blocks, and the sinks'
  int order;                // the CTA's items before it; -1: there are no more
  int cta0, cta1, slot0;    // a cut item: its CTAs, and whether it is not the first of cta0's
  ELSAA_DEV int block(int n) const { return n < sink_blocks ? n : first + n - sink_blocks; }
  // whether the stream uses half h of block n
  ELSAA_DEV bool uses(int s, int n, int h) const {
    if (split && (n & 1) != s) return false;
    const int x = 2 * block(n) + h;
    return x <= pick(l64, s) && (x >= pick(f64, s) || x < s64);
  }
  // the last half (2 n + h) of [n0, n1) that the stream uses; 2 n0 - 1: none
  ELSAA_DEV int last_use(int s) const {
    int x = 2 * n1 - 1;
    while (x >= 2 * n0 && !uses(s, x >> 1, x & 1)) --x;
    return x;
  }
};

ELSAA_DEV void item_blocks(Item& it, const AttendArgs& a) {
  it.s64 = (int)(((int64_t)a.sinks + 63) / 64);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int lo = it.p_first[s] - a.window + 1;
    it.f64[s] = lo > 0 ? lo / 64 : 0;
    it.l64[s] = it.p_last[s] >= 0 ? it.p_last[s] / 64 : -1;
  }
  // the union: stream 0 starts and ends no later than stream 1 (where that has rows)
  it.nblk = it.sink_blocks = it.first = 0;
  if (it.p_last[0] < 0) return;
  it.first = it.f64[0] >> 1;
  it.sink_blocks = min((it.s64 + 1) >> 1, it.first);
  it.nblk = it.sink_blocks + (max(it.l64[0], it.l64[1]) >> 1) - it.first + 1;
}

// Where a paged CTA's run begins, and its length (0: no work).
struct Cut {
  int b, pair, hk, off, units;
  int start, tokens, len;       // of sequence b
};

constexpr int kItems = 4;
struct Bars {
  uint64_t full[8], empty[8];   // ring slots
  uint64_t q_full, q_empty;
  uint64_t s_full[2][2], p_full[2][2];   // [stream][half]
  uint64_t pv_done[2], o_full[2];
  uint64_t x_full, x_done;      // a split item: O of stream 1 given, and read
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t drain;
  uint32_t loads[2];            // copies into the ring that K's and V's warp have started
  uint32_t tmem;
  Cut cut;                      // a paged CTA's first item
  int64_t per;                  // units of a run
  Item items[kItems];
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// ---- window items ----------------------------------------------------------

// Item x, the longest (last) tiles first, heads and batches inside.
ELSAA_DEV Item window_item(const AttendArgs& a, const Shape& sh, int64_t x) {
  Item it;
  const int hh = sh.pair_heads ? a.H / 2 : a.H;
  const int t = sh.tiles - 1 - (int)(x / ((int64_t)a.B * hh));
  const int bh = (int)(x % ((int64_t)a.B * hh));
  it.b = bh / hh;
  const int h = sh.pair_heads ? bh % hh * 2 : bh % hh;
  it.hk = h / a.g;
  it.len = a.lengths ? min(max(a.lengths[it.b], 0), a.N) : a.N;
  it.split = false;
  it.start = it.tokens = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    it.h[s] = sh.pair_heads ? h + s : h;
    it.r0[s] = sh.pair_heads ? t * kBlock : (2 * t + s) * kBlock;
    it.p_first[s] = it.r0[s];
    it.p_last[s] = it.r0[s] < it.len ? min(it.len, it.r0[s] + kBlock) - 1 : -1;
  }
  item_blocks(it, a);
  it.n0 = 0;
  it.n1 = it.nblk;
  return it;
}

// ---- paged items -----------------------------------------------------------

ELSAA_DEV int pairs_of(int tokens, int tt) { return (tokens + 2 * tt - 1) / (2 * tt); }

// Tile pair `pair` of sequence b (tokens new tokens from row start, context len).
ELSAA_DEV Item paged_item(const AttendArgs& a, const Shape& sh, int b, int pair, int hk, int start,
                          int tokens, int len) {
  Item it;
  it.b = b;
  it.hk = hk;
  it.len = len;
  it.start = start;
  it.tokens = tokens;
  const int t0 = 2 * pair * sh.tt;
  it.split = t0 + sh.tt >= tokens;   // the pair has one tile
  const int pos0 = len - tokens;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int r = it.split ? t0 : t0 + s * sh.tt;
    it.h[s] = 0;
    it.r0[s] = r;
    it.p_first[s] = pos0 + r;
    it.p_last[s] = pos0 + min(tokens, r + sh.tt) - 1;
  }
  item_blocks(it, a);
  it.n0 = 0;
  it.n1 = it.nblk;
  return it;
}

// Blocks of tile pair `pair` (paged_item's nblk; a pair's rows are successive, so its
// list is that of its first and last row).
ELSAA_DEV int pair_blocks(const AttendArgs& a, const Shape& sh, int pair, int tokens, int len) {
  const int t0 = 2 * pair * sh.tt, p_lo = len - tokens + t0;
  const int p_hi = len - tokens + min(tokens, t0 + 2 * sh.tt) - 1;
  const int lo = p_lo - a.window + 1, first = lo > 0 ? lo >> 7 : 0;
  const int s128 = (int)(((int64_t)a.sinks + 127) >> 7);
  return min(s128, first) + (p_hi >> 7) - first + 1;
}
// Units (tile pair, key head, block) of a sequence.
ELSAA_DEV int64_t seq_units(const AttendArgs& a, const Shape& sh, int tokens, int len) {
  int64_t u = 0;
  const int pairs = pairs_of(tokens, sh.tt);
  for (int p = 0; p < pairs; ++p) u += pair_blocks(a, sh, p, tokens, len);
  return u * a.Hkv;
}

// The run of CTA `cta` of `ctas`, by one warp; *per: units of a run.
ELSAA_DEV Cut find_run(const AttendArgs& a, const Shape& sh, int cta, int ctas, int64_t* per) {
  const int lane = threadIdx.x & 31;
  Cut c{0, 0, 0, 0, 0, 0, 0, 0};
  int64_t total = 0, mine = 0;
  int start = 0, len = 0, n = 0;
  for (int b = lane; b < a.seqs; b += 32) {
    n = new_tokens(a, b, &start, &len, cta == 0);
    total += mine = seq_units(a, sh, n, len);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  *per = div64(total + ctas - 1, ctas);
  if (*per < kMinUnits) *per = kMinUnits;
  int64_t w = *per * cta;
  if (w >= total) return c;
  c.units = (int)(*per < total - w ? *per : total - w);
  for (int b0 = 0; b0 < a.seqs; b0 += 32) {
    if (a.seqs > 32) {
      mine = n = 0;
      if (b0 + lane < a.seqs) {
        n = new_tokens(a, b0 + lane, &start, &len, false);
        mine = seq_units(a, sh, n, len);
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
      const int pairs = pairs_of(c.tokens, sh.tt);
      for (; c.pair < pairs; ++c.pair) {
        const int blk = pair_blocks(a, sh, c.pair, c.tokens, c.len);
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

// Walks a CTA's items.
template <bool PAGED>
struct Walk {
  const AttendArgs& a;
  const Shape& sh;
  int64_t x, items;                          // window
  int b, pair, hk, off, left, start, tokens, len;   // pages
  int order;                                 // items so far
  int64_t per, at;                           // pages: units of a run, and the next unit
  ELSAA_DEV Walk(const AttendArgs& a_, const Shape& sh_, int64_t items_, const Cut& c, int64_t per_)
      : a(a_), sh(sh_), x(blockIdx.x), items(items_), order(0), per(per_) {
    if (PAGED) {
      at = per * blockIdx.x;
      b = c.b, pair = c.pair, hk = c.hk, off = c.off, left = c.units;
      start = c.start, tokens = c.tokens, len = c.len;
    }
  }
  ELSAA_DEV bool next(Item& it) {
    if (!PAGED) {
      if (x >= items) return false;
      it = window_item(a, sh, x);
      it.order = order++;
      x = next_item(a.counters, items);
      return true;
    }
    if (left <= 0) return false;
    while (pair >= pairs_of(tokens, sh.tt)) {   // (a later sequence holds the units left)
      if (++b >= a.seqs) return false;
      pair = hk = off = 0;
      tokens = new_tokens(a, b, &start, &len, false);
    }
    it = paged_item(a, sh, b, pair, hk, start, tokens, len);
    it.n0 = off;
    it.n1 = min(it.nblk, off + left);
    it.cta0 = it.cta1 = it.slot0 = 0;
    if (it.n1 - it.n0 < it.nblk) {
      const int64_t begin = at - off;
      it.cta0 = (int)div64(begin, per);
      it.cta1 = (int)div64(begin + it.nblk - 1, per);
      it.slot0 = begin == it.cta0 * per ? 0 : 1;
    }
    left -= it.n1 - it.n0;
    at += it.n1 - it.n0;
    off = 0;
    if (++hk == a.Hkv) hk = 0, ++pair;
    it.order = order++;
    return true;
  }
};

// ---- kernel ------------------------------------------------------------------

// The scratch of a paged call: partial rows [slot][row][D] and (m, l) [slot][row];
// slot = ((cta * 2 + (not the run's first item)) * 2 + stream).
struct Partial {
  float* o;
  float2* ml;
};
ELSAA_DEV Partial partial_row(const AttendArgs& a, const Shape& sh, int d, int slot, int row) {
  const int64_t slots = (int64_t)kMaxCtas * 4, at = (int64_t)slot * sh.slot_rows + row;
  float* o = reinterpret_cast<float*>(a.scratch);
  return {o + at * d, reinterpret_cast<float2*>(o + slots * sh.slot_rows * d) + at};
}

// R rows of a cut item (merge_rows), from row x0 of the warp's on; lanes over the
// columns.  m: the maximum of row `lane`.
template <int D, int R>
ELSAA_DEV void merge_group(const AttendArgs& a, const Shape& sh, const Item& it, int st, int row0,
                           int x0, int rows, float m) {
  constexpr int V = D / 32;   // values of a lane
  const int lane = threadIdx.x & 31, cta0 = it.cta0, cta1 = it.cta1, slot0 = it.slot0;
  float o[R][V], l = 0.f;
#pragma unroll
  for (int x = 0; x < R; ++x)
#pragma unroll
    for (int e = 0; e < V; ++e) o[x][e] = 0.f;
#pragma unroll(16 / R)
  for (int i = cta0; i <= cta1; ++i) {
    const int slot = (i * 2 + (i == cta0 ? slot0 : 0)) * 2 + st;
    const float2 ml = __ldcg(partial_row(a, sh, D, slot, row0 + min(lane, rows - 1)).ml);
    const float* p = partial_row(a, sh, D, slot, row0).o + lane * V;
    float v[R][V];
#pragma unroll
    for (int x = 0; x < R; ++x) {   // (past the last row: that one again)
      const float* q = p + (int64_t)min(x0 + x, rows - 1) * D;
      if (V == 4) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(q));
        v[x][0] = u.x, v[x][1] = u.y, v[x][2 % V] = u.z, v[x][3 % V] = u.w;
      } else {
        const float2 u = __ldcg(reinterpret_cast<const float2*>(q));
        v[x][0] = u.x, v[x][1] = u.y;
      }
    }
    const float w = ml.x > -INFINITY ? ex2(ml.x - m) : 0.f;   // (no blocks of the stream there)
    l += ml.y * w;
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const float wx = __shfl_sync(0xffffffffu, w, min(x0 + x, rows - 1));
#pragma unroll
      for (int e = 0; e < V; ++e) o[x][e] += v[x][e] * wx;
    }
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
  for (int x = 0; x < R; ++x) {
    const float f = __shfl_sync(0xffffffffu, inv, min(x0 + x, rows - 1));
    if (x0 + x >= rows) break;
    const int row = row0 + x0 + x;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) +
                       (int64_t)(it.start + pick(it.r0, st) + row / a.g) * a.sy.n +
                       (int64_t)(it.hk * a.g + row % a.g) * a.sy.h + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(y + e) =
          __floats2bfloat162_rn(o[x][e] * f, o[x][(e + 1) % V] * f);
  }
}

// The rows of one warp of a cut item from the partials of all its CTAs, in their
// order: m = max m_i, y = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
template <int D>
ELSAA_DEV void merge_rows(const AttendArgs& a, const Shape& sh, const Item& it, int st, int row0) {
  const int lane = threadIdx.x & 31, cta0 = it.cta0, cta1 = it.cta1, slot0 = it.slot0;
  const int rows = min(min(sh.tt, it.tokens - pick(it.r0, st)) * a.g - row0, 32);   // (at least 1)
  float m = -INFINITY;   // of row `lane`
#pragma unroll 8
  for (int i = cta0; i <= cta1; ++i)
    m = fmaxf(m, __ldcg(partial_row(a, sh, D, (i * 2 + (i == cta0 ? slot0 : 0)) * 2 + st,
                                    row0 + min(lane, rows - 1)).ml).x);
  if (rows <= 4) {
    merge_group<D, 4>(a, sh, it, st, row0, 0, rows, m);
  } else {
    for (int x0 = 0; x0 < rows; x0 += 8) merge_group<D, 8>(a, sh, it, st, row0, x0, rows, m);
  }
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
attend_fwd_kernel(const __grid_constant__ Maps maps, const AttendArgs a, const Shape sh,
                  int64_t items) {
  using L = Lay<D>;
  constexpr int SL = L::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((sbase & 1023u) != 0) {
    if (tid == 0) raise_error(a.err, ERR_CHECK);
    return;
  }
  if (tid == 32 * kKWarp) {
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  if (tid == 0) {
    for (int i = 0; i < SL; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 2);       // both MMA warps
    }
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);
    for (int s = 0; s < 2; ++s) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bars->s_full[s][h], 1);
        mbar_init(&bars->p_full[s][h], 4);   // a stream's warps
      }
      mbar_init(&bars->pv_done[s], 1);
      mbar_init(&bars->o_full[s], 1);
    }
    mbar_init(&bars->x_full, 4);
    mbar_init(&bars->x_done, 4);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], 12);   // eight softmax warps, K, V, two MMA
    }
    mbar_init(&bars->drain, 2);
    fence_mbar_init();
  }
  if (PAGED && warp == 0) {   // this CTA's run of units
    int64_t per;
    const Cut c = find_run(a, sh, blockIdx.x, gridDim.x, &per);
    if (lane == 0) {
      bars->cut = c;
      bars->per = per;
    }
  }
  __syncthreads();
  if (PAGED && bars->cut.units == 0) return;
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;
  bool ok = true;
  uint32_t ni = 0;   // items taken so far
  // the next item, or null behind the last one (or where a wait gave up)
  auto take = [&]() -> const Item* {
    if (!ok) return nullptr;
    ok = warp_wait(&bars->item_full[ni % kItems], (ni / kItems) & 1, a.err);
    const Item* it = &bars->items[ni % kItems];
    return ok && it->order >= 0 ? it : nullptr;
  };
  auto give_back = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[ni % kItems]);
    ++ni;
  };

  if (warp < kKWarp) {
    regs_up<kSoftmaxRegs>();
    // ------------------------------------------------------------------ softmax and output
    const int st = warp >> 2, row = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + 128 * st + lane_off, tO = tmem + kTO + 128 * st + lane_off;
    float* ml1 = reinterpret_cast<float*>(smem + L::kMl);
    uint32_t ns = 0, np = 0, no = 0, nx = 0;   // ns: phases of both halves' S, one bit each
    const int tok_of_row = PAGED ? row / a.g : row;
    while (const Item* item = take()) {
      const Item& it = *item;
      // the row's position; rows past the tile or its tokens have none
      const int r = pick(it.r0, st) + tok_of_row;
      const int pos = pick(it.p_first, st) + tok_of_row;
      const bool live = PAGED ? tok_of_row < sh.tt && r < it.tokens : r < it.len;
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m = -INFINITY, l = 0.f;
      bool any = false;
      const int n1 = it.n1, sink_blocks = it.sink_blocks, shift = it.first - sink_blocks;
      const int p_first = pick(it.p_first, st), edge = pick(it.p_last, st) - a.window;
      const int f64 = pick(it.f64, st), l64 = pick(it.l64, st), s64 = it.s64;
      const bool split = it.split;
#pragma unroll 1
      for (int x = 2 * it.n0; x < 2 * n1 && ok; ++x) {   // half x & 1 of block x >> 1
        const int n = x >> 1, h = x & 1, k64 = 2 * (n < sink_blocks ? n : n + shift) + h;
        if ((split && (n & 1) != st) || k64 > l64 || (k64 < f64 && k64 >= s64)) continue;
        ok = warp_wait(&bars->s_full[st][h], (ns >> h) & 1, a.err);
        if (!ok) break;
        ns ^= 1u << h;
        fence_after();
        if (warp_live) {
          const int j0 = k64 * 64;
          float sv[64];
          tmem_ld32(tS + 64 * h, sv);
          tmem_ld32(tS + 64 * h + 32, sv + 32);
          tmem_ld_wait();
          // some row of the tile does not see all of the half
          if (j0 + 63 > p_first || j0 <= edge) {
            const int hi = pos - j0, lo = pos - a.window + 1 - j0;
            const int sk = (int)min((int64_t)a.sinks - j0, (int64_t)64);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t see = upto_bits(hi - 32 * c) &
                                   (~upto_bits(lo - 1 - 32 * c) | upto_bits(sk - 1 - 32 * c));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see >> e) & 1u)) sv[32 * c + e] = -INFINITY;
            }
          }
          float t0 = sv[0], t1 = sv[1], t2 = sv[2], t3 = sv[3];
#pragma unroll
          for (int e = 4; e < 64; e += 4) {
            t0 = fmaxf(t0, sv[e]);
            t1 = fmaxf(t1, sv[e + 1]);
            t2 = fmaxf(t2, sv[e + 2]);
            t3 = fmaxf(t3, sv[e + 3]);
          }
          const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * sh.scale_log2;   // scale > 0
          const bool grow = top > m + kGrow;
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? ex2(m - top) : 1.f;
            if (grow) m = top;
            l *= f;
            if (any) {
              // the last product into O has ended
              ok = warp_wait(&bars->pv_done[st], (np - 1) & 1, a.err);
              fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                float ov[16];
                uint32_t ow[16];
                tmem_ld16(tO + 16 * c, ov);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(ov[e] * f);
                tmem_st16(tO + 16 * c, ow);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float a0 = sv[32 * c + e], a1 = sv[32 * c + e + 1];
              fma2(a0, a1, sh.scale_log2, sh.scale_log2, -base, -base);
              exp2_pair<true>(e >> 1, a0, a1);
              add2(l0, l1, a0, a1);
              const __nv_bfloat162 hv = __floats2bfloat162_rn(a0, a1);
              packed[e >> 1] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            tmem_st16(tS + 64 * h + 16 * c, packed);   // over S, which is all in registers
          }
          l += l0 + l1;
          tmem_st_wait();
        }
        any = true;
        ++np;
        fence_before();
        warp_arrive(&bars->p_full[st][h]);
      }
      if (!ok) break;
      if (any) {
        ok = warp_wait(&bars->o_full[st], no & 1, a.err);
        if (!ok) break;
        ++no;
        fence_after();
      }
      // rows of the result: final (the item is whole in this CTA) or partial
      const bool whole = !PAGED || (it.n0 == 0 && it.n1 == it.nblk);
      // weights of O of this stream and of stream 1 (0: no keys seen there, O not read; a row
      // whose scores were all NaN has no maximum either, but a NaN sum, and stays NaN)
      float w0 = any ? 1.f : 0.f, w1 = 0.f;
      if (PAGED && it.split) {
        // stream 0 reads both O (a row's lane is the same in both)
        if (st == 1) {
          ml1[row] = any ? m : -INFINITY;
          ml1[128 + row] = any ? l : 0.f;
          fence_before();
          warp_arrive(&bars->x_full);
        } else {
          ok = warp_wait(&bars->x_full, nx & 1, a.err);
          if (!ok) break;
          fence_after();
          const float m1 = ml1[row], l1 = ml1[128 + row], mm = fmaxf(m, m1);
          w0 = m > -INFINITY ? ex2(m - mm) : 0.f * l;
          w1 = m1 > -INFINITY ? ex2(m1 - mm) : 0.f * l1;
          l = l * w0 + l1 * w1;
          m = mm;
        }
      }
      const bool out = !(PAGED && it.split && st == 1);
      if (out && PAGED && warp_live) {
        const bool two = it.split && __any_sync(0xffffffffu, w1 != 0.f);
        const int slot = ((int)blockIdx.x * 2 + (it.order > 0 ? 1 : 0)) * 2 + st;
        const float inv = !whole ? 1.f : l > 0.f ? 1.0f / l : 0.f;
        __nv_bfloat16* yrow = nullptr;
        float* prow = nullptr;
        if (live && whole)
          yrow = static_cast<__nv_bfloat16*>(a.y) + (int64_t)(it.start + r) * a.sy.n +
                 (int64_t)(it.hk * a.g + row % a.g) * a.sy.h;
        if (live && !whole) {
          const Partial p = partial_row(a, sh, D, slot, row);
          *p.ml = make_float2(m, l);
          prow = p.o;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float ov[32], ow[32];
          tmem_ld32(tO + 32 * c, ov);
          if (two) tmem_ld32(tO + 128 + 32 * c, ow);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            ov[e] = w0 != 0.f ? ov[e] * (w0 * inv) : 0.f;
            if (two && w1 != 0.f) ov[e] += ow[e] * (w1 * inv);
          }
          if (yrow != nullptr) store32(yrow + 32 * c, ov);
          if (prow != nullptr) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(prow + 32 * c + 4 * q) =
                  make_float4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
          }
        }
        if (!whole) {
          // the last of the item's CTAs to come here with this warp's rows adds them up
          uint32_t* counter = a.counters + it.cta0 * 8 + warp;
          uint32_t before = 0;
          __threadfence();
          __syncwarp();
          if (lane == 0) before = atomicAdd(counter, 1u);
          before = __shfl_sync(0xffffffffu, before, 0);
          if (before == (uint32_t)(it.cta1 - it.cta0)) {
            __threadfence();
            merge_rows<D>(a, sh, it, st, 32 * (warp & 3));
            if (lane == 0) *counter = 0;
          }
        }
      }
      if (!PAGED) {
        // rows at and behind the length: zeros (a live row sees its own key: l > 0, or NaN)
        const float inv = live ? 1.0f / l : 0.f;
        const bool store = r < a.N;
        if (store)
          a.lse[((int64_t)it.b * a.H + pick(it.h, st)) * a.N + r] =
              live ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        __nv_bfloat16* yrow = static_cast<__nv_bfloat16*>(a.y) + (int64_t)it.b * a.sy.b +
                              (int64_t)pick(it.h, st) * a.sy.h + (int64_t)r * a.sy.n;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float ov[32];
          if (warp_live) {
            tmem_ld32(tO + 32 * c, ov);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = live ? ov[e] * inv : 0.f;
          if (store) store32(yrow + 32 * c, ov);
        }
      }
      fence_before();
      if (PAGED && it.split) {
        if (st == 0) {
          warp_arrive(&bars->x_done);
        } else {
          ok = warp_wait(&bars->x_done, nx & 1, a.err);
          if (!ok) break;
        }
        ++nx;
      }
      give_back();
    }
  } else {
    regs_down<kOtherRegs>();
    if (warp == kKWarp || warp == kVWarp) {
      // ------------------------------------------------------------------ copies (and items)
      const int kv = warp == kVWarp ? 1 : 0;
      const CUtensorMap* map = kv ? &maps.v : &maps.k;
      const int subs = PAGED ? kBlock / sh.sub : 1;
      RingPos<SL> at;            // K and V take the slots in turn
      if (kv) at.next();
      uint32_t loads = 0, nq = 0;
      // pages: this lane's box of block n; boxes behind the length, or that no row of the
      // item sees, are not looked up, and a page outside the pool reads as zeros
      auto lookup = [&](const Item& it, int n) -> int {
        if (!PAGED || lane >= subs || n >= it.n1) return a.pages;
        const int j = it.block(n) * kBlock + lane * sh.sub;
        if (j > max(it.p_last[0], it.p_last[1]) ||
            !(j < a.sinks || (int64_t)j + sh.sub - 1 > (int64_t)it.p_first[0] - a.window))
          return a.pages;
        const int page = page_of(a, it.b, j);
        return page < 0 ? a.pages : page;
      };
      auto load_block = [&](const Item& it, int n, int page) {
        // (a fresh barrier counts as released)
        ok = ok && warp_wait(&bars->empty[at.slot], at.phase ^ 1, a.err);
        if (!ok) return;
        uint64_t* bar = &bars->full[at.slot];
        if (lane == 0) mbar_arrive_expect_tx(bar, L::kTile);
        __syncwarp();
        const int j0 = it.block(n) * kBlock;
        const uint32_t dst = sbase + L::kRing + at.slot * L::kTile;
        if (lane < subs) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            if (PAGED)
              tma_load_4d(dst + c * kAtom + lane * sh.sub * 128, map, 64 * c,
                          (j0 + lane * sh.sub) % a.page_size, it.hk, page, bar);
            else
              tma_load_4d(dst + c * kAtom, map, 64 * c, j0, it.hk, it.b, bar);
          }
        }
        __syncwarp();
        at.next(), at.next();
        ++loads;
      };
      auto load_q = [&](const Item& it) {
        if (nq > 0) ok = ok && warp_wait(&bars->q_empty, (nq - 1) & 1, a.err);
        if (!ok) return;
        if (lane == 0) {
          const int tiles = it.split ? 1 : 2;
          const uint32_t rows = PAGED ? sh.tt * a.g : kBlock;
          mbar_arrive_expect_tx(&bars->q_full, tiles * rows * D * 2);
#pragma unroll
          for (int s = 0; s < 2; ++s)
            for (int c = 0; c < (s < tiles ? D / 64 : 0); ++c) {
              const uint32_t dst = sbase + L::kQ + s * L::kTile + c * kAtom;
              if (PAGED)
                tma_load_4d(dst, &maps.q, 64 * c, it.hk * a.g, it.start + it.r0[s], 0, &bars->q_full);
              else
                tma_load_4d(dst, &maps.q, 64 * c, it.r0[s], it.h[s], it.b, &bars->q_full);
            }
        }
        __syncwarp();
        ++nq;
      };
      Walk<PAGED> walk(a, sh, items, bars->cut, bars->per);   // (V's warp, lane 0)
      uint32_t given = 0;
      bool more = kv == 1;
      auto hand_out = [&]() {
        if (!more) return;
        const uint32_t i = given % kItems;
        ok = ok && warp_wait(&bars->item_empty[i], ((given / kItems) & 1) ^ 1, a.err);
        if (!ok) return;
        if (lane == 0) {
          Item it;
          more = walk.next(it);
          if (!more) it.order = -1;
          bars->items[i] = it;
          mbar_arrive(&bars->item_full[i]);
        }
        more = __shfl_sync(0xffffffffu, more, 0);
        ++given;
      };
      hand_out();
      for (;;) {
        hand_out();   // one ahead of what is copied
        const Item* item = take();
        if (item == nullptr) break;
        const Item& it = *item;
        const int n0 = it.n0, n1 = it.n1;
        if (n0 < n1) {
          int page = lookup(it, n0);
          // Q of the first item first; later ones behind the first block, which need not
          // wait for the last item's scores
          const bool late = nq > 0;
          if (!kv && !late) load_q(it);
          for (int n = n0; n < n1 && ok; ++n) {
            const int now = page;
            page = lookup(it, n + 1);   // (in flight while the slot is awaited)
            load_block(it, n, now);
            if (!kv && late && n == n0) load_q(it);
          }
        }
        if (!ok) break;
        give_back();
      }
      if (lane == 0) {
        bars->loads[kv] = loads;
        if (nq > 0) mbar_wait(&bars->q_full, (nq - 1) & 1, a.err);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ products
      // a warp a stream: one's waits and bookkeeping run under the other's products
      constexpr uint32_t id_pv = idesc_bf16(128, D, false, true);
      constexpr uint32_t kStep = L::kTile >> 4;   // a slot further, in descriptor units
      const int st = warp - kMmaWarp;
      const uint32_t tS = uniform(tmem + 128 * st), tO = uniform(tmem + kTO + 128 * st);
      const uint32_t q_d = row_desc(sbase + L::kQ);
      const uint32_t k_d = row_desc(sbase + L::kRing), v_d = col_desc(sbase + L::kRing);
      uint32_t nq = 0, np = 0;   // np: phases of both halves' P, one bit each
      RingPos<SL> at;   // the ring slot of the next load: K of a block, then V
      auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, a.err); };
      while (const Item* item = take()) {
        const Item& it = *item;
        const int n0 = it.n0, n1 = it.n1, len = it.len;
        if (n0 >= n1) {
          give_back();
          continue;
        }
        const int last = it.last_use(st);
        const uint32_t qd = uniform(q_d + (it.split || st == 0 ? 0 : kStep));
        bool pend[2] = {false, false};
        uint32_t add = 0, sv = 0;          // slot of V of block n - 1
        for (int n = n0; n <= n1 && ok; ++n) {
          // what block n needs is awaited before the softmax of block n - 1
          const bool more = n < n1;
          const uint32_t sk = at.slot;
          if (more) {
            ok = wait(&bars->full[sk], at.phase);
            if (ok && n == n0) ok = wait(&bars->q_full, nq & 1);
            at.next();
          }
          const uint32_t kd = uniform(k_d + sk * kStep), vd = uniform(v_d + sv * kStep);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool use = more && it.uses(st, n, h);
            const uint32_t acc = uniform(add);
            if (pend[h]) {
              ok = ok && wait(&bars->p_full[st][h], (np >> h) & 1);
              np ^= 1u << h;
            }
            if (!ok) break;
            fence_after();
            if (elect_one()) {
              if (pend[h]) {               // O (+)= P V of half h of block n - 1
#pragma unroll
                for (int x = 0; x < 64; x += 16)
                  mma_ts(tO, tS + 64 * h + (x >> 1), vd + (64 * h + x) * 8, id_pv, x > 0 ? 1u : acc);
                mma_commit(&bars->pv_done[st]);
                if (2 * (n - 1) + h == last) mma_commit(&bars->o_full[st]);
              }
              if (use) {                   // S = Q K^T of half h of block n
                mma_tiles<D, 64>(tS + 64 * h, qd, kd + 512 * h);
                mma_commit(&bars->s_full[st][h]);
              }
            }
            __syncwarp();
            if (pend[h]) add = 1;
            pend[h] = use;
          }
          if (!ok) break;
          if (elect_one()) {
            if (n > n0) mma_commit(&bars->empty[sv]);
            if (more) mma_commit(&bars->empty[sk]);
            if (n + 1 == n1) mma_commit(&bars->q_empty);
          }
          __syncwarp();
          if (more) {                      // V of block n
            sv = at.slot;
            ok = wait(&bars->full[sv], at.phase);
            at.next();
            const int live = len - it.block(n) * kBlock;
            if (ok && (pend[0] || pend[1]) && live < kBlock && (PAGED || a.lengths != nullptr)) {
              // value rows behind the length: zeros (both warps may write them)
              uint8_t* v = smem + L::kRing + sv * L::kTile;
              for (int r = live * 8 + lane; r < kBlock * 8; r += 32)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  *reinterpret_cast<uint4*>(v + c * kAtom + r * 16) = make_uint4(0, 0, 0, 0);
              fence_async_smem();
              __syncwarp();
            }
          }
        }
        ++nq;
        give_back();
      }
      if (elect_one()) {   // the products issued so far end before TMEM is freed
        mma_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, a.err);
      }
      __syncwarp();
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 32 * kKWarp) {   // every copy has landed before the CTA exits, after a wait that gave up too
    const RingDrain ring{SL, bars->loads[0], bars->loads[1]};
    for (uint32_t i = ring.begin(); i < ring.end(); ++i)
      if (ring.open(i)) mbar_wait(&bars->full[i % SL], (i / SL) & 1, a.err);
  }
  if (warp == kMmaWarp) {
    fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- launches ------------------------------------------------------------------

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

int slot_rows(int64_t rows, int g) {
  const int64_t most = (128 / g) * g;
  return (int)(rows * g < most ? rows * g : most);
}

template <int D>
cudaError_t window(const AttendArgs& a, cudaStream_t s) {
  Shape sh = {};
  sh.pair_heads = a.g % 2 == 0;
  const int t = (a.N + kBlock - 1) / kBlock;
  sh.tiles = sh.pair_heads ? t : (t + 1) / 2;
  sh.scale_log2 = a.scale * 1.4426950408889634f;
  const int64_t items = (int64_t)a.B * (sh.pair_heads ? a.H / 2 : a.H) * sh.tiles;
  Maps maps;
  cudaError_t e;
  const uint32_t box[4] = {64, kBlock, 1, 1};
  if ((e = make_map_4d(&maps.q, a.q, D, a.N, a.H, a.B, a.sq.n, a.sq.h, a.sq.b, box)) != cudaSuccess ||
      (e = make_map_4d(&maps.k, a.k, D, a.N, a.Hkv, a.B, a.sk.n, a.sk.h, a.sk.b, box)) != cudaSuccess ||
      (e = make_map_4d(&maps.v, a.v, D, a.N, a.Hkv, a.B, a.sv.n, a.sv.h, a.sv.b, box)) != cudaSuccess)
    return e;
  e = cudaFuncSetAttribute(attend_fwd_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)Lay<D>::kDyn);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  attend_fwd_kernel<D, false><<<(int)(items < sms ? items : sms), kThreads, Lay<D>::kDyn, s>>>(
      maps, a, sh, items);
  return cudaGetLastError();
}

template <int D>
cudaError_t pages(const AttendArgs& a, cudaStream_t s) {
  Shape sh = {};
  sh.tt = 128 / a.g;
  sh.sub = a.page_size & -a.page_size;
  if (sh.sub > kBlock) sh.sub = kBlock;
  sh.scale_log2 = a.scale * 1.4426950408889634f;
  sh.slot_rows = slot_rows(a.rows, a.g);
  Maps maps;
  cudaError_t e;
  const uint32_t qbox[4] = {64, (uint32_t)a.g, (uint32_t)sh.tt, 1};
  const uint32_t box[4] = {64, (uint32_t)sh.sub, 1, 1};
  if ((e = make_map_4d(&maps.q, a.q, D, a.H, a.rows, 1, a.sq.h, a.sq.n, a.sq.b, qbox)) != cudaSuccess ||
      (e = make_map_4d(&maps.k, a.k, D, a.page_size, a.Hkv, a.pages, a.sk.n, a.sk.h, a.sk.b, box)) !=
          cudaSuccess ||
      (e = make_map_4d(&maps.v, a.v, D, a.page_size, a.Hkv, a.pages, a.sv.n, a.sv.h, a.sv.b, box)) !=
          cudaSuccess)
    return e;
  e = cudaFuncSetAttribute(attend_fwd_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)Lay<D>::kDyn);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(), ctas = sms < kMaxCtas ? sms : kMaxCtas;
  attend_fwd_kernel<D, true><<<ctas, kThreads, Lay<D>::kDyn, s>>>(maps, a, sh, 0);
  return cudaGetLastError();
}

}  // namespace

bool attend_tc_supported(int d, bool bf16) { return bf16 && (d == 64 || d == 128); }

size_t paged_scratch_bytes(int d, int64_t rows, int g) {
  return (size_t)kMaxCtas * 4 * slot_rows(rows, g) * (d + 2) * sizeof(float);
}

cudaError_t launch_window_fwd_tc(const AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? window<64>(a, s) : window<128>(a, s);
}
cudaError_t launch_paged_tc(const AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? pages<64>(a, s) : pages<128>(a, s);
}

}  // namespace elsaa
