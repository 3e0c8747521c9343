// Backward of the window attention on the tensor cores (bf16, d = 64 or 128).
//
//   P = exp(scale q k - lse),  dS = P (dy v - delta),  delta = y . dy,
//   dv = P^T dy,  dk = scale dS^T q,  dq = scale dS k.
//
// Two persistent warp-specialized tcgen05 kernels, so that every output element
// has one writer and no atomics:
//   window_dkv_kernel  key tiles: S^T = K Q^T and dP^T = V dY^T, keys in the TMEM
//                      lanes; P^T and dS^T go back over them as bf16 and are the A
//                      operands of dV += P^T dY, dK += dS^T Q.  All query heads of
//                      the group walk past a key tile, so grouped heads add up in
//                      TMEM.  4 products a block.
//   window_dq_kernel   query tiles: S = Q K^T, dP = dY V^T, dQ += dS K.  3 products.
// A single kernel would save two products of seven and one exponential a block,
// but would add 64 KB of fp32 dQ a block to memory in an order that changes.
//
// window_dkv_kernel's work is one list of (key tile, query head, query block) units
// cut into equal runs, one per CTA: a tile of sinks is seen by every query behind
// it, an order of magnitude more than the others.  A tile cut between CTAs leaves
// fp32 partials, and the last CTA to get there adds them up, in the CTAs' order
// whichever it is (a counter a warp: a row's partials come from the same warp of
// every CTA).
//
// Elementwise work of a block: 256 threads, each one lane and 64 of the 128
// columns.  The products of one block run under the elementwise work of the
// previous one: dV and the next S under dS, dK and the next dP under P.
//
// P and dS are rounded to bf16, the other operand's type, before the gradients'
// products (half a step each, random; the sums are fp32): dq, dk and dv are off by
// 0.0024 of their norm against 64 bits (their own rounding alone: 0.0017).
//
// Bound: a block's floor at d = 128 is 2048 (dkv) and 1536 (dq) cycles of products,
// at d = 64 half of that, against 1024 of exponentials and about as many of other
// instructions.  At d = 64 nothing is full (issue slots 38 and 41 % active, the tensor
// pipe 33 %): what counts is the latency of the chain of a block (S read from TMEM,
// exponentials, P written, dP read, dS written), with one block's worth in flight.
// stats_kernel (rows of y and dy once) is bound by HBM.
// Measured: 8192 tokens, 32 query and 8 key heads, window 4096: d = 128 1306 us (790
// TFLOP/s by the formulas' five products), d = 64 927 us; text-32k (2 x 12 heads of
// d = 64, 32768 tokens) at window 1024: dkv 685 us, dq 512, stats 49.
//
// Every wait is bounded; one that gives up records ERR_TIMEOUT, every role leaves
// its loop, and copies and products in flight end before TMEM is freed.
#include <math.h>

#include "attend_tc.cuh"
#include "internal.h"

namespace elsaa {
namespace {

using namespace tc;

constexpr int kThreads = 384;            // 8 elementwise warps, TMA, two MMA, items
constexpr int kTmaWarp = 8, kMmaWarp = 9, kItemWarp = 11;
// registers a thread: 384 x 168 at launch = 256 x 216 + 128 x 72
constexpr int kWorkRegs = 216, kOtherRegs = 72;
constexpr uint32_t kTmemCols = 512;
constexpr int kItems = 3;
constexpr int kMinUnits = 2;

template <int D>
struct Lay {
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr uint32_t kFix = 0;                          // K, V (dkv) or Q, dY (dq)
  static constexpr uint32_t kRing = 2 * kTile;
  // dkv: query blocks' statistics, each in a ring of its own.  They are written with
  // the loads of Q and dY, whose ring slots came free with the dV or dK of an earlier
  // block: with 5 slots Q of block t + 3 waits for dV of t (-lse of t has been read)
  // and dY of t + 2 for dK of t (-delta too); with 8, Q of t + 4 for dK of t and dY
  // of t + 5 for dV of t + 1.
  static constexpr int kNl = D == 128 ? 3 : 4, kNd = D == 128 ? 2 : 5;
  static constexpr uint32_t kStatL = kRing + kSlots * kTile;   // [kNl][128]
  static constexpr uint32_t kStatD = kStatL + kNl * 512;       // [kNd][128]
  static constexpr uint32_t kBars = kStatD + kNd * 512;
  static constexpr uint32_t kDyn = kBars + 512;
};
static_assert(Lay<128>::kDyn <= 232448, "shared memory at d = 128");

struct Maps {
  CUtensorMap q, k, v, dy;
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t fix_full[2], fix_empty[2];    // dkv: K, V; dq: Q, dY
  uint64_t s_full[2], s_read[2], dp_full, p_full, ds_full, acc_full;
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t drain;
  uint32_t tmem;
  int32_t cut[5];
  int64_t per;
  int32_t items[kItems][12];
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// Row statistics in the workspace, rows padded to whole blocks per head:
// -log2e lse and -delta; (-inf, 0) for rows without keys, which makes P zero.
struct Stats {
  float *nl, *nd;
  int64_t pad;   // rows of a head
};

ELSAA_DEV int length_of(const AttendArgs& a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
}

// ---- row statistics (and the zeros of empty tiles) ------------------------------------------------------------

// -delta of row x from sum_j p_j dy . v_j where it sees at most kFewKeys keys, by its lane
// group; the whole warp takes as many turns as one of its rows needs.  c: the lane's first
// column.
template <int D>
ELSAA_DEV void few_delta(const AttendArgs& a, const Stats& st, int x, int rows, int c) {
  constexpr int LANES = D / 8;
  const int pad = (int)st.pad, bh = x / pad, n = x - bh * pad, b = bh / a.H, h = bh - b * a.H;
  const bool mine = x < rows && n < length_of(a, b) && seen_keys(n, a.window, a.sinks) <= kFewKeys;
  const int few = mine ? seen_keys(n, a.window, a.sinks) : 0;
  const int turns = __reduce_max_sync(0xffffffffu, few);
  if (turns == 0) return;
  const auto at = [&](const void* base, const Strides& s, int head, int64_t j, bool in) {
    return in ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + b * s.b +
                                                head * s.h + j * s.n + c)
              : make_uint4(0, 0, 0, 0);
  };
  const auto dot = [](const uint4& y, const uint4& z) {
    const uint32_t ya[4] = {y.x, y.y, y.z, y.w}, za[4] = {z.x, z.y, z.z, z.w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s += __uint_as_float(ya[e] << 16) * __uint_as_float(za[e] << 16) +
           __uint_as_float(ya[e] & 0xffff0000u) * __uint_as_float(za[e] & 0xffff0000u);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  const uint4 q = at(a.q, a.sq, h, n, mine), g = at(a.dy, a.sdy, h, n, mine);
  const float nl = mine ? a.lse[(int64_t)bh * a.N + n] * -1.4426950408889634f : 0.f;
  float sum = 0.f;
  for (int t = 0; t < turns; t += 4) {
    uint4 k[4], v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = t + e < few;
      const int64_t j = in ? seen_key(t + e, n, a.window, a.sinks) : 0;
      k[e] = at(a.k, a.sk, h / a.g, j, in);
      v[e] = at(a.v, a.sv, h / a.g, j, in);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = dot(q, k[e]), r = dot(g, v[e]);
      if (t + e < few) sum += ex2(s * (a.scale * 1.4426950408889634f) + nl) * r;
    }
  }
  if (mine && c == 0) st.nd[x] = -sum;
}

// Four rows a lane group, all their loads in flight before the first sum.
constexpr int kStatRows = 4;
template <int D>
__global__ void __launch_bounds__(256) stats_kernel(const AttendArgs a, const Stats st) {
  constexpr int LANES = D / 8, ROWS = 256 / LANES;
  const int c = (threadIdx.x % LANES) * 8;
  const int pad = (int)st.pad, rows = a.B * a.H * pad;   // (below 2^31)
  // (a block's rows are one head's; the first blocks of all heads, which may hold rows that
  // see few keys, go first)
  static_assert(kBlock % (ROWS * kStatRows) == 0, "blocks within a head");
  const int heads = a.B * a.H, n0 = (int)blockIdx.x / heads * (ROWS * kStatRows);
  const int x0 = (int)blockIdx.x % heads * pad + n0 + threadIdx.x / LANES;
  uint4 u[kStatRows], w[kStatRows];
  float nl[kStatRows];
  bool empty[kStatRows];
#pragma unroll
  for (int i = 0; i < kStatRows; ++i) {
    const int x = x0 + i * ROWS;
    u[i] = w[i] = make_uint4(0, 0, 0, 0);
    nl[i] = INFINITY;
    empty[i] = false;
    if (x < rows) {
      const int bh = x / pad, n = x - bh * pad, b = bh / a.H, h = bh - b * a.H, len = length_of(a, b);
      if (n < len) {
        u[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.y) + b * a.sy.b +
                                               h * a.sy.h + n * a.sy.n + c);
        w[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dy) + b * a.sdy.b +
                                               h * a.sdy.h + n * a.sdy.n + c);
        nl[i] = a.lse[(int64_t)bh * a.N + n];
      }
      empty[i] = n < a.N && n / kBlock * kBlock >= len;
    }
  }
#pragma unroll
  for (int i = 0; i < kStatRows; ++i) {
    const int x = x0 + i * ROWS;
    const uint32_t ua[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, wa[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s += __uint_as_float(ua[e] << 16) * __uint_as_float(wa[e] << 16) +
           __uint_as_float(ua[e] & 0xffff0000u) * __uint_as_float(wa[e] & 0xffff0000u);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (x < rows && c == 0) {
      // (a row without keys has lse -inf; like a row behind the length it gets P = 0)
      st.nl[x] = fabsf(nl[i]) == INFINITY ? -INFINITY : -nl[i] * 1.4426950408889634f;
      st.nd[x] = -s;
    }
    if (empty[i]) {   // a tile behind the length is no item of the kernels below: its zeros
      const int bh = x / pad, n = x - bh * pad, b = bh / a.H, h = bh - b * a.H;
      const uint4 z = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dq) + b * a.sdq.b + h * a.sdq.h +
                                n * a.sdq.n + c) = z;
      if (h % a.g == 0) {
        const int hk = h / a.g;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dk) + b * a.sdk.b + hk * a.sdk.h +
                                  n * a.sdk.n + c) = z;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dv) + b * a.sdv.b + hk * a.sdv.h +
                                  n * a.sdv.n + c) = z;
      }
    }
  }
  // rows that see few keys, read anew (in the loop above: text-32k 72 us); later rows of a
  // head see no fewer
  if (seen_keys(n0, a.window, a.sinks) > kFewKeys) return;
#pragma unroll 1
  for (int i = 0; i < kStatRows; ++i) few_delta<D>(a, st, x0 + i * ROWS, rows, c);
}

// ---- shared pieces ---------------------------------------------------------------

// 16-byte-aligned bytes (a multiple of 16) into shared memory.
ELSAA_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Rows live .. 127 of a tile in shared memory become zeros (rows behind a length
// may hold anything, and meet zero factors in a product); one warp.
template <int D>
ELSAA_DEV void zero_rows(uint8_t* tile, int live) {
  for (int r = live * 8 + (threadIdx.x & 31); r < kBlock * 8; r += 32)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<uint4*>(tile + c * kAtom + r * 16) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  __syncwarp();
}

// D[128 x D] (+)= A X, A the bf16 tile that both halves of the elementwise threads
// left in TMEM (columns 0..63 packed from `a`, 64..127 from a + 64), X [128, D] in
// shared memory.
template <int D>
ELSAA_DEV void mma_packed(uint32_t d_tmem, uint32_t a, uint32_t xd, uint32_t accumulate) {
  constexpr uint32_t id = idesc_bf16(128, D, false, true);
#pragma unroll
  for (int x = 0; x < kBlock; x += 16)
    mma_ts(d_tmem, a + (uint32_t)((x >> 6) * 64 + ((x & 63) >> 1)), xd + (uint32_t)x * 8, id,
           x > 0 ? 1u : accumulate);
}

// 64 fp32 values to 32 packed columns.
ELSAA_DEV void store_packed(uint32_t taddr, const float* v) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[32 * c + 2 * e], v[32 * c + 2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    tmem_st16(taddr + 16 * c, w);
  }
}

// The item ring between the items warp and the others.
struct ItemRing {
  Bars* bars;
  uint32_t* err;
  uint32_t taken = 0;
  // the next item, or null behind the last one; ok turns false where a wait gave up
  ELSAA_DEV const int32_t* take(bool& ok) {
    if (!ok) return nullptr;
    const uint32_t i = taken % kItems;
    ok = warp_wait(&bars->item_full[i], (taken / kItems) & 1, err);
    const int32_t* it = bars->items[i];
    if (!ok || it[0] < 0) return nullptr;
    ++taken;
    return it;
  }
  ELSAA_DEV void give_back(const int32_t* it) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
      mbar_arrive(&bars->item_empty[(it - &bars->items[0][0]) / 12]);
  }
};

ELSAA_DEV void init_bars(Bars* b, int acc) {
  for (int i = 0; i < 8; ++i) {
    mbar_init(&b->full[i], 1);
    mbar_init(&b->empty[i], 2);            // both MMA warps
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&b->fix_full[i], 1);
    mbar_init(&b->fix_empty[i], 1);
    mbar_init(&b->s_full[i], 1);
    mbar_init(&b->s_read[i], 8);   // elementwise warps
  }
  mbar_init(&b->dp_full, 1);
  mbar_init(&b->p_full, 8);
  mbar_init(&b->ds_full, 8);
  mbar_init(&b->acc_full, acc);            // MMA warps with an accumulator
  for (int i = 0; i < kItems; ++i) {
    mbar_init(&b->item_full[i], 1);
    mbar_init(&b->item_empty[i], 11);   // eight elementwise warps, TMA, two MMA
  }
  mbar_init(&b->drain, 2);
  fence_mbar_init();
}

// ---- dk, dv ----------------------------------------------------------------------

// Fields of a key tile's item; [0] < 0: no more items.
enum { kB, kHk, kLen, kKt, kNb, kNq, kN0, kN1, kOrder, kCta0, kCta1, kSlot0 };

// Query blocks (of one head) that see key tile kt.
ELSAA_DEV int query_blocks(const AttendArgs& a, int len, int kt) {
  const int j0 = kt * kBlock;
  if (j0 >= len) return 0;
  const int64_t reach = j0 < a.sinks ? len : (int64_t)j0 + kBlock - 1 + a.window;
  return ((int)(reach < len ? reach : len) - 1) / kBlock - kt + 1;
}

// Units of one key head of a sequence, by one warp.
ELSAA_DEV int64_t head_units(const AttendArgs& a, int len) {
  int64_t u = 0;
  for (int kt = threadIdx.x & 31; kt * kBlock < len; kt += 32) u += query_blocks(a, len, kt);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  return u * a.g;
}
ELSAA_DEV int64_t all_units(const AttendArgs& a) {
  if (!a.lengths) return head_units(a, a.N) * a.Hkv * a.B;
  int64_t u = 0;
  for (int b = 0; b < a.B; ++b) u += head_units(a, length_of(a, b)) * a.Hkv;
  return u;
}
ELSAA_DEV int64_t run_length(int64_t total, int ctas) {
  const int64_t per = (total + ctas - 1) / ctas;
  return per > kMinUnits ? per : kMinUnits;
}

struct Cut {
  int b, hk, kt, off;
};

// The key tile and block of unit w (0 <= w < all units), by one warp.
ELSAA_DEV Cut find_unit(const AttendArgs& a, int64_t w) {
  const int lane = threadIdx.x & 31;
  Cut c{0, 0, 0, 0};
  int64_t per_head = 0;
  if (!a.lengths) {
    per_head = head_units(a, a.N);
    c.b = (int)(w / (per_head * a.Hkv));
    w -= c.b * per_head * a.Hkv;
  } else {
    for (; c.b < a.B; ++c.b) {
      per_head = head_units(a, length_of(a, c.b));
      if (w < per_head * a.Hkv) break;
      w -= per_head * a.Hkv;
    }
    if (c.b == a.B) return c;   // (w was no unit)
  }
  c.hk = (int)(w / per_head);
  w -= c.hk * per_head;
  const int len = length_of(a, c.b);
  for (int t0 = 0; t0 * kBlock < len; t0 += 32) {
    const int64_t mine = (int64_t)query_blocks(a, len, t0 + lane) * a.g;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w < upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      c.kt = t0 + l;
      c.off = (int)(w - __shfl_sync(0xffffffffu, upto - mine, l));
      return c;
    }
    w -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return c;
}

// The partials of a key tile cut between CTAs: [slot][dv, dk][128][D], slot = 2 cta +
// (not the run's first item).
ELSAA_DEV float* partial(const AttendArgs& a, int d, int slot, int which, int row) {
  return reinterpret_cast<float*>(a.scratch) + (((int64_t)slot * 2 + which) * kBlock + row) * d;
}

// 32 rows of a cut tile's dV (which = 0) or dK (1) from the partials of all its CTAs,
// in their order; lanes over the columns, eight rows at a time.
template <int D>
ELSAA_DEV void merge_rows(const AttendArgs& a, const int32_t* it, int which, int warp_row) {
  constexpr int V = D / 32, R = 8;   // values of a lane, rows at a time
  const int lane = threadIdx.x & 31, cta0 = it[kCta0], cta1 = it[kCta1], slot0 = it[kSlot0];
  const int j0 = it[kKt] * kBlock, len = it[kLen];
  const float f = which ? a.scale : 1.f;
  const Strides so = which ? a.sdk : a.sdv;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(which ? a.dk : a.dv) + it[kB] * so.b +
                       it[kHk] * so.h + lane * V;
  for (int x0 = warp_row; x0 < warp_row + 32; x0 += R) {
    float o[R][V];
#pragma unroll
    for (int x = 0; x < R; ++x)
#pragma unroll
      for (int e = 0; e < V; ++e) o[x][e] = 0.f;
#pragma unroll 2
    for (int i = cta0; i <= cta1; ++i) {
      const float* p = partial(a, D, i * 2 + (i == cta0 ? slot0 : 0), which, x0) + lane * V;
#pragma unroll
      for (int x = 0; x < R; ++x) {
        if (V == 4) {
          const float4 u = __ldcg(reinterpret_cast<const float4*>(p + x * D));
          o[x][0] += u.x, o[x][1] += u.y, o[x][2 % V] += u.z, o[x][3 % V] += u.w;
        } else {
          const float2 u = __ldcg(reinterpret_cast<const float2*>(p + x * D));
          o[x][0] += u.x, o[x][1] += u.y;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const int j = j0 + x0 + x;
      if (j >= a.N) break;
#pragma unroll
      for (int e = 0; e < V; e += 2)   // rows behind the length: zeros
        *reinterpret_cast<__nv_bfloat162*>(out + (int64_t)j * so.n + e) =
            __floats2bfloat162_rn(j < len ? o[x][e] * f : 0.f, j < len ? o[x][(e + 1) % V] * f : 0.f);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dkv_kernel(const __grid_constant__ Maps maps, const AttendArgs a, const Stats stats) {
  using L = Lay<D>;
  constexpr int SL = L::kSlots;
  constexpr uint32_t kTS = 0, kTP = 128, kTV = 256, kTK = 256 + D;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((sbase & 1023u) != 0) {
    if (tid == 0) raise_error(a.err, ERR_CHECK);
    return;
  }
  if (tid == 0) init_bars(bars, 2);
  if (warp == 0) {   // this CTA's run of units
    const int64_t total = all_units(a), per = run_length(total, gridDim.x), w0 = per * blockIdx.x;
    Cut c{0, 0, 0, 0};
    int units = 0;
    if (w0 < total) {
      c = find_unit(a, w0);
      units = (int)(per < total - w0 ? per : total - w0);
    }
    if (lane == 0) {
      bars->cut[0] = c.b, bars->cut[1] = c.hk, bars->cut[2] = c.kt, bars->cut[3] = c.off;
      bars->cut[4] = units;
      bars->per = per;
    }
  }
  __syncthreads();
  if (bars->cut[4] == 0) return;
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;
  bool ok = true;
  ItemRing ring{bars, a.err};
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, a.err);
  };

  if (warp < kTmaWarp) {
    // ------------------------------------------------------------------ elementwise
    regs_up<kWorkRegs>();
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + kTS + 64 * half + lane_off, tP = tmem + kTP + 64 * half + lane_off;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    uint32_t t = 0, ni = 0;
    while (const int32_t* it = ring.take(ok)) {
      const int kt = it[kKt], nq = it[kNq], j0 = kt * kBlock, j = j0 + row;
      int q = it[kN0] % nq;   // query block of the head, from the key tile's on
      for (int left = it[kN1] - it[kN0]; left > 0; --left, ++t) {
        const int i0 = j0 + q * kBlock;
        if (++q == nq) q = 0;
        // (S^T is there: its Q has landed before it, and -lse with Q)
        ok = wait(&bars->s_full[0], t & 1);
        if (!ok) break;
        fence_after();
        const float* nl = reinterpret_cast<const float*>(smem + L::kStatL) + (t % L::kNl) * 128 + 64 * half;
        const float* nd = reinterpret_cast<const float*>(smem + L::kStatD) + (t % L::kNd) * 128 + 64 * half;
        float p[64];
        tmem_ld32(tS, p);
        tmem_ld32(tS + 32, p + 32);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 l = *reinterpret_cast<const float4*>(nl + e);
          fma2(p[e], p[e + 1], scale_log2, scale_log2, l.x, l.y);
          fma2(p[e + 2], p[e + 3], scale_log2, scale_log2, l.z, l.w);
          exp2_pair<D == 64>(e >> 1, p[e], p[e + 1]);
          exp2_pair<D == 64>((e >> 1) + 1, p[e + 2], p[e + 3]);
        }
        if (i0 < j0 + kBlock - 1 ||
            (j0 + kBlock > a.sinks && (int64_t)i0 + kBlock - 1 >= (int64_t)j0 + a.window)) {
          const int lo = j - i0 - 64 * half;   // queries from the key on
          const int hi = j < a.sinks ? 63
                                     : (int)min((int64_t)j + a.window - 1 - i0 - 64 * half, (int64_t)63);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t see = upto_bits(hi - 32 * c) & ~upto_bits(lo - 1 - 32 * c);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) p[32 * c + e] = 0.f;
          }
        }
        store_packed(tS, p);   // P^T over S^T
        tmem_st_wait();
        fence_before();
        warp_arrive(&bars->p_full);
        ok = wait(&bars->dp_full, t & 1);   // (and -delta with dY)
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float dp[32];
          tmem_ld32(tP + 32 * c, dp);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 x = *reinterpret_cast<const float4*>(nd + 32 * c + e);
            add2(dp[e], dp[e + 1], x.x, x.y);
            add2(dp[e + 2], dp[e + 3], x.z, x.w);
            mul2(p[32 * c + e], p[32 * c + e + 1], dp[e], dp[e + 1]);
            mul2(p[32 * c + e + 2], p[32 * c + e + 3], dp[e + 2], dp[e + 3]);
          }
        }
        store_packed(tP, p);   // dS^T over dP^T
        tmem_st_wait();
        fence_before();
        warp_arrive(&bars->ds_full);
      }
      if (!ok) break;
      ok = wait(&bars->acc_full, ni & 1);
      if (!ok) break;
      ++ni;
      fence_after();
      // dV by the first half of the threads, dK by the second
      const bool whole = it[kN0] == 0 && it[kN1] == it[kNb];
      const uint32_t acc = tmem + (half ? kTK : kTV) + lane_off;
      const float f = half ? a.scale : 1.f;
      float* prow = partial(a, D, (int)blockIdx.x * 2 + (it[kOrder] > 0 ? 1 : 0), half, row);
      const Strides so = half ? a.sdk : a.sdv;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(half ? a.dk : a.dv) + it[kB] * so.b +
                            it[kHk] * so.h + (int64_t)j * so.n;
      const bool live = j < it[kLen];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        tmem_ld32(acc + 32 * c, v);
        tmem_ld_wait();
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = live ? v[e] * f : 0.f;
          if (j < a.N) store32(orow + 32 * c, v);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(prow + 32 * c + 4 * q) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
      if (!whole) {
        // the last of the tile's CTAs to come here with this warp's rows adds them up
        uint32_t* counter = a.counters + it[kCta0] * 8 + warp;
        uint32_t before = 0;
        __threadfence();
        __syncwarp();
        if (lane == 0) before = atomicAdd(counter, 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == (uint32_t)(it[kCta1] - it[kCta0])) {
          __threadfence();
          merge_rows<D>(a, it, half, 32 * (warp & 3));
          if (lane == 0) *counter = 0;
        }
      }
      fence_before();
      ring.give_back(it);
    }
  } else {
    regs_down<kOtherRegs>();
    if (warp == kTmaWarp) {
      // ---------------------------------------------------------------- copies
      uint32_t nr = 0, t = 0, nf[2] = {0, 0};
      auto load = [&](const CUtensorMap* map, uint32_t dst, int n, int h, int b, uint64_t* bar) {
        if (lane < D / 64) tma_load_4d(dst + lane * kAtom, map, 64 * lane, n, h, b, bar);
        __syncwarp();
      };
      // the item's fixed tile x (0: K, 1: V)
      auto load_fix = [&](const int32_t* it, int x) {
        if (nf[x] > 0) ok = ok && wait(&bars->fix_empty[x], (nf[x] - 1) & 1);
        if (!ok) return;
        ++nf[x];
        if (lane == 0) mbar_arrive_expect_tx(&bars->fix_full[x], L::kTile);
        __syncwarp();
        load(x ? &maps.v : &maps.k, sbase + L::kFix + x * L::kTile, it[kKt] * kBlock, it[kHk], it[kB],
             &bars->fix_full[x]);
      };
      // Q and -lse (x = 0) or dY and -delta (1) of block n
      auto load_block = [&](const int32_t* it, int n, int x) {
        const uint32_t s = nr % SL;
        if (nr >= SL) ok = ok && wait(&bars->empty[s], (nr / SL - 1) & 1);
        if (!ok) return;
        const int nq = it[kNq], h = it[kHk] * a.g + n / nq, qb = it[kKt] + n % nq;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->full[s], L::kTile + 512);
          const int64_t at = ((int64_t)it[kB] * a.H + h) * stats.pad + (int64_t)qb * kBlock;
          if (x)
            bulk_load(sbase + L::kStatD + (t % L::kNd) * 512, stats.nd + at, 512, &bars->full[s]);
          else
            bulk_load(sbase + L::kStatL + (t % L::kNl) * 512, stats.nl + at, 512, &bars->full[s]);
        }
        __syncwarp();
        load(x ? &maps.dy : &maps.q, sbase + L::kRing + s * L::kTile, qb * kBlock, h, it[kB],
             &bars->full[s]);
        ++nr;
        if (x) ++t;
      };
      while (const int32_t* it = ring.take(ok)) {
        const int n0 = it[kN0], n1 = it[kN1];
        load_fix(it, 0);
        load_block(it, n0, 0);
        load_fix(it, 1);
        load_block(it, n0, 1);
        for (int n = n0 + 1; n < n1 && ok; ++n) {
          load_block(it, n, 0);
          load_block(it, n, 1);
        }
        ring.give_back(it);
      }
      if (lane == 0) {   // every copy has landed before the CTA may exit
        for (uint32_t i = nr > SL ? nr - SL : 0; i < nr; ++i)
          mbar_wait(&bars->full[i % SL], (i / SL) & 1, a.err);
        for (int x = 0; x < 2; ++x)
          if (nf[x] > 0) mbar_wait(&bars->fix_full[x], (nf[x] - 1) & 1, a.err);
      }
      __syncwarp();
    } else if (warp < kItemWarp) {
      // ---------------------------------------------------------------- products
      // Warp x = 0: S^T (from Q) and dV (from dY); x = 1: dP^T (from dY) and dK (from
      // Q).  One warp's waits and bookkeeping run under the other's products.
      const int x = warp - kMmaWarp;
      const uint32_t tm = uniform(tmem);
      const uint32_t fix_d = uniform(row_desc(sbase + L::kFix + x * L::kTile));
      const uint32_t row_d = row_desc(sbase + L::kRing), col_d = col_desc(sbase + L::kRing);
      constexpr uint32_t kStep = L::kTile >> 4;   // a slot further, in descriptor units
      const uint32_t t_new = uniform(tm + (x ? kTP : kTS)), t_acc = uniform(tm + (x ? kTK : kTV));
      uint64_t* const gate = x ? &bars->ds_full : &bars->p_full;
      uint64_t* const done = x ? &bars->dp_full : &bars->s_full[0];
      // the block whose S^T or dP^T comes next
      const int32_t* it = nullptr;
      int left = 0, q = 0, nq = 1, j0 = 0, len = 0, live = 0;   // blocks of its item from it on
      bool first = false;
      uint32_t items = 0;
      auto open = [&]() {   // the next item's first block
        it = ring.take(ok);
        if (it == nullptr) return;
        left = it[kN1] - it[kN0];
        nq = it[kNq];
        q = it[kN0] % nq;
        j0 = it[kKt] * kBlock;
        len = it[kLen];
        first = true;
        ++items;
      };
      // a tile is in shared memory, zeros behind the length
      auto ready = [&](const RingPos<SL>& at, int rows) {
        ok = ok && wait(&bars->full[at.slot], at.phase);
        if (ok && a.lengths && rows < kBlock) zero_rows<D>(smem + L::kRing + at.slot * L::kTile, rows);
      };
      RingPos<SL> own, other;   // Q, dY (x = 0) or dY, Q (1)
      if (x) own.next(); else other.next();
      // the next block's operand, awaited before the elementwise work
      auto prepare = [&]() {
        live = len - j0 - q * kBlock;
        ready(own, live);
        if (ok && first) ok = wait(&bars->fix_full[x], (items - 1) & 1);
      };
      auto issue = [&](uint32_t d) {   // its product (the elected lane)
        mma_tiles<D>(t_new, fix_d, d);
        mma_commit(done);
        mma_commit(&bars->empty[own.slot]);
        if (left == 1) mma_commit(&bars->fix_empty[x]);
      };
      auto advance = [&]() {
        own.next(), own.next();
        if (++q == nq) q = 0;
        --left;
        first = false;
      };
      open();
      if (it != nullptr) {
        prepare();
        const uint32_t d = uniform(row_d + own.slot * kStep);
        fence_after();
        if (ok && elect_one()) issue(d);
        __syncwarp();
        advance();
      }
      uint32_t add = 0;
      for (uint32_t t = 0; it != nullptr && ok; ++t) {   // block t's accumulation and the next product
        const int rows = live;
        const bool end = left == 0;
        if (end) {
          ring.give_back(it);   // (before the next is asked for: its place may be needed)
          open();
        }
        const bool more = it != nullptr;
        if (more) prepare();
        ready(other, rows);
        const uint32_t d = uniform(row_d + own.slot * kStep), od = uniform(col_d + other.slot * kStep);
        const uint32_t acc = uniform(add);
        ok = ok && wait(gate, t & 1);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          mma_packed<D>(t_acc, t_new, od, acc);
          mma_commit(&bars->empty[other.slot]);
          if (end) mma_commit(&bars->acc_full);
          if (more) issue(d);
        }
        __syncwarp();
        add = end ? 0 : 1;
        other.next(), other.next();
        if (more) advance();
      }
      if (elect_one()) {
        mma_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, a.err);
      }
      __syncwarp();
    } else if (lane == 0) {
      // ---------------------------------------------------------------- items
      int b = bars->cut[0], hk = bars->cut[1], kt = bars->cut[2], off = bars->cut[3], left = bars->cut[4];
      int order = 0;
      const int64_t per = bars->per;
      int64_t at = per * blockIdx.x;   // the next unit
      for (uint32_t n = 0;; ++n) {
        if (n >= kItems && !mbar_wait(&bars->item_empty[n % kItems], (n / kItems - 1) & 1, a.err)) break;
        int32_t* it = bars->items[n % kItems];
        int len = b < a.B ? length_of(a, b) : 0;
        while (b < a.B && kt * kBlock >= len) {   // the next key head, the next sequence
          kt = 0;
          if (++hk == a.Hkv) {
            hk = 0;
            ++b;
            len = b < a.B ? length_of(a, b) : 0;
          }
        }
        const bool more = left > 0 && b < a.B;
        if (more) {
          const int nq = query_blocks(a, len, kt), nb = nq * a.g;
          it[kB] = b, it[kHk] = hk, it[kLen] = len, it[kKt] = kt, it[kNb] = nb, it[kNq] = nq;
          it[kN0] = off;
          it[kN1] = min(nb, off + left);
          it[kOrder] = order++;
          if (it[kN1] - off < nb) {   // cut: its CTAs, and its slot in the first one's run
            const int64_t begin = at - off;
            it[kCta0] = (int)(begin / per);
            it[kCta1] = (int)((begin + nb - 1) / per);
            it[kSlot0] = begin == it[kCta0] * per ? 0 : 1;
          }
          at += it[kN1] - off;
          left -= it[kN1] - off;
          off = 0;
          ++kt;
        } else {
          it[kB] = -1;
        }
        mbar_arrive(&bars->item_full[n % kItems]);
        if (!more) break;
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- dq ----------------------------------------------------------------------------

// Fields of a query tile's item.
enum { qB, qH, qLen, qT, qSink, qFirst, qN };
ELSAA_DEV int key_block(const int32_t* it, int n) {
  return n < it[qSink] ? n : it[qFirst] + n - it[qSink];
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dq_kernel(const __grid_constant__ Maps maps, const AttendArgs a, const Stats stats, int tiles) {
  using L = Lay<D>;
  constexpr int SL = L::kSlots;
  constexpr uint32_t kTP = 256, kTQ = 384;   // S at 0 and 128
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((sbase & 1023u) != 0) {
    if (tid == 0) raise_error(a.err, ERR_CHECK);
    return;
  }
  if (tid == 0) init_bars(bars, 1);
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;
  bool ok = true;
  ItemRing ring{bars, a.err};
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, a.err);
  };

  if (warp < kTmaWarp) {
    // ------------------------------------------------------------------ elementwise
    regs_up<kWorkRegs>();
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    uint32_t t = 0, ni = 0;
    while (const int32_t* it = ring.take(ok)) {
      const int r0 = it[qT] * kBlock, r = r0 + row, blocks = it[qN], len = it[qLen];
      const int64_t at = ((int64_t)it[qB] * a.H + it[qH]) * stats.pad + r;
      const float nl = stats.nl[at], nd = stats.nd[at];
      const int p_last = min(len, r0 + kBlock) - 1;
      for (int n = 0; n < blocks; ++n, ++t) {
        const int j0 = key_block(it, n) * kBlock;
        ok = wait(&bars->s_full[t & 1], (t >> 1) & 1);
        if (!ok) break;
        fence_after();
        float p[64];
        const uint32_t tS = tmem + 128 * (t & 1) + 64 * half + lane_off;
        const uint32_t tP = tmem + kTP + 64 * half + lane_off;
        tmem_ld32(tS, p);
        tmem_ld32(tS + 32, p + 32);
        tmem_ld_wait();
        fence_before();
        warp_arrive(&bars->s_read[t & 1]);
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          fma2(p[e], p[e + 1], scale_log2, scale_log2, nl, nl);
          exp2_pair<D == 64>(e >> 1, p[e], p[e + 1]);
        }
        if (j0 + kBlock - 1 > r0 || (int64_t)j0 <= (int64_t)p_last - a.window) {
          const int hi = r - j0 - 64 * half, lo = r - a.window + 1 - j0 - 64 * half;
          const int sk = (int)min((int64_t)a.sinks - j0 - 64 * half, (int64_t)64);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t see =
                upto_bits(hi - 32 * c) & (~upto_bits(lo - 1 - 32 * c) | upto_bits(sk - 1 - 32 * c));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) p[32 * c + e] = 0.f;
          }
        }
        ok = wait(&bars->dp_full, t & 1);
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float dp[32];
          tmem_ld32(tP + 32 * c, dp);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            add2(dp[e], dp[e + 1], nd, nd);
            mul2(p[32 * c + e], p[32 * c + e + 1], dp[e], dp[e + 1]);
          }
        }
        store_packed(tP, p);   // dS over dP
        tmem_st_wait();
        fence_before();
        warp_arrive(&bars->ds_full);
      }
      if (!ok) break;
      ok = wait(&bars->acc_full, ni & 1);
      if (!ok) break;
      ++ni;
      fence_after();
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.dq) + it[qB] * a.sdq.b + it[qH] * a.sdq.h +
                            (int64_t)r * a.sdq.n + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        float v[32];
        tmem_ld32(tmem + kTQ + half * (D / 2) + 32 * c + lane_off, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = r < len ? v[e] * a.scale : 0.f;
        if (r < a.N) store32(orow + 32 * c, v);
      }
      fence_before();
      ring.give_back(it);
    }
  } else {
    regs_down<kOtherRegs>();
    if (warp == kTmaWarp) {
      // ---------------------------------------------------------------- copies
      uint32_t nr = 0, nf[2] = {0, 0};
      auto load = [&](const CUtensorMap* map, uint32_t dst, int n, int h, int b, uint64_t* bar) {
        if (lane < D / 64) tma_load_4d(dst + lane * kAtom, map, 64 * lane, n, h, b, bar);
        __syncwarp();
      };
      auto load_fix = [&](const int32_t* it, int x) {   // Q, dY
        if (nf[x] > 0) ok = ok && wait(&bars->fix_empty[x], (nf[x] - 1) & 1);
        if (!ok) return;
        ++nf[x];
        if (lane == 0) mbar_arrive_expect_tx(&bars->fix_full[x], L::kTile);
        __syncwarp();
        load(x ? &maps.dy : &maps.q, sbase + L::kFix + x * L::kTile, it[qT] * kBlock, it[qH], it[qB],
             &bars->fix_full[x]);
      };
      auto load_block = [&](const int32_t* it, int n, int x) {   // K, V
        const uint32_t s = nr % SL;
        if (nr >= SL) ok = ok && wait(&bars->empty[s], (nr / SL - 1) & 1);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], L::kTile);
        __syncwarp();
        load(x ? &maps.v : &maps.k, sbase + L::kRing + s * L::kTile, key_block(it, n) * kBlock,
             it[qH] / a.g, it[qB], &bars->full[s]);
        ++nr;
      };
      while (const int32_t* it = ring.take(ok)) {
        const int blocks = it[qN];
        load_fix(it, 0);
        load_block(it, 0, 0);
        load_fix(it, 1);
        load_block(it, 0, 1);
        for (int n = 1; n < blocks && ok; ++n) {
          load_block(it, n, 0);
          load_block(it, n, 1);
        }
        ring.give_back(it);
      }
      if (lane == 0) {   // every copy has landed before the CTA may exit
        for (uint32_t i = nr > SL ? nr - SL : 0; i < nr; ++i)
          mbar_wait(&bars->full[i % SL], (i / SL) & 1, a.err);
        for (int x = 0; x < 2; ++x)
          if (nf[x] > 0) mbar_wait(&bars->fix_full[x], (nf[x] - 1) & 1, a.err);
      }
      __syncwarp();
    } else if (warp < kItemWarp) {
      // ---------------------------------------------------------------- products
      // Warp x = 0: S (from K); x = 1: dP (from V) and dQ (from K).
      const int x = warp - kMmaWarp;
      const uint32_t tm = uniform(tmem);
      const uint32_t fix_d = uniform(row_desc(sbase + L::kFix + x * L::kTile));
      const uint32_t row_d = row_desc(sbase + L::kRing), col_d = col_desc(sbase + L::kRing);
      constexpr uint32_t kStep = L::kTile >> 4;   // a slot further, in descriptor units
      const int32_t* it = nullptr;
      int n = 0, blocks = 0, len = 0;
      uint32_t items = 0;
      auto open = [&]() {   // the next item's first block
        it = ring.take(ok);
        if (it == nullptr) return;
        n = 0;
        blocks = it[qN];
        len = it[qLen];
        ++items;
      };
      RingPos<SL> own, other;   // K, V (x = 0) or V, K (1)
      if (x) own.next(); else other.next();
      // the next block's operand is in shared memory, zeros behind the length
      auto prepare = [&]() {
        ok = ok && wait(&bars->full[own.slot], own.phase);
        if (ok && n == 0) ok = wait(&bars->fix_full[x], (items - 1) & 1);
        if (ok && a.lengths) {
          const int live = len - key_block(it, n) * kBlock;
          if (live < kBlock) zero_rows<D>(smem + L::kRing + own.slot * L::kTile, live);
        }
      };
      auto advance = [&]() {
        own.next(), own.next();
        ++n;
      };
      open();
      if (x == 0) {
        for (uint32_t t = 0; it != nullptr && ok; ++t) {   // S of block t
          prepare();
          const uint32_t d = uniform(row_d + own.slot * kStep), td = uniform(tm + 128 * (t & 1));
          if (t >= 2) ok = ok && wait(&bars->s_read[t & 1], ((t >> 1) - 1) & 1);
          if (!ok) break;
          fence_after();
          const bool end = n + 1 == blocks;
          if (elect_one()) {
            mma_tiles<D>(td, fix_d, d);
            mma_commit(&bars->s_full[t & 1]);
            mma_commit(&bars->empty[own.slot]);
            if (end) mma_commit(&bars->fix_empty[0]);
          }
          __syncwarp();
          advance();
          if (end) {
            ring.give_back(it);   // (before the next is asked for: its place may be needed)
            open();
          }
        }
      } else {
        auto issue = [&](uint32_t d) {   // dP (the elected lane; V is this warp's alone)
          mma_tiles<D>(tm + kTP, fix_d, d);
          mma_commit(&bars->dp_full);
          mma_commit(&bars->empty[own.slot]);
          mma_commit(&bars->empty[own.slot]);
          if (n + 1 == blocks) mma_commit(&bars->fix_empty[1]);
        };
        if (it != nullptr) {
          prepare();
          const uint32_t d = uniform(row_d + own.slot * kStep);
          fence_after();
          if (ok && elect_one()) issue(d);
          __syncwarp();
          advance();
        }
        uint32_t add = 0;
        for (uint32_t t = 0; it != nullptr && ok; ++t) {   // dQ of block t and the next dP
          const bool end = n == blocks;
          if (end) {
            ring.give_back(it);   // (before the next is asked for: its place may be needed)
            open();
          }
          const bool more = it != nullptr;
          if (more) prepare();
          const uint32_t d = uniform(row_d + own.slot * kStep), kd = uniform(col_d + other.slot * kStep);
          const uint32_t acc = uniform(add);
          ok = ok && wait(&bars->ds_full, t & 1);
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            mma_packed<D>(tm + kTQ, tm + kTP, kd, acc);
            mma_commit(&bars->empty[other.slot]);
            if (end) mma_commit(&bars->acc_full);
            if (more) issue(d);
          }
          __syncwarp();
          add = end ? 0 : 1;
          other.next(), other.next();
          if (more) advance();
        }
      }
      if (elect_one()) {
        mma_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, a.err);
      }
      __syncwarp();
    } else if (lane == 0) {
      // ---------------------------------------------------------------- items
      const int64_t bh = (int64_t)a.B * a.H, items = bh * tiles;
      int64_t x = blockIdx.x;
      // Every item has blocks: a product warp asks for the next one before it ends the
      // last, and must not wait there for items in between to pass.
      for (uint32_t n = 0;; ++n) {
        if (n >= kItems && !mbar_wait(&bars->item_empty[n % kItems], (n / kItems - 1) & 1, a.err)) break;
        int32_t* it = bars->items[n % kItems];
        it[qB] = -1;
        for (; x < items && it[qB] < 0; x = next_item(a.counters, items)) {
          // the longest (last) tiles first, heads and batches inside
          const int t = tiles - 1 - (int)(x / bh), b = (int)(x % bh / a.H), h = (int)(x % a.H);
          const int len = length_of(a, b);
          const KeyBlocks k = key_blocks(t * kBlock, min(len, (t + 1) * kBlock) - 1, a.window, a.sinks, kBlock);
          if (k.count() == 0) continue;
          it[qH] = h, it[qLen] = len, it[qT] = t;
          it[qSink] = k.sink_blocks, it[qFirst] = k.first, it[qN] = k.count();
          it[qB] = b;
        }
        const bool more = it[qB] >= 0;
        mbar_arrive(&bars->item_full[n % kItems]);
        if (!more) break;
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- launches ------------------------------------------------------------------------

int64_t padded_rows(int N) { return ((int64_t)N + kBlock - 1) / kBlock * kBlock; }

template <int D>
cudaError_t backward(const AttendArgs& args, cudaStream_t s) {
  AttendArgs a = args;
  const int tiles = (a.N + kBlock - 1) / kBlock;
  Stats st;
  st.pad = padded_rows(a.N);
  const int64_t rows = (int64_t)a.B * a.H * st.pad;
  st.nl = a.delta;
  st.nd = st.nl + rows;
  a.scratch = reinterpret_cast<char*>(st.nd + rows);
  Maps maps;
  cudaError_t e;
  const uint32_t box[4] = {64, kBlock, 1, 1};
  if ((e = make_map_4d(&maps.q, a.q, D, a.N, a.H, a.B, a.sq.n, a.sq.h, a.sq.b, box)) != cudaSuccess ||
      (e = make_map_4d(&maps.k, a.k, D, a.N, a.Hkv, a.B, a.sk.n, a.sk.h, a.sk.b, box)) != cudaSuccess ||
      (e = make_map_4d(&maps.v, a.v, D, a.N, a.Hkv, a.B, a.sv.n, a.sv.h, a.sv.b, box)) != cudaSuccess ||
      (e = make_map_4d(&maps.dy, a.dy, D, a.N, a.H, a.B, a.sdy.n, a.sdy.h, a.sdy.b, box)) != cudaSuccess)
    return e;
  constexpr int kRows = 256 / (D / 8) * kStatRows;
  stats_kernel<D><<<(unsigned)((rows + kRows - 1) / kRows), 256, 0, s>>>(a, st);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int smem = (int)Lay<D>::kDyn;
  e = cudaFuncSetAttribute(window_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(window_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  window_dkv_kernel<D><<<ctas, kThreads, smem, s>>>(maps, a, st);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t items = (int64_t)a.B * a.H * tiles;
  window_dq_kernel<D><<<(int)(items < sms ? items : sms), kThreads, smem, s>>>(maps, a, st, tiles);
  return cudaGetLastError();
}

}  // namespace

size_t window_tc_scratch_bytes(int d, int64_t B, int64_t H, int64_t N) {
  return (size_t)(B * H * padded_rows((int)N)) * 2 * sizeof(float) +
         (size_t)kMaxCtas * 2 * 2 * kBlock * d * sizeof(float);
}

cudaError_t launch_window_bwd_tc(const AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? backward<64>(a, s) : backward<128>(a, s);
}

}  // namespace elsaa
