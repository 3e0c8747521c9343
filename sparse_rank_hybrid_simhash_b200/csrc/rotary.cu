// RMS norm of query and key rows and the position rotation, in one pass, with
// the gradients, and their serving form that writes keys and values into the
// pages of a cache.
//
// A row x of d values:  n = x r,  r = 1 / sqrt(mean(x^2) + eps),  u = n w, and
// for each of its rot / 2 pairs (a, b) with the angle of (position, pair)
//   y_a = u_a cos - u_b sin,   y_b = u_b cos + u_a sin.
// Backward: du is the transposed rotation of dy, dw = sum over rows of du n,
// dn = du w, dx = r (dn - n mean(dn n)).
//
// Bound: HBM, each row read once and written once (backward: x and dy read, dx
// written); what keeps the backward from it (136 us against 92 of bytes) is latency: issue
// slots are active 67 % of the time, loads first among the stalls, with two heads' rows
// and their shuffles in flight.  A row is held by a group of d / V
// lanes with one 16-byte load each (V = 8 bf16 or 4 fp32 values), so the sums are
// shuffles within the group; in halves a lane's partner values sit rot / (2 V) lanes
// away and come over as the raw 16 bytes.  A group walks several heads of its token
// and keeps what does not depend on the head in registers, weight and angle folded:
//   y_i = r (x_i A_i + x_o B_i),  A_i = w_i cos,  B_i = -+ w_o sin  (o: i's partner)
// (text-32k queries and keys, 2 x 12 heads of d = 64 over 32768 tokens: 71 us, issue
// active 69 % of the time; backward 135 and the weights' sums 4).  Four heads' rows are
// in flight at a time, the first of them while the angles are fetched (an output may be
// its input, so the compiler must keep a later row's load behind an earlier store: 102 us
// without); in the backward two heads' x and dy.
#include "attend.cuh"
#include "common.cuh"
#include "internal.h"
#include "layer.h"

namespace elsaa {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;       // heads whose rows are in flight
constexpr int kFwdBlocks = 4, kBackBlocks = 3;   // resident blocks an SM
constexpr int kStarts = 2048;   // sequence starts kept in shared memory

template <typename T>
struct Vec {
  static constexpr int V = 16 / sizeof(T);
};

// A lane's 16 bytes of a row as fp32.
template <typename T>
ELSAA_DEV void unpack(const uint4& v, float* x);
template <>
ELSAA_DEV void unpack<float>(const uint4& v, float* x) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
template <>
ELSAA_DEV void unpack<__nv_bfloat16>(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
ELSAA_DEV void store_row(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
ELSAA_DEV void store_row(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the lane group of a row.
template <int LANES>
ELSAA_DEV float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The partner values of a lane's 16 bytes: those of the lane `from` (halves), or the
// neighbours in a pair (interleaved).
template <typename T, bool IL>
ELSAA_DEV void partners(const uint4& raw, int from, const float* x, float* o) {
  constexpr int V = Vec<T>::V;
  if (IL) {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = x[i ^ 1];
  } else {
    const uint4 r = make_uint4(__shfl_sync(0xffffffffu, raw.x, from), __shfl_sync(0xffffffffu, raw.y, from),
                               __shfl_sync(0xffffffffu, raw.z, from), __shfl_sync(0xffffffffu, raw.w, from));
    unpack<T>(r, o);
  }
}
// The lane that holds the partners of this lane's columns (halves).
template <int V>
ELSAA_DEV int partner_lane(int col, int rot) {
  const int lane = threadIdx.x & 31, hop = rot / (2 * V);
  return col >= rot ? lane : col < rot / 2 ? lane + hop : lane - hop;
}

// The rotation of a lane's V values at a table row, u_i = x_i a_i + x_o b_i; columns
// past the rotated part: (1, 0).
template <int V, bool IL>
struct Turn {
  float a[V], b[V];
  ELSAA_DEV Turn(const float* row, int col, int rot) {
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 1.f, b[i] = 0.f;
    if (col >= rot) return;
    const int first = IL ? col / 2 : (col < rot / 2 ? col : col - rot / 2);
    constexpr int C = IL ? V / 2 : V;   // pairs of these columns
#pragma unroll
    for (int i = 0; i < C; i += 2) {
      const float4 t = *reinterpret_cast<const float4*>(row + 2 * (first + i));
      const float c[2] = {t.x, t.z}, sn[2] = {t.y, t.w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (IL) {
          a[2 * (i + e)] = a[2 * (i + e) + 1] = c[e];
          b[2 * (i + e)] = -sn[e];
          b[2 * (i + e) + 1] = sn[e];
        } else {
          a[i + e] = c[e];
          b[i + e] = col < rot / 2 ? -sn[e] : sn[e];
        }
      }
    }
  }
  // the weights of the values (w) and of their partners folded in
  ELSAA_DEV void weigh(const float* w, int col, int rot) {
    if (w == nullptr) return;
    const int other = col >= rot ? col : col < rot / 2 ? col + rot / 2 : col - rot / 2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      a[i] *= __ldg(w + col + i);
      b[i] *= __ldg(w + (IL ? col + (i ^ 1) : other + i));
    }
  }
};

// One row forward: x (its raw 16 bytes) to y.
template <typename T, int D, bool IL>
ELSAA_DEV void row_forward(const uint4& raw, const Turn<Vec<T>::V, IL>& t, int from, const RotaryArgs& g,
                           float* y) {
  constexpr int V = Vec<T>::V, LANES = D / V;
  float x[V], o[V], r = 1.f;
  unpack<T>(raw, x);
  partners<T, IL>(raw, from, x, o);
  if (g.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss += x[i] * x[i];
    r = rsqrtf(group_sum<LANES>(ss) * (1.0f / D) + g.eps);   // (2 units off at most)
  }
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = r * (x[i] * t.a[i] + o[i] * t.b[i]);
}

template <int V>
ELSAA_DEV void load_weight(const float* w, int col, float* out) {
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = w ? __ldg(w + col + i) : 1.f;
}

// The table row of a token's position; null (recorded) where it is none.
ELSAA_DEV const float* table_row(const RotaryArgs& a, int pos, bool lead) {
  if (a.rot == 0) return a.table;
  if (pos < 0 || pos >= a.max_pos) {
    if (lead) raise_error(a.err, ERR_CHECK);
    return nullptr;
  }
  return a.table + (int64_t)pos * a.rot;
}

// blockIdx.y: chunks of HP query heads, then of HP key heads.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kThreads, kFwdBlocks)
norm_rotate_kernel(const RotaryArgs a, int hp, int q_chunks) {
  constexpr int V = Vec<T>::V, LANES = D / V, ROWS = kThreads / LANES;
  const int col = (threadIdx.x % LANES) * V;
  const int tok = blockIdx.x * ROWS + threadIdx.x / LANES;   // (B N < 2^31 / H)
  const bool live = tok < a.B * a.N;
  const int b = live ? tok / a.N : 0, n = live ? tok - b * a.N : 0;
  const bool is_q = (int)blockIdx.y < q_chunks;
  const int h0 = (is_q ? blockIdx.y : blockIdx.y - q_chunks) * hp;
  const int h1 = min(h0 + hp, is_q ? a.H : a.Hkv);
  const Strides si = is_q ? a.sq : a.sk, so = is_q ? a.sqo : a.sko;
  const T* in = static_cast<const T*>(is_q ? a.q : a.k) + b * si.b + n * si.n + col;
  T* out = static_cast<T*>(is_q ? a.qo : a.ko) + b * so.b + n * so.n + col;
  const int pos = a.positions && live ? a.positions[tok] : n;
  const float* tab = table_row(a, pos, live && col == 0);
  const bool ok = a.rot == 0 || tab != nullptr;
  uint4 raw[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      if (live && h + u < h1) raw[u] = *reinterpret_cast<const uint4*>(in + (h + u) * si.h);
    }
  };
  load(h0);   // (in flight while the angles are fetched)
  Turn<V, IL> turn(tab, live && ok ? col : D, live && ok ? a.rot : 0);
  turn.weigh(is_q ? a.wq : a.wk, col, a.rot);
  const int from = partner_lane<V>(col, a.rot);
  for (int h = h0; h < h1; h += kBatch) {
    if (h > h0) load(h);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (h + u >= h1) break;
      float x[V];
      row_forward<T, D, IL>(raw[u], turn, from, a, x);
      if (!ok)
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0.f;
      if (live) store_row(out + (h + u) * so.h, x);
    }
  }
}

// Backward: blocks [0, q_blocks) walk (token group, head chunk) items of the
// queries, the rest those of the keys; each block leaves one partial sum of
// its weight's gradient.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kThreads, kBackBlocks)
norm_rotate_back_kernel(const RotaryArgs a, int hp, int q_blocks) {
  constexpr int V = Vec<T>::V, LANES = D / V, ROWS = kThreads / LANES;
  const int col = (threadIdx.x % LANES) * V;
  const bool is_q = (int)blockIdx.x < q_blocks;
  const int heads = is_q ? a.H : a.Hkv;
  const int chunks = (heads + hp - 1) / hp;
  const int tokens = a.B * a.N;   // (tokens and items: below 2^31)
  const int items = (tokens + ROWS - 1) / ROWS * chunks;
  const int first = is_q ? blockIdx.x : blockIdx.x - q_blocks;
  const int step = is_q ? q_blocks : gridDim.x - q_blocks;
  const Strides si = is_q ? a.sq : a.sk, sg = is_q ? a.sdqo : a.sdko, so = is_q ? a.sqo : a.sko;
  const int from = partner_lane<V>(col, a.rot);
  float w[V], dw[V];
  load_weight<V>(is_q ? a.wq : a.wk, col, w);
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.f;
  for (int it = first; it < items; it += step) {
    const int group = it / chunks, tok = group * ROWS + threadIdx.x / LANES;
    const int chunk = it - group * chunks;   // (of equal size: a block may only ever get one of them)
    const int h0 = chunk * heads / chunks, h1 = (chunk + 1) * heads / chunks;
    const bool live = tok < tokens;
    const int b = live ? tok / a.N : 0, n = live ? tok - b * a.N : 0;
    const T* in = static_cast<const T*>(is_q ? a.q : a.k) + b * si.b + n * si.n + col;
    const T* dy = static_cast<const T*>(is_q ? a.dqo : a.dko) + b * sg.b + n * sg.n + col;
    T* out = static_cast<T*>(is_q ? a.qo : a.ko) + b * so.b + n * so.n + col;
    const int pos = a.positions && live ? a.positions[tok] : n;
    const float* tab = table_row(a, pos, live && col == 0);
    const bool ok = a.rot == 0 || tab != nullptr;
    uint4 cx[2], cg[2];
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        cx[u] = cg[u] = make_uint4(0, 0, 0, 0);
        if (live && ok && h + u < h1) {   // (a row without a position was written as zeros: no gradient)
          cx[u] = *reinterpret_cast<const uint4*>(in + (h + u) * si.h);
          cg[u] = *reinterpret_cast<const uint4*>(dy + (h + u) * sg.h);
        }
      }
    };
    load(h0);   // (in flight while the angles are fetched)
    const Turn<V, IL> turn(tab, live && ok ? col : D, live && ok ? a.rot : 0);
    for (int h = h0; h < h1; h += 2) {
      if (h > h0) load(h);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (h + u >= h1) break;
        // du, the transposed rotation of dy (b turns its sign); with n = x r, t = du x:
        // dw += t r,  dx = du w r - x r^3 mean(t w)
        float x[V], g[V], o[V];
        unpack<T>(cg[u], g);
        partners<T, IL>(cg[u], from, g, o);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = g[i] * turn.a[i] - o[i] * turn.b[i];
        if (a.norm) {
          unpack<T>(cx[u], x);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            ss += x[i] * x[i];
            o[i] = g[i] * x[i];
            dot += o[i] * w[i];
          }
          ss = group_sum<LANES>(ss);   // (every lane of the warp, whatever its row)
          dot = group_sum<LANES>(dot);
          const float r = ok ? rsqrtf(ss * (1.0f / D) + a.eps) : 0.f;
          const float f = (r * r) * (r * (1.0f / D) * dot);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dw[i] += o[i] * r;
            g[i] = g[i] * (w[i] * r) - x[i] * f;
          }
        }
        if (live) store_row(out + (h + u) * so.h, g);
      }
    }
  }
  if ((is_q ? a.dwq : a.dwk) == nullptr) return;
  // the block's sum, lane groups in order
  __shared__ float part[ROWS][D + 1];
#pragma unroll
  for (int i = 0; i < V; ++i) part[threadIdx.x / LANES][col + i] = dw[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int r = 0; r < ROWS; ++r) s += part[r][threadIdx.x];
    a.partials[(int64_t)blockIdx.x * D + threadIdx.x] = s;
  }
}

// dw of the queries (block y = 0) and keys (1): 32 columns a block, 32 warps over
// the partials in a fixed order, in 64 bits.
__global__ void __launch_bounds__(1024)
weight_reduce_kernel(const RotaryArgs a, int d, int q_blocks, int blocks) {
  const bool is_q = blockIdx.y == 0;
  float* to = is_q ? a.dwq : a.dwk;
  if (to == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int lo = is_q ? 0 : q_blocks, hi = is_q ? q_blocks : blocks;
  double s = 0.0;
#pragma unroll 8
  for (int r = lo + warp; r < hi; r += 32) s += (double)a.partials[(int64_t)r * d + c];
  __shared__ double part[32][33];
  part[lane][warp] = s;
  __syncthreads();
  // warp x adds column x up
  double v = part[warp][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) to[blockIdx.x * 32 + warp] = (float)v;
}

// The write into the cache: blockIdx.y walks chunks of hp query heads, key
// heads and value heads.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kThreads)
paged_write_kernel(const RotaryArgs a, int hp, int q_chunks, int k_chunks) {
  constexpr int V = Vec<T>::V, LANES = D / V, ROWS = kThreads / LANES;
  __shared__ int32_t first[kStarts + 1];
  const bool cached = a.seqs <= kStarts;
  if (cached) {
    for (int i = threadIdx.x; i <= a.seqs; i += kThreads) first[i] = a.starts[i];
    __syncthreads();
  }
  const int32_t* st = cached ? first : a.starts;
  const int col = (threadIdx.x % LANES) * V;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
  const int64_t context = (int64_t)a.page_size * a.table_width;
  // sequences that do not fit are recorded by one block, whether they have rows here or not
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.seqs; i += kThreads)
      if (!tokens_fit(st[i], st[i + 1], a.lengths[i], a.N, context)) raise_error(a.err, ERR_CHECK);
  // the last sequence that starts at or before the row (empty ones share a start)
  int lo = 0, hi = a.seqs - 1;
  while (row < a.N && lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (st[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int seq = lo, s0 = st[seq], s1 = st[seq + 1];
  const bool mine = row < a.N && row >= s0 && row < s1;
  const int len = mine ? a.lengths[seq] : 0;
  const bool live = mine && tokens_fit(s0, s1, len, a.N, context);   // (else the row stays as it was)
  const int pos = live ? len - s1 + (int)row : 0;
  const int kind = (int)blockIdx.y < q_chunks ? 0 : (int)blockIdx.y < q_chunks + k_chunks ? 1 : 2;
  const int y = blockIdx.y - (kind == 0 ? 0 : kind == 1 ? q_chunks : q_chunks + k_chunks);
  const int h0 = y * hp, h1 = min(h0 + hp, kind == 0 ? a.H : a.Hkv);
  // keys and values: the token's page and slot, checked before anything is written
  int64_t page = -1;
  bool ok = live;
  if (ok && kind != 0) {
    page = a.page_table[(int64_t)seq * a.table_width + pos / a.page_size];
    ok = page >= 0 && page < a.pages;
  }
  if (live && !ok && col == 0) raise_error(a.err, ERR_CHECK);
  const int slot = ok ? pos % a.page_size : 0;
  if (kind == 2) {
    const T* in = static_cast<const T*>(a.v) + row * a.sv.n + col;
    T* out = static_cast<T*>(a.v_pages) + page * a.svp.b + slot * a.svp.n + col;
    if (ok)
      for (int h = h0; h < h1; h += kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (h + u < h1) raw[u] = *reinterpret_cast<const uint4*>(in + (h + u) * a.sv.h);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (h + u < h1) *reinterpret_cast<uint4*>(out + (h + u) * a.svp.h) = raw[u];
      }
    return;
  }
  const Strides si = kind == 0 ? a.sq : a.sk;
  const T* in = static_cast<const T*>(kind == 0 ? a.q : a.k) + row * si.n + col;
  T* out = kind == 0 ? static_cast<T*>(a.qo) + row * a.sqo.n + col
                     : static_cast<T*>(a.k_pages) + page * a.skp.b + slot * a.skp.n + col;
  const int64_t oh = kind == 0 ? a.sqo.h : a.skp.h;
  const float* tab = ok ? table_row(a, pos, col == 0) : nullptr;
  const bool pos_ok = ok && (a.rot == 0 || tab != nullptr);
  Turn<V, IL> turn(tab, pos_ok ? col : D, pos_ok ? a.rot : 0);
  turn.weigh(kind == 0 ? a.wq : a.wk, col, a.rot);
  const int from = partner_lane<V>(col, a.rot);
  for (int h = h0; h < h1; h += kBatch) {
    uint4 raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      if (pos_ok && h + u < h1) raw[u] = *reinterpret_cast<const uint4*>(in + (h + u) * si.h);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (h + u >= h1) break;
      float x[V];
      row_forward<T, D, IL>(raw[u], turn, from, a, x);
      if (!pos_ok)
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0.f;
      // a query row without a position is zeros; a key row is written with a page only
      if (kind == 0 ? live : ok) store_row(out + (h + u) * oh, x);
    }
  }
}

// Heads that a lane group walks: as many as leave the card (148 SMs x 1024 threads) filled,
// at most `most`.  More of them share an angle and are loaded together; the forward on
// text-32k 78 us with at most 8, 71 with 16, a fused projection of 32 and 8 heads over 4099
// tokens 19.9, 17.8 (22.1 with 32), 24.4 where the card had to be filled four times.
int head_chunk(int64_t tokens, int lanes, int heads, int most) {
  int hp = most;
  while (hp > 1 && tokens * lanes * ((heads + hp - 1) / hp) < (int64_t)148 * 1024) hp >>= 1;
  return hp;
}

template <typename F>
cudaError_t by_shape(int d, bool bf16, bool il, F&& f) {
#define ELSAA_ROW(T, D)                                         \
  return il ? f.template operator()<T, D, true>() : f.template operator()<T, D, false>()
  if (bf16) {
    if (d == 32) ELSAA_ROW(__nv_bfloat16, 32);
    if (d == 64) ELSAA_ROW(__nv_bfloat16, 64);
    ELSAA_ROW(__nv_bfloat16, 128);
  }
  if (d == 32) ELSAA_ROW(float, 32);
  if (d == 64) ELSAA_ROW(float, 64);
  ELSAA_ROW(float, 128);
#undef ELSAA_ROW
}

struct Forward {
  const RotaryArgs& a;
  cudaStream_t s;
  template <typename T, int D, bool IL>
  cudaError_t operator()() const {
    constexpr int LANES = D / Vec<T>::V, ROWS = kThreads / LANES;
    const int64_t tokens = (int64_t)a.B * a.N;
    const int hp = head_chunk(tokens, LANES, a.H + a.Hkv, 16);
    const int qc = (a.H + hp - 1) / hp, kc = (a.Hkv + hp - 1) / hp;
    const dim3 grid((unsigned)((tokens + ROWS - 1) / ROWS), qc + kc);
    norm_rotate_kernel<T, D, IL><<<grid, kThreads, 0, s>>>(a, hp, qc);
    return cudaGetLastError();
  }
};

struct Backward {
  const RotaryArgs& a;
  cudaStream_t s;
  template <typename T, int D, bool IL>
  cudaError_t operator()() const {
    constexpr int LANES = D / Vec<T>::V, ROWS = kThreads / LANES;
    const int64_t tokens = (int64_t)a.B * a.N, groups = (tokens + ROWS - 1) / ROWS;
    const int hp = head_chunk(tokens, LANES, a.H + a.Hkv, 8);
    const int64_t qi = groups * ((a.H + hp - 1) / hp), ki = groups * ((a.Hkv + hp - 1) / hp);
    // blocks by the share of the heads, all resident at once
    const int64_t cap = kRotaryPartials;
    int64_t qb = qi, kb = ki;
    if (qi + ki > cap) {
      kb = cap * a.Hkv / (a.H + a.Hkv);
      kb = kb > ki ? ki : a.Hkv && kb < 1 ? 1 : kb;
      qb = cap - kb > qi ? qi : cap - kb;
    }
    norm_rotate_back_kernel<T, D, IL><<<(unsigned)(qb + kb), kThreads, 0, s>>>(a, hp, (int)qb);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.dwq && !a.dwk)) return e;
    weight_reduce_kernel<<<dim3(D / 32, 2), 1024, 0, s>>>(a, D, (int)qb, (int)(qb + kb));
    return cudaGetLastError();
  }
};

struct Write {
  const RotaryArgs& a;
  cudaStream_t s;
  template <typename T, int D, bool IL>
  cudaError_t operator()() const {
    constexpr int LANES = D / Vec<T>::V, ROWS = kThreads / LANES;
    const int hp = head_chunk(a.N, LANES, a.H + 2 * a.Hkv, 16);
    const int qc = (a.H + hp - 1) / hp, kc = (a.Hkv + hp - 1) / hp;
    const dim3 grid((unsigned)((a.N + ROWS - 1) / ROWS), qc + 2 * kc);
    paged_write_kernel<T, D, IL><<<grid, kThreads, 0, s>>>(a, hp, qc, kc);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_rotary_forward(const RotaryArgs& a, int d, bool bf16, bool interleaved,
                                  cudaStream_t s) {
  return by_shape(d, bf16, interleaved, Forward{a, s});
}
cudaError_t launch_rotary_backward(const RotaryArgs& a, int d, bool bf16, bool interleaved,
                                   cudaStream_t s) {
  return by_shape(d, bf16, interleaved, Backward{a, s});
}
cudaError_t launch_paged_write(const RotaryArgs& a, int d, bool bf16, bool interleaved,
                               cudaStream_t s) {
  return by_shape(d, bf16, interleaved, Write{a, s});
}

}  // namespace elsaa
