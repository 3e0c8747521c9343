// Causal attention over a sliding window with sinks, and over a paged cache, on
// CUDA cores: fp32 at every head dim (fp32 data keep fp32 products, which the tensor
// cores do not have), and d = 32.
//
// Query at position i sees the keys j <= i with i - j < window or j < sinks.
// y_i = sum_j p_ij v_j, p = exp(scale q k - lse).  Backward, D_i = y_i . dy_i:
//   dS = p (dy v - D),  dq = scale dS k,  dk = scale dS^T q,  dv = p^T dy.
//
// Tiles of R rows (64, or 16 where 64 would leave most of the card idle) against
// 64-row blocks in shared memory (fp32), 256 threads as 16 x 16 with an R / 16 x 4
// score tile and R / 16 x D / 16 output values each; one pass over the keys with the
// running maximum and sum.  Only the blocks that some row of the tile sees are
// visited: the sinks' and the window's.  The backward runs one kernel for dq (query
// tiles) and one for dk and dv (key tiles, over all query heads of the group): every
// output has one writer and no atomics.  Paged work is one list of (row tile, key
// head, key block) units cut into equal runs, one per CTA; an item cut between CTAs
// leaves unnormalised partial rows, which the last CTA to get there adds up in the
// CTAs' order.
// Bound: the shared-memory reads that feed the products (a 4 x 4 score tile reads 8
// vectors for 64 FMA a thread) and instruction issue.  fp32, 8 heads of d = 64, 8192 tokens,
// window 512, 4 sinks, forward 368 us: L1 and shared memory 76 % busy, issue slots 72 %, the
// FMA pipe 55 %; warps wait for shared reads (1.3 an issue), then for their turn, and for a
// block's copy and its barriers (0.5), which two CTAs an SM cover (at d = 128 there is one).
#include <math.h>

#include "attend.cuh"
#include "paged_runs.cuh"
#include "common.cuh"
#include "internal.h"
#include "layer.h"

namespace elsaa {
namespace {

constexpr int kThreads = 256;
constexpr int kPs = kBlk + 4;    // pitch of a score tile's rows

template <int D>
constexpr int pitch() { return D + 4; }

ELSAA_DEV float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
ELSAA_DEV float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

// `rows` rows x D of fp32 in shared memory from row pointers (null: zeros).
template <typename T, int D, int ROWS, typename F>
ELSAA_DEV void load_tile(float* dst, F&& row_ptr) {
  constexpr int PER = D / 4, STEPS = ROWS * PER / kThreads;   // 4 values a step
  static_assert(ROWS * PER % kThreads == 0 || ROWS * PER < kThreads, "whole steps");
  auto step = [&](int i) {
    const int r = i / PER, c = (i % PER) * 4;
    const T* p = row_ptr(r);
    *reinterpret_cast<float4*>(dst + r * pitch<D>() + c) = p ? load4(p + c) : make_float4(0, 0, 0, 0);
  };
  if constexpr (STEPS == 0) {
    if (threadIdx.x < ROWS * PER) step(threadIdx.x);
  } else {
#pragma unroll 8
    for (int s = 0; s < STEPS; ++s) step(threadIdx.x + s * kThreads);
  }
}

// s[a][c] = A[RT ty + a] . B[tx + 16 c] over D
template <int D, int RT>
ELSAA_DEV void scores(const float* A, const float* B, float s[RT][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[a][c] = 0.f;
#pragma unroll 4
  for (int x = 0; x < D; x += 4) {
    float4 u[RT], w[4];
#pragma unroll
    for (int a = 0; a < RT; ++a) u[a] = load4(A + (RT * ty + a) * pitch<D>() + x);
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = load4(B + (tx + 16 * c) * pitch<D>() + x);
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s[a][c] += u[a].x * w[c].x + u[a].y * w[c].y + u[a].z * w[c].z + u[a].w * w[c].w;
  }
}

// The output columns of a thread: R runs of W consecutive ones.
template <int D>
struct Cols {
  static constexpr int W = D >= 64 ? 4 : 2;
  static constexpr int R = D / 16 / W;
  ELSAA_DEV static int at(int r) { return (threadIdx.x & 15) * W + r * 64; }
};

// o[a][] += sum_j P[RT ty + a][j] X[j][] over 64 j (P pitch kPs)
template <int D, int RT>
ELSAA_DEV void accumulate(const float* P, const float* X, float o[RT][D / 16]) {
  using C = Cols<D>;
  const int ty = threadIdx.x >> 4;
#pragma unroll 4
  for (int j = 0; j < kBlk; j += 4) {
    float p[RT][4];
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      const float4 v = load4(P + (RT * ty + a) * kPs + j);
      p[a][0] = v.x, p[a][1] = v.y, p[a][2] = v.z, p[a][3] = v.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int r = 0; r < C::R; ++r) {
        const float* x = X + (j + jj) * pitch<D>() + C::at(r);
        float v[4];
        if (C::W == 4) {
          const float4 u = load4(x);
          v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        } else {
          const float2 u = *reinterpret_cast<const float2*>(x);
          v[0] = u.x, v[1] = u.y;
        }
#pragma unroll
        for (int e = 0; e < C::W; ++e)
#pragma unroll
          for (int a = 0; a < RT; ++a) o[a][r * C::W + e] += p[a][jj] * v[e];
      }
  }
}

template <typename T, int D>
ELSAA_DEV void store_cols(T* row, const float* o) {
  using C = Cols<D>;
#pragma unroll
  for (int r = 0; r < C::R; ++r)
#pragma unroll
    for (int e = 0; e < C::W; ++e) row[C::at(r) + e] = from_f32<T>(o[r * C::W + e]);
}

ELSAA_DEV float row_max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
ELSAA_DEV float row_sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The running softmax of a thread's rows (replicated over the 16 threads of a row).
template <int D, int RT>
struct Rows {
  float o[RT][D / 16], m[RT], l[RT];
  ELSAA_DEV void clear() {
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[x][c] = 0.f;
    }
  }
  // one block of keys j0 .. j0 + 63; pos[x]: the row's position, -1 where it has none
  ELSAA_DEV void block(const float* Qs, const float* Ks, const float* Vs, float* Ps, int j0,
                       const int* pos, const AttendArgs& a) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float s[RT][4];
    scores<D, RT>(Qs, Ks, s);
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        s[x][c] = sees(pos[x], j, a.window, a.sinks) ? s[x][c] * a.scale : -INFINITY;
        top = fmaxf(top, s[x][c]);
      }
      top = fmaxf(m[x], row_max16(top));
      const float base = top == -INFINITY ? 0.f : top;
      const float f = expf(m[x] - base);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = expf(s[x][c] - base);
        sum += p;
        Ps[(RT * ty + x) * kPs + tx + 16 * c] = p;
      }
      l[x] = l[x] * f + row_sum16(sum);
      m[x] = top;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[x][c] *= f;
    }
    __syncwarp();   // a row of P is written and read by the same half warp
    accumulate<D, RT>(Ps, Vs, o);
  }
};

// ---- window forward --------------------------------------------------------------

ELSAA_DEV int length_of(const AttendArgs& a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
}

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads)
window_fwd_simt_kernel(const AttendArgs a, int tiles) {
  constexpr int RT = ROWS / 16;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + ROWS * pitch<D>();
  float* Vs = Ks + kBlk * pitch<D>();
  float* Ps = Vs + kBlk * pitch<D>();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int bh = blockIdx.x / tiles, b = bh / a.H, h = bh % a.H, hk = h / a.g;
  const int r0 = (tiles - 1 - (int)(blockIdx.x % tiles)) * ROWS;   // the longest rows first
  const int len = length_of(a, b);
  auto row = [&](const void* base, const Strides& s, int head, int n) -> const T* {
    return n < len ? static_cast<const T*>(base) + b * s.b + head * s.h + n * s.n : nullptr;
  };
  load_tile<T, D, ROWS>(Qs, [&](int r) { return row(a.q, a.sq, h, r0 + r); });
  const KeyBlocks kb = key_blocks(r0, min(len, r0 + ROWS) - 1, a.window, a.sinks, kBlk);
  Rows<D, RT> st;
  st.clear();
  int pos[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) pos[x] = r0 + RT * ty + x < len ? r0 + RT * ty + x : -1;
  for (int n = 0; n < kb.count(); ++n) {
    const int j0 = kb.block(n) * kBlk;
    __syncthreads();
    load_tile<T, D, kBlk>(Ks, [&](int r) { return row(a.k, a.sk, hk, j0 + r); });
    load_tile<T, D, kBlk>(Vs, [&](int r) { return row(a.v, a.sv, hk, j0 + r); });
    __syncthreads();
    st.block(Qs, Ks, Vs, Ps, j0, pos, a);
  }
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int n = r0 + RT * ty + x;
    if (n >= a.N) continue;
    const bool some = st.l[x] != 0.f;   // (NaN too: a score was)
    const float inv = some ? 1.0f / st.l[x] : 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) st.o[x][c] *= inv;
    store_cols<T, D>(static_cast<T*>(a.y) + b * a.sy.b + h * a.sy.h + n * a.sy.n, st.o[x]);
    if (tx == 0)
      a.lse[(int64_t)bh * a.N + n] = some ? st.m[x] + logf(st.l[x]) : -INFINITY;
  }
}

// ---- paged -----------------------------------------------------------------------

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads)
paged_simt_kernel(const AttendArgs a) {
  constexpr int RT = ROWS / 16;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + ROWS * pitch<D>();
  float* Vs = Ks + kBlk * pitch<D>();
  float* Ps = Vs + kBlk * pitch<D>();
  __shared__ Run run;
  __shared__ int pages[kBlk], last;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, g = a.g, tt = ROWS / g;
  if (threadIdx.x < 32) {
    const Run c = find_run(a, tt, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) run = c;
  }
  __syncthreads();
  int b = run.b, tile = run.tile, hk = run.hk, off = run.off, left = run.units;
  int start = run.start, len = run.len, tokens = run.tokens;
  int64_t at = run.per * blockIdx.x;   // the next unit
  for (int order = 0; left > 0; ++order) {
    while (tile * tt >= tokens) {
      if (++b >= a.seqs) return;       // (a later sequence holds the units left)
      tile = hk = off = 0;
      tokens = new_tokens(a, b, &start, &len, false);
    }
    const PagedItem it = paged_item(a, tt, tile, tokens, len);
    const int nblk = it.kb.count(), n0 = off, n1 = min(nblk, off + left);
    // row r of the tile: token tile tt + r / g, head hk g + r % g
    auto live = [&](int r) { return r / g < tt && tile * tt + r / g < tokens; };
    auto at_row = [&](const Strides& s, int r) -> int64_t {
      return (int64_t)(start + tile * tt + r / g) * s.n + (int64_t)(hk * g + r % g) * s.h;
    };
    __syncthreads();
    load_tile<T, D, ROWS>(Qs, [&](int r) -> const T* {
      return live(r) ? static_cast<const T*>(a.q) + at_row(a.sq, r) : nullptr;
    });
    Rows<D, RT> st;
    st.clear();
    int pos[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) pos[x] = live(RT * ty + x) ? it.p_lo + (RT * ty + x) / g : -1;
    for (int n = n0; n < n1; ++n) {
      const int j0 = it.kb.block(n) * kBlk;
      __syncthreads();
      if (threadIdx.x < kBlk) {
        // entries that no row of the tile sees are not looked up
        const int j = j0 + threadIdx.x;
        const bool need = j <= it.p_hi && (j < a.sinks || (int64_t)j > (int64_t)it.p_lo - a.window);
        pages[threadIdx.x] = need ? page_of(a, b, j) : -1;
      }
      __syncthreads();
      auto key = [&](const void* base, const Strides& s, int r) -> const T* {
        return pages[r] >= 0 ? static_cast<const T*>(base) + (int64_t)pages[r] * s.b + (int64_t)hk * s.h +
                                   (int64_t)((j0 + r) % a.page_size) * s.n
                             : nullptr;
      };
      load_tile<T, D, kBlk>(Ks, [&](int r) { return key(a.k, a.sk, r); });
      load_tile<T, D, kBlk>(Vs, [&](int r) { return key(a.v, a.sv, r); });
      __syncthreads();
      st.block(Qs, Ks, Vs, Ps, j0, pos, a);
    }
    const bool whole = n0 == 0 && n1 == nblk;
    const int slot = (int)blockIdx.x * 2 + (order > 0 ? 1 : 0);
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int r = RT * ty + x;
      if (!live(r)) continue;
      if (whole) {
        const float inv = st.l[x] > 0.f ? 1.0f / st.l[x] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) st.o[x][c] *= inv;
        store_cols<T, D>(static_cast<T*>(a.y) + at_row(a.sy, r), st.o[x]);
      } else {
        store_cols<float, D>(partial_o<ROWS>(a, D, slot, r), st.o[x]);
        if (tx == 0) *partial_ml<ROWS>(a, D, slot, r) = make_float2(st.m[x], st.l[x]);
      }
    }
    if (!whole) {
      const Ctas c = ctas_of(at - off, nblk, run.per);
      const int cta0 = c.first, cta1 = c.last, slot0 = c.slot0;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        last = atomicAdd(a.counters + cta0, 1u) == (uint32_t)(cta1 - cta0) ? 1 : 0;
      __syncthreads();
      if (last) {
        __threadfence();
        for (int x = threadIdx.x; x < ROWS * (D / 4); x += kThreads) {
          const int r = x / (D / 4), c = x % (D / 4) * 4;
          if (!live(r)) break;   // (rows end with the tokens)
          auto slot_of = [&](int i) { return 2 * i + (i == cta0 ? slot0 : 0); };
          float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
          for (int i = cta0; i <= cta1; ++i) m = fmaxf(m, __ldcg(partial_ml<ROWS>(a, D, slot_of(i), r)).x);
#pragma unroll 4
          for (int i = cta0; i <= cta1; ++i) {
            const float2 ml = __ldcg(partial_ml<ROWS>(a, D, slot_of(i), r));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(partial_o<ROWS>(a, D, slot_of(i), r) + c));
            const float w = ml.x > -INFINITY ? expf(ml.x - m) : 0.f;
            l += ml.y * w;
            o[0] += v.x * w, o[1] += v.y * w, o[2] += v.z * w, o[3] += v.w * w;
          }
          const float inv = l > 0.f ? 1.0f / l : 0.f;
          T* y = static_cast<T*>(a.y) + at_row(a.sy, r) + c;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(o[e] * inv);
        }
        if (threadIdx.x == 0) a.counters[cta0] = 0;
      }
    }
    left -= n1 - n0;
    at += n1 - n0;
    off = 0;
    if (++hk == a.Hkv) hk = 0, ++tile;
  }
}

// ---- backward --------------------------------------------------------------------

// delta = rowsum(y dy), one warp a row (rows behind a length are not read).
template <typename T>
__global__ void __launch_bounds__(kThreads) window_delta_kernel(const AttendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= (int64_t)a.B * a.H * a.N) return;
  const int n = (int)(row % a.N), h = (int)(row / a.N % a.H), b = (int)(row / a.N / a.H);
  float s = 0.f;
  if (n < length_of(a, b)) {
    const T* y = static_cast<const T*>(a.y) + b * a.sy.b + h * a.sy.h + n * a.sy.n;
    const T* g = static_cast<const T*>(a.dy) + b * a.sdy.b + h * a.sdy.h + n * a.sdy.n;
    for (int c = lane; c < a.d; c += 32) s += to_f32(y[c]) * to_f32(g[c]);
  }
  s = warp_sum(s);
  // bf16 rows that see few keys (kFewKeys)
  if (sizeof(T) == 2 && n < length_of(a, b) && seen_keys(n, a.window, a.sinks) <= kFewKeys) {
    const int few = seen_keys(n, a.window, a.sinks), hk = h / a.g;
    const T* q = static_cast<const T*>(a.q) + b * a.sq.b + h * a.sq.h + n * a.sq.n;
    const T* g = static_cast<const T*>(a.dy) + b * a.sdy.b + h * a.sdy.h + n * a.sdy.n;
    const float lse = a.lse[row];
    s = 0.f;
    for (int x = 0; x < few; ++x) {
      const int64_t j = seen_key(x, n, a.window, a.sinks);
      const T* k = static_cast<const T*>(a.k) + b * a.sk.b + hk * a.sk.h + j * a.sk.n;
      const T* v = static_cast<const T*>(a.v) + b * a.sv.b + hk * a.sv.h + j * a.sv.n;
      float e = 0.f, r = 0.f;
      for (int c = lane; c < a.d; c += 32) {
        e += to_f32(q[c]) * to_f32(k[c]);
        r += to_f32(g[c]) * to_f32(v[c]);
      }
      s += expf(warp_sum(e) * a.scale - lse) * warp_sum(r);
    }
  }
  if (lane == 0) a.delta[row] = s;
}

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads) window_dq_simt_kernel(const AttendArgs a, int tiles) {
  constexpr int RT = ROWS / 16;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Gs = Qs + ROWS * pitch<D>();
  float* Ks = Gs + ROWS * pitch<D>();
  float* Vs = Ks + kBlk * pitch<D>();
  float* Ps = Vs + kBlk * pitch<D>();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int bh = blockIdx.x / tiles, b = bh / a.H, h = bh % a.H, hk = h / a.g;
  const int r0 = (tiles - 1 - (int)(blockIdx.x % tiles)) * ROWS;
  const int len = length_of(a, b);
  auto row = [&](const void* base, const Strides& s, int head, int n) -> const T* {
    return n < len ? static_cast<const T*>(base) + b * s.b + head * s.h + n * s.n : nullptr;
  };
  load_tile<T, D, ROWS>(Qs, [&](int r) { return row(a.q, a.sq, h, r0 + r); });
  load_tile<T, D, ROWS>(Gs, [&](int r) { return row(a.dy, a.sdy, h, r0 + r); });
  float lse[RT], del[RT], o[RT][D / 16];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int n = r0 + RT * ty + x;
    const bool live = n < len;
    lse[x] = live ? a.lse[(int64_t)bh * a.N + n] : 0.f;
    del[x] = live ? a.delta[(int64_t)bh * a.N + n] : 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[x][c] = 0.f;
  }
  const KeyBlocks kb = key_blocks(r0, min(len, r0 + ROWS) - 1, a.window, a.sinks, kBlk);
  for (int n = 0; n < kb.count(); ++n) {
    const int j0 = kb.block(n) * kBlk;
    __syncthreads();
    load_tile<T, D, kBlk>(Ks, [&](int r) { return row(a.k, a.sk, hk, j0 + r); });
    load_tile<T, D, kBlk>(Vs, [&](int r) { return row(a.v, a.sv, hk, j0 + r); });
    __syncthreads();
    float s[RT][4], t[RT][4];
    scores<D, RT>(Qs, Ks, s);
    scores<D, RT>(Gs, Vs, t);
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int pos = r0 + RT * ty + x;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        const bool see = pos < len && sees(pos, j, a.window, a.sinks);
        Ps[(RT * ty + x) * kPs + tx + 16 * c] =
            see ? expf(s[x][c] * a.scale - lse[x]) * (t[x][c] - del[x]) * a.scale : 0.f;
      }
    }
    __syncwarp();
    accumulate<D, RT>(Ps, Ks, o);
  }
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int n = r0 + RT * ty + x;
    if (n < a.N) store_cols<T, D>(static_cast<T*>(a.dq) + b * a.sdq.b + h * a.sdq.h + n * a.sdq.n, o[x]);
  }
}

// How many CTAs share a key tile's (head of the group, query block) list: a head's first
// `sinks` tiles, which every query behind them sees, `sink` each, the others `other`.
struct Parts {
  int sinks, sink, other;
};

// With more than one CTA a tile, each leaves its sums in `partial` ([tile][part][2][ROWS][D])
// and the last to come adds them up in order.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads)
window_dkv_simt_kernel(const AttendArgs a, int tiles, const Parts share, float* partial) {
  constexpr int RT = ROWS / 16;
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + ROWS * pitch<D>();
  float* Qs = Vs + ROWS * pitch<D>();
  float* Gs = Qs + kBlk * pitch<D>();
  float* Ps = Gs + kBlk * pitch<D>();   // [key][query]
  float* Ds = Ps + ROWS * kPs;
  __shared__ int last;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lead = share.sinks * share.sink, per = lead + (tiles - share.sinks) * share.other;
  const int bk = blockIdx.x / per, b = bk / a.Hkv, hk = bk % a.Hkv, at = blockIdx.x % per;
  const bool sink = at < lead;
  const int parts = sink ? share.sink : share.other, part = (sink ? at : at - lead) % parts;
  const int tile = sink ? at / parts : share.sinks + (at - lead) / parts;
  const int j0 = tile * ROWS;
  const int len = length_of(a, b);
  auto row = [&](const void* base, const Strides& s, int head, int n) -> const T* {
    return n < len ? static_cast<const T*>(base) + b * s.b + head * s.h + n * s.n : nullptr;
  };
  load_tile<T, D, ROWS>(Ks, [&](int r) { return row(a.k, a.sk, hk, j0 + r); });
  load_tile<T, D, ROWS>(Vs, [&](int r) { return row(a.v, a.sv, hk, j0 + r); });
  float ok[RT][D / 16], ov[RT][D / 16];
#pragma unroll
  for (int x = 0; x < RT; ++x)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) ok[x][c] = ov[x][c] = 0.f;
  const int64_t reach = j0 < a.sinks ? len : (int64_t)j0 + ROWS - 1 + a.window;
  const int i_end = (int)(reach < len ? reach : len);   // queries j0 .. i_end - 1 may see the tile
  const int nq = i_end > j0 ? (i_end - j0 + kBlk - 1) / kBlk : 0;
  const int64_t list = (int64_t)nq * a.g;
  for (int n = (int)(list * part / parts); n < (int)(list * (part + 1) / parts); ++n) {
    const int h = hk * a.g + n / nq, i0 = j0 + n % nq * kBlk;
    const int64_t rows = ((int64_t)b * a.H + h) * a.N;
    __syncthreads();
    load_tile<T, D, kBlk>(Qs, [&](int r) { return row(a.q, a.sq, h, i0 + r); });
    load_tile<T, D, kBlk>(Gs, [&](int r) { return row(a.dy, a.sdy, h, i0 + r); });
    __syncthreads();
    float s[RT][4], t[RT][4];
    scores<D, RT>(Ks, Qs, s);
    scores<D, RT>(Vs, Gs, t);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = i0 + tx + 16 * c;
      const float lse = i < len ? a.lse[rows + i] : 0.f, del = i < len ? a.delta[rows + i] : 0.f;
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        const int j = j0 + RT * ty + x;
        const bool see = i < len && sees(i, j, a.window, a.sinks);
        const float p = see ? expf(s[x][c] * a.scale - lse) : 0.f;
        Ps[(RT * ty + x) * kPs + tx + 16 * c] = p;
        Ds[(RT * ty + x) * kPs + tx + 16 * c] = see ? p * (t[x][c] - del) * a.scale : 0.f;
      }
    }
    __syncwarp();
    accumulate<D, RT>(Ps, Gs, ov);
    accumulate<D, RT>(Ds, Qs, ok);
  }
  if (parts > 1) {
    // (the sinks' tiles of all heads, then the others)
    const int heads = a.B * a.Hkv, most = heads * share.sinks;
    const int item = sink ? bk * share.sinks + tile : most + bk * (tiles - share.sinks) + tile - share.sinks;
    const int64_t slot = sink ? (int64_t)item * parts
                              : (share.sink > 1 ? (int64_t)most * share.sink : 0) + (int64_t)(item - most) * parts;
    float* base = partial + slot * 2 * ROWS * D;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      store_cols<float, D>(base + ((int64_t)part * 2 * ROWS + RT * ty + x) * D, ov[x]);
      store_cols<float, D>(base + (((int64_t)part * 2 + 1) * ROWS + RT * ty + x) * D, ok[x]);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.counters + item, 1u) == (uint32_t)(parts - 1) ? 1 : 0;
    __syncthreads();
    if (!last) return;
    __threadfence();
    using C = Cols<D>;
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float sv = 0.f, sk = 0.f;
        const int col = C::at(c / C::W) + c % C::W;
#pragma unroll 4
        for (int q = 0; q < parts; ++q) {
          sv += __ldcg(base + ((int64_t)q * 2 * ROWS + RT * ty + x) * D + col);
          sk += __ldcg(base + (((int64_t)q * 2 + 1) * ROWS + RT * ty + x) * D + col);
        }
        ov[x][c] = sv;
        ok[x][c] = sk;
      }
    if (threadIdx.x == 0) a.counters[item] = 0;
  }
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int n = j0 + RT * ty + x;
    if (n >= a.N) continue;
    store_cols<T, D>(static_cast<T*>(a.dk) + b * a.sdk.b + hk * a.sdk.h + n * a.sdk.n, ok[x]);
    store_cols<T, D>(static_cast<T*>(a.dv) + b * a.sdv.b + hk * a.sdv.h + n * a.sdv.n, ov[x]);
  }
}

// ---- launches --------------------------------------------------------------------

template <typename K, typename... A>
cudaError_t run(K kernel, int64_t blocks, size_t smem, cudaStream_t s, A... args) {
  if (blocks <= 0 || blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)blocks, kThreads, smem, s>>>(args...);
  return cudaGetLastError();
}

// Bytes of `tiles` R-row tiles, `blocks` 64-row blocks and `scores` R x 64 score tiles.
template <int D>
constexpr size_t bytes(int R, int tiles, int blocks, int scores) {
  return sizeof(float) * ((size_t)(tiles * R + blocks * kBlk) * pitch<D>() + (size_t)scores * R * kPs);
}

// 16-row query tiles where 64-row ones would leave two thirds of the SMs idle: a tile of 16
// does a quarter of the work of one of 64 in two thirds of its time (fp32, d = 64, window 72:
// forward of 20 tiles 17 against 25 us, of 80 tiles 28 against 25.5, of 120 39 against 26).
bool small_tiles(int64_t heads, int N) { return heads * ((N + 63) / 64) < 50; }

// Query blocks that see a key tile of 64 without sinks, and all of them.
int64_t near_blocks(int N, int64_t window, int R) {
  const int64_t all = (N + kBlk - 1) / kBlk, few = (window + R - 1 + kBlk - 1) / kBlk + 1;
  return few < all ? few : all;
}
// 16-row key tiles where 64-row ones would not fill the card even with their lists (g heads x
// query blocks) shared by up to 16 CTAs (fp32, d = 64, window 72, g = 1: 20 tiles 28 against 56
// us, 40 tiles 34 against 42, 80 tiles 51 against 43; 24 tiles of a group of 8 over 1500 tokens
// at d = 128 866 against 374).
bool small_key_tiles(int64_t heads, int g, int N, int window) {
  const int64_t list = g * near_blocks(N, window, 64);
  return heads * ((N + 63) / 64) * (list < 16 ? list : 16) < 200;
}

template <typename T, int D, int R>
cudaError_t forward(const AttendArgs& a, cudaStream_t s) {
  const int tiles = (a.N + R - 1) / R;
  return run(window_fwd_simt_kernel<T, D, R>, (int64_t)a.B * a.H * tiles, bytes<D>(R, 1, 2, 1), s, a, tiles);
}
template <typename T, int D, int R>
cudaError_t dq(const AttendArgs& a, cudaStream_t s) {
  const int tiles = (a.N + R - 1) / R;
  return run(window_dq_simt_kernel<T, D, R>, (int64_t)a.B * a.H * tiles, bytes<D>(R, 2, 2, 1), s, a, tiles);
}
// CTAs that share a key tile: as many as give every SM two; for the sinks' tiles as many as
// make their lists as short as the others' (fp32, 8 heads of d = 64, 8192 tokens, a window of
// 512 and 4 sinks: the backward 2439 us with one CTA each, 1247 so).  At most 16, and no more
// tiles than counters.
Parts dkv_parts(int64_t heads, int N, int R, int window, int sinks) {
  const int64_t tiles = (N + R - 1) / R, items = heads * tiles, p = (296 + items - 1) / items;
  Parts s{0, 1, (int)(p > 16 ? 16 : p)};
  if (sinks == 0 || window >= N) return s;
  const int64_t most = ((int64_t)sinks + R - 1) / R;
  int64_t n = (N + kBlk - 1) / kBlk / near_blocks(N, window, R);
  n = n > 16 ? 16 : n;
  if (n <= s.other || heads * most > 1024) return s;
  s.sinks = (int)(most < tiles ? most : tiles);
  s.sink = (int)n;
  return s;
}
// Partial sums of the shared tiles, [2][R][d] each.
int64_t dkv_slots(const Parts& s, int64_t heads, int64_t tiles) {
  return (s.sink > 1 ? heads * s.sinks * s.sink : 0) + (s.other > 1 ? heads * (tiles - s.sinks) * s.other : 0);
}
template <typename T, int D, int R>
cudaError_t dkv(const AttendArgs& a, cudaStream_t s) {
  const int tiles = (a.N + R - 1) / R;
  const int64_t heads = (int64_t)a.B * a.Hkv;
  const Parts p = dkv_parts(heads, a.N, R, a.window, a.sinks);
  return run(window_dkv_simt_kernel<T, D, R>, heads * (p.sinks * p.sink + (int64_t)(tiles - p.sinks) * p.other),
             bytes<D>(R, 2, 2, 2), s, a, tiles, p,
             a.delta + align_up((size_t)a.B * a.H * a.N * sizeof(float)) / sizeof(float));
}

template <typename T, int D>
cudaError_t pages(const AttendArgs& a, cudaStream_t s) {
  if (paged_tile_rows(a.rows, a.seqs, a.g) == 16)
    return run(paged_simt_kernel<T, D, 16>, 296, bytes<D>(16, 1, 2, 1), s, a);
  return run(paged_simt_kernel<T, D, 64>, 296, bytes<D>(64, 1, 2, 1), s, a);
}

template <typename T, int D>
struct Launch {
  static cudaError_t fwd(const AttendArgs& a, cudaStream_t s) {
    return small_tiles((int64_t)a.B * a.H, a.N) ? forward<T, D, 16>(a, s) : forward<T, D, 64>(a, s);
  }
  static cudaError_t bwd(const AttendArgs& a, cudaStream_t s) {
    const cudaError_t e = small_tiles((int64_t)a.B * a.H, a.N) ? dq<T, D, 16>(a, s) : dq<T, D, 64>(a, s);
    if (e != cudaSuccess) return e;
    return small_key_tiles((int64_t)a.B * a.Hkv, a.g, a.N, a.window) ? dkv<T, D, 16>(a, s) : dkv<T, D, 64>(a, s);
  }
  static cudaError_t paged(const AttendArgs& a, cudaStream_t s) { return pages<T, D>(a, s); }
};

// f<T, D> of the problem's type and head dim (bf16 at d = 64, 128 has the tensor cores).
#define ELSAA_BY_SHAPE(f)                                \
  (bf16        ? Launch<__nv_bfloat16, 32>::f(a, s)      \
   : a.d == 32 ? Launch<float, 32>::f(a, s)              \
   : a.d == 64 ? Launch<float, 64>::f(a, s)              \
               : Launch<float, 128>::f(a, s))

}  // namespace

size_t window_simt_scratch_bytes(int d, int64_t B, int64_t H, int64_t Hkv, int N, int window, int sinks) {
  const int R = small_key_tiles(B * Hkv, (int)(H / Hkv), N, window) ? 16 : 64;
  const Parts p = dkv_parts(B * Hkv, N, R, window, sinks);
  return align_up((size_t)(B * H * N) * sizeof(float)) +
         (size_t)dkv_slots(p, B * Hkv, (N + R - 1) / R) * 2 * R * d * sizeof(float);
}

cudaError_t launch_window_delta(const AttendArgs& a, bool bf16, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.H * a.N, warps = kThreads / 32;
  const unsigned blocks = (unsigned)((rows + warps - 1) / warps);
  if (bf16)
    window_delta_kernel<__nv_bfloat16><<<blocks, kThreads, 0, s>>>(a);
  else
    window_delta_kernel<float><<<blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_window_fwd_simt(const AttendArgs& a, bool bf16, cudaStream_t s) {
  return ELSAA_BY_SHAPE(fwd);
}
cudaError_t launch_window_bwd_simt(const AttendArgs& a, bool bf16, cudaStream_t s) {
  return ELSAA_BY_SHAPE(bwd);
}
cudaError_t launch_paged_simt(const AttendArgs& a, bool bf16, cudaStream_t s) {
  return ELSAA_BY_SHAPE(paged);
}

}  // namespace elsaa
