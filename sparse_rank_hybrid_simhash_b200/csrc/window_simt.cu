// Causal attention over a sliding window with sinks, and over a paged cache,
// on CUDA cores: every type and head dim (fp32 data keep fp32 products, which
// the tensor cores do not have).
//
// Query at position i sees the keys j <= i with i - j < window or j < sinks.
// y_i = sum_j p_ij v_j, p = exp(scale q k - lse).  Backward, D_i = y_i . dy_i:
//   dS = p (dy v - D),  dq = scale dS k,  dk = scale dS^T q,  dv = p^T dy.
//
// Tiles of 64 query rows against 64-key blocks in shared memory (fp32), a
// 16 x 16 thread grid with a 4 x 4 score tile and 4 x D / 16 output values each;
// one pass over the keys with the running maximum and sum.  Only the blocks
// that some row of the tile sees are visited: the sinks' and the window's.
// Bound: fp32 FMA issue (the products); the backward runs one kernel for dq
// (query tiles) and one for dk and dv (key tiles, over all query heads of the
// group), so every output has one writer and no atomics.
#include <math.h>

#include "attend.cuh"
#include "common.cuh"
#include "internal.h"
#include "layer.h"

namespace elsaa {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;
constexpr int kPs = kTile + 4;   // pitch of a 64 x 64 score tile

template <int D>
constexpr int pitch() { return D + 4; }

// 64 rows x D of fp32 in shared memory from row pointers (null: zeros).
template <typename T, int D, typename F>
ELSAA_DEV void load_tile(float* dst, F&& row_ptr) {
  constexpr int PER = D / 4;   // 4 values a step
  for (int i = threadIdx.x; i < kTile * PER; i += kThreads) {
    const int r = i / PER, c = (i % PER) * 4;
    const T* p = row_ptr(r);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p != nullptr) x = make_float4(to_f32(p[c]), to_f32(p[c + 1]), to_f32(p[c + 2]), to_f32(p[c + 3]));
    *reinterpret_cast<float4*>(dst + r * pitch<D>() + c) = x;
  }
}

// s[a][c] = A[4 ty + a] . B[tx + 16 c] over D
template <int D>
ELSAA_DEV void scores(const float* A, const float* B, float s[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[a][c] = 0.f;
#pragma unroll 4
  for (int x = 0; x < D; x += 4) {
    float4 u[4], w[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) u[a] = *reinterpret_cast<const float4*>(A + (4 * ty + a) * pitch<D>() + x);
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * pitch<D>() + x);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s[a][c] += u[a].x * w[c].x + u[a].y * w[c].y + u[a].z * w[c].z + u[a].w * w[c].w;
  }
}

// The output columns of a thread: CW consecutive ones from col(c).
template <int D>
struct Cols {
  static constexpr int W = D >= 64 ? 4 : 2;      // width of a run
  static constexpr int R = D / 16 / W;           // runs
  ELSAA_DEV static int at(int r) { return (threadIdx.x & 15) * W + r * 64; }
};

// o[a][] += sum_j P[4 ty + a][j] X[j][] over 64 j (P pitch kPs)
template <int D>
ELSAA_DEV void accumulate(const float* P, const float* X, float o[4][D / 16]) {
  using C = Cols<D>;
  const int ty = threadIdx.x >> 4;
#pragma unroll 4
  for (int j = 0; j < kTile; ++j) {
    float p[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) p[a] = P[(4 * ty + a) * kPs + j];
#pragma unroll
    for (int r = 0; r < C::R; ++r)
#pragma unroll
      for (int e = 0; e < C::W; ++e) {
        const float x = X[j * pitch<D>() + C::at(r) + e];
#pragma unroll
        for (int a = 0; a < 4; ++a) o[a][r * C::W + e] += p[a] * x;
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

// ---- forward -------------------------------------------------------------------

// PAGED: a tile's rows are (token, head of the group) pairs, head fastest;
// else 64 tokens of one head.
template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(kThreads)
attend_simt_kernel(const AttendArgs a, int tiles) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + kTile * pitch<D>();
  float* Vs = Ks + kTile * pitch<D>();
  float* Ps = Vs + kTile * pitch<D>();
  __shared__ PagedTile found;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int b, h, hk, r0, len, pos0, rows;   // rows of the tile's (batch, head) or (sequence, key head)
  if (PAGED) {
    hk = blockIdx.x / tiles;
    if (threadIdx.x < 32) {
      const PagedTile t = find_paged_tile(a, blockIdx.x % tiles, kTile);
      if (threadIdx.x == 0) found = t;
    }
    __syncthreads();
    if (found.seq < 0) return;
    b = found.seq;
    r0 = found.tile * kTile;
    rows = found.rows;
    pos0 = found.pos0;
    len = found.len;
    h = 0;
  } else {
    const int bh = blockIdx.x / tiles;
    b = bh / a.H;
    h = bh % a.H;
    hk = h / a.g;
    r0 = (tiles - 1 - blockIdx.x % tiles) * kTile;   // the longest rows first
    rows = a.N;
    pos0 = 0;
    len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
  }
  const int g = PAGED ? a.g : 1;
  auto token_of = [&](int r) { return (r0 + r) / g; };
  auto q_off = [&](int r, const Strides& s) -> int64_t {
    if (PAGED) return (int64_t)(found.start + token_of(r)) * s.n + (int64_t)(hk * g + (r0 + r) % g) * s.h;
    return (int64_t)b * s.b + (int64_t)h * s.h + (int64_t)(r0 + r) * s.n;
  };
  auto key_ptr = [&](const void* base, const Strides& s, int j) -> const T* {
    if (j >= len) return nullptr;
    const T* p = static_cast<const T*>(base);
    if (PAGED) {
      const int page = page_of(a, b, j);
      if (page < 0) return nullptr;
      return p + (int64_t)page * s.b + (int64_t)hk * s.h + (int64_t)(j % a.page_size) * s.n;
    }
    return p + (int64_t)b * s.b + (int64_t)hk * s.h + (int64_t)j * s.n;
  };
  load_tile<T, D>(Qs, [&](int r) -> const T* {
    return r0 + r < rows ? static_cast<const T*>(a.q) + q_off(r, a.sq) : nullptr;
  });
  // positions of the tile's first and last row
  const int p_lo = pos0 + token_of(0), p_hi = min(len - 1, pos0 + token_of(min(kTile, rows - r0) - 1));
  const KeyBlocks kb = key_blocks(max(p_lo, 0), p_hi, a.window, a.sinks, kTile);
  float o[4][D / 16], m[4], l[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[x][c] = 0.f;
  }
  for (int n = 0; n < kb.count(); ++n) {
    const int j0 = kb.block(n) * kTile;
    // a page entry that no row of the tile sees (holes between sinks and window) is not read
    auto needed = [&](int j) { return j < a.sinks || (int64_t)j > (int64_t)p_lo - a.window; };
    __syncthreads();
    load_tile<T, D>(Ks, [&](int r) { return needed(j0 + r) ? key_ptr(a.k, a.sk, j0 + r) : nullptr; });
    load_tile<T, D>(Vs, [&](int r) { return needed(j0 + r) ? key_ptr(a.v, a.sv, j0 + r) : nullptr; });
    __syncthreads();
    float s[4][4];
    scores<D>(Qs, Ks, s);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = 4 * ty + x;
      const int pos = pos0 + token_of(r);
      const bool live = r0 + r < rows && pos < len;
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        s[x][c] = live && sees(pos, j, a.window, a.sinks) ? s[x][c] * a.scale : -INFINITY;
        top = fmaxf(top, s[x][c]);
      }
      top = fmaxf(m[x], row_max16(top));
      const float base = top == -INFINITY ? 0.f : top;
      const float f = __expf(m[x] - base);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = expf(s[x][c] - base);
        sum += p;
        Ps[r * kPs + tx + 16 * c] = p;
      }
      l[x] = l[x] * f + row_sum16(sum);
      m[x] = top;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[x][c] *= f;
    }
    __syncwarp();   // a row of P is written and read by the same half warp
    accumulate<D>(Ps, Vs, o);
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int r = 4 * ty + x;
    if (r0 + r >= rows) continue;
    const float inv = l[x] > 0.f ? 1.0f / l[x] : 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[x][c] *= inv;
    store_cols<T, D>(static_cast<T*>(a.y) + q_off(r, a.sy), o[x]);
    if (!PAGED && tx == 0)
      a.lse[((int64_t)b * a.H + h) * a.N + r0 + r] = l[x] > 0.f ? m[x] + logf(l[x]) : -INFINITY;
  }
}

// ---- backward ------------------------------------------------------------------

// delta = rowsum(y dy), one warp a row (rows behind a length are not read).
template <typename T>
__global__ void __launch_bounds__(kThreads) window_delta_kernel(const AttendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= (int64_t)a.B * a.H * a.N) return;
  const int n = (int)(row % a.N), h = (int)(row / a.N % a.H), b = (int)(row / a.N / a.H);
  float s = 0.f;
  if (!a.lengths || n < a.lengths[b]) {
    const T* y = static_cast<const T*>(a.y) + b * a.sy.b + h * a.sy.h + n * a.sy.n;
    const T* g = static_cast<const T*>(a.dy) + b * a.sdy.b + h * a.sdy.h + n * a.sdy.n;
    for (int c = lane; c < a.d; c += 32) s += to_f32(y[c]) * to_f32(g[c]);
  }
  s = warp_sum(s);
  if (lane == 0) a.delta[row] = s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_dq_simt_kernel(const AttendArgs a, int tiles) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Gs = Qs + kTile * pitch<D>();
  float* Ks = Gs + kTile * pitch<D>();
  float* Vs = Ks + kTile * pitch<D>();
  float* Ps = Vs + kTile * pitch<D>();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int bh = blockIdx.x / tiles, b = bh / a.H, h = bh % a.H, hk = h / a.g;
  const int r0 = (tiles - 1 - blockIdx.x % tiles) * kTile;
  const int len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
  auto row = [&](const void* base, const Strides& s, int head, int n) -> const T* {
    return n < len ? static_cast<const T*>(base) + b * s.b + head * s.h + n * s.n : nullptr;
  };
  load_tile<T, D>(Qs, [&](int r) { return row(a.q, a.sq, h, r0 + r); });
  load_tile<T, D>(Gs, [&](int r) { return row(a.dy, a.sdy, h, r0 + r); });
  float lse[4], del[4], o[4][D / 16];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int n = r0 + 4 * ty + x;
    const bool live = n < len;
    lse[x] = live ? a.lse[(int64_t)bh * a.N + n] : 0.f;
    del[x] = live ? a.delta[(int64_t)bh * a.N + n] : 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[x][c] = 0.f;
  }
  const KeyBlocks kb = key_blocks(r0, min(len, r0 + kTile) - 1, a.window, a.sinks, kTile);
  for (int n = 0; n < kb.count(); ++n) {
    const int j0 = kb.block(n) * kTile;
    __syncthreads();
    load_tile<T, D>(Ks, [&](int r) { return row(a.k, a.sk, hk, j0 + r); });
    load_tile<T, D>(Vs, [&](int r) { return row(a.v, a.sv, hk, j0 + r); });
    __syncthreads();
    float s[4][4], t[4][4];
    scores<D>(Qs, Ks, s);
    scores<D>(Gs, Vs, t);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int pos = r0 + 4 * ty + x;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        const bool see = pos < len && sees(pos, j, a.window, a.sinks);
        Ps[(4 * ty + x) * kPs + tx + 16 * c] =
            see ? expf(s[x][c] * a.scale - lse[x]) * (t[x][c] - del[x]) * a.scale : 0.f;
      }
    }
    __syncwarp();
    accumulate<D>(Ps, Ks, o);
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int n = r0 + 4 * ty + x;
    if (n < a.N) store_cols<T, D>(static_cast<T*>(a.dq) + b * a.sdq.b + h * a.sdq.h + n * a.sdq.n, o[x]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_dkv_simt_kernel(const AttendArgs a, int tiles) {
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + kTile * pitch<D>();
  float* Qs = Vs + kTile * pitch<D>();
  float* Gs = Qs + kTile * pitch<D>();
  float* Ps = Gs + kTile * pitch<D>();   // [key][query]
  float* Ds = Ps + kTile * kPs;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int bk = blockIdx.x / tiles, b = bk / a.Hkv, hk = bk % a.Hkv;
  const int j0 = (int)(blockIdx.x % tiles) * kTile;   // the sinks' tile, the longest, first
  const int len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
  auto row = [&](const void* base, const Strides& s, int head, int n) -> const T* {
    return n < len ? static_cast<const T*>(base) + b * s.b + head * s.h + n * s.n : nullptr;
  };
  load_tile<T, D>(Ks, [&](int r) { return row(a.k, a.sk, hk, j0 + r); });
  load_tile<T, D>(Vs, [&](int r) { return row(a.v, a.sv, hk, j0 + r); });
  float ok[4][D / 16], ov[4][D / 16];
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) ok[x][c] = ov[x][c] = 0.f;
  const int64_t last = j0 < a.sinks ? len : (int64_t)j0 + kTile - 1 + a.window;
  const int i_end = (int)(last < len ? last : len);   // queries j0 .. i_end - 1 may see the tile
  for (int h = hk * a.g; h < (hk + 1) * a.g; ++h) {
    const int64_t rows = ((int64_t)b * a.H + h) * a.N;
    for (int i0 = j0; i0 < i_end; i0 += kTile) {
      __syncthreads();
      load_tile<T, D>(Qs, [&](int r) { return row(a.q, a.sq, h, i0 + r); });
      load_tile<T, D>(Gs, [&](int r) { return row(a.dy, a.sdy, h, i0 + r); });
      __syncthreads();
      float s[4][4], t[4][4];
      scores<D>(Ks, Qs, s);
      scores<D>(Vs, Gs, t);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = i0 + tx + 16 * c;
        const float lse = i < len ? a.lse[rows + i] : 0.f, del = i < len ? a.delta[rows + i] : 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = j0 + 4 * ty + x;
          const bool see = i < len && sees(i, j, a.window, a.sinks);
          const float p = see ? expf(s[x][c] * a.scale - lse) : 0.f;
          Ps[(4 * ty + x) * kPs + tx + 16 * c] = p;
          Ds[(4 * ty + x) * kPs + tx + 16 * c] = see ? p * (t[x][c] - del) * a.scale : 0.f;
        }
      }
      __syncwarp();
      accumulate<D>(Ps, Gs, ov);
      accumulate<D>(Ds, Qs, ok);
    }
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int n = j0 + 4 * ty + x;
    if (n >= a.N) continue;
    store_cols<T, D>(static_cast<T*>(a.dk) + b * a.sdk.b + hk * a.sdk.h + n * a.sdk.n, ok[x]);
    store_cols<T, D>(static_cast<T*>(a.dv) + b * a.sdv.b + hk * a.sdv.h + n * a.sdv.n, ov[x]);
  }
}

// ---- launches ------------------------------------------------------------------

template <typename K>
cudaError_t run(K kernel, int64_t blocks, size_t smem, const AttendArgs& a, int tiles,
                cudaStream_t s) {
  if (blocks <= 0 || blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)blocks, kThreads, smem, s>>>(a, tiles);
  return cudaGetLastError();
}

template <int D>
constexpr size_t tile_bytes(int row_tiles, int score_tiles) {
  return sizeof(float) * kTile * ((size_t)row_tiles * pitch<D>() + (size_t)score_tiles * kPs);
}

template <typename T, int D>
cudaError_t forward(const AttendArgs& a, cudaStream_t s) {
  const int tiles = (a.N + kTile - 1) / kTile;
  return run(attend_simt_kernel<T, D, false>, (int64_t)a.B * a.H * tiles, tile_bytes<D>(3, 1), a,
             tiles, s);
}
template <typename T, int D>
cudaError_t backward(const AttendArgs& a, cudaStream_t s) {
  const int tiles = (a.N + kTile - 1) / kTile;
  const cudaError_t e = run(window_dq_simt_kernel<T, D>, (int64_t)a.B * a.H * tiles,
                            tile_bytes<D>(4, 1), a, tiles, s);
  if (e != cudaSuccess) return e;
  return run(window_dkv_simt_kernel<T, D>, (int64_t)a.B * a.Hkv * tiles, tile_bytes<D>(4, 2), a,
             tiles, s);
}
template <typename T, int D>
cudaError_t pages(const AttendArgs& a, cudaStream_t s) {
  const int64_t tiles = paged_tiles(a, kTile);
  return run(attend_simt_kernel<T, D, true>, tiles * a.Hkv, tile_bytes<D>(3, 1), a, (int)tiles, s);
}

template <int D>
struct Launch {
  static cudaError_t fwd(const AttendArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? forward<__nv_bfloat16, D>(a, s) : forward<float, D>(a, s);
  }
  static cudaError_t bwd(const AttendArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? backward<__nv_bfloat16, D>(a, s) : backward<float, D>(a, s);
  }
  static cudaError_t paged(const AttendArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? pages<__nv_bfloat16, D>(a, s) : pages<float, D>(a, s);
  }
};

}  // namespace

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
  return a.d == 32 ? Launch<32>::fwd(a, bf16, s)
         : a.d == 64 ? Launch<64>::fwd(a, bf16, s) : Launch<128>::fwd(a, bf16, s);
}
cudaError_t launch_window_bwd_simt(const AttendArgs& a, bool bf16, cudaStream_t s) {
  return a.d == 32 ? Launch<32>::bwd(a, bf16, s)
         : a.d == 64 ? Launch<64>::bwd(a, bf16, s) : Launch<128>::bwd(a, bf16, s);
}
cudaError_t launch_paged_simt(const AttendArgs& a, bool bf16, cudaStream_t s) {
  return a.d == 32 ? Launch<32>::paged(a, bf16, s)
         : a.d == 64 ? Launch<64>::paged(a, bf16, s) : Launch<128>::paged(a, bf16, s);
}

}  // namespace elsaa
