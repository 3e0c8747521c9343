// Attention of a few new rows a sequence over a paged cache (decoding: bf16, at most
// 16 (token, head of the group) rows a sequence on average).
//
// Bound: HBM, each key and value of the contexts read once; the products of 16 rows
// are a hundredth of what the bytes cost.  So the work per byte is kept small and many
// loads in flight: a warp is a pipeline of its own with 16 keys a stage (K and V
// rows by cp.async into 16-byte chunks swizzled by their row, no barrier but the
// warp's), four warps a CTA take the 16-key quarters of each 64-key block, two or three
// CTAs an SM, 128 KB in flight.  Scores, softmax and output stay in registers: S = Q K^T
// and O += P V by 16 x 8 x 16 tensor instructions (a 128-row tcgen05 tile holds 8 to
// 16 live rows here, its S, P and O go through TMEM with a barrier each way, and the
// blocks that wait there take the ring's slots: 50 % of the bandwidth at contexts of
// 1000 to 5000 keys).  The row reference grows only by more than 2^8.  P is rounded to bf16,
// V's type, for its product (half a step of a probability, random: the error of y against 64
// bits 0.0021 to 0.0023 of its norm, y's own rounding alone 0.0016); P in two bf16 parts
// would leave that alone, at 416 -> 444 us for 64 sequences over up to 16k keys: not taken.
// Measured against that kernel: 64 sequences over up to 16k keys (32 query and 8 key
// heads of d = 128) 361 against 398 us, 93 % of the copy bandwidth; 87 over a window of
// 1318 151 against 214; one sequence 13.6 against 18.5.  A long chunk among single
// tokens comes here too where the average stays small, which bounds the number of tiles
// but not their keys: each walks its sequence's context, out of L2 behind the first.  900
// tokens beside 63 single ones, 8 heads of d = 128 over contexts of 4000: 293 us, against
// 172 for the tokens and 54 for the chunk in two calls.
//
// Items (row tile, key head) are cut into equal runs of 64-key blocks (paged_runs.cuh);
// the four warps' rows are joined in shared memory at an item's end, cut items by the
// last CTA to get there, in the CTAs' order.
#include <math.h>

#include "internal.h"
#include "paged_runs.cuh"
#include "tc_common.cuh"

namespace elsaa {
namespace {

using namespace tc;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16, kKeys = 16;        // rows of a tile, keys of a stage
constexpr float kGrow = 8.0f;                // log2 of the growth that rescales O
constexpr int kAhead = 4;                    // page lookups in flight

template <int D>
struct Lay {
  static constexpr int kRow = D * 2;                      // bytes of a row
  static constexpr int kStage = 2 * kKeys * kRow;         // K and V
  static constexpr int kStages = D == 128 ? 3 : D == 64 ? 4 : 8;
  static constexpr int kCtas = D == 128 ? 2 : 3;          // an SM
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kPitch = D + 4;                    // floats of a joined row
  static constexpr int kDyn = kWarps * kWarpBytes;
  static_assert(kWarps * kRows * kPitch * 4 <= kDyn, "the joined rows reuse the stages");
};

ELSAA_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
ELSAA_DEV void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
ELSAA_DEV void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
ELSAA_DEV void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
ELSAA_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
ELSAA_DEV uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Where chunk c of row r lies in its row: the eight rows that an ldmatrix reads at one
// chunk fall into different banks.
template <int D>
ELSAA_DEV int place(int c, int r) { return D == 32 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); }

template <int D>
__global__ void __launch_bounds__(kThreads, Lay<D>::kCtas) paged_decode_kernel(const AttendArgs a, float scale_log2) {
  using L = Lay<D>;
  constexpr int ST = L::kStages, CH = D / 8;   // 16-byte chunks of a row
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Run run;
  __shared__ float ml[kWarps][2][kRows];
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, part = lane & 3;
  const uint32_t base = smem_u32(smem) + warp * L::kWarpBytes;
  const int g = a.g, tt = kRows / g;
  if (warp == 0) {
    const Run c = find_run(a, tt, blockIdx.x, gridDim.x);
    if (lane == 0) run = c;
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
    const int rows = min(tt, tokens - tile * tt) * g;   // live rows: token tile tt + r / g, head hk g + r % g
    auto at_row = [&](const Strides& s, int r) -> int64_t {
      return (int64_t)(start + tile * tt + r / g) * s.n + (int64_t)(hk * g + r % g) * s.h;
    };

    // ---- the warp's keys of block n: rows j0 .. j0 + 15 ----
    // the page of this lane's key (lanes 0 .. 15); -1: not read (no row sees it, or no page)
    auto lookup = [&](int n) -> int {
      if (n >= n1 || lane >= kKeys) return -1;
      const int j = it.kb.block(n) * kBlk + warp * kKeys + lane;
      if (j > it.p_hi || !(j < a.sinks || (int64_t)j > (int64_t)it.p_lo - a.window)) return -1;
      return page_of(a, b, j);
    };
    auto load = [&](int n, int page) {
      if (n < n1) {
        const uint32_t dst = base + (uint32_t)((n - n0) % ST) * L::kStage;
        const int j0 = it.kb.block(n) * kBlk + warp * kKeys;
        const int slot0 = j0 % a.page_size;   // (16 keys lie in one page: its size is a multiple of 16)
#pragma unroll
        for (int x = 0; x < kKeys * CH / 32; ++x) {
          const int r = (x * 32 + lane) / CH, c = (x * 32 + lane) % CH;
          const int pg = __shfl_sync(0xffffffffu, page, r);
          const uint32_t to = dst + r * L::kRow + (place<D>(c, r) << 4);
          const int64_t p = pg >= 0 ? pg : 0;
          const int64_t in = (int64_t)(slot0 + r);
          const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + p * a.sk.b +
                                   (int64_t)hk * a.sk.h + in * a.sk.n + c * 8;
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + p * a.sv.b +
                                   (int64_t)hk * a.sv.h + in * a.sv.n + c * 8;
          cp_async16(to, k, pg >= 0 ? 16 : 0);   // (zeros where nothing is read)
          cp_async16(to + kKeys * L::kRow, v, pg >= 0 ? 16 : 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int x = 0; x < ST - 1; ++x) load(n0 + x, lookup(n0 + x));
    int ahead[kAhead];   // pages of the next loads (a lookup takes about as long as two blocks)
#pragma unroll
    for (int x = 0; x < kAhead; ++x) ahead[x] = lookup(n0 + ST - 1 + x);

    // Q as the A operand of every K step (rows quad and quad + 8)
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = quad + 8 * h;
      const uint32_t* q = r < rows ? reinterpret_cast<const uint32_t*>(
                                         static_cast<const __nv_bfloat16*>(a.q) + at_row(a.sq, r))
                                   : nullptr;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][h] = q ? q[8 * k + part] : 0u;
        qf[k][h + 2] = q ? q[8 * k + 4 + part] : 0u;
      }
    }
    int pos[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) pos[h] = quad + 8 * h < rows ? it.p_lo + (quad + 8 * h) / g : -1;
#pragma unroll
    for (int t = 0; t < D / 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;

    for (int n = n0; n < n1; ++n) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      const uint32_t ks = base + (uint32_t)((n - n0) % ST) * L::kStage, vs = ks + kKeys * L::kRow;
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
      {
        const int r = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t kf[4];
          ldsm4(ks + r * L::kRow + (place<D>(2 * k + ((lane >> 3) & 1), r) << 4), kf);
          mma16816(s[0], qf[k], kf[0], kf[1]);
          mma16816(s[1], qf[k], kf[2], kf[3]);
        }
      }
      // the row's scores: elements (t, 2 h + e) are keys j + 8 t + e of row quad + 8 h
      const int j = it.kb.block(n) * kBlk + warp * kKeys + 2 * part;
      float top[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[t][2 * h + e];
            x = sees(pos[h], j + 8 * t + e, a.window, a.sinks) ? x * scale_log2 : -INFINITY;
            top[h] = fmaxf(top[h], x);
          }
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] + kGrow || top[1] > m[1] + kGrow)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool grow = top[h] > m[h] + kGrow;
          const float f = grow ? ex2(m[h] - top[h]) : 1.f;
          if (grow) m[h] = top[h];
          l[h] *= f;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) o[t][2 * h] *= f, o[t][2 * h + 1] *= f;
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2(s[t][2 * h] - ref), p1 = ex2(s[t][2 * h + 1] - ref);
          l[h] += p0 + p1;
          pf[2 * t + h] = pack2(p0, p1);
        }
      }
      {
        const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t vf[4];
          ldsm4_t(vs + r * L::kRow + (place<D>(2 * c + (lane >> 4), r) << 4), vf);
          mma16816(o[2 * c], pf, vf[0], vf[1]);
          mma16816(o[2 * c + 1], pf, vf[2], vf[3]);
        }
      }
      __syncwarp();   // the stage has been read by every lane
      load(n + ST - 1, ahead[0]);
#pragma unroll
      for (int x = 0; x + 1 < kAhead; ++x) ahead[x] = ahead[x + 1];
      ahead[kAhead - 1] = lookup(n + ST - 1 + kAhead);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the four warps' rows joined ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (part == 0) ml[warp][0][quad + 8 * h] = m[h], ml[warp][1][quad + 8 * h] = l[h];
    }
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = quad + 8 * h;
      float top = ml[0][0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, ml[w][0][r]);
      const float f = m[h] > -INFINITY ? ex2(m[h] - top) : 0.f;
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
        *reinterpret_cast<float2*>(join + (warp * kRows + r) * L::kPitch + 8 * t + 2 * part) =
            make_float2(o[t][2 * h] * f, o[t][2 * h + 1] * f);
    }
    __syncthreads();
    const bool whole = n0 == 0 && n1 == nblk;
    const int slot = (int)blockIdx.x * 2 + (order > 0 ? 1 : 0);
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      float top = ml[0][0][r], sum = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, ml[w][0][r]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(join + (w * kRows + r) * L::kPitch + c);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        if (ml[w][0][r] > -INFINITY) sum += ml[w][1][r] * ex2(ml[w][0][r] - top);
      }
      if (whole) {
        const float inv = sum > 0.f ? 1.0f / sum : 0.f;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at_row(a.sy, r) + c) =
            make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
      } else {
        *reinterpret_cast<float4*>(partial_o<kRows>(a, D, slot, r) + c) = v;
        if (c == 0) *partial_ml<kRows>(a, D, slot, r) = make_float2(top, sum);
      }
    }
    if (!whole) {
      const Ctas ct = ctas_of(at - off, nblk, run.per);
      __threadfence();
      __syncthreads();
      if (tid == 0) last = atomicAdd(a.counters + ct.first, 1u) == (uint32_t)(ct.last - ct.first) ? 1 : 0;
      __syncthreads();
      if (last) {
        __threadfence();
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
          const int r = x / (D / 4), c = x % (D / 4) * 4;
          auto slot_of = [&](int i) { return 2 * i + (i == ct.first ? ct.slot0 : 0); };
          float top = -INFINITY, sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int i = ct.first; i <= ct.last; ++i)
            top = fmaxf(top, __ldcg(partial_ml<kRows>(a, D, slot_of(i), r)).x);
#pragma unroll 8
          for (int i = ct.first; i <= ct.last; ++i) {
            const float2 pm = __ldcg(partial_ml<kRows>(a, D, slot_of(i), r));
            const float4 u = __ldcg(reinterpret_cast<const float4*>(partial_o<kRows>(a, D, slot_of(i), r) + c));
            const float f = pm.x > -INFINITY ? ex2(pm.x - top) : 0.f;
            sum += pm.y * f;
            v.x += u.x * f, v.y += u.y * f, v.z += u.z * f, v.w += u.w * f;
          }
          const float inv = sum > 0.f ? 1.0f / sum : 0.f;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at_row(a.sy, r) + c) =
              make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
        }
        if (tid == 0) a.counters[ct.first] = 0;
      }
    }
    __syncthreads();   // the stages and ml may be written again
    left -= n1 - n0;
    at += n1 - n0;
    off = 0;
    if (++hk == a.Hkv) hk = 0, ++tile;
  }
}

template <int D>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(
      paged_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kDyn);
  if (e != cudaSuccess) return e;
  static_assert(148 * Lay<D>::kCtas <= kRuns, "partials of every CTA");
  paged_decode_kernel<D><<<148 * Lay<D>::kCtas, kThreads, Lay<D>::kDyn, s>>>(a, a.scale * 1.4426950408889634f);
  return cudaGetLastError();
}

}  // namespace

bool paged_decode_supported(int d, bool bf16, int64_t rows, int seqs, int g) {
  return bf16 && (d == 32 || d == 64 || d == 128) && paged_tile_rows(rows, seqs, g) == kRows;
}

cudaError_t launch_paged_decode(const AttendArgs& a, cudaStream_t s) {
  return a.d == 32 ? launch<32>(a, s) : a.d == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace elsaa
