// Pieces shared by the tcgen05 kernels of the window and paged attention.
#pragma once

#include "attend.cuh"
#include "tc_common.cuh"

namespace elsaa {
namespace tc {

constexpr int kBlock = 128;              // rows of a tile, keys of a block
constexpr uint32_t kAtom = 128 * 128;    // 128 rows x 64 bf16
constexpr int kMaxCtas = 160;            // CTAs of a call cut into runs (the workspace holds their partials)

// x[s] of a pair that stays in registers.
template <typename T>
ELSAA_DEV T pick(const T (&x)[2], int s) { return s ? x[1] : x[0]; }

// 2^x on the special-function unit (approximate, flushes denormals).
ELSAA_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
ELSAA_DEV void tma_load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// Registers of this thread, by whole warpgroups.
template <int N>
ELSAA_DEV void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
ELSAA_DEV void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

ELSAA_DEV void store32(__nv_bfloat16* p, const float* v) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * q + 2 * e], v[8 * q + 2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Columns <= x of 32.
ELSAA_DEV uint32_t upto_bits(int x) { return x < 0 ? 0u : x >= 31 ? ~0u : (2u << x) - 1u; }

}  // namespace tc
}  // namespace elsaa
