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
// One lane of the warp (always the same one), by the instruction that tells the
// compiler so: operands of the tensor-core instructions live in uniform registers,
// and behind a plain lane test each is moved there by itself (a 128 x 128 x 128
// product took 1400 cycles to issue instead of about 100).
ELSAA_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// A value that is the same in every lane, known to be.
ELSAA_DEV uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Low words of the shared-memory descriptors of a tile at `saddr` (128-byte
// swizzle, 8-row groups 1024 bytes apart): read by rows (K-major), or by columns
// (the next 64 of them kAtom further on).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
ELSAA_DEV uint32_t row_desc(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
ELSAA_DEV uint32_t col_desc(uint32_t saddr) { return (saddr >> 4) | ((kAtom >> 4) << 16); }

// D[tmem] (+)= A B of descriptors' low words (mma_bf16_ss, _ts); the elected lane.
ELSAA_DEV void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
ELSAA_DEV void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}

// 128 x N product of two K-major tiles over D.
template <int D, int N = kBlock>
ELSAA_DEV void mma_tiles(uint32_t d_tmem, uint32_t ad, uint32_t bd) {
  constexpr uint32_t id = idesc_bf16(128, N, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((uint32_t)(kk >> 2) * kAtom + (uint32_t)(kk & 3) * 32) >> 4;
    mma_ss(d_tmem, ad + off, bd + off, id, kk > 0 ? 1u : 0u);
  }
}

// A place in a ring of N slots, and the parity of its phase there.
template <int N>
struct RingPos {
  uint32_t slot = 0, phase = 0;
  ELSAA_DEV void next() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

// The whole warp waits for the barrier's phase; bounded (ERR_TIMEOUT).
ELSAA_DEV bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err) {
  for (uint32_t i = 0; i < kMaxSpin; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  raise_error(err, ERR_TIMEOUT);
  return false;
}

// One arrival for the warp: what its lanes did before is ordered by the warp's
// barrier (32 arrivals at one address would queue up).
ELSAA_DEV void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
ELSAA_DEV void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
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
