// Pieces shared by the tcgen05 kernels of the window and paged attention.
#pragma once

#include "attend.cuh"
#include "tc_common.cuh"

namespace elsaa {
namespace tc {

constexpr int kBlock = 128;              // rows of a tile, keys of a block
constexpr uint32_t kAtom = 128 * 128;    // 128 rows x 64 bf16
constexpr int kMaxCtas = 160;            // CTAs of a call cut into runs (the workspace holds their partials)

// The next of `items` window items for a CTA that has ended one (its first is its own
// number): whoever is free takes the next, longest first, so that the CTAs end together.
// (Every gridDim.x-th item each: a padded batch of 4 x 16 heads of d = 128, 4001 tokens,
// window 1000, forward 165 and dq 205 us, 132 and 170 so; 16384 tokens, 32 and 8 heads,
// window 4096, forward 925 -> 890.)  The last of the `items` calls leaves the counter at zero.
ELSAA_DEV int64_t next_item(uint32_t* counter, int64_t items) {
  const uint32_t n = atomicAdd(counter, 1u);
  if (n == (uint32_t)(items - 1)) *counter = 0;
  return (int64_t)gridDim.x + n;
}

// x[s] of a pair that stays in registers.
template <typename T>
ELSAA_DEV T pick(const T (&x)[2], int s) { return s ? x[1] : x[0]; }

// 2^x on the special-function unit (approximate, flushes denormals).
ELSAA_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x of a pair on the FMA pipe, relative error below 2.4e-7 (ex2.approx: 2^-22):
// x = n + f with n the nearest whole number (Cody and Waite's reduction, by adding
// and taking off 1.5 2^23) and a degree-5 polynomial of f in [-1/2, 1/2], minimax in
// the relative error (Remez exchange).  x below -127 counts as -127, where n = x and f = 0:
// the last coefficient's bits (one unit over 1) less 127 in the exponent are 2^-149, so a
// masked score's probability is zero once it is bf16 and no value behind it enters the row,
// however large (at -125 a value of 2^127 came through as 4).  Between -127 and -126 the
// result is off by up to 2^-127.  NaN does not come out finite and small.
ELSAA_DEV void exp2_fma(float& x0, float& x1) {
  constexpr float kMagic = 12582912.0f;
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x0));   // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x1));
  float t0 = x0, t1 = x1;
  add2(t0, t1, kMagic, kMagic);
  float n0 = t0, n1 = t1;
  add2(n0, n1, -kMagic, -kMagic);
  fma2(n0, n1, -1.0f, -1.0f, x0, x1);   // f
  float p0 = 1.3276472454890609e-3f, p1 = p0;
  fma2(p0, p1, n0, n1, 9.675540961325169e-3f, 9.675540961325169e-3f);
  fma2(p0, p1, n0, n1, 5.550713092088699e-2f, 5.550713092088699e-2f);
  fma2(p0, p1, n0, n1, 2.4022120237350464e-1f, 2.4022120237350464e-1f);
  fma2(p0, p1, n0, n1, 6.931469440460205e-1f, 6.931469440460205e-1f);
  fma2(p0, p1, n0, n1, 1.0000001192092896f, 1.0000001192092896f);
  x0 = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
  x1 = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
}
// 2^x of pair i of an unrolled row.  MIX: one pair of four on the FMA pipe, the others on
// the special-function unit, which two warps a scheduler keep busy for 9.4 cycles a warp
// value.  Measured (8192 tokens, 32 heads, window 4096): forward 407 -> 382 us at d = 64,
// 434 -> 431 at d = 128; backward 974 -> 941 at d = 64, 1316 -> 1378 at d = 128, where the
// products are the bound and the longer chain costs (so not there).  Three of eight, or
// half of the pairs, are slower.
template <bool MIX>
ELSAA_DEV void exp2_pair(int i, float& x0, float& x1) {
  if (MIX && i % 4 == 1) {
    exp2_fma(x0, x1);
  } else {
    x0 = ex2(x0);
    x1 = ex2(x1);
  }
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
