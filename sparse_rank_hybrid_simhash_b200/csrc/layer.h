// Host-side problem descriptions of the operators next to ELSAA (norm and
// rotation, window attention, the paged cache) and the launchers each .cu file
// provides.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/elsaa.h"

namespace elsaa {

// Element strides of a [batch, heads, tokens, d] tensor (d contiguous).
struct Strides {
  int64_t b, h, n;
};

// Head of every workspace, zeroed once by the caller: the error word, and the
// arrival counters of work cut between CTAs (which the calls leave at zero).
constexpr size_t kHeadBytes = 8192;
constexpr size_t kCounters = 256;   // byte offset of the counters (at most 1984)

// ---- norm and rotation -------------------------------------------------------

// Most blocks that leave a partial sum of a weight's gradient (queries' and
// keys' together): a fixed number, so the summation order is fixed.
constexpr int kRotaryPartials = 444;   // 3 x 148: all resident

struct RotaryArgs {
  const void *q, *k;
  void *qo, *ko;              // outputs (forward), dq and dk (backward)
  const void *dqo, *dko;      // backward
  Strides sq, sk, sqo, sko, sdqo, sdko;
  const int32_t* positions;   // [B, N] or null
  const float* table;         // [max_pos, rot / 2, 2]
  const float *wq, *wk;       // [d] or null
  float *dwq, *dwk;           // [d] or null
  float* partials;            // [kRotaryPartials][d]
  uint32_t* err;
  int B, H, Hkv, N, rot, norm, max_pos;
  float eps;
  // the write into pages
  const void* v;
  Strides sv;
  void *k_pages, *v_pages;
  Strides skp, svp;           // (page, head, slot)
  const int32_t *page_table, *starts, *lengths;
  int seqs, page_size, pages, table_width;
};

cudaError_t launch_rotary_forward(const RotaryArgs& a, int d, bool bf16, bool interleaved,
                                  cudaStream_t s);
cudaError_t launch_rotary_backward(const RotaryArgs& a, int d, bool bf16, bool interleaved,
                                   cudaStream_t s);
cudaError_t launch_paged_write(const RotaryArgs& a, int d, bool bf16, bool interleaved,
                               cudaStream_t s);

// ---- attention ---------------------------------------------------------------

struct AttendArgs {
  const void *q, *k, *v;
  void* y;
  float* lse;                 // [B, H, N] (window forward, backward)
  const void* dy;
  void *dq, *dk, *dv;
  Strides sq, sk, sv, sy, sdy, sdq, sdk, sdv;   // pages: sk, sv are (page, head, slot)
  const int32_t* lengths;     // window: [B] or null; pages: [S]
  int B, H, Hkv, N, d, g;     // g = H / Hkv
  int window;                 // INT32_MAX: no limit
  int sinks;
  float scale;
  uint32_t* err;
  uint32_t* counters;         // [CTAs][8 warps], or [CTAs]
  float* delta;               // backward: the row statistics and partials
  // pages
  const int32_t *page_table, *starts;
  int seqs, rows, page_size, pages, table_width;
  char* scratch;              // split partials
};

// CUDA-core kernels: fp32, and bf16 at d = 32.
cudaError_t launch_window_delta(const AttendArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_window_fwd_simt(const AttendArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_window_bwd_simt(const AttendArgs& a, bool bf16, cudaStream_t s);
// (a.delta: window_simt_scratch_bytes of workspace, row statistics and partials of shared tiles)
// (window: INT32_MAX for no limit)
size_t window_simt_scratch_bytes(int d, int64_t B, int64_t H, int64_t Hkv, int N, int window, int sinks);
cudaError_t launch_paged_simt(const AttendArgs& a, bool bf16, cudaStream_t s);

// tcgen05 kernels: bf16, d = 64 or 128.
bool attend_tc_supported(int d, bool bf16);
cudaError_t launch_window_fwd_tc(const AttendArgs& a, cudaStream_t s);
// (a.delta: window_tc_scratch_bytes of workspace)
cudaError_t launch_window_bwd_tc(const AttendArgs& a, cudaStream_t s);
cudaError_t launch_paged_tc(const AttendArgs& a, cudaStream_t s);
// Workspace bytes of launch_window_bwd_tc: row statistics, and partials of cut tiles.
size_t window_tc_scratch_bytes(int d, int64_t B, int64_t H, int64_t N);
// Workspace bytes of launch_paged_tc's partial rows.
size_t paged_scratch_bytes(int d, int64_t rows, int g);
// A few rows a sequence (decoding), bf16.
bool paged_decode_supported(int d, bool bf16, int64_t rows, int seqs, int g);
cudaError_t launch_paged_decode(const AttendArgs& a, cudaStream_t s);

// A 128-byte-swizzled bf16 tensor map of a [n3, n2, n1, d] tensor with the
// given element strides (d contiguous) and box.
cudaError_t make_map_4d(CUtensorMap* map, const void* base, uint64_t d, uint64_t n1, uint64_t n2,
                        uint64_t n3, int64_t s1, int64_t s2, int64_t s3, const uint32_t* box);

}  // namespace elsaa
