// Host side of the TMA copies: 2-D tensor maps over [rows, 64] or [rows, 128]
// bf16 matrices (a box of one row of 64 columns, 128-byte swizzle) for the
// attention kernels' row gathers, and 3-D maps over [units, N, d] bf16 with
// 8-column boxes for the RACE slab kernels, and 4-D maps of strided tensors for
// the window and paged attention; encoded through the driver entry
// point the runtime resolves (no direct driver-API calls).
#include <cudaTypedefs.h>
#include <mutex>

#include "internal.h"
#include "layer.h"

namespace elsaa {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The encoder wants a context current on the calling thread.  A thread whose first call into
// CUDA this is (a server's worker, the thread that autograd runs a backward on) has none until
// the runtime is initialised there, which setting its device does (once a thread and device;
// no work on a stream, so captures go on).
cudaError_t bind_thread() {
  static thread_local int bound = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != bound && (e = cudaSetDevice(dev)) == cudaSuccess) bound = dev;
  return e;
}

// The encoder, or null where there is none (*e: why).
PFN_cuTensorMapEncodeTiled_v12000 encoder(cudaError_t* e) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  *e = fn == nullptr ? cudaErrorNotSupported : bind_thread();
  return *e == cudaSuccess ? fn : nullptr;
}
}  // namespace

cudaError_t make_row_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t width) {
  cudaError_t e;
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder(&e);
  if (fn == nullptr) return e;
  const cuuint64_t dims[2] = {width, rows};
  const cuuint64_t strides[1] = {width * 2};
  const cuuint32_t box[2] = {64, 1};
  const cuuint32_t elem[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_slab_map(CUtensorMap* map, const void* base, uint64_t units, uint64_t n,
                          uint64_t d, uint32_t box_rows) {
  cudaError_t e;
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder(&e);
  if (fn == nullptr) return e;
  const cuuint64_t dims[3] = {d, n, units};
  const cuuint64_t strides[2] = {d * 2, n * d * 2};
  const cuuint32_t box[3] = {8, box_rows, 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_map_4d(CUtensorMap* map, const void* base, uint64_t d, uint64_t n1, uint64_t n2,
                        uint64_t n3, int64_t s1, int64_t s2, int64_t s3, const uint32_t* box) {
  cudaError_t e;
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder(&e);
  if (fn == nullptr) return e;
  const cuuint64_t dims[4] = {d, n1, n2, n3};
  const cuuint64_t strides[3] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2, (cuuint64_t)s3 * 2};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                        strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace elsaa
