// Host side of rows_map.cuh.
#include "rows_map.cuh"

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>

namespace la {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  auto fn = encoder();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn != nullptr &&
         fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_rows_map(CUtensorMap* m, const void* base, int W, int heads, long ld, int N, int B) {
  const cuuint64_t dims[4] = {(cuuint64_t)W, (cuuint64_t)heads, (cuuint64_t)N, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)W * 2, (cuuint64_t)ld * 2, (cuuint64_t)N * ld * 2};
  const cuuint32_t box[4] = {64, 1, 128, 1};
  return encode(m, base, 4, dims, strides, box);
}

bool make_state_map(CUtensorMap* m, const void* base, int M, int D, long n) {
  const cuuint64_t dims[3] = {(cuuint64_t)M, (cuuint64_t)D, (cuuint64_t)n};
  const cuuint64_t strides[2] = {(cuuint64_t)M * 2, (cuuint64_t)D * M * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  return encode(m, base, 3, dims, strides, box);
}

}  // namespace la
