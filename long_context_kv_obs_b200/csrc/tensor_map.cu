// Tensor maps of the TMA loads.  cuTensorMapEncodeTiled is a driver call: it is looked up once, and wants
// a context on the calling thread, which a thread has only once it made a runtime call that binds one.
#include <cudaTypedefs.h>

#include <atomic>

#include "tc_sm100.cuh"

namespace kvc {
namespace tc {

bool bf16_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> entry{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 enc = entry.load();
  if (!enc) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    entry.store(enc);
  }
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  auto encode = [&] {
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  int dev = 0;                                  // perhaps the thread's first call: bind its device's context
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

}  // namespace tc
}  // namespace kvc
