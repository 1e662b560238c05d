// Host-side TMA tensor-map encoding through the driver entry point, so the
// library needs no link against libcuda.
#include <atomic>

#include "sm100.cuh"

namespace kvattn {

namespace {
// looked up once; where that fails, the next call looks again
std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode{nullptr};
}  // namespace

CUresult encode_tiled(CUtensorMap *map, CUtensorMapDataType dtype, cuuint32_t rank, void *base,
                      const cuuint64_t *dims, const cuuint64_t *strides_bytes, const cuuint32_t *box,
                      CUtensorMapSwizzle swizzle)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = g_encode.load(std::memory_order_relaxed);
    if (!encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess) {
            cudaGetLastError();      // a failed query leaves its error as the last error: clear it
            return CUDA_ERROR_NOT_SUPPORTED;
        }
        if (q != cudaDriverEntryPointSuccess)
            return CUDA_ERROR_NOT_SUPPORTED;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        g_encode.store(encode, std::memory_order_relaxed);
    }
    const cuuint32_t elem_strides[5] = {1, 1, 1, 1, 1};
    return encode(map, dtype, rank, base, dims, strides_bytes, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace kvattn
