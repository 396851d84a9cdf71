// tensor_map.cu -- TMA descriptors of arrays of rows, encoded on the host through the driver's entry point.
#include "tensor_map.h"

#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"

namespace sd {

namespace {

struct Encoder {
    std::mutex mu;
    PFN_cuTensorMapEncodeTiled fn = nullptr;
};
Encoder g_encoder;

cudaError_t encoder(PFN_cuTensorMapEncodeTiled* out) {
    std::lock_guard<std::mutex> lock(g_encoder.mu);
    if (g_encoder.fn == nullptr) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
        g_encoder.fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled>(fn);
    }
    *out = g_encoder.fn;
    return cudaSuccess;
}

}  // namespace

cudaError_t encode_rows_map(CUtensorMap* m, const void* base, bool bytes, long heads, long rows, int x, int y, int z,
                            bool swizzle) {
    PFN_cuTensorMapEncodeTiled fn;
    const cudaError_t e = encoder(&fn);
    if (e != cudaSuccess) return e;
    const cuuint64_t esz = bytes ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {kHeadDim * esz, kHeadDim * esz * (cuuint64_t)heads};
    const cuuint32_t box[3] = {(cuuint32_t)x, (cuuint32_t)y, (cuuint32_t)z};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult res = fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return res == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace sd
