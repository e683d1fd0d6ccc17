// Host side of TMA: tensor-map encoding through the driver entry point
// (fetched once per process through the runtime, so the library links no
// driver library and loads on a machine without a GPU).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kernels.h"

namespace orthrus {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        else
            cudaGetLastError();
    });
    return fn;
}

}  // namespace

static bool encode_sw128(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
                         const uint64_t *strides, const uint32_t *box)
{
    auto fn = encode_fn();
    if (!fn || rank < 1 || rank > 5) return false;
    cuuint64_t d[5], st[4];
    cuuint32_t b[5], e[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        e[i] = 1;
        if (i + 1 < rank) st[i] = strides[i];
    }
    return fn(m, type, (cuuint32_t)rank, const_cast<void *>(base), d, st, b,
              e, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_bf16_sw128(CUtensorMap *m, int rank, const void *base, const uint64_t *dims,
                       const uint64_t *strides, const uint32_t *box)
{
    return encode_sw128(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box);
}

bool encode_u8_sw128(CUtensorMap *m, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                     const uint32_t *box)
{
    return encode_sw128(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, base, dims, strides, box);
}

}  // namespace orthrus
