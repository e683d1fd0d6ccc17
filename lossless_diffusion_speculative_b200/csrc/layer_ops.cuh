// Element types and small helpers shared by the layer operators (rmsnorm.cu,
// rope.cu, paged_attn.cu, fp8_matmul.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace orthrus {

template <> __device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Two values packed into (unpacked from) one 32-bit word of a 16-bit type.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Eight consecutive values at a 16-byte aligned address, as loaded (not yet converted), so that loads can be
// in flight without holding fp32 registers.
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) / 2];
};
template <typename T> __device__ __forceinline__ Raw8<T> load_raw(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
template <typename T> __device__ __forceinline__ void unpack8(const Raw8<T> &r, float2 (&x)[4])
{
    if constexpr (sizeof(T) == 2) {
        x[0] = unpack2<T>(r.w[0].x), x[1] = unpack2<T>(r.w[0].y);
        x[2] = unpack2<T>(r.w[0].z), x[3] = unpack2<T>(r.w[0].w);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[2 * i] = make_float2(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
            x[2 * i + 1] = make_float2(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
        }
    }
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float2 (&x)[4])
{
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2<T>(x[0].x, x[0].y), pack2<T>(x[1].x, x[1].y), pack2<T>(x[2].x, x[2].y), pack2<T>(x[3].x, x[3].y));
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
}

// Host: the size of an orthrus_dtype's element, 0 for anything else.
inline int elem_size(int dtype)
{
    return dtype == ORTHRUS_BF16 || dtype == ORTHRUS_F16 ? 2 : dtype == ORTHRUS_F32 ? 4 : 0;
}

// Host: launch with programmatic stream serialisation: the grid may become
// resident while the previous kernel of the stream drains; its griddepcontrol.wait
// holds it back before the first access to memory.
template <class... P, class... A>
inline cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace orthrus
