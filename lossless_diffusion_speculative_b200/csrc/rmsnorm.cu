// RMS norm of rows with the residual's addition in front and an 8-bit output
// with scales behind it, and plain quantisation to the same 8-bit form.
//
//     s = x + r;  y = s * rsqrt(mean(s^2) + eps) * w
//     scale = max(max|y| / 448, 2^-126) per 128 columns;  value = e4m3(y / scale)
//
// One pass: a row's values stay in registers (fp32) between the sum of squares
// and the outputs, so each input is read and each output written once.  A row
// belongs to W warps (1..32), each lane holding NC chunks of 8 values; the sum
// of squares goes through shuffles and, for W > 1, shared memory.  A 128-column
// group lies within one warp's chunk of 256 columns: 16 lanes of 8 consecutive
// values on the vector path, or four strips of 32 lanes where rows are not
// 16-byte aligned (V = 1), so its maximum needs shuffles only.  HBM-bound.
#include <math.h>

#include "kernels.h"
#include "layer_ops.cuh"

namespace orthrus {

namespace {

struct NormArgs {
    const void *x, *residual, *weight;
    int64_t x_stride;
    void *sum_out, *out;
    uint8_t *out_fp8;
    float *out_scale;
    int T, H, W;                    // W: warps per row
    float eps;
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Maximum over 2 * o lanes; fmaxf drops a NaN operand.
__device__ __forceinline__ float lanes_max(float v, int o)
{
    for (; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax / 448.0f, 1.17549435e-38f); }

template <typename T, int V, int NC, bool NORM, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_kernel(const NormArgs p)
{
    __shared__ float part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // without the norm a row's warps need not share a block
    const int W = p.W;
    const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
    const int64_t row = unit / W;
    const int wr = (int)(unit - row * W);
    const bool live = row < p.T;
    const int H = p.H;
    sm100::pdl_trigger();
    sm100::pdl_wait();

    // column of value j of chunk c: chunk c of warp wr covers 256 columns
    auto col = [&](int c, int j) { return (c * W + wr) * 256 + (V == 8 ? lane * 8 + j : j * 32 + lane); };
    const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
    const T *r = static_cast<const T *>(p.residual) + row * H;
    float s[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] = 0.f;
        if (V == 8) {
            if (live && col(c, 0) < H) load8(x + col(c, 0), s[c]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (live && col(c, j) < H) s[c][j] = to_f32<T>(x[col(c, j)]);
        }
    }
    if (NORM && p.residual) {
        T *so = static_cast<T *>(p.sum_out) + row * H;
        float a[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (V == 8) {
                if (live && col(c, 0) < H) load8(r + col(c, 0), a[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (live && col(c, j) < H) a[c][j] = to_f32<T>(r[col(c, j)]);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (V == 8) {
                if (!live || col(c, 0) >= H) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) s[c][j] += a[c][j];
                store8(so + col(c, 0), s[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (live && col(c, j) < H) {
                        s[c][j] += a[c][j];
                        so[col(c, j)] = from_f32<T>(s[c][j]);
                    }
            }
        }
    }
    if (NORM) {
        float q = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) q += s[c][j] * s[c][j];
        q = warp_sum(q);
        if (W > 1) {
            if (lane == 0) part[warp] = q;
            __syncthreads();
            q = 0.f;
            for (int w = 0; w < W; ++w) q += part[warp - wr + w];
        }
        const float inv = 1.0f / sqrtf(q / (float)H + p.eps);
        const T *wt = static_cast<const T *>(p.weight);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float w[8];
            if (V == 8) {
                if (col(c, 0) < H) load8(wt + col(c, 0), w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (V != 8) w[j] = col(c, j) < H ? to_f32<T>(wt[col(c, j)]) : 0.f;
                s[c][j] = col(c, j) < H ? s[c][j] * inv * w[j] : 0.f;
            }
        }
    }
    if (NORM && p.out && live) {
        T *o = static_cast<T *>(p.out) + row * H;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (V == 8) {
                if (col(c, 0) < H) store8(o + col(c, 0), s[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(c, j) < H) o[col(c, j)] = from_f32<T>(s[c][j]);
            }
        }
    }
    if (!NORM || p.out_fp8) {
        uint8_t *o = p.out_fp8 + row * H;
        float *os = p.out_scale + row * ((H + 127) / 128);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int g0 = ((c * W + wr) * 256) >> 7;               // first of the chunk's two groups
            if (V == 8) {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(s[c][j]));
                const float sc = scale_of(lanes_max(m, 8)), inv = 1.0f / sc;
                if (!live || col(c, 0) >= H) continue;
                uint32_t w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[c][4 * h] * inv, s[c][4 * h + 1] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(s[c][4 * h + 2] * inv, s[c][4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                    w[h] = lo | (hi << 16);
                }
                *reinterpret_cast<uint2 *>(o + col(c, 0)) = make_uint2(w[0], w[1]);
                if ((lane & 15) == 0) os[g0 + (lane >> 4)] = sc;
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float m = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(s[c][4 * h + j]));
                    const float sc = scale_of(lanes_max(m, 16)), inv = 1.0f / sc;
                    if (!live) continue;
#pragma unroll
                    for (int j = 4 * h; j < 4 * h + 4; ++j)
                        if (col(c, j) < H) o[col(c, j)] = __nv_cvt_float_to_fp8(s[c][j] * inv, __NV_SATFINITE, __NV_E4M3);
                    if (lane == 0 && (g0 + h) * 128 < H) os[g0 + h] = sc;
                }
            }
        }
    }
}

template <typename T, int V, int NC, bool NORM> cudaError_t launch_norm(const NormArgs &a, cudaStream_t st)
{
    const int warps = NORM && a.W > 8 ? a.W : 8;
    const dim3 grid((unsigned)(((int64_t)a.T * a.W + warps - 1) / warps));
    if (warps > 8) return launch_pdl(rmsnorm_kernel<T, V, NC, NORM, 1024>, grid, warps * 32, 0, st, a);
    return launch_pdl(rmsnorm_kernel<T, V, NC, NORM, 256>, grid, warps * 32, 0, st, a);
}

template <typename T, bool NORM> cudaError_t launch_norm_v(NormArgs &a, bool vec, cudaStream_t st)
{
    // Chunks per lane and warps per row: few rows spread a row over as many
    // warps as it has chunks (latency); many rows give a lane up to four chunks
    // (more loads in flight, fewer partial sums).
    const int chunks = (a.H + 255) / 256;
    int nc = a.T <= 296 ? 1 : chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
    while (NORM && nc < 4 && nc * 32 < chunks) nc *= 2;
    a.W = (chunks + nc - 1) / nc;
    if (NORM) {                                  // a block holds whole rows
        int w = 1;
        while (w < a.W) w *= 2;
        a.W = w;
    }
    if (vec)
        return nc == 1   ? launch_norm<T, 8, 1, NORM>(a, st)
               : nc == 2 ? launch_norm<T, 8, 2, NORM>(a, st)
                         : launch_norm<T, 8, 4, NORM>(a, st);
    return nc == 1   ? launch_norm<T, 1, 1, NORM>(a, st)
           : nc == 2 ? launch_norm<T, 1, 2, NORM>(a, st)
                     : launch_norm<T, 1, 4, NORM>(a, st);
}

template <bool NORM> int norm_call(int dtype, NormArgs &a, void *stream)
{
    const int e = elem_size(dtype);
    const uintptr_t ptrs = (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.weight | (uintptr_t)a.sum_out |
                           (uintptr_t)a.out | (uintptr_t)a.out_fp8;
    if (((uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.weight | (uintptr_t)a.sum_out | (uintptr_t)a.out) &
        (uintptr_t)(e - 1))
        return ORTHRUS_ERR_ALIGN;
    if ((uintptr_t)a.out_scale & 3u) return ORTHRUS_ERR_ALIGN;
    const bool vec = (ptrs & 15u) == 0 && a.H % 8 == 0 && a.x_stride % 8 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t r;
    if (dtype == ORTHRUS_BF16)
        r = launch_norm_v<__nv_bfloat16, NORM>(a, vec, st);
    else if (dtype == ORTHRUS_F16)
        r = launch_norm_v<__half, NORM>(a, vec, st);
    else
        r = launch_norm_v<float, NORM>(a, vec, st);
    return r == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_LAUNCH;
}

}  // namespace

}  // namespace orthrus

using namespace orthrus;

extern "C" int orthrus_rmsnorm(orthrus_dtype dtype, const void *x, int64_t x_stride, const void *residual,
                               const void *weight, int T, int H, float eps, void *sum_out, void *out, void *out_fp8,
                               float *out_scale, void *stream)
{
    if (!x || !weight || !elem_size(dtype) || T <= 0 || H <= 0 || !(eps >= 0.f) || isinf(eps)) return ORTHRUS_ERR_ARG;
    if ((residual == nullptr) != (sum_out == nullptr) || (out_fp8 == nullptr) != (out_scale == nullptr))
        return ORTHRUS_ERR_ARG;
    if ((!out && !out_fp8) || x_stride < (T > 1 ? H : 0)) return ORTHRUS_ERR_ARG;
    if (H > ORTHRUS_MAX_NORM_WIDTH) return ORTHRUS_ERR_UNSUPPORTED;
    // rows of x that are not dense must not be written through another stride
    if (x_stride != H && T > 1 && (sum_out == x || out == x)) return ORTHRUS_ERR_ARG;
    NormArgs a = {x, residual, weight, x_stride, sum_out, out, static_cast<uint8_t *>(out_fp8), out_scale, T, H, 1, eps};
    return norm_call<true>(dtype, a, stream);
}

extern "C" int orthrus_quantize_fp8(orthrus_dtype dtype, const void *x, int64_t x_stride, int T, int H, void *out_fp8,
                                    float *out_scale, void *stream)
{
    if (!x || !out_fp8 || !out_scale || !elem_size(dtype) || T <= 0 || H <= 0) return ORTHRUS_ERR_ARG;
    if (x_stride < (T > 1 ? H : 0)) return ORTHRUS_ERR_ARG;
    NormArgs a = {x, nullptr, nullptr, x_stride, nullptr, nullptr, static_cast<uint8_t *>(out_fp8), out_scale, T, H, 1, 0.f};
    if ((int64_t)T * ((H + 255) / 256) >= (8ll << 31)) return ORTHRUS_ERR_UNSUPPORTED;   // (blocks of the grid)
    return norm_call<false>(dtype, a, stream);
}
