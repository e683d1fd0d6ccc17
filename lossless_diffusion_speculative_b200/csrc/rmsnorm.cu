// RMS norm of rows with the residual's addition in front and an 8-bit output
// with scales behind it, and plain quantisation to the same 8-bit form.
//
//     s = x + r;  y = s * rsqrt(mean(s^2) + eps) * w
//     scale = max(max|y| (1 / 448), 2^-126) per 128 columns;  value = e4m3(y / scale)
//
// One pass: a row's values stay in registers (fp32) between the sum of squares
// and the outputs, so each input is read and each output written once.  A row
// belongs to W warps (1..32), each lane holding NC chunks of 8 values; the sum
// of squares goes through shuffles and, for W > 1, shared memory.  A 128-column
// group lies within one warp's chunk of 256 columns: 16 lanes of 8 consecutive
// values on the vector path, or strips of 32 lanes where rows are not 16-byte
// aligned, so its maximum needs shuffles only.  HBM-bound, measured: 16384 x 4096 bf16 with
// residual to 8 bits 73 us (6.4 TB/s, 98 % of a copy's rate) in short runs and 79-82
// where the power limit holds, 8192 x 12288 quantised 50 us (94 %) and 54-56.
// (The 1024-thread instances, 64 registers a thread, keep part of two and four
// chunks a lane in local memory: 2000 x 32768 with residual to 8 bits 181 us, floor 70.)
#include <math.h>

#include <type_traits>

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

// Scale of a group from its maximum, and the scale's reciprocal (the nearest fp32
// value), or 0 from 2^80 on, where the reciprocal's own error would fall below the
// smallest numbers, and for a scale of infinity.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(float amax)
{
    Scale o;
    o.s = fmaxf(amax * (1.0f / 448.0f), 1.17549435e-38f);
    o.inv = o.s < 0x1p80f ? __frcp_rn(o.s) : 0.f;
    return o;
}

// Where inv is 0: a factor for the group's values that keeps their quotients by
// the scale, which is changed with them (finite / infinity: zeros).
__device__ __forceinline__ float lower(Scale &sc)
{
    const bool finite = sc.s < INFINITY;
    sc.s = finite ? sc.s * 0x1p-100f : 1.0f;
    sc.inv = __frcp_rn(sc.s);
    return finite ? 0x1p-100f : 0.f;
}

// Maxima of NC chunks' values over 16 lanes, as scales: the butterfly folds chunks
// together as it goes (with four chunks 5 exchanges instead of 16), each lane
// makes one scale, and every lane then takes all chunks' from the lanes that
// hold them.
template <int NC> __device__ __forceinline__ void scales_of(const float (&m)[NC], Scale (&sc)[NC])
{
    const int lane = threadIdx.x & 31;
    float v;
    if constexpr (NC == 4) {
        const bool b0 = lane & 1, b1 = lane & 2;         // the lane keeps chunk (lane & 3)
        const float a = fmaxf(b0 ? m[1] : m[0], __shfl_xor_sync(~0u, b0 ? m[0] : m[1], 1));
        const float b = fmaxf(b0 ? m[3] : m[2], __shfl_xor_sync(~0u, b0 ? m[2] : m[3], 1));
        v = fmaxf(b1 ? b : a, __shfl_xor_sync(~0u, b1 ? a : b, 2));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
    } else if constexpr (NC == 2) {
        const bool b0 = lane & 1;
        v = fmaxf(b0 ? m[1] : m[0], __shfl_xor_sync(~0u, b0 ? m[0] : m[1], 1));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
    } else {
        v = fmaxf(m[0], __shfl_xor_sync(~0u, m[0], 1));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
    }
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
    const Scale own = scale_of(v);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        sc[c] = own;
        if (NC > 1) {
            sc[c].s = __shfl_sync(~0u, own.s, (lane & 16) + c);
            sc[c].inv = __shfl_sync(~0u, own.inv, (lane & 16) + c);
        }
    }
}

// 1 / s as the nearest fp32 value and the rest: together good to 2^-48 (1 - s inv is
// exact, an fma).
struct Inverse {
    float2 hi, lo;
};
__device__ __forceinline__ Inverse inverse_of(const Scale &sc)
{
    const float rest = fmaf(-sc.s, sc.inv, 1.0f) * sc.inv;
    return {make_float2(sc.inv, sc.inv), make_float2(rest, rest)};
}

// y / scale as e4m3: two values, low byte first.  The quotient is rounded to fp32
// once, from y (hi + lo) within 2^-47 of it: 16-bit inputs lie on the borders
// between two e4m3 values often, and a quotient that is one fp32 step off can go to
// the wrong neighbour there (with y hi alone 21 of 8192 x 12288 bf16 values did).
// At every border the result equals the division's, for every significand of a scale.
__device__ __forceinline__ uint32_t quotient2(float2 y, const Inverse &v)
{
    return __nv_cvt_float2_to_fp8x2(sm100::ffma2(y, v.hi, sm100::fmul2(y, v.lo)), __NV_SATFINITE, __NV_E4M3);
}

// ---- vector path
//
// A row belongs to W warps (W <= 32, a power of two with the norm), a lane
// holds NC chunks of 8 consecutive values.  Blocks are resident for the whole
// call and walk the rows, the next row's loads issued (unconverted) before the
// current one is worked on, so that the memory never waits for the arithmetic;
// the weights stay in registers.  Without the norm a warp's part of a row is a
// unit of its own.
template <typename T, int NC, bool NORM, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_rows_kernel(const NormArgs p)
{
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int W = p.W, H = p.H, groups = (H + 127) >> 7;
    sm100::pdl_trigger();
    sm100::pdl_wait();

    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    const bool add = NORM && p.residual != nullptr;
    // unit = (row, part of the row); a block's warps take consecutive units
    const unsigned units = (unsigned)p.T * W, step = gridDim.x * warps;
    unsigned unit = blockIdx.x * warps + warp;
    Raw8<T> nx[NC], nr[NORM ? NC : 1], wt[NORM ? NC : 1];
    unsigned row = unit / W;
    int c0 = (int)(unit - row * W) * 256 + lane * 8;                  // columns c0 + 256 W c of chunk c
    auto fetch = [&](unsigned r, int col, bool live) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = col + c * W * 256;
            nx[c] = Raw8<T>{};
            if (live && k < H) nx[c] = load_raw(x + (int64_t)r * p.x_stride + k);
            if constexpr (NORM) {
                if (add) {
                    nr[c] = Raw8<T>{};
                    if (live && k < H) nr[c] = load_raw(res + (int64_t)r * H + k);
                }
            }
        }
    };
    fetch(row, c0, unit < units);
    if constexpr (NORM) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            wt[c] = Raw8<T>{};
            if (c0 + c * W * 256 < H) wt[c] = load_raw(static_cast<const T *>(p.weight) + c0 + c * W * 256);
        }
    }
    // (with the norm every warp of a block makes the same number of rounds)
    const unsigned first = blockIdx.x * warps;
    for (unsigned it = 0; (NORM ? first + it * step : unit) < units; ++it) {
        const bool live = unit < units;
        float2 s[NC][4];
#pragma unroll
        for (int c = 0; c < NC; ++c) unpack8<T>(nx[c], s[c]);
        if constexpr (NORM) {
            if (add) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float2 a[4];
                    unpack8<T>(nr[c], a);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[c][j] = sm100::fadd2(s[c][j], a[j]);
                }
            }
        }
        const unsigned r = row;
        const int k0 = c0;
        unit += step;
        row = unit / W;
        c0 = (int)(unit - row * W) * 256 + lane * 8;                  // (with the norm: unchanged, W divides the step)
        fetch(row, c0, unit < units);
        if constexpr (NORM) {
            float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (add && live && k0 + c * W * 256 < H)
                    store8(static_cast<T *>(p.sum_out) + (int64_t)r * H + k0 + c * W * 256, s[c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) q2 = sm100::ffma2(s[c][j], s[c][j], q2);
            }
            float q = warp_sum(q2.x + q2.y);
            if (W > 1) {
                if (lane == 0) part[it & 1][warp] = q;
                __syncthreads();
                q = 0.f;
                const int w0 = warp & ~(W - 1);
                for (int w = 0; w < W; ++w) q += part[it & 1][w0 + w];
            }
            const float inv = 1.0f / sqrtf(q / (float)H + p.eps);
            const float2 i2 = make_float2(inv, inv);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float2 w[4];
                unpack8<T>(wt[c], w);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[c][j] = sm100::fmul2(sm100::fmul2(s[c][j], i2), w[j]);
                if (p.out && live && k0 + c * W * 256 < H)
                    store8(static_cast<T *>(p.out) + (int64_t)r * H + k0 + c * W * 256, s[c]);
            }
        }
        if (!NORM || p.out_fp8) {
            float m[NC];
            Scale sc[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                m[c] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) m[c] = sm100::fmax3(m[c], fabsf(s[c][j].x), fabsf(s[c][j].y));
            }
            scales_of<NC>(m, sc);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = k0 + c * W * 256;
                const float scale = sc[c].s;
                if (sc[c].inv == 0.f) {
                    const float f = lower(sc[c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[c][j] = sm100::fmul2(s[c][j], make_float2(f, f));
                }
                const Inverse v = inverse_of(sc[c]);
                const uint32_t lo = quotient2(s[c][0], v) | (quotient2(s[c][1], v) << 16);
                const uint32_t hi = quotient2(s[c][2], v) | (quotient2(s[c][3], v) << 16);
                if (live && k < H) {
                    *reinterpret_cast<uint2 *>(p.out_fp8 + (int64_t)r * H + k) = make_uint2(lo, hi);
                    if ((lane & 15) == 0) p.out_scale[(int64_t)r * groups + (k >> 7)] = scale;
                }
            }
        }
    }
}

// ---- element path: rows that are not 16-byte aligned, or whose width is not a
// multiple of 8.  The same parts of a row; a lane's 8 values of a chunk are V at
// a time, strips of 32 V columns: four values, pairs or single ones, as every
// row is aligned for them (1113 x 10780 with residual to 8 bits, with four 39 us, with pairs 50).
template <typename T, int V> union Few {
    using Raw = std::conditional_t<sizeof(T) * V == 2, uint16_t,
                                   std::conditional_t<sizeof(T) * V == 4, uint32_t,
                                                      std::conditional_t<sizeof(T) * V == 8, uint2, uint4>>>;
    Raw raw;                        // (one access; the values' own copy may be split into theirs)
    T v[V];
    __device__ Few() : raw() {}
};
template <typename T, int V, int NC, bool NORM, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_any_kernel(const NormArgs p)
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

    // first column of piece j (V columns) of chunk c: chunk c of warp wr covers 256 columns
    auto col = [&](int c, int j) { return (c * W + wr) * 256 + (j * 32 + lane) * V; };
    auto load = [&](const T *src, float (&f)[NC][8]) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8 / V; ++j) {
                Few<T, V> w;
                if (live && col(c, j) < H) w.raw = *reinterpret_cast<const typename Few<T, V>::Raw *>(src + col(c, j));
#pragma unroll
                for (int e = 0; e < V; ++e) f[c][j * V + e] = to_f32<T>(w.v[e]);
            }
    };
    auto store = [&](T *dst, const float (&f)[NC][8]) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8 / V; ++j) {
                Few<T, V> w;
#pragma unroll
                for (int e = 0; e < V; ++e) w.v[e] = from_f32<T>(f[c][j * V + e]);
                if (live && col(c, j) < H) *reinterpret_cast<typename Few<T, V>::Raw *>(dst + col(c, j)) = w.raw;
            }
    };
    float s[NC][8];
    load(static_cast<const T *>(p.x) + row * p.x_stride, s);
    if constexpr (NORM) {
        if (p.residual) {
            float a[NC][8];
            load(static_cast<const T *>(p.residual) + row * H, a);
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[c][j] += a[c][j];
            store(static_cast<T *>(p.sum_out) + row * H, s);
        }
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
        float w[NC][8];
        load(static_cast<const T *>(p.weight), w);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[c][j] = col(c, j / V) < H ? s[c][j] * inv * w[c][j] : 0.f;
        if (p.out) store(static_cast<T *>(p.out) + row * H, s);
    }
    if (!NORM || p.out_fp8) {
        uint8_t *o = p.out_fp8 + row * H;
        float *os = p.out_scale + row * ((H + 127) / 128);
        // one lane makes each group's scale (chunk c has two groups), and every lane
        // takes all of them: a scale costs as much as five exchanges
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(s[i / 2][4 * (i & 1) + j]));
            m = lanes_max(m, 16);
            if (lane == i) mine = m;
        }
        const Scale own = scale_of(mine);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int g0 = ((c * W + wr) * 256) >> 7;               // first of the chunk's two groups
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Scale sc = {__shfl_sync(~0u, own.s, 2 * c + h), __shfl_sync(~0u, own.inv, 2 * c + h)};
                const float scale = sc.s;
                if (!live) continue;
                if (sc.inv == 0.f) {
                    const float f = lower(sc);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[c][4 * h + j] *= f;
                }
                const Inverse inv = inverse_of(sc);
#pragma unroll
                for (int j = 4 * h; j < 4 * h + 4; j += V == 4 ? 4 : 2) {
                    const uint32_t v = quotient2(make_float2(s[c][j], s[c][j + 1]), inv);
                    if constexpr (V == 4) {
                        const uint32_t hi = quotient2(make_float2(s[c][j + 2], s[c][j + 3]), inv);
                        if (col(c, h) < H) *reinterpret_cast<uint32_t *>(o + col(c, h)) = v | hi << 16;
                    } else if constexpr (V == 2) {
                        if (col(c, j / 2) < H) *reinterpret_cast<uint16_t *>(o + col(c, j / 2)) = (uint16_t)v;
                    } else {
                        if (col(c, j) < H) o[col(c, j)] = (uint8_t)v;
                        if (col(c, j + 1) < H) o[col(c, j + 1)] = (uint8_t)(v >> 8);
                    }
                }
                if (lane == 0 && (g0 + h) * 128 < H) os[g0 + h] = scale;
            }
        }
    }
}

template <typename T, int NC, bool NORM> cudaError_t launch_norm(const NormArgs &a, int vec, int sms, cudaStream_t st)
{
    const int warps = NORM && a.W > 8 ? a.W : 8;
    int64_t blocks = ((int64_t)a.T * a.W + warps - 1) / warps;
    if (vec < 8) {
        const dim3 grid((unsigned)blocks);
        const auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            if constexpr (NORM) {
                if (warps > 8) return launch_pdl(norm_any_kernel<T, V, NC, NORM, 1024>, grid, warps * 32, 0, st, a);
            }
            return launch_pdl(norm_any_kernel<T, V, NC, NORM, 256>, grid, warps * 32, 0, st, a);
        };
        return vec == 4   ? go(std::integral_constant<int, 4>{})
               : vec == 2 ? go(std::integral_constant<int, 2>{})
                          : go(std::integral_constant<int, 1>{});
    }
    const int64_t resident = (int64_t)sms * (warps > 8 ? 1 : NORM ? 2 : NC < 4 ? 5 : sizeof(T) == 2 ? 3 : 2);
    const dim3 grid((unsigned)(blocks < resident ? blocks : resident));
    if constexpr (NORM) {
        if (warps > 16) return launch_pdl(norm_rows_kernel<T, NC, NORM, 1024>, grid, warps * 32, 0, st, a);
        if (warps > 8) return launch_pdl(norm_rows_kernel<T, NC, NORM, 512>, grid, warps * 32, 0, st, a);
    }
    return launch_pdl(norm_rows_kernel<T, NC, NORM, 256>, grid, warps * 32, 0, st, a);
}

template <typename T, bool NORM> cudaError_t launch_norm_v(NormArgs &a, int vec, int sms, cudaStream_t st)
{
    // Chunks per lane and warps per row: few rows spread a row over as many
    // warps as it has chunks (latency); many rows give a lane up to four chunks
    // (more loads in flight, fewer partial sums).
    const int chunks = (a.H + 255) / 256;
    // The element path holds no loads back: one chunk up to eight warps, then two.
    // 4000 rows with residual to 8 bits take with one and two 45 and 37 us at 4095
    // columns, with two and four 71 and 76 at 4597, 75 and 111 at 4598, 65 and 97 at
    // 8188.  Without the norm four chunks share a scale's cost, but have fewer
    // warps: from three rounds of them on, and where no lane goes empty; two and four
    // take 58 and 54 us at 8192 x 12288, 31.6 and 27.5 at 8192 x 4096 fp32, but 15.8
    // and 16.9 at 16384 x 1536, 4.1 and 4.6 at 400 x 12288, and 17.8 and 24.7 on the
    // element path at 4000 x 4596.
    int nc = a.T <= 2 * sms ? 1
             : vec < 8      ? (chunks <= 8 ? 1 : chunks <= 32 ? 2 : 4)
                            : (chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1);
    const bool four = vec == 8 && (chunks % 4 == 0 || chunks > 16) && (int64_t)a.T * chunks >= 3ll * 96 * sms;
    if (!NORM && nc > 2 && !four) nc = 2;
    while (NORM && nc < 4 && nc * 32 < chunks) nc *= 2;
    a.W = (chunks + nc - 1) / nc;
    if (NORM) {                                  // a block holds whole rows
        int w = 1;
        while (w < a.W) w *= 2;
        a.W = w;
    }
    return nc == 1   ? launch_norm<T, 1, NORM>(a, vec, sms, st)
           : nc == 2 ? launch_norm<T, 2, NORM>(a, vec, sms, st)
                     : launch_norm<T, 4, NORM>(a, vec, sms, st);
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
    // values at a time: 8 (a 16-byte load of a 16-bit type), or 4, 2 or 1
    const auto fits = [&](int n) {
        return (ptrs & ((uintptr_t)n * e - 1)) == 0 && a.H % n == 0 && a.x_stride % n == 0;
    };
    const int vec = (ptrs & 15u) == 0 && a.H % 8 == 0 && a.x_stride % 8 == 0 ? 8 : fits(4) ? 4 : fits(2) ? 2 : 1;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ORTHRUS_ERR_DEVICE;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) return ORTHRUS_ERR_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t r = dtype == ORTHRUS_BF16  ? launch_norm_v<__nv_bfloat16, NORM>(a, vec, sms, st)
                          : dtype == ORTHRUS_F16 ? launch_norm_v<__half, NORM>(a, vec, sms, st)
                                                 : launch_norm_v<float, NORM>(a, vec, sms, st);
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
    if ((!out && !out_fp8) || (out && out == sum_out) || x_stride < (T > 1 ? H : 0)) return ORTHRUS_ERR_ARG;
    if (H > ORTHRUS_MAX_NORM_WIDTH) return ORTHRUS_ERR_UNSUPPORTED;
    if ((int64_t)T * 32 >= (1ll << 31)) return ORTHRUS_ERR_UNSUPPORTED;                  // (units of work are 32-bit)
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
    if (H > 1 << 30) return ORTHRUS_ERR_UNSUPPORTED;                                     // (columns are 32-bit)
    NormArgs a = {x, nullptr, nullptr, x_stride, nullptr, nullptr, static_cast<uint8_t *>(out_fp8), out_scale, T, H, 1, 0.f};
    if ((int64_t)T * ((H + 255) / 256) >= (1ll << 31)) return ORTHRUS_ERR_UNSUPPORTED;   // (units of work are 32-bit)
    return norm_call<false>(dtype, a, stream);
}
