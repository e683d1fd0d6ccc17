// Rotary positions of queries and keys, with an optional RMS norm of each head
// in front, and (orthrus_rope_append) the rotated keys and the values written
// into their rows of a paged cache.
//
// For pair i of the first rot elements of a head at position t:
//     (a, b) <- m (a cos p - b sin p, b cos p + a sin p),  p = 2 pi frac(t * turns_i)
// The product t * turns_i and its fraction are fp64: at position 2^20 an fp32
// angle would be off by 2^-4 radians.  sincospi gets an fp32 fraction in [-1, 1]
// of a half turn, and what its rounding lost is added to first order.
//
// Vector path: a warp takes a token and a run of its heads, LP lanes of 16
// values each per head.  A lane's two 8-value vectors are the two sides of 8
// pairs (halves layout: elements 8u.. and rot/2 + 8u..; interleaved:
// 16u..16u+15), so a rotation needs no exchange between lanes and the lane's 8
// (cos, sin) pairs stay in registers for all of its heads (each computed by one
// lane, passed on through shared memory); the norm's sum of squares is a shuffle
// over the LP lanes.  U heads' loads are issued before any of them is worked on
// and before the angles are.  HBM-bound: every value is read and written once
// (16384 tokens, 40 heads of 128: 59 us, 5.7 TB/s, 87 % of a copy's rate).
//
// Element path (misaligned tensors, D or rot not a multiple of 16): a warp per
// (token, head), lanes over single pairs.
#include <math.h>

#include "kernels.h"
#include "layer_ops.cuh"

namespace orthrus {

namespace {

struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t qt, qh, qot, qoh, kt, kh, kot, koh, vt, vh;     // strides in elements
    const int32_t *positions;        // [T]; NULL: ctx_lens[b] + i
    const double *turns;
    const void *q_norm, *k_norm;
    float magnitude, eps;
    int T, Hq, Hkv, D, rot, layout;
    // paged destination (orthrus_rope_append)
    int append, K;
    int heads;                       // Hq + Hkv, + Hkv where values are written
    void *k_pages, *v_pages;
    int num_pages, page_size, max_pages;
    const int32_t *block_table, *ctx_lens;
    int32_t *status;
};

// Where item (token t, head h) is read and written; false: nothing to do.
template <typename T> struct Item {
    const T *src;
    T *dst;
    const T *norm;
    bool rotate;
};

__device__ __forceinline__ int position_of(const RopeArgs &p, int t)
{
    if (p.positions) return p.positions[t];
    const int b = t / p.K;
    return p.ctx_lens[b] + (t - b * p.K);
}

// Row of token t in the paged cache, KV head 0: (page * Hkv) * page_size + row,
// or -1 where it has none (the caller's error, raised in the status word).
__device__ __forceinline__ int64_t cache_row(const RopeArgs &p, int t)
{
    const int b = t / p.K, i = t - b * p.K;
    const int c = p.ctx_lens[b];
    if (c < 0 || (int64_t)c + p.K > (int64_t)p.max_pages * p.page_size) {
        if (i == 0) raise_status(p.status, ORTHRUS_STATUS_CAPACITY);
        return -1;
    }
    const int pos = c + i, e = pos / p.page_size;
    const int page = p.block_table[(int64_t)b * p.max_pages + e];
    if (page < 0 || page >= p.num_pages) {
        raise_status(p.status, ORTHRUS_STATUS_PAGE);
        return -1;
    }
    return (int64_t)page * p.Hkv * p.page_size + (pos - e * p.page_size);
}

template <typename T>
__device__ __forceinline__ bool item_of(const RopeArgs &p, int t, int h, int64_t crow, Item<T> &it)
{
    if (h < p.Hq) {
        it.src = static_cast<const T *>(p.q) + t * p.qt + h * p.qh;
        it.dst = static_cast<T *>(p.q_out) + t * p.qot + h * p.qoh;
        it.norm = static_cast<const T *>(p.q_norm);
        it.rotate = true;
        return true;
    }
    int g = h - p.Hq;
    const bool value = g >= p.Hkv;
    if (value) g -= p.Hkv;
    it.rotate = !value;
    it.norm = value ? nullptr : static_cast<const T *>(p.k_norm);
    if (!p.append) {
        it.src = static_cast<const T *>(p.k) + t * p.kt + g * p.kh;
        it.dst = static_cast<T *>(p.k_out) + t * p.kot + g * p.koh;
        return true;
    }
    if (crow < 0) return false;
    it.dst = static_cast<T *>(value ? p.v_pages : p.k_pages) + (crow + (int64_t)g * p.page_size) * p.D;
    it.src = value    ? static_cast<const T *>(p.v) + t * p.vt + g * p.vh
             : !p.k ? it.dst
                    : static_cast<const T *>(p.k) + t * p.kt + g * p.kh;
    return true;
}

// The fp32 fraction's rest d, up to pi 2^-25 radians, turns the pair by itself
// (its square is below 2^-46).
__device__ __forceinline__ float2 cos_sin(const RopeArgs &p, int pos, int i)
{
    const double turn = (double)pos * p.turns[i], half_turns = 2.0 * (turn - rint(turn));
    const float f = (float)half_turns, d = (float)(half_turns - (double)f) * 3.14159265f;
    float s, c;
    sincospif(f, &s, &c);
    return make_float2(fmaf(-s, d, c) * p.magnitude, fmaf(c, d, s) * p.magnitude);
}

constexpr int kRopeThreads = 256;

template <typename T, int LP, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs p, int run, int runs, int64_t units)
{
    constexpr int HPI = 32 / LP;                      // heads per pass of the warp
    __shared__ float4 cs[kRopeThreads / 32][LP * 4];  // (cos, sin) of the token's pairs
    sm100::pdl_trigger();
    sm100::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int u = lane % LP, hg = lane / LP;
    const int half = p.rot >> 1;
    const bool pairs = u < p.rot >> 4, mine = u < p.D >> 4;
    const bool norm = p.q_norm || p.k_norm;
    // the lane's two vectors: the two sides of 8 pairs, or 16 values that only pass
    const int e0 = pairs && p.layout == ORTHRUS_ROPE_HALF ? 8 * u : 16 * u;
    const int e1 = pairs && p.layout == ORTHRUS_ROPE_HALF ? half + 8 * u : 16 * u + 8;
    const int64_t step = (int64_t)gridDim.x * (kRopeThreads / 32);
    for (int64_t unit = (int64_t)blockIdx.x * (kRopeThreads / 32) + warp; unit < units; unit += step) {
        const int t = (int)(unit / runs), h_lo = (int)(unit - (int64_t)t * runs) * run;
        const int h_hi = h_lo + run < p.heads ? h_lo + run : p.heads;
        const int pos = position_of(p, t);
        const int64_t crow = p.append && h_hi > p.Hq ? cache_row(p, t) : 0;
        float2 f[8];
        for (int hb = h_lo; hb < h_hi; hb += U * HPI) {
            Raw8<T> ra[U], rb[U];
            Item<T> it[U];
            bool live[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * HPI + hg;
                live[i] = h < h_hi && mine && item_of(p, t, h, crow, it[i]);
                if (live[i]) {
                    ra[i] = load_raw(it[i].src + e0);
                    rb[i] = load_raw(it[i].src + e1);
                }
            }
            if (hb == h_lo) {
                __syncwarp();                         // (the last unit's pairs have been read)
                for (int i = lane; i < half; i += 32) reinterpret_cast<float2 *>(cs[warp])[i] = cos_sin(p, pos, i);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 v = cs[warp][4 * u + j];
                    f[2 * j] = make_float2(v.x, v.y);
                    f[2 * j + 1] = make_float2(v.z, v.w);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float2 a[4], b[4];
                if (live[i]) {
                    unpack8<T>(ra[i], a);
                    unpack8<T>(rb[i], b);
                }
                if (norm) {
                    float ss = 0.f;
                    if (live[i]) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            ss += a[j].x * a[j].x + a[j].y * a[j].y + b[j].x * b[j].x + b[j].y * b[j].y;
                    }
#pragma unroll
                    for (int o = LP / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                    if (live[i] && it[i].norm) {
                        const float inv = 1.0f / sqrtf(ss / (float)p.D + p.eps);
                        float2 w[4];
                        unpack8<T>(load_raw(it[i].norm + e0), w);
#pragma unroll
                        for (int j = 0; j < 4; ++j) a[j] = make_float2(a[j].x * inv * w[j].x, a[j].y * inv * w[j].y);
                        unpack8<T>(load_raw(it[i].norm + e1), w);
#pragma unroll
                        for (int j = 0; j < 4; ++j) b[j] = make_float2(b[j].x * inv * w[j].x, b[j].y * inv * w[j].y);
                    }
                }
                if (!live[i]) continue;
                if (it[i].rotate && pairs) {
                    if (p.layout == ORTHRUS_ROPE_HALF) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = a[j], y = b[j], f0 = f[2 * j], f1 = f[2 * j + 1];
                            a[j] = make_float2(x.x * f0.x - y.x * f0.y, x.y * f1.x - y.y * f1.y);
                            b[j] = make_float2(y.x * f0.x + x.x * f0.y, y.y * f1.x + x.y * f1.y);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = a[j], y = b[j];
                            a[j] = make_float2(x.x * f[j].x - x.y * f[j].y, x.y * f[j].x + x.x * f[j].y);
                            b[j] = make_float2(y.x * f[4 + j].x - y.y * f[4 + j].y, y.y * f[4 + j].x + y.x * f[4 + j].y);
                        }
                    }
                }
                store8(it[i].dst + e0, a);
                store8(it[i].dst + e1, b);
            }
        }
    }
}

template <typename T> __global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const RopeArgs p)
{
    sm100::pdl_trigger();
    sm100::pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t items = (int64_t)p.T * p.heads, step = (int64_t)gridDim.x * (kRopeThreads / 32);
    const int half = p.rot >> 1, pairs = half + (p.D - p.rot + 1) / 2;
    for (int64_t idx = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); idx < items; idx += step) {
        const int t = (int)(idx / p.heads), h = (int)(idx - (int64_t)t * p.heads);
        const int pos = position_of(p, t);
        Item<T> it;
        // (one token's error is raised by every head: an idempotent OR)
        if (!item_of(p, t, h, p.append && h >= p.Hq ? cache_row(p, t) : 0, it)) continue;
        // pair i: elements (e0, e1); past the rotated part, two values that only pass
        float a[4], b[4], ss = 0.f;
        int n = 0;
        for (int i = lane; i < pairs; i += 32, ++n) {
            const int e0 = i >= half                             ? p.rot + 2 * (i - half)
                           : p.layout == ORTHRUS_ROPE_HALF ? i
                                                                 : 2 * i;
            const int e1 = i < half && p.layout == ORTHRUS_ROPE_HALF ? half + i : e0 + 1;
            a[n] = to_f32<T>(it.src[e0]);
            b[n] = e1 < p.D ? to_f32<T>(it.src[e1]) : 0.f;
            ss += a[n] * a[n] + b[n] * b[n];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float inv = 1.0f / sqrtf(ss / (float)p.D + p.eps);
        n = 0;
        for (int i = lane; i < pairs; i += 32, ++n) {
            const int e0 = i >= half                             ? p.rot + 2 * (i - half)
                           : p.layout == ORTHRUS_ROPE_HALF ? i
                                                                 : 2 * i;
            const int e1 = i < half && p.layout == ORTHRUS_ROPE_HALF ? half + i : e0 + 1;
            float x = a[n], y = b[n];
            if (it.norm) {
                x = x * inv * to_f32<T>(it.norm[e0]);
                if (e1 < p.D) y = y * inv * to_f32<T>(it.norm[e1]);
            }
            if (it.rotate && i < half) {
                const float2 f = cos_sin(p, pos, i);
                const float r = x * f.x - y * f.y;
                y = y * f.x + x * f.y;
                x = r;
            }
            it.dst[e0] = from_f32<T>(x);
            if (e1 < p.D) it.dst[e1] = from_f32<T>(y);
        }
    }
}

template <typename T, int LP> cudaError_t launch_rope_v(const RopeArgs &p, int sms, cudaStream_t st)
{
    // Heads per warp: all of a token's (one set of angles) once the tokens alone
    // fill the SMs' warps, else as few passes as it takes to fill them.
    constexpr int U = sizeof(T) == 2 ? 4 : 2, HPI = 32 / LP;
    const int64_t want = 16ll * sms;                  // warps
    const int passes = (p.heads + HPI - 1) / HPI;
    int64_t runs = (want + p.T - 1) / p.T;
    if (runs > passes) runs = passes;
    const int run = (int)((passes + runs - 1) / runs) * HPI;
    runs = (p.heads + run - 1) / run;
    const int64_t units = (int64_t)p.T * runs, blocks = (units + 7) / 8, most = 8ll * sms;
    return launch_pdl(rope_kernel<T, LP, U>, dim3((unsigned)(blocks < most ? blocks : most)), kRopeThreads, 0, st, p, run,
                      (int)runs, units);
}

template <typename T> cudaError_t launch_rope_t(const RopeArgs &p, bool vec, int sms, cudaStream_t st)
{
    if (!vec) {
        const int64_t blocks = ((int64_t)p.T * p.heads + 7) / 8, most = 8ll * sms;
        return launch_pdl(rope_any_kernel<T>, dim3((unsigned)(blocks < most ? blocks : most)), kRopeThreads, 0, st, p);
    }
    int lp = 1;
    while (lp * 16 < p.D) lp *= 2;
    switch (lp) {
    case 1: return launch_rope_v<T, 1>(p, sms, st);
    case 2: return launch_rope_v<T, 2>(p, sms, st);
    case 4: return launch_rope_v<T, 4>(p, sms, st);
    case 8: return launch_rope_v<T, 8>(p, sms, st);
    default: return launch_rope_v<T, 16>(p, sms, st);
    }
}

int rope_call(int dtype, RopeArgs &p, void *stream)
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ORTHRUS_ERR_DEVICE;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) return ORTHRUS_ERR_DEVICE;
    const int e = elem_size(dtype);
    const uintptr_t ptrs = (uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)p.q_out | (uintptr_t)p.k_out |
                           (uintptr_t)p.k_pages | (uintptr_t)p.v_pages | (uintptr_t)p.q_norm | (uintptr_t)p.k_norm;
    const int64_t strides = p.qt | p.qh | p.qot | p.qoh | p.kt | p.kh | p.kot | p.koh | p.vt | p.vh;
    const bool vec = (ptrs & 15u) == 0 && strides % 8 == 0 && p.D % 16 == 0 && p.rot % 16 == 0;
    if (ptrs & (uintptr_t)(e - 1)) return ORTHRUS_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t r = dtype == ORTHRUS_BF16  ? launch_rope_t<__nv_bfloat16>(p, vec, sms, st)
                          : dtype == ORTHRUS_F16 ? launch_rope_t<__half>(p, vec, sms, st)
                                                 : launch_rope_t<float>(p, vec, sms, st);
    return r == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_LAUNCH;
}

// Checks and fields that both entry points share.
int rope_common(RopeArgs &p, int dtype, int layout, const double *turns, float magnitude, int64_t T, int Hq, int Hkv,
                int D, int rot, const void *q_norm, const void *k_norm, float eps)
{
    if (!elem_size(dtype) || (layout != ORTHRUS_ROPE_HALF && layout != ORTHRUS_ROPE_INTERLEAVED)) return ORTHRUS_ERR_ARG;
    if (!turns || T <= 0 || Hq < 0 || Hkv < 0 || Hq + Hkv <= 0 || D <= 0 || rot <= 0 || rot > D) return ORTHRUS_ERR_ARG;
    if (!isfinite(magnitude) || !(eps >= 0.f) || isinf(eps)) return ORTHRUS_ERR_ARG;
    if ((uintptr_t)turns & 7u) return ORTHRUS_ERR_ALIGN;
    if (rot % 2 || D > ORTHRUS_MAX_HEAD_DIM || Hq > 65536 || Hkv > 65536 || T > (1 << 30)) return ORTHRUS_ERR_UNSUPPORTED;
    p.turns = turns;
    p.magnitude = magnitude;
    p.T = (int)T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.rot = rot;
    p.layout = layout;
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.eps = eps;
    return ORTHRUS_OK;
}

}  // namespace

}  // namespace orthrus

using namespace orthrus;

extern "C" int orthrus_rope_table(orthrus_rope_scaling kind, int rot_dim, double theta, double factor, double orig_len,
                                  double beta_fast, double beta_slow, double *turns, float *magnitude)
{
    const double pi = 3.14159265358979323846;
    if (!turns || !magnitude || rot_dim <= 0 || rot_dim % 2 || !(theta > 1.0) || isinf(theta)) return ORTHRUS_ERR_ARG;
    if (kind < ORTHRUS_ROPE_PLAIN || kind > ORTHRUS_ROPE_YARN) return ORTHRUS_ERR_ARG;
    if (kind != ORTHRUS_ROPE_PLAIN && (!(factor >= 1.0) || isinf(factor))) return ORTHRUS_ERR_ARG;
    if (kind == ORTHRUS_ROPE_NTK && rot_dim < 4) return ORTHRUS_ERR_UNSUPPORTED;
    if (kind == ORTHRUS_ROPE_YARN &&
        (!(orig_len > 0.0) || isinf(orig_len) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || isinf(beta_fast)))
        return ORTHRUS_ERR_ARG;
    if (kind == ORTHRUS_ROPE_NTK) theta *= pow(factor, (double)rot_dim / (rot_dim - 2));
    double low = 0.0, high = 0.0;
    if (kind == ORTHRUS_ROPE_YARN) {
        // the (real) pair index whose wavelength makes `beta` turns in orig_len positions
        auto index_of = [&](double beta) { return rot_dim * log(orig_len / (beta * 2.0 * pi)) / (2.0 * log(theta)); };
        low = fmax(floor(index_of(beta_fast)), 0.0);
        high = fmin(ceil(index_of(beta_slow)), rot_dim - 1.0);
        if (high <= low) high = low + 0.001;           // a step instead of a ramp
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(theta, -2.0 * i / rot_dim);
        if (kind == ORTHRUS_ROPE_LINEAR) f /= factor;
        if (kind == ORTHRUS_ROPE_YARN) {
            const double r = fmin(1.0, fmax(0.0, (i - low) / (high - low)));
            f = f / factor * r + f * (1.0 - r);
        }
        turns[i] = f / (2.0 * pi);
    }
    *magnitude = kind == ORTHRUS_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return ORTHRUS_OK;
}

extern "C" int orthrus_rope(orthrus_dtype dtype, orthrus_rope_layout layout, const void *q, void *q_out, const void *k,
                            void *k_out, const int64_t *strides, const int32_t *positions, const double *turns,
                            float magnitude, int T, int Hq, int Hkv, int D, int rot_dim, const void *q_norm,
                            const void *k_norm, float eps, void *stream)
{
    RopeArgs p = {};
    if (!q || !q_out || !positions || Hq <= 0 || (k == nullptr) != (k_out == nullptr) || (k == nullptr) != (Hkv == 0))
        return ORTHRUS_ERR_ARG;
    const int rc = rope_common(p, dtype, layout, turns, magnitude, T, Hq, Hkv, D, rot_dim, q_norm, k_norm, eps);
    if (rc != ORTHRUS_OK) return rc;
    p.q = q;
    p.q_out = q_out;
    p.k = k;
    p.k_out = k_out;
    p.positions = positions;
    p.heads = Hq + Hkv;
    const int64_t dense[8] = {(int64_t)Hq * D, D, (int64_t)Hq * D, D, (int64_t)Hkv * D, D, (int64_t)Hkv * D, D};
    const int64_t *s = strides ? strides : dense;
    p.qt = s[0], p.qh = s[1], p.qot = s[2], p.qoh = s[3];
    if (k) p.kt = s[4], p.kh = s[5], p.kot = s[6], p.koh = s[7];
    // in place means the same layout
    if ((q == q_out && (p.qt != p.qot || p.qh != p.qoh)) || (k && k == k_out && (p.kt != p.kot || p.kh != p.koh)))
        return ORTHRUS_ERR_ARG;
    return rope_call(dtype, p, stream);
}

extern "C" int orthrus_rope_append(orthrus_dtype dtype, orthrus_rope_layout layout, const void *q, void *q_out,
                                   const void *k, const void *v, const int64_t *strides, const double *turns,
                                   float magnitude, int B, int K, int Hq, int Hkv, int D, int rot_dim,
                                   const void *q_norm, const void *k_norm, float eps, void *k_pages, void *v_pages,
                                   int num_pages, int page_size, const int32_t *block_table, int max_pages,
                                   const int32_t *ctx_lens, int32_t *status, void *stream)
{
    RopeArgs p = {};
    if ((q == nullptr) != (q_out == nullptr) || (q == nullptr) != (Hq == 0) || (k == nullptr) != (v == nullptr))
        return ORTHRUS_ERR_ARG;
    if (!k_pages || (v && !v_pages) || !block_table || !ctx_lens || Hkv <= 0 || B <= 0 || K <= 0) return ORTHRUS_ERR_ARG;
    if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return ORTHRUS_ERR_ARG;
    const int rc = rope_common(p, dtype, layout, turns, magnitude, (int64_t)B * K, Hq, Hkv, D, rot_dim, q_norm, k_norm, eps);
    if (rc != ORTHRUS_OK) return rc;
    if ((int64_t)max_pages * page_size >= 1ll << 31) return ORTHRUS_ERR_UNSUPPORTED;
    p.q = q;
    p.q_out = q_out;
    p.k = k;
    p.v = v;
    const int64_t dense[8] = {(int64_t)Hq * D, D, (int64_t)Hq * D, D, (int64_t)Hkv * D, D, (int64_t)Hkv * D, D};
    const int64_t *s = strides ? strides : dense;
    if (q) p.qt = s[0], p.qh = s[1], p.qot = s[2], p.qoh = s[3];
    if (k) p.kt = s[4], p.kh = s[5], p.vt = s[6], p.vh = s[7];
    if (q && q == q_out && (p.qt != p.qot || p.qh != p.qoh)) return ORTHRUS_ERR_ARG;
    p.append = 1;
    p.K = K;
    p.heads = Hq + Hkv + (v ? Hkv : 0);
    p.k_pages = k_pages;
    p.v_pages = v ? v_pages : nullptr;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.block_table = block_table;
    p.ctx_lens = ctx_lens;
    p.status = status;
    return rope_call(dtype, p, stream);
}
