// Matrix product of e4m3 operands with a scale per 1 x 128 block of a and per
// 128 x 128 block of w, on the tcgen05 tensor cores (kind::f8f6f4):
//
//     out[m, n] = sum_kb sa[m, kb] sw[n / 128, kb] sum_{k in kb} a[m, k] w[n, k]
//
// The scales change every 128 values of K, so the tensor cores cannot carry one
// accumulator through: each block's product (four K = 32 instructions) goes to
// its own TMEM buffer, and the epilogue warps add it, scaled, to fp32 sums in
// registers while the next blocks are multiplied.  (The sum of a block is exact
// to fp32 in the tensor cores.)
//
// Few token rows (this file): the weight rows are the MMA's 128 rows and up to
// 128 token rows its columns, so that no part of the MMA is padding and the
// weights are streamed once; bound by HBM.  The weight rows are cut into ranges
// of 16-row granules, one per block, walked in tiles of up to 128 rows with the
// loads running ahead across tiles.  Where whole tiles are too few for the SMs
// a range goes to a cluster of blocks that split K (partials joined through
// distributed shared memory, in rank order).  The steps of the pipeline are
// groups of GRP k-blocks: every wait, signal and issue of a step costs 50-150
// cycles of latency, which per single block (530 cycles a block measured, 16 KB
// of weights) was more than the SM's share of HBM takes to deliver it.
// (Now: 4 x 151936 x 4096 99 us, 97 % of a copy's rate; 32 x 6144 x 4096 9 us.)
// Many token rows: fp8_pair.cuh.
//
// Roles: warps 0..3 epilogue, then a TMA producer warp and an MMA warp (one
// elected thread each).
#include <mutex>

#include "kernels.h"
#include "layer_ops.cuh"

namespace orthrus {

namespace f8 {

using namespace sm100;

struct Maps {
    CUtensorMap w, w32, w16, a;          // weights: boxes of 128, 32 and 16 rows; tokens: NT rows
};

struct Args {
    const float *a_scale, *w_scale;
    void *out;
    int32_t *status;
    int M, N, K, nkb;
    int split;                           // blocks of a cluster, along K
    int tiles_x, tiles_y;                // tiles of the weight (pair: token) rows, of the others
    int ranges;                          // blocks (clusters) that share the weight rows of one token tile
    int out_dtype;
    int vec;                             // columns of out that one aligned store takes: 4, 2 or 1 (pairs of CTAs: 16 bytes' worth)
};

constexpr int kXBytes = 128 * 128;

template <int NT, int GRP, int NST> struct Conf {
    static constexpr int threads = 6 * 32;
    static constexpr int stage = GRP * (kXBytes + NT * 128);
    static constexpr int cols = 2 * GRP * NT;                         // two sets of GRP buffers; a power of two
    static constexpr int tile = NST * stage;                          // the output tile, [token][weight row] in fp32
    static constexpr int bars = tile + NT * 128 * 4;
    static constexpr int nbars = 2 * NST + 4 + 1;                     // stage full / empty, set full / empty, drain
    static constexpr int svec = (bars + nbars * 8 + 16 + 15) & ~15;   // [2][2 weight blocks][GRP][NT] scales
    static constexpr int total = svec + 2 * 2 * GRP * NT * 4 + 1024;
    static_assert(cols >= 32 && cols <= 512 && (cols & (cols - 1)) == 0, "TMEM");
    static_assert(total <= 227 * 1024, "shared memory");
    // (so that a block of the next call, which may start early, cannot take the
    // TMEM that a block of this one is about to allocate)
    static_assert(total > 114 * 1024, "one block per SM: TMEM is never waited for");
};

// Four consecutive columns of one row, the first n of them inside the matrix,
// stored `vec` (4, 2, 1) at a time.
template <typename T> __device__ __forceinline__ void put2(T *out, float a, float b)
{
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t *>(out) = pack2<T>(a, b);
    else *reinterpret_cast<float2 *>(out) = make_float2(a, b);
}
template <typename T> __device__ __forceinline__ void put4(T *out, float4 x, int n, int vec)
{
    if (vec == 2 && n >= 2) {                  // (n is even where the rows are)
        put2(out, x.x, x.y);
        if (n >= 4) put2(out + 2, x.z, x.w);
    } else if (vec == 4 && n >= 4) {
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(x.x, x.y), pack2<T>(x.z, x.w));
        else
            *reinterpret_cast<float4 *>(out) = x;
    } else {
        if (n > 0) out[0] = from_f32<T>(x.x);
        if (n > 1) out[1] = from_f32<T>(x.y);
        if (n > 2) out[2] = from_f32<T>(x.z);
        if (n > 3) out[3] = from_f32<T>(x.w);
    }
}
__device__ __forceinline__ void put4_any(const Args &p, size_t at, float4 x, int n)
{
    if (p.out_dtype == ORTHRUS_BF16) put4(static_cast<__nv_bfloat16 *>(p.out) + at, x, n, p.vec);
    else if (p.out_dtype == ORTHRUS_F16) put4(static_cast<__half *>(p.out) + at, x, n, p.vec);
    else put4(static_cast<float *>(p.out) + at, x, n, p.vec);
}

template <int NT, int GRP, int NST>
__global__ void __launch_bounds__(Conf<NT, GRP, NST>::threads, 1)
    fp8_rows_kernel(const __grid_constant__ Maps mp, const Args p)
{
    using C = Conf<NT, GRP, NST>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw);
    const uint32_t b_full = base + C::bars, b_empty = b_full + 8 * NST, b_tfull = b_empty + 8 * NST,
                   b_tempty = b_tfull + 16, b_drain = b_tempty + 16;
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::bars + C::nbars * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_tfull + 8 * i, 1);
            mbar_init(b_tempty + 8 * i, 4);
        }
        mbar_init(b_drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 && lane == 0) {
        tma_prefetch(&mp.w);
        tma_prefetch(&mp.w32);
        tma_prefetch(&mp.w16);
        tma_prefetch(&mp.a);
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::bars +
                                                                                               C::nbars * 8),
                     "r"(C::cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    // this block's weight rows [r_lo, r_hi), token rows from y0, k-blocks [k_lo, k_hi)
    const int rank = blockIdx.x % p.split, unit = blockIdx.x / p.split, range = unit % p.ranges;
    const int g16 = (p.N + 15) >> 4, y0 = unit / p.ranges * NT;
    const int r_lo = 16 * (int)((int64_t)range * g16 / p.ranges);
    int r_hi = 16 * (int)((int64_t)(range + 1) * g16 / p.ranges);
    if (r_hi > p.N) r_hi = p.N;
    const int k_lo = (int)((int64_t)rank * p.nkb / p.split), k_hi = (int)((int64_t)(rank + 1) * p.nkb / p.split);
    const int ng = (k_hi - k_lo + GRP - 1) / GRP;                     // groups of a tile
    pdl_wait();

    if (warp < 4) {
        const int row = warp * 32 + lane;
        const uint32_t t_row = tmem + ((uint32_t)(warp * 32) << 16);
        float *svec = reinterpret_cast<float *>(sm + C::svec);
        float *tile_o = reinterpret_cast<float *>(sm + C::tile);
        // scales of a group, fetched a group ahead: this thread's entries (k-block j, token c)
        constexpr int E = (GRP * NT + 127) / 128;
        float na[E], nw[E][2];
        auto fetch = [&](int x0, int g) {
            const int b0 = x0 >> 7, b1 = b0 + 1 < p.tiles_x ? b0 + 1 : b0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = e * 128 + threadIdx.x, j = i / NT, c = i - j * NT, k = k_lo + g * GRP + j;
                const bool in = i < GRP * NT && k < k_hi && y0 + c < p.M;
                na[e] = in ? __ldg(p.a_scale + (size_t)(y0 + c) * p.nkb + k) : 0.f;
                nw[e][0] = in ? __ldg(p.w_scale + (size_t)b0 * p.nkb + k) : 0.f;
                nw[e][1] = in ? __ldg(p.w_scale + (size_t)b1 * p.nkb + k) : 0.f;
            }
        };
        int it = 0;
        bool ok = true;
        fetch(r_lo, 0);
#pragma unroll 1
        for (int x0 = r_lo; x0 < r_hi; x0 += 128) {
            float acc[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) acc[c] = 0.f;
            const int blk = ((x0 + row) >> 7) - (x0 >> 7);            // 0 or 1: the row's weight block in the tile
#pragma unroll 1
            for (int g = 0; g < ng; ++g, ++it) {
                const int set = it & 1;
                float *sv = svec + set * 2 * GRP * NT;                // [2][GRP][NT]
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = e * 128 + threadIdx.x;
                    if (i < GRP * NT) {
                        sv[i] = na[e] * nw[e][0];
                        sv[GRP * NT + i] = na[e] * nw[e][1];
                    }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");        // (after an abort too: all four warps come here)
                if (g + 1 < ng) fetch(x0, g + 1);
                else if (x0 + 128 < r_hi) fetch(x0 + 128, 0);
                if (ok) ok = __all_sync(~0u, wait_bar_near(b_tfull + 8 * set, (it >> 1) & 1, abort_flag, p.status));
                if (!ok) continue;
                tc_fence_after();
                const float *s = sv + blk * GRP * NT;
                const int here = k_hi - k_lo - g * GRP;               // blocks of this group
                // chunks of 16 columns, the next on its way while one is added
                constexpr int CH = GRP * NT / 16;
                uint32_t v[2][16];
                tmem_ld16(t_row + set * GRP * NT, v[0]);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    tmem_wait_ld();
                    if (c + 1 < CH) {
                        tmem_ld16(t_row + set * GRP * NT + (c + 1) * 16, v[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_tempty + 8 * set);
                    }
                    const uint32_t(&w)[16] = v[c & 1];
                    constexpr int per = NT / 16;
                    const int j = c / per, c0 = c % per * 16;
                    if (j < here) {                                   // (buffers past the last block hold old sums)
#pragma unroll
                        for (int q = 0; q < 16; q += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(s + j * NT + c0 + q);
                            acc[c0 + q] = fmaf(__uint_as_float(w[q]), f.x, acc[c0 + q]);
                            acc[c0 + q + 1] = fmaf(__uint_as_float(w[q + 1]), f.y, acc[c0 + q + 1]);
                            acc[c0 + q + 2] = fmaf(__uint_as_float(w[q + 2]), f.z, acc[c0 + q + 2]);
                            acc[c0 + q + 3] = fmaf(__uint_as_float(w[q + 3]), f.w, acc[c0 + q + 3]);
                        }
                    }
                }
            }
            // ---- out: through shared memory, so that the stores are runs of a token's row
#pragma unroll
            for (int c = 0; c < NT; ++c) tile_o[c * 128 + row] = acc[c];
            if (p.split > 1) break;                                   // (one tile: joined below)
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int rows = r_hi - x0 < 128 ? r_hi - x0 : 128;
            if (!*abort_flag) {
#pragma unroll 1
                for (int c = warp; c < NT && y0 + c < p.M; c += 4)
                    if (lane * 4 < rows)
                        put4_any(p, (size_t)(y0 + c) * p.N + x0 + lane * 4,
                                 *reinterpret_cast<const float4 *>(tile_o + c * 128 + lane * 4), rows - lane * 4);
            }
            // (the next tile's sums are written after the group barriers above: at least one)
        }
    } else if (warp == 4) {
        if (elect_one()) {
            const uint64_t once = make_policy_evict_first(), keep = make_policy_evict_last();
            const uint64_t pw = p.tiles_y > 1 ? keep : once;
            int it = 0;
            bool ok = true;
            for (int x0 = r_lo; x0 < r_hi && ok; x0 += 128) {
                const int rows = r_hi - x0 < 128 ? (r_hi - x0 + 15) & ~15 : 128;
#pragma unroll 1
                for (int g = 0; g < ng; ++g, ++it) {
                    const int st = it % NST, n = it / NST;
                    if (n > 0) ok = wait_bar_near(b_empty + 8 * st, (n - 1) & 1, abort_flag, p.status);
                    if (!ok) break;
                    const int k0 = k_lo + g * GRP, here = k_hi - k0 < GRP ? k_hi - k0 : GRP;
                    const uint32_t full = b_full + 8 * st, dx = base + st * C::stage, dy = dx + GRP * kXBytes;
                    mbar_expect_tx(full, here * (rows * 128 + NT * 128));
                    for (int j = 0; j < here; ++j) {
                        if (rows == 128) {
                            tma_load_2d_hint(dx + j * kXBytes, &mp.w, full, (k0 + j) * 128, x0, pw);
                        } else {
                            int r = 0;
                            for (; r + 32 <= rows; r += 32)
                                tma_load_2d_hint(dx + j * kXBytes + r * 128, &mp.w32, full, (k0 + j) * 128, x0 + r, pw);
                            if (r < rows)
                                tma_load_2d_hint(dx + j * kXBytes + r * 128, &mp.w16, full, (k0 + j) * 128, x0 + r, pw);
                        }
                    }
                    for (int j = 0; j < here; ++j)
                        tma_load_2d_hint(dy + j * NT * 128, &mp.a, full, (k0 + j) * 128, y0, keep);
                }
            }
            if (!ok) {                                                // abort: let the copies in flight land
                for (int st = 0; st < NST; ++st) {
                    const int fills = it / NST + (st < it % NST ? 1 : 0);
                    if (fills) wait_bar_quiet(b_full + 8 * st, (fills - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else {
        if (elect_one()) {
            constexpr uint32_t idesc = instr_desc_e4m3(128, NT);
            const int steps = (r_hi - r_lo + 127) / 128 * ng;
            bool ok = true;
            int g = 0;
#pragma unroll 1
            for (int it = 0; it < steps; ++it) {
                const int st = it % NST, set = it & 1, n = it >> 1;
                ok = wait_bar_near(b_full + 8 * st, (it / NST) & 1, abort_flag, p.status) &&
                     (n == 0 || wait_bar_near(b_tempty + 8 * set, (n - 1) & 1, abort_flag, p.status));
                if (!ok) break;
                tc_fence_after();
                const int here = k_hi - k_lo - g * GRP;
                if (++g == ng) g = 0;
                const uint32_t dx = base + st * C::stage;
                const uint64_t aw = smem_desc(dx, 16, 1024), at = smem_desc(dx + GRP * kXBytes, 16, 1024);
#pragma unroll
                for (int j = 0; j < GRP; ++j) {
                    if (j < here) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tc_mma_f8(tmem + (set * GRP + j) * NT, aw + j * (kXBytes >> 4) + 2 * q,
                                      at + j * (NT * 128 >> 4) + 2 * q, idesc, q);
                    }
                }
                tc_commit(b_tfull + 8 * set);
                tc_commit(b_empty + 8 * st);
            }
            if (!ok) {
                tc_commit(b_drain);
                wait_bar_quiet(b_drain, 0);
            }
        }
        __syncwarp();
    }

    if (p.split > 1) {
        // each rank writes its share of the token rows, added over the ranks in order
        cluster_sync();
        if (!*abort_flag) {
#pragma unroll 1
            for (int c = rank + warp * p.split; c < NT; c += 6 * p.split) {
                const int n = r_lo + lane * 4;
                if (y0 + c >= p.M || n >= r_hi) continue;
                const uint32_t at = base + C::tile + (uint32_t)(c * 128 + lane * 4) * 4u;
                float4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < p.split) v[r] = ld_cluster_f32x4(at, r);
                float4 x = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < p.split) x.x += v[r].x, x.y += v[r].y, x.z += v[r].z, x.w += v[r].w;
                put4_any(p, (size_t)(y0 + c) * p.N + n, x, r_hi - n);
            }
        }
        cluster_sync_relaxed();                                       // no block leaves while its partials are read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::cols) : "memory");
    }
}

}  // namespace f8
}  // namespace orthrus

#include "fp8_pair.cuh"

namespace orthrus {
namespace f8 {

constexpr int kMaxDevices = 64;

// Per device: the kernel's shared memory allowed, and how many clusters of 1, 2,
// 4 and 8 of its blocks the device holds at once (clusters do not cross the
// device's processor groups, so these are fewer than SMs / size).
template <int NT, int GRP, int NST> const int *rows_ready(int dev)
{
    static std::once_flag once[kMaxDevices];
    static int held[kMaxDevices][4];
    if (dev < 0 || dev >= kMaxDevices) return nullptr;
    std::call_once(once[dev], [dev] {
        using C = Conf<NT, GRP, NST>;
        bool ok = cudaFuncSetAttribute(fp8_rows_kernel<NT, GRP, NST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::total) == cudaSuccess;
        for (int i = 0; i < 4 && ok; ++i) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << i);
            cfg.blockDim = dim3(C::threads);
            cfg.dynamicSmemBytes = C::total;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << i;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            ok = cudaOccupancyMaxActiveClusters(&held[dev][i], fp8_rows_kernel<NT, GRP, NST>, &cfg) == cudaSuccess;
        }
        if (!ok) {
            cudaGetLastError();
            held[dev][0] = 0;
        }
    });
    return held[dev][0] > 0 ? held[dev] : nullptr;
}

template <int NT, int GRP, int NST>
int launch_rows(Args &p, const void *a, const void *w, int dev, cudaStream_t st)
{
    using C = Conf<NT, GRP, NST>;
    p.tiles_x = (p.N + 127) / 128;
    p.tiles_y = (p.M + NT - 1) / NT;
    const uintptr_t oe = (uintptr_t)elem_size(p.out_dtype);
    p.vec = ((uintptr_t)p.out & (4 * oe - 1)) == 0 && p.N % 4 == 0   ? 4
            : ((uintptr_t)p.out & (2 * oe - 1)) == 0 && p.N % 2 == 0 ? 2
                                                                     : 1;
    const int *held = rows_ready<NT, GRP, NST>(dev);
    if (!held) return ORTHRUS_ERR_LAUNCH;
    // The largest K split whose clusters, all resident at once, cover the weight
    // rows with one tile of up to 128 rows each: a second wave of clusters costs
    // a whole kernel time (32 x 6144 x 4096: 48 clusters of 3, of which 46 fit,
    // took 13.4 us).
    const int g16 = (p.N + 15) / 16;
    int split = 1;
    p.ranges = p.tiles_y >= held[0] ? 1 : held[0] / p.tiles_y;
    for (int i = 1; i < 4; ++i) {
        const int r = held[i] / p.tiles_y;
        if ((int64_t)r * 8 < g16 || (1 << i) > p.nkb) continue;
        split = 1 << i;
        p.ranges = r;
    }
    if (p.ranges > g16) p.ranges = g16;
    p.split = split;
    const int64_t blocks = (int64_t)p.ranges * p.tiles_y * split;
    if (blocks >= 1ll << 31) return ORTHRUS_ERR_UNSUPPORTED;
    Maps mp;
    const uint64_t str[1] = {(uint64_t)p.K};
    const uint64_t dw[2] = {(uint64_t)p.K, (uint64_t)p.N}, da[2] = {(uint64_t)p.K, (uint64_t)p.M};
    const uint32_t bw[2] = {128, 128}, b32[2] = {128, 32}, b16[2] = {128, 16}, ba[2] = {128, NT};
    if (!encode_u8_sw128(&mp.w, 2, w, dw, str, bw) || !encode_u8_sw128(&mp.w32, 2, w, dw, str, b32) ||
        !encode_u8_sw128(&mp.w16, 2, w, dw, str, b16) ||
        !encode_u8_sw128(&mp.a, 2, a, da, str, ba))
        return ORTHRUS_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(C::threads);
    cfg.dynamicSmemBytes = C::total;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_rows_kernel<NT, GRP, NST>, mp, p);
    return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_LAUNCH;
}

template <typename T, bool TMA> bool pair_ready(int dev)
{
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return false;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(fp8_pair_kernel<T, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PairConf::total) == cudaSuccess;
        if (!ok[dev]) cudaGetLastError();
    });
    return ok[dev];
}

template <typename T>
int launch_pair_t(Args &p, const void *a, const void *w, int dev, int sms, cudaStream_t st)
{
    using C = PairConf;
    p.tiles_x = (p.M + 255) / 256;
    p.tiles_y = (p.N + kPairN - 1) / kPairN;
    const int64_t tiles = (int64_t)p.tiles_x * p.tiles_y;
    const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
    if (tiles >= 1ll << 30 || (tiles / pairs + 1) * p.nkb >= 1ll << 31) return ORTHRUS_ERR_UNSUPPORTED;   // (32-bit steps)
    const uintptr_t oa = (uintptr_t)p.out;
    const int64_t row = (int64_t)p.N * (int)sizeof(T);
    p.vec = (oa & 15u) == 0 && row % 16 == 0 && row < 1ll << 31 ? 16 / (int)sizeof(T)
            : (oa & (2 * sizeof(T) - 1)) == 0 && p.N % 2 == 0   ? 2
                                                                : 1;
    PairMaps mp;
    const uint64_t str[1] = {(uint64_t)p.K}, ostr[1] = {(uint64_t)p.N * sizeof(T)};
    const uint64_t dx[2] = {(uint64_t)p.K, (uint64_t)p.M}, dy[2] = {(uint64_t)p.K, (uint64_t)p.N},
                   dz[2] = {(uint64_t)p.N * sizeof(T), (uint64_t)p.M};
    const uint32_t bx[2] = {128, 128}, by[2] = {128, 64};
    if (!encode_u8_sw128(&mp.x, 2, a, dx, str, bx) || !encode_u8_sw128(&mp.y, 2, w, dy, str, by)) return ORTHRUS_ERR_LAUNCH;
    if (p.vec > 2) {
        if (!encode_u8_sw128(&mp.o, 2, p.out, dz, ostr, bx)) return ORTHRUS_ERR_LAUNCH;
    } else {
        mp.o = mp.x;                                                  // (not used)
    }
    const bool tma = p.vec > 2;
    if (!(tma ? pair_ready<T, true>(dev) : pair_ready<T, false>(dev))) return ORTHRUS_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = C::total;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = tma ? cudaLaunchKernelEx(&cfg, fp8_pair_kernel<T, true>, mp, p)
                              : cudaLaunchKernelEx(&cfg, fp8_pair_kernel<T, false>, mp, p);
    return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_LAUNCH;
}

int launch_pair(Args &p, const void *a, const void *w, int dev, int sms, cudaStream_t st)
{
    return p.out_dtype == ORTHRUS_BF16  ? launch_pair_t<__nv_bfloat16>(p, a, w, dev, sms, st)
           : p.out_dtype == ORTHRUS_F16 ? launch_pair_t<__half>(p, a, w, dev, sms, st)
                                        : launch_pair_t<float>(p, a, w, dev, sms, st);
}

}  // namespace f8

}  // namespace orthrus

using namespace orthrus;

extern "C" int orthrus_fp8_matmul(const void *a, const float *a_scale, const void *w, const float *w_scale, int M, int N,
                                  int K, orthrus_dtype out_dtype, void *out, int32_t *status, void *stream)
{
    if (!a || !a_scale || !w || !w_scale || !out || M <= 0 || N <= 0 || K <= 0) return ORTHRUS_ERR_ARG;
    const int e = elem_size(out_dtype);
    if (!e) return ORTHRUS_ERR_ARG;
    if (K % 16 || K > 1 << 30 || M > 1 << 30 || N > 1 << 30) return ORTHRUS_ERR_UNSUPPORTED;
    if (((uintptr_t)a | (uintptr_t)w) & 15u) return ORTHRUS_ERR_ALIGN;
    if (((uintptr_t)out & (uintptr_t)(e - 1)) || (((uintptr_t)a_scale | (uintptr_t)w_scale) & 3u)) return ORTHRUS_ERR_ALIGN;
    int dev = 0, sms = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ORTHRUS_ERR_DEVICE;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (sms <= 0 || major != 10) return ORTHRUS_ERR_DEVICE;
    f8::Args p = {};
    p.a_scale = a_scale;
    p.w_scale = w_scale;
    p.out = out;
    p.status = status;
    p.M = M;
    p.N = N;
    p.K = K;
    p.nkb = (K + ORTHRUS_FP8_BLOCK - 1) / ORTHRUS_FP8_BLOCK;
    p.out_dtype = out_dtype;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M <= 16) return f8::launch_rows<16, 4, 3>(p, a, w, dev, st);
    if (M <= 32) return f8::launch_rows<32, 4, 2>(p, a, w, dev, st);
    if (M <= 64) return f8::launch_rows<64, 2, 3>(p, a, w, dev, st);
    // Pairs from 129 rows on, unless their 256 x 256 tiles (no K split) would be so few
    // that the row form can give each tile of 128 x 128 two SMs, which split K.  At
    // K = 4096, by rows and by pairs: 256 x 4608 14.2 and 19.6 us, 1024 x 1152 14.0 and
    // 19.7, 8192 x 128 15.3 and 19.6; without a split 256 x 5120 21.1 and 19.8, 1024 x
    // 1280 20.8 and 19.7, 512 x 6144 39.3 and 21.0.  (K <= 256: within 0.7 us.)
    const int weight_tiles = sms / 2 / ((M + 127) / 128);
    if (M <= 128 || (int64_t)weight_tiles * 128 >= N) return f8::launch_rows<128, 2, 2>(p, a, w, dev, st);
    return f8::launch_pair(p, a, w, dev, sms, st);
}
