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
// Two forms of one kernel.  SWAP (few token rows): the weight rows are the
// MMA's 128 rows and up to 128 token rows its columns, so that no part of the
// MMA is padding and the weights are streamed once; bound by HBM.  Otherwise a
// thread owns a token row of a 128 x NT tile; bound by the tensor cores.  A K
// split over a cluster of blocks (partials joined through distributed shared
// memory, in rank order) fills the SMs where there are few tiles.
//
// Roles: warps 0..EW-1 epilogue, then a TMA producer warp and an MMA warp.
#include <mutex>

#include "kernels.h"
#include "layer_ops.cuh"

namespace orthrus {

namespace f8 {

using namespace sm100;

struct Maps {
    CUtensorMap x, y;                    // 128-row operand (box 128 x 128), NT-row operand (box 128 x NT)
};

struct Args {
    const float *a_scale, *w_scale;
    void *out;
    int32_t *status;
    int M, N, K, nkb;
    int split;                           // blocks of a cluster, along K
    int tiles_x, tiles_y;                // tiles of the 128-row operand, of the other
    int out_dtype;
    int vec;                             // every fourth column of out is aligned for four
};

constexpr int kXBytes = 128 * 128;
constexpr int kRing = 192 * 1024;

template <int NT, bool SWAP, int CPS> struct Conf {
    static constexpr int EW = NT > 128 ? 8 : 4;                       // epilogue warps
    static constexpr int CPT = NT > 128 ? NT / 2 : NT;                // columns of a thread
    static constexpr int threads = (EW + 2) * 32;
    static constexpr int stage = CPS * (kXBytes + NT * 128);
    static constexpr int nst = kRing / stage;
    static constexpr int nbuf = NT > 128 ? 2 : 4;                     // TMEM buffers
    static constexpr int cols = nbuf * NT;                            // a power of two, >= 32
    static constexpr int scales = 2 * 4 * (SWAP ? NT : EW * 32) * 4;  // two groups of four k-blocks' scales
    // the output tile on its way out, [token row][weight row] in fp32 in place of the ring
    static constexpr int lines = SWAP ? NT : 128, len = SWAP ? 128 : NT, pitch = SWAP ? 128 : NT + 4;
    // barriers: stage full / empty, buffer full / empty, drain
    static constexpr int bars = nst * stage;
    static constexpr int nbars = 2 * nst + 2 * nbuf + 1;
    static constexpr int svec = (bars + nbars * 8 + 16 + 15) & ~15;
    static constexpr int total = svec + scales + 1024;
    static_assert(nst >= 2 && lines * pitch * 4 <= nst * stage, "ring");
};

// Four consecutive columns of one row, the first n of them inside the matrix.
template <typename T> __device__ __forceinline__ void put4(T *out, float4 x, int n, bool vec)
{
    if (vec && n >= 4) {
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

template <int NT, bool SWAP, int CPS>
__global__ void __launch_bounds__(Conf<NT, SWAP, CPS>::threads, 1)
    fp8_matmul_kernel(const __grid_constant__ Maps mp, const Args p)
{
    using C = Conf<NT, SWAP, CPS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw);
    const uint32_t b_full = base + C::bars, b_empty = b_full + 8 * C::nst, b_tfull = b_empty + 8 * C::nst,
                   b_tempty = b_tfull + 8 * C::nbuf, b_drain = b_tempty + 8 * C::nbuf;
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::bars + C::nbars * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::nst; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < C::nbuf; ++i) {
            mbar_init(b_tfull + 8 * i, 1);
            mbar_init(b_tempty + 8 * i, C::EW);
        }
        mbar_init(b_drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::EW && lane == 0) {
        tma_prefetch(&mp.x);
        tma_prefetch(&mp.y);
    }
    if (warp == C::EW + 1) {
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

    const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
    const int tx = tile % p.tiles_x, ty = tile / p.tiles_x;
    const int x0 = tx * 128, y0 = ty * NT;
    const int k_lo = (int)((int64_t)rank * p.nkb / p.split), k_hi = (int)((int64_t)(rank + 1) * p.nkb / p.split);
    const int nk = k_hi - k_lo;
    pdl_wait();

    float acc[C::CPT];
#pragma unroll
    for (int i = 0; i < C::CPT; ++i) acc[i] = 0.f;
    bool ok = true;

    if (warp < C::EW) {
        const int half = warp >> 2;                                   // which CPT columns
        const int row = (warp & 3) * 32 + lane;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * C::CPT;
        // scales of a group of four k-blocks, fetched one group ahead: of the
        // thread's own row, or (SWAP) of the columns, shared by the four warps.
        // They go through shared memory in both forms so that the loop over
        // k-blocks is one small body: unrolled over a group it drove the
        // producer's and the MMA warp's code out of the instruction cache, and
        // each of their steps took ~350 cycles.
        constexpr int NS = SWAP ? NT : C::EW * 32;
        float *svec = reinterpret_cast<float *>(sm + C::svec);        // [2][4][NS]
        float next[4];
        const int sr = SWAP ? y0 + (int)threadIdx.x : x0 + row;
        const bool mine = sr < p.M && (SWAP ? (int)threadIdx.x < NT : y0 + half * 128 < p.N);
        const float *sa = p.a_scale + (size_t)(mine ? sr : 0) * p.nkb;
        const float *sw = p.w_scale + (size_t)(SWAP ? tx : mine ? (y0 + half * 128) / 128 : 0) * p.nkb;
        auto fetch = [&](int k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) next[j] = mine && k + j < k_hi ? __ldg(sa + k + j) * __ldg(sw + k + j) : 0.f;
        };
        fetch(k_lo);
#pragma unroll 1
        for (int it = 0; it < nk; ++it) {
            if ((it & 3) == 0) {                   // (after an abort too: the warps meet at barrier 1)
                float *sv = svec + ((it >> 2) & 1) * 4 * NS;
                if (!SWAP || (int)threadIdx.x < NT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) sv[j * NS + threadIdx.x] = next[j];
                }
                if (SWAP) asm volatile("bar.sync 1, 128;" ::: "memory");
                fetch(k_lo + it + 4);
            }
            if (!ok) continue;
            const float *sv = svec + (it & 7) * NS;
            const float own_scale = SWAP ? 0.f : sv[threadIdx.x];
            const int buf = it % C::nbuf;
            ok = __all_sync(~0u, wait_bar_near(b_tfull + 8 * buf, (it / C::nbuf) & 1, abort_flag, p.status));
            if (!ok) continue;
            tc_fence_after();
            constexpr int W = C::CPT < 32 ? 16 : 32;
#pragma unroll
            for (int c = 0; c < C::CPT; c += W) {
                uint32_t v[W];
                if constexpr (W == 32) tmem_ld32(t_row + buf * NT + c, v);
                else tmem_ld16(t_row + buf * NT + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < W; q += 4) {
                    const float4 s = SWAP ? *reinterpret_cast<const float4 *>(sv + c + q)
                                          : make_float4(own_scale, own_scale, own_scale, own_scale);
                    const float2 u = ffma2(make_float2(__uint_as_float(v[q]), __uint_as_float(v[q + 1])),
                                           make_float2(s.x, s.y), make_float2(acc[c + q], acc[c + q + 1]));
                    const float2 w = ffma2(make_float2(__uint_as_float(v[q + 2]), __uint_as_float(v[q + 3])),
                                           make_float2(s.z, s.w), make_float2(acc[c + q + 2], acc[c + q + 3]));
                    acc[c + q] = u.x, acc[c + q + 1] = u.y, acc[c + q + 2] = w.x, acc[c + q + 3] = w.y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_tempty + 8 * buf);
        }
    } else if (warp == C::EW) {
        if (lane == 0) {
            const uint64_t first = make_policy_evict_first(), last = make_policy_evict_last();
            const uint64_t px = SWAP ? first : last;                  // streamed once, or re-read by other tiles
            const int ns = (nk + CPS - 1) / CPS;
            int it = 0;
            for (; it < ns; ++it) {
                const int st = it % C::nst, n = it / C::nst;
                if (n > 0 && !wait_bar_near(b_empty + 8 * st, (n - 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                const int here = nk - it * CPS < CPS ? nk - it * CPS : CPS;
                const uint32_t full = b_full + 8 * st, dx = base + st * C::stage, dy = dx + CPS * kXBytes;
                mbar_expect_tx(full, here * (kXBytes + NT * 128));
                for (int j = 0; j < here; ++j) {
                    const int k = (k_lo + it * CPS + j) * 128;
                    tma_load_2d_hint(dx + j * kXBytes, &mp.x, full, k, x0, px);
                    tma_load_2d_hint(dy + j * NT * 128, &mp.y, full, k, y0, last);
                }
            }
            if (!ok) {                                                // abort: let the copies in flight land
                for (int st = 0; st < C::nst; ++st) {
                    const int fills = it / C::nst + (st < it % C::nst ? 1 : 0);
                    if (fills) wait_bar_quiet(b_full + 8 * st, (fills - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            const uint32_t idesc = instr_desc_e4m3(128, NT);
            const int ns = (nk + CPS - 1) / CPS;
            for (int it = 0; it < ns && ok; ++it) {
                const int st = it % C::nst;
                if (!wait_bar_near(b_full + 8 * st, (it / C::nst) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int j = 0; j < CPS && it * CPS + j < nk; ++j) {
                    const int kb = it * CPS + j, buf = kb % C::nbuf, n = kb / C::nbuf;
                    if (n > 0 && !wait_bar_near(b_tempty + 8 * buf, (n - 1) & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t dx = base + st * C::stage + j * kXBytes,
                                   dy = base + st * C::stage + CPS * kXBytes + j * NT * 128;
                    const uint64_t ax = smem_desc(dx, 16, 1024), ay = smem_desc(dy, 16, 1024);
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_mma_f8(tmem + buf * NT, ax + 2 * q, ay + 2 * q, idesc, q);
                    tc_commit(b_tfull + 8 * buf);
                }
                if (ok) tc_commit(b_empty + 8 * st);
            }
            if (!ok) {
                tc_commit(b_drain);
                wait_bar_quiet(b_drain, 0);
            }
        }
        __syncwarp();
    }

    // ---- output: the tile goes through shared memory (the ring: every load has
    // been consumed) so that the stores are whole rows of it; with a split each
    // rank writes its share of the token rows, added over the ranks in order.
    float *tile_o = reinterpret_cast<float *>(sm);
    __syncthreads();
    if (warp < C::EW) {
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        if (SWAP) {
#pragma unroll
            for (int c = 0; c < C::CPT; ++c) tile_o[c * C::pitch + row] = acc[c];
        } else {
#pragma unroll
            for (int c = 0; c < C::CPT; c += 4)
                *reinterpret_cast<float4 *>(tile_o + row * C::pitch + half * C::CPT + c) =
                    make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        }
    }
    if (p.split > 1) cluster_sync();
    else __syncthreads();
    const int m0 = SWAP ? y0 : x0, n0 = SWAP ? x0 : y0;
    if (!*abort_flag) {
        constexpr int per = C::len / 4;                               // threads of a token row
#pragma unroll 1
        for (int i = threadIdx.x; i < C::lines * per; i += C::threads) {
            const int line = i / per, e = (i % per) * 4;
            const int m = m0 + line, n = n0 + e;
            if (m >= p.M || n >= p.N || (p.split > 1 && line % p.split != rank)) continue;
            float4 x;
            if (p.split > 1) {
                x = make_float4(0.f, 0.f, 0.f, 0.f);
                const uint32_t at = base + (uint32_t)(line * C::pitch + e) * 4u;
                for (int r = 0; r < p.split; ++r) {
                    const float4 v = ld_cluster_f32x4(at, r);
                    x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
                }
            } else {
                x = *reinterpret_cast<const float4 *>(tile_o + line * C::pitch + e);
            }
            const size_t at = (size_t)m * p.N + n;
            if (p.out_dtype == ORTHRUS_BF16) put4(static_cast<__nv_bfloat16 *>(p.out) + at, x, p.N - n, p.vec);
            else if (p.out_dtype == ORTHRUS_F16) put4(static_cast<__half *>(p.out) + at, x, p.N - n, p.vec);
            else put4(static_cast<float *>(p.out) + at, x, p.N - n, p.vec);
        }
    }
    if (p.split > 1) cluster_sync();                                  // no block leaves while its partials are read
    tc_fence_before();
    __syncthreads();
    if (warp == C::EW + 1) {
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

template <int NT, bool SWAP, int CPS> bool smem_ready(int dev)
{
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return false;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(fp8_matmul_kernel<NT, SWAP, CPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Conf<NT, SWAP, CPS>::total) == cudaSuccess;
        if (!ok[dev]) cudaGetLastError();
    });
    return ok[dev];
}

template <int NT, bool SWAP, int CPS>
int launch(Args &p, const void *a, const void *w, int dev, int sms, cudaStream_t st)
{
    using C = Conf<NT, SWAP, CPS>;
    static_assert(C::total <= 227 * 1024, "shared memory");
    const void *x = SWAP ? w : a, *y = SWAP ? a : w;
    const int xr = SWAP ? p.N : p.M, yr = SWAP ? p.M : p.N;
    p.tiles_x = (xr + 127) / 128;
    p.tiles_y = (yr + NT - 1) / NT;
    const int64_t tiles = (int64_t)p.tiles_x * p.tiles_y;
    // fewer tiles than half the SMs: split K over a cluster
    int split = (int)(tiles * 2 <= sms ? sms / tiles : 1);
    if (split > 8) split = 8;
    if (split > p.nkb) split = p.nkb;
    p.split = split;
    if (tiles * split >= 1ll << 31) return ORTHRUS_ERR_UNSUPPORTED;
    Maps mp;
    const uint64_t str[1] = {(uint64_t)p.K};
    const uint64_t dx[2] = {(uint64_t)p.K, (uint64_t)xr}, dy[2] = {(uint64_t)p.K, (uint64_t)yr};
    const uint32_t bx[2] = {128, 128}, by[2] = {128, NT};
    if (!encode_u8_sw128(&mp.x, 2, x, dx, str, bx) || !encode_u8_sw128(&mp.y, 2, y, dy, str, by)) return ORTHRUS_ERR_LAUNCH;
    if (!smem_ready<NT, SWAP, CPS>(dev)) return ORTHRUS_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_matmul_kernel<NT, SWAP, CPS>, mp, p);
    return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_LAUNCH;
}

template <typename T> bool pair_ready(int dev)
{
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return false;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(fp8_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    if (tiles >= 1ll << 28) return ORTHRUS_ERR_UNSUPPORTED;
    p.vec = ((uintptr_t)p.out & 15u) == 0 && (int64_t)p.N * (int)sizeof(T) % 16 == 0 &&
            (int64_t)p.N * (int)sizeof(T) < 1ll << 31;
    PairMaps mp;
    const uint64_t str[1] = {(uint64_t)p.K}, ostr[1] = {(uint64_t)p.N * sizeof(T)};
    const uint64_t dx[2] = {(uint64_t)p.K, (uint64_t)p.M}, dy[2] = {(uint64_t)p.K, (uint64_t)p.N},
                   dz[2] = {(uint64_t)p.N * sizeof(T), (uint64_t)p.M};
    const uint32_t bx[2] = {128, 128}, by[2] = {128, 128};
    if (!encode_u8_sw128(&mp.x, 2, a, dx, str, bx) || !encode_u8_sw128(&mp.y, 2, w, dy, str, by)) return ORTHRUS_ERR_LAUNCH;
    if (p.vec) {
        if (!encode_u8_sw128(&mp.o, 2, p.out, dz, ostr, bx)) return ORTHRUS_ERR_LAUNCH;
    } else {
        mp.o = mp.x;                                                  // (not used)
    }
    if (!pair_ready<T>(dev)) return ORTHRUS_ERR_LAUNCH;
    const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_pair_kernel<T>, mp, p);
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
    if (K % 16) return ORTHRUS_ERR_UNSUPPORTED;
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
    p.vec = ((uintptr_t)out & (uintptr_t)(4 * e - 1)) == 0 && N % 4 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M <= 16) return f8::launch<16, true, 4>(p, a, w, dev, sms, st);
    if (M <= 32) return f8::launch<32, true, 4>(p, a, w, dev, sms, st);
    if (M <= 64) return f8::launch<64, true, 2>(p, a, w, dev, sms, st);
    if (M <= 128) return f8::launch<128, true, 2>(p, a, w, dev, sms, st);
    return f8::launch_pair(p, a, w, dev, sms, st);
}
