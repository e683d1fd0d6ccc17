// Attention of one new token per sequence over a paged KV cache, split over the
// cache's length and joined in the same launch.
//
//     out[b,h] = sum_j softmax_j(scale <q[b,h], K[b,g,j]>) V[b,g,j],  j < len_b
//
// What bounds it: each key and value is used by the G = Hq / Hkv query heads of
// its KV head only, 2 G flop per byte, so the keys and values are streamed once
// from HBM and everything else has to hide behind that stream, within the
// board's power: under a sustained load that reaches the power limit the clocks,
// and the memory rate with them, fall (by 11 % for twice the matrix
// instructions).  Measured, 8 KV heads of 128: 8 long sequences of 273,000 keys in
// all 170 us (6.6 TB/s, a copy's rate; 178 to 186 at the power limit), 16 ragged ones
// of 154,000 103 us (94 %), one of 300 keys 7.7.  G <= 16 rows would fill an eighth of
// a tcgen05 tile's 128 and pay its TMEM round trips per tile, so the products run
// on mma.sync m16n8k16, transposed: 16 keys (then 16 dims) are the instruction's rows and 8 heads its
// columns, so that up to 8 heads waste nothing.  The weights go from the first
// product's layout to the second's by 8 x 8 transposes in registers.
//
// Work split: every sequence's keys are cut into tiles of 64 (128 for D = 64);
// the tiles of all (sequence, KV head, group of 16 heads) segments are laid end
// to end and cut into equal contiguous ranges, one per block, computed on the device from
// ctx_lens.  Each of the block's four warps takes a quarter of a tile and runs its
// own cp.async ring and its own running maximum and sum (no block-wide barrier
// inside a segment); the four are combined through shared memory when the block
// leaves a segment.  A segment that spans blocks is joined by the last of them
// to arrive, which adds the partials in block order.  Its counter is the one of its
// first block (a block leaves at most one segment unfinished), so the counters'
// place does not depend on a call's shape: calls of any shapes can share a workspace.
//
// Numerics: q.k in fp32 from exact products, running maximum with a lazy
// rescale (only when a row's maximum grows by more than 2^8), p = 2^(s - m) split
// into 16-bit terms for the second product: three of bf16, which hold all of p's 24
// bits, or two of fp16, 22 bits.  (The third of bf16 hides behind the stream for up
// to 8 heads: 168.8 and 169.1 us for 8 long sequences; 16 heads take 61.2 and 63.5
// us, of 256 values 126 and 138.)  fp16
// weights are held 2^7 up (2^15 at most): a step of 2^-24 at the bottom of the
// type's range, against a largest weight of 1, lost up to 0.8 % of the many small
// weights of a long cache beside one dominant key.
#include <math.h>

#include <mutex>
#include <type_traits>

#include "kernels.h"
#include "layer_ops.cuh"

namespace orthrus {

namespace paged {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                        // query heads per segment, at most
constexpr int kMaxB = 4096;
constexpr float kLazy = 8.f;                     // log2 units

struct Args {
    const void *q, *k_pages, *v_pages;
    const int32_t *block_table, *ctx_lens;
    void *out;
    int32_t *counters;                           // [2 * SMs], zero between calls
    float *part_ml;                              // [2 * grid][kRows][2]: maximum, sum
    float *part_o;                               // [2 * grid][rows][D], not normalised
    int32_t *status;
    int n_new, B, Hq, Hkv, G, HG;                // HG: groups of 16 heads per KV head
    int num_pages, page_size, max_pages;
    float scale_log2;
};

__device__ __forceinline__ int visible(const Args &p, int b, bool report)
{
    const int c = p.ctx_lens[b];
    const int64_t n = (int64_t)c + p.n_new;
    if (c < 0 || n > (int64_t)p.max_pages * p.page_size) {
        if (report) raise_status(p.status, ORTHRUS_STATUS_CAPACITY);
        return 0;
    }
    return (int)n;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

// Transpose of an 8 x 8 matrix of 16-bit values spread over the warp (row lane / 4).
__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two weights as sums of 16-bit terms, each term's two values packed.  Every term
// but the last is the largest value below what it stands for, so that none is zero
// or negative beside a weight that is not, and an infinite value of a key stays the
// infinity it is (0 times it would be a NaN).  (Up to 1 % of a call's time.)
__device__ __forceinline__ float below(float x)          // x >= 0; 0 stays
{
    const uint32_t u = __float_as_uint(x);
    return __uint_as_float(u - (u < 1u ? u : 1u));
}
template <typename T> struct Split;
template <> struct Split<__nv_bfloat16> {
    static constexpr int terms = 3;                      // truncated to 8 bits each, exact together
    static __device__ __forceinline__ void of(float a, float b, uint32_t (&w)[3])
    {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t x = __float_as_uint(i < 2 ? below(a) : a), y = __float_as_uint(i < 2 ? below(b) : b);
            w[i] = __byte_perm(x, y, 0x7632);
            a -= __uint_as_float(x & 0xffff0000u);
            b -= __uint_as_float(y & 0xffff0000u);
        }
    }
};
template <> struct Split<__half> {
    static constexpr int terms = 2;
    static __device__ __forceinline__ void of(float a, float b, uint32_t (&w)[2])
    {
        const __half2 h = __halves2half2(__float2half_rz(below(a)), __float2half_rz(below(b)));
        w[0] = *reinterpret_cast<const uint32_t *>(&h);
        const float2 back = unpack2<__half>(w[0]);
        w[1] = pack2<__half>(a - back.x, b - back.y);
    }
};

// Position in the flat tile order: sequence b, segment g (KV head x head
// group), tile t of its n tiles.
struct Pos {
    int b, g, t, n, len;
};

// Shared memory of one block: the warps' rings, the running maxima and sums at
// a segment's end, the rings' key masks, and after them the first flat tile of
// every sequence (prefix, in tiles of one segment).
template <int D> struct Layout {
    // keys per warp and tile: 8 KB of keys and values, so that a tile's fixed
    // costs (lookup, softmax, signals) weigh the same for heads of 64 and 128
    static constexpr int kStrip = D == 64 ? 32 : 16, kTile = kWarps * kStrip;
    static constexpr int kStripBytes = kStrip * D * 2;               // keys (or values) of a strip
    static constexpr int kStages = 3;
    static constexpr int kRing = kWarps * kStages * 2 * kStripBytes;
    static constexpr int kML = kWarps * kRows * 2 * 4;               // m, l per warp and row
    static constexpr int kMask = kWarps * kStages * 4;
    static constexpr int kFixed = kRing + kML + kMask;
    // a warp's O of 16 rows takes the place of the strip it has just read
    static_assert(2 * kStripBytes >= kRows * D * 4 && 2 * kStripBytes >= 2048, "O and a join's sums fit a stage");
};

// A row's joint maximum and 1 / sum over a segment's n partials (0 and 0 where no
// key was seen; a sum that is not a number stays one), LP lanes per row.
template <int LP, class S>
__device__ __forceinline__ void join_statistics(const Args &p, int rows, int n, S slot_of, float2 *seg_ml)
{
    const int r = threadIdx.x / LP;
    float M = -INFINITY, l = 0.f;
    if (r < rows) {
#pragma unroll 8
        for (int j = threadIdx.x % LP; j < n; j += LP) {
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + (slot_of(j) + r) * 2));
            const float m = fmaxf(M, ml.x);
            if (m != -INFINITY) l = l * fast_exp2(M - m) + ml.y * fast_exp2(ml.x - m);
            M = m;
        }
    }
    float A = M;
#pragma unroll
    for (int d = LP / 2; d; d >>= 1) A = fmaxf(A, __shfl_xor_sync(~0u, A, d));
    l = M == -INFINITY ? 0.f : l * fast_exp2(M - A);
#pragma unroll
    for (int d = LP / 2; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
    if (threadIdx.x % LP == 0 && r < rows)
        seg_ml[r] = make_float2(A == -INFINITY ? 0.f : A, l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l);
}

// Output of a segment from its n partials, a lane up to 4 four-value pieces of the
// rows with the loads of four partials in flight (a segment of one sequence can
// have a partial from every block of the grid).  With pieces enough each of the
// four warps has its own (2 sequences of 16,000, 8 heads of 128, 16 rows each:
// 36.6 -> 34.8 us);
// else every warp takes every fourth partial, and the four sums are added in order
// through shared memory (`area(w)`: 2 KB of warp w).  All threads of the block.
template <typename T, int D, class S, class A>
__device__ __forceinline__ void join_segment(const Args &p, T *dst, int rows, int n, S slot_of, A area, float2 *seg_ml)
{
    constexpr int U = 4;                               // partials in flight per warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (rows <= 4) join_statistics<32>(p, rows, n, slot_of, seg_ml);
    else if (rows <= 8) join_statistics<16>(p, rows, n, slot_of, seg_ml);
    else join_statistics<8>(p, rows, n, slot_of, seg_ml);
    __syncthreads();
    constexpr int Q = 4;
    const int items = rows * (D / 4);
    // enough pieces for every warp to have its own: no sums to exchange
    const bool apart = items >= kWarps * 32 * Q;
    const int first = apart ? 0 : warp, step = apart ? 1 : kWarps;      // this warp's partials
    for (int base = apart ? warp * 32 * Q : 0; base < items; base += (apart ? kWarps : 1) * 32 * Q) {
        float4 a[Q];
        float E[Q];
        const float *ml[Q], *po[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {                  // (past the last piece: the last again, not stored)
            int i = base + q * 32 + lane;
            i = i < items ? i : items - 1;
            a[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            E[q] = seg_ml[i / (D / 4)].x;
            ml[q] = p.part_ml + i / (D / 4) * 2;
            po[q] = p.part_o + (i / (D / 4)) * D + i % (D / 4) * 4;
        }
#pragma unroll 1
        for (int j = first; j < n; j += step * U) {
            float m[U][Q];
            float4 v[U][Q];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ju = j + u * step;
                const size_t slot = slot_of(ju < n ? ju : j);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    m[u][q] = __ldcg(ml[q] + slot * 2);
                    v[u][q] = __ldcg(reinterpret_cast<const float4 *>(po[q] + slot * D));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float f = j + u * step < n ? fast_exp2(m[u][q] - E[q]) : 0.f;
                    if (j + u * step < n)
                        a[q].x += v[u][q].x * f, a[q].y += v[u][q].y * f, a[q].z += v[u][q].z * f, a[q].w += v[u][q].w * f;
                }
            }
        }
        if (apart) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int i = base + q * 32 + lane;
                if (i < items) {
                    const int r = i / (D / 4);
                    const float inv = seg_ml[r].y;
                    *reinterpret_cast<uint2 *>(dst + r * D + i % (D / 4) * 4) =
                        make_uint2(pack2<T>(a[q].x * inv, a[q].y * inv), pack2<T>(a[q].z * inv, a[q].w * inv));
                }
            }
            continue;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (base + q * 32 + lane < items) area(warp)[q * 32 + lane] = a[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 32 * Q / kThreads; ++q) {
            const int k = q * kThreads + threadIdx.x, i = base + k;
            if (i < items) {
                float4 x = area(0)[k];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 v = area(w)[k];
                    x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
                }
                const int r = i / (D / 4), d = i % (D / 4) * 4;
                const float inv = seg_ml[r].y;
                *reinterpret_cast<uint2 *>(dst + r * D + d) =
                    make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
            }
        }
        __syncthreads();
    }
}

// (blocks of D = 64 and 128 fit twice into an SM)
// NH: groups of 8 heads per segment (1 or 2).
template <typename T, int D, int NH>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) paged_attn_kernel(const Args p)
{
    using L = Layout<D>;
    constexpr int kStages = L::kStages, kStrip = L::kStrip, kTile = L::kTile;
    constexpr int CH = D / 8;                                        // 16-byte chunks of a row
    constexpr int NS = kStrip / 16;                                  // 16-key steps of a strip
    constexpr float kUp = std::is_same<T, __half>::value ? 7.f : 0.f;
    extern __shared__ __align__(128) uint8_t smem[];
    float2 *comb_ml = reinterpret_cast<float2 *>(smem + L::kRing);   // [warp][row]
    volatile uint32_t *masks = reinterpret_cast<uint32_t *>(smem + L::kRing + L::kML);
    int *pre = reinterpret_cast<int *>(smem + L::kFixed);            // [B + 1]
    __shared__ int flag, blocks;
    __shared__ float2 seg_ml[kRows];                                 // a join's maxima and 1 / sums
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int segs = p.Hkv * p.HG;
    pdl_trigger();
    pdl_wait();

    // ---- the flat tile order: exclusive prefix of the sequences' tile counts
    for (int b = threadIdx.x; b < p.B; b += kThreads) pre[b] = (visible(p, b, blockIdx.x == 0) + kTile - 1) / kTile;
    __syncthreads();
    if (warp == 0) {
        int run = 0, n_max = 0, n_min = 0x7fffffff, held = 0;     // tiles per segment, sequences with any
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            const int n = b < p.B ? pre[b] : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            if (b < p.B) pre[b] = run + x - n;
            run += __shfl_sync(~0u, x, 31);
            if (n) {
                n_max = n > n_max ? n : n_max;
                n_min = n < n_min ? n : n_min;
                ++held;
            }
        }
        n_max = __reduce_max_sync(~0u, n_max);
        n_min = __reduce_min_sync(~0u, n_min);
        held = __reduce_add_sync(~0u, held);
        if (lane == 0) {
            pre[p.B] = run;
            // Blocks with work: not so many that a join's partials (~0.05 us each
            // and 128 pieces of output) outweigh the tiles a block is spared
            // (~0.9 us each), and for a segment of up to 3 tiles one (a join
            // takes ~3 us even of two).  Segments of equal length take whole
            // blocks each, so that none straddles two.
            const int64_t total = (int64_t)run * segs, seg = (int64_t)held * segs;
            const int rows = p.G < kRows ? p.G : kRows, pieces = (rows * (D / 4) + 127) / 128;
            int64_t P = total < gridDim.x ? total : gridDim.x;
            if (seg > 0) {
                const int64_t most = (int64_t)sqrtf(18.f * ((float)total / (float)seg) / (float)pieces) + 1;
                if (n_max == n_min && seg <= gridDim.x) {
                    int64_t k = gridDim.x / seg;
                    k = k < most ? k : most;
                    P = seg * (n_max <= 3 ? 1 : k < n_max ? k : n_max);
                } else if (P > seg * most) {
                    P = seg * most;
                }
            }
            blocks = (int)P;
        }
    }
    __syncthreads();
    const int64_t total = (int64_t)pre[p.B] * segs;
    // sequences with nothing to see: zeros
    T *out = static_cast<T *>(p.out);
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
        if (pre[b + 1] == pre[b])
            for (int i = threadIdx.x; i < p.Hq * D; i += kThreads) out[(size_t)b * p.Hq * D + i] = from_f32<T>(0.f);
    const int64_t P = blocks;
    if (blockIdx.x >= P) return;
    auto range = [&](int64_t c) { return c * total / P; };
    const int64_t lo = range(blockIdx.x), hi = range(blockIdx.x + 1);

    Pos cur;
    {
        int l = 0, r = p.B - 1;                                      // the sequence that holds flat tile lo
        while (l < r) {
            const int m = (l + r + 1) >> 1;
            if ((int64_t)pre[m] * segs <= lo) l = m; else r = m - 1;
        }
        cur.b = l;
        cur.n = pre[l + 1] - pre[l];
        const int64_t o = lo - (int64_t)pre[l] * segs;
        cur.g = (int)(o / cur.n);
        cur.t = (int)(o - (int64_t)cur.g * cur.n);
        cur.len = visible(p, l, false);
    }
    auto advance = [&](Pos &x) {
        if (++x.t < x.n) return;
        x.t = 0;
        if (++x.g < segs) return;
        x.g = 0;
        do {
            if (++x.b >= p.B) {
                x.n = 0;
                return;
            }
            x.n = pre[x.b + 1] - pre[x.b];
        } while (x.n == 0);
        x.len = visible(p, x.b, false);
    };

    // ---- this warp's ring
    const uint32_t ring = smem_u32(smem) + warp * kStages * 2 * L::kStripBytes;
    const T *kp = static_cast<const T *>(p.k_pages), *vp = static_cast<const T *>(p.v_pages);
    Pos iss = cur;
    int64_t issued = lo;
    // row offset (in rows of D) of the strip's key `lane`, -1 where there is none
    int64_t next_row = -1;
    auto look_up = [&]() {
        next_row = -1;
        if (issued < hi) {
            const int j = iss.t * kTile + warp * kStrip + lane;
            if (lane < kStrip && j < iss.len) {
                const int e = j / p.page_size;
                const int page = p.block_table[(int64_t)iss.b * p.max_pages + e];
                if (page >= 0 && page < p.num_pages)
                    next_row = ((int64_t)page * p.Hkv + iss.g / p.HG) * p.page_size + (j - e * p.page_size);
                else
                    raise_status(p.status, ORTHRUS_STATUS_PAGE);
            }
        }
    };
    look_up();
    auto issue = [&](int stage) {
        const uint32_t dk = ring + stage * 2 * L::kStripBytes, dv = dk + L::kStripBytes;
        const uint32_t m = __ballot_sync(~0u, next_row >= 0);
        if (lane == 0) masks[warp * kStages + stage] = m;
        if (m) {
#pragma unroll
            for (int i = 0; i < kStrip * CH / 32; ++i) {
                const int id = i * 32 + lane, r = id / CH, c = id % CH;
                const int64_t row = __shfl_sync(~0u, next_row, r);
                const uint32_t o = (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
                const int64_t src = (row < 0 ? 0 : row) * D + c * 8;
                cp_async16(dk + o, kp + src, row >= 0);
                cp_async16(dv + o, vp + src, row >= 0);
            }
        }
        if (issued < hi) {
            advance(iss);
            ++issued;
        }
        look_up();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        issue(s);
        cp_commit();
    }

    // ---- per-segment state.  This thread's heads in group h: 8 h + 2 (lane & 3)
    // + {0, 1}; its dims 16 d + lane / 4 + {0, 8}.
    uint32_t qf[D / 16][NH][2];
    float o[D / 16][NH][4], m[NH][2], l[NH][2];
    auto load_q = [&]() {
        const int g = cur.g / p.HG, h0 = (cur.g - g * p.HG) * kRows;
        const T *q = static_cast<const T *>(p.q) + ((size_t)cur.b * p.Hq + g * p.G) * D + (lane & 3) * 2;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const int r = h0 + h * 8 + (lane >> 2);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][h][0] = r < p.G ? *reinterpret_cast<const uint32_t *>(q + r * D + k * 16) : 0u;
                qf[k][h][1] = r < p.G ? *reinterpret_cast<const uint32_t *>(q + r * D + k * 16 + 8) : 0u;
            }
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[d][h][j] = 0.f;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h][0] = m[h][1] = -INFINITY;
            l[h][0] = l[h][1] = 0.f;
        }
    };
    load_q();
    clear();

    int stage = 0;
    for (int64_t x = lo; x < hi; ++x) {
        cp_wait<kStages - 2>();
        __syncwarp();              // (also: every lane is done with the stage that this iteration issues into)
        const uint32_t mask = masks[warp * kStages + stage];
        const uint32_t sk = ring + stage * 2 * L::kStripBytes, sv = sk + L::kStripBytes;
        if (mask) {
            // scores: rows are keys (lane / 4 and + 8 of each 16), columns heads.  Where
            // there is one accumulator per k, two take turns (the chain of dependent
            // instructions is half as long).
            constexpr int CN = NS * NH == 1 ? 2 : 1;
            float s[NS][NH][4], s2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[j] = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][h][j] = 0.f;
            {
                // matrices: dims lo | keys 0-7, 8-15, then dims hi | keys 0-7, 8-15
                const int r = lane & 15, cc = lane >> 4;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        uint32_t a[4];
                        ldsm4(a, sk + (i * 16 + r) * D * 2 + (((2 * k + cc) ^ (r & 7)) << 4));
#pragma unroll
                        for (int h = 0; h < NH; ++h) mma<T>(CN == 2 && (k & 1) ? s2 : s[i][h], a, qf[k][h][0], qf[k][h][1]);
                    }
                }
            }
            if (CN == 2) {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[0][0][j] += s2[j];
            }
            if (mask != (kStrip == 32 ? ~0u : 0xffffu)) {
                const uint32_t mk = mask >> (lane >> 2);
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (!((mk >> (16 * i + 8 * (j >> 1))) & 1u)) s[i][h][j] = -INFINITY;
            }
            float a[NH][2];
            bool grow = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NS; ++i) v = fmax3(v, s[i][h][e], s[i][h][2 + e]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
                    a[h][e] = v * p.scale_log2;
                    grow |= a[h][e] > m[h][e] + kLazy;
                }
            }
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float n = fmaxf(m[h][e], a[h][e]);
                        const float f = m[h][e] == -INFINITY ? 0.f : fast_exp2(m[h][e] - n);
                        m[h][e] = n;
                        l[h][e] *= f;
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            o[d][h][e] *= f;
                            o[d][h][2 + e] *= f;
                        }
                    }
                }
            }
            constexpr int TERMS = Split<T>::terms;
            uint32_t pw[TERMS][NS][NH][2];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                // a head whose scores so far are all -inf keeps the weights at zero
                const float e0 = m[h][0] == -INFINITY ? 0.f : m[h][0] - kUp, e1 = m[h][1] == -INFINITY ? 0.f : m[h][1] - kUp;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {                     // keys lane / 4, + 8
                        const float x0 = fast_exp2(fmaf(s[i][h][2 * k], p.scale_log2, -e0));
                        const float x1 = fast_exp2(fmaf(s[i][h][2 * k + 1], p.scale_log2, -e1));
                        l[h][0] += x0;
                        l[h][1] += x1;
                        uint32_t w[TERMS];
                        Split<T>::of(x0, x1, w);
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) pw[t][i][h][k] = transpose8(w[t]);
                    }
                }
            }
            // the values' transpose: matrices keys 0-7 | dims lo, hi, then keys 8-15 | dims lo, hi
            const int r = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    uint32_t v[4];
                    ldsm4_t(v, sv + (i * 16 + r) * D * 2 + (((2 * d + cc) ^ (r & 7)) << 4));
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) mma<T>(o[d][h], v, pw[t][i][h][0], pw[t][i][h][1]);
                }
            }
        }
        issue((stage + kStages - 1) % kStages);
        cp_commit();

        if (cur.t + 1 == cur.n || x + 1 == hi) {   // the block leaves this segment
            const Pos seg_ = cur;
            if (x + 1 < hi) {
                advance(cur);
                load_q();                          // (on its way during the rest)
            }
            const int rowsG = p.G - (seg_.g % p.HG) * kRows, rows = rowsG < kRows ? rowsG : kRows;
            // the stage just read holds O now (its next load is issued an iteration
            // later); 8-value chunk i of row r sits at i ^ (r & 7)
            auto comb_o = [&](int w) {
                return reinterpret_cast<float *>(smem + ((w * kStages + stage) * 2) * L::kStripBytes);
            };
#pragma unroll
            for (int h = 0; h < NH; ++h) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[h][e] += __shfl_xor_sync(~0u, l[h][e], d);
                    const int r = 8 * h + 2 * (lane & 3) + e;
                    if (lane < 4) comb_ml[warp * kRows + r] = make_float2(m[h][e], l[h][e]);
                    if (r < rows) {
                        float *c = comb_o(warp) + r * D + (lane >> 2);
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            c[((2 * d) ^ (r & 7)) * 8] = o[d][h][e];
                            c[((2 * d + 1) ^ (r & 7)) * 8] = o[d][h][2 + e];
                        }
                    }
                }
            }
            __syncthreads();
            const int64_t s0 = (int64_t)pre[seg_.b] * segs + (int64_t)seg_.g * seg_.n;      // the segment's flat tiles
            const bool whole = lo <= s0 && hi >= s0 + seg_.n;
            const int g = seg_.g / p.HG, h0 = (seg_.g - g * p.HG) * kRows;
            T *dst = out + ((size_t)seg_.b * p.Hq + g * p.G + h0) * D;
            const size_t slot = 2 * (size_t)blockIdx.x + (lo < s0 ? 1 : 0);
            for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
                const int r = i / (D / 4), d = (i % (D / 4)) * 4;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, comb_ml[w * kRows + r].x);
                const float E = M == -INFINITY ? 0.f : M;
                float l = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 ml = comb_ml[w * kRows + r];
                    const float f = fast_exp2(ml.x - E);
                    const float4 v = *reinterpret_cast<const float4 *>(comb_o(w) + r * D + ((d >> 3) ^ (r & 7)) * 8 + (d & 7));
                    l += ml.y * f;
                    a.x += v.x * f, a.y += v.y * f, a.z += v.z * f, a.w += v.w * f;
                }
                if (whole) {
                    const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;           // (NaN stays NaN)
                    *reinterpret_cast<uint2 *>(dst + r * D + d) =
                        make_uint2(pack2<T>(a.x * inv, a.y * inv), pack2<T>(a.z * inv, a.w * inv));
                } else {
                    *reinterpret_cast<float4 *>(p.part_o + (slot * kRows + r) * D + d) = a;
                    if (d == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * kRows + r) * 2) = make_float2(M, l);
                }
            }
            if (!whole) {
                // blocks [c0, c1] hold the segment; the last to arrive joins it
                const int c_first = (int)(((s0 + 1) * P - 1) / total), c_last = (int)(((s0 + seg_.n) * P - 1) / total);
                const int n = c_last - c_first + 1;
                __syncthreads();                   // every partial store of the block, before the release
                if (threadIdx.x == 0) {
                    const int old = counter_fetch_add_acq_rel(p.counters + c_first, 1);
                    flag = old == n - 1;
                    if (flag) p.counters[c_first] = 0;
                }
                __syncthreads();
                if (flag) {
                    // (the first block may have come to the segment from another one;
                    // every other block's range begins inside it)
                    const size_t slot0 = 2 * (size_t)c_first + (range(c_first) < s0 ? 1 : 0);
                    auto slot_of = [&](int j) { return (j ? 2 * (size_t)(c_first + j) : slot0) * kRows; };
                    join_segment<T, D>(p, dst, rows, n, slot_of,
                                       [&](int w) { return reinterpret_cast<float4 *>(comb_o(w)); }, seg_ml);
                }
            }
            __syncthreads();                       // the combine buffer and the flag are free again
            clear();
        } else {
            ++cur.t;
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_wait<0>();
}

// The launch's block count.
inline int grid_of(int D, int sms) { return D == 256 ? sms : 2 * sms; }

struct Plan {
    int grid;
    size_t ml, o, total;                         // partials' places; the counters come first
};

// The counters sit at the same place for every shape; the partials, which may lie
// anywhere behind them, leave a word per segment free at the head as well.
inline Plan plan(int B, int Hq, int Hkv, int D, int sms)
{
    Plan w;
    const int G = Hq / Hkv, HG = (G + kRows - 1) / kRows;
    w.grid = grid_of(D, sms);
    const size_t words = (size_t)B * Hkv * HG, counters = 2 * (size_t)sms;
    w.ml = ((words > counters ? words : counters) * sizeof(int32_t) + 255) & ~(size_t)255;
    w.o = w.ml + (((size_t)2 * w.grid * kRows * 2 * sizeof(float) + 255) & ~(size_t)255);
    w.total = w.o + (size_t)2 * w.grid * kRows * D * sizeof(float);
    return w;
}

constexpr int kMaxDevices = 64;

template <typename T, int D, int NH> bool smem_ready()
{
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(paged_attn_kernel<T, D, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Layout<D>::kFixed + (kMaxB + 1) * (int)sizeof(int)) == cudaSuccess;
        if (!ok[dev]) cudaGetLastError();
    });
    return ok[dev];
}

template <typename T, int D, int NH> cudaError_t launch_h(const Args &a, int grid, cudaStream_t st)
{
    if (!smem_ready<T, D, NH>()) return cudaErrorInvalidValue;
    const size_t smem = Layout<D>::kFixed + ((size_t)a.B + 1) * sizeof(int);
    return launch_pdl(paged_attn_kernel<T, D, NH>, dim3(grid), kThreads, smem, st, a);
}

template <typename T, int D> cudaError_t launch(const Args &a, int grid, cudaStream_t st)
{
    return a.G <= 8 ? launch_h<T, D, 1>(a, grid, st) : launch_h<T, D, 2>(a, grid, st);
}

template <typename T> cudaError_t launch_d(const Args &a, int D, int grid, cudaStream_t st)
{
    return D == 64 ? launch<T, 64>(a, grid, st) : D == 128 ? launch<T, 128>(a, grid, st) : launch<T, 256>(a, grid, st);
}

int current_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

bool shape_ok(int B, int Hq, int Hkv, int D) { return B > 0 && Hq > 0 && Hkv > 0 && D > 0 && Hq % Hkv == 0; }
bool shape_supported(int B, int Hq, int D)
{
    return B <= kMaxB && (D == 64 || D == 128 || D == 256) && Hq <= 65536;
}

}  // namespace paged

}  // namespace orthrus

using namespace orthrus;

extern "C" size_t orthrus_paged_attn_workspace_size(int B, int Hq, int Hkv, int D)
{
    if (!paged::shape_ok(B, Hq, Hkv, D) || !paged::shape_supported(B, Hq, D)) return 0;
    const int sms = paged::current_sms();
    return sms > 0 ? paged::plan(B, Hq, Hkv, D, sms).total : 0;
}

extern "C" int orthrus_paged_attn(orthrus_dtype dtype, const void *q, const void *k_pages, const void *v_pages,
                                  const int32_t *block_table, const int32_t *ctx_lens, int n_new, int B, int Hq, int Hkv,
                                  int D, int num_pages, int page_size, int max_pages, float scale, void *out,
                                  void *workspace, size_t workspace_bytes, int32_t *status, void *stream)
{
    if (!q || !k_pages || !v_pages || !block_table || !ctx_lens || !out) return ORTHRUS_ERR_ARG;
    if (!paged::shape_ok(B, Hq, Hkv, D) || n_new < 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0)
        return ORTHRUS_ERR_ARG;
    if (!(scale == scale) || isinf(scale)) return ORTHRUS_ERR_ARG;
    if (dtype != ORTHRUS_BF16 && dtype != ORTHRUS_F16) return dtype == ORTHRUS_F32 ? ORTHRUS_ERR_UNSUPPORTED : ORTHRUS_ERR_ARG;
    if (!paged::shape_supported(B, Hq, D)) return ORTHRUS_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page_size > (1ll << 31) - 128 ||
        ((int64_t)max_pages * page_size / 64 + 1) * B >= (1ll << 31))
        return ORTHRUS_ERR_UNSUPPORTED;          // (positions and the tile prefix are 32-bit)
    if (((uintptr_t)q | (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)out | (uintptr_t)workspace) & 15u)
        return ORTHRUS_ERR_ALIGN;
    const int sms = paged::current_sms();
    if (sms <= 0) return ORTHRUS_ERR_DEVICE;
    const paged::Plan w = paged::plan(B, Hq, Hkv, D, sms);
    if (!workspace || workspace_bytes < w.total) return ORTHRUS_ERR_WORKSPACE;
    paged::Args a;
    a.q = q;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.block_table = block_table;
    a.ctx_lens = ctx_lens;
    a.out = out;
    char *ws = static_cast<char *>(workspace);
    a.counters = reinterpret_cast<int32_t *>(ws);
    a.part_ml = reinterpret_cast<float *>(ws + w.ml);
    a.part_o = reinterpret_cast<float *>(ws + w.o);
    a.status = status;
    a.n_new = n_new;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.HG = (a.G + paged::kRows - 1) / paged::kRows;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == ORTHRUS_BF16 ? paged::launch_d<__nv_bfloat16>(a, D, w.grid, st)
                                                : paged::launch_d<__half>(a, D, w.grid, st);
    return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_LAUNCH;
}
