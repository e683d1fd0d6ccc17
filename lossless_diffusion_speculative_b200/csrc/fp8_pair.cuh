// The form of orthrus_fp8_matmul for many token rows: pairs of CTAs on tiles of
// 256 token rows x 256 weight rows (tcgen05 cta_group::2).  Bound by the tensor
// cores; what the layout has to keep out of their way:
//   - operands.  In a pair each CTA holds half of both operands (32 KB per
//     k-block instead of the 48 KB of a single CTA on 128 x 256).
//   - the scales.  Each k-block's sums are read from TMEM and added, scaled, to
//     fp32 registers: eight warps, a token row per lane, 128 columns each (half
//     of the register file holds the CTA's 128 x 256 sums).  A buffer's round
//     trip (multiply, signal, read and add, signal back) takes ~1500 cycles
//     against the 512 of a block's multiplication, so the two column halves
//     have two TMEM buffers each and are multiplied, signalled and freed
//     separately (706k cycles a call at 8192 x 12288 x 4096 with both halves
//     together, 610k apart; the multiplications alone are 340k).  The issuing
//     thread shares its scheduler with two epilogue warps, so what it and they
//     issue counts: the sums use two-element FMAs but for one pair in eight
//     (595k; for none: 610k, for half: 685k, for all: 746k), chunks of 16 columns (8: 688k, 32:
//     715k), no votes between signals, one issuing thread (one per half: 770k).
//   - the row scales lie [row][k-block] in memory, a line per row: a warp of
//     its own copies 16 k-blocks of all rows at a time, coalesced along k.
//     (Loaded by the epilogue's lanes, a row each, the same copies took the L1
//     ~1300 cycles per four blocks.)
//   - the output.  The pair walks its tiles; a finished tile leaves through
//     shared memory by TMA stores while the next tile is being multiplied.
// Measured at 8192 x 12288 x 4096: 352 us a call (2.34 PFLOP/s), 410-430 repeated
// for seconds (the power limit), against 325 of a library product with one scale
// per tensor there.
#pragma once

namespace orthrus {
namespace f8 {

constexpr int kEpiWarps = 8;
constexpr int kPairThreads = (kEpiWarps + 3) * 32;    // and a producer, an MMA and a scale warp
constexpr int kPairN = 256;
constexpr int kScaleGroup = 16;                       // k-blocks whose scales are fetched at once
constexpr int kScalePitch = 129;                      // row scales [k-block][row], padded for the copies' banks

struct PairMaps {
    CUtensorMap x, y, o;                 // a: box 128 x 128; w: box 128 x 64; out: box 128 bytes x 128 rows
};

struct PairConf {
    static constexpr int stage = 2 * kXBytes;                         // 128 token rows, 2 x 64 weight rows
    static constexpr int nst = 4;
    static constexpr int out_half = 32 * 1024;                        // staging of one column half: two boxes
    static constexpr int out = nst * stage;
    static constexpr int bars = out + 2 * out_half;
    // stage full / empty, TMEM buffer [half][2] full / empty, scale group full / empty, drain
    static constexpr int nbars = 2 * nst + 8 + 4 + 1;
    static constexpr int sa = (bars + nbars * 8 + 16 + 15) & ~15;     // [2][16][129] row scales
    static constexpr int sw = sa + 2 * kScaleGroup * kScalePitch * 4; // [2][2 halves][16] weight scales
    static constexpr int total = sw + 2 * 2 * kScaleGroup * 4 + 1024;
    static_assert(total > 114 * 1024, "one block per SM: TMEM is never waited for");
    static_assert(total <= 227 * 1024 && nst == 4, "shared memory; the MMA loop's parities");
};

// Token tiles first, in strips of 32, so that the pairs at work share few weight
// tiles and all token rows come from L2 (strips of 8: 431 us sustained, 32: 420).
__device__ __forceinline__ void pair_tile(const Args &p, int t, int &x, int &y)
{
    constexpr int G = 32;
    const int strip = t / (G * p.tiles_y), r = t - strip * G * p.tiles_y;
    const int h = p.tiles_x - strip * G < G ? p.tiles_x - strip * G : G;
    y = r / h;
    x = strip * G + (r - y * h);
}

// The four warps of one column half meet.
__device__ __forceinline__ void half_sync(int half)
{
    if (half) asm volatile("bar.sync 2, 128;" ::: "memory");
    else asm volatile("bar.sync 1, 128;" ::: "memory");
}

// They meet and agree: whether all of them are ok.
__device__ __forceinline__ bool half_agree(int half, bool ok)
{
    uint32_t r;
    if (half)
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                     "barrier.cta.red.and.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(r)
                     : "r"((uint32_t)ok)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                     "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(r)
                     : "r"((uint32_t)ok)
                     : "memory");
    return r != 0;
}

// Staged rows of up to 128 16-bit values (two boxes, chunks swizzled by the row)
// to rows of global memory at any element's alignment: whole 16-byte chunks of each
// destination row, put together from the words around them, then the few
// elements before and after (565 x 116147 x 416: 262 us element by element, 123 so).
// The 128 threads of a column half.
__device__ __noinline__ void copy_rows(const uint8_t *src, uint8_t *dst, size_t pitch, int rows, int len)
{
    const int tid = threadIdx.x & 127;
    auto at = [&](int r, int b) { return src + (b >> 7) * 16384 + r * 128 + ((((b >> 4) & 7) ^ (r & 7)) << 4) + (b & 15); };
#pragma unroll 4
    for (int i = tid; i < rows * 16; i += 128) {
        const int r = i >> 4, k = i & 15;
        uint8_t *d = dst + r * pitch;
        const int lead = (int)(-reinterpret_cast<uintptr_t>(d) & 15), b = lead + 16 * k;
        if (b + 16 > len) continue;
        uint32_t w[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            const int q = (b & ~3) + 4 * j;
            w[j] = *reinterpret_cast<const uint32_t *>(at(r, q < 252 ? q : 252));
        }
        const uint32_t sel = b & 2 ? 0x5432u : 0x3210u;
        *reinterpret_cast<uint4 *>(d + b) = make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[1], w[2], sel),
                                                       __byte_perm(w[2], w[3], sel), __byte_perm(w[3], w[4], sel));
    }
    if (tid < rows) {
        uint8_t *d = dst + tid * pitch;
        int lead = (int)(-reinterpret_cast<uintptr_t>(d) & 15);
        lead = lead < len ? lead : len;
        const int tail = lead + ((len - lead) & ~15);
#pragma unroll 2
        for (int b = 0; b < len; b += 2) {
            if (b == lead) b = tail;
            if (b >= len) break;
            *reinterpret_cast<uint16_t *>(d + b) = *reinterpret_cast<const uint16_t *>(at(tid, b));
        }
    }
}

// TMA: rows of out are aligned for TMA stores.  (A form of its own: the other
// path's registers made the sums' loop spill, 676k cycles instead of 610k.)
template <typename T, bool TMA>
__global__ void __launch_bounds__(kPairThreads, 1) fp8_pair_kernel(const __grid_constant__ PairMaps mp, const Args p)
{
    using C = PairConf;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw);
    const uint32_t b_full = base + C::bars, b_empty = b_full + 8 * C::nst, b_tfull = b_empty + 8 * C::nst,
                   b_tempty = b_tfull + 32, b_sfull = b_tempty + 32, b_sempty = b_sfull + 16, b_drain = b_sempty + 16;
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::bars + C::nbars * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::nst; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(b_tfull + 8 * i, 1);
            mbar_init(b_tempty + 8 * i, kEpiWarps);                   // four warps of both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_sfull + 8 * i, 1);
            mbar_init(b_sempty + 8 * i, kEpiWarps);
        }
        mbar_init(b_drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kEpiWarps && lane == 0) {
        tma_prefetch(&mp.x);
        tma_prefetch(&mp.y);
        if (TMA) tma_prefetch(&mp.o);
    }
    if (warp == kEpiWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + C::bars +
                                                                                                C::nbars * 8)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const int tiles = p.tiles_x * p.tiles_y;
    pdl_wait();

    if (warp < kEpiWarps) {
        constexpr int CPT = kPairN / 2;
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 2 * CPT;
        const uint32_t tfull = b_tfull + 16 * half, lead_tempty = map_to_rank(b_tempty + 16 * half, 0);
        const float *sa = reinterpret_cast<const float *>(sm + C::sa) + row;
        const float *sw = reinterpret_cast<const float *>(sm + C::sw) + half * kScaleGroup;
        // staging of this half: boxes of 128 rows x 128 bytes, 16-byte chunks swizzled by the row
        const uint32_t stage_out = base + C::out + half * C::out_half;
        const uint32_t my_row = stage_out + row * 128;
        constexpr int BOX = 128 / (int)sizeof(T);                    // columns of a box
        constexpr int PASS = CPT < 2 * BOX ? CPT : 2 * BOX;           // columns of a pass
        int it = 0, g = 0;                           // k-blocks and scale groups so far
        bool ok = true;
        for (int t = pair; t < tiles; t += pairs) {
            float2 acc[CPT / 2];
#pragma unroll
            for (int i = 0; i < CPT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int kb = 0; kb < p.nkb; ++kb, ++it) {
                const int in = kb % kScaleGroup;
                if (in == 0) {
                    ok &= wait_bar_near(b_sfull + 8 * (g & 1), (g >> 1) & 1, abort_flag, p.status);
                    __syncwarp();
                    ++g;
                }
                const int gb = (g - 1) & 1, buf = it & 1;
                const float sc = sa[(gb * kScaleGroup + in) * kScalePitch] * sw[gb * 2 * kScaleGroup + in];
                const float2 s2 = make_float2(sc, sc);
                // (no vote here: after an abort the warp goes on with what it reads
                // and leaves at the tile's end)
                ok &= wait_bar_near(tfull + 8 * buf, (it >> 1) & 1, abort_flag, p.status);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < CPT; c += 16) {
                    uint32_t w[16];
                    tmem_ld16(t_row + buf * CPT + c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        // seven pairs in eight by two-element FMAs (half of the FMA pipe,
                        // half the issue slots), one by the pipe's other half
                        float2 &x = acc[c / 2 + q];
                        const float y0 = __uint_as_float(w[2 * q]), y1 = __uint_as_float(w[2 * q + 1]);
                        if (q == 7) x = make_float2(fmaf(y0, sc, x.x), fmaf(y1, sc, x.y));
                        else x = ffma2(make_float2(y0, y1), s2, x);
                    }
                }
                // (signalled after the last sums, not after the last load: the MMA
                // warp's steps are slow while this partition still adds)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster(lead_tempty + 8 * buf);
                    if (in == kScaleGroup - 1 || kb + 1 == p.nkb) mbar_arrive(b_sempty + 8 * gb);
                }
            }
            ok = half_agree(half, ok);               // (after an abort all four warps leave together)
            if (!ok) break;
            // ---- out: through the staging buffer, PASS columns at a time
            int x, y;
            pair_tile(p, t, x, y);
            const int m0 = x * 256 + rank * 128, n0 = y * kPairN + half * CPT;
#pragma unroll
            for (int c0 = 0; c0 < CPT; c0 += PASS) {
                if ((threadIdx.x & 127) == 0) bulk_wait_read();       // the last stores have left the buffer
                half_sync(half);
#pragma unroll
                for (int b = 0; b < PASS / BOX; ++b) {
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {                  // 16-byte chunks of the box's row
                        const float2 *f = acc + (c0 + b * BOX) / 2 + ch * (BOX / 16);
                        uint4 w;
                        if constexpr (sizeof(T) == 2)
                            w = make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y),
                                           pack2<T>(f[3].x, f[3].y));
                        else
                            w = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                                           __float_as_uint(f[1].y));
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(my_row + b * 16384 +
                                                                                      ((ch ^ (row & 7)) << 4)),
                                     "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                                     : "memory");
                    }
                }
                fence_proxy_async();
                half_sync(half);
                if constexpr (TMA) {
                    if ((threadIdx.x & 127) == 0) {
#pragma unroll
                        for (int b = 0; b < PASS / BOX; ++b)
                            if (n0 + c0 + b * BOX < p.N && m0 < p.M)
                                tma_store_2d(&mp.o, stage_out + b * 16384, (n0 + c0 + b * BOX) * (int)sizeof(T), m0);
                        bulk_commit();
                    }
                } else {                                              // rows of out not 16-byte aligned
                    const uint8_t *src = sm + C::out + half * C::out_half;
                    if constexpr (sizeof(T) == 2) {
                        const int cols = p.N - n0 - c0 < PASS ? p.N - n0 - c0 : PASS, rows = p.M - m0 < 128 ? p.M - m0 : 128;
                        if (cols > 0)
                            copy_rows(src, reinterpret_cast<uint8_t *>(static_cast<T *>(p.out) + (size_t)m0 * p.N + n0 + c0),
                                      (size_t)p.N * 2, rows, cols * 2);
                    } else {
                        // (by pairs or elements: the second pass' sums are still in
                        // registers here, where the copy of whole chunks made them spill)
                        const int V = p.vec;
#pragma unroll 4
                        for (int i = threadIdx.x & 127; i < 128 * PASS / V; i += 128) {
                            const int r = i * V / PASS, c = i * V % PASS, e = c % BOX * 4;
                            const uint8_t *at = src + (c / BOX) * 16384 + r * 128 + ((e >> 4 ^ (r & 7)) << 4) + (e & 15);
                            if (m0 + r < p.M && n0 + c0 + c < p.N) {
                                T *dst = static_cast<T *>(p.out) + (size_t)(m0 + r) * p.N + n0 + c0 + c;
                                if (V == 2) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(at);
                                else *dst = *reinterpret_cast<const T *>(at);
                            }
                        }
                    }
                    half_sync(half);
                }
            }
        }
        if ((threadIdx.x & 127) == 0) bulk_wait_all();
    } else if (warp == kEpiWarps) {
        // ---- producer: this CTA's token rows, and its 64 weight rows of either column half
        if (elect_one()) {
            const uint64_t keep = make_policy_evict_last();
            int it = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int x, y;
                pair_tile(p, t, x, y);
                const int m0 = x * 256 + rank * 128, n0 = y * kPairN + rank * 64;
#pragma unroll 1
                for (int kb = 0; kb < p.nkb; ++kb, ++it) {
                    const int st = it % C::nst, n = it / C::nst;
                    if (n > 0) ok = wait_bar_near(b_empty + 8 * st, (n - 1) & 1, abort_flag, p.status);
                    if (!ok) break;
                    const uint32_t full = map_to_rank(b_full + 8 * st, 0), dst = base + st * C::stage;
                    if (rank == 0) mbar_expect_tx(b_full + 8 * st, 2 * C::stage);
                    tma_load_2d_pair(dst, &mp.x, full, kb * 128, m0, keep);
                    tma_load_2d_pair(dst + kXBytes, &mp.y, full, kb * 128, n0, keep);
                    tma_load_2d_pair(dst + kXBytes + 8192, &mp.y, full, kb * 128, n0 + 128, keep);
                }
            }
            if (!ok && rank == 0) {                                   // abort: let both CTAs' copies in flight land
                for (int st = 0; st < C::nst; ++st) {
                    const int fills = it / C::nst + (st < it % C::nst ? 1 : 0);
                    if (fills) wait_bar_quiet(b_full + 8 * st, (fills - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == kEpiWarps + 1) {
        // ---- MMA: the even CTA issues for both
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = instr_desc_e4m3(256, kPairN / 2);
            const int steps = (tiles - pair + pairs - 1) / pairs * p.nkb;
            const uint64_t ax0 = smem_desc(base, 16, 1024), ay0 = smem_desc(base + kXBytes, 16, 1024);
            bool ok = true;
            uint32_t par = 0;                                         // parity of the stage ring's round
#pragma unroll 1
            for (int it = 0; ok && it < steps; it += C::nst, par ^= 1) {
#pragma unroll
                for (int st = 0; st < C::nst; ++st) {                 // (nst is even: buffer st & 1, used twice a round)
                    if (it + st >= steps) break;
                    ok = wait_bar_near(b_full + 8 * st, par, abort_flag, p.status);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && (it + st < 2 || wait_bar_near(b_tempty + 16 * h + 8 * (st & 1), ((st >> 1) & 1) ^ 1,
                                                                 abort_flag, p.status));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tc_mma_f8_pair(tmem + (h * 2 + (st & 1)) * (kPairN / 2), ax0 + st * (C::stage >> 4) + 2 * q,
                                           ay0 + st * (C::stage >> 4) + h * (8192 >> 4) + 2 * q, idesc, q);
                        tc_commit_pair(b_tfull + 16 * h + 8 * (st & 1));
                    }
                    if (!ok) break;
                    tc_commit_pair(b_empty + 8 * st);
                }
            }
            if (!ok) {
                tc_commit_pair_own(b_drain);
                wait_bar_quiet(b_drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ---- scales: 16 k-blocks of the CTA's 128 rows and of the two column halves
        int g = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int x, y;
            pair_tile(p, t, x, y);
            const int m0 = x * 256 + rank * 128, nb = y * 2 + (lane >> 4), blocks = (p.N + 127) / 128;
            const int k16 = lane & 15;
#pragma unroll 1
            for (int kb = 0; kb < p.nkb; kb += kScaleGroup, ++g) {
                const int b = g & 1, n = g >> 1, k = kb + k16;
                if (n > 0) ok = __all_sync(~0u, wait_bar_near(b_sempty + 8 * b, (n - 1) & 1, abort_flag, p.status));
                if (!ok) break;
                const uint32_t dst = base + C::sa + ((b * kScaleGroup + k16) * kScalePitch + (lane >> 4)) * 4;
                const float *src = p.a_scale + (size_t)m0 * p.nkb + k;
#pragma unroll 8
                for (int r = 0; r < 128; r += 2) {                    // two rows, 16 k-blocks each
                    const int m = r + (lane >> 4);
                    const bool in = k < p.nkb && m0 + m < p.M;
                    cp_async4(dst + r * 4, in ? src + (size_t)m * p.nkb : p.a_scale, in);
                }
                const bool in = k < p.nkb && nb < blocks;
                cp_async4(base + C::sw + (b * 2 * kScaleGroup + lane) * 4,
                          in ? p.w_scale + (size_t)nb * p.nkb + k : p.w_scale, in);
                cp_commit();
                cp_wait<0>();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_sfull + 8 * b);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                                   // neither CTA leaves while the other may signal it
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace f8
}  // namespace orthrus
