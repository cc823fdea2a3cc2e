// attn_kernel_decode_q4.cuh -- sm_103a attention of a few query rows over a
// key/value cache held in 4 bits (format: attn_cache_q4.cuh).
//
//     O = softmax(scale Q K^T + bias + M) V,   K, V = s (u - u0) per group of 64 channels
//
// The work is reading the cache once (17/32 of a byte a value), so the kernel streams
// blocks of 64 slots and keeps everything else in registers. At the copy rate an SM
// has about 400 cycles per block of 64 x (128 + 128) values, fewer than the CUDA
// cores would need for an FMA per value and row, so the products run on the tensor
// cores with the codes as the A operand (mma.sync m16n8k16, 16 slots or 16 value
// channels by 8 query rows; a tcgen05 tile of 128 rows would be mostly padding, and
// its operand would have to pass through shared memory as bf16, four times the bytes).
//
// Unpacking. The low nibble of each 16-bit half, masked, is an fp16 subnormal
// u 2^-24; the next nibble, masked in place, is u 2^-20. So a word of eight codes
// becomes four operand registers with four ANDs and one shift, exactly and without an
// offset to take out again. The fp16 partner carries the scales: the query row times a
// power of two that brings its largest magnitude to [2^14, 2^15) (and 2^-4 for the
// odd nibbles), for V the weights p s R, R a power of two per group and warp that
// keeps the largest s R in [2^12, 2^15).
//
//   scores   S^T[slot][row] = s (sum_c u_c q_c - u0 sum_c q_c), summed over the groups
//   output   O^T[c][row]    = sum_j (p_j s_j R) u_jc - sum_j (p_j s_j R) u0_j, over R l
//
// The scores' accumulator has a slot in its row and two query rows in its columns; the
// weights go to the second product's B operand through movmatrix (an 8 x 8 transpose
// in registers). Row r of a 16-slot tile is slot 4 (r % 2) + (r % 8) / 2 + 8 (r / 8), so that
// a thread's four V slots are t, t + 4, t + 8, t + 12 and a warp reads 16 contiguous rows.
//
// A warp streams its own blocks through its own ring (lane 0 issues a bulk copy per
// block as soon as the warp has consumed the stage) with an online softmax of its own;
// the CTA's warps share one (b, cache head, row tile) at a time, block by block, and
// merge at its end. With `split` the blocks of all pairs, as the entries' lengths have
// them on the device, are dealt out evenly: CTA c takes units [T c / G, T (c + 1) / G). A
// pair that lies in one CTA is written there; of one that is cut, each CTA writes its
// part (max, sum, unnormalised O) to its slot 0 (the pair began in an earlier CTA) or
// slot 1, and a second kernel merges the parts in order.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_cache_q4.cuh"
#include "attn_internal.h"
#include "sm103a.cuh"

namespace attn {

using namespace sm103a;

namespace dq4 {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr float LN2 = 0.693147180559945309f;
constexpr float LOG2E = 1.44269504088896341f;
constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
constexpr float TWO20 = 1048576.f, TWO24 = 16777216.f;

template <int DK, int DV, int NT>
struct Layout {
    static constexpr int ROWS = 8 * NT;
    static constexpr int BYTES_BLOCK = q4::block_bytes(DK, DV);
    // 2 blocks of 8704 or 6528 bytes, or 3 of 4352, in flight per warp
    static constexpr int STAGES = DK + DV == 128 ? 3 : 2;
    static constexpr int RING = WARPS * STAGES * BYTES_BLOCK;
    // the merge of the warps reuses the ring: per warp max and sum [ROWS], O [ROWS][DV]
    static constexpr int RED_WARP = ROWS * (DV + 2);
    static_assert(WARPS * RED_WARP * 4 <= RING, "merge area inside the ring");
    static constexpr int BAR_OFF = RING;
    static constexpr int MISC_OFF = BAR_OFF + (WARPS * STAGES + 1) * 8;
    static constexpr int BYTES = MISC_OFF + 16 + 128;
    static_assert(BYTES * decode_q4_ctas_per_sm(DK, DV, ROWS) <= 232448 - 3 * 1024, "shared memory budget");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Exponent of a finite positive x (subnormals: -127).
__device__ __forceinline__ int exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }

// Step and zero of a group word in the lower half of w.
__device__ __forceinline__ float word_step(uint32_t w) { return __uint_as_float((w << 16) & 0xFFF00000u); }
__device__ __forceinline__ float word_zero(uint32_t w)
{
    return __uint_as_float(((w << 19) & 0x00780000u) | 0x41800000u) - 16.f;   // (16 + u0) - 16
}

// The slots of entry b that some row sees end here; kv_len: its filled slots.
__device__ __forceinline__ int visible_end(const DecodeQ4Params& p, int b, int* kv_len)
{
    int len = p.m;
    if (mask_has_lengths(p.mask)) {
        const int l = __ldg(p.key_lengths + b);
        len = l < 0 ? 0 : (l > p.m ? p.m : l);
    }
    *kv_len = len;
    if (!mask_is_causal(p.mask)) return len;
    const int off = causal_offset(p.mask, p.m - p.n, len, p.n);
    return min(len, max(0, p.n + off));          // row n - 1 sees slots up to n - 1 + off
}

// Blocks of each pair of entry b; a pair without a visible slot keeps one, so that its rows are written.
__device__ __forceinline__ int pair_blocks(const DecodeQ4Params& p, int b)
{
    int kv;
    return max(1, (visible_end(p, b, &kv) + q4::BLOCK - 1) / q4::BLOCK);
}

template <int DK, int DV, int NT>
__global__ void __launch_bounds__(THREADS, decode_q4_ctas_per_sm(DK, DV, 8 * NT))
attn_decode_q4_kernel(const DecodeQ4Params p)
{
    using L = Layout<DK, DV, NT>;
    constexpr int NGK = DK / q4::GROUP, NGV = DV / q4::GROUP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t bar0 = sbase + L::BAR_OFF + 8u * static_cast<uint32_t>(warp * L::STAGES);   // this warp's ring
    const uint32_t bar_never = sbase + L::BAR_OFF + 8u * static_cast<uint32_t>(WARPS * L::STAGES);
    volatile uint32_t* abort_word = reinterpret_cast<volatile uint32_t*>(smem + L::MISC_OFF);
    if (threadIdx.x == 0) {
        for (int s = 0; s < WARPS * L::STAGES + 1; ++s) mbar_init(sbase + L::BAR_OFF + 8u * s, 1);
        *abort_word = 0u;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();   // the previous grid's writes (Q, the cache, the lengths) are visible

    // ------------------------------------------------ this CTA's units
    const int cta = static_cast<int>(blockIdx.x);
    const int pairs_b = p.H_kv * p.row_tiles;            // pairs per entry
    int b = 0, pr = 0, blk = 0;                          // entry, pair inside it, first block
    int64_t todo;                                        // units to take
    bool mid_pair = false;                               // the first segment began in an earlier CTA
    if (!p.split) {
        b = cta / pairs_b;
        pr = cta - b * pairs_b;
        todo = pair_blocks(p, b);
    } else {
        int64_t total;
        const bool ragged = mask_has_lengths(p.mask);
        if (ragged) {
            int64_t sum = 0;
            for (int i = lane; i < p.B; i += 32) sum += pair_blocks(p, i);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            total = sum * pairs_b;
        } else {
            total = static_cast<int64_t>(p.B) * pairs_b * pair_blocks(p, 0);
        }
        // at least one block per warp
        const int64_t ctas = max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.ctas), total / WARPS));
        if (cta >= ctas) {
            if (threadIdx.x == 0) p.part_flags[cta] = make_int2(-1, 0);
            return;
        }
        const int64_t u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
        todo = u1 - u0;
        int64_t before = 0;                              // units of the entries before b
        if (ragged) {
            for (int base = 0; base < p.B; base += 32) {
                const int64_t nb = base + lane < p.B ? static_cast<int64_t>(pair_blocks(p, base + lane)) * pairs_b : 0;
                int64_t incl = nb;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += v;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, before + incl > u0);
                if (past != 0u) {
                    const int l = __ffs(past) - 1;
                    b = base + l;
                    before += __shfl_sync(0xffffffffu, incl - nb, l);
                    break;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
        } else {
            const int64_t per = static_cast<int64_t>(pairs_b) * pair_blocks(p, 0);
            b = static_cast<int>(u0 / per);
            before = per * b;
        }
        const int nb = pair_blocks(p, b);
        pr = static_cast<int>((u0 - before) / nb);
        blk = static_cast<int>((u0 - before) - static_cast<int64_t>(pr) * nb);
        mid_pair = blk > 0;
    }

    bool ok = true;
    if (p.debug_flags & DEBUG_FORCE_TIMEOUT) {
        ok = mbar_wait(bar_never, 0, abort_word, p.status, STATUS_FORCED, 20000000ull);
        ok = __all_sync(0xffffffffu, ok);
    }
    uint32_t landed = 0;                                 // blocks this warp has waited for, over all segments
    int tail_pair = -1, head_end = 0;
    const int pi = 4 * (g & 1) + (g >> 1);               // slot of tile row g inside a 16-slot tile
    // byte offsets of this thread's codes and words inside a block
    const int k_lo = q4::k_row(pi, DK) * (DK / 2) + t * 8 * NGK, k_hi = q4::k_row(pi + 8, DK) * (DK / 2) + t * 8 * NGK;
    const int v_0 = q4::v_off(DK) + q4::v_code_off(t, 0, g, DV);
    const int w_lo = 2 * NGK * pi, vw_lo = 2 * NGV * pi;

    while (todo > 0) {
        int kv_len;
        const int end = visible_end(p, b, &kv_len);      // slots past it are seen by no row
        const int nb = max(1, (end + q4::BLOCK - 1) / q4::BLOCK);
        const int take = static_cast<int>(min(static_cast<int64_t>(nb - blk), todo));
        const int hk = pr / p.row_tiles, rt = pr - hk * p.row_tiles;
        const int64_t pair_bh = static_cast<int64_t>(b) * p.H_kv + hk;
        const uint8_t* src = p.cache + (pair_bh * p.blocks + blk) * L::BYTES_BLOCK;
        const int mine = take > warp ? (take - warp + WARPS - 1) / WARPS : 0;   // blocks warp, warp + 4, ...
        const int count = end > 0 ? mine : 0;
        auto issue = [&](int i) {                        // block i of this warp into its stage
            const uint32_t s = (landed + static_cast<uint32_t>(i)) % L::STAGES;
            mbar_arrive_expect_tx(bar0 + 8u * s, L::BYTES_BLOCK);
            bulk_load(sbase + (warp * L::STAGES + s) * L::BYTES_BLOCK, src + static_cast<int64_t>(warp + WARPS * i) * L::BYTES_BLOCK,
                      L::BYTES_BLOCK, bar0 + 8u * s);
        };
        int issued = 0;
        if (ok) {
            issued = min(count, L::STAGES);
            if (lane == 0)
                for (int i = 0; i < issued; ++i) issue(i);
        }

        // -------------------------------------------- the query rows, as fp16 B operands
        uint32_t bq[NT][NGK][4][2];
        float sq[NT][2][NGK], fac[NT][2];
        float slope[NT][2];
        int lim[NT][2], pos[NT][2];
        const int r0 = rt * L::ROWS;
        const int off = causal_offset(p.mask, p.m - p.n, kv_len, p.n);
        int min_lim = end;                               // every row sees the slots below it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = r0 + 8 * nt + g;
            uint32_t qv[NGK][8];
            uint32_t top = 0u;
#pragma unroll
            for (int q = 0; q < NGK; ++q) {
#pragma unroll
                for (int i = 0; i < 8; ++i) qv[q][i] = 0u;
                if (r < p.R) {
                    const uint4* qp = reinterpret_cast<const uint4*>(p.Q + (pair_bh * p.R + r) * DK + 64 * q + 16 * t);
                    const uint4 x = __ldg(qp), y = __ldg(qp + 1);
                    qv[q][0] = x.x; qv[q][1] = x.y; qv[q][2] = x.z; qv[q][3] = x.w;
                    qv[q][4] = y.x; qv[q][5] = y.y; qv[q][6] = y.z; qv[q][7] = y.w;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, max(qv[q][i] & 0x7FFFu, (qv[q][i] >> 16) & 0x7FFFu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^e q has its largest magnitude in [2^14, 2^15); an infinity or NaN stays one
            const int e = max(-113, min(110, 14 - (static_cast<int>(top >> 7) - 127)));
            const float up = pow2i(e);
            float sum[NGK];
#pragma unroll
            for (int q = 0; q < NGK; ++q) {
                float x[16];
                sum[q] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[2 * i] = __uint_as_float(qv[q][i] << 16) * up;
                    x[2 * i + 1] = __uint_as_float(qv[q][i] & 0xFFFF0000u) * up;
                    sum[q] += x[2 * i] + x[2 * i + 1];
                }
                // word w, half h: nibbles 2 h (u 2^-24) and 2 h + 1 (u 2^-20) of both 16-bit halves
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = 8 * w + 2 * h;
                        bq[nt][q][2 * w + h][0] = pack_f16x2(x[c], x[c + 4]);
                        bq[nt][q][2 * w + h][1] = pack_f16x2(x[c + 1] * 0.0625f, x[c + 5] * 0.0625f);
                    }
                sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 1);
                sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 2);
            }
            // per column of the accumulators (query rows 2 t and 2 t + 1 of this tile)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int srcl = 4 * (2 * t + c);
#pragma unroll
                for (int q = 0; q < NGK; ++q) sq[nt][c][q] = __shfl_sync(0xffffffffu, sum[q], srcl) * (1.f / TWO24);
                const int ec = __shfl_sync(0xffffffffu, e, srcl);
                // scale * log2(e) * 2^(24 - e), kept finite
                fac[nt][c] = fminf(p.scale_log2 * pow2i(24 - max(ec, -100)) * pow2i(max(0, -100 - ec)), 3e38f);
                const int rc = r0 + 8 * nt + 2 * t + c;
                const int i = rc % p.n;
                pos[nt][c] = i + off;
                lim[nt][c] = mask_is_causal(p.mask) ? min(kv_len, i + off + 1) : kv_len;
                slope[nt][c] = p.slopes != nullptr && rc < p.R ? __ldg(p.slopes + hk * (p.R / p.n) + rc / p.n) * LOG2E : 0.f;
                min_lim = min(min_lim, lim[nt][c]);
            }
        }
        min_lim = __reduce_min_sync(0xffffffffu, min_lim);
        const bool biased = p.slopes != nullptr;

        float m_run[NT][2], l_run[NT][2], corr[NT][2][NGV], o[NT][NGV][4][4], rg[NGV];
#pragma unroll
        for (int q = 0; q < NGV; ++q) rg[q] = 0.f;       // 0: no reference yet
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m_run[nt][c] = -INFINITY;
                l_run[nt][c] = 0.f;
#pragma unroll
                for (int q = 0; q < NGV; ++q) corr[nt][c][q] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < NGV; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[nt][q][j][c] = 0.f;
        }

        // -------------------------------------------- the blocks
        for (int it = 0; ok && it < count; ++it) {
            const uint32_t stage = landed % L::STAGES;
            ok = mbar_wait(bar0 + 8u * stage, (landed / L::STAGES) & 1u, abort_word, p.status, STATUS_SOFTMAX_WAIT,
                           p.watchdog_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t* sb = smem + (warp * L::STAGES + stage) * L::BYTES_BLOCK;
            const int key0 = (blk + warp + WARPS * it) * q4::BLOCK;
            const bool masked = key0 + q4::BLOCK > min_lim;

            // scores, scaled to the log2 domain
            float x[4][NT][4];
#pragma unroll
            for (int tile = 0; tile < 4; ++tile) {
                uint32_t lo[2 * NGK], hi[2 * NGK];
                const uint8_t* kb = sb + tile * 16 * (DK / 2);
                if (NGK == 2) {
                    const uint4 a = *reinterpret_cast<const uint4*>(kb + k_lo), c = *reinterpret_cast<const uint4*>(kb + k_hi);
                    lo[0] = a.x; lo[1] = a.y; lo[2 * NGK - 2] = a.z; lo[2 * NGK - 1] = a.w;
                    hi[0] = c.x; hi[1] = c.y; hi[2 * NGK - 2] = c.z; hi[2 * NGK - 1] = c.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2*>(kb + k_lo), c = *reinterpret_cast<const uint2*>(kb + k_hi);
                    lo[0] = a.x; lo[1] = a.y;
                    hi[0] = c.x; hi[1] = c.y;
                }
                const uint8_t* wb = sb + q4::k_words_off(DK) + tile * 16 * 2 * NGK + w_lo;
                uint32_t wl, wh;
                if (NGK == 2) {
                    wl = *reinterpret_cast<const uint32_t*>(wb);
                    wh = *reinterpret_cast<const uint32_t*>(wb + 8 * 2 * NGK);
                } else {
                    wl = *reinterpret_cast<const uint16_t*>(wb);
                    wh = *reinterpret_cast<const uint16_t*>(wb + 8 * 2 * NGK);
                }
#pragma unroll
                for (int q = 0; q < NGK; ++q) {
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[nt][c] = 0.f;
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a = lo[2 * q + w] >> (8 * h), c = hi[2 * q + w] >> (8 * h);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(acc[nt], a & LO, c & LO, a & HI, c & HI, bq[nt][q][2 * w + h][0],
                                        bq[nt][q][2 * w + h][1]);
                        }
                    const float s0 = word_step(wl >> (16 * q)), s1 = word_step(wh >> (16 * q));
                    const float z0 = word_zero(wl >> (16 * q)), z1 = word_zero(wh >> (16 * q));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float v = fmaf(c < 2 ? -z0 : -z1, sq[nt][c & 1][q], acc[nt][c]);
                            const float s = c < 2 ? s0 : s1;
                            x[tile][nt][c] = q == 0 ? v * s : fmaf(v, s, x[tile][nt][c]);
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[tile][nt][c] *= fac[nt][c & 1];
            }
            if (biased) {
#pragma unroll
                for (int tile = 0; tile < 4; ++tile)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int key = key0 + 16 * tile + pi + 8 * (c >> 1);
                            x[tile][nt][c] = fmaf(-slope[nt][c & 1], fabsf(static_cast<float>(pos[nt][c & 1] - key)),
                                                  x[tile][nt][c]);
                        }
            }
            if (masked) {
#pragma unroll
                for (int tile = 0; tile < 4; ++tile)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (key0 + 16 * tile + pi + 8 * (c >> 1) >= lim[nt][c & 1]) x[tile][nt][c] = -INFINITY;
            }

            // online softmax: x becomes the weights
            bool grew = false;
            float alpha[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(x[0][nt][c], x[0][nt][c + 2]);
#pragma unroll
                    for (int tile = 1; tile < 4; ++tile) mx = max3f(mx, x[tile][nt][c], x[tile][nt][c + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float m_new = fmaxf(m_run[nt][c], mx);
                    const float m_use = m_new == -INFINITY ? 0.f : m_new;
                    alpha[nt][c] = ex2_approx(m_run[nt][c] - m_use);
                    grew = grew || m_new > m_run[nt][c];
                    float sum = 0.f;
#pragma unroll
                    for (int tile = 0; tile < 4; ++tile) {
                        x[tile][nt][c] = ex2_approx(x[tile][nt][c] - m_use);
                        x[tile][nt][c + 2] = ex2_approx(x[tile][nt][c + 2] - m_use);
                        sum += x[tile][nt][c] + x[tile][nt][c + 2];
                    }
                    l_run[nt][c] = fmaf(l_run[nt][c], alpha[nt][c], sum);
                    m_run[nt][c] = m_new;
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int q = 0; q < NGV; ++q) {
                        corr[nt][0][q] *= alpha[nt][0];
                        corr[nt][1][q] *= alpha[nt][1];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[nt][q][j][c] *= alpha[nt][c & 1];
                    }
            }

            // the value groups' steps, and the power of two that keeps p s R inside fp16
            uint32_t vw[4][2];
            float smax[NGV];
#pragma unroll
            for (int q = 0; q < NGV; ++q) smax[q] = 0.f;
#pragma unroll
            for (int tile = 0; tile < 4; ++tile)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* wb = sb + q4::v_words_off(DK, DV) + (16 * tile + 8 * h) * 2 * NGV + vw_lo;
                    uint32_t w = NGV == 2 ? *reinterpret_cast<const uint32_t*>(wb) : *reinterpret_cast<const uint16_t*>(wb);
                    if (masked && key0 + 16 * tile + 8 * h + pi >= end) w = 0u;   // never written, perhaps
                    vw[tile][h] = w;
#pragma unroll
                    for (int q = 0; q < NGV; ++q) smax[q] = fmaxf(smax[q], word_step(w >> (16 * q)));   // a NaN step is passed over
                }
            bool over = false;
#pragma unroll
            for (int q = 0; q < NGV; ++q) over = over || rg[q] == 0.f || smax[q] * rg[q] > 32768.f;
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int q = 0; q < NGV; ++q) {
                    const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(smax[q])));
                    if (rg[q] != 0.f && top * rg[q] <= 32768.f) continue;
                    const float r_new = pow2i(max(-126, min(126, 12 - exponent(top))));
                    const float f = rg[q] == 0.f ? 0.f : r_new / rg[q];
                    rg[q] = r_new;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        corr[nt][0][q] *= f;
                        corr[nt][1][q] *= f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[nt][q][j][c] *= f;
                    }
                }
            }

            // O^T += V^T (p s R)^T
#pragma unroll
            for (int tile = 0; tile < 4; ++tile) {
                uint32_t bp[NT][NGV][2];
#pragma unroll
                for (int q = 0; q < NGV; ++q) {
                    const float s0 = word_step(vw[tile][0] >> (16 * q)) * rg[q], s1 = word_step(vw[tile][1] >> (16 * q)) * rg[q];
                    const float z0 = word_zero(vw[tile][0] >> (16 * q)), z1 = word_zero(vw[tile][1] >> (16 * q));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float w[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            w[c] = x[tile][nt][c] * (c < 2 ? s0 : s1);
                            // a masked weight is 0 whatever the group's step (0 times NaN otherwise)
                            if (masked && x[tile][nt][c] == 0.f) w[c] = 0.f;
                            corr[nt][c & 1][q] = fmaf(w[c], c < 2 ? z0 : z1, corr[nt][c & 1][q]);
                        }
                        bp[nt][q][0] = transpose8(pack_f16x2(w[0], w[1]));
                        bp[nt][q][1] = transpose8(pack_f16x2(w[2], w[3]));
                    }
                }
                uint32_t vc[4][NGV];                     // slots t, t + 4, t + 8, t + 12 of the tile
                const uint8_t* vb = sb + v_0 + tile * 16 * (DV / 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (NGV == 2) {
                        const uint2 a = *reinterpret_cast<const uint2*>(vb + 4 * i * (DV / 2));
                        vc[i][0] = a.x;
                        vc[i][NGV - 1] = a.y;
                    } else {
                        vc[i][0] = *reinterpret_cast<const uint32_t*>(vb + 4 * i * (DV / 2));
                    }
                }
#pragma unroll
                for (int q = 0; q < NGV; ++q)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {     // codes 4 hf .. 4 hf + 3 of both slots of a pair
                        const uint32_t a = __byte_perm(vc[0][q], vc[1][q], hf ? 0x7632 : 0x5410);
                        const uint32_t c = __byte_perm(vc[2][q], vc[3][q], hf ? 0x7632 : 0x5410);
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj) {
                            const uint32_t as = a >> (8 * jj), cs = c >> (8 * jj);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(o[nt][q][2 * hf + jj], as & LO, as & HI, cs & LO, cs & HI, bp[nt][q][0], bp[nt][q][1]);
                        }
                    }
            }
            ++landed;
            __syncwarp();                                // every lane is done with the stage
            if (it + L::STAGES < count) {
                // (issue() counts from the first block that has not landed)
                if (lane == 0) {
                    const uint32_t s = stage;
                    mbar_arrive_expect_tx(bar0 + 8u * s, L::BYTES_BLOCK);
                    bulk_load(sbase + (warp * L::STAGES + s) * L::BYTES_BLOCK,
                              src + static_cast<int64_t>(warp + WARPS * (it + L::STAGES)) * L::BYTES_BLOCK, L::BYTES_BLOCK,
                              bar0 + 8u * s);
                }
                ++issued;
            }
        }
        if (!ok) {
            // land what is still in flight before the ring is written or the CTA ends
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t i = landed % L::STAGES, k = 0; issued > 0 && k < L::STAGES; ++k, i = (i + 1) % L::STAGES)
                while (!mbar_test(bar0 + 8u * i, ((landed + k) / L::STAGES) & 1u) && globaltimer_ns() - t0 < 100000000ull) {
                }
        }

        // -------------------------------------------- merge the four warps (the ring is free now)
        __syncthreads();
        float* red = reinterpret_cast<float*>(smem) + warp * L::RED_WARP;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * nt + 2 * t + c;
                float l = l_run[nt][c];
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
                if (g == 0) {
                    red[row] = m_run[nt][c];
                    red[L::ROWS + row] = l;
                }
#pragma unroll
                for (int q = 0; q < NGV; ++q) {
                    float z = corr[nt][c][q];
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) z += __shfl_xor_sync(0xffffffffu, z, sh);
                    const float inv = rg[q] == 0.f ? 0.f : 1.f / rg[q];
                    float* dst = red + 2 * L::ROWS + row * DV + 64 * q + 8 * g;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dst[2 * j] = fmaf(o[nt][q][j][c], TWO24, -z) * inv;
                        dst[2 * j + 1] = fmaf(o[nt][q][j][c + 2], TWO20, -z) * inv;
                    }
                }
            }
        __syncthreads();
        const bool ends = blk + take == nb;
        const bool whole = ends && !mid_pair;
        const int part = 2 * cta + (mid_pair ? 0 : 1);
        const int rows = min(L::ROWS, p.R - r0);
        const float* all = reinterpret_cast<const float*>(smem);
        for (int e = threadIdx.x; e < rows * DV; e += THREADS) {
            const int row = e / DV, c = e % DV;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) M = fmaxf(M, all[w * L::RED_WARP + row]);
            const float M_use = M == -INFINITY ? 0.f : M;
            float Lsum = 0.f, Oc = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float* rw = all + w * L::RED_WARP;
                const float f = ex2_approx(rw[row] - M_use);
                Lsum = fmaf(rw[L::ROWS + row], f, Lsum);
                Oc = fmaf(rw[2 * L::ROWS + row * DV + c], f, Oc);
            }
            if (whole) {
                const int64_t orow = pair_bh * p.R + r0 + row;
                // (a NaN sum is not 0: it reaches the output)
                const float out = Lsum == 0.f ? 0.f : Oc / Lsum;
                p.O[orow * DV + c] = static_cast<uint16_t>(pack_bf16x2(out, 0.f) & 0xFFFFu);
                if (c == 0 && p.LSE != nullptr) p.LSE[orow] = Lsum == 0.f ? -INFINITY : (M_use + __log2f(Lsum)) * LN2;
            } else {
                const int64_t prow = static_cast<int64_t>(part) * p.part_rows + row;
                p.part_o[prow * DV + c] = Oc;
                if (c == 0) {
                    p.part_ml[2 * prow] = M;
                    p.part_ml[2 * prow + 1] = Lsum;
                }
            }
        }
        if (!whole) {
            if (mid_pair) head_end = ends ? 1 : 0;
            else tail_pair = static_cast<int>(pair_bh) * p.row_tiles + rt;
        }
        fence_proxy_async_smem();                        // the merge's writes come before the next copies into the ring
        __syncthreads();

        todo -= take;
        blk = 0;
        mid_pair = false;
        if (++pr == pairs_b) {
            pr = 0;
            ++b;
        }
    }
    if (p.split && threadIdx.x == 0) p.part_flags[cta] = make_int2(tail_pair, head_end);
}

// Merge of the parts of a cut pair: CTA (c, row) for the pair whose first part is
// CTA c's slot 1; the parts after it are the slots 0 of CTAs c + 1, c + 2, ... up to the
// one that ends the pair. One thread per output column.
template <int DV>
__global__ void __launch_bounds__(DV)
attn_decode_q4_merge_kernel(const DecodeQ4Params p, int tile_rows)
{
    griddep_wait();   // the parts are visible
    const int c = static_cast<int>(blockIdx.x), row = static_cast<int>(blockIdx.y);
    const int pair = p.part_flags[c].x;
    if (pair < 0) return;
    const int64_t pair_bh = pair / p.row_tiles;
    const int r = (pair % p.row_tiles) * tile_rows + row;
    if (r >= p.R) return;
    int parts = 1;                                       // one warp-wide look at the flags per 32 parts
    for (int base = c + 1;; base += 32) {
        const int i = base + static_cast<int>(threadIdx.x % 32);
        const uint32_t ends = __ballot_sync(0xffffffffu, i >= p.ctas || p.part_flags[i].y != 0);
        if (ends != 0u) {
            parts += __ffs(ends);
            break;
        }
        parts += 32;
    }
    parts = min(parts, p.ctas - c);
    auto part_row = [&](int s) -> int64_t {
        return static_cast<int64_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)) * p.part_rows + row;
    };
    float M = -INFINITY;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) M = fmaxf(M, p.part_ml[2 * part_row(s)]);
    const float M_use = M == -INFINITY ? 0.f : M;
    float Lsum = 0.f, Oc = 0.f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const int64_t pr = part_row(s);
        const float f = ex2_approx(p.part_ml[2 * pr] - M_use);
        Lsum = fmaf(p.part_ml[2 * pr + 1], f, Lsum);
        Oc = fmaf(p.part_o[pr * DV + threadIdx.x], f, Oc);
    }
    const int64_t orow = pair_bh * p.R + r;
    const float out = Lsum == 0.f ? 0.f : Oc / Lsum;
    p.O[orow * DV + threadIdx.x] = static_cast<uint16_t>(pack_bf16x2(out, 0.f) & 0xFFFFu);
    if (threadIdx.x == 0 && p.LSE != nullptr) p.LSE[orow] = Lsum == 0.f ? -INFINITY : (M_use + __log2f(Lsum)) * LN2;
}

template <int DK, int DV, int NT>
cudaError_t launch(const DecodeQ4Params& p, cudaStream_t stream)
{
    using L = Layout<DK, DV, NT>;
    auto kern = attn_decode_q4_kernel<DK, DV, NT>;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    e = launch_pdl(kern, dim3(static_cast<unsigned>(p.ctas)), dim3(THREADS), L::BYTES, stream, p);
    if (e != cudaSuccess || !p.split) return e;
    return launch_pdl(attn_decode_q4_merge_kernel<DV>, dim3(static_cast<unsigned>(p.ctas), static_cast<unsigned>(p.part_rows)),
                      dim3(DV), 0, stream, p, L::ROWS);
}

}  // namespace dq4
}  // namespace attn
