// attn_cache_q4.cu -- writing into a key/value cache held in 4 bits, and reading it
// back as bf16. Both move each byte once; what keeps them from HBM's rate is the
// instructions per channel, so a lane takes 16 channels (a quarter of a group) at a time:
// the group's step, zero and addresses are then shared by 16, and loads and stores of
// bf16 rows are 32 bytes a lane, 1 KB a warp.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_cache_q4.cuh"
#include "attn_internal.h"
#include "sm103a.cuh"

namespace attn {

using namespace sm103a;

namespace {

// 32 bytes of a row of bf16; `wide`: the address is a multiple of 32 (else of 16).
__device__ __forceinline__ void load32(const uint16_t* src, bool wide, uint32_t (&w)[8])
{
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(src));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}

__device__ __forceinline__ void store32(uint16_t* dst, bool wide, const uint32_t (&w)[8])
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Packed bf16 minimum and maximum that give NaN if either operand is one.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

constexpr float RINT = 12582912.f;                       // 1.5 * 2^23: a sum with it holds a whole number in its low bits
constexpr uint32_t RINT_BITS = 0x4B400000u;

// rint(x / s) + RINT for a bf16 x and a step s of four significant bits, |x / s| <= 15,
// with r = 1 / s to within 2^-22. x / s = X / M 2^c with whole X < 256, 8 <= M < 16, so it is
// either exactly halfway between two whole numbers or 1 / 512 or more away from
// halfway. x r is off by less than 2^-18; adding 1.5 * 2^12 rounds it to a multiple of
// 2^-11, which restores an exact half and moves nothing else across one. The second
// sum is round half to even, as the definition has it (RINT is even).
__device__ __forceinline__ float rint_ratio(float x, float r)
{
    const float c = 6144.f;                              // 1.5 * 2^12
    return __fadd_rn(__fmaf_rn(x, r, c), RINT - c);
}

// One lane of four quantises channels 16 t .. 16 t + 15 of a group (t = lane % 4): the
// codes as 16 nibbles, and the group's word (the same in all four lanes).
__device__ __forceinline__ uint2 quantise(const uint32_t (&w)[8], uint32_t* word)
{
    uint32_t hx = w[0], lx = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        hx = max_bf16x2(hx, w[i]);
        lx = min_bf16x2(lx, w[i]);
    }
    // (max x, max -x), at least 0, of the lane and then of the group
    lx ^= 0x80008000u;
    uint32_t top = max_bf16x2(__byte_perm(hx, lx, 0x5410), __byte_perm(hx, lx, 0x7632));
    top = max_bf16x2(top, 0u);
    top = max_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float hi = __uint_as_float(top << 16), neg = __uint_as_float(top & 0xFFFF0000u);
    const float big = 1.7014118346046923e38f;            // 2^127
    if (!(hi < big && neg < big)) {
        *word = q4::BAD_WORD;
        return make_uint2(0u, 0u);
    }
    const float range = __fadd_rn(hi, neg);
    uint2 codes;
    uint32_t u0, sb;
    if (range >= 2.4074124304840448e-35f) {              // 2^-115: steps and their reciprocals are normal numbers
        // The smallest four-bit step with 15 s >= range: the product may be off either
        // way, but only by less than a step, and 15 s has eight bits. (The definition
        // rounds range / 15 to fp32 first, which never reaches a four-bit number from above it.)
        sb = __float_as_uint(range * (1.f / 15.f)) & 0xFFF00000u;
        if (15.f * __uint_as_float(sb) < range) sb += 0x00100000u;
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float(sb)));
        u0 = __float_as_uint(rint_ratio(neg, r)) - RINT_BITS;
        // rint(x / s) + u0 is in 0..15 (rint is odd and monotone, |x| <= hi or neg), except
        // that two exact halves at the ends may add up to 16
        const bool sixteen = __float_as_uint(rint_ratio(hi, r)) - RINT_BITS + u0 > 15u;
        const float most = RINT + 15.f - static_cast<float>(u0);
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t sum = 0u;                           // the rounded sums' bits times 16^i, modulo 2^32
#pragma unroll
            for (int i = 7; i >= 0; --i) {
                const uint32_t pair = w[4 * h + i / 2];
                const float x = __uint_as_float(i % 2 ? pair & 0xFFFF0000u : pair << 16);
                float y = rint_ratio(x, r);
                if (sixteen) y = fminf(y, most);
                sum = sum * 16u + __float_as_uint(y);
            }
            c[h] = sum - (RINT_BITS - u0) * 0x11111111u;
        }
        codes = make_uint2(c[0], c[1]);
    } else {
        sb = (__float_as_uint(__fdiv_rn(range, 15.f)) + 0xFFFFFu) & 0xFFF00000u;
        const float s = __uint_as_float(sb);
        if (sb == 0u) {                                  // every channel is 0
            *word = 0u;
            return make_uint2(0u, 0u);
        }
        u0 = static_cast<uint32_t>(rintf(__fdiv_rn(neg, s)));
        uint32_t c[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
            const int u = static_cast<int>(rintf(__fdiv_rn(x, s))) + static_cast<int>(u0);
            c[i / 8] |= static_cast<uint32_t>(min(max(u, 0), 15)) << (4 * (i % 8));
        }
        codes = make_uint2(c[0], c[1]);
    }
    *word = (sb >> 16) | u0;
    return codes;
}

constexpr int WRITE_GROUPS = 64;                         // groups a CTA takes at once
constexpr int WRITE_ROUNDS = 1;

// Four lanes take one group of one row; the codes of a warp's eight groups fill whole
// 32-byte sectors of the cache.
__global__ void __launch_bounds__(256) cache_q4_write_kernel(const CacheQ4WriteParams p)
{
    griddep_wait();   // K, V and the positions of the earlier kernels are visible, their reads of the cache done
    const int t = threadIdx.x % 4;
    uint32_t w[WRITE_ROUNDS][8];
    uint8_t* dst[WRITE_ROUNDS];                          // codes, or null for a row that is not written
    int slot_k[WRITE_ROUNDS];
#pragma unroll
    for (int u = 0; u < WRITE_ROUNDS; ++u) {
        const uint32_t gi = (blockIdx.x * WRITE_ROUNDS + u) * WRITE_GROUPS + threadIdx.x / 4u;
        const bool is_v = gi >= p.k_groups;
        const uint32_t gj = is_v ? gi - p.k_groups : gi;
        const int d = is_v ? p.d_v : p.d_k;
        const uint32_t row = d == 128 ? gj >> 1 : gj;
        const int q = d == 128 ? static_cast<int>(gj & 1u) : 0;
        const uint32_t bh = p.by_n.divide(row);
        const int i = static_cast<int>(row - bh * static_cast<uint32_t>(p.n));
        const int b = static_cast<int>(p.by_H.divide(bh));
        dst[u] = nullptr;
        slot_k[u] = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) w[u][k] = 0u;
        if (gi < p.groups) {
            const int start = p.starts != nullptr ? __ldg(p.starts + b) : 0;
            const int count = p.counts != nullptr ? __ldg(p.counts + b) : p.n;
            const int64_t slot = static_cast<int64_t>(start) + i;
            if (i < count && slot >= 0 && slot < p.m) {
                load32((is_v ? p.V : p.K) + static_cast<int64_t>(row) * d + q * q4::GROUP + 16 * t, p.wide, w[u]);
                const int k = static_cast<int>(slot) % q4::BLOCK;
                dst[u] = p.cache + (static_cast<int64_t>(bh) * p.blocks + slot / q4::BLOCK) * q4::block_bytes(p.d_k, p.d_v) +
                         (is_v ? q4::v_off(p.d_k) : 0);
                slot_k[u] = (is_v ? 256 : 0) | q << 7 | k;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < WRITE_ROUNDS; ++u) {
        uint32_t word;
        const uint2 codes = quantise(w[u], &word);
        if (dst[u] == nullptr) continue;
        const bool is_v = slot_k[u] & 256;
        const int q = slot_k[u] >> 7 & 1, k = slot_k[u] & 127;
        const int d = is_v ? p.d_v : p.d_k;
        if (is_v) {
            *reinterpret_cast<uint32_t*>(dst[u] + q4::v_code_off(k, q, 2 * t, d)) = codes.x;
            *reinterpret_cast<uint32_t*>(dst[u] + q4::v_code_off(k, q, 2 * t + 1, d)) = codes.y;
        } else {
            *reinterpret_cast<uint2*>(dst[u] + q4::k_code_off(k, q, 2 * t, d)) = codes;
        }
        if (t == 0) *reinterpret_cast<uint16_t*>(dst[u] + 32 * d + 2 * (k * (d / q4::GROUP) + q)) = static_cast<uint16_t>(word);
    }
}

// Values of 16 codes, s (u - u0), in packed bf16: 128 + u and 128 + u0 have eight bits, so
// their difference is exact, and the value itself is a bf16 number.
__device__ __forceinline__ void values(uint2 codes, uint32_t word, uint32_t (&out)[8])
{
    const uint32_t s2 = (word & 0xFFF0u) * 0x10001u;
    const uint32_t z2 = (word & 15u) * 0x10001u | 0x43004300u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = h ? codes.y : codes.x;
        uint32_t v[4];                                   // channels i and i + 4
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"((c >> (4 * i) & 0x000F000Fu) | 0x43004300u), "r"(z2));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(s2));
        }
        out[4 * h] = __byte_perm(v[0], v[1], 0x5410);
        out[4 * h + 1] = __byte_perm(v[2], v[3], 0x5410);
        out[4 * h + 2] = __byte_perm(v[0], v[1], 0x7632);
        out[4 * h + 3] = __byte_perm(v[2], v[3], 0x7632);
    }
}

constexpr int READ_ROUNDS = 1;                           // 16-channel pieces a lane has in flight

// One CTA per (b, cache head, 64 slots): the slots' K and V as bf16 for each of the
// query heads that share them. Slots at or past the entry's length give 0.
__global__ void __launch_bounds__(256) cache_q4_read_kernel(const CacheQ4ReadParams p)
{
    griddep_wait();   // the earlier kernels' writes into the cache are visible, their reads of K and V done
    const uint32_t tiles = static_cast<uint32_t>(p.tiles);
    const uint32_t bh = blockIdx.x / tiles;
    const int j0 = static_cast<int>(blockIdx.x - bh * tiles) * q4::BLOCK;      // first output row
    const int b = static_cast<int>(bh / static_cast<uint32_t>(p.H_kv));
    const int hk = static_cast<int>(bh - static_cast<uint32_t>(b) * p.H_kv);
    const int len = p.key_lengths != nullptr ? __ldg(p.key_lengths + b) : p.m;
    const uint8_t* base = p.cache + static_cast<int64_t>(bh) * p.blocks * q4::block_bytes(p.d_k, p.d_v);
    const int rows = min(q4::BLOCK, p.n - j0);
    const int64_t head0 = (static_cast<int64_t>(b) * p.H + static_cast<int64_t>(hk) * p.group);
    const int k_pieces = rows * (p.d_k / 16), pieces = k_pieces + rows * (p.d_v / 16);
    for (int e0 = threadIdx.x; e0 < pieces; e0 += 256 * READ_ROUNDS) {
        uint2 codes[READ_ROUNDS];
        uint32_t word[READ_ROUNDS];
        uint16_t* dst[READ_ROUNDS];
#pragma unroll
        for (int u = 0; u < READ_ROUNDS; ++u) {
            const int e = e0 + 256 * u;
            const bool is_v = e >= k_pieces;
            const int ee = is_v ? e - k_pieces : e;
            const int d = is_v ? p.d_v : p.d_k;
            const int r = d == 128 ? ee >> 3 : ee >> 2;
            const int piece = ee & (d / 16 - 1), q = piece >> 2, t = piece & 3;
            const int slot = p.first + j0 + r;
            codes[u] = make_uint2(0u, 0u);
            word[u] = 0u;
            dst[u] = e < pieces ? (is_v ? p.V : p.K) + (head0 * p.n + j0 + r) * d + 16 * piece : nullptr;
            if (e < pieces && slot < len) {
                const int k = slot % q4::BLOCK;
                const uint8_t* blk = base + static_cast<int64_t>(slot / q4::BLOCK) * q4::block_bytes(p.d_k, p.d_v) +
                                     (is_v ? q4::v_off(p.d_k) : 0);
                if (is_v) {
                    codes[u].x = __ldg(reinterpret_cast<const uint32_t*>(blk + q4::v_code_off(k, q, 2 * t, d)));
                    codes[u].y = __ldg(reinterpret_cast<const uint32_t*>(blk + q4::v_code_off(k, q, 2 * t + 1, d)));
                } else {
                    codes[u] = __ldg(reinterpret_cast<const uint2*>(blk + q4::k_code_off(k, q, 2 * t, d)));
                }
                word[u] = __ldg(reinterpret_cast<const uint16_t*>(blk + 32 * d) + k * (d / q4::GROUP) + q);
            }
        }
#pragma unroll
        for (int u = 0; u < READ_ROUNDS; ++u) {
            if (dst[u] == nullptr) continue;
            uint32_t out[8];
            values(codes[u], word[u], out);
            const int64_t head = static_cast<int64_t>(p.n) * (e0 + 256 * u >= k_pieces ? p.d_v : p.d_k);
            for (int g = 0; g < p.group; ++g) store32(dst[u] + g * head, p.wide, out);
        }
    }
}

}  // namespace

cudaError_t launch_cache_q4_write(const CacheQ4WriteParams& p, cudaStream_t stream)
{
    const uint32_t per = WRITE_GROUPS * WRITE_ROUNDS;
    return launch_pdl(cache_q4_write_kernel, dim3((p.groups + per - 1) / per), dim3(256), 0, stream, p);
}

cudaError_t launch_cache_q4_read(const CacheQ4ReadParams& p, cudaStream_t stream)
{
    return launch_pdl(cache_q4_read_kernel, dim3(static_cast<unsigned>(p.B) * p.H_kv * p.tiles), dim3(256), 0, stream, p);
}

}  // namespace attn
