// attn_cache_q4.cu -- writing into a key/value cache held in 4 bits, and reading it
// back as bf16. Both move each byte once and are bound by HBM.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_cache_q4.cuh"
#include "attn_internal.h"
#include "sm103a.cuh"

namespace attn {

using namespace sm103a;

namespace {

// rint(x / s) for a bf16 x and a step s of four significant bits, |x / s| <= 15, with
// r = 1 / s rounded. x / s = X / M 2^c with whole X < 256, 8 <= M < 16, so it is either
// exactly halfway between two whole numbers or 1 / 512 or more away from halfway. x r is off by less than 2^-19; adding 1.5 * 2^12 rounds it to a multiple of
// 2^-11, which restores an exact half and moves nothing else across one. The last
// sum is round half to even, as the definition has it. Returns the whole number in
// the low bits of 1.5 * 2^23.
__device__ __forceinline__ float rint_ratio(float x, float r)
{
    const float c = 6144.f;                            // 1.5 * 2^12
    const float y = __fadd_rn(__fmaf_rn(x, r, c), -c);
    return __fadd_rn(y, 12582912.f);                   // 1.5 * 2^23
}

// One lane of eight quantises channels 8 c .. 8 c + 7 of a group (c = lane % 8): the
// codes as eight nibbles, and the group's word (the same in all eight lanes).
__device__ __forceinline__ uint32_t quantise(const uint4 v, uint32_t* word)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    float lo = 0.f, hi = 0.f, poison = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        poison = fmaf(x[i], 0.f, poison);              // NaN from a NaN or an infinity
    }
    if (!(poison == 0.f)) hi = INFINITY;
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    const float big = 1.7014118346046923e38f;          // 2^127
    if (!(hi < big && lo > -big)) {
        *word = q4::BAD_WORD;
        return 0u;
    }
    const float t = __fdiv_rn(__fadd_rn(hi, -lo), 15.f);
    const uint32_t sb = (__float_as_uint(t) + 0xFFFFFu) & 0xFFF00000u;
    if (sb == 0u) {                                    // every channel is 0
        *word = 0u;
        return 0u;
    }
    const float s = __uint_as_float(sb);
    uint32_t u[8];
    int u0;
    if (sb >= 0x03000000u) {                           // 1 / s is a normal number
        const float r = __frcp_rn(s);
        u0 = __float_as_int(rint_ratio(-lo, r)) & 15;
        const int base = u0 - 0x4B400000;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = static_cast<uint32_t>(min(max(__float_as_int(rint_ratio(x[i], r)) + base, 0), 15));
    } else {
        u0 = static_cast<int>(rintf(__fdiv_rn(-lo, s)));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = static_cast<uint32_t>(min(max(static_cast<int>(rintf(__fdiv_rn(x[i], s))) + u0, 0), 15));
    }
    *word = (sb >> 16) | static_cast<uint32_t>(u0);
    uint32_t codes = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= u[i] << (4 * i);
    return codes;
}

// Eight lanes take one group of one row; a warp's four groups are 512 contiguous bytes
// of K or V, and their codes fill whole 32-byte sectors of the cache.
__global__ void __launch_bounds__(256) cache_q4_write_kernel(const CacheQ4WriteParams p)
{
    griddep_wait();   // K, V and the positions of the earlier kernels are visible, their reads of the cache done
    const uint32_t gi = blockIdx.x * 32u + threadIdx.x / 8u;
    const int c = threadIdx.x % 8;
    const bool is_v = gi >= p.k_groups;
    const uint32_t gj = is_v ? gi - p.k_groups : gi;
    const int d = is_v ? p.d_v : p.d_k;
    const int ng = d / q4::GROUP;                      // 1 or 2
    const bool live = gi < p.groups;
    const uint32_t row = live ? (ng == 2 ? gj >> 1 : gj) : 0u;
    const int q = static_cast<int>(gj & static_cast<uint32_t>(ng - 1));
    const uint32_t bh = row / static_cast<uint32_t>(p.n);
    const int i = static_cast<int>(row - bh * static_cast<uint32_t>(p.n));
    const int b = static_cast<int>(bh / static_cast<uint32_t>(p.H));
    const int start = p.starts != nullptr ? __ldg(p.starts + b) : 0;
    const int count = p.counts != nullptr ? __ldg(p.counts + b) : p.n;
    const int64_t slot = static_cast<int64_t>(start) + i;
    const bool keep = live && i < count && slot >= 0 && slot < p.m;

    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (keep)
        v = __ldg(reinterpret_cast<const uint4*>((is_v ? p.V : p.K) + static_cast<int64_t>(row) * d + q * q4::GROUP) + c);
    uint32_t word;
    const uint32_t codes = quantise(v, &word);
    if (!keep) return;
    const int k = static_cast<int>(slot) % q4::BLOCK;
    uint8_t* blk = p.cache + (static_cast<int64_t>(bh) * p.blocks + slot / q4::BLOCK) * q4::block_bytes(p.d_k, p.d_v) +
                   (is_v ? q4::v_off(p.d_k) : 0);
    *reinterpret_cast<uint32_t*>(blk + (is_v ? q4::v_code_off(k, q, c, d) : q4::k_code_off(k, q, c, d))) = codes;
    if (c == 0) *reinterpret_cast<uint16_t*>(blk + 32 * d + 2 * (k * ng + q)) = static_cast<uint16_t>(word);
}

// Values of eight codes: s (u - u0), each a bf16 number, so the upper half of the fp32.
__device__ __forceinline__ uint4 values(uint32_t codes, uint32_t word)
{
    const float s = __uint_as_float((word & 0xFFF0u) << 16);
    const float zero = 8388608.f + static_cast<float>(word & 15u);   // 2^23 + u0
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = __float_as_uint((__uint_as_float(((codes >> (4 * i)) & 15u) | 0x4B000000u) - zero) * s);
    return make_uint4(__byte_perm(f[0], f[1], 0x7632), __byte_perm(f[2], f[3], 0x7632),
                      __byte_perm(f[4], f[5], 0x7632), __byte_perm(f[6], f[7], 0x7632));
}

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
    const int kc = p.d_k / 8, vc = p.d_v / 8;                                  // 16-byte pieces a row
    const int rows = min(q4::BLOCK, p.n - j0);
    const int64_t head0 = (static_cast<int64_t>(b) * p.H + static_cast<int64_t>(hk) * p.group);
    for (int e = threadIdx.x; e < rows * (kc + vc); e += 256) {
        const bool is_v = e >= rows * kc;
        const int ee = is_v ? e - rows * kc : e;
        const int pieces = is_v ? vc : kc;                                     // 8 or 16
        const int r = pieces == 16 ? ee >> 4 : ee >> 3;
        const int piece = ee & (pieces - 1);
        const int q = piece >> 3, c = piece & 7;
        const int d = is_v ? p.d_v : p.d_k;
        const int slot = p.first + j0 + r;
        uint4 out = make_uint4(0u, 0u, 0u, 0u);
        if (slot < len) {
            const int k = slot % q4::BLOCK;
            const uint8_t* blk = base + static_cast<int64_t>(slot / q4::BLOCK) * q4::block_bytes(p.d_k, p.d_v) +
                                 (is_v ? q4::v_off(p.d_k) : 0);
            const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>(
                blk + (is_v ? q4::v_code_off(k, q, c, d) : q4::k_code_off(k, q, c, d))));
            const uint32_t word = __ldg(reinterpret_cast<const uint16_t*>(blk + 32 * d) + k * (d / q4::GROUP) + q);
            out = values(codes, word);
        }
        uint16_t* dst = (is_v ? p.V : p.K) + (head0 * p.n + j0 + r) * d + 8 * piece;
        for (int g = 0; g < p.group; ++g)
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(g) * p.n * d) = out;
    }
}

}  // namespace

cudaError_t launch_cache_q4_write(const CacheQ4WriteParams& p, cudaStream_t stream)
{
    return launch_pdl(cache_q4_write_kernel, dim3((p.groups + 31u) / 32u), dim3(256), 0, stream, p);
}

cudaError_t launch_cache_q4_read(const CacheQ4ReadParams& p, cudaStream_t stream)
{
    return launch_pdl(cache_q4_read_kernel, dim3(static_cast<unsigned>(p.B) * p.H_kv * p.tiles), dim3(256), 0, stream, p);
}

}  // namespace attn
