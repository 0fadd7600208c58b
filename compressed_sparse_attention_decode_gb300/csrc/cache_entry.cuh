// What an entry of the cache is made of: one or two bf16 rows, merged, quantised, and projected to the
// indexer key.  Shared by the cache write (every sequence at one position) and the append (each at its own).
#pragma once
#include "common.cuh"

namespace csa2 {

// 16 bf16 values as fp32
__device__ __forceinline__ void bf16x16_to_f32(const uint4& a, const uint4& b, float* x) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = bf16_bits_to_f32((c & 1) ? (w[c >> 1] >> 16) : (w[c >> 1] & 0xffffu));
}
// .. read from memory that the kernel does not write
__device__ __forceinline__ void row16(const uint16_t* __restrict__ p, float* x) {
    bf16x16_to_f32(__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p) + 1), x);
}

// x <- fmaf(w1, h1, float(w0 * x)), 16 channels: one rounded product, one fused multiply-add
__device__ __forceinline__ void merge16(float* x, const float* h1, const float* __restrict__ w0,
                                        const float* __restrict__ w1) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const float4 p = __ldg(reinterpret_cast<const float4*>(w0) + v);
        const float4 q = __ldg(reinterpret_cast<const float4*>(w1) + v);
        const float pw[4] = {p.x, p.y, p.z, p.w};
        const float qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) x[4 * v + t] = __fmaf_rn(qw[t], h1[4 * v + t], __fmul_rn(pw[t], x[4 * v + t]));
    }
}

// E4M3 value times 2^9 (an integer below 2^18: the smallest E4M3 value is 2^-9)
__device__ __forceinline__ int cw_e4m3_x512(uint32_t b) {
    const uint32_t e = (b >> 3) & 15u, m = b & 7u;
    return e ? (int)((8u + m) << (e - 1u)) : (int)m;
}

}  // namespace csa2
