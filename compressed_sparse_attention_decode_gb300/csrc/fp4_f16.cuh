// FP4 rows as exact fp16 operands, and bf16 rows as fp16 after a power-of-two scale.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

namespace csa2 {

// 2^e as a float, for -126 <= e <= 127
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// the largest bf16 magnitude (as bits, sign cleared) of the eight values in v
__device__ __forceinline__ uint32_t bf16_absmax8(const uint4& v) {
    const uint32_t a = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), b = __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
    const uint32_t m = __vmaxu2(a, b);
    return max(m & 0xffffu, m >> 16);
}

// The exponent E by which values whose largest magnitude has bf16 bits `mx` are divided
// before they go to fp16: 0 while that magnitude lies in [2^-10, 2^15) or is 0, else the E
// that brings it into [2^14, 2^15), kept within [-100, 100].
__device__ __forceinline__ int f16_range_exp(uint32_t mx) {
    if (mx == 0u) return 0;
    const int e = (int)((mx >> 7) & 0xffu) - 127;
    if (e >= -10 && e < 15) return 0;
    return max(-100, min(100, e - 14));
}

__device__ __forceinline__ uint32_t f16x2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// eight bf16 values times d (a power of two) as fp16: exact unless a value leaves fp16's range
__device__ __forceinline__ uint4 bf16x8_to_f16x8(const uint4& v, float d) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f16x2_bits(__uint_as_float(w[i] << 16) * d, __uint_as_float(w[i] & 0xffff0000u) * d);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// two E4M3 bytes (low byte -> low half) to fp16, exactly
__device__ __forceinline__ __half2 e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(r) : "r"(two));
    return *reinterpret_cast<__half2*>(&r);
}
// eight E2M1 codes to fp16
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, __half2* o) {
    uint32_t r[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<__half2*>(&r[i]);
}
// eight E2M1 codes times their scale, as packed fp16 (exact)
__device__ __forceinline__ uint4 e2m1x8_scaled(uint32_t w, __half2 s) {
    __half2 h[4];
    e2m1x8_to_f16x8(w, h);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hmul2(h[i], s);
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

namespace umma {
// true in one lane of the (whole) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}
}  // namespace umma

}  // namespace csa2
