// Element types of the operators that take bf16, fp16 or fp32 rows: loads to and
// stores from fp32 (one rounding, to nearest even, where the type is narrower).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace csa2 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The N consecutive elements at p as fp32, p aligned to min(16, N * sizeof(T)) bytes.
template <typename T, int N>
struct ElemVec {
    static constexpr int BYTES = N * (int)sizeof(T);
    static constexpr int WORDS = BYTES >= 4 ? BYTES / 4 : 1;
    uint32_t w[WORDS];                       // the raw bits

    __device__ __forceinline__ void load(const T* p) {
        if constexpr (BYTES % 16 == 0) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (BYTES % 16 == 0) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (BYTES == 4) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
        }
    }
    // the same one element at a time, for rows that the wide accesses' alignment does not hold for
    __device__ __forceinline__ void load_each(const T* p) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + 2 * i;
                w[i] = q[0] | (N > 1 ? (uint32_t)q[N > 1 ? 1 : 0] << 16 : 0u);
            }
        }
    }
    __device__ __forceinline__ void store_each(T* p) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                uint16_t* q = reinterpret_cast<uint16_t*>(p) + 2 * i;
                q[0] = (uint16_t)w[i];
                if (N > 1) q[N > 1 ? 1 : 0] = (uint16_t)(w[i] >> 16);
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else {
            const uint16_t b = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            return to_f32(*reinterpret_cast<const T*>(&b));
        }
    }
    // N fp32 values, rounded
    __device__ __forceinline__ void pack(const float* v) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (N == 1) {
            const T e = from_f32<T>(v[0]);
            w[0] = *reinterpret_cast<const uint16_t*>(&e);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&p);
                } else {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
        }
    }
};

}  // namespace csa2
