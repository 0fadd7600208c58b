// Joining the shares of a row of attention: each has its unnormalised output, the reference (log2) that its weights were
// taken against, and their sum.
#pragma once
#include "common.cuh"
#include "elem.cuh"

namespace csa2 {

// One row of 512 dims, four a thread (dim = tid % 128): SPREAD 1, 128 threads; SPREAD 4, four groups of 128 that take every
// fourth share and are added up in order.  `share(s)` is the row of share s in part_o and part_ml; shares whose sum is zero
// are not taken into account, whatever their outputs hold.
template <typename TO, int SPREAD, typename F>
__device__ __forceinline__ void join_row(const float* part_o, const float2* part_ml, int n, F&& share, TO* out, float* lse) {
    __shared__ float4 sums[SPREAD > 1 ? 3 : 1][128];
    const int tid = threadIdx.x, dim = tid & 127, group = SPREAD > 1 ? tid >> 7 : 0, lane = tid & 31;
    constexpr int NB = 8;                            // shares in flight
    float m = -INFINITY, l = 0.0f;
    for (int s = lane; s < n; s += 32) {
        const float2 v = part_ml[share(s)];
        if (v.y != 0.0f) m = fmaxf(m, v.x);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int s = lane; s < n; s += 32) {
        const float2 v = part_ml[share(s)];
        if (v.y != 0.0f) l = fmaf(exp2f(v.x - m), v.y, l);
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float o[4] = {};
    for (int s0 = group; s0 < n; s0 += NB * SPREAD) {
        float4 x[NB];
        float2 v[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t at = share(min(s0 + i * SPREAD, n - 1));
            x[i] = reinterpret_cast<const float4*>(part_o + at * D_LAT)[dim];
            v[i] = part_ml[at];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (s0 + i * SPREAD >= n || v[i].y == 0.0f) continue;
            const float f = exp2f(v[i].x - m);
            o[0] = fmaf(f, x[i].x, o[0]), o[1] = fmaf(f, x[i].y, o[1]);
            o[2] = fmaf(f, x[i].z, o[2]), o[3] = fmaf(f, x[i].w, o[3]);
        }
    }
    if constexpr (SPREAD > 1) {
        if (group > 0) sums[group - 1][dim] = make_float4(o[0], o[1], o[2], o[3]);
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const float4 x = sums[i][dim];
            o[0] += x.x, o[1] += x.y, o[2] += x.z, o[3] += x.w;
        }
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    ElemVec<TO, 4> y;
    y.pack(o);
    y.store(out + 4 * dim);
    if (lse != nullptr && dim == 0) *lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace csa2
