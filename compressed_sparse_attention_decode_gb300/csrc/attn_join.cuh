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
    constexpr int NB = SPREAD > 1 ? 8 : 4, NK = 3;   // shares in flight; at most 96 in all
    float4 x[NB];
    auto load = [&](int s0) {                        // (past the end: the last one again, times nothing)
#pragma unroll
        for (int i = 0; i < NB; ++i)
            if (i == 0 || s0 + i * SPREAD < n)
                x[i] = reinterpret_cast<const float4*>(part_o + (int64_t)share(min(s0 + i * SPREAD, n - 1)) * D_LAT)[dim];
    };
    load(group);                                     // before the factors are known
    float f[NK], m = -INFINITY, l = 0.0f;
    float2 v[NK];
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        v[k] = make_float2(-INFINITY, 0.0f);
        if (32 * k + lane < n) v[k] = part_ml[share(32 * k + lane)];
        if (v[k].y != 0.0f) m = fmaxf(m, v[k].x);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        f[k] = v[k].y != 0.0f ? exp2f(v[k].x - m) : 0.0f;
        l = fmaf(f[k], v[k].y, l);
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float o[4] = {};
    for (int s0 = group; s0 < n;) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int s = s0 + i * SPREAD;
            if (s >= n) break;
            const float w = __shfl_sync(0xffffffffu, s < 32 ? f[0] : s < 64 ? f[1] : f[2], s & 31);
            if (w == 0.0f) continue;
            o[0] = fmaf(w, x[i].x, o[0]), o[1] = fmaf(w, x[i].y, o[1]);
            o[2] = fmaf(w, x[i].z, o[2]), o[3] = fmaf(w, x[i].w, o[3]);
        }
        s0 += NB * SPREAD;
        if (s0 < n) load(s0);
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
