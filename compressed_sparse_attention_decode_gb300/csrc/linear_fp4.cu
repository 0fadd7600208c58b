// Products with FP4 weights (E2M1 codes, one E4M3 scale per 16 values, the
// cache's format) for the few tokens of a decode step or a small chunk:
//     y[t][g][m] = alpha * sum_k W[g][m][k] x[t][g][k]
// W is never expanded in memory: 9/16 of a byte per weight is read once.
//
// One warp per output row and 8 tokens; lane l takes the scale groups l, l+32, ..
// of the row (8 bytes of codes and one scale byte), fp32 sums per token, joined
// by shuffles.
#include "common.cuh"
#include "elem.cuh"

namespace csa2 {

constexpr int LF_TOK = 8;

__device__ __forceinline__ float e2m1_to_f32(uint32_t code) {
    const uint32_t m = code & 7u;
    const float v = m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (code & 8u) ? -v : v;
}
// as e4m3_to_f32, with the format's NaN bytes
__device__ __forceinline__ float e4m3_to_f32_nan(uint32_t b) {
    return (b & 127u) == 127u ? __int_as_float(0x7fc00000) : e4m3_to_f32(b);
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(256) k_linear_fp4_rows(const TX* __restrict__ x, int64_t x_tok, int64_t x_group,
                                                         int n_tok, int n_in, int n_out,
                                                         const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, float alpha,
                                                         TY* __restrict__ y, int64_t y_tok, int64_t y_group) {
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.x * 8 + warp, g = blockIdx.y, t0 = blockIdx.z * LF_TOK;
    if (m < n_out) {
        const int64_t row = (int64_t)g * n_out + m;
        const uint2* cw = reinterpret_cast<const uint2*>(codes + row * (n_in / 2));
        const uint8_t* sc = scales + row * (n_in / 16);
        const int nt = min(LF_TOK, n_tok - t0);
        const TX* xp = x + t0 * x_tok + g * x_group;
        float acc[LF_TOK] = {};
        for (int i = lane; i < n_in / 16; i += 32) {
            const uint2 c = cw[i];
            const float s = e4m3_to_f32_nan(sc[i]);
            for (int e = 0; e < 16; ++e) {
                const float w = e2m1_to_f32(((e < 8 ? c.x : c.y) >> (4 * (e & 7))) & 15u) * s;
#pragma unroll
                for (int t = 0; t < LF_TOK; ++t)
                    if (t < nt) acc[t] = fmaf(w, to_f32(xp[t * x_tok + i * 16 + e]), acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < LF_TOK; ++t) {
            for (int o = 16; o; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
            if (lane == 0 && t < nt) y[(t0 + t) * y_tok + g * y_group + m] = from_f32<TY>(alpha * acc[t]);
        }
    }
    __threadfence();    // the attention may stage these rows as its queries before it waits (see norm_rope.cu)
}

namespace {
template <typename TX, typename TY>
cudaError_t lf_launch(const void* x, int64_t x_tok, int64_t x_group, int n_tok, int n_groups, int n_in, int n_out,
                      const uint8_t* codes, const uint8_t* scales, float alpha, void* y, int64_t y_tok,
                      int64_t y_group, cudaStream_t st) {
    const dim3 grid((n_out + 7) / 8, n_groups, (n_tok + LF_TOK - 1) / LF_TOK);
    launch_k(k_linear_fp4_rows<TX, TY>, grid, 256, 0, st, reinterpret_cast<const TX*>(x), x_tok, x_group, n_tok, n_in,
             n_out, codes, scales, alpha, reinterpret_cast<TY*>(y), y_tok, y_group);
    note_launch();
    return cudaGetLastError();
}
template <typename TX, typename... A>
cudaError_t lf_pick_y(int y_type, A... a) {
    if (y_type == CSA2_BF16) return lf_launch<TX, __nv_bfloat16>(a...);
    if (y_type == CSA2_F16) return lf_launch<TX, __half>(a...);
    return lf_launch<TX, float>(a...);
}
}  // namespace

cudaError_t launch_linear_fp4(const void* x, int x_type, int64_t x_tok, int64_t x_group, int n_tok, int n_groups,
                              int n_in, int n_out, const uint8_t* codes, const uint8_t* scales, float alpha, void* y,
                              int y_type, int64_t y_tok, int64_t y_group, cudaStream_t st) {
    if (x_type == CSA2_BF16)
        return lf_pick_y<__nv_bfloat16>(y_type, x, x_tok, x_group, n_tok, n_groups, n_in, n_out, codes, scales, alpha, y,
                                        y_tok, y_group, st);
    if (x_type == CSA2_F16)
        return lf_pick_y<__half>(y_type, x, x_tok, x_group, n_tok, n_groups, n_in, n_out, codes, scales, alpha, y, y_tok,
                                 y_group, st);
    return lf_pick_y<float>(y_type, x, x_tok, x_group, n_tok, n_groups, n_in, n_out, codes, scales, alpha, y, y_tok,
                            y_group, st);
}

}  // namespace csa2
