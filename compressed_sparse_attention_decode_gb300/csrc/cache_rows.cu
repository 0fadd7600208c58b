// Rows into the cache of a ragged batch, and entries back out of it.
//
// csa2_cache_append: what a step has accepted, for sequences that each stand at a position of their own.  Of
// sequence b the rows path[b][0], path[b][1], .. (node numbers of a drafted tree, or rows 0, 1, .. without a path)
// are raw positions pos0[b], pos0[b] + 1, ..; every entry whose last position is among them is written.  In a cache
// of merged pairs an odd pos0 completes the pair whose first half, the row of position pos0 - 1, was carried in
// `prev`; `prev_out` carries the last row on.  The arithmetic is csa2_cache_write's ("DeepSeek-v4.1 Flash:
// KVキャッシュ圧縮の限界を押し広げる" §1.1, §2.3.1).
#include <algorithm>
#include <type_traits>

#include "cache_entry.cuh"
#include "common.cuh"
#include "elem.cuh"
#include "fp4_f16.cuh"

namespace csa2 {

constexpr int CA_WARPS = 8;

struct AppendArgs {
    uint8_t *lat_codes, *lat_scales, *ik_codes, *ik_scales;
    int capacity, ratio, d_idx;
    const uint16_t* rows;
    int n_rows;
    const int32_t* path;
    int n_path;
    const int64_t* pos0;
    const uint16_t* prev;
    uint16_t* prev_out;
    const float *w0, *w1;
    const uint8_t *wik_codes, *wik_scales;
    int per_warp;                // entries a warp takes
};

// how many of the first `upto` steps of a path are rows that exist, the block together
__device__ __forceinline__ int ca_length(const int32_t* path, int upto, int n_rows) {
    if (path == nullptr) return upto;
    for (int j0 = 0; j0 < upto; j0 += CA_WARPS * 32) {
        const int j = j0 + (int)threadIdx.x;
        const bool there = j < upto && (unsigned)path[j] < (unsigned)n_rows;
        const int n = __syncthreads_count(there);
        if (n == min(CA_WARPS * 32, upto - j0)) continue;
        // the first that is not there: a minimum over the block
        __shared__ int first;
        if (threadIdx.x == 0) first = upto;
        __syncthreads();
        if (!there) atomicMin(&first, min(j, upto));
        __syncthreads();
        return first;
    }
    return upto;
}

// One warp an entry, lane g owning channels 16g .. 16g+15, one scale group.  KEYS: the indexer keys are projected
// from the stored entry, W in shared memory as in k_cache_write_proj.
template <int DI>
__global__ void __launch_bounds__(CA_WARPS * 32) k_cache_append(const __grid_constant__ AppendArgs a) {
    extern __shared__ int smw[];
    constexpr int WS = 129;
    int* Wq = smw;                                   // [DI][WS] doubled E2M1 values, int8 x4
    int* Ws = Wq + DI * WS;                          // [DI][33] scales x 2^9
    int* Lq = Ws + DI * 33;                          // per warp: the entry's 128 words and 32 scales
    float* Kf = reinterpret_cast<float*>(Lq + CA_WARPS * 160);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
    pdl_wait();
    pdl_launch_next();
    const int64_t pos0 = a.pos0[b];
    const int odd = a.ratio == 2 ? (int)(pos0 & 1) : 0;
    const int64_t e0 = min(a.ratio == 2 ? (pos0 - odd) / 2 : pos0, (int64_t)a.capacity);
    const int32_t* path = a.path ? a.path + (int64_t)b * a.n_path : nullptr;
    const uint16_t* rows = a.rows + (int64_t)b * a.n_rows * D_LAT;
    const int i0 = blockIdx.x * CA_WARPS * a.per_warp;
    const int64_t last = (int64_t)(i0 + CA_WARPS * a.per_warp) * a.ratio;
    const int length = ca_length(path, blockIdx.x == 0 ? a.n_path : (int)min((int64_t)a.n_path, last), a.n_rows);
    if (DI > 0) {
        for (int i = tid; i < DI * 128; i += CA_WARPS * 32)
            Wq[(i >> 7) * WS + (i & 127)] =
                (int)unpack4_int8(reinterpret_cast<const uint16_t*>(a.wik_codes + (int64_t)(i >> 7) * (D_LAT / 2))[i & 127]);
        for (int i = tid; i < DI * 32; i += CA_WARPS * 32) Ws[(i >> 5) * 33 + (i & 31)] = cw_e4m3_x512(a.wik_scales[i]);
        __syncthreads();
    }
    auto row_of = [&](int j) { return rows + (int64_t)(path ? path[j] : j) * D_LAT + lane * 16; };
    for (int n = 0; n < a.per_warp; ++n) {
        const int i = i0 + warp + n * CA_WARPS;
        const int j = i * a.ratio - odd;                 // the row of the entry's first position; -1: the carried one
        const int64_t e = e0 + i;
        if (j + a.ratio - 1 >= length || e < 0 || e >= a.capacity) continue;         // warp-uniform
        const int64_t entry = (int64_t)b * a.capacity + e;
        float x[16];
        row16(j < 0 ? a.prev + (int64_t)b * D_LAT + lane * 16 : row_of(j), x);
        if (a.ratio == 2) {
            float y[16];
            row16(row_of(j + 1), y);
            merge16(x, y, a.w0 + lane * 16, a.w1 + lane * 16);
        }
        uint32_t q0, q1, sb;
        quant_group16(x, q0, q1, sb);
        reinterpret_cast<uint2*>(a.lat_codes + entry * (D_LAT / 2))[lane] = make_uint2(q0, q1);
        a.lat_scales[entry * (D_LAT / 16) + lane] = (uint8_t)sb;
        if constexpr (DI > 0) {
            int* Lw = Lq + warp * 160;
            float* Kw = Kf + warp * DI;
            Lw[4 * lane] = (int)unpack4_int8(q0 & 0xffffu);
            Lw[4 * lane + 1] = (int)unpack4_int8(q0 >> 16);
            Lw[4 * lane + 2] = (int)unpack4_int8(q1 & 0xffffu);
            Lw[4 * lane + 3] = (int)unpack4_int8(q1 >> 16);
            Lw[128 + lane] = cw_e4m3_x512(sb);
            __syncwarp();
#pragma unroll
            for (int t = 0; t < DI / 32; ++t) {
                const int d = lane + 32 * t;
                long long D = 0;
#pragma unroll 8
                for (int g = 0; g < 32; ++g) {
                    const int G4 = group_dot4(Wq + d * WS + 4 * g, reinterpret_cast<const uint32_t*>(Lw + 4 * g));
                    D += (long long)(G4 * Ws[d * 33 + g]) * Lw[128 + g];
                }
                Kw[d] = __ll2float_rn(D) * 0x1p-20f;        // one rounding; the power of two is exact
            }
            __syncwarp();
            if (lane < DI / 16) {
                float kx[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) kx[c] = Kw[16 * lane + c];
                quant_group16(kx, q0, q1, sb);
                reinterpret_cast<uint2*>(a.ik_codes + entry * (DI / 2))[lane] = make_uint2(q0, q1);
                a.ik_scales[entry * (DI / 16) + lane] = (uint8_t)sb;
            }
            __syncwarp();
        }
    }
    if (blockIdx.x == 0 && a.prev_out != nullptr) {
        __syncthreads();                                 // prev_out may be prev: its last reader is this block
        const uint4* src = reinterpret_cast<const uint4*>(
            length > 0 ? rows + (int64_t)(path ? path[length - 1] : length - 1) * D_LAT : a.prev + (int64_t)b * D_LAT);
        if (tid < D_LAT / 8) reinterpret_cast<uint4*>(a.prev_out + (int64_t)b * D_LAT)[tid] = src[tid];
    }
}

// Entries as values: eight a thread (one 4-byte word of codes, its group's scale), exact in every output type: an E2M1
// value times an E4M3 scale has at most 6 significant bits and lies in [2^-10, 2688].
template <typename TO>
__global__ void __launch_bounds__(256) k_cache_read(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                    int capacity, int d, const int32_t* __restrict__ idx, int64_t first,
                                                    int64_t n, int64_t total, TO* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    const int per_row = d / 8;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        const int64_t row = u / per_row;
        const int c = (int)(u - row * per_row);
        const int64_t b = row / n;
        const int64_t e = idx ? (int64_t)idx[row] : first + (row - b * n);
        uint32_t w = 0u, s = 0u;
        if (e >= 0 && e < capacity) {
            const int64_t at = b * capacity + e;
            w = reinterpret_cast<const uint32_t*>(codes + at * (d / 2))[c];
            s = scales[at * (d / 16) + (c >> 1)];
        }
        __half2 h[4];
        e2m1x8_to_f16x8(w, h);
        const __half2 s2 = __half2half2(__low2half(e4m3x2_to_f16x2(s)));
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(__hmul2(h[i], s2));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
        ElemVec<TO, 8> y;
        y.pack(v);
        y.store(out + row * d + 8 * c);
    }
}

cudaError_t launch_cache_append(const csa2_cache& c, const uint16_t* rows, int n_rows, const int32_t* path, int n_path,
                                const int64_t* pos0, const uint16_t* prev, uint16_t* prev_out, const float* w0,
                                const float* w1, const uint8_t* wik_codes, const uint8_t* wik_scales, cudaStream_t st) {
    const int n_ent = c.ratio == 2 ? n_path / 2 + (n_path & 1) : n_path;
    const bool carry = c.ratio == 2 && prev_out != nullptr;
    if (n_ent == 0 && (!carry || prev_out == prev)) return cudaSuccess;
    const int di = wik_codes ? c.d_idx : 0;
    AppendArgs a{c.lat_codes, c.lat_scales, c.ikey_codes, c.ikey_scales, c.capacity, c.ratio, c.d_idx, rows, n_rows, path, n_path,
                 pos0, prev, carry ? prev_out : nullptr, w0, w1, wik_codes, wik_scales, n_ent > 64 ? 8 : 1};
    const auto kern = di == 128 ? k_cache_append<128> : di == 64 ? k_cache_append<64> : k_cache_append<0>;
    const size_t smem = di ? ((size_t)di * (129 + 33) + CA_WARPS * 160 + CA_WARPS * di) * sizeof(int) : 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int per = CA_WARPS * a.per_warp;
    e = launch_k(kern, dim3((unsigned)std::max(1, (n_ent - 1) / per + 1), c.batch), CA_WARPS * 32, smem, st, a);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_read(const csa2_cache& c, bool keys, const int32_t* idx, int64_t first, int64_t n, void* out,
                              int out_type, cudaStream_t st) {
    const int d = keys ? c.d_idx : D_LAT;
    const int64_t total = (int64_t)c.batch * n * (d / 8);
    const uint8_t *codes = keys ? c.ikey_codes : c.lat_codes, *scales = keys ? c.ikey_scales : c.lat_scales;
    const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 152 * 64);
    auto go = [&](auto* y) {
        using TO = std::remove_pointer_t<decltype(y)>;
        launch_k(k_cache_read<TO>, dim3(grid), 256, 0, st, codes, scales, (int)c.capacity, d, idx, first, n, total, y);
    };
    if (out_type == CSA2_F32)
        go(reinterpret_cast<float*>(out));
    else if (out_type == CSA2_F16)
        go(reinterpret_cast<__half*>(out));
    else
        go(reinterpret_cast<__nv_bfloat16*>(out));
    note_launch();
    return cudaGetLastError();
}

}  // namespace csa2
