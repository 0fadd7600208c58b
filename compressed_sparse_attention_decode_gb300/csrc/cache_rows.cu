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
#include "tree.cuh"

namespace csa2 {

struct AppendArgs {
    uint8_t *lat_codes, *lat_scales, *ik_codes, *ik_scales;
    int capacity, ratio;
    const uint16_t* rows;
    int n_rows;
    const int32_t* path;
    int n_path, n_ent;           // entries of a sequence at most
    const int64_t* pos0;
    const uint16_t* prev;
    uint16_t* prev_out;
    const float *w0, *w1;
    const uint8_t *wik_codes, *wik_scales;
};

// Sequence b of a call
struct AppendSeq {
    int64_t e0;                  // the entry of the first position, outside the cache where that is
    int odd;                     // the first position completes a pair
    const int32_t* path;
    const uint16_t* rows;
    __device__ __forceinline__ AppendSeq(const AppendArgs& a, int b) {
        const int64_t pos0 = a.pos0[b];
        odd = a.ratio == 2 ? (int)(pos0 & 1) : 0;
        e0 = min(a.ratio == 2 ? (pos0 - odd) / 2 : pos0, (int64_t)a.capacity);
        path = a.path ? a.path + (int64_t)b * a.n_path : nullptr;
        rows = a.rows + (int64_t)b * a.n_rows * D_LAT;
    }
    // how many of the path's first `upto` steps are rows that exist, a whole warp together
    __device__ __forceinline__ int length(const AppendArgs& a, int upto) const {
        if (path == nullptr) return upto;
        const int lane = threadIdx.x & 31;
        for (int j0 = 0; j0 < upto; j0 += 32) {
            const unsigned there = __ballot_sync(0xffffffffu, j0 + lane < upto && (unsigned)path[j0 + lane] < (unsigned)a.n_rows);
            if (there != 0xffffffffu) return min(upto, j0 + __ffs(~there) - 1);
        }
        return upto;
    }
    __device__ __forceinline__ const uint16_t* row(int j) const { return rows + (int64_t)(path ? path[j] : j) * D_LAT; }
    // the entry's 16 channels of this lane's group, quantised; its first row is step j (-1: the carried row)
    __device__ __forceinline__ void entry(const AppendArgs& a, int b, int j, uint32_t& q0, uint32_t& q1, uint32_t& sb) const {
        const int at = (threadIdx.x & 31) * 16;
        float x[16];
        row16((j < 0 ? a.prev + (int64_t)b * D_LAT : row(j)) + at, x);
        if (a.ratio == 2) {
            float y[16];
            row16(row(j + 1) + at, y);
            merge16(x, y, a.w0 + at, a.w1 + at);
        }
        quant_group16(x, q0, q1, sb);
    }
};
__device__ __forceinline__ void store_latent(const AppendArgs& a, int64_t entry, uint32_t q0, uint32_t q1, uint32_t sb) {
    const int lane = threadIdx.x & 31;
    reinterpret_cast<uint2*>(a.lat_codes + entry * (D_LAT / 2))[lane] = make_uint2(q0, q1);
    a.lat_scales[entry * (D_LAT / 16) + lane] = (uint8_t)sb;
}
// the row of the path's last position, or the carried one, to prev_out (which may be prev: whoever reads it is done)
__device__ __forceinline__ void carry_on(const AppendArgs& a, const AppendSeq& s, int b, int length) {
    const int lane = threadIdx.x & 31;
    const uint4* src = reinterpret_cast<const uint4*>(length > 0 ? s.row(length - 1) : a.prev + (int64_t)b * D_LAT);
    uint4* dst = reinterpret_cast<uint4*>(a.prev_out + (int64_t)b * D_LAT);
    const uint4 x = src[lane], y = src[32 + lane];
    dst[lane] = x, dst[32 + lane] = y;
}

// Few entries, or no indexer keys.  DI = 0: a warp an entry.  Else a block an entry and a warp a group of 16 key dims (it
// makes the entry for itself: nothing is handed from warp to warp): lane g multiplies latent group g with 16 rows of W,
// exactly (k_cache_write_proj has the bounds), the 16 sums over the lanes are halved in turn, and the group is quantised.
// What bounds it are five loads in a row, position, path, rows, weights' products, stores: 64 entries of 128 keys take 3.6 us.
template <int DI>
__global__ void __launch_bounds__(256) k_cache_append(const __grid_constant__ AppendArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
    pdl_wait();
    pdl_launch_next();
    const AppendSeq s(a, b);
    const int i = DI > 0 ? (int)blockIdx.x : (int)blockIdx.x * 8 + warp;
    const int j = i * a.ratio - s.odd;                   // the step of the entry's first position; -1: the carried row
    const bool first = blockIdx.x == 0 && warp == 0 && a.prev_out != nullptr;
    const int length = s.length(a, first ? a.n_path : min(a.n_path, j + a.ratio));
    const int64_t e = s.e0 + i;
    const bool there = i < a.n_ent && j + a.ratio <= length && e >= 0 && e < a.capacity;
    uint2 wc[16];
    uint32_t wsc[16], q0 = 0u, q1 = 0u, sb = 0u;
    if constexpr (DI > 0) {
        if (there)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int64_t d = warp * 16 + k;
                wc[k] = reinterpret_cast<const uint2*>(a.wik_codes + d * (D_LAT / 2))[lane];
                wsc[k] = a.wik_scales[d * (D_LAT / 16) + lane];
            }
    }
    if (there) s.entry(a, b, j, q0, q1, sb);
    if (DI > 0 && blockIdx.x == 0) __syncthreads();      // every warp (every lane) has read the carried row
    __syncwarp();
    if (first) carry_on(a, s, b, length);
    if (!there) return;
    const int64_t entry = (int64_t)b * a.capacity + e;
    if (DI == 0 || warp == 0) store_latent(a, entry, q0, q1, sb);
    if constexpr (DI > 0) {
        const uint32_t L[4] = {unpack4_int8(q0 & 0xffffu), unpack4_int8(q0 >> 16), unpack4_int8(q1 & 0xffffu), unpack4_int8(q1 >> 16)};
        const int sl = cw_e4m3_x512(sb);
        long long t[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int w[4] = {(int)unpack4_int8(wc[k].x & 0xffffu), (int)unpack4_int8(wc[k].x >> 16),
                              (int)unpack4_int8(wc[k].y & 0xffffu), (int)unpack4_int8(wc[k].y >> 16)};
            t[k] = (long long)(group_dot4(w, L) * cw_e4m3_x512(wsc[k])) * sl;
        }
        // sums over the lanes: each step a lane keeps half of the dims, and has dim lane / 2 in the end
        const auto halve = [&](auto left, int o) {
            constexpr int n = decltype(left)::value;
            const bool up = lane & o;
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const long long give = up ? t[k] : t[k + n], keep = up ? t[k + n] : t[k];
                t[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        };
        halve(std::integral_constant<int, 8>{}, 16);
        halve(std::integral_constant<int, 4>{}, 8);
        halve(std::integral_constant<int, 2>{}, 4);
        halve(std::integral_constant<int, 1>{}, 2);
        t[0] += __shfl_xor_sync(0xffffffffu, t[0], 1);
        const float mine = __ll2float_rn(t[0]) * 0x1p-20f;       // one rounding; the power of two is exact
        float kx[16];
#pragma unroll
        for (int d = 0; d < 16; ++d) kx[d] = __shfl_sync(0xffffffffu, mine, 2 * d);
        quant_group16(kx, q0, q1, sb);
        if (lane == 0) {
            *reinterpret_cast<uint2*>(a.ik_codes + entry * (DI / 2) + warp * 8) = make_uint2(q0, q1);
            a.ik_scales[entry * (DI / 16) + warp] = (uint8_t)sb;
        }
    }
}

// Many entries with their indexer keys.  A key is sum_g G_g sL_g sW_g over 32 groups; G, sixteen products of E2M1 values, has 12
// bits in quarters, the scales 4 each, so that a group's term has 20 bits and comes exactly out of one m16n8k16 product of the
// scaled values (fp16 holds them exactly).  The sum has to be exact too, over 53 bits.  It is held in three fp32 sums: the
// first two start at 1.5 x 2^33 and 1.5 x 2^15 and are never more than 2^32 and 2^14 away from there, so that their last bits
// stay 2^10 and 2^-8; adding a term to the first leaves a remainder (exact, at most 2^9), which is added to the second; its
// remainder (at most 2^-9, a multiple of 2^-20) goes into the third.  Seven additions a term, no 64-bit arithmetic.  The
// products bound the kernel: an SM's quarter takes an m16n8k16 every 32 clocks or so, and the additions some of what is left
// (4 x 4,096 entries of 128 keys: 48 us; int8 products and 64-bit sums took 105).
// W is expanded to shared memory once a block, in the products' order.  Sixteen warps quantise a tile of 32 entries (two each,
// whose rows they have asked for a tile ahead) while the other sixteen multiply the tile before; one of those has 16 entries
// and a key group of 16 dims, which it quantises from its sums (all warps doing one after the other: 60 us).
constexpr int CM_TILE = 32, CM_MAKERS = 16, CM_THREADS = 1024;
constexpr int CM_A = CM_TILE * 1024, CM_RAW = CM_MAKERS * 2048;      // bytes of a tile's entries (fp16), of the rows under way

__device__ __forceinline__ void mma16816(float* d, const uint32_t* x, uint32_t y0, uint32_t y1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(y0), "r"(y1), "f"(0.0f));
}
// two codes of a byte (low nibble first) times the scale
__device__ __forceinline__ uint32_t pair_scaled(uint32_t byte, __half2 s) {
    uint32_t r;
    asm("{\n .reg .b8 x, y, z, w;\n mov.b32 {x, y, z, w}, %1;\n cvt.rn.f16x2.e2m1x2 %0, x;\n}" : "=r"(r) : "r"(byte));
    const __half2 v = __hmul2(*reinterpret_cast<__half2*>(&r), s);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int DI>
__global__ void __launch_bounds__(CM_THREADS, 1) k_cache_append_many(const __grid_constant__ AppendArgs a, int tiles, int batch) {
    extern __shared__ __align__(16) uint8_t A[];             // two tiles: entries x 512 fp16, 16-byte pieces at p ^ (entry & 7)
    uint2* W = reinterpret_cast<uint2*>(A + 2 * CM_A + CM_RAW);      // [DI / 8][32 groups][32 lanes] the products' B
    __shared__ int64_t entry_at[2][CM_TILE];                 // -1: not there
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, all = tiles * batch;
    pdl_wait();
    pdl_launch_next();
    // B of a group: rows 2 (lane % 4) + {0, 1} and 8 further, column lane / 4: bytes lane % 4 and 4 + lane % 4 of the dim's eight
#pragma unroll 4
    for (int u = warp; u < DI / 8 * 32; u += CM_THREADS / 32) {
        const int64_t d = (u >> 5) * 8 + (lane >> 2);
        const int g = u & 31;
        const uint2 c = reinterpret_cast<const uint2*>(a.wik_codes + d * (D_LAT / 2))[g];
        // (the scale as the exact integers take it)
        const __half2 s = __float2half2_rn((float)cw_e4m3_x512(a.wik_scales[d * (D_LAT / 16) + g]) * 0x1p-9f);
        W[u * 32 + lane] = make_uint2(pair_scaled(c.x >> (8 * (lane & 3)), s), pair_scaled(c.y >> (8 * (lane & 3)), s));
    }
    __syncthreads();
    // named barriers: 1 + buf the tile in buffer buf is made, 3 + buf it is read
    if (warp < CM_MAKERS) {
        // ================= entries: warp w makes entries w and 16 + w of a tile, lane g its channel group g
        uint8_t* raw = A + 2 * CM_A + warp * 2048;
        int64_t entry = -1;
        int length = 0;
        auto fetch = [&](int tile, int r) {                  // entry r's rows, if it is there
            const int b = tile / tiles, i = (tile - b * tiles) * CM_TILE + r;
            const AppendSeq s(a, b);
            const int j = i * a.ratio - s.odd;
            length = s.length(a, i == 0 && a.prev_out != nullptr ? a.n_path : min(a.n_path, j + a.ratio));
            const int64_t e = s.e0 + i;
            const bool there = i < a.n_ent && j + a.ratio <= length && e >= 0 && e < a.capacity;
            entry = there ? (int64_t)b * a.capacity + e : -1;
            if (there)
                for (int k = 0; k < a.ratio; ++k) {
                    const uint16_t* src = j + k < 0 ? a.prev + (int64_t)b * D_LAT : s.row(j + k);
                    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(raw + k * 1024);
                    copy16(dst + lane * 16, src + lane * 8, true);
                    copy16(dst + (32 + lane) * 16, src + (32 + lane) * 8, true);
                }
        };
        if ((int)blockIdx.x < all) fetch(blockIdx.x, warp);
        int n = 0;
        for (int tile = blockIdx.x; tile < all; tile += gridDim.x, ++n) {
            const int buf = n & 1;
            if (n >= 2) asm volatile("bar.sync %0, %1;" ::"r"(3 + buf), "r"(CM_THREADS) : "memory");
#pragma unroll 1
            for (int r = warp; r < CM_TILE; r += CM_MAKERS) {
                copy16_wait();
                __syncwarp();
                const int b = tile / tiles;
                if (r == 0 && tile == b * tiles && a.prev_out != nullptr) carry_on(a, AppendSeq(a, b), b, length);     // (it is here)
                const int64_t at = entry;
                float x[16], y[16];
                auto take = [&](int k, float* v) {           // 32 bytes of a row
                    const uint4* p = reinterpret_cast<const uint4*>(raw + k * 1024) + 2 * lane;
                    const uint4 c = p[0], d = p[1];
                    const uint32_t w[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = bf16_bits_to_f32((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xffffu));
                };
                if (at >= 0) {
                    take(0, x);
                    if (a.ratio == 2) take(1, y);
                }
                __syncwarp();
                if (r + CM_MAKERS < CM_TILE)
                    fetch(tile, r + CM_MAKERS);
                else if (tile + (int)gridDim.x < all)
                    fetch(tile + gridDim.x, warp);
                uint32_t q0 = 0u, q1 = 0u, sb = 0u;
                if (at >= 0) {
                    if (a.ratio == 2) merge16(x, y, a.w0 + lane * 16, a.w1 + lane * 16);
                    quant_group16(x, q0, q1, sb);
                    store_latent(a, at, q0, q1, sb);
                }
                const __half2 sc = __half2half2(__low2half(e4m3x2_to_f16x2(sb)));
                uint8_t* row = A + buf * CM_A + r * 1024;
                *reinterpret_cast<uint4*>(row + (((2 * lane) ^ (r & 7)) << 4)) = e2m1x8_scaled(q0, sc);
                *reinterpret_cast<uint4*>(row + (((2 * lane + 1) ^ (r & 7)) << 4)) = e2m1x8_scaled(q1, sc);
                if (lane == 0) entry_at[buf][r] = at;
            }
            __threadfence_block();
            asm volatile("bar.arrive %0, %1;" ::"r"(1 + buf), "r"(CM_THREADS) : "memory");
        }
    } else {
        // ================= products: warp w has entries 16 (w % 2) .. + 15 and key group w / 2 (with 64 dims half of the warps
        // have none)
        const int w = warp - CM_MAKERS, m = w & 1, group = w >> 1;
        const bool busy = group < DI / 16;
        const uint32_t abase = (uint32_t)__cvta_generic_to_shared(A);
        const uint2* B = W + group * 2048 + lane;
        int n = 0;
        for (int tile = blockIdx.x; tile < all; tile += gridDim.x, ++n) {
            const int buf = n & 1;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + buf), "r"(CM_THREADS) : "memory");
            float key[2][4];                                 // rows lane / 4 and 8 further, dims 8 h + 2 (lane % 4) + {0, 1}
            int64_t at[2] = {-1, -1};
            if (busy) {
                const int r = m * 16 + (lane & 15);
                at[0] = entry_at[buf][m * 16 + (lane >> 2)], at[1] = entry_at[buf][m * 16 + 8 + (lane >> 2)];
                float s1[2][4], s2[2][4], s3[2][4];
#pragma unroll
                for (int v = 0; v < 8; ++v) s1[v >> 2][v & 3] = 0x1.8p33f, s2[v >> 2][v & 3] = 0x1.8p15f, s3[v >> 2][v & 3] = 0.0f;
#pragma unroll 2
                for (int g = 0; g < 32; ++g) {
                    uint32_t x[4];
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                 : "r"(abase + buf * CM_A + r * 1024 + (((2 * g + (lane >> 4)) ^ (r & 7)) << 4)));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 y = B[h * 1024 + g * 32];
                        float t[4];
                        mma16816(t, x, y.x, y.y);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float n1 = __fadd_rn(s1[h][v], t[v]), r1 = __fsub_rn(t[v], __fsub_rn(n1, s1[h][v]));
                            const float n2 = __fadd_rn(s2[h][v], r1), r2 = __fsub_rn(r1, __fsub_rn(n2, s2[h][v]));
                            s1[h][v] = n1, s2[h][v] = n2, s3[h][v] = __fadd_rn(s3[h][v], r2);
                        }
                    }
                }
#pragma unroll
                for (int v = 0; v < 8; ++v) {                // the three as one number of 2^-20: exact, then one rounding
                    const int h = v >> 2, c = v & 3;
                    const long long sum = ((long long)__float2int_rn(__fsub_rn(s1[h][c], 0x1.8p33f) * 0x1p-10f) << 30) +
                                          ((long long)__float2int_rn(__fsub_rn(s2[h][c], 0x1.8p15f) * 0x1p8f) << 12) +
                                          __float2int_rn(s3[h][c] * 0x1p20f);
                    key[h][c] = __ll2float_rn(sum) * 0x1p-20f;
                }
            }
            if (tile + 2 * (int)gridDim.x < all) {
                __threadfence_block();
                asm volatile("bar.arrive %0, %1;" ::"r"(3 + buf), "r"(CM_THREADS) : "memory");
            }
            // a row's group lies in four lanes, four values each
            if (busy)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v[4] = {key[0][2 * i], key[0][2 * i + 1], key[1][2 * i], key[1][2 * i + 1]};
                    float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const uint32_t sb = f32_to_e4m3_satfinite(__fdiv_rn(top, 6.0f));
                    const float s = e4m3_to_f32(sb);
                    uint32_t c[2] = {0u, 0u};
                    if (s > 0.0f)
#pragma unroll
                        for (int h = 0; h < 2; ++h) c[h] = e2m1_code(v[2 * h], s) | (e2m1_code(v[2 * h + 1], s) << 4);
                    if (at[i] >= 0) {
                        uint8_t* codes = a.ik_codes + at[i] * (DI / 2) + group * 8 + (lane & 3);
                        codes[0] = (uint8_t)c[0], codes[4] = (uint8_t)c[1];
                        if ((lane & 3) == 0) a.ik_scales[at[i] * (DI / 16) + group] = (uint8_t)sb;
                    }
                }
        }
    }
}

// Entries as values: a unit is eight of them (one 4-byte word of codes, its group's scale), exact in every output type: an
// E2M1 value times an E4M3 scale has at most 6 significant bits and lies in [2^-10, 2688].  HBM bounds it, with eight units of a
// thread asked for at once (8 x 65,536 latents in fp16: 101 us, 6.8 TB/s; with one 152 us); a call that one unit a thread of
// all SMs holds has one, which is 2 us shorter.
template <typename TO, int CR_UNITS>
__global__ void __launch_bounds__(256) k_cache_read(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                    int capacity, int shift, int batch, const int32_t* __restrict__ idx, int64_t first,
                                                    int64_t n, TO* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    const int d = 8 << shift;
    const int64_t units = n << shift, u0 = (int64_t)blockIdx.x * (256 * CR_UNITS) + threadIdx.x;
    for (int b = blockIdx.y; b < batch; b += gridDim.y) {
        int64_t at[CR_UNITS];
        uint32_t w[CR_UNITS], s[CR_UNITS];
#pragma unroll
        for (int i = 0; i < CR_UNITS; ++i) {
            const int64_t u = u0 + i * 256, row = u >> shift;
            at[i] = -1;
            if (u < units) {
                const int64_t e = idx ? (int64_t)idx[b * n + row] : first + row;
                if (e >= 0 && e < capacity) at[i] = (int64_t)b * capacity + e;
            }
        }
#pragma unroll
        for (int i = 0; i < CR_UNITS; ++i) {
            const int c = (int)((u0 + i * 256) & ((1 << shift) - 1));
            w[i] = s[i] = 0u;
            if (at[i] >= 0) {
                w[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + at[i] * (d / 2)) + c);
                s[i] = __ldg(scales + at[i] * (d / 16) + (c >> 1));
            }
        }
#pragma unroll
        for (int i = 0; i < CR_UNITS; ++i) {
            const int64_t u = u0 + i * 256;
            if (u >= units) break;
            __half2 h[4];
            e2m1x8_to_f16x8(w[i], h);
            const __half2 s2 = __half2half2(__low2half(e4m3x2_to_f16x2(s[i])));
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(__hmul2(h[k], s2));
                v[2 * k] = f.x, v[2 * k + 1] = f.y;
            }
            ElemVec<TO, 8> y;
            y.pack(v);
            y.store(out + (b * units + u) * 8);
        }
    }
}

// Entries of a call from which on the tensor cores make their keys (512 entries: 12 us without them, 14 with them; 1,024:
// 22 and 15)
constexpr int64_t CA_MANY = 768;

cudaError_t launch_cache_append(const csa2_cache& c, const uint16_t* rows, int n_rows, const int32_t* path, int n_path,
                                const int64_t* pos0, const uint16_t* prev, uint16_t* prev_out, const float* w0,
                                const float* w1, const uint8_t* wik_codes, const uint8_t* wik_scales, cudaStream_t st) {
    const int n_ent = c.ratio == 2 ? n_path / 2 + (n_path & 1) : n_path;
    const bool carry = c.ratio == 2 && prev_out != nullptr;
    if (n_ent == 0 && (!carry || prev_out == prev)) return cudaSuccess;
    const int di = wik_codes ? c.d_idx : 0;
    const AppendArgs a{c.lat_codes, c.lat_scales, c.ikey_codes, c.ikey_scales, c.capacity, c.ratio, rows, n_rows, path, n_path, n_ent,
                       pos0, prev, carry ? prev_out : nullptr, w0, w1, wik_codes, wik_scales};
    if (di > 0 && (int64_t)n_ent * c.batch >= CA_MANY) {
        const int tiles = (n_ent - 1) / CM_TILE + 1;
        const unsigned grid = (unsigned)std::min<int64_t>((int64_t)tiles * c.batch, 152);
        const auto kern = di == 128 ? k_cache_append_many<128> : k_cache_append_many<64>;
        const int smem = 2 * CM_A + CM_RAW + di * 1024;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        launch_k(kern, dim3(grid), CM_THREADS, (size_t)smem, st, a, tiles, (int)c.batch);
    } else if (di > 0) {
        launch_k(di == 128 ? k_cache_append<128> : k_cache_append<64>, dim3((unsigned)std::max(1, n_ent), c.batch), di * 2, 0, st, a);
    } else {
        launch_k(k_cache_append<0>, dim3((unsigned)std::max(1, (n_ent + 7) / 8), c.batch), 256, 0, st, a);
    }
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const csa2_cache& c, bool keys, const int32_t* idx, int64_t first, int64_t n, void* out,
                              int out_type, cudaStream_t st) {
    const int shift = keys ? (c.d_idx == 128 ? 4 : 3) : 6;           // units of a row: 2^shift
    const uint8_t *codes = keys ? c.ikey_codes : c.lat_codes, *scales = keys ? c.ikey_scales : c.lat_scales;
    const bool few = ((n << shift) * c.batch) <= 152 * 2048;
    const int64_t per = 256 * (few ? 1 : 8), blocks = ((n << shift) + per - 1) / per;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)std::min(c.batch, 65535));
    auto go = [&](auto* y) {
        using TO = std::remove_pointer_t<decltype(y)>;
        launch_k(few ? k_cache_read<TO, 1> : k_cache_read<TO, 8>, grid, 256, 0, st, codes, scales, (int)c.capacity, shift, (int)c.batch,
                 idx, first, n, y);
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
