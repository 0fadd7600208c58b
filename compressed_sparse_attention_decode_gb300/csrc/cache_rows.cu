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
#include "umma.cuh"

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
    // how many of the path's first `upto` steps are rows that exist, its first `from` being known to be; a whole warp together
    __device__ __forceinline__ int length(const AppendArgs& a, int upto, int from = 0) const {
        if (path == nullptr) return upto;
        const int lane = threadIdx.x & 31;
        for (int j0 = from & ~31; j0 < upto; j0 += 128) {
            unsigned there[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {                    // (four loads under way: 8,192 steps are 64 times their latency)
                const int j = j0 + 32 * k + lane;
                there[k] = __ballot_sync(0xffffffffu, j < upto && (unsigned)path[j] < (unsigned)a.n_rows);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (there[k] != 0xffffffffu) return min(upto, j0 + 32 * k + __ffs(~there[k]) - 1);
        }
        return upto;
    }
    // the step of entry i's first position; -1: the carried row
    __device__ __forceinline__ int step(const AppendArgs& a, int i) const { return i * a.ratio - odd; }
    // where in the cache's planes entry i of the path's goes, -1 where it is not complete within `length` steps or not inside
    __device__ __forceinline__ int64_t place(const AppendArgs& a, int b, int i, int length) const {
        const int64_t e = e0 + i;
        return i < a.n_ent && step(a, i) + a.ratio <= length && e >= 0 && e < a.capacity ? (int64_t)b * a.capacity + e : -1;
    }
    __device__ __forceinline__ const uint16_t* row(int j) const { return rows + (int64_t)(path ? path[j] : j) * D_LAT; }
    // the entry's 16 channels of this lane's group, quantised; its first row is step j (-1: the carried row)
    __device__ __forceinline__ void entry(const AppendArgs& a, int b, int j, uint32_t& q0, uint32_t& q1, uint32_t& sb) const {
        const int at = (threadIdx.x & 31) * 16;
        float x[16];
        // (plain loads: the carried row may be written by this kernel)
        const uint4* src = reinterpret_cast<const uint4*>((j < 0 ? a.prev + (int64_t)b * D_LAT : row(j)) + at);
        const uint4 c0 = src[0], c1 = src[1];
        if (a.ratio == 2) {
            src = reinterpret_cast<const uint4*>(row(j + 1) + at);
            const uint4 d0 = src[0], d1 = src[1];
            float y[16];
            bf16x16_to_f32(c0, c1, x);
            bf16x16_to_f32(d0, d1, y);
            merge16(x, y, a.w0 + at, a.w1 + at);
        } else {
            bf16x16_to_f32(c0, c1, x);
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
    const int j = s.step(a, i);
    const bool first = blockIdx.x == 0 && warp == 0 && a.prev_out != nullptr;
    const int length = s.length(a, first ? a.n_path : min(a.n_path, j + a.ratio));
    const int64_t entry = s.place(a, b, i, length);
    const bool there = entry >= 0;
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

// Many entries with their indexer keys.  A key is the exact sum of W . L over 512 dims, rounded once and quantised: what is
// kept of it is a scale byte of 16 dims and four bits each.  So the tensor cores sum in fp32, in eight accumulators of 64 dims,
// which err by no more than CM_ERR |W_d| |L| together (no product and no partial sum is larger than its part's two norms'
// product, and these add up to no more than the whole's; four steps of 17 terms, each cut at 2^-24 of that or better, as
// measured (2^-26; it is not documented), and seven additions: 75 x 2^-24, held as 80).  Where both ends of that interval have the same scale and code, those are the
// exact sum's; the others, one in a thousand of random rows, are summed again exactly: a term of 16 dims, sixteen
// products of E2M1 values times two scales, has 20 bits and comes exactly out of fp32 additions, and the 32 terms go into 64 bits.
// W is expanded to shared memory once a block, 128 dims x 512 in fp16 (with 64 dims the other half is zeros).  A tile is 16
// entries: sixteen warps make one each (its rows are asked for a tile ahead, and the entry kept as it is stored, in fp16), two
// warps issue half of its sixteen-dim steps each (one thread issues a product per 65 to 85 clocks, whatever its size), and two
// sets of four warps take the sums of every second tile: TMEM lane = key dim, turned in shared memory so that a thread
// has an entry's group of 16 dims.  Merging, quantising and expanding are 57 % of all issue slots, and no unit is full: 4 x 4,096 entries of 128
// keys take 38 us, 10 of them start and end (in one accumulator 62, half of it exact sums; exact terms of 16 dims added up in
// fp32, by mma.sync, 58).
constexpr int CM_TILE = 16, CM_MAKERS = 16, CM_MMA = 16, CM_OUT = 18, CM_THREADS = 26 * 32;
constexpr int CM_BUFS = 4;
constexpr uint32_t CM_W = 128 * 1024, CM_A = CM_TILE * 1024, CM_TURN = CM_TILE * 36 * 4;     // W, a tile, a warp's sums
constexpr uint32_t CM_DYN = CM_W + CM_BUFS * CM_A + 8 * CM_TURN + 4096 + 1024;                 // + w0 and w1, alignment
constexpr float CM_ERR = 0x1.4p-18f;

// where entry e (0 .. 15, of each lane) of a tile goes, found out anew; a whole warp together
__device__ __noinline__ int64_t cm_place(const AppendArgs& a, int tile, int tiles, int e) {
    const int b = tile / tiles, i = (tile - b * tiles) * CM_TILE + e;
    const AppendSeq s(a, b);
    return s.place(a, b, i, s.length(a, a.n_path));
}

// sixteen fp16 values of a row of a 128-byte swizzled slab (rows of 64)
__device__ __forceinline__ void cm_row16(const uint8_t* slab, int row, int g, uint4* v) {
    const uint8_t* at = slab + row * 128;
    v[0] = *reinterpret_cast<const uint4*>(at + (((2 * (g & 3)) ^ (row & 7)) << 4));
    v[1] = *reinterpret_cast<const uint4*>(at + (((2 * (g & 3) + 1) ^ (row & 7)) << 4));
}

template <int DI>
__global__ void __launch_bounds__(CM_THREADS, 1) k_cache_append_many(const __grid_constant__ AppendArgs a, int tiles, int batch) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) unsigned long long b_w, b_full[CM_BUFS], b_free[CM_BUFS], b_sum[2], b_taken[2];
    __shared__ int64_t entry_at[CM_BUFS][CM_TILE];           // -1: not there
    __shared__ float norm_l[CM_BUFS][CM_TILE], norm_w[128];
    __shared__ uint32_t tmem_base;
    const uint32_t raw0 = umma::smem_u32(dyn), base = (raw0 + 1023u) & ~1023u;
    uint8_t* W = dyn + (base - raw0);                        // 8 slabs of 128 rows x 64 dims
    uint8_t* A = W + CM_W;                                   // buffers of 8 slabs of 16 rows x 64 dims
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, all = tiles * batch;
    auto sa = [&](const void* x) { return umma::smem_u32(x); };
    if (tid == 0) {
        umma::mbar_init(sa(&b_w), CM_THREADS / 32 - CM_MAKERS);
        for (int i = 0; i < CM_BUFS; ++i) umma::mbar_init(sa(&b_full[i]), CM_MAKERS), umma::mbar_init(sa(&b_free[i]), 4);
        for (int i = 0; i < 2; ++i) umma::mbar_init(sa(&b_sum[i]), 2), umma::mbar_init(sa(&b_taken[i]), 4);
        umma::fence_mbar_init();
    }
    if (warp == CM_MMA) umma::tmem_alloc(sa(&tmem_base), 256);
    float4* merge = reinterpret_cast<float4*>(A + CM_BUFS * CM_A + 8 * CM_TURN);     // [w0, w1][4][32 lanes] four of a lane's 16 dims
    pdl_wait();
    pdl_launch_next();
    if (a.ratio == 2 && tid < 256)
        merge[(tid & 128) + ((tid & 3) << 5) + ((tid & 127) >> 2)] = reinterpret_cast<const float4*>(tid < 128 ? a.w0 : a.w1)[tid & 127];
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    if (warp < CM_MAKERS) {
        // ================= entries: a warp makes one of a tile, lane g its channel group g
        // Two tiles ahead where its rows are, and a request for them to L2; one tile ahead the rows.
        struct Place {
            int64_t entry;                                   // -1: not there
            const uint4 *x, *y;
            int length;
        };
        int fb = (int)blockIdx.x / tiles, ft = (int)blockIdx.x - fb * tiles;         // the tile that is found next
        int seen_b = -1, seen = 0;
        bool ends = false;
        auto find = [&]() {
            Place p{-1, nullptr, nullptr, 0};
            if (fb >= batch) return p;
            const int b = fb, i = ft * CM_TILE + warp;
            for (ft += gridDim.x; ft >= tiles && fb < batch; ft -= tiles) ++fb;
            const AppendSeq s(a, b);
            const int j = s.step(a, i);
            // (of a path that it goes along the warp looks at each step once)
            const int upto = i == 0 && a.prev_out != nullptr ? a.n_path : min(a.n_path, j + a.ratio);
            if (b != seen_b) seen_b = b, seen = 0, ends = false;
            if (!ends && seen < upto) seen = s.length(a, upto, seen), ends = seen < upto;
            p.length = min(seen, upto);
            p.entry = s.place(a, b, i, p.length);
            if (p.entry >= 0) {
                p.x = reinterpret_cast<const uint4*>(j < 0 ? a.prev + (int64_t)b * D_LAT : s.row(j));
                p.y = a.ratio == 2 ? reinterpret_cast<const uint4*>(s.row(j + 1)) : p.x;
                if (lane < 16) umma::prefetch_l2((lane & 8 ? p.y : p.x) + 8 * (lane & 7));      // (lines of 128 bytes)
            }
            return p;
        };
        uint4 raw[4];
        auto fetch = [&](const Place& p) {
            if (p.entry < 0) return;
            raw[0] = p.x[2 * lane], raw[1] = p.x[2 * lane + 1];
            if (a.ratio == 2) raw[2] = p.y[2 * lane], raw[3] = p.y[2 * lane + 1];
        };
        Place now = find();
        fetch(now);
        Place next = find();
        int n = 0;
        for (int tile = blockIdx.x; tile < all; tile += gridDim.x, ++n) {
            const int buf = n % CM_BUFS;
            const int64_t at = now.entry;
            float x[16];
            if (at >= 0) {
                bf16x16_to_f32(raw[0], raw[1], x);
                if (a.ratio == 2) {
                    float y[16];
                    bf16x16_to_f32(raw[2], raw[3], y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {            // (merge16, of weights in shared memory)
                        const float4 f0 = merge[k * 32 + lane], f1 = merge[128 + k * 32 + lane];
                        const float w0[4] = {f0.x, f0.y, f0.z, f0.w}, w1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * k + i] = __fmaf_rn(w1[i], y[4 * k + i], __fmul_rn(w0[i], x[4 * k + i]));
                    }
                }
            }
            __syncwarp();
            if (warp == 0 && tile % tiles == 0 && a.prev_out != nullptr) {   // (its rows are here)
                const int b = tile / tiles;
                carry_on(a, AppendSeq(a, b), b, now.length);
            }
            now = next;
            fetch(now);
            next = find();
            uint32_t q0 = 0u, q1 = 0u, sb = 0u;
            if (at >= 0) {
                quant_group16(x, q0, q1, sb);
                store_latent(a, at, q0, q1, sb);
            }
            const __half2 sc = __half2half2(__low2half(e4m3x2_to_f16x2(sb)));
            __half2 h[8], sq = __half2half2(__ushort_as_half(0));
            e2m1x8_to_f16x8(q0, h), e2m1x8_to_f16x8(q1, h + 4);
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sq = __hfma2(h[i], h[i], sq);                // (quarters up to 288: exact)
                const __half2 v = __hmul2(h[i], sc);
                o[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            const float s = __low2float(sc);
            float norm = (__low2float(sq) + __high2float(sq)) * s * s;
#pragma unroll
            for (int k = 16; k; k >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, k);
            // (a buffer that is not known to be free is left alone: the keys' warps then wait for it in vain, and say so)
            if (n >= CM_BUFS) ok = ok && umma::mbar_wait_fast(sa(&b_free[buf]), ((n / CM_BUFS) - 1) & 1);
            uint8_t* row = A + buf * CM_A + (lane >> 2) * (CM_TILE * 128) + warp * 128;
            if (ok) {
                *reinterpret_cast<uint4*>(row + (((2 * (lane & 3)) ^ (warp & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(row + (((2 * (lane & 3) + 1) ^ (warp & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                if (lane == 0) entry_at[buf][warp] = at, norm_l[buf][warp] = sqrtf(norm);
            }
            umma::fence_proxy_async();
            const bool all = __all_sync(0xffffffffu, ok);
            __syncwarp();
            if (all && lane == 0) umma::mbar_arrive(sa(&b_full[buf]));
        }
    } else {
        // ================= W: a warp makes a row, lane g its dims 16 g .. + 15
        constexpr int N = (128 + CM_THREADS / 32 - CM_MAKERS - 1) / (CM_THREADS / 32 - CM_MAKERS);
        uint2 wc[N];
        float ws[N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int d = warp - CM_MAKERS + r * (CM_THREADS / 32 - CM_MAKERS);
            wc[r] = make_uint2(0u, 0u), ws[r] = 0.0f;
            if (d < DI) {
                wc[r] = reinterpret_cast<const uint2*>(a.wik_codes + d * (D_LAT / 2))[lane];
                ws[r] = (float)cw_e4m3_x512(a.wik_scales[d * (D_LAT / 16) + lane]) * 0x1p-9f;    // (as the exact integers take it)
            }
        }
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int d = warp - CM_MAKERS + r * (CM_THREADS / 32 - CM_MAKERS);
            if (d >= 128) break;
            const uint2 c = wc[r];
            const float sw = ws[r];
            const __half2 sc = __float2half2_rn(sw);
            __half2 h[8], sq = __half2half2(__ushort_as_half(0));
            e2m1x8_to_f16x8(c.x, h), e2m1x8_to_f16x8(c.y, h + 4);
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sq = __hfma2(h[i], h[i], sq);
                const __half2 v = __hmul2(h[i], sc);
                o[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            float norm = (__low2float(sq) + __high2float(sq)) * sw * sw;
#pragma unroll
            for (int k = 16; k; k >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, k);
            uint8_t* row = W + (lane >> 2) * (128 * 128) + d * 128;
            *reinterpret_cast<uint4*>(row + (((2 * (lane & 3)) ^ (d & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(row + (((2 * (lane & 3) + 1) ^ (d & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            if (lane == 0) norm_w[d] = sqrtf(norm);
        }
        umma::fence_proxy_async();
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(sa(&b_w));
        ok = umma::mbar_wait_fast(sa(&b_w), 0);
        if (warp < CM_OUT) {
            // ================= sums: dims 256 half .. + 255 of every tile
            const int half = warp - CM_MMA;
            const uint32_t id = umma::idesc_f16(128, CM_TILE, 0, 0);
            const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
            const uint64_t wd = umma::desc(base, 16, 1024, umma::LAYOUT_SW128);
            int n = 0;
            for (int tile = blockIdx.x; tile < all; tile += gridDim.x, ++n) {
                const int buf = n % CM_BUFS, set = n & 1;
                ok = ok && umma::mbar_wait_fast(sa(&b_full[buf]), (n / CM_BUFS) & 1);
                if (n >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_taken[set]), ((n >> 1) - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                umma::fence_after();
                const uint64_t ad = umma::desc(base + CM_W + buf * CM_A, 16, 1024, umma::LAYOUT_SW128);
                if (umma::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk) {
                        const int ks = 16 * half + kk;
                        umma::mma_f16(tm + 128 * set + 16 * (ks >> 2), wd + (uint64_t)(((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4),
                                      ad + (uint64_t)(((ks >> 2) * (CM_TILE * 128) + (ks & 3) * 32) >> 4), id, (kk & 3) > 0);
                    }
                    umma::commit(sa(&b_sum[set]));
                }
                __syncwarp();
            }
        } else {
            // ================= keys: set s has tiles s, s + 2, ..; warp q of it (TMEM lanes 32 q .. + 31) key groups 2 q and
            // 2 q + 1, a thread an entry's group
            const int qd = warp & 3, set = (warp - CM_OUT) >> 2, e = lane & 15, group = 2 * qd + (lane >> 4);
            float* turn = reinterpret_cast<float*>(A + CM_BUFS * CM_A + (warp - CM_OUT) * CM_TURN);
            float nw = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) nw = fmaxf(nw, norm_w[group * 16 + i]);
            bool made = true;                                // the entries are (if a wait for them ran out, where they go is found out here)
            int n = 0;
            for (int tile = blockIdx.x; tile < all; tile += gridDim.x, ++n) {
                if ((n & 1) != set) continue;
                const int buf = n % CM_BUFS;
                made = __all_sync(0xffffffffu, made && umma::mbar_wait_fast(sa(&b_full[buf]), (n / CM_BUFS) & 1));
                ok = ok && made && umma::mbar_wait_fast(sa(&b_sum[set]), (n >> 1) & 1);
                umma::fence_after();
                {
                    const uint32_t at = tmem + ((uint32_t)(qd * 32) << 16) + 128 * set;
                    float v[16], w[16], x[16];
                    umma::tmem_ld16(at, v);
#pragma unroll
                    for (int k = 1; k < 7; k += 2) {
                        umma::tmem_ld16(at + 16 * k, w);
                        umma::tmem_ld16(at + 16 * (k + 1), x);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] += w[i] + x[i];
                    }
                    umma::tmem_ld16(at + 112, w);
                    umma::tmem_wait_ld();
                    umma::fence_before();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(sa(&b_taken[set]));
#pragma unroll
                    for (int i = 0; i < 16; ++i) turn[i * 36 + lane] = v[i] + w[i];
                }
                __syncwarp();
                if (qd < DI / 32) {
                    float v[16];
                    auto load = [&]() {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(turn + e * 36 + (group & 1) * 16 + i);
                            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
                        }
                    };
                    load();
                    const int64_t at = made ? entry_at[buf][e] : cm_place(a, tile, tiles, e);
                    const float err = CM_ERR * nw * norm_l[buf][e];
                    // the values that `open` names, summed again exactly, one after the other: lane g the term of latent group g
                    auto settle = [&](uint32_t open) {
                        const bool mine = open != 0u;
                        for (unsigned who = __ballot_sync(0xffffffffu, mine); who;) {
                            const int src = __ffs(who) - 1;
                            const uint32_t left = __shfl_sync(0xffffffffu, open, src);
                            const int i = __ffs(left) - 1, es = src & 15, d = (2 * qd + (src >> 4)) * 16 + i;
                            uint4 l[2], w[2];
                            cm_row16(A + buf * CM_A + (lane >> 2) * (CM_TILE * 128), es, lane, l);
                            cm_row16(W + (lane >> 2) * (128 * 128), d, lane, w);
                            const __half2 *lh = reinterpret_cast<const __half2*>(l), *wh = reinterpret_cast<const __half2*>(w);
                            float t = 0.0f;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float2 x = __half22float2(lh[k]), y = __half22float2(wh[k]);
                                t = fmaf(x.y, y.y, fmaf(x.x, y.x, t));
                            }
                            long long sum = __float2ll_rn(t * 0x1p20f);
#pragma unroll
                            for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
                            if (lane == 0) turn[es * 36 + (src >> 4) * 16 + i] = __ll2float_rn(sum) * 0x1p-20f;
                            if (lane == src) open &= open - 1u;
                            if ((left & (left - 1u)) == 0u) who &= who - 1u;
                        }
                        __syncwarp();
                        if (mine) load();
                    };
                    auto largest = [&]() {
                        float top = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));
                        return top;
                    };
                    const bool there = at >= 0 && ok;
                    float top = largest();
                    uint32_t sb = f32_to_e4m3_satfinite(__fdiv_rn(fmaxf(top - err, 0.0f), 6.0f)), done = 0u;
                    if (there && sb != f32_to_e4m3_satfinite(__fdiv_rn(top + err, 6.0f)))
#pragma unroll
                        for (int i = 0; i < 16; ++i) done |= fabsf(v[i]) >= top - 2.0f * err ? 1u << i : 0u;
                    if (__any_sync(0xffffffffu, done != 0u)) {       // the scale is open: it takes the largest ones
                        settle(done);
                        if (done != 0u) sb = f32_to_e4m3_satfinite(__fdiv_rn(largest(), 6.0f));
                    }
                    uint32_t q0 = 0u, q1 = 0u, open = 0u;
                    if (sb != 0u) {
                        const float s = e4m3_to_f32(sb);
                        float lo[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) lo[i] = v[i] - err, v[i] += err;
                        q0 = e2m1_codes8(lo, s), q1 = e2m1_codes8(lo + 8, s);
                        const uint32_t d0 = q0 ^ e2m1_codes8(v, s), d1 = q1 ^ e2m1_codes8(v + 8, s);
                        if (there && (d0 | d1) != 0u)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                open |= (((d0 >> (4 * i)) & 15u) ? 1u << i : 0u) | (((d1 >> (4 * i)) & 15u) ? 256u << i : 0u);
                    }
                    if (__any_sync(0xffffffffu, open != 0u)) {
                        settle(open);
                        if (open != 0u) {                    // (the other codes are those of their exact sums as they are)
                            const float s = e4m3_to_f32(sb);
                            q0 = e2m1_codes8(v, s), q1 = e2m1_codes8(v + 8, s);
                        }
                    }
                    if (!ok) q0 = q1 = 0u, sb = 0x7fu;
                    if (at >= 0) {
                        *reinterpret_cast<uint2*>(a.ik_codes + at * (DI / 2) + group * 8) = make_uint2(q0, q1);
                        a.ik_scales[at * (DI / 16) + group] = (uint8_t)sb;
                    }
                }
                __syncwarp();                                // (sums and entries are read)
                if (lane == 0) umma::mbar_arrive(sa(&b_free[buf]));
            }
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == CM_MMA) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, 256);
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

cudaError_t launch_cache_append(const csa2_cache& c, const uint16_t* rows, int n_rows, const int32_t* path, int n_path,
                                const int64_t* pos0, const uint16_t* prev, uint16_t* prev_out, const float* w0,
                                const float* w1, const uint8_t* wik_codes, const uint8_t* wik_scales, cudaStream_t st) {
    const int n_ent = c.ratio == 2 ? n_path / 2 + (n_path & 1) : n_path;
    const bool carry = c.ratio == 2 && prev_out != nullptr;
    if (n_ent == 0 && (!carry || prev_out == prev)) return cudaSuccess;
    const int di = wik_codes ? c.d_idx : 0;
    const AppendArgs a{c.lat_codes, c.lat_scales, c.ikey_codes, c.ikey_scales, c.capacity, c.ratio, rows, n_rows, path, n_path, n_ent,
                       pos0, prev, carry ? prev_out : nullptr, w0, w1, wik_codes, wik_scales};
    // the tensor cores make the keys where that is the faster: about 10 us and 4 more for every further round of tiles, and
    // 24 ns an entry otherwise (64 sequences' 256 entries: 12.5 us without them and 14 with; 512: 18.7 and 14; one entry of each of
    // 304 sequences: 12.5 and 18)
    const int tiles = (n_ent + CM_TILE - 1) / CM_TILE;
    const int64_t rounds = ((int64_t)tiles * c.batch + 151) / 152;
    if (di > 0 && (int64_t)n_ent * c.batch >= 160 * (1 + rounds) && (int64_t)tiles * c.batch <= INT32_MAX) {
        const unsigned grid = (unsigned)std::min<int64_t>((int64_t)tiles * c.batch, 152);
        const auto kern = di == 128 ? k_cache_append_many<128> : k_cache_append_many<64>;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CM_DYN);
        if (e != cudaSuccess) return e;
        launch_k(kern, dim3(grid), CM_THREADS, CM_DYN, st, a, tiles, (int)c.batch);
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
