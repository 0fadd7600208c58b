// Products with FP4 weights (E2M1 codes, one E4M3 scale per 16 values, the
// cache's format):  y[t][g][m] = alpha * sum_k W[g][m][k] x[t][g][k].
//
// W is never expanded in memory: 9/16 of a byte per weight is read once per pass
// over the tokens, and the weights become fp16 in registers.  That is exact: an
// E2M1 value times an E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688].  x goes to fp16 too, each token (of a group, or of a 128-value
// chunk) times the power of two 2^-E that brings its largest magnitude into [2^14,
// 2^15): fp16 x needs no scale, bf16 x loses only what lies 2^39 below the largest
// value, and fp32 x is split into two fp16 parts (2^-22 of each value).  Products
// are exact, sums fp32; y is rounded once.
//
// Two kernels:
//  - k_linear_few (up to 8 tokens, 4 of fp32, and twice as many where the matrix is
//    small).  The weights' bytes are its floor: one token, 1,536 -> 32,768 (28 MB) takes
//    8.7 us, 3.2 TB/s, for a floor of 4.2.  Neither memory (26 % busy) nor the SMs' issue
//    slots (44 %) bound it: launch, set-up, the weights' first bytes (asked for only after
//    the wait for the kernel before) and the conversion of x take 2.5 us one after the
//    other, and a block's few tiles then overlap little.  mma.sync m16n8k16, the weights as the A fragments.  The order of
//    k within a product is free as long as both operands agree, so a lane takes 16
//    consecutive bytes of a row (32 weights, two scale groups) and feeds them, four at a
//    time, to eight products, and x comes from global memory in the matching order.  The
//    weights come by bulk copies, all at once.
//  - k_linear_many: tcgen05, M = 128 rows, N = up to 128 tokens.  Expanded
//    weights go from registers to TMEM (the A operand), so shared memory carries
//    the tokens alone: with both operands there, N = 128 would need 192 bytes per
//    clock of the 128 it gives.  x comes by bulk copies in the layout that
//    k_linear_x has written to the workspace; fp16 tokens by tensor copies from where
//    they are.  When there are few row tiles a cluster of blocks splits n_in and adds
//    up through distributed shared memory.
//    What bounds it is the tensor pipe with 128 tokens (busy 512 of the 600 clocks that
//    128 values of a row tile take), and with fewer its pipeline's start (2.5 us to the
//    first product: codes, expansion, x) and end (1.5 us).  64 bf16 tokens, 1,536 ->
//    32,768: 14.5 us with k_linear_x, which overlaps its start, and in fp16 13.6 without;
//    256 fp16 tokens, 4,096 -> 8,192: 16.6 us (1,040 TFLOP/s on 128 of the 152 SMs).
#include <algorithm>
#include <type_traits>

#include <cuda.h>

#include "common.cuh"
#include "elem.cuh"
#include "fp4_f16.cuh"
#include "umma.cuh"

namespace csa2 {

struct LinArgs {
    const void* x;
    int64_t x_tok, x_group;
    int n_tok, n_groups, n_in, n_out;
    const uint8_t* codes;
    const uint8_t* scales;
    float alpha;
    void* y;
    int y_type;
    int64_t y_tok, y_group;
};

__device__ __forceinline__ void lin_store(const LinArgs& a, int t, int g, int m, float v) {
    const int64_t i = t * a.y_tok + g * a.y_group + m;
    if (a.y_type == CSA2_BF16)
        reinterpret_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
    else if (a.y_type == CSA2_F16)
        reinterpret_cast<__half*>(a.y)[i] = __float2half_rn(v);
    else
        reinterpret_cast<float*>(a.y)[i] = v;
}

// The exponent E of a token whose largest finite magnitude is mx: mx * 2^-E in [2^14, 2^15)
__device__ __forceinline__ int lin_exp(float mx) {
    if (mx == 0.0f) return 0;
    return max(-126, (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 14);
}
// the largest finite magnitude of eight values: the largest magnitude as bits and, where that is an infinity or
// a NaN (which stay what they are in fp16), one by one
template <typename TX>
__device__ __forceinline__ float lin_absmax(const ElemVec<TX, 8>& v) {
    uint32_t m = 0u;
    if constexpr (sizeof(TX) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, v.w[i] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16) << 16;                 // bf16: the upper half of the fp32 bits
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, v.w[i] & 0x7fffffffu);
    }
    if (__builtin_expect(m < 0x7f800000u, 1)) return __uint_as_float(m);
    float f = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = fabsf(v.get(e));
        if (a < INFINITY) f = fmaxf(f, a);
    }
    return f;
}
// eight values times d as fp16, and for fp32 what that leaves (0 where it is not finite)
template <typename TX>
__device__ __forceinline__ void lin_split(const ElemVec<TX, 8>& v, float d, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(TX) == 2 && !std::is_same<TX, __nv_bfloat16>::value) {
            h[i] = v.w[i];
        } else {
            const float a = v.get(2 * i) * d, b = v.get(2 * i + 1) * d;
            const __half2 p = __floats2half2_rn(a, b);
            h[i] = *reinterpret_cast<const uint32_t*>(&p);
            if constexpr (sizeof(TX) == 4) {
                const float ra = a - __low2float(p), rb = b - __high2float(p);
                l[i] = f16x2_bits(fabsf(ra) < INFINITY ? ra : 0.0f, fabsf(rb) < INFINITY ? rb : 0.0f);
            }
        }
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// the eight elements at p, by 16-byte loads where the rows allow it
template <typename TX>
__device__ __forceinline__ ElemVec<TX, 8> lin_load8(const TX* p, bool vec) {
    ElemVec<TX, 8> v;
    if (vec)
        v.load(p);
    else
        v.load_each(p);
    return v;
}

// ================================================================ up to 16 tokens

constexpr int LF_TOK = 16;
constexpr int LF_MAXW = 8;                       // warps of a block
constexpr int LF_SMEM = 184 * 1024;              // the weights of a block, at most

__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bytes [start, start + n) of `src` into shared memory at dst (16-byte aligned), byte i at dst + start % 16 + i:
// a bulk copy of the whole 16-byte pieces, counted on `bar`, and plain loads of the rest by the calling warp.
__device__ __forceinline__ uint32_t lf_bulk_bytes(uint64_t start, uint32_t n) {
    return (uint32_t)(((start + n) & ~15ull) - (start & ~15ull));
}
__device__ __forceinline__ void lf_copy(uint8_t* dst, const uint8_t* src, uint64_t start, uint32_t n, uint32_t bar, int lane) {
    const uint64_t a = start & ~15ull;
    const uint32_t whole = lf_bulk_bytes(start, n);
    if (lane == 0 && whole > 0) umma::bulk_g2s(umma::smem_u32(dst), src + a, whole, bar);
    const uint32_t rest = (uint32_t)(start + n - a) - whole;
    if (lane < (int)rest) dst[whole + lane] = src[a + whole + lane];
}

// A block takes up to R tiles of 16 rows: `each`, the first `more` blocks one more.  Rows are contiguous, so a
// tile's codes and scales are one piece of memory each: all of them are requested by bulk copies as the block
// starts, which keeps more bytes in flight than registers could (one token, 1,536 x 32,768: every block's rows at once), and each tile has a
// barrier of its own.  The warps split n_in in chunks of 128, warp w taking chunks w, w + warps, ..; per
// chunk a warp holds the tokens' fragments in registers and runs all R tiles over them.  The warps' sums are
// joined at the end, in order.
template <typename TX, int NT, int R>
__global__ void __launch_bounds__(LF_MAXW * 32, 2) k_linear_few(const LinArgs a, int x_vec, int each, int more) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(8) unsigned long long b_tile[R];
    constexpr bool SPLIT = sizeof(TX) == 4, SCALED = !std::is_same<TX, __half>::value;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    const int K = a.n_in, T = a.n_tok, g = blockIdx.y;
    const int chunks = (K + 127) / 128;
    const int m0 = 16 * ((int)blockIdx.x * each + min((int)blockIdx.x, more));
    const int r = lane >> 2, c = lane & 3;
    const int rows = min(16 * (each + ((int)blockIdx.x < more)), a.n_out - m0);
    // tile i's codes at sm + i * (8 K + 16), its scales after all codes at i * (K + 16) (both with the source's
    // offset to 16 bytes)
    const uint32_t c_tile = 8u * K + 16, s_tile = (uint32_t)K + 16;
    uint8_t* sm_s = sm + R * c_tile;
    const uint64_t row0 = (uint64_t)g * a.n_out + m0;
    const uint64_t c0 = row0 * (uint64_t)(K / 2), s0 = row0 * (uint64_t)(K / 16);
    if (tid == 0) {
        for (int i = 0; i < R; ++i) umma::mbar_init(umma::smem_u32(&b_tile[i]), 1);
        umma::fence_mbar_init();
    }
    pdl_wait();                                  // x, and weights just quantised, may come from the preceding kernel
    __syncthreads();                             // the barriers
#pragma unroll 1
    for (int i = warp; i < R; i += warps) {      // a tile's copies are some 150 instructions: a warp for each
        const int n = max(0, min(16, rows - 16 * i));
        const uint64_t cb = c0 + (uint64_t)i * 8 * K, sb = s0 + (uint64_t)i * K;
        const uint32_t nc = (uint32_t)n * (K / 2), ns = (uint32_t)n * (K / 16);
        const uint32_t bar = umma::smem_u32(&b_tile[i]);
        if (lane == 0) umma::mbar_arrive_expect_tx(bar, n > 0 ? lf_bulk_bytes(cb, nc) + lf_bulk_bytes(sb, ns) : 0u);
        __syncwarp();
        if (n > 0) {
            lf_copy(sm + i * c_tile, a.codes, cb, nc, bar, lane);
            lf_copy(sm_s + i * s_tile, a.scales, sb, ns, bar, lane);
        }
    }

    const TX* x = reinterpret_cast<const TX*>(a.x) + (int64_t)g * a.x_group;
    uint4 bh[NT][4], bl[SPLIT ? NT : 1][4];      // 32 values of token n * 8 + r: this lane's B fragments of a chunk
    float back[NT][2];                           // 2^E of tokens n * 8 + 2c and + 1
    ElemVec<TX, 8> v[4];
    auto fetch = [&](int ch, int n) {            // chunk ch of token n * 8 + r: this lane's segment
        const int t = n * 8 + r, k0 = ch * 128 + c * 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t < T && k0 + 8 * j < K)
                v[j] = lin_load8(x + t * a.x_tok + k0 + 8 * j, x_vec);
            else
#pragma unroll
                for (int i = 0; i < ElemVec<TX, 8>::WORDS; ++i) v[j].w[i] = 0u;
        }
    };
    auto convert = [&](int n) {
        float m = 0.0f, d = 1.0f;
        if (SCALED) {
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, lin_absmax(v[j]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const int e = lin_exp(m);
            d = pow2f(-e);
            const float up = pow2f(e);           // of token r (of 8); this lane's results are of tokens 2c, 2c + 1
            back[n][0] = __shfl_sync(0xffffffffu, up, 8 * c);
            back[n][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 lo;
            lin_split(v[j], d, bh[n][j], lo);
            if (SPLIT) bl[n][j] = lo;
        }
    };
    // up to 8 tokens: the loads run a chunk ahead (more would not fit the registers)
    constexpr bool EARLY = NT == 1 && !(SPLIT && R > 1);
    if (EARLY && warp < chunks) fetch(warp, 0);  // while the weights arrive
    __syncthreads();                             // the barriers, and the copies' plain ends

    // one row's 32 weights (16 bytes of codes, two scales) from k on; rows past the end repeat the last one (their
    // results are not stored), and values from n_in on are zeros
    const uint32_t co = (uint32_t)(c0 & 15), so = (uint32_t)(s0 & 15);     // of every tile: a tile is a multiple of 16 bytes
    const bool wide = K % 32 == 0;               // codes 16 bytes apart from a 16-byte boundary, scales in pairs
    const bool full = rows % 16 == 0 && K % 128 == 0 && co == 0;         // nothing to check, few addresses to find
    const uint8_t* cl = sm + (uint32_t)r * (K / 2) + c * 16;
    const uint8_t* sl = sm_s + so + (uint32_t)r * (K / 16) + c * 2;
    auto segment = [&](int tile, int hi, int ch, uint4& cw, uint32_t& sw) {
        if (full) {
            cw = *reinterpret_cast<const uint4*>(cl + tile * c_tile + hi * (K / 2) + ch * 64);
            sw = *reinterpret_cast<const uint16_t*>(sl + tile * s_tile + hi * (K / 16) + ch * 8);
            return;
        }
        const int row = r + hi, k = ch * 128 + c * 32;
        const int rr = min(row, rows - 1 - tile * 16);
        const uint8_t* cp = sm + tile * c_tile + co + (uint32_t)rr * (K / 2) + k / 2;
        const uint8_t* sp = sm_s + tile * s_tile + so + (uint32_t)rr * (K / 16) + k / 16;
        cw = make_uint4(0, 0, 0, 0);
        sw = 0u;
        if (k >= K) return;
        if (wide && co == 0) {
            cw = *reinterpret_cast<const uint4*>(cp);
            sw = sp[0] | ((uint32_t)sp[1] << 8);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(cp);
            cw.x = u.x, cw.y = u.y;
            sw = sp[0];
            if (k + 16 < K) {
                const uint2 w = *reinterpret_cast<const uint2*>(cp + 8);
                cw.z = w.x, cw.w = w.y;
                sw |= (uint32_t)sp[1] << 8;
            }
        }
    };
    bool ok = true;
    float acc[R][NT][4] = {};
    for (int ch = warp; ch < chunks; ch += warps) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (!EARLY) fetch(ch, n);
            convert(n);
        }
        if (EARLY && ch + warps < chunks) fetch(ch + warps, 0);
#pragma unroll
        for (int tile = 0; tile < R; ++tile) {
            if (tile * 16 >= rows) break;
            if (ch == warp) ok = ok && umma::mbar_wait_fast(umma::smem_u32(&b_tile[tile]), 0);
            uint4 va, vb;
            uint32_t sa, sb;
            segment(tile, 0, ch, va, sa);
            segment(tile, 8, ch, vb, sb);
            const __half2 pa = e4m3x2_to_f16x2(sa), pb = e4m3x2_to_f16x2(sb);
            const uint32_t xa[4] = {va.x, va.y, va.z, va.w}, xb[4] = {vb.x, vb.y, vb.z, vb.w};
            float d[NT][2][4] = {};              // two sums: consecutive products do not wait for each other
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint4 fa = e2m1x8_scaled(xa[w], w < 2 ? __low2half2(pa) : __high2half2(pa));
                const uint4 fb = e2m1x8_scaled(xb[w], w < 2 ? __low2half2(pb) : __high2half2(pb));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_16816(d[n][0], fa.x, fb.x, fa.y, fb.y, bh[n][w].x, bh[n][w].y);
                    mma_16816(d[n][1], fa.z, fb.z, fa.w, fb.w, bh[n][w].z, bh[n][w].w);
                    if (SPLIT) {
                        mma_16816(d[n][0], fa.x, fb.x, fa.y, fb.y, bl[n][w].x, bl[n][w].y);
                        mma_16816(d[n][1], fa.z, fb.z, fa.w, fb.w, bl[n][w].z, bl[n][w].w);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = d[n][0][i] + d[n][1][i];
                    acc[tile][n][i] = SCALED ? fmaf(v, back[n][i & 1], acc[tile][n][i]) : acc[tile][n][i] + v;
                }
        }
    }
    // every copy has landed before the block's memory is used again or given up: each tile's barrier is waited
    // for by warp 0 even where it has no chunk
    if (warp == 0 && chunks == 0)
        for (int i = 0; i < R; ++i) ok = ok && umma::mbar_wait_fast(umma::smem_u32(&b_tile[i]), 0);
    // ---- join the warps in order and store with the rows along the lanes
    float* red = reinterpret_cast<float*>(sm);   // [warp][token][R * 16 rows]
    __syncthreads();                             // the weights are read no more
#pragma unroll
    for (int tile = 0; tile < R; ++tile)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = n * 8 + 2 * c + (i & 1);
                if (t < T)
                    red[(warp * T + t) * (R * 16) + tile * 16 + r + 8 * (i >> 1)] = ok ? acc[tile][n][i] : __int_as_float(0x7fc00000);
            }
    __syncthreads();
    for (int u = tid; u < T * R * 16; u += blockDim.x) {
        const int t = u / (R * 16), m = u % (R * 16);
        if (m >= rows) continue;
        float v = 0.0f;
        for (int w = 0; w < warps; ++w) v += red[w * T * (R * 16) + u];
        lin_store(a, t, g, m0 + m, v * a.alpha);
    }
    __syncthreads();
    if (tid == 0) __threadfence();               // the attention may stage these rows before it waits (see norm_rope.cu)
}

// ================================================================ more tokens

constexpr int LM_EXPAND = 16, LM_EPI = 4;        // warps 0-15 expand weights, 16-19 store results,
constexpr int LM_XW = LM_EXPAND + LM_EPI;        // 20 copies x, 21 copies codes, 22 and 23 issue MMAs
constexpr int LM_THREADS = (LM_XW + 4) * 32;
constexpr int LM_M = 128, LM_K = 128;            // rows of a block, values per stage
constexpr int LM_MAXC = 9;                       // code stages, at most
constexpr int LM_S = 4;                          // stages: x in shared memory, expanded weights in TMEM (64 columns each)
constexpr int LM_CK = 2 * LM_K;                  // values per code stage: 128 bytes of each row, whole lines
constexpr uint32_t LM_CODES = LM_M * LM_CK / 2;  // bytes of codes of a stage

struct LinPrep {                                 // the workspace's layout
    int nb, tiles, chunks, planes;               // tokens per tile, token tiles, 128-value chunks, fp16 parts
    __host__ __device__ int cols() const { return nb * planes; }         // a product's: the parts of x side by side
    __host__ __device__ int64_t half_bytes() const { return (int64_t)cols() * 128; }
    __host__ __device__ int64_t stage_bytes() const { return half_bytes() * 2; }
    // [group][token tile][chunk][half chunk][part] tiles of nb rows x 64 values in the MMA's swizzled layout
    __host__ __device__ int64_t stage(int g, int tt, int ch) const {
        return (((int64_t)g * tiles + tt) * chunks + ch) * stage_bytes();
    }
    __host__ __device__ int64_t scales_at(int groups) const { return (int64_t)groups * tiles * chunks * stage_bytes(); }
};

// one block per token and group: its scale, and its values in the layout above
template <typename TX>
__global__ void __launch_bounds__(256) k_linear_x(const LinArgs a, LinPrep p, uint8_t* __restrict__ ws, int x_vec) {
    constexpr bool SPLIT = sizeof(TX) == 4, SCALED = !std::is_same<TX, __half>::value;
    constexpr int KEEP = SCALED ? 2 : 1;         // pieces of 2,048 values that stay in registers between the passes
    __shared__ unsigned int tmax;
    const int t = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
    const TX* x = reinterpret_cast<const TX*>(a.x) + t * a.x_tok + (int64_t)g * a.x_group;
    if (SCALED && tid == 0) tmax = 0u;
    pdl_wait();
    pdl_launch_next();                           // the product's blocks start expanding weights meanwhile
    ElemVec<TX, 8> v[KEEP];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (tid * 8 + i * 2048 < a.n_in) v[i] = lin_load8(x + tid * 8 + i * 2048, x_vec);
    float d = 1.0f;
    float* scale = reinterpret_cast<float*>(ws + p.scales_at(a.n_groups)) + (int64_t)g * a.n_tok + t;
    if (SCALED) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (tid * 8 + i * 2048 < a.n_in) m = fmaxf(m, lin_absmax(v[i]));
        for (int k = tid * 8 + KEEP * 2048; k < a.n_in; k += 2048) m = fmaxf(m, lin_absmax(lin_load8(x + k, x_vec)));
        const unsigned int w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if ((tid & 31) == 0 && w) atomicMax(&tmax, w);
        __syncthreads();
        const int e = lin_exp(__uint_as_float(tmax));
        d = pow2f(-e);
        if (tid == 0) *scale = pow2f(e);
    } else if (tid == 0) {
        *scale = 1.0f;
    }
    const int tt = t / p.nb, r = t - tt * p.nb;
    auto put = [&](int k, const ElemVec<TX, 8>& e) {
        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
        if (k < a.n_in) lin_split(e, d, hi, lo);
        uint8_t* at = ws + p.stage(g, tt, k >> 7) + ((k >> 6) & 1) * p.half_bytes() + r * 128 + ((((k >> 3) & 7) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = hi;
        if (SPLIT) *reinterpret_cast<uint4*>(at + p.nb * 128) = lo;
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (tid * 8 + i * 2048 < p.chunks * LM_K) put(tid * 8 + i * 2048, v[i]);
    for (int k = tid * 8 + KEEP * 2048; k < p.chunks * LM_K; k += 2048)
        put(k, k < a.n_in ? lin_load8(x + k, x_vec) : v[0]);
}

// D[tmem] += A[tmem: 128 rows x 16 fp16, two per column] . B[smem]
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
// a box of the codes (128 bytes of 128 rows) at byte column x (a multiple of 64) and row y
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(mbar)
        : "memory");
}

// a box of the tokens (64 values of p.nb tokens) at value x (a multiple of 64), token y and group z
__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(mbar)
        : "memory");
}

// the four scales of 64 weights of one row from k on; zeros from n_in on
__device__ __forceinline__ uint32_t lin_scales4(const uint8_t* __restrict__ s, int k, int n_in, int wide) {
    if (k >= n_in) return 0u;
    if (wide == 2) return __ldg(reinterpret_cast<const uint32_t*>(s + k / 16));
    uint32_t v = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k + 16 * i < n_in) v |= (uint32_t)__ldg(s + k / 16 + i) << (8 * i);
    return v;
}
// 64 weights of one row: 32 bytes of codes
struct LinSeg64 {
    uint4 c[2];
    __device__ __forceinline__ void load(const uint8_t* __restrict__ codes, int k, int n_in) {
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = make_uint2(0, 0);
            if (k + 16 * i < n_in) w[i] = __ldg(reinterpret_cast<const uint2*>(codes + k / 2) + i);
        }
        c[0] = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
        c[1] = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
    }
};

// after a wait that gave up: this thread's copies in flight (the last of `issued` into a ring) land before
// the block ends
__device__ __forceinline__ void lin_drain(bool ok, unsigned long long* full, uint32_t stages, uint32_t issued) {
    if (!ok)
        for (uint32_t j = issued > stages ? issued - stages : 0; j < issued; ++j)
            umma::mbar_wait(umma::smem_u32(&full[j % stages]), (j / stages) & 1, 1u << 16);
}

struct LinRings {
    int tiles_m, log_splits, wide, c_stages;
};

// Tiles (row tile, token tile, group) in that order of change from slow to fast: group, row tile, token
// tile, so that blocks side by side read the same codes.  Without splits the blocks walk the tiles,
// the results of one being stored while the next is summed; with splits a cluster takes one tile and
// its blocks a share of the chunks each.  TMA: the codes come by tensor copies (n_in a multiple of 32:
// rows a multiple of 16 bytes apart), else by plain loads.  DIRECT: fp16 tokens are read where they are, with
// no k_linear_x before this kernel (a variant of its own: as a test at run time it cost the others 4 %).
template <bool TMA, bool DIRECT>
__global__ void __launch_bounds__(LM_THREADS, 1)
    k_linear_many(const __grid_constant__ CUtensorMap tmap, const LinArgs a, LinPrep p, const uint8_t* __restrict__ ws,
                  int* __restrict__ err, LinRings rg, const __grid_constant__ CUtensorMap xmap) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) unsigned long long b_a[LM_S], b_x[LM_S], b_free[LM_S], b_c[LM_MAXC], b_cfree[LM_MAXC], b_d[2],
        b_dfree[2];
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int splits = 1 << rg.log_splits, CS = rg.c_stages, NB = p.nb, NC = p.cols();
    const uint32_t raw = umma::smem_u32(dyn), base = (raw + 1023u) & ~1023u;
    uint8_t* sm = dyn + (base - raw);
    const uint32_t stage_bytes = (uint32_t)p.stage_bytes(), xb = base + (TMA ? CS * LM_CODES : 0u);
    const int tiles = rg.tiles_m * p.tiles * a.n_groups;
    const int split = blockIdx.x & (splits - 1);                 // (a power of two of them)
    const int first = blockIdx.x >> rg.log_splits, step = gridDim.x >> rg.log_splits;
    const int ch0 = (p.chunks * split) >> rg.log_splits, n = ((p.chunks * (split + 1)) >> rg.log_splits) - ch0;
    struct Tile {
        int m, t, g;
    };
    auto tile_of = [&](int i) {                  // (in 32 bits: two 64-bit divisions are 1,500 clocks)
        Tile v;
        const int j = (unsigned)i / (unsigned)p.tiles;
        v.t = i - j * p.tiles;
        v.g = (unsigned)j / (unsigned)rg.tiles_m;
        v.m = j - v.g * rg.tiles_m;
        return v;
    };
    // TMEM: results in columns 0-255, (buffer, issuer) tiles of NC: two buffers up to 64 columns, else one;
    // expanded weights in LM_S x 64 columns from 256 on
    constexpr uint32_t cols = 512, t_a = 256;
    const int bufs = NC <= 64 ? 2 : 1;
    auto sa = [&](const void* q) { return umma::smem_u32(q); };
    static_assert(LM_S <= 32 && LM_MAXC <= 32, "a lane each");
    if (warp == 0) {
        if (lane < LM_S) {
            umma::mbar_init(sa(&b_a[lane]), 8);                  // four lane quarters x two halves of a chunk
            umma::mbar_init(sa(&b_x[lane]), 1);
            umma::mbar_init(sa(&b_free[lane]), 1);
        }
        if (lane < LM_MAXC) {
            umma::mbar_init(sa(&b_c[lane]), 1);
            umma::mbar_init(sa(&b_cfree[lane]), LM_EXPAND);
        }
        if (lane < 2) {
            umma::mbar_init(sa(&b_d[lane]), 2);                  // both issuers
            umma::mbar_init(sa(&b_dfree[lane]), LM_EPI);
        }
        umma::fence_mbar_init();
    }
    if (TMA && warp == LM_XW + 1 && lane == 0)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap)) : "memory");
    if (DIRECT && warp == LM_XW && lane == 0)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&xmap)) : "memory");
    if (DIRECT) pdl_wait();                      // else k_linear_x has waited: the weights may have just been quantised
    __syncthreads();
    // the copies start at once; whoever touches TMEM meets here after its allocation
    uint32_t tmem = 0;
    auto tmem_ready = [&]() {
        umma::fence_before();
        umma::bar_named(1, LM_THREADS - 64);
        umma::fence_after();
        tmem = tmem_base;
    };
    bool ok = true;
    const int my_tiles = first < tiles ? (tiles - 1 - first) / step + 1 : 0;
    // Results of tile ti: this warp's lane quarter (rows along the lanes), token columns 16 (part + i * parts),
    // both issuers' sums (and of fp32 both parts') added.  With splits, to this block's shared memory as [token][128 rows].
    auto store = [&](int ti, int part, int parts) {
        const Tile v = tile_of(first + ti * step);
        const int q = warp & 3, buf = ti % bufs, m = v.m * LM_M + q * 32 + lane, t0 = v.t * NB, nt = min(NB, a.n_tok - t0);
        const float* scale = DIRECT ? nullptr : reinterpret_cast<const float*>(ws + p.scales_at(a.n_groups)) + (int64_t)v.g * a.n_tok + t0;
        float* mine = reinterpret_cast<float*>(sm);
        const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + 2 * buf * NC;
        const int one = n == 1 ? ti & 1 : 0;                     // the issuer that has a tile's only chunk
        float f[16];
        auto scales = [&](int c) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = DIRECT ? 1.0f : c + i < nt ? scale[c + i] : 0.0f;
        };
        if (splits == 1) scales(16 * part);                      // in flight while the sums are waited for
        if (n > 0) ok = ok && umma::mbar_wait_fast(sa(&b_d[buf]), (ti / bufs) & 1);
        umma::fence_after();
        for (int c = 16 * part; c < nt; c += 16 * parts) {
            float r[16], r1[16];
            umma::tmem_ld16(d + one * NC + c, r);
            umma::tmem_ld16(d + NC + c, r1);
            umma::tmem_wait_ld();
            // with a single chunk one issuer has products, without any none
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = n > 1 ? r[i] + r1[i] : n > 0 ? r[i] : 0.0f;
            for (int k = 0; k < (p.planes > 1 ? min(n, 2) : 0); ++k) {
                umma::tmem_ld16(d + (k + one) * NC + NB + c, r1);
                umma::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] += r1[i];
            }
            if (!ok)
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __int_as_float(0x7fc00000);
            if (splits > 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[(c + i) * LM_M + q * 32 + lane] = r[i];
                continue;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = r[i] * f[i] * a.alpha;           // (2^E alpha itself may leave fp32's range)
            if (c + 16 * parts < nt) scales(c + 16 * parts);
            if (m < a.n_out) {
                const int64_t y0 = (int64_t)(t0 + c) * a.y_tok + v.g * a.y_group + m;
                auto put = [&](auto* y) {
                    y += y0;
#pragma unroll
                    for (int i = 0; i < 16; ++i, y += a.y_tok)
                        if (i < nt - c) *y = from_f32<std::remove_pointer_t<decltype(y)>>(r[i]);
                };
                if (a.y_type == CSA2_BF16)
                    put(reinterpret_cast<__nv_bfloat16*>(a.y));
                else if (a.y_type == CSA2_F16)
                    put(reinterpret_cast<__half*>(a.y));
                else
                    put(reinterpret_cast<float*>(a.y));
            }
        }
        umma::fence_before();
    };

    if (warp < LM_EXPAND) {
        // ================= weights: warp w takes rows 32(w%4) .. +31 of the tile, half (w/4)%2 of a chunk and
        // every second of the block's chunks, as the issuers do (not of a tile's: a stage then has the same warps
        // each time, which have waited for its phase before, so that no wait can meet a barrier two phases back).
        // Only x and its scales come from the kernel before this one: nothing waits here.
        const int q = warp & 3, hf = (warp >> 2) & 1, par = warp >> 3, rt = q * 32 + lane;
        const uint8_t *cr = nullptr, *sr = nullptr;
        const int pairs = (n + 1) / 2;                           // of a tile's chunks; a code stage holds a pair
        const int total = my_tiles * pairs;
        constexpr int AHEAD = TMA ? 4 : 2;                       // own chunks whose scales (and plain codes) are in flight
        LinSeg64 seg[TMA ? 1 : AHEAD];
        uint32_t sc[AHEAD];
        int at = 0, ai = 0;                                      // tile and pair to load next
        auto ahead = [&](int i) {
            int k = a.n_in;
            if (at < my_tiles) {
                if (ai == 0) {
                    const Tile v = tile_of(first + at * step);
                    const int64_t row = (int64_t)v.g * a.n_out + min(v.m * LM_M + rt, a.n_out - 1);
                    cr = a.codes + row * (a.n_in / 2);
                    sr = a.scales + row * (a.n_in / 16);
                }
                const int jj = 2 * ai + (par ^ (at & n & 1));    // tile `at` begins with chunk at * n of the block's
                if (jj < n) k = (ch0 + jj) * LM_K + hf * 64;
                if (++ai == pairs) ai = 0, ++at;
            }
            sc[i] = lin_scales4(sr, k, a.n_in, rg.wide);
            if constexpr (!TMA) seg[i].load(cr, k, a.n_in);
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (total > 0) ahead(i);
        uint4 c[2];
        int cs = 0, cph = 0;                                     // code stage of the pair in c, and its phase
        auto take = [&](int stage, int odd) {                    // the even or the odd chunk of a stage's pair
            const uint8_t* src = sm + stage * LM_CODES + rt * 128;
            const int u = odd * 4 + hf * 2;
            c[0] = *reinterpret_cast<const uint4*>(src + ((u ^ (rt & 7)) << 4));
            c[1] = *reinterpret_cast<const uint4*>(src + (((u + 1) ^ (rt & 7)) << 4));
        };
        if (TMA && total > 0) {
            ok = ok && umma::mbar_wait_fast(sa(&b_c[0]), 0);
            take(0, par);
        }
        tmem_ready();
        int j = par;                                             // chunk within the tile
        uint32_t it = par;                                       // and among the block's
        for (int p0 = 0; p0 < total; p0 += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (p0 + i >= total) break;
                // the barriers that this round waits for are asked first, so that their answers (and the next
                // codes) arrive behind the arithmetic
                const uint32_t st = it % LM_S;
                const bool more = TMA && p0 + i + 1 < total;
                const int ncs = cs + 1 == CS ? 0 : cs + 1, ncph = cph ^ (ncs == 0);
                const bool c_there = more && umma::mbar_test(sa(&b_c[ncs]), ncph);
                const bool st_free = it < LM_S || umma::mbar_test(sa(&b_free[st]), (it / LM_S - 1) & 1);
                const uint32_t s4 = sc[i];
                if constexpr (!TMA) c[0] = seg[TMA ? 0 : i].c[0], c[1] = seg[TMA ? 0 : i].c[1];
                ahead(i);
                uint32_t o[32];
                const __half2 s01 = e4m3x2_to_f16x2(s4 & 0xffffu), s23 = e4m3x2_to_f16x2(s4 >> 16);
                const __half2 f4[4] = {__low2half2(s01), __high2half2(s01), __low2half2(s23), __high2half2(s23)};
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const uint4& cc = c[w >> 2];
                    const uint32_t word = (w & 3) == 0 ? cc.x : (w & 3) == 1 ? cc.y : (w & 3) == 2 ? cc.z : cc.w;
                    const uint4 f = e2m1x8_scaled(word, f4[w >> 1]);
                    o[4 * w] = f.x, o[4 * w + 1] = f.y, o[4 * w + 2] = f.z, o[4 * w + 3] = f.w;
                }
                if constexpr (TMA) {
                    __syncwarp();                                // every lane has its codes in registers
                    if (lane == 0) umma::mbar_arrive(sa(&b_cfree[cs]));
                    if (more) {
                        if (!c_there) ok = ok && umma::mbar_wait(sa(&b_c[ncs]), ncph);
                        take(ncs, (j ^ (j + 2 >= 2 * pairs ? n : 0)) & 1);
                    }
                    cs = ncs, cph = ncph;
                }
                if (j < n) {
                    if (!st_free) ok = ok && umma::mbar_wait(sa(&b_free[st]), (it / LM_S - 1) & 1);
                    if (it >= LM_S) umma::fence_after();
                    tmem_st32(tmem + ((uint32_t)(q * 32) << 16) + t_a + 64 * st + 32 * hf, o);
                    umma::tmem_wait_st();
                    umma::fence_before();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(sa(&b_a[st]));
                }
                j += 2, it += 2;
                if (j >= 2 * pairs) {                            // the next tile, of which it has the other chunks where n is odd
                    const int nj = (j ^ n) & 1;
                    it += n + nj - j, j = nj;
                }
            }
        }
    } else if (warp < LM_XW) {
        // ================= results of all tiles but the last, while the next is summed
        tmem_ready();
        pdl_wait();                                              // the tokens' scales, and y
        for (int ti = 0; ti + 1 < my_tiles; ++ti) {
            store(ti, 0, 1);
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(sa(&b_dfree[ti % bufs]));
        }
    } else if (warp == LM_XW) {
        // ================= x: bulk copies of the prepared stages, or the tokens themselves into the same layout
        if (lane == 0) {
            pdl_wait();
            uint32_t it = 0;
            for (int ti = 0; ti < my_tiles && ok; ++ti) {
                const Tile v = tile_of(first + ti * step);
                for (int j = 0; j < n; ++j, ++it) {
                    const uint32_t st = it % LM_S;
                    if (it >= LM_S) ok = ok && umma::mbar_wait_fast(sa(&b_free[st]), (it / LM_S - 1) & 1);
                    if (!ok) break;
                    umma::mbar_arrive_expect_tx(sa(&b_x[st]), stage_bytes);
                    if constexpr (DIRECT)
                        for (int h = 0; h < 2; ++h)
                            tma_box3(xb + st * stage_bytes + h * (uint32_t)p.half_bytes(), &xmap, (ch0 + j) * LM_K + h * 64, v.t * NB,
                                     v.g, sa(&b_x[st]));
                    else
                        umma::bulk_g2s(xb + st * stage_bytes, ws + p.stage(v.g, v.t, ch0 + j), stage_bytes, sa(&b_x[st]));
                }
            }
            lin_drain(ok, b_x, LM_S, it);
        }
    } else if (warp == LM_XW + 1) {
        // ================= codes
        if (TMA && lane == 0) {
            int st = 0, ph = 1;                                  // a fresh barrier passes a wait for phase 1
            uint32_t it = 0;
            for (int ti = 0; ti < my_tiles && ok; ++ti) {
                const Tile v = tile_of(first + ti * step);
                const int y = (int)((int64_t)v.g * a.n_out + v.m * LM_M);
                for (int j = 0; j < n; j += 2, ++it) {
                    ok = ok && umma::mbar_wait_fast(sa(&b_cfree[st]), ph);
                    if (!ok) break;
                    umma::mbar_arrive_expect_tx(sa(&b_c[st]), LM_CODES);
                    tma_box(base + st * LM_CODES, &tmap, (ch0 + j) * (LM_K / 2), y, sa(&b_c[st]));
                    if (++st == CS) st = 0, ph ^= 1;
                }
            }
            lin_drain(ok, b_c, CS, it);
        }
    } else {
        // ================= MMAs: two issuers, for the even and the odd chunks of the block (one thread issues an MMA per
        // 65 clocks and is held 200 by a commit, whatever the sizes; a chunk's halves for one each meant two
        // commits a chunk, 740-800 clocks); a whole warp walks the chunks, so that descriptors and addresses stay
        // in uniform registers, and one elected lane issues
        const int hf = warp - (LM_XW + 2);
        if (hf == 0) umma::tmem_alloc(sa(&tmem_base), cols);
        tmem_ready();
        const uint32_t id = umma::idesc_f16(LM_M, NC, 0, 0);
        const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem), half_bytes = (uint32_t)p.half_bytes();
        bool there = false;
        for (int ti = 0; ti < my_tiles && ok; ++ti) {
            const int buf = ti % bufs;
            if (ti >= bufs) ok = ok && umma::mbar_wait_fast(sa(&b_dfree[buf]), (ti / bufs - 1) & 1);
            for (int j = (hf ^ (ti & n)) & 1; j < n && ok; j += 2) {
                const uint32_t it = (uint32_t)ti * n + j, st = it % LM_S, ph = (it / LM_S) & 1;
                if (!there) ok = ok && umma::mbar_wait_fast(sa(&b_x[st]), ph) && umma::mbar_wait_fast(sa(&b_a[st]), ph);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // asked while this chunk's products are issued
                const uint32_t nst = (it + 2) % LM_S, nph = ((it + 2) / LM_S) & 1;
                const bool nx = umma::mbar_test(sa(&b_x[nst]), nph), na = umma::mbar_test(sa(&b_a[nst]), nph);
                umma::fence_after();
                const uint64_t bd = umma::desc(xb + st * stage_bytes, 16, 1024, umma::LAYOUT_SW128);
                if (umma::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_f16_ta(tm + (2 * buf + hf) * NC, tm + t_a + 64 * st + 8 * ks,
                                   bd + (uint64_t)(((ks >> 2) * half_bytes + (ks & 3) * 32) >> 4), id, j > 1 || ks > 0);
                    umma::commit(sa(&b_free[st]));
                }
                __syncwarp();
                there = __all_sync(0xffffffffu, nx && na);
            }
            if (ok && umma::elect_one()) umma::commit(sa(&b_d[buf]));
            __syncwarp();
        }
    }
    __syncwarp();                                // two warps ran their loops in one lane
    // The last tile's results: by twenty warps where the expanding ones cannot take an older phase of its
    // barrier for this one's: in the barrier's first phase, or when their last chunks waited for products of
    // this very tile
    const bool wide = my_tiles <= bufs || n >= LM_S + 2;
    if (my_tiles > 0 && warp < LM_XW && (wide || warp >= LM_EXPAND)) {
        pdl_wait();
        store(my_tiles - 1, wide ? warp >> 2 : 0, wide ? LM_XW / 4 : 1);
    }
    if (splits > 1) {
        // block r of the cluster adds the splits up, in order, and stores every splits-th token
        pdl_wait();
        const Tile v = tile_of(first);
        const int t0 = v.t * NB, nt = min(NB, a.n_tok - t0);
        const float* mine = reinterpret_cast<const float*>(sm);
        const float* scale = DIRECT ? nullptr : reinterpret_cast<const float*>(ws + p.scales_at(a.n_groups)) + (int64_t)v.g * a.n_tok + t0;
        umma::cluster_sync();
        for (int u = tid; u < ((nt - split + splits - 1) / splits) * LM_M; u += LM_THREADS) {
            const int c = split + (u / LM_M) * splits, row = u % LM_M;
            float x = 0.0f;
            for (int s = 0; s < splits; ++s) {
                float w;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(umma::mapa(sa(mine + c * LM_M + row), s)));
                x += w;
            }
            const int m = v.m * LM_M + row;
            if (m < a.n_out) lin_store(a, t0 + c, v.g, m, (DIRECT ? x : x * scale[c]) * a.alpha);
        }
        umma::cluster_sync();                    // no block leaves while another reads its sums
    }
    if (!ok && err != nullptr) atomicExch(err, 1);
    umma::fence_before();
    __syncthreads();
    if (tid == 0) __threadfence();               // as in k_linear_few
    if (warp == LM_XW + 2) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, cols);
    }
}

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime (no link to libcuda)
typedef CUresult (*LinEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static LinEncodeFn lin_encode() {
    static const LinEncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<LinEncodeFn>(p);
    }();
    return fn;
}

namespace {
constexpr size_t LM_HEAD = 256;                  // the error word and padding

// how the rows of codes and scales may be read: 2: 64 values at a time, 1: 32, 0: 16
int lin_wide(const LinArgs& a) {
    const uintptr_t s = reinterpret_cast<uintptr_t>(a.scales);
    return a.n_in % 64 == 0 && s % 4 == 0 ? 2 : a.n_in % 32 == 0 && s % 2 == 0 ? 1 : 0;
}
int lin_planes(int x_type) { return x_type == CSA2_F32 ? 2 : 1; }

// whether the few-token kernel can take them: up to 16 tokens, 8 where x has two parts, of rows that fit a
// block's shared memory
bool lin_few(int x_type, int n_tok, int n_in) {
    return n_tok <= (x_type == CSA2_F32 ? LF_TOK / 2 : LF_TOK) && 9 * (int64_t)n_in + 32 <= LF_SMEM;
}
// In the upper half of that range it is the better one for small matrices only: below some 20 million weights
// (16 bf16 tokens, few-token kernel and the other: 1,536 x 8,192 7.6 and 8.2 us, 4,096 x 8,192 13.3 and 11.6,
// 1,536 x 32,768 16.1 and 13.3; 8 fp32 tokens, 1,536 x 1,024 5.0 and 7.7, 16 groups of 2,048 x 1,024 13.1 and 11.5)
bool lin_between(int x_type, int n_tok) { return n_tok > (x_type == CSA2_F32 ? LF_TOK / 4 : LF_TOK / 2); }
constexpr int64_t LIN_BIG = 20 << 20;
LinPrep lin_prep(int x_type, int n_tok, int n_in) {
    LinPrep p;
    p.nb = n_tok <= 32 ? 32 : n_tok <= 64 || x_type == CSA2_F32 ? 64 : 128;
    p.tiles = (n_tok + p.nb - 1) / p.nb;
    p.chunks = (n_in + LM_K - 1) / LM_K;
    p.planes = lin_planes(x_type);
    return p;
}

template <typename TX, int NT, int R>
cudaError_t lf_launch(const LinArgs& a, int x_vec, int warps, cudaStream_t st) {
    const size_t smem = std::max<size_t>((size_t)warps * a.n_tok * R * 16 * sizeof(float), R * (9 * (size_t)a.n_in + 32));
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_linear_few<TX, NT, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    // As many blocks as R tiles each need, and then as many more as there are SMs without one in the last round:
    // the SMs' shares differ by a tile, not by a block (32,768 rows: 608 blocks of 3 or 4 tiles for 512 of 4,
    // one token 8.9 us for 9.7)
    const int tiles = (a.n_out + 15) / 16;
    const int64_t need = (int64_t)((tiles + R - 1) / R) * a.n_groups;
    const int blocks = (int)std::min<int64_t>(tiles, (need + 151) / 152 * 152 / a.n_groups);
    launch_k(k_linear_few<TX, NT, R>, dim3(blocks, a.n_groups), warps * 32, smem, st, a, x_vec, tiles / blocks, tiles % blocks);
    note_launch();
    return cudaGetLastError();
}
template <typename TX, int NT>
cudaError_t lf_pick(const LinArgs& a, int x_vec, cudaStream_t st) {
    // Row tiles per block: four or two (the tokens' fragments are made once for all) when that still gives every
    // SM blocks and two of them fit an SM's shared memory, else one (one token, 4,096 x 8,192: two tiles 8.1 us,
    // one 13.2; 1,536 x 32,768: four 9.0, two 16.1)
    const int chunks = std::max(1, (a.n_in + 127) / 128);
    const int64_t tiles = (int64_t)((a.n_out + 15) / 16) * a.n_groups;
    auto fit = [&](int r) { return tiles >= 152 * r && r * (9 * a.n_in + 32) <= LF_SMEM / 2; };
    const bool four = fit(4);
    // Warps: the most, up to 8, that divide the chunks (nearly) as evenly as any number does; up to 4 with four
    // row tiles, so that four blocks stay on an SM (1,536 x 32,768, one token: 10.6 us against 13.6 with six)
    const int most = std::min(chunks, four ? 4 : LF_MAXW);
    int warps = 1;
    double best = 0.0;
    for (int w = std::min(chunks, 3); w <= most; ++w) {
        const double even = (double)chunks / ((double)w * ((chunks + w - 1) / w));
        if (even >= best - 0.02) best = std::max(best, even), warps = w;
    }
    return four     ? lf_launch<TX, NT, 4>(a, x_vec, warps, st)
           : fit(2) ? lf_launch<TX, NT, 2>(a, x_vec, warps, st)
                    : lf_launch<TX, NT, 1>(a, x_vec, warps, st);
}
template <typename TX>
cudaError_t lin_launch(const LinArgs& a, int x_type, void* wsp, cudaStream_t st) {
    const int x_vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_tok * (int64_t)sizeof(TX) % 16 == 0 &&
                      a.x_group * (int64_t)sizeof(TX) % 16 == 0;
    const bool tma = a.n_in % 32 == 0 && a.n_in > 0 && (int64_t)a.n_groups * a.n_out <= 0x7fffffff && lin_encode() != nullptr;
    // fp16 tokens need no scale: the product reads them itself where a tensor copy can (256 x 4,096 -> 8,192:
    // 16.6 us, 18.9 with a copy first)
    const LinPrep p = lin_prep(x_type, a.n_tok, a.n_in);
    CUtensorMap xm = {};
    bool direct = false;
    const bool few = lin_few(x_type, a.n_tok, a.n_in);
    const bool big = lin_between(x_type, a.n_tok) && (int64_t)a.n_groups * a.n_out * a.n_in >= LIN_BIG;
    if constexpr (std::is_same<TX, __half>::value)
        if ((!few || big) && tma && x_vec && a.x_tok > 0 && (a.n_groups == 1 || a.x_group > 0)) {
            const cuuint64_t dims[3] = {(cuuint64_t)a.n_in, (cuuint64_t)a.n_tok, (cuuint64_t)a.n_groups};
            const cuuint64_t strides[2] = {(cuuint64_t)a.x_tok * 2, (cuuint64_t)(a.n_groups == 1 ? a.x_tok : a.x_group) * 2};
            const cuuint32_t box[3] = {64, (cuuint32_t)p.nb, 1}, estr[3] = {1, 1, 1};
            direct = lin_encode()(&xm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(a.x), dims, strides, box, estr,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
        }
    // (fp16 tokens come without a workspace up to 16 of them)
    if (few && !(big && (direct || !std::is_same<TX, __half>::value))) {
        if constexpr (sizeof(TX) == 2)
            if (a.n_tok > 8) return lf_pick<TX, 2>(a, x_vec, st);
        return lf_pick<TX, 1>(a, x_vec, st);
    }
    uint8_t* ws = reinterpret_cast<uint8_t*>(wsp);
    cudaError_t e;
    if (!direct) launch_k(k_linear_x<TX>, dim3(a.n_tok, a.n_groups), 256, 0, st, a, p, ws + LM_HEAD, x_vec);
    // Splits of n_in: while the row and token tiles leave SMs idle and a split keeps four chunks
    const int tiles_m = (a.n_out + LM_M - 1) / LM_M;
    const int64_t tiles = (int64_t)tiles_m * p.tiles * a.n_groups;
    if (tiles > 0x7fffffff) return cudaErrorInvalidValue;        // y alone would be past any memory
    LinRings rg{tiles_m, 0, lin_wide(a), 0};
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= 152 && p.chunks >= splits * 2 * 4) splits *= 2, ++rg.log_splits;
    // code stages: what the token ring leaves (a tensor copy lands about 2 us after its issue)
    rg.c_stages = (int)std::min<int64_t>(LM_MAXC, (224 * 1024 - LM_S * p.stage_bytes()) / LM_CODES);
    CUtensorMap tm = {};
    if (tma) {
        const cuuint64_t dims[2] = {(cuuint64_t)(a.n_in / 2), (cuuint64_t)a.n_groups * (cuuint64_t)a.n_out};
        const cuuint64_t strides[1] = {(cuuint64_t)(a.n_in / 2)};
        const cuuint32_t box[2] = {LM_CK / 2, LM_M}, estr[2] = {1, 1};
        if (lin_encode()(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const auto kern = !tma ? k_linear_many<false, false> : direct ? k_linear_many<true, true> : k_linear_many<true, false>;
    const size_t smem = std::max<size_t>((tma ? rg.c_stages * (size_t)LM_CODES : 0) + (size_t)LM_S * p.stage_bytes(),
                                         splits > 1 ? (size_t)p.nb * LM_M * 4 : 0) + 1024;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(splits > 1 ? tiles * splits : std::min<int64_t>(tiles, 152)));
    cfg.blockDim = dim3(LM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, tm, a, p, (const uint8_t*)(ws + LM_HEAD), reinterpret_cast<int*>(ws), rg, xm);
    note_launch(direct ? 1 : 2);
    return e != cudaSuccess ? e : cudaGetLastError();
}
}  // namespace

size_t linear_fp4_ws(int x_type, int n_tok, int n_groups, int n_in) {
    if (lin_few(x_type, n_tok, n_in) && !(lin_between(x_type, n_tok) && x_type != CSA2_F16)) return 0;
    const LinPrep p = lin_prep(x_type, n_tok, n_in);
    return LM_HEAD + (size_t)p.scales_at(n_groups) + (size_t)n_groups * n_tok * sizeof(float);
}

cudaError_t launch_linear_fp4(const void* x, int x_type, int64_t x_tok, int64_t x_group, int n_tok, int n_groups,
                              int n_in, int n_out, const uint8_t* codes, const uint8_t* scales, float alpha, void* y,
                              int y_type, int64_t y_tok, int64_t y_group, void* ws, cudaStream_t st) {
    const LinArgs a{x, x_tok, x_group, n_tok, n_groups, n_in, n_out, codes, scales, alpha, y, y_type, y_tok, y_group};
    if (x_type == CSA2_BF16) return lin_launch<__nv_bfloat16>(a, x_type, ws, st);
    if (x_type == CSA2_F16) return lin_launch<__half>(a, x_type, ws, st);
    return lin_launch<float>(a, x_type, ws, st);
}

}  // namespace csa2
