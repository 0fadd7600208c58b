// Attention over every visible entry of the FP4 cache and the sliding window,
// with no index list: the form for contexts and layers that have no indexer
// ("DeepSeek-v4.1 Flash: KVキャッシュ圧縮の限界を押し広げる", §1.1: one 512-dim latent,
// key and value of every head; §2.3.1: the local window).  Per query and head:
//     s_j = scale * (q_h . L_j),  o_h = sum_j softmax_j(s) L_j,  lse_h = log sum_j exp(s_j)
// over the n = floor((p - 127) / ratio) entries before the window of raw position
// p and the window rows max(0, p - 127) .. p that are present.
//
// Work.  2 x 512 multiply-adds per head and entry against 288 bytes: with 64 heads
// 455 flop per byte, so the tensor cores bound it; with few heads the heads pad the
// MMA's 64 rows.  One block takes one (query, 64 heads, split of the entries); the
// window is a split of its own, since its bf16 rows may need a scale of their own.
// Each block leaves its running max, row sum and unnormalised output in the
// workspace; k_dense_combine joins the splits of a query.  The split count comes
// from the batch and the capacity alone (dense_splits).
//
// One block, 64-key tiles, double-buffered (L, S, P):
//   S^T = Q . L^T   (tcgen05 kind::f16, M = 64 heads, N = 64 keys, K = 512; two
//                    issuers take dims 0-255 and 256-511 into two TMEM partials)
//   online softmax, one head and 32 keys per thread; the running max is raised, and
//   O rescaled in TMEM, only when a score rises more than 2^8 above it; row sums in fp32
//   O^T += L^T . P  (M = 4 x 128 dims, N = 64 heads, K = 64 keys; two issuers)
// Warps: 0-7 softmax and epilogue, 8-9 score MMAs, 10-11 value MMAs, 12-19 load the
// FP4 rows and expand them to fp16 (exact: an E2M1 value times an E4M3 scale has at
// most 6 significant bits and lies in [2^-10, 2688]).
//
// Roundings: scores and sums fp32; P in fp16 (2^-11 of each weight, the tensor
// cores' operand type), as in the sparse attention; q exact in fp16 after a
// power-of-two scale per head, the window rows after one per window.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "fp4_f16.cuh"
#include "umma.cuh"

namespace csa2 {

constexpr int DA_TILE = 64;                          // keys per tile
constexpr int DA_H = 64;                             // heads per block
constexpr int DA_THREADS = 640;
constexpr int DA_SMW = 8;                            // softmax warps 0-7
constexpr int DA_SMT = DA_SMW * 32;
constexpr int DA_MMA1 = 8;                           // warps 8, 9: score MMAs
constexpr int DA_MMA2 = 10;                          // warps 10, 11: value MMAs
constexpr int DA_LOADW = 12;                         // warps 12-19: rows
constexpr int DA_LOADERS = 256;
constexpr uint32_t DA_SLAB = 64 * 128;               // 64 rows x 64 dims fp16, 128-byte swizzle
constexpr uint32_t DA_SQ = 0;                        // Q: 8 slabs
constexpr uint32_t DA_SL = 8 * DA_SLAB;              // L: 2 buffers x 8 slabs
constexpr uint32_t DA_LBUF = 8 * DA_SLAB;
constexpr uint32_t DA_SP = DA_SL + 2 * DA_LBUF;      // P^T: 2 buffers
constexpr uint32_t DA_PBUF = DA_H * 128;
constexpr uint32_t DA_RED = DA_SP + 2 * DA_PBUF;     // [2 key halves][64 heads]
constexpr uint32_t DA_MISC = DA_RED + 512;           // m_run[64], fac[64], qexp[64], flag[8], wmax
constexpr uint32_t DA_DYN = DA_MISC + 1024 + 1024;   // + alignment
constexpr uint32_t DAT_S = 0, DAT_O = 256, DAT_COLS = 512;
constexpr float DA_LAZY = 8.0f;                      // log2 headroom before the running max is raised

__device__ __forceinline__ uint32_t da_swz(uint32_t row, uint32_t chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

struct DenseArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    int capacity, ratio;
    const uint16_t* q;
    int n_q, n_heads, hgroups;
    const int64_t* q_pos;
    const uint16_t* swa;
    const int64_t* swa_pos0;
    int swa_len;
    float scale_log2e;
    int64_t query0;              // first query of this pass (b * n_q + i)
    int n_items, splits;         // (query, head group) pairs of this pass
    float* part_o;               // [item][splits + 1][64][512]
    float2* part_ml;             // [item][splits + 1][64] running max (log2) and row sum
    int* err;
};

__device__ __forceinline__ int64_t da_visible(int64_t p, int ratio, int capacity) {
    const int64_t n = p >= WINDOW - 1 ? (p - (WINDOW - 1)) / ratio : 0;
    return n < capacity ? n : capacity;
}

__global__ void __launch_bounds__(DA_THREADS, 1) k_dense_attn(const DenseArgs a) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) unsigned long long b_lhalf[2], b_lfull[2], b_lfree[2], b_sfull[2], b_sfree[2], b_pfull[2],
        b_odone[2];
    __shared__ uint32_t tmem_base;
    pdl_wait();                  // q, the positions and the window may come from the preceding kernel
    pdl_launch_next();

    const uint32_t raw = umma::smem_u32(dyn);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* sm = dyn + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto sa = [&](const void* x) { return umma::smem_u32(x); };

    // this block's work: FP4 splits first, then the windows
    const int64_t n_fp4 = (int64_t)a.n_items * a.splits;
    const bool window = (int64_t)blockIdx.x >= n_fp4;
    const int item = window ? (int)(blockIdx.x - n_fp4) : (int)(blockIdx.x / a.splits);
    const int split = window ? a.splits : (int)(blockIdx.x % a.splits);
    const int64_t gq = a.query0 + item / a.hgroups;
    const int h0 = (item % a.hgroups) * DA_H, nh = min(DA_H, a.n_heads - h0);
    const int b = (int)(gq / a.n_q);
    const int64_t p = a.q_pos[gq];
    int64_t row0 = 0;            // first row of this split, and how many
    int rows = 0;
    if (window) {
        const int64_t s0 = a.swa_pos0 != nullptr ? a.swa_pos0[b] : 0;
        const int64_t lo = max(max((int64_t)0, p - (WINDOW - 1)), s0), hi = min(p, s0 + a.swa_len - 1);
        rows = hi >= lo ? (int)(hi - lo + 1) : 0;
        row0 = lo - s0;
    } else {
        const int64_t n = da_visible(p, a.ratio, a.capacity), tiles = (n + DA_TILE - 1) / DA_TILE;
        row0 = tiles * split / a.splits * DA_TILE;
        const int64_t end = min(n, tiles * (split + 1) / a.splits * DA_TILE);
        rows = (int)max((int64_t)0, end - row0);
    }
    const int T = (rows + DA_TILE - 1) / DA_TILE;
    const int64_t part = ((int64_t)item * (a.splits + 1) + split) * DA_H;
    if (T == 0) {                // nothing here: an empty share, which the combine skips
        if (tid < DA_H) a.part_ml[part + tid] = make_float2(-INFINITY, 0.0f);
        return;
    }

    float* red = reinterpret_cast<float*>(sm + DA_RED);
    float* m_run = reinterpret_cast<float*>(sm + DA_MISC);
    float* fac = m_run + DA_H;
    int* qexp = reinterpret_cast<int*>(fac + DA_H);
    int* flag = qexp + DA_H;
    unsigned int* wmax = reinterpret_cast<unsigned int*>(flag + 8);

    // FP4 rows: a tile is 64 rows x 16 units of 32 dims (16 bytes of codes, 2 of scales); the first one is
    // fetched before anything else is set up
    const int lt = tid - DA_LOADW * 32;
    const uint8_t* codes = a.codes + ((int64_t)b * a.capacity + row0) * (D_LAT / 2);
    const uint8_t* scales = a.scales + ((int64_t)b * a.capacity + row0) * (D_LAT / 16);
    constexpr int NU = DA_TILE * 16 / DA_LOADERS;
    // unit u: a warp takes 4 rows x 8 units, so that a load touches whole 128-byte lines and the
    // 8 threads of a quarter warp write different bank groups; units below 512 hold dims 0-255
    auto unit_rc = [](int u, int& r, int& c) {
        const int qq = u >> 5, l = u & 31;
        r = 4 * (qq & 15) + (l & 3);
        c = 8 * (qq >> 4) + (l >> 2);
    };
    uint4 cw[NU];
    uint32_t sc[NU];
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            int r, c;
            unit_rc(lt + i * DA_LOADERS, r, c);
            cw[i] = make_uint4(0, 0, 0, 0);      // rows past the end expand to zeros
            sc[i] = 0u;
            const int j = t * DA_TILE + r;
            if (j < rows) {
                cw[i] = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)j * (D_LAT / 2)) + c);
                sc[i] = __ldg(reinterpret_cast<const uint16_t*>(scales + (int64_t)j * (D_LAT / 16)) + c);
            }
        }
    };
    if (warp >= DA_LOADW && !window) fetch(0);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(sa(&b_lhalf[i]), DA_LOADERS / 32);
            umma::mbar_init(sa(&b_lfull[i]), DA_LOADERS / 32);
            umma::mbar_init(sa(&b_lfree[i]), 2);
            umma::mbar_init(sa(&b_sfull[i]), 2);
            umma::mbar_init(sa(&b_sfree[i]), DA_SMW);
            umma::mbar_init(sa(&b_pfull[i]), DA_SMW);
            umma::mbar_init(sa(&b_odone[i]), 2);
        }
        umma::fence_mbar_init();
        *wmax = 0u;
    }
    if (tid < DA_H) m_run[tid] = -INFINITY;
    if (warp == DA_LOADW - 1) umma::tmem_alloc(sa(&tmem_base), DAT_COLS);
    // ---- Q: heads h0 .. h0+63 (zero rows past n_heads), bf16 -> fp16 slabs, by warps 0-11; a head whose
    // largest magnitude lies outside [2^-10, 2^15) is scaled by a power of two on the way
    if (warp < DA_LOADW) {
        const uint4* qsrc = reinterpret_cast<const uint4*>(a.q + (gq * a.n_heads + h0) * D_LAT);
        constexpr int HPW = (DA_H + DA_LOADW - 1) / DA_LOADW;
        uint4 qv[HPW][2];
#pragma unroll
        for (int r = 0; r < HPW; ++r) {
            const int h = warp + DA_LOADW * r;
            qv[r][0] = qv[r][1] = make_uint4(0, 0, 0, 0);
            if (h < nh) {
                qv[r][0] = qsrc[h * 64 + lane];
                qv[r][1] = qsrc[h * 64 + 32 + lane];
            }
        }
#pragma unroll
        for (int r = 0; r < HPW; ++r) {
            const int h = warp + DA_LOADW * r;
            if (h < DA_H) {
                const uint32_t mx = __reduce_max_sync(0xffffffffu, max(bf16_absmax8(qv[r][0]), bf16_absmax8(qv[r][1])));
                const int e = f16_range_exp(mx);
                const float d = pow2f(-e);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int c = lane + 32 * hh;
                    *reinterpret_cast<uint4*>(sm + DA_SQ + (c >> 3) * DA_SLAB + da_swz(h, c & 7)) =
                        bf16x8_to_f16x8(qv[r][hh], d);
                }
                if (lane == 0) qexp[h] = e;
            }
        }
        umma::fence_proxy_async();
        umma::fence_before();
    }
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;

    if (warp >= DA_LOADW) {
        if (window) {
            // ================= window rows: bf16, one scale for all of them
            const uint4* src = reinterpret_cast<const uint4*>(a.swa + ((int64_t)b * a.swa_len + row0) * D_LAT);
            uint32_t mx = 0u;
            for (int u = lt; u < rows * 64; u += DA_LOADERS) mx = max(mx, bf16_absmax8(src[u]));
            mx = __reduce_max_sync(0xffffffffu, mx);
            if (lane == 0) atomicMax(wmax, mx);
            umma::bar_named(2, DA_LOADERS);
            const float d = pow2f(-f16_range_exp(*reinterpret_cast<volatile unsigned int*>(wmax)));
            for (int t = 0; t < T; ++t) {              // at most two tiles: no buffer is used twice
                uint8_t* L = sm + DA_SL + t * DA_LBUF;
                for (int u = lt; u < DA_TILE * 64; u += DA_LOADERS) {
                    const int r = u >> 6, c = u & 63;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (t * DA_TILE + r < rows) v = src[t * DA_TILE * 64 + u];
                    *reinterpret_cast<uint4*>(L + (c >> 3) * DA_SLAB + da_swz(r, c & 7)) = bf16x8_to_f16x8(v, d);
                }
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    umma::mbar_arrive(sa(&b_lhalf[t]));
                    umma::mbar_arrive(sa(&b_lfull[t]));
                }
            }
        } else {
            // ================= FP4 rows
            for (int t = 0; t < T; ++t) {
                const int buf = t & 1;
                uint8_t* L = sm + DA_SL + buf * DA_LBUF;
                if (t > 0) fetch(t);
                if (lt < DA_TILE && (t + 1) * DA_TILE + lt < rows) {
                    const int64_t j = (t + 1) * DA_TILE + lt;
                    umma::prefetch_l2(codes + j * (D_LAT / 2));
                    umma::prefetch_l2(codes + j * (D_LAT / 2) + 128);
                    if ((lt & 3) == 0) umma::prefetch_l2(scales + j * (D_LAT / 16));
                }
                if (t >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_lfree[buf]), ((t >> 1) - 1) & 1);
#pragma unroll
                for (int i = 0; i < NU; ++i) {
                    int r, c;
                    unit_rc(lt + i * DA_LOADERS, r, c);
                    const uint32_t words[4] = {cw[i].x, cw[i].y, cw[i].z, cw[i].w};
                    const __half2 sp = e4m3x2_to_f16x2(sc[i]);
                    const __half2 s_lo = __low2half2(sp), s_hi = __high2half2(sp);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int cc = c * 4 + w;
                        *reinterpret_cast<uint4*>(L + (cc >> 3) * DA_SLAB + da_swz(r, cc & 7)) =
                            e2m1x8_scaled(words[w], (w >> 1) ? s_hi : s_lo);
                    }
                    if (i == NU / 2 - 1) {
                        umma::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(sa(&b_lhalf[buf]));
                    }
                }
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(sa(&b_lfull[buf]));
            }
        }
    } else if (warp == DA_MMA1 || warp == DA_MMA1 + 1) {
        // ================= scores of tile t once its dims are expanded and the softmax has read tile t-2's
        if (lane == 0) {
            const int half = warp - DA_MMA1;
            const uint32_t id = umma::idesc_f16(64, DA_TILE, 0, 0);
            const uint64_t qd = umma::desc(base + DA_SQ, 16, 1024, umma::LAYOUT_SW128);
            unsigned long long* ready = half == 0 ? b_lhalf : b_lfull;
            for (int t = 0; t < T && ok; ++t) {
                const int buf = t & 1;
                ok = ok && umma::mbar_wait_fast(sa(&ready[buf]), (t >> 1) & 1);
                if (t >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_sfree[buf]), ((t >> 1) - 1) & 1);
                if (!ok) break;
                umma::fence_after();
                const uint64_t ld = umma::desc(base + DA_SL + buf * DA_LBUF, 16, 1024, umma::LAYOUT_SW128);
#pragma unroll
                for (int kk = 0; kk < 16; ++kk) {
                    const int ks = 16 * half + kk;
                    const uint64_t off = (uint64_t)(((ks >> 2) * DA_SLAB + (ks & 3) * 32) >> 4);
                    umma::mma_f16(tmem + DAT_S + 64 * (2 * buf + half), qd + off, ld + off, id, kk > 0);
                }
                umma::commit(sa(&b_sfull[buf]));
            }
        }
    } else if (warp == DA_MMA2 || warp == DA_MMA2 + 1) {
        // ================= values of tile t once P is written; completion frees the L and P buffers
        if (lane == 0) {
            const int half = warp - DA_MMA2;
            const uint32_t id = umma::idesc_f16(128, DA_H, 1, 0);
            for (int t = 0; t < T && ok; ++t) {
                const int buf = t & 1;
                ok = ok && umma::mbar_wait_fast(sa(&b_pfull[buf]), (t >> 1) & 1);
                if (!ok) break;
                umma::fence_after();
                const uint64_t la = umma::desc(base + DA_SL + buf * DA_LBUF, DA_SLAB, 1024, umma::LAYOUT_SW128);
                const uint64_t pb = umma::desc(base + DA_SP + buf * DA_PBUF, 16, 1024, umma::LAYOUT_SW128);
#pragma unroll
                for (int mt = 2 * half; mt < 2 * half + 2; ++mt)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma::mma_f16(tmem + DAT_O + 64 * mt, la + (uint64_t)((2 * mt * DA_SLAB + ks * 2048) >> 4),
                                      pb + (uint64_t)((ks * 32) >> 4), id, (t > 0 || ks > 0) ? 1u : 0u);
                umma::commit(sa(&b_odone[buf]));
                umma::commit(sa(&b_lfree[buf]));
            }
        }
    } else {
        // ================= softmax: lane l of warp w has head 16(w%4) + l/4 + 8(l%2) and, of keys
        // 32(w/4) .. +31, those of parity (l/2)%2 (the 16x64b TMEM shape)
        const int qd = warp & 3, half = warp >> 2;
        const int h = qd * 16 + (lane >> 2) + 8 * (lane & 1);
        const int par = (lane >> 1) & 1;
        const uint32_t lane_base = tmem + ((uint32_t)(qd * 32) << 16);
        float lsum = 0.0f, mul = 0.0f;
        for (int t = 0; t < T; ++t) {
            const int buf = t & 1;
            float x[16];
            ok = ok && umma::mbar_wait_fast(sa(&b_sfull[buf]), (t >> 1) & 1);
            umma::fence_after();
            {
                float x1[16];
                umma::tmem_ld16x64b_x16(lane_base + DAT_S + 64 * (2 * buf) + 32 * half, x);
                umma::tmem_ld16x64b_x16(lane_base + DAT_S + 64 * (2 * buf + 1) + 32 * half, x1);
                umma::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] += x1[i];
            }
            umma::fence_before();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(sa(&b_sfree[buf]));
            // the scores times scale and this head's and the window's powers of two (known once tile 0 is in)
            if (t == 0 && window) ok = ok && umma::mbar_wait_fast(sa(&b_lfull[0]), 0);
            if (t == 0)
                mul = a.scale_log2e * pow2f(qexp[h]) *
                      (window ? pow2f(f16_range_exp(*reinterpret_cast<volatile unsigned int*>(wmax))) : 1.0f);
            const float mh = m_run[h];
            const int left = rows - t * DA_TILE - 32 * half;     // valid keys of this half
            bool exceed = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = par + 2 * i < left ? x[i] * mul : -INFINITY;
                exceed |= x[i] > mh + DA_LAZY;
            }
            if (umma::bar_red_or(1, DA_SMT, exceed)) {
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) mx = fmaxf(mx, x[i]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (par == 0) red[half * DA_H + h] = mx;
                umma::bar_named(1, DA_SMT);
                if (half == 0) {
                    float f = 1.0f;
                    if (par == 0) {
                        const float mt = fmaxf(red[h], red[DA_H + h]), mo = m_run[h];
                        if (mt > -INFINITY && (mo == -INFINITY || mt > mo + DA_LAZY)) {
                            f = mo == -INFINITY ? 0.0f : umma::ex2(mo - mt);
                            m_run[h] = mt;
                        }
                        fac[h] = f;
                    }
                    const unsigned any = __ballot_sync(0xffffffffu, f != 1.0f);
                    if (lane == 0) flag[qd] = any != 0;
                }
                if (t >= 1) ok = ok && umma::mbar_wait_fast(sa(&b_odone[(t - 1) & 1]), ((t - 1) >> 1) & 1);   // O settled
                umma::bar_named(1, DA_SMT);
                umma::fence_after();
                if (t >= 1 && (flag[0] | flag[1] | flag[2] | flag[3])) {
#pragma unroll 1
                    for (int mt = 2 * half; mt < 2 * half + 2; ++mt)
#pragma unroll 1
                        for (int c = 0; c < DA_H; c += 16) {
                            float v[16];
                            umma::tmem_ld16(lane_base + DAT_O + 64 * mt + c, v);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] *= fac[c + i];
                            umma::tmem_st16(lane_base + DAT_O + 64 * mt + c, v);
                        }
                    umma::tmem_wait_st();
                }
                lsum *= fac[h];
            }
            if (t >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_odone[buf]), ((t >> 1) - 1) & 1);   // P buffer free
            const float m = m_run[h];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = (x[i] == -INFINITY || m == -INFINITY) ? 0.0f : umma::ex2_ftz(x[i] - m);
                lsum += x[i];
            }
            // row h of P^T: trade half of the values with the lane of the other parity for 16 consecutive keys
            float rv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) rv[i] = __shfl_xor_sync(0xffffffffu, par ? x[i] : x[8 + i], 2);
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __half2 hp = par ? __floats2half2_rn(rv[j], x[8 + j]) : __floats2half2_rn(x[j], rv[j]);
                w[j] = *reinterpret_cast<const uint32_t*>(&hp);
            }
            uint8_t* P = sm + DA_SP + buf * DA_PBUF;
            *reinterpret_cast<uint4*>(P + da_swz(h, 4 * half + 2 * par)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(P + da_swz(h, 4 * half + 2 * par + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
            umma::fence_proxy_async();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(sa(&b_pfull[buf]));
        }
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
        if (par == 0) red[half * DA_H + h] = lsum;
        umma::bar_named(1, DA_SMT);
        if (tid < DA_H) a.part_ml[part + tid] = make_float2(m_run[tid], red[tid] + red[DA_H + tid]);
        // ---- this block's O^T (the window's back on the common scale) to the workspace, [head][dim]
        ok = ok && umma::mbar_wait_fast(sa(&b_odone[(T - 1) & 1]), ((T - 1) >> 1) & 1);
        umma::fence_after();
        const float up = window ? pow2f(f16_range_exp(*wmax)) : 1.0f;
#pragma unroll 1
        for (int mt = 2 * half; mt < 2 * half + 2; ++mt) {
            float* dst = a.part_o + part * D_LAT + mt * 128 + qd * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < nh; c += 16) {
                float v[16];
                umma::tmem_ld16(lane_base + DAT_O + 64 * mt + c, v);
                umma::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < nh) dst[(int64_t)(c + i) * D_LAT] = ok ? v[i] * up : __int_as_float(0x7fc00000);
            }
        }
    }
    if (!ok) atomicExch(a.err, 1);
    umma::fence_before();
    __syncthreads();
    if (warp == DA_LOADW - 1) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, DAT_COLS);
    }
}

// Joins the splits of one query and head: 128 threads, four dims each.  The shares' factors are found by
// the threads side by side, then the outputs are read eight at a time.
constexpr int DA_MAX_SPLITS = 152;

template <typename TO>
__global__ void __launch_bounds__(128) k_dense_combine(const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                                                       int splits, int hgroups, int n_heads, int64_t query0,
                                                       TO* __restrict__ out, float* __restrict__ lse) {
    __shared__ float fac[DA_MAX_SPLITS + 1], wm[4], wl[4];
    __shared__ int live[DA_MAX_SPLITS + 1], n_live;
    const int64_t ql = blockIdx.x / n_heads;                      // query of this pass
    const int head = (int)(blockIdx.x - ql * n_heads);
    const int64_t first = (ql * hgroups + head / DA_H) * (splits + 1) * DA_H + head % DA_H;
    const int tid = threadIdx.x, warp = tid >> 5;
    pdl_wait();
    float2 v[2];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = tid + 128 * i;
        v[i] = s <= splits ? part_ml[first + (int64_t)s * DA_H] : make_float2(-INFINITY, 0.0f);
        if (v[i].y != 0.0f) m = fmaxf(m, v[i].x);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) wm[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
    float l = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = tid + 128 * i;
        const float f = v[i].y != 0.0f ? exp2f(v[i].x - m) : 0.0f;
        if (s <= splits) fac[s] = f;
        l = fmaf(f, v[i].y, l);
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if ((tid & 31) == 0) wl[warp] = l;
    __syncthreads();
    l = (wl[0] + wl[1]) + (wl[2] + wl[3]);
    if (warp == 0) {                                              // shares that hold an output, in order
        int n = 0;
        for (int s0 = 0; s0 <= splits; s0 += 32) {
            const bool is = s0 + tid <= splits && !(fac[s0 + tid] == 0.0f);
            const unsigned b = __ballot_sync(0xffffffffu, is);
            if (is) live[n + __popc(b & ((1u << tid) - 1u))] = s0 + tid;
            n += __popc(b);
        }
        if (tid == 0) n_live = n;
    }
    __syncthreads();
    const int n = n_live;
    float o[4] = {};
    const float4* src = reinterpret_cast<const float4*>(part_o + first * D_LAT) + tid;
    for (int s0 = 0; s0 < n; s0 += 8) {
        float4 x[8];
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = 0.0f;
            x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s0 + i < n) {
                const int s = live[s0 + i];
                f[i] = fac[s];
                x[i] = src[(int64_t)s * DA_H * (D_LAT / 4)];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[0] = fmaf(f[i], x[i].x, o[0]), o[1] = fmaf(f[i], x[i].y, o[1]);
            o[2] = fmaf(f[i], x[i].z, o[2]), o[3] = fmaf(f[i], x[i].w, o[3]);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t row = (query0 + ql) * n_heads + head;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    ElemVec<TO, 4> y;
    y.pack(o);
    y.store(out + row * D_LAT + 4 * tid);
    if (lse != nullptr && tid == 0) lse[row] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

namespace {
constexpr int DA_SMS = 152;
constexpr size_t DA_HEAD = 256;                                   // the error word and padding

// Splits of each query's entries: the count whose whole waves of blocks finish first, at about 2 us a
// tile and 5 us a block, plus the combine's reading of the shares.
int dense_splits(int64_t items, int64_t capacity) {
    const int64_t tiles = (capacity + DA_TILE - 1) / DA_TILE;
    int best = 1;
    double best_us = 1e30;
    for (int s = 1; s <= DA_MAX_SPLITS && s <= tiles; ++s) {
        const int64_t waves = (items * s + DA_SMS - 1) / DA_SMS;
        const double us = (double)waves * (2.0 * (double)((tiles + s - 1) / s) + 5.0) + 0.03 * (double)(items * s);
        if (us < best_us) best_us = us, best = s;
    }
    return best;
}
// (query, head group) pairs of one pass: the shares of a pass stay near 160 MB
int64_t dense_pass(int splits) { return std::max<int64_t>(1, 8 * DA_SMS / (splits + 1)); }

struct DensePlan {
    int hgroups, splits;
    int64_t items, pass_queries;
    size_t o_bytes, ml_bytes;
};
DensePlan dense_plan(int64_t queries, int n_heads, int64_t capacity) {
    DensePlan p;
    p.hgroups = (n_heads + DA_H - 1) / DA_H;
    p.items = queries * p.hgroups;
    p.splits = dense_splits(p.items, capacity);
    p.pass_queries = std::max<int64_t>(1, dense_pass(p.splits) / p.hgroups);
    if (p.pass_queries > queries) p.pass_queries = queries;
    const size_t rows = (size_t)p.pass_queries * p.hgroups * (p.splits + 1) * DA_H;
    p.o_bytes = rows * D_LAT * sizeof(float);
    p.ml_bytes = rows * sizeof(float2);
    return p;
}
}  // namespace

size_t dense_attn_ws(int batch, int n_q, int n_heads, int64_t capacity) {
    const DensePlan p = dense_plan((int64_t)batch * n_q, n_heads, capacity);
    return DA_HEAD + p.o_bytes + p.ml_bytes;
}

cudaError_t launch_dense_attn(const csa2_cache& c, const uint16_t* q, int n_q, int n_heads, const int64_t* q_pos,
                              const uint16_t* swa, const int64_t* swa_pos0, int swa_len, float scale, void* out,
                              int out_type, float* lse, void* ws, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_dense_attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DA_DYN);
    if (e != cudaSuccess) return e;
    const int64_t queries = (int64_t)c.batch * n_q;
    const DensePlan p = dense_plan(queries, n_heads, c.capacity);
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    DenseArgs a{c.lat_codes, c.lat_scales, c.capacity, c.ratio, q, n_q, n_heads, p.hgroups, q_pos, swa, swa_pos0, swa_len,
                scale * 1.4426950408889634f, 0, 0, p.splits, reinterpret_cast<float*>(w + DA_HEAD),
                reinterpret_cast<float2*>(w + DA_HEAD + p.o_bytes), reinterpret_cast<int*>(w)};
    for (int64_t q0 = 0; q0 < queries; q0 += p.pass_queries) {
        const int64_t nq = queries - q0 < p.pass_queries ? queries - q0 : p.pass_queries;
        a.query0 = q0;
        a.n_items = (int)(nq * p.hgroups);
        launch_k(k_dense_attn, dim3((unsigned)(a.n_items * (p.splits + 1))), DA_THREADS, DA_DYN, st, a);
        const dim3 grid((unsigned)(nq * n_heads));
        if (out_type == CSA2_F32)
            launch_k(k_dense_combine<float>, grid, 128, 0, st, a.part_o, a.part_ml, p.splits, p.hgroups, n_heads, q0,
                     reinterpret_cast<float*>(out), lse);
        else if (out_type == CSA2_F16)
            launch_k(k_dense_combine<__half>, grid, 128, 0, st, a.part_o, a.part_ml, p.splits, p.hgroups, n_heads, q0,
                     reinterpret_cast<__half*>(out), lse);
        else
            launch_k(k_dense_combine<__nv_bfloat16>, grid, 128, 0, st, a.part_o, a.part_ml, p.splits, p.hgroups, n_heads,
                     q0, reinterpret_cast<__nv_bfloat16*>(out), lse);
        note_launch(2);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace csa2
