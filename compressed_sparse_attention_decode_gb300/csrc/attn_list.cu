// The nodes of drafted trees over index lists (csa2_tree_attn with k >= 0): what csa2_sparse_attn computes, with a node's
// window ending in the draft rows of its chain (attn_tree.cu has the definition; "DeepSeek-v4.1 Flash:
// KVキャッシュ圧縮の限界を押し広げる" §2.3.1).  Lists differ from node to node, so an item is one node and 64 of its heads.
//
// Work.  2 x 512 multiply-adds per head and key; 64 heads make 455 flop of a 288-byte entry, so the tensor cores bound it and
// shared memory feeds them.  An item has two units for its window (at most 128 rows) and one for each 64 slots of its list,
// known on the host; block i (one per SM) takes the i-th even part of all units, and the shares of an item that several
// blocks have are joined.  Where whole items a block are not much longer than even parts, the parts are whole items, stored
// by their block (16 x 16 nodes of 512 slots: 16.8 units a block or 2 items of 10, and no join).
//
// One tile of 64 keys, double-buffered (L, S, P):
//   S = Q . L^T     (tcgen05 kind::f16, M = 64 heads, N = 64 keys, K = 512; two issuers take dims 0-255 and 256-511 into two
//                    TMEM partials)
//   softmax         one head and 16 keys per thread, weights against a reference that is raised, and O rescaled in TMEM, only
//                   when a score rises far above it
//   O^T += L^T . P  (M = 4 x 128 dims, N = the heads in steps of 16, K = 64 keys; two issuers)
// Weights are fp16 (2^-11 of each) where the output is of 16 bits, and two fp16 parts (2^-22) where it is fp32: the value MMAs
// double, and the second part, in a P buffer of its own, waits for the values of the tile before.
// Window rows and drafts of another size than most are fp16 values of a power-of-two scale of their own (tree_prep.cu); their weights
// enter O times that scale, and references are taken from these products.
// Warps: 0-7 softmax and epilogue, 8-9 score MMAs, 10-11 value MMAs, 12-19 rows, 20-23 the queries, fetched for the next item
// while this one's last values and outputs are under way (k_tree_prep has them in fp16: converted here they were 10,000
// clocks late, mostly for their own code).  Nothing waits for a P or S buffer: a tile's keys are expanded
// only after the values of the tile before it in that buffer, which had read and written both.
#include <algorithm>
#include <type_traits>

#include "attn_join.cuh"
#include "common.cuh"
#include "elem.cuh"
#include "fp4_f16.cuh"
#include "tree.cuh"
#include "umma.cuh"

namespace csa2 {

constexpr int TL_TILE = 64, TL_H = 64;
constexpr int TL_THREADS = 768;
constexpr int TL_SMW = 8, TL_SMT = TL_SMW * 32;
constexpr int TL_MMA1 = 8, TL_MMA2 = 10, TL_LOADW = 12, TL_LOADERS = 256, TL_QW = 20, TL_QWARPS = 4;
constexpr uint32_t TL_SLAB = 64 * 128;               // 64 heads or keys x 64 fp16, 128-byte swizzle
constexpr uint32_t TL_SQ = 0;
constexpr uint32_t TL_SL = 8 * TL_SLAB, TL_LBUF = 8 * TL_SLAB;
constexpr uint32_t TL_SP = TL_SL + 2 * TL_LBUF, TL_PBUF = TL_SLAB;    // P: 2 buffers, and an fp32 output's second parts
constexpr uint32_t TL_SLOTS = TL_SP + 3 * TL_PBUF;   // the share's entries, -1 for none
constexpr uint32_t TL_DYN = TL_SLOTS + MAX_K * 4 + 1024;
constexpr uint32_t TLT_S = 0, TLT_O = 256, TLT_COLS = 512;       // S partial p of buffer b at TLT_S + 64 (2b + p)
// Weights are 2^(score - m), m a whole number TL_UP, or where the output is fp32 TL_UP32, below the largest score's when it was set,
// and raised when one is more than TL_TOP above it: the largest weight lies in [2^7, 2^16) or [2^10, 2^16), within fp16's range, and
// fp16's last place (of both parts together, if there are two) is 2^-32 or 2^-35 of it at most.  The higher m is, the more tiles
// raise it: 16 nodes of 16 sequences, 512 entries each, 64 heads take 69.3 us with 7, 69.6 with 10, 71.1 with 11, 77 with 12.
constexpr float TL_UP = 7.0f, TL_UP32 = 10.0f, TL_TOP = 15.9f;
// Tiles of a run of sums for an fp32 output, as in attn_tree.cu: 48 steps (16 nodes of 16 sequences, 512 entries each, 64 heads: 64 us in
// one run and 1.3e-6 off, 74 us and 7.6e-7 with runs of six tiles, 81 us with runs of four; 69 us since the weights' second
// part has a buffer of its own)
constexpr int TL_RUN = 6;
constexpr int TL_SMS = 152;
constexpr int TL_WIN = 2;                            // units of an item's window
static_assert(WINDOW <= TL_WIN * TL_TILE, "the window's rows have a unit per tile");

struct ListArgs {
    const uint8_t *codes, *scales;
    int capacity;
    int n_q, n_heads, hgroups;
    TreeNodes t;
    const int32_t* idx;
    int k;
    float scale_log2e;
    void* out;
    float* lse;
    int per;                     // units of an item
    int grain, each, more;       // the first `more` blocks have each + 1 grains of units, the others `each`
    float* part_o;               // [2 blocks][64][512]
    float2* part_ml;             // [2 blocks][64] reference (log2) and sum
    int* err;
    __device__ __forceinline__ int start(int b) const { return grain * (each * b + min(b, more)); }
    __device__ __forceinline__ int block_of(int u) const {           // (of grains of one unit)
        const int longer = (each + 1) * more;
        return u < longer ? (unsigned)u / (unsigned)(each + 1) : more + (int)((unsigned)(u - longer) / (unsigned)each);
    }
};

// Item i: a node, its first head, and how many window rows and drafts it attends to
struct ListItem {
    int64_t gq;
    int b, h0, rows;             // rows = 0: the node is not there
    __device__ __forceinline__ int wtiles() const { return (rows + TL_TILE - 1) / TL_TILE; }
};
__device__ __forceinline__ ListItem tl_item(const ListArgs& a, int item) {
    ListItem w;
    const int g = a.hgroups == 1 ? item : item >> 1;                 // at most 128 heads: one or two groups
    w.h0 = a.hgroups == 1 ? 0 : (item & 1) * TL_H;
    w.gq = g;
    w.b = (int)((unsigned)g / (unsigned)a.n_q);
    const uint4* m = reinterpret_cast<const uint4*>(a.t.mask + w.gq * 8);
    const uint4 x = m[0], y = m[1];
    w.rows = __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w) + __popc(y.x) + __popc(y.y) + __popc(y.z) + __popc(y.w);
    return w;
}

template <typename TO>
__global__ void __launch_bounds__(TL_THREADS, 1) k_tree_lists(const __grid_constant__ ListArgs a) {
    constexpr bool FINE = std::is_same<TO, float>::value;           // weights in two parts
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) unsigned long long b_lhalf[2], b_lfull[2], b_lfree[2], b_sfull[2], b_pfull[2], b_odone[2], b_q, b_plow;
    __shared__ float red[2][TL_H], m_run[TL_H];
    __shared__ __align__(16) float fac[TL_H], held[FINE ? TL_H : 4];     // (held: FINE's factor of what lies in part_o)
    __shared__ int any[4];
    __shared__ uint32_t slot_ok[2][2], tmem_base;
    __shared__ uint8_t wrows[2][WINDOW];                     // the rows of rows16 that a share's node attends to
    const uint32_t raw = umma::smem_u32(dyn), base = (raw + 1023u) & ~1023u;
    uint8_t* sm = dyn + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto sa = [&](const void* x) { return umma::smem_u32(x); };
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(sa(&b_lhalf[i]), TL_LOADERS / 32);
            umma::mbar_init(sa(&b_lfull[i]), TL_LOADERS / 32);
            umma::mbar_init(sa(&b_lfree[i]), 2);
            umma::mbar_init(sa(&b_sfull[i]), 2);
            umma::mbar_init(sa(&b_pfull[i]), TL_SMW);
            umma::mbar_init(sa(&b_odone[i]), 2);
        }
        umma::mbar_init(sa(&b_q), TL_QWARPS);
        umma::mbar_init(sa(&b_plow), TL_SMW);
        umma::fence_mbar_init();
    }
    if (warp == TL_LOADW - 1) umma::tmem_alloc(sa(&tmem_base), TLT_COLS);
    pdl_wait();
    pdl_launch_next();
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    uint32_t tb = 0, nq = 0;                         // tiles and shares with tiles done so far: the rings go on from share to share
    const int u1 = a.start(blockIdx.x + 1);
    int u = a.start(blockIdx.x);
    const int lt = tid - TL_LOADW * 32;

    // every warp goes through the block's shares: units t0 .. t1-1 of an item, units 0 and 1 its window's tiles
    for (int k = 0; u < u1; ++k) {
        const int item = (unsigned)u / (unsigned)a.per, t0 = u - item * a.per, t1 = min(a.per, t0 + u1 - u);
        u += t1 - t0;
        const bool loader = warp >= TL_LOADW && warp < TL_QW;
        const ListItem w = tl_item(a, item);
        uint8_t* wrow = wrows[nq & 1];
        const int wt = w.wtiles();
        // the tiles that are there, counted on: window tiles first, then the list's
        const int wa = min(t0, wt), wb = min(t1, wt), la = max(t0, TL_WIN), lb = max(t1, TL_WIN);
        const int nwt = max(0, min(wb, TL_WIN) - wa), T = w.rows == 0 ? 0 : nwt + (lb - la);
        const int nh = min(TL_H, a.n_heads - w.h0);
        if (loader) {
            // ================= rows
            const uint8_t* codes = a.codes + (int64_t)w.b * a.capacity * (D_LAT / 2);
            const uint8_t* scales = a.scales + (int64_t)w.b * a.capacity * (D_LAT / 16);
            int* slots = reinterpret_cast<int*>(sm + TL_SLOTS);
            umma::bar_named(2, TL_LOADERS);          // the slots of the share before are read
            if (nwt > 0 && T > 0) {
                // (once the softmax is done with the share before the last, which had its rows here)
                if (tb >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_lfree[tb & 1]), ((tb >> 1) - 1) & 1);
                // row lt is the node's if its bit is set: as many of its rows come before it as bits lie below
                const uint32_t* m = a.t.mask + w.gq * 8;
                const uint32_t mine = m[lt >> 5];
                int at = __popc(mine & ((1u << lane) - 1u));
                for (int i = 0; i < (lt >> 5); ++i) at += __popc(m[i]);
                if ((mine >> lane) & 1u) wrow[at] = (uint8_t)lt;
            }
            const int s0 = (la - TL_WIN) * TL_TILE;
            if (T > nwt)
                for (int j = lt; j < (T - nwt) * TL_TILE; j += TL_LOADERS) {
                    const int e = s0 + j < a.k ? a.idx[w.gq * a.k + s0 + j] : -1;
                    slots[j] = (unsigned)e < (unsigned)a.capacity ? e : -1;
                    if (j < TL_TILE && (unsigned)e < (unsigned)a.capacity) {         // (later tiles: a tile ahead)
                        umma::prefetch_l2(codes + (int64_t)e * (D_LAT / 2));
                        umma::prefetch_l2(codes + (int64_t)e * (D_LAT / 2) + 128);
                        umma::prefetch_l2(scales + (int64_t)e * (D_LAT / 16));
                    }
                }
            umma::bar_named(2, TL_LOADERS);
            constexpr int NU = TL_TILE * 16 / TL_LOADERS;
            // unit i of a tile: a warp takes 4 rows x 8 units of 32 dims, whole 128-byte lines of codes; the 8 threads of a
            // quarter warp write different bank groups; units below NU / 2 are dims 0-255
            auto unit_rc = [&](int i, int& r, int& c) {
                const int qq = (lt >> 5) + 8 * i;
                r = 4 * (qq & 15) + (lane & 3);
                c = 8 * (qq >> 4) + (lane >> 2);
            };
            for (int t = 0; t < T; ++t) {
                const uint32_t tg = tb + t, buf = tg & 1, before = ((tg >> 1) - 1) & 1;
                uint8_t* L = sm + TL_SL + buf * TL_LBUF;
                if (t < nwt) {
                    // ---- window rows and drafts
                    const int v0 = (wa + t) * TL_TILE;
                    if (tg >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_lfree[buf]), before);
                    const uint16_t* rows16 = a.t.rows16 + (int64_t)w.b * a.t.row_stride * D_LAT;
#pragma unroll
                    for (int i = 0; i < TL_TILE * 64 / TL_LOADERS; ++i) {
                        const int r = (lt >> 6) + 4 * i, c = lt & 63;
                        const bool there = v0 + r < w.rows;
                        copy16(sa(L + (c >> 3) * TL_SLAB + tree_swz(r, c & 7)), rows16 + (there ? (int)wrow[v0 + r] : 0) * D_LAT + 8 * c, there);
                    }
                    copy16_wait();
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        umma::mbar_arrive(sa(&b_lhalf[buf]));
                        umma::mbar_arrive(sa(&b_lfull[buf]));
                    }
                } else {
                    // ---- the list's entries
                    const int* sl = slots + (t - nwt) * TL_TILE;
                    uint4 cw[NU];
                    uint32_t sc[NU];
#pragma unroll
                    for (int i = 0; i < NU; ++i) {
                        int r, c;
                        unit_rc(i, r, c);
                        cw[i] = make_uint4(0u, 0u, 0u, 0u);          // empty slots expand to zeros
                        sc[i] = 0u;
                        const int e = sl[r];
                        if (e >= 0) {
                            cw[i] = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)e * (D_LAT / 2)) + c);
                            sc[i] = __ldg(reinterpret_cast<const uint16_t*>(scales + (int64_t)e * (D_LAT / 16)) + c);
                        }
                    }
                    if (lt < TL_TILE && t + 1 < T) {
                        const int e = sl[TL_TILE + lt];
                        if (e >= 0) {
                            umma::prefetch_l2(codes + (int64_t)e * (D_LAT / 2));
                            umma::prefetch_l2(codes + (int64_t)e * (D_LAT / 2) + 128);
                            umma::prefetch_l2(scales + (int64_t)e * (D_LAT / 16));
                        }
                    }
                    if (tg >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_lfree[buf]), before);
                    if (lt < TL_TILE) {
                        const uint32_t there = __ballot_sync(0xffffffffu, sl[lt] >= 0);
                        if (lane == 0) slot_ok[buf][lt >> 5] = there;
                    }
#pragma unroll
                    for (int i = 0; i < NU; ++i) {
                        int r, c;
                        unit_rc(i, r, c);
                        if (i == NU / 2) {               // dims 0-255 are done
                            umma::fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) umma::mbar_arrive(sa(&b_lhalf[buf]));
                        }
                        const uint32_t words[4] = {cw[i].x, cw[i].y, cw[i].z, cw[i].w};
                        const __half2 sp = e4m3x2_to_f16x2(sc[i]);
                        const __half2 s_lo = __low2half2(sp), s_hi = __high2half2(sp);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int cc = c * 4 + j;
                            *reinterpret_cast<uint4*>(L + (cc >> 3) * TL_SLAB + tree_swz(r, cc & 7)) =
                                e2m1x8_scaled(words[j], (j >> 1) ? s_hi : s_lo);
                        }
                    }
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(sa(&b_lfull[buf]));
                }
            }
        } else if (T > 0 || warp < TL_SMW) {
            if (warp >= TL_QW) {
                // ================= Q: heads h0 .. h0+63 (zero rows past n_heads) once the softmax of the share before is done
                if (tb > 0) ok = ok && umma::mbar_wait_fast(sa(&b_pfull[(tb - 1) & 1]), ((tb - 1) >> 1) & 1);
                const uint16_t* src = a.t.q16 + (w.gq * a.n_heads + w.h0) * D_LAT;
#pragma unroll 4
                for (int i = tid - TL_QW * 32; i < TL_H * 64; i += TL_QWARPS * 32) {
                    const int r = i >> 6, c = i & 63;
                    copy16(sa(sm + TL_SQ + (c >> 3) * TL_SLAB + tree_swz(r, c & 7)), src + (r < nh ? r : 0) * D_LAT + 8 * c, r < nh);
                }
                copy16_wait();
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(sa(&b_q));
                // the next share's queries, if it is another item's, on their way to L2 while this one runs
                if (u < u1) {
                    const int next = (unsigned)u / (unsigned)a.per;
                    const int64_t g = a.hgroups == 1 ? next : next >> 1;
                    const int nh0 = a.hgroups == 1 ? 0 : (next & 1) * TL_H;
                    const char* ahead = reinterpret_cast<const char*>(a.t.q16 + (g * a.n_heads + nh0) * D_LAT);
                    for (int i = tid - TL_QW * 32; i < min(TL_H, a.n_heads - nh0) * 8; i += TL_QWARPS * 32) umma::prefetch_l2(ahead + i * 128);
                }
                // every phase in turn, the last one at the next share: a wait tells a phase from the next by its parity alone
                for (int t = 0; t + 1 < T; ++t) ok = ok && umma::mbar_wait_fast(sa(&b_pfull[(tb + t) & 1]), ((tb + t) >> 1) & 1);
            } else if (warp >= TL_MMA1 && warp < TL_MMA2) {
                // ================= scores of tile t once its dims are expanded.  The whole warp walks the tiles, so that
                // descriptors and addresses stay in uniform registers; one elected lane issues.
                const int half = warp - TL_MMA1;
                const uint32_t id = umma::idesc_f16(64, TL_TILE, 0, 0);
                const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
                const uint64_t qd = umma::desc(base + TL_SQ, 16, 1024, umma::LAYOUT_SW128);
                ok = ok && umma::mbar_wait_fast(sa(&b_q), nq & 1);
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t, buf = tg & 1;
                    ok = ok && umma::mbar_wait_fast(sa(half == 0 ? &b_lhalf[buf] : &b_lfull[buf]), (tg >> 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    umma::fence_after();
                    const uint64_t ld = umma::desc(base + TL_SL + buf * TL_LBUF, 16, 1024, umma::LAYOUT_SW128);
                    if (umma::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 16; ++kk) {
                            const int ks = 16 * half + kk;
                            const uint64_t off = (uint64_t)(((ks >> 2) * TL_SLAB + (ks & 3) * 32) >> 4);
                            umma::mma_f16(tm + TLT_S + 64 * (2 * buf + half), qd + off, ld + off, id, kk > 0);
                        }
                        umma::commit(sa(&b_sfull[buf]));
                    }
                    __syncwarp();
                }
            } else if (warp >= TL_MMA2) {
                // ================= values of tile t once P is written; completion frees the L and P buffers
                const int half = warp - TL_MMA2;
                const uint32_t id = umma::idesc_f16(128, (nh + 15) & ~15, 1, 0);     // heads that are there, in MMA steps
                const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t, buf = tg & 1;
                    ok = ok && umma::mbar_wait_fast(sa(&b_pfull[buf]), (tg >> 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    umma::fence_after();
                    const uint64_t ld = umma::desc(base + TL_SL + buf * TL_LBUF, TL_SLAB, 1024, umma::LAYOUT_SW128);
                    // part 0 from the tile's own P buffer, FINE's second part from the third
                    auto part = [&](uint32_t pb, bool first) {
                        const uint64_t pd = umma::desc(base + TL_SP + pb * TL_PBUF, 16, 1024, umma::LAYOUT_SW128);
#pragma unroll
                        for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
                            for (int ks = 0; ks < TL_TILE / 16; ++ks) {
                                const int mt = 2 * half + m2;
                                umma::mma_f16(tm + TLT_O + 64 * mt, ld + (uint64_t)((2 * mt * TL_SLAB + ks * 2048) >> 4),
                                              pd + (uint64_t)((ks * 32) >> 4), id, (!first || ks > 0) ? 1u : 0u);
                            }
                    };
                    if (umma::elect_one()) part(buf, (FINE ? t % TL_RUN : t) == 0);
                    if (FINE) {
                        __syncwarp();
                        ok = ok && umma::mbar_wait_fast(sa(&b_plow), tg & 1);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        umma::fence_after();
                    }
                    if (umma::elect_one()) {
                        if (FINE) part(2, false);
                        umma::commit(sa(&b_lfree[buf]));
                        umma::commit(sa(&b_odone[buf]));
                    }
                    __syncwarp();
                }
            } else {
                // ================= softmax: lane l of warp w has head 16 (w % 4) + l / 4 + 8 (l % 2) and, of keys 32 (w / 4) .. + 31,
                // those of parity (l / 2) % 2 (the 16x64b TMEM shape)
                const int qd = warp & 3, half = warp >> 2;
                const int h = qd * 16 + (lane >> 2) + 8 * (lane & 1), par = (lane >> 1) & 1;
                const uint32_t lane_base = tmem + ((uint32_t)(qd * 32) << 16);
                if (tid < TL_H) {
                    m_run[tid] = -INFINITY;
                    if constexpr (FINE) held[tid] = 1.0f;
                }
                umma::bar_named(1, TL_SMT);
                const int q_exp = T > 0 && h < nh ? a.t.q_exps[w.gq * a.n_heads + w.h0 + h] : 0;
                // never zero, so that a masked score stays -inf, nor infinite, so that nothing stays nothing
                const float mul4 = fminf(fmaxf(fabsf(a.scale_log2e) * pow2f(q_exp), 0x1p-100f), 0x1p126f);
                const bool scaled = tree_scaled(a.t, w.b, a.t.seq[w.b].n_rows);
                float lsum = 0.0f;
                // FINE: the sums of the runs before this one lie in the share's slot of part_o, in this order of its own
                float4* runs = reinterpret_cast<float4*>(a.part_o + (int64_t)(2 * blockIdx.x + (k == 0 ? 0 : 1)) * TL_H * D_LAT) + tid;
                // the run that ends with tile t - 1 is added to them; the share's last one: they to it, back in TMEM
                auto add_run = [&](int t, bool last) {
                    const uint32_t tp = tb + t - 1;
                    ok = ok && umma::mbar_wait_fast(sa(&b_odone[tp & 1]), (tp >> 1) & 1);
                    umma::fence_after();
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        const uint32_t at = lane_base + TLT_O + 64 * (2 * half + (g >> 2)) + 16 * (g & 3);
                        const float* fh = held + 16 * (g & 3);
                        float v[16];
                        float4 y[4] = {};
                        if (last || t > TL_RUN)
#pragma unroll
                            for (int i = 0; i < 4; ++i) y[i] = runs[(4 * g + i) * TL_SMT];
                        umma::tmem_ld16(at, v);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[4 * i] = fmaf(y[i].x, fh[4 * i], v[4 * i]), v[4 * i + 1] = fmaf(y[i].y, fh[4 * i + 1], v[4 * i + 1]);
                            v[4 * i + 2] = fmaf(y[i].z, fh[4 * i + 2], v[4 * i + 2]), v[4 * i + 3] = fmaf(y[i].w, fh[4 * i + 3], v[4 * i + 3]);
                        }
                        if (last) {
                            umma::tmem_st16(at, v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                runs[(4 * g + i) * TL_SMT] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                    if (last) umma::tmem_wait_st();
                    umma::bar_named(1, TL_SMT);              // held is read
                    if (!last && tid < TL_H) held[tid] = 1.0f;
                };
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t, buf = tg & 1, ph = (tg >> 1) & 1;
                    if (FINE && t > 0 && t % TL_RUN == 0) add_run(t, false);
                    float x[16];
                    // what does not need the scores comes first: the loaders' words, the reference
                    ok = ok && umma::mbar_wait_fast(sa(&b_lfull[buf]), ph);
                    const bool window = t < nwt;
                    uint32_t see;                    // which of the half's 32 keys are there
                    if (window) {
                        const int left = w.rows - (wa + t) * TL_TILE - 32 * half;
                        see = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
                    } else {
                        see = *reinterpret_cast<volatile uint32_t*>(&slot_ok[buf][half]);
                    }
                    const float mh = m_run[h];
                    ok = ok && umma::mbar_wait_fast(sa(&b_sfull[buf]), ph);
                    umma::fence_after();
                    {
                        float x1[16];
                        umma::tmem_ld16x64b_x16(lane_base + TLT_S + 64 * (2 * buf) + 32 * half, x);
                        umma::tmem_ld16x64b_x16(lane_base + TLT_S + 64 * (2 * buf + 1) + 32 * half, x1);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] += x1[i];
                    }
                    // exponent of the row that key par + 2i is, 0 for none
                    auto rexp = [&](int i) {
                        return (see >> (par + 2 * i)) & 1u ? (int)a.t.exps[w.b * 256 + wrow[(wa + t) * TL_TILE + 32 * half + par + 2 * i]] : 0;
                    };
                    const bool odd = window && scaled;
                    float mx = -INFINITY;
                    if (odd) {                       // references are of the weights that O takes: times 2^(the row's exponent)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int e = rexp(i);
                            x[i] = (see >> (par + 2 * i)) & 1u ? tree_score(x[i], fabsf(a.scale_log2e), q_exp + e) : -INFINITY;
                            mx = fmaxf(mx, x[i] + (float)e);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] *= mul4;
                        if (see != 0xffffffffu)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (!((see >> (par + 2 * i)) & 1u)) x[i] = -INFINITY;
                        const auto max3 = [](float p, float q, float r) { return fmaxf(p, fmaxf(q, r)); };
                        mx = max3(max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), x[6]),
                                  max3(max3(x[7], x[8], x[9]), max3(x[10], x[11], x[12]), x[13]), fmaxf(x[14], x[15]));
                    }
                    if (umma::bar_red_or(1, TL_SMT, mx - mh > TL_TOP)) {
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        if (par == 0) red[half][h] = mx;
                        umma::bar_named(1, TL_SMT);
                        if (half == 0) {
                            float f = 1.0f;
                            if (par == 0) {
                                const float mt = fmaxf(red[0][h], red[1][h]), mo = m_run[h], mu = floorf(mt) - (FINE ? TL_UP32 : TL_UP);
                                const float mn = mt - mu > TL_TOP ? floorf(mt) : mu;     // (whole: factors are exact; beyond 2^27 not every number is there)
                                if (mt > -INFINITY && (mo == -INFINITY || mt - mo > TL_TOP)) {
                                    f = mo == -INFINITY ? 0.0f : umma::ex2(mo - mn);
                                    m_run[h] = mn;
                                }
                                fac[h] = f;
                                if constexpr (FINE) held[h] *= f;
                            }
                            const unsigned some = __ballot_sync(0xffffffffu, f != 1.0f);
                            if (lane == 0) any[qd] = some != 0;
                        }
                        if (t >= 1) ok = ok && umma::mbar_wait_fast(sa(&b_odone[buf ^ 1]), ((tg - 1) >> 1) & 1);   // O settled
                        umma::bar_named(1, TL_SMT);
                        umma::fence_after();
                        if (t >= 1 && (any[0] | any[1] | any[2] | any[3])) {
#pragma unroll 1
                            for (int mt = 2 * half; mt < 2 * half + 2; ++mt)
#pragma unroll 1
                                for (int c = 0; c < TL_H; c += 16) {
                                    float v[16];
                                    umma::tmem_ld16(lane_base + TLT_O + 64 * mt + c, v);
                                    umma::tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) v[i] *= fac[c + i];
                                    umma::tmem_st16(lane_base + TLT_O + 64 * mt + c, v);
                                }
                            umma::tmem_wait_st();
                        }
                        lsum *= fac[h];
                    }
                    const float mr = m_run[h], m = mr == -INFINITY ? 0.0f : mr;      // (a tile may have no key)
                    float sum[2] = {0.0f, 0.0f};
                    if (odd) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int e = rexp(i);
                            x[i] = umma::ex2_ftz(fminf(x[i] + ((float)e - m), TL_TOP));    // (above it by a rounding at most)
                            sum[i & 1] = fmaf(x[i], pow2f(-e), sum[i & 1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[i] = umma::ex2_ftz(x[i] - m);
                            sum[i & 1] += x[i];
                        }
                    }
                    lsum += sum[0] + sum[1];
                    // row h of P^T: trade half of the values with the lane of the other parity for 16 consecutive keys
                    float rv[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) rv[i] = __shfl_xor_sync(0xffffffffu, par ? x[i] : x[8 + i], 2);
                    uint32_t p2[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) p2[j] = par ? f16x2_bits(rv[j], x[8 + j]) : f16x2_bits(x[j], rv[j]);
                    auto put = [&](uint32_t pb) {
                        uint8_t* P = sm + TL_SP + pb * TL_PBUF;
                        *reinterpret_cast<uint4*>(P + tree_swz(h, 4 * half + 2 * par)) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                        *reinterpret_cast<uint4*>(P + tree_swz(h, 4 * half + 2 * par + 1)) = make_uint4(p2[4], p2[5], p2[6], p2[7]);
                        umma::fence_proxy_async();
                        umma::fence_before();
                        __syncwarp();
                    };
                    put(buf);
                    if (lane == 0) umma::mbar_arrive(sa(&b_pfull[buf]));
                    if constexpr (FINE) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {        // what the first part leaves
                            const float2 part = __half22float2(*reinterpret_cast<const __half2*>(&p2[j]));
                            p2[j] = par ? f16x2_bits(rv[j] - part.x, x[8 + j] - part.y) : f16x2_bits(x[j] - part.x, rv[j] - part.y);
                        }
                        if (t > 0) ok = ok && umma::mbar_wait_fast(sa(&b_odone[buf ^ 1]), ((tg - 1) >> 1) & 1);
                        put(2);
                        if (lane == 0) umma::mbar_arrive(sa(&b_plow));
                    }
                }
                // ---- the share's end: sums, then O^T as [head][dim]
                if (FINE && T > TL_RUN) add_run(T, true);
                lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
                if (par == 0) red[half][h] = lsum;
                umma::bar_named(1, TL_SMT);
                const bool whole = t1 - t0 == a.per;
                const int64_t orow = w.gq * a.n_heads + w.h0, prow = (int64_t)(2 * blockIdx.x + (k == 0 ? 0 : 1)) * TL_H;
                if (tid < TL_H) {
                    const float l = T > 0 ? red[0][tid] + red[1][tid] : 0.0f, m = T > 0 ? m_run[tid] : -INFINITY;
                    if (!whole)
                        a.part_ml[prow + tid] = make_float2(m, l);
                    else if (tid < nh && a.lse != nullptr)
                        a.lse[orow + tid] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                    fac[tid] = !whole ? 1.0f : l > 0.0f || l != l ? 1.0f / l : 0.0f;
                }
                umma::bar_named(1, TL_SMT);
                if (T > 0) {
                    const uint32_t tl = tb + T - 1;
                    ok = ok && umma::mbar_wait_fast(sa(&b_odone[tl & 1]), (tl >> 1) & 1);
                    umma::fence_after();
                    const float up = ok ? 1.0f : __int_as_float(0x7fc00000);
                    auto store = [&](auto* dst) {            // row 0's first dim
                        using TD = std::remove_pointer_t<decltype(dst)>;
                        // 16 heads of a dim tile at a time, the next ones' load under way while these are stored
                        float v[2][16];
                        const int n = (nh + 15) / 16;            // groups of 16 heads
                        auto load = [&](int g, float* to) { umma::tmem_ld16(lane_base + TLT_O + 64 * (2 * half + g / n) + 16 * (g % n), to); };
                        auto put = [&](int g, const float* x) {
                            TD* d = dst + (2 * half + g / n) * 128 + qd * 32 + lane;
                            const int c = 16 * (g % n);
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(fac + c + i);
                                const float f4[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if (c + i + j < nh) d[(c + i + j) * D_LAT] = from_f32<TD>(x[i + j] * f4[j] * up);
                            }
                        };
                        load(0, v[0]);
#pragma unroll 1
                        for (int g = 0; g < 2 * n; g += 2) {
                            umma::tmem_wait_ld();
                            load(g + 1, v[1]);
                            put(g, v[0]);
                            umma::tmem_wait_ld();
                            if (g + 2 < 2 * n) load(g + 2, v[0]);
                            put(g + 1, v[1]);
                        }
                    };
                    if (whole)
                        store(reinterpret_cast<TO*>(a.out) + orow * D_LAT);
                    else
                        store(a.part_o + prow * D_LAT);
                } else if (whole) {
                    for (int i = tid; i < nh * D_LAT; i += TL_SMT) reinterpret_cast<TO*>(a.out)[orow * D_LAT + i] = from_f32<TO>(0.0f);
                }
                umma::fence_before();
                umma::bar_named(1, TL_SMT);              // what the softmax keeps is read
            }
        }
        tb += T;
        nq += T > 0;
    }
    if (!ok) atomicExch(a.err, 1);
    umma::fence_before();
    __syncthreads();
    if (warp == TL_LOADW - 1) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, TLT_COLS);
    }
}

// Joins the shares of an item that several blocks worked on, four heads a block: block x joins the item whose units begin
// with block x of k_tree_lists and go on in the next one.
template <typename TO>
__global__ void __launch_bounds__(512) k_tree_lists_join(const __grid_constant__ ListArgs a) {
    pdl_wait();
    const int blk = blockIdx.x, bound = a.start(blk + 1), item = (unsigned)bound / (unsigned)a.per, first = item * a.per;
    const int head = (int)blockIdx.y * 4 + ((int)threadIdx.x >> 7);
    if (bound == first || first < a.start(blk)) return;
    const int64_t g = a.hgroups == 1 ? item : item >> 1;
    const int h0 = a.hgroups == 1 ? 0 : (item & 1) * TL_H;
    if (h0 + head >= a.n_heads || head >= TL_H) return;
    const int n = a.block_of(first + a.per - 1) - blk + 1, slot = 2 * blk + (first == a.start(blk) ? 0 : 1);
    auto share = [&](int s) { return (int64_t)(s == 0 ? slot : 2 * (blk + s)) * TL_H + head; };
    const int64_t row = g * a.n_heads + h0 + head;
    join_row<TO, 1>(a.part_o, a.part_ml, n, share, reinterpret_cast<TO*>(a.out) + row * D_LAT, a.lse != nullptr ? a.lse + row : nullptr);
}

namespace {
constexpr size_t TL_HEAD = 256;                      // the error word and padding

struct ListPlan {
    int hgroups, per, blocks, grain, each, more;
    ListPlan(int batch, int n_q, int n_heads, int k) {
        hgroups = (n_heads + TL_H - 1) / TL_H;
        per = TL_WIN + (k + TL_TILE - 1) / TL_TILE;
        const int items = batch * n_q * hgroups;     // at most 65,536
        blocks = std::min(TL_SMS, items * per);
        // Whole items a block where that is at most 6 units (20,000 clocks) more than an even part: about what the shares'
        // stores and the join cost with all blocks at it.  With fewer units than blocks they cost 2.4 us and 0.03 more a unit, of
        // which one takes 1.9: 10 items of 4 units 15.6 us whole and 13.2 in parts, 24 of 6 21.6 and 19.0, 38 of 4 18.4 and 19.6.
        const int units = items * per, whole = (items + blocks - 1) / blocks * per;
        grain = whole <= units / blocks + 6 && !(units <= TL_SMS && per >= 3 + units / 50) ? per : 1;
        const int grains = items * per / grain;
        blocks = std::min(blocks, grains);
        each = grains / blocks, more = grains % blocks;
    }
};
}  // namespace

size_t tree_lists_ws(int batch, int n_q, int n_heads, int k) {
    const int nb = tree_pass(batch, n_q * n_heads);
    const size_t rows = (size_t)2 * TL_SMS * TL_H;
    return TL_HEAD + tree_nodes_bytes(nb, n_q, n_q * n_heads) + rows * (D_LAT * sizeof(float) + sizeof(float2));
}

cudaError_t launch_tree_lists(const csa2_cache& c, const uint16_t* q, int n_q, int n_heads, const int64_t* q_pos,
                              const int32_t* parent, const uint16_t* draft, const int32_t* idx, int k, const uint16_t* swa,
                              const int64_t* swa_pos0, int swa_len, float scale, void* out, int out_type, float* lse, void* ws,
                              cudaStream_t st) {
    auto go = [&](auto* y) {
        using TO = std::remove_pointer_t<decltype(y)>;
        cudaError_t e = cudaFuncSetAttribute(k_tree_lists<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TL_DYN);
        const int pass = tree_pass(c.batch, n_q * n_heads);
        for (int b0 = 0; b0 < c.batch && e == cudaSuccess; b0 += pass) {
            const int nb = std::min(pass, c.batch - b0);
            const int64_t n0 = (int64_t)b0 * n_q, r0 = n0 * n_heads;         // nodes and rows before the pass
            const ListPlan p(nb, n_q, n_heads, k);
            TreeCall call{nb, c.capacity, c.ratio, n_q, n_heads, q_pos + n0, parent + n0, draft + n0 * D_LAT,
                          swa ? swa + (int64_t)b0 * swa_len * D_LAT : nullptr, swa_pos0 ? swa_pos0 + b0 : nullptr, swa_len, {},
                          q + r0 * D_LAT, scale < 0.0f, false, nullptr, nullptr, 0};
            uint8_t* w = tree_nodes_take(call.t, nb, n_q, n_q * n_heads, reinterpret_cast<uint8_t*>(ws) + TL_HEAD);
            ListArgs a{c.lat_codes + (int64_t)b0 * c.capacity * (D_LAT / 2), c.lat_scales + (int64_t)b0 * c.capacity * (D_LAT / 16),
                       c.capacity, n_q, n_heads, p.hgroups, call.t, idx ? idx + n0 * k : nullptr, k, scale * 1.4426950408889634f,
                       y + r0 * D_LAT, lse ? lse + r0 : nullptr, p.per, p.grain, p.each, p.more, nullptr, nullptr,
                       reinterpret_cast<int*>(ws)};
            a.part_o = reinterpret_cast<float*>(w);
            a.part_ml = reinterpret_cast<float2*>(w + (size_t)2 * TL_SMS * TL_H * D_LAT * sizeof(float));
            e = launch_tree_prep(call, st);
            if (e != cudaSuccess) break;
            launch_k(k_tree_lists<TO>, dim3((unsigned)p.blocks), TL_THREADS, TL_DYN, st, a);
            note_launch();
            if (p.grain == 1 && p.blocks > 1) {
                launch_k(k_tree_lists_join<TO>, dim3((unsigned)(p.blocks - 1), (unsigned)((std::min(n_heads, TL_H) + 3) / 4)), 512, 0, st, a);
                note_launch();
            }
            e = cudaGetLastError();
        }
        return e;
    };
    return out_type == CSA2_F32   ? go(reinterpret_cast<float*>(out))
           : out_type == CSA2_F16 ? go(reinterpret_cast<__half*>(out))
                                  : go(reinterpret_cast<__nv_bfloat16*>(out));
}

}  // namespace csa2
