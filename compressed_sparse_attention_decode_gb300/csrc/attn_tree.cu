// Attention of a tree of drafted tokens over the FP4 cache: what csa2_dense_attn and csa2_sparse_attn compute for
// queries in a row, for the nodes of a tree whose own rows are not in the cache yet ("DeepSeek-v4.1 Flash:
// KVキャッシュ圧縮の限界を押し広げる" §1.1: one 512-dim latent, key and value of every head; §2.3.1: the top-k entries
// and the local window).  Node i at raw position p, with the chain of its `len` last tokens that are drafted (itself
// and its ancestors), attends to
//     the entries 0 .. floor((p - 127) / ratio) - 1, or those that its index list names;
//     the committed window rows of positions max(0, p - 127) .. p - len;
//     the draft rows of its chain (at most 128, so that they always lie in the window).
//
// Every visible entry: k_tree_prep, k_tree_attn, k_tree_join.  The nodes of a sequence see the same entries but for the
// last few, so their (node, head) rows are one matrix against the same keys: 4 x 512 flop per row and entry, 2,048
// per byte of an entry and row.  The tensor cores bound it, and what feeds them is shared memory.
//
// Work.  An item is 128 consecutive rows of a sequence, worked on by a pair of CTAs with 64 rows each (tcgen05
// cta_group::2); its units are its 128-key tiles: the committed window rows and the drafts first (at most 255 rows,
// two tiles), then the entries.  Pair i takes the i-th even part of all units; an item that several pairs
// share leaves each one's reference, row sums and unnormalised output in the workspace, and k_tree_join joins
// them; all others are stored by their pair.
//
// One tile, CTA r of the pair:
//   S = Q . L^T   M = 128 rows (64 from each CTA), N = 128 keys (64 from each CTA), K = 512 dims: a CTA expands its own
//                 64 keys alone, so a key's fp16 row is made once for 128 rows
//   softmax       a row has four threads, 32 keys each; weights against a reference that is raised, and O rescaled in
//                 TMEM, only when a score rises far above it
//   O += P . V    M = 128 rows, N = 2 x 256 dims, K = 128 keys.  Each CTA brings half of every N: dims 128 r .. + 127 and
//                 256 + 128 r .. + 127 of all 128 keys.  Half of that are its own keys, where they are; the other CTA's
//                 keys' dims it expands itself, over those dims of its own keys that only S needed: slab s of 64 dims
//                 goes to place s ^ 2, which gives both CTAs the same address for the same keys, as the MMA asks.
// Rows, running maxima, sums and outputs of a row stay in its CTA: the pair shares nothing but the MMAs.
//
// Roundings: entries are exact in fp16, window rows and queries to 2^-22 of a row's largest magnitude (tree_prep.cu); scores, sums
// and outputs fp32.
// The weights are fp16 (2^-11 of each) where the output is of 16 bits, and two fp16 parts (2^-22) where it is fp32, which
// doubles the value MMAs; both parts then take the two P buffers, and P waits for the values of the tile before.  An fp32
// output's sums are also taken out of the tensor cores every few tiles (TR_RUN).
#include <algorithm>
#include <type_traits>

#include "attn_join.cuh"
#include "common.cuh"
#include "elem.cuh"
#include "fp4_f16.cuh"
#include "tree.cuh"
#include "umma.cuh"

namespace csa2 {

// ---------------------------------------------------------------- every visible entry

constexpr int TR_TILE = 128;                         // keys per tile, 64 of each CTA
constexpr int TR_ROWS = 128;                         // rows of an item, 64 of each CTA
constexpr int TR_THREADS = 768;
constexpr int TR_SMW = 8, TR_SMT = TR_SMW * 32;      // warps 0-7: softmax, epilogue
constexpr int TR_MMA1 = 8, TR_MMA2 = 9;              // warps 8 and 9 of CTA 0: score MMAs, value MMAs
constexpr int TR_QW = 10;                            // a thread of warp 10: the queries of the next item
constexpr int TR_OWNW = 12, TR_OWN = 256;            // warps 12-19: a CTA's own keys
constexpr int TR_FORW = 20, TR_FOR = 128;            // warps 20-23: the other CTA's keys, this CTA's dims
constexpr uint32_t TR_SLAB = 64 * 128;               // 64 rows or keys x 64 fp16, 128-byte swizzle
constexpr uint32_t TR_SQ = 0;                        // Q: 8 slabs
constexpr uint32_t TR_SL = 8 * TR_SLAB;              // L: 2 buffers x 8 slabs
constexpr uint32_t TR_LBUF = 8 * TR_SLAB;
constexpr uint32_t TR_SP = TR_SL + 2 * TR_LBUF;      // P: 2 buffers x 2 slabs (64 keys each)
constexpr uint32_t TR_PBUF = 2 * TR_SLAB;
constexpr uint32_t TR_DYN = TR_SP + 2 * TR_PBUF + 1024;                  // + alignment
constexpr uint32_t TRT_S = 0, TRT_RUN = 128, TRT_O = 256, TRT_COLS = 512;   // S of buffer b at TRT_S + 64 b
// Weights are 2^(score - m), m a whole number TR_UP below the largest score's when it was set, and raised when one is more than
// TR_TOP above it: the largest weight lies in [2^7, 2^15], within fp16's range, and fp16's last place (of both parts together, if
// there are two) is 2^-32 of it at most.  Where the output is fp32 a run has an m of its own, so that this counts against the
// largest weight of 384 keys (against that of all, a million keys 22 nats below one lost their 2e-4 of the output).
constexpr float TR_UP = 7.0f, TR_TOP = 15.0f;
// Tiles of a run of sums for an fp32 output: a tensor-core sum loses some 2^-26 of itself at each 16-key step, always to zero's
// side (200,000 entries: 5.4e-6 of the output, a million 2.6e-5), so that after 48 steps it is added to fp32 sums (6.6e-7 after 32
// steps, 8.9e-7 after 48, 1.1e-6 after 64), half of them in the columns of TMEM that are free, half in global memory, where they
// stay in L2.  16 sequences of 32K positions take 564 us in one run and 762 in runs of three tiles;
// with all sums in global memory 820, 921 in runs of two and 744 of four.
constexpr int TR_RUN = 3;
constexpr int TR_PAIRS = 76;                         // pairs of CTAs at most: one CTA per SM
// Units of an item beside its tiles: its queries and its epilogue, some 12,000 clocks, and a tile 3,600 (ragged-7x21: 55.5 us with one,
// 50.8 with two, 45.9 with three or four; 20 ragged sequences of up to 3,000 positions 63.9, 52.9, 51.1 and 51.3)
constexpr int TR_OVER = 3;

// (d0, d1) += (a0, a1), one packed instruction
__device__ __forceinline__ void add2_rn(float& d0, float& d1, float a0, float a1) {
    asm("{\n .reg .b64 ra, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rd, {%0, %1};\n add.rn.f32x2 rd, rd, ra;\n"
        " mov.b64 {%0, %1}, rd;\n}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// an item that several pairs share: the slot of its first share, and how many there are
struct TreeHead {
    int b, rt, slot, n;
};
struct TreeArgs {
    const uint8_t *codes, *scales;
    int batch, capacity;
    int n_q, n_heads;
    float scale_log2e;
    void* out;
    float* lse;
    TreeNodes t;
    TreeHead* heads;             // [pairs]
    float* part_o;               // [2 pairs][128][512]
    float2* part_ml;             // [2 pairs][128] reference (log2) and row sum
    int* err;
};

__device__ __forceinline__ int tr_tiles(const TreeSeq& s) {
    return (s.n_rows + TR_TILE - 1) / TR_TILE + (int)(((unsigned)s.n_vis + TR_TILE - 1) / TR_TILE);
}

// Where a pair stands in its part of all units, and the share that comes next.  (32 bits: a cache that fills the memory has
// 7.6 million tiles of entries, times 128 items a sequence.)
struct TreeCursor {
    int left, off, b;            // units left, the next one's place among its sequence's
};
struct TreeShare {
    int b, rt, t0, t1, T, wt;    // tiles t0 .. t1-1 of the item's T, of which the first wt are window rows and drafts
};
__device__ __forceinline__ bool tr_next(const TreeArgs& a, TreeCursor& c, TreeShare& h) {
    while (c.left > 0) {
        const TreeSeq* s = a.t.seq + c.b;
        h.wt = (s->n_rows + TR_TILE - 1) / TR_TILE;
        h.T = tr_tiles(*s);
        const int per = h.T + TR_OVER;
        if (c.off >= s->row_tiles * per) {
            ++c.b, c.off = 0;
            continue;
        }
        h.b = c.b;
        h.rt = (int)((unsigned)c.off / (unsigned)per);
        h.t0 = c.off - h.rt * per;
        const int n = min(per - h.t0, c.left);
        h.t1 = min(h.t0 + n, h.T);
        c.left -= n, c.off += n;
        if (h.t1 > h.t0) return true;
    }
    return false;
}

template <typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(TR_THREADS, 1) k_tree_attn(const __grid_constant__ TreeArgs a) {
    constexpr bool FINE = std::is_same<TO, float>::value;           // weights in two parts
    extern __shared__ uint8_t dyn[];
    // in CTA 0, counting warps of both CTAs: dims 0-255 of a tile's keys ready, all of them, the other CTA's keys ready, P
    // written, the queries staged.  In each CTA, arrived on by the MMAs: scores done, values of dims 0-255
    // done (their places are free), all values done
    __shared__ __align__(8) unsigned long long b_half[2], b_full[2], b_for[2], b_pfull[2], b_q, b_sfull[2], b_ohalf[2],
        b_odone[2], b_qfree, b_qhere;
    __shared__ uint32_t tmem_base;
    __shared__ float red_l[256];
    __shared__ int64_t wsum[TR_THREADS / 32];
    __shared__ int start_b, start_off, part_each, part_more;
    const uint32_t raw = umma::smem_u32(dyn), base = (raw + 1023u) & ~1023u;
    uint8_t* sm = dyn + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = umma::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    auto sa = [&](const void* x) { return umma::smem_u32(x); };
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(sa(&b_half[i]), 2 * TR_OWN / 32);
            umma::mbar_init(sa(&b_full[i]), 2 * TR_OWN / 32);
            umma::mbar_init(sa(&b_for[i]), 2 * TR_FOR / 32);
            umma::mbar_init(sa(&b_pfull[i]), 2 * TR_SMW);
            umma::mbar_init(sa(&b_sfull[i]), 1);
            umma::mbar_init(sa(&b_ohalf[i]), 1);
            umma::mbar_init(sa(&b_odone[i]), 1);
        }
        umma::mbar_init(sa(&b_q), 2);
        umma::mbar_init(sa(&b_qfree), 1);
        umma::mbar_init(sa(&b_qhere), 1);
        umma::fence_mbar_init();
        start_b = 0, start_off = 0;
    }
    if (warp == TR_OWNW - 1) umma::tmem_alloc_pair(sa(&tmem_base), TRT_COLS);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    umma::cluster_sync();        // the other CTA's barriers are there
    const uint32_t tmem = tmem_base;
    pdl_wait();
    pdl_launch_next();

    // ---- this pair's part of all units: a sum over the sequences, each thread taking consecutive ones
    const int per = (a.batch + TR_THREADS - 1) / TR_THREADS;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    auto units = [&](int b) {
        const TreeSeq s = a.t.seq[b];
        return (int64_t)s.row_tiles * (tr_tiles(s) + TR_OVER);
    };
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += units(b);
    int64_t upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) wsum[warp] = upto;
    __syncthreads();
    int64_t total = 0;
    for (int i = 0; i * per * 32 < a.batch; ++i) {                   // warps that have sequences
        if (i < warp) upto += wsum[i];
        total += wsum[i];
    }
    // total % pairs of the parts have one unit more than the others, and come first
    const int64_t each = total < 0x7fffffff ? (int64_t)((unsigned)total / (unsigned)pairs) : total / pairs;
    const int64_t more = total - each * pairs;
    const int64_t u0 = each * pair + min((int64_t)pair, more);
    const int n_units = (int)each + (pair < more ? 1 : 0);
    if (tid == 0) {
        part_each = (int)each, part_more = (int)more;
        if (rank == 0) a.heads[pair] = TreeHead{0, 0, 0, 0};
    }
    {
        int64_t s = upto - mine;
        if (n_units > 0 && s <= u0 && u0 < upto)
            for (int b = b0; b < b1; ++b) {
                const int64_t n = per == 1 ? mine : units(b);
                if (u0 < s + n) {
                    start_b = b, start_off = (int)(u0 - s);
                    break;
                }
                s += n;
            }
    }
    __syncthreads();
    TreeCursor cur{n_units, start_off, start_b};
    TreeShare h{};
    bool ok = true;
    uint32_t tb = 0;                                 // tiles done so far: the rings go on from share to share

    if (warp >= TR_OWNW) {
        // ================= rows.  A unit is 32 dims of a key: 16 bytes of codes, 2 of scales.
        auto load = [&](const uint8_t* codes, const uint8_t* scales, int j, int n, int c, uint4& w, uint32_t& s) {
            w = make_uint4(0u, 0u, 0u, 0u), s = 0u;              // keys past the end expand to zeros
            if (j < n) {
                w = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)j * (D_LAT / 2)) + c);
                s = __ldg(reinterpret_cast<const uint16_t*>(scales + (int64_t)j * (D_LAT / 16)) + c);
            }
        };
        auto expand = [&](uint8_t* L, int r, int c, int flip, const uint4& w, uint32_t s) {
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
            const __half2 sp = e4m3x2_to_f16x2(s);
            const __half2 s_lo = __low2half2(sp), s_hi = __high2half2(sp);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int cc = 4 * c + k;
                *reinterpret_cast<uint4*>(L + ((cc >> 3) ^ flip) * TR_SLAB + tree_swz(r, cc & 7)) =
                    e2m1x8_scaled(words[k], (k >> 1) ? s_hi : s_lo);
            }
        };
        // row v of the window rows and drafts, 8 dims at chunk cc, to dst
        auto copy_row = [&](int v, int cc, uint8_t* dst) {
            const bool there = v < a.t.seq[h.b].n_rows;
            copy16(sa(dst), a.t.rows16 + ((int64_t)h.b * a.t.row_stride + (there ? v : 0)) * D_LAT + 8 * cc, there);
        };
        // each thread orders its own writes for the tensor core, then one arrival per warp, in CTA 0
        auto arrive = [&](unsigned long long* bar) {
            umma::fence_proxy_async();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive_pair(umma::mapa(sa(bar), 0));
        };
        const int kr = lane & 3, ku = lane >> 2;
        if (warp < TR_FORW) {
            // ---- this CTA's 64 keys of every tile, dims 0-255 first.  A warp takes 4 keys x 8 units at a time: whole 128-byte
            // lines of codes, and the 8 threads of a quarter warp write different bank groups
            const int lt = tid - TR_OWNW * 32, lw = warp - TR_OWNW;
            while (tr_next(a, cur, h)) {
                const int T = h.t1 - h.t0, wt = h.wt, n_vis = a.t.seq[h.b].n_vis;
                const uint8_t* codes = a.codes + (int64_t)h.b * a.capacity * (D_LAT / 2);
                const uint8_t* scales = a.scales + (int64_t)h.b * a.capacity * (D_LAT / 16);
                uint4 cw[4];
                uint32_t sc[4];
                auto fetch = [&](int t) {            // units 0, 1: dims 0-255, keys 4 lw .. and 32 + 4 lw ..; units 2, 3: the rest
                    const int j0 = (h.t0 + t - wt) * TR_TILE + 64 * (int)rank + 4 * lw + kr;
                    if (t < T && h.t0 + t >= wt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) load(codes, scales, j0 + 32 * (i & 1), n_vis, 8 * (i >> 1) + ku, cw[i], sc[i]);
                };
                fetch(0);
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t, buf = tg & 1, before = ((tg >> 1) - 1) & 1;
                    uint8_t* L = sm + TR_SL + buf * TR_LBUF;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (tg >= 2) ok = ok && umma::mbar_wait_fast(sa(half == 0 ? &b_ohalf[buf] : &b_odone[buf]), before);
                        if (h.t0 + t < wt) {
                            const int v0 = (h.t0 + t) * TR_TILE + 64 * (int)rank;
#pragma unroll 4
                            for (int i = lt; i < 64 * 32; i += TR_OWN) {
                                const int r = i >> 5, cc = 32 * half + (i & 31);
                                copy_row(v0 + r, cc, L + (cc >> 3) * TR_SLAB + tree_swz(r, cc & 7));
                            }
                            copy16_wait();
                        } else {
#pragma unroll
                            for (int i = 2 * half; i < 2 * half + 2; ++i)
                                expand(L, 32 * (i & 1) + 4 * lw + kr, 8 * half + ku, 0, cw[i], sc[i]);
                        }
                        arrive(half == 0 ? &b_half[buf] : &b_full[buf]);
                    }
                    fetch(t + 1);
                }
                tb += T;
            }
        } else {
            // ---- the other CTA's 64 keys, this CTA's 256 dims, over the dims of its own keys that only the scores needed
            const int lt = tid - TR_FORW * 32, lw = warp - TR_FORW;
            const int c = 8 * (ku >> 2) + 4 * (int)rank + (ku & 3);
            while (tr_next(a, cur, h)) {
                const int T = h.t1 - h.t0, wt = h.wt, n_vis = a.t.seq[h.b].n_vis;
                const uint8_t* codes = a.codes + (int64_t)h.b * a.capacity * (D_LAT / 2);
                const uint8_t* scales = a.scales + (int64_t)h.b * a.capacity * (D_LAT / 16);
                uint4 cw[4];
                uint32_t sc[4];
                auto fetch = [&](int t) {
                    const int j0 = (h.t0 + t - wt) * TR_TILE + 64 * (int)(rank ^ 1u) + 4 * lw + kr;
                    if (t < T && h.t0 + t >= wt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) load(codes, scales, j0 + 16 * i, n_vis, c, cw[i], sc[i]);
                };
                fetch(0);
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t, buf = tg & 1;
                    uint8_t* L = sm + TR_SL + buf * TR_LBUF;
                    ok = ok && umma::mbar_wait_fast(sa(&b_sfull[buf]), (tg >> 1) & 1);
                    if (h.t0 + t < wt) {
                        const int v0 = (h.t0 + t) * TR_TILE + 64 * (int)(rank ^ 1u);
#pragma unroll 4
                        for (int i = lt; i < 64 * 32; i += TR_FOR) {
                            const int r = i >> 5, cs = i & 31;       // this CTA's 32 chunks: 16 of dims 128 r .., 16 of 256 + 128 r ..
                            const int cc = 32 * (cs >> 4) + 16 * (int)rank + (cs & 15);
                            copy_row(v0 + r, cc, L + ((cc >> 3) ^ 2) * TR_SLAB + tree_swz(r, cc & 7));
                        }
                        copy16_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) expand(L, 16 * i + 4 * lw + kr, c, 2, cw[i], sc[i]);
                    }
                    arrive(&b_for[buf]);
                    fetch(t + 1);
                }
                tb += T;
            }
        }
    } else if (warp >= TR_QW) {
        // ================= queries: this CTA's 64 rows of the next item, once the last scores of the one before are done.
        // k_tree_prep has them as fp16 in this very layout (bf16 rows converted by the softmax warps were 5,000 clocks before an
        // item's first scores, fp16 rows copied 16 bytes at a time 4,000).  Rows that are not there hold anything: a row's scores
        // and outputs are its own.
        if (tid == TR_QW * 32) {
            const uint32_t r_q = umma::mapa(sa(&b_q), 0);
            const uint8_t* q16 = reinterpret_cast<const uint8_t*>(a.t.q16);
            const int tiles = (a.n_q * a.n_heads + TR_ROWS - 1) / TR_ROWS;
            for (uint32_t k = 0; tr_next(a, cur, h); ++k) {
                if (k > 0) ok = ok && umma::mbar_wait_fast(sa(&b_qfree), (k - 1) & 1);
                const uint8_t* src = q16 + (((int64_t)h.b * tiles + h.rt) * 2 + rank) * (8 * TR_SLAB);
                umma::mbar_arrive_expect_tx(sa(&b_qhere), 8 * TR_SLAB);
#pragma unroll 1
                for (int i = 0; i < 8; ++i) umma::bulk_g2s(base + TR_SQ + i * TR_SLAB, src + i * TR_SLAB, TR_SLAB, sa(&b_qhere));
                ok = umma::mbar_wait(sa(&b_qhere), k & 1) && ok;
                umma::mbar_arrive_pair(r_q);
            }
        }
        __syncwarp();
    } else if (warp >= TR_MMA1 && rank == 0) {
        // ================= MMAs of the pair.  The whole warp walks the tiles, so that descriptors and addresses stay in
        // uniform registers; one elected lane issues.
        const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
        auto both = [&] { return ok = __all_sync(0xffffffffu, ok); };
        if (warp == TR_MMA1) {
            // ---- scores of tile t: dims 0-255 as soon as they are expanded and the softmax has read those of tile t-2
            const uint32_t id = umma::idesc_f16(128, 128, 0, 0);
            const uint64_t qd = umma::desc(base + TR_SQ, 16, 1024, umma::LAYOUT_SW128);
            uint32_t k = 0;
            while (ok && tr_next(a, cur, h)) {
                ok = umma::mbar_wait_fast(sa(&b_q), k & 1);
                for (int t = h.t0; t < h.t1; ++t, ++tb) {
                    const uint32_t buf = tb & 1, ph = (tb >> 1) & 1;
                    const uint64_t ld = umma::desc(base + TR_SL + buf * TR_LBUF, 16, 1024, umma::LAYOUT_SW128);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && umma::mbar_wait_fast(sa(half == 0 ? &b_half[buf] : &b_full[buf]), ph);
                        if (!both()) break;
                        umma::fence_after();
                        if (umma::elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk) {
                                const int ks = 16 * half + kk;
                                const uint64_t off = (uint64_t)(((ks >> 2) * TR_SLAB + (ks & 3) * 32) >> 4);
                                umma::mma_f16_pair(tm + TRT_S + 64 * buf, qd + off, ld + off, id, ks > 0);
                            }
                            if (half == 1) umma::commit_pair(sa(&b_sfull[buf]));
                            if (half == 1 && t == h.t1 - 1) umma::commit_pair(sa(&b_qfree));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                ++k;
            }
        } else if (warp == TR_MMA2) {
            // ---- values of tile t, dims 0-255 first.  Keys 0-63 (CTA 0's) in places 4 n, 4 n + 1, keys 64-127 in the two
            // after them
            const uint32_t id = umma::idesc_f16(128, 256, 0, 1);
            while (ok && tr_next(a, cur, h)) {
                for (int t = h.t0; t < h.t1; ++t, ++tb) {
                    const uint32_t buf = tb & 1, ph = (tb >> 1) & 1;
                    ok = ok && umma::mbar_wait_fast(sa(&b_for[buf]), ph);
                    ok = ok && umma::mbar_wait_fast(sa(&b_pfull[buf]), ph);
                    if (!both()) break;
                    umma::fence_after();
                    if (umma::elect_one()) {
                        const uint64_t pd = umma::desc(base + TR_SP + (FINE ? 0 : buf) * TR_PBUF, 16, 1024, umma::LAYOUT_SW128);
                        const uint64_t vd = umma::desc(base + TR_SL + buf * TR_LBUF, TR_SLAB, 1024, umma::LAYOUT_SW128);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
#pragma unroll
                            for (int ks = 0; ks < (FINE ? 16 : 8); ++ks) {
                                const int k8 = ks & 7;               // (P's second part lies one buffer on)
                                umma::mma_f16_pair(tm + TRT_O + 128 * n,
                                                   pd + (uint64_t)(((ks >> 3) * TR_PBUF + (k8 >> 2) * TR_SLAB + (k8 & 3) * 32) >> 4),
                                                   vd + (uint64_t)(((4 * n + 2 * (k8 >> 2)) * TR_SLAB + (k8 & 3) * 2048) >> 4), id,
                                                   ((FINE ? (t - h.t0) % TR_RUN : t - h.t0) > 0 || ks > 0) ? 1u : 0u);
                            }
                            umma::commit_pair(sa(n == 0 ? &b_ohalf[buf] : &b_odone[buf]));
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp < TR_SMW) {
        // ================= softmax, outputs: a thread has one row (TMEM lane 32 (warp % 4) + lane: row lane % 64) and,
        // of the tile's keys, 64 (lane / 64) + 32 (warp / 4) .. + 31; of the row's output, 128 dims
        const int qd = warp & 3, ch = warp >> 2, kh = qd >> 1, row = 32 * (qd & 1) + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(qd * 32) << 16);
        const uint32_t r_pfull[2] = {umma::mapa(sa(&b_pfull[0]), 0), umma::mapa(sa(&b_pfull[1]), 0)};
        bool first_share = true;
        while (tr_next(a, cur, h)) {
            const int T = h.t1 - h.t0, wt = h.wt;
            const int n_rows_q = a.n_q * a.n_heads, q0 = h.rt * TR_ROWS + 64 * (int)rank;
            const bool scaled = tree_scaled(a.t, h.b, a.t.seq[h.b].n_rows);
            const int q_exp = q0 + row < n_rows_q ? a.t.q_exps[(int64_t)h.b * n_rows_q + q0 + row] : 0;
            // never zero, so that a masked score stays -inf (a score of nearly nothing for a scale of nothing), nor infinite, so that
            // nothing stays nothing
            const float mul4 = fminf(fmaxf(fabsf(a.scale_log2e) * pow2f(q_exp), 0x1p-100f), 0x1p126f);
            int vis = 0;
            const uint32_t* mask = nullptr;
            if (q0 + row < n_rows_q) {
                const int64_t node = (int64_t)h.b * a.n_q + (int)((unsigned)(q0 + row) / (unsigned)a.n_heads);
                vis = a.t.vis[node];
                mask = a.t.mask + node * 8 + 2 * kh + ch;
            }
            float m = -INFINITY, lsum = 0.0f;
            // this row's O times f
            auto scale_o = [&](float f) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                    float v[16];
                    umma::tmem_ld16(lane_base + TRT_O + 128 * ch + c, v);
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] *= f;
                    umma::tmem_st16(lane_base + TRT_O + 128 * ch + c, v);
                }
                umma::tmem_wait_st();
            };
            // FINE: the sums of the runs before this one: half of a thread's dims in TMEM and half in the share's slot of part_o, in this
            // order of its own; before them the reference that they were taken against and the sum of the weights in two parts
            // (thousands of runs may each be less than half of its last place).  The run that ends with tile t - 1 is added to them,
            // and the next one begins with no reference; the share's last one: they to it, back in TMEM.
            const int slot = 2 * pair + (first_share ? 0 : 1);
            float4* runs = reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * TR_ROWS + 64 * (int)rank) * D_LAT) + tid;
            auto add_run = [&](int t, bool last) {
                const uint32_t tp = tb + t - 1;
                const bool more = last || t > TR_RUN;
                float4 y[2][4] = {};                 // the next 16 columns' under way
                float4 of = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);    // the sums' reference, the weights' sum, what that rounded off
                if (more) of = runs[0];
                ok = ok && umma::mbar_wait_fast(sa(&b_odone[tp & 1]), (tp >> 1) & 1);
                umma::fence_after();
                const float top = fmaxf(of.x, m);
                const float held = of.x == -INFINITY ? 0.0f : umma::ex2(of.x - top), run = m == -INFINITY ? 0.0f : umma::ex2(m - top);
                const float l0 = __fmul_rn(of.y, held), l1 = __fmul_rn(lsum, run), l = __fadd_rn(l0, l1), took = __fsub_rn(l, l0);
                const float low = fmaf(of.z, held, __fadd_rn(__fsub_rn(l0, __fsub_rn(l, took)), __fsub_rn(l1, took)));
                if (!last) runs[0] = make_float4(top, l, low, 0.0f);
                lsum = last ? l + low : 0.0f, m = last ? top : -INFINITY;
                auto load = [&](int g, float4* to) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) to[i] = runs[(4 * g + i) * TR_SMT];
                };
                auto add = [&](int g, const float4* y) {
                    const uint32_t at = lane_base + TRT_O + 128 * ch + 16 * g;
                    float v[16];
                    umma::tmem_ld16(at, v);
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[4 * i] = fmaf(y[i].x, held, v[4 * i] * run), v[4 * i + 1] = fmaf(y[i].y, held, v[4 * i + 1] * run);
                        v[4 * i + 2] = fmaf(y[i].z, held, v[4 * i + 2] * run), v[4 * i + 3] = fmaf(y[i].w, held, v[4 * i + 3] * run);
                    }
                    if (last) {
                        umma::tmem_st16(at, v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            runs[(4 * g + i) * TR_SMT] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                };
                if (more) load(4, y[0]);
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    const uint32_t at = lane_base + TRT_O + 128 * ch + 16 * g, sum = lane_base + TRT_RUN + 64 * ch + 16 * g;
                    float v[16], w[16];
                    umma::tmem_ld16(at, v);
                    umma::tmem_ld16(sum, w);
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = more ? fmaf(w[i], held, v[i] * run) : v[i] * run;
                    umma::tmem_st16(last ? at : sum, v);
                }
#pragma unroll 1
                for (int g = 4; g < 8; g += 2) {
                    if (more) load(g + 1, y[1]);
                    add(g, y[0]);
                    if (more && g + 2 < 8) load(g + 2, y[0]);
                    add(g + 1, y[1]);
                }
                umma::tmem_wait_st();
            };
            // one tile, of the window or of entries (two copies, so that the entries' carries nothing of the window's)
            auto step = [&](auto is_window, int t) {
                constexpr bool window = decltype(is_window)::value;
                const uint32_t tg = tb + t, buf = tg & 1, ph = (tg >> 1) & 1;
                const int tile = h.t0 + t;
                uint32_t see = 0xffffffffu;          // which of the 32 keys this row attends to
                if constexpr (window) {
                    see = mask != nullptr ? mask[4 * tile] : 0u;
                } else {
                    const int left = vis - ((tile - wt) * TR_TILE + 64 * kh + 32 * ch);
                    if (left < 32) see = left <= 0 ? 0u : (1u << left) - 1u;
                }
                const bool fresh = FINE && !window && t > 0 && t % TR_RUN == 0;      // a run begins: O is of the one before
                if (fresh) add_run(t, false);
                float x[32];
                ok = ok && umma::mbar_wait_fast(sa(&b_sfull[buf]), ph);
                umma::fence_after();
                umma::tmem_ld16(lane_base + TRT_S + 64 * buf + 32 * ch, x);
                umma::tmem_ld16(lane_base + TRT_S + 64 * buf + 32 * ch + 16, x + 16);
                umma::tmem_wait_ld();
                // A row with an exponent e of its own enters O with its weight times 2^e.  The reference is one of these products
                // then: O stands for itself all the time, the sum takes the weights as they are, and both have their full precision
                // where rows of any size lie side by side, seen or not.
                const bool odd = window && scaled;
                const int8_t* rexp = a.t.exps + h.b * 256 + (window ? tile : 0) * TR_TILE + 64 * kh + 32 * ch;
                auto exp_of = [&](int i) { return (see >> i) & 1u ? (int)rexp[i] : 0; };     // (in masked places there may be none)
                float mul = odd ? 1.0f : mul4;
                float mx = -INFINITY;
                if (odd) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int e = exp_of(i);
                        x[i] = (see >> i) & 1u ? tree_score(x[i], fabsf(a.scale_log2e), q_exp + e) : -INFINITY;
                        mx = fmaxf(mx, x[i] + (float)e);
                    }
                } else {
                    if (see != 0xffffffffu)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((see >> i) & 1u)) x[i] = -INFINITY;
                    float m4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m4[i] = max3(max3(x[8 * i], x[8 * i + 1], x[8 * i + 2]), max3(x[8 * i + 3], x[8 * i + 4], x[8 * i + 5]),
                                     fmaxf(x[8 * i + 6], x[8 * i + 7]));
                    mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * mul;
                }
                const bool raise = umma::bar_red_or(1 + (qd & 1), TR_SMT / 2, mx - m > TR_TOP);
                // (the P buffer is free: these scores' keys were expanded after the values of the tile before in it; and S is
                // read before P is handed on, without which its buffer is not written again)
                if (FINE && t > 0) ok = ok && umma::mbar_wait_fast(sa(&b_odone[buf ^ 1]), ((tg - 1) >> 1) & 1);
                uint8_t* Pbuf = sm + TR_SP + (FINE ? 0 : buf) * TR_PBUF;
                if (raise) {
                    // [4][32] of this half of the rows, where their own P goes afterwards
                    float* red = reinterpret_cast<float*>(Pbuf + 4096 * (qd & 1)) + lane;
                    red[32 * (2 * kh + ch)] = mx;
                    umma::bar_named(1 + (qd & 1), TR_SMT / 2);
                    float mt = red[0];
#pragma unroll
                    for (int i = 1; i < 4; ++i) mt = fmaxf(mt, red[32 * i]);
                    float f = 1.0f;
                    if (mt > -INFINITY && (m == -INFINITY || mt - m > TR_TOP)) {
                        const float mn = floorf(mt) - TR_UP;     // (whole, so that exponents and factors of two are exact)
                        f = m == -INFINITY ? 0.0f : umma::ex2(m - mn);
                        m = mn;
                    }
                    lsum *= f;
                    if (t >= 1 && !fresh) {
                        ok = ok && umma::mbar_wait_fast(sa(&b_odone[buf ^ 1]), ((tg - 1) >> 1) & 1);      // O settled
                        umma::fence_after();
                        if (__any_sync(0xffffffffu, f != 1.0f)) scale_o(f);
                    }
                    umma::bar_named(1 + (qd & 1), TR_SMT / 2);        // red is read
                }
                float ref = m == -INFINITY ? 0.0f : -m;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (!odd && fabsf(ref) >= 0x1p23f) { // scores rounded as their largest was: half of its last place may be more than 2^15
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] *= mul4;
                    mul = 1.0f;
                }
                if (odd) {                           // the sum is of the weights as they are, P of what their rows need
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int e = exp_of(i);
                        x[i] = fminf(x[i] + ((float)e + ref), TR_TOP);      // (above it by a rounding at most)
                        lsum = fmaf(umma::ex2_ftz(x[i]), pow2f(-e), lsum);
                    }
                    ref = 0.0f;
                }
                uint8_t* P = Pbuf + kh * TR_SLAB;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
                    [[maybe_unused]] uint32_t low[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float d0 = ref, d1 = ref;
                        fma2_rn(d0, d1, x[8 * c + 2 * i], x[8 * c + 2 * i + 1], mul, mul);
                        d0 = umma::ex2_ftz(d0), d1 = umma::ex2_ftz(d1);
                        add2_rn(sum[2 * (i & 1)], sum[2 * (i & 1) + 1], d0, d1);
                        w[i] = f16x2_bits(d0, d1);
                        if constexpr (FINE) {
                            const float2 part = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                            low[i] = f16x2_bits(d0 - part.x, d1 - part.y);
                        }
                    }
                    *reinterpret_cast<uint4*>(P + tree_swz(row, 4 * ch + c)) = make_uint4(w[0], w[1], w[2], w[3]);
                    if constexpr (FINE)
                        *reinterpret_cast<uint4*>(P + TR_PBUF + tree_swz(row, 4 * ch + c)) = make_uint4(low[0], low[1], low[2], low[3]);
                }
                if (!odd) lsum += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                umma::fence_proxy_async();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive_pair(r_pfull[buf]);
            };
            const int T_win = max(0, min(wt - h.t0, T));
#pragma unroll 1
            for (int t = 0; t < T_win; ++t) step(std::true_type{}, t);
#pragma unroll 1
            for (int t = T_win; t < T; ++t) step(std::false_type{}, t);
            // ---- the share's end: the row's sum over its four threads, then O
            const uint32_t tl = tb + T - 1;
            ok = ok && umma::mbar_wait_fast(sa(&b_odone[tl & 1]), (tl >> 1) & 1);
            umma::fence_after();
            if (FINE && T > TR_RUN) add_run(T, true);
            red_l[64 * (2 * kh + ch) + row] = lsum;
            umma::bar_named(3, TR_SMT);
            float l = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) l += red_l[64 * i + row];
            const bool whole = T == h.T;
            const int64_t gr = (int64_t)h.b * n_rows_q + q0 + row;
            const bool there = q0 + row < n_rows_q;
            const int64_t pr = (int64_t)slot * TR_ROWS + 64 * (int)rank + row;
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            const int d0 = 256 * ch + 128 * kh;
            // 128 bytes of each of the warp's 32 rows at a time through the P buffers (both free), so that rows are stored as whole
            // lines: a thread has a row, and rows lie far apart
            auto store = [&](auto* dst, int rows, float f) {         // dst: the warp's first row, first dim
                using TD = std::remove_pointer_t<decltype(dst)>;
                constexpr int E = 16 / (int)sizeof(TD), N = 8 * E;   // elements of a piece, of a round
                uint8_t* mine = sm + TR_SP + warp * 4096;
                f = ok ? f : __int_as_float(0x7fc00000);
#pragma unroll 1
                for (int c0 = 0; c0 < 128; c0 += N) {
#pragma unroll 1
                    for (int c = 0; c < N; c += 16) {
                        float v[16];
                        umma::tmem_ld16(lane_base + TRT_O + 128 * ch + c0 + c, v);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] *= f;
#pragma unroll
                        for (int i = 0; i < 16; i += E) {
                            ElemVec<TD, E> y;
                            y.pack(v + i);
                            y.store(reinterpret_cast<TD*>(mine + lane * 128 + ((((c + i) / E) ^ (lane & 7)) << 4)));
                        }
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3), k = lane & 7;
                        const uint4 y = *reinterpret_cast<const uint4*>(mine + r * 128 + ((k ^ (r & 7)) << 4));
                        if (r < rows) *reinterpret_cast<uint4*>(dst + (int64_t)r * D_LAT + c0 + k * E) = y;
                    }
                    __syncwarp();
                }
            };
            const int wrow = 32 * (qd & 1);                          // the warp's first row
            if (!whole)
                store(a.part_o + (pr - lane) * D_LAT + d0, 32, 1.0f);
            else
                store(reinterpret_cast<TO*>(a.out) + (gr - lane) * D_LAT + d0, n_rows_q - q0 - wrow, inv);
            if (2 * kh + ch == 0) {
                if (!whole)
                    a.part_ml[pr] = make_float2(m, l);
                else if (there && a.lse != nullptr)
                    a.lse[gr] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            }
            // an item that begins here and goes on in other pairs is joined from their shares
            if (!whole && h.t0 == 0 && rank == 0 && tid == 0) {
                int n = 1;
                for (int rest = h.T - h.t1; rest > 0; ++n) rest -= part_each + (pair + n < part_more ? 1 : 0);
                a.heads[pair] = TreeHead{h.b, h.rt, slot, n};
            }
            first_share = false;
            tb += T;
            umma::fence_before();
            umma::bar_named(3, TR_SMT);              // sums, pieces and O are read
            umma::fence_after();
        }
    }
    if (!ok) atomicExch(a.err, 1);
    umma::fence_before();
    __syncthreads();
    umma::cluster_sync();
    if (warp == TR_OWNW - 1) {
        umma::fence_after();
        umma::tmem_dealloc_pair(tmem, TRT_COLS);
    }
}

// Joins the shares of an item that several pairs worked on, four dims a thread.  SPREAD 1: block (pair, four rows);
// SPREAD 4, for few items: block (item, row), four groups of 128 threads that take every fourth share.
template <typename TO, int SPREAD>
__global__ void __launch_bounds__(512) k_tree_join(const __grid_constant__ TreeArgs a, int pairs, int row_tiles) {
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    TreeHead hd{0, 0, 0, 0};
    int row;
    if (SPREAD == 1) {
        hd = a.heads[blockIdx.x];
        row = (int)blockIdx.y * 4 + (tid >> 7);
    } else {
        row = (int)blockIdx.y;
        for (int i = lane; i < pairs; i += 32) {
            const TreeHead x = a.heads[i];
            if (x.n > 0 && x.b * row_tiles + x.rt == (int)blockIdx.x) hd = x;
        }
        const unsigned who = __ballot_sync(0xffffffffu, hd.n > 0);
        const int src = who ? __ffs(who) - 1 : 0;
        hd.b = __shfl_sync(0xffffffffu, hd.b, src), hd.rt = __shfl_sync(0xffffffffu, hd.rt, src);
        hd.slot = __shfl_sync(0xffffffffu, hd.slot, src), hd.n = __shfl_sync(0xffffffffu, hd.n, src);
    }
    const int in_seq = hd.rt * TR_ROWS + row;
    if (hd.n == 0 || in_seq >= a.n_q * a.n_heads) return;
    // the first share's slot, then the first slots of the pairs after it
    auto share = [&](int s) { return (int64_t)(s == 0 ? hd.slot : ((hd.slot >> 1) + s) * 2) * TR_ROWS + row; };
    const int64_t gr = (int64_t)hd.b * a.n_q * a.n_heads + in_seq;
    join_row<TO, SPREAD>(a.part_o, a.part_ml, hd.n, share, reinterpret_cast<TO*>(a.out) + gr * D_LAT,
                         a.lse != nullptr ? a.lse + gr : nullptr);
}

// ---------------------------------------------------------------- launches

size_t tree_lists_ws(int batch, int n_q, int n_heads, int k);
cudaError_t launch_tree_lists(const csa2_cache& c, const uint16_t* q, int n_q, int n_heads, const int64_t* q_pos,
                              const int32_t* parent, const uint16_t* draft, const int32_t* idx, int k, const uint16_t* swa,
                              const int64_t* swa_pos0, int swa_len, float scale, void* out, int out_type, float* lse, void* ws,
                              cudaStream_t st);

namespace {
constexpr size_t TR_HEAD = 256;                      // the error word and padding

struct TreePlan {
    int row_tiles, pairs;
    size_t heads, o, ml;                             // bytes of the workspace's parts after the nodes'
    TreePlan(int batch, int n_q, int n_heads, int64_t capacity) {
        row_tiles = (n_q * n_heads + TR_ROWS - 1) / TR_ROWS;
        // fewer pairs where even a full cache has fewer tiles
        const int64_t tiles = (capacity + TR_TILE - 1) / TR_TILE + 2;
        pairs = (int)std::min<int64_t>(TR_PAIRS, (int64_t)batch * row_tiles * (tiles + TR_OVER));
        heads = ((size_t)pairs * sizeof(TreeHead) + 255) / 256 * 256;
        o = (size_t)2 * pairs * TR_ROWS * D_LAT * sizeof(float);
        ml = (size_t)2 * pairs * TR_ROWS * sizeof(float2);
    }
};
}  // namespace

size_t tree_attn_ws(int batch, int n_q, int n_heads, int k, int64_t capacity) {
    const size_t lists = k >= 0 ? tree_lists_ws(batch, n_q, n_heads, k) : 0;
    if (k > 0) return lists;
    const int q_rows = tree_q_rows(n_q, n_heads, true), nb = tree_pass(batch, q_rows);      // (a last pass of fewer sequences has fewer pairs, if any)
    const TreePlan p(nb, n_q, n_heads, capacity);
    return std::max(lists, TR_HEAD + tree_nodes_bytes(nb, n_q, q_rows) + p.heads + p.o + p.ml);
}

cudaError_t launch_tree_attn(const csa2_cache& c, const uint16_t* q, int n_q, int n_heads, const int64_t* q_pos,
                             const int32_t* parent, const uint16_t* draft, const int32_t* idx, int k, const uint16_t* swa,
                             const int64_t* swa_pos0, int swa_len, float scale, void* out, int out_type, float* lse, void* ws,
                             cudaStream_t st) {
    if (k >= 0)
        return launch_tree_lists(c, q, n_q, n_heads, q_pos, parent, draft, idx, k, swa, swa_pos0, swa_len, scale, out, out_type, lse,
                                 ws, st);
    auto go = [&](auto* y) {
        using TO = std::remove_pointer_t<decltype(y)>;
        cudaError_t e = cudaFuncSetAttribute(k_tree_attn<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TR_DYN);
        const int q_rows = tree_q_rows(n_q, n_heads, true), pass = tree_pass(c.batch, q_rows), rows = std::min(TR_ROWS, n_q * n_heads);
        for (int b0 = 0; b0 < c.batch && e == cudaSuccess; b0 += pass) {
            const int nb = std::min(pass, c.batch - b0);
            const int64_t n0 = (int64_t)b0 * n_q, r0 = n0 * n_heads;         // nodes and rows before the pass
            const TreePlan p(nb, n_q, n_heads, c.capacity);
            TO* o = y + r0 * D_LAT;
            float* l = lse ? lse + r0 : nullptr;
            TreeCall call{nb, c.capacity, c.ratio, n_q, n_heads, q_pos + n0, parent + n0, draft + n0 * D_LAT,
                          swa ? swa + (int64_t)b0 * swa_len * D_LAT : nullptr, swa_pos0 ? swa_pos0 + b0 : nullptr, swa_len, {},
                          q + r0 * D_LAT, scale < 0.0f, true, o, l, (int)sizeof(TO)};
            uint8_t* w = tree_nodes_take(call.t, nb, n_q, q_rows, reinterpret_cast<uint8_t*>(ws) + TR_HEAD);
            TreeArgs a{c.lat_codes + (int64_t)b0 * c.capacity * (D_LAT / 2), c.lat_scales + (int64_t)b0 * c.capacity * (D_LAT / 16), nb,
                       c.capacity, n_q, n_heads, scale * 1.4426950408889634f, o, l, call.t, nullptr, nullptr, nullptr,
                       reinterpret_cast<int*>(ws)};
            a.heads = reinterpret_cast<TreeHead*>(w);
            a.part_o = reinterpret_cast<float*>(w + p.heads);
            a.part_ml = reinterpret_cast<float2*>(w + p.heads + p.o);
            e = launch_tree_prep(call, st);
            if (e != cudaSuccess) break;
            launch_k(k_tree_attn<TO>, dim3((unsigned)(2 * p.pairs)), TR_THREADS, TR_DYN, st, a);
            // few items: many shares each, so a block per row
            const int64_t items = (int64_t)nb * p.row_tiles;
            if (items * 8 <= p.pairs)
                launch_k(k_tree_join<TO, 4>, dim3((unsigned)items, (unsigned)rows), 512, 0, st, a, p.pairs, p.row_tiles);
            else
                launch_k(k_tree_join<TO, 1>, dim3((unsigned)p.pairs, (unsigned)((rows + 3) / 4)), 512, 0, st, a, p.pairs, p.row_tiles);
            note_launch(2);
            e = cudaGetLastError();
        }
        return e;
    };
    return out_type == CSA2_F32   ? go(reinterpret_cast<float*>(out))
           : out_type == CSA2_F16 ? go(reinterpret_cast<__half*>(out))
                                  : go(reinterpret_cast<__nv_bfloat16*>(out));
}

}  // namespace csa2
