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
// MMA's 64 rows.  Lengths are known on the device alone, so the blocks (one per SM)
// share the work there: each (query, 64 heads) is as many units as it has 64-key
// tiles, plus some for each tile of its window, and block i takes the i-th even part of
// all units.
// A part that covers several queries is worked through one after the other; a query
// that several blocks share leaves each one's reference (below), row sum and unnormalised
// output in the workspace, and k_dense_combine joins them.  The window is always a
// share of its own, since its bf16 rows may need a scale of their own.
//
// One share, 64-key tiles, double-buffered (L, S, P):
//   S^T = Q . L^T   (tcgen05 kind::f16, M = 64 heads, N = 64 keys, K = 512; two
//                    issuers take dims 0-255 and 256-511 into two TMEM partials)
//   online softmax, one head and 32 keys per thread.  Weights are taken against a reference that
//   is set 7 (in log2) below the running max, so that they use fp16's range; it is raised, and O
//   rescaled in TMEM, only when a score rises more than 15 above it; row sums in fp32
//   O^T += L^T . P  (M = 4 x 128 dims, N = the heads in steps of 16 (8 heads, 16 queries of 9K entries: 35.0 us, 36.0
//                    with N = 64), K = 64 keys; two issuers)
// What bounds a tile is shared memory: 64 KB written, 128 KB read by the score MMAs (64
// of them the query again) and 96 KB by the value MMAs, 2,250 clocks at 128 bytes a
// clock, against 3,200 measured (64 queries of 64 heads at 32K, 16,320 entries each: 206 us
// with the join, 670 TFLOP/s).  Three buffers of 48 keys, which take the buffers'
// round off the critical path, read more per key and were slower (2,700 per 48).
// Warps: 0-7 softmax and epilogue, 8-9 score MMAs, 10-11 value MMAs, 12-19 load the
// FP4 rows and expand them to fp16 (exact: an E2M1 value times an E4M3 scale has at
// most 6 significant bits and lies in [2^-10, 2688]).
//
// Roundings: scores and sums fp32; P in fp16, the tensor cores' operand type (2^-11 of each
// weight, or 2^-32 of the head's largest where that is more); q and the window rows in fp16,
// exact from 2^-17 up and to 2^-25 below, after a power-of-two scale per head or share where the
// largest magnitude lies outside [2^-10, 2^15).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "fp4_f16.cuh"
#include "umma.cuh"

namespace csa2 {

constexpr int DA_TILE = 64;                          // keys per tile
constexpr int DA_H = 64;                             // heads per share
constexpr int DA_THREADS = 640;
constexpr int DA_SMW = 8;                            // softmax warps 0-7
constexpr int DA_SMT = DA_SMW * 32;
constexpr int DA_MMA1 = 8;                           // warps 8, 9: score MMAs
constexpr int DA_MMA2 = 10;                          // warps 10, 11: value MMAs
constexpr int DA_LOADW = 12;                         // warps 12-19: rows
constexpr int DA_LOADERS = 256;
constexpr int DA_NL = 2;                             // L buffers: a window has at most as many tiles
static_assert(WINDOW <= DA_NL * DA_TILE && DA_TILE == 64, "the window's tiles have a buffer each");
constexpr uint32_t DA_QSLAB = DA_H * 128;            // 64 heads x 64 dims fp16, 128-byte swizzle
constexpr uint32_t DA_LSLAB = DA_TILE * 128;         // 64 keys x 64 dims
constexpr uint32_t DA_SQ = 0;                        // Q: 8 slabs
static_assert(DA_QSLAB == DA_LSLAB, "the score MMAs step both operands alike");
constexpr uint32_t DA_SL = 8 * DA_QSLAB;             // L: 2 buffers x 8 slabs
constexpr uint32_t DA_LBUF = 8 * DA_LSLAB;
constexpr uint32_t DA_SP = DA_SL + DA_NL * DA_LBUF;  // P^T: 2 buffers x 64 heads x 64 keys
constexpr uint32_t DA_PBUF = DA_H * 128;
constexpr uint32_t DA_RED = DA_SP + 2 * DA_PBUF;     // [2 key halves][64 heads]
constexpr uint32_t DA_MISC = DA_RED + 512;           // m_run[64], fac[64], qexp[64], flag[4], wmax[2]
constexpr uint32_t DA_DYN = DA_MISC + 832 + 1024;    // + alignment
constexpr uint32_t DAT_S = 0, DAT_O = 256, DAT_COLS = 512;   // S^T partial p of buffer b at DAT_S + 64 (2b + p)
// A head's weights are 2^(score - m), m set DA_UP below the largest score and raised when one is more than DA_TOP
// above it: the largest weight lies in [2^7, 2^15], within fp16's range, and what fp16 rounds to zero is below
// 2^-32 of it.
constexpr float DA_UP = 7.0f, DA_TOP = 15.0f;
constexpr int DA_SMS = 152;                          // blocks at most: one per SM
constexpr int DA_WIN = 4;                            // units of a window tile: 64 rows, their scale and the share's epilogue

__device__ __forceinline__ uint32_t da_swz(uint32_t row, uint32_t chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

struct DenseItem {               // the shares of an item: blocks b0 .. b0 + n_fp4 - 1; the window's blocks, or -1
    int b0, n_fp4, w0, w1;
};
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
    int n_items;                 // (query, head group) pairs of this pass
    DenseItem* items;            // [n_items]
    float* part_o;               // [share][64][512]
    float2* part_ml;             // [share][64] reference (log2) of the weights and their sum
    int* err;
};
// Shares: block b's part of item i's tiles is number i + b (both only grow along the units, so no two
// meet), its part of item i's window n_items + blocks - 1 further.

// The units' parts: total % parts of them have one unit more than the others, and come first
struct DenseParts {
    int parts, each, more;
    __device__ __forceinline__ DenseParts(int total, int blocks) {
        parts = min(blocks, total);                      // every part has a unit, so a query's shares have no holes
        each = total <= blocks ? 1 : (int)((unsigned)total / (unsigned)blocks);
        more = total - each * parts;
    }
    __device__ __forceinline__ int start(int b) const { return each * min(b, parts) + min(b, more); }
    __device__ __forceinline__ int block_of(int u) const {
        const int longer = (each + 1) * more;
        return u < longer ? (unsigned)u / (unsigned)(each + 1) : more + (unsigned)(u - longer) / (unsigned)each;
    }
};

// what item i of the pass attends to: FP4 entries 0 .. n-1 and `rows` window rows from `row0` on
struct DenseWork {
    int64_t gq, row0;
    int b, h0, n, rows;
    __device__ __forceinline__ int tiles() const { return (int)(((unsigned)n + DA_TILE - 1) / DA_TILE); }
    __device__ __forceinline__ int win() const { return (rows + DA_TILE - 1) / DA_TILE * DA_WIN; }
};
__device__ __forceinline__ DenseWork da_work(const DenseArgs& a, int item) {
    DenseWork w;
    const int ql = a.hgroups == 1 ? item : item >> 1;                    // at most 128 heads: one or two groups
    w.h0 = a.hgroups == 1 ? 0 : (item & 1) * DA_H;
    w.gq = a.query0 + ql;
    w.b = (int)(a.n_q == 1 ? w.gq : a.query0 == 0 ? (unsigned)ql / (unsigned)a.n_q : w.gq / a.n_q);
    const int64_t p = a.q_pos[w.gq];
    const int64_t s0 = a.swa_pos0 != nullptr ? a.swa_pos0[w.b] : 0;
    const int64_t v = p >= WINDOW - 1 ? (p - (WINDOW - 1)) >> (a.ratio - 1) : 0;      // ratio 1 or 2
    w.n = (int)min(v, (int64_t)a.capacity);
    const int64_t lo = max(max((int64_t)0, p - (WINDOW - 1)), s0), hi = min(p, s0 + a.swa_len - 1);
    w.rows = hi >= lo ? (int)(hi - lo + 1) : 0;
    w.row0 = lo - s0;
    return w;
}

// One share of a block, and where the block's units go on after it
struct DenseShare {
    int64_t row;                 // its first row: of the FP4 planes, or of the window rows
    int64_t gq;                  // its query
    int u, start;                // the next unit, and the first unit of the item that has it
    int h0, rows, share, item, next_item, window;
};
// The share that begins at unit u < u1 of item `item` (work w, units from `start` on), if there is one there
__device__ __forceinline__ bool da_part(const DenseArgs& a, const DenseWork& w, int& u, int u1, int& start, int& item,
                                        DenseShare* out) {
    const int ws = start + w.tiles(), end = ws + w.win();
    const bool window = u >= ws;
    const int upto = min(u1, window ? end : ws);
    // of the window the tiles whose first units are among these (none: the rest of another block's tile)
    const int t0 = window ? (u - ws + DA_WIN - 1) / DA_WIN : u - start;
    const int t1 = window ? (upto - ws + DA_WIN - 1) / DA_WIN : upto - start;
    const int row0 = t0 * DA_TILE;
    out->row = (window ? (int64_t)w.b * a.swa_len + w.row0 : (int64_t)w.b * a.capacity) + row0;
    out->rows = (int)min((int64_t)(t1 - t0) * DA_TILE, (int64_t)(window ? w.rows : w.n) - row0);
    out->share = (window ? a.n_items + (int)gridDim.x - 1 : 0) + item + (int)blockIdx.x;
    out->gq = w.gq, out->h0 = w.h0, out->item = item, out->window = window;
    u = upto;
    if (u >= end) start = end, ++item;
    out->u = u, out->start = start, out->next_item = item;
    return t1 > t0;
}
// The next share of the units u .. u1-1, `item` with units from `start` on being the one that has unit u;
// rows = -1 when there is none.  One thread calls it while the block works on the share before, so that
// this state lives in shared memory and not in everybody's registers.
__device__ __noinline__ void da_next(const DenseArgs& a, int u, int u1, int start, int item, DenseShare* out) {
    while (u < u1)
        if (da_part(a, da_work(a, item), u, u1, start, item, out)) return;
    out->rows = -1;
}

__global__ void __launch_bounds__(DA_THREADS, 1) k_dense_attn(const __grid_constant__ DenseArgs a) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) unsigned long long b_lhalf[DA_NL], b_lfull[DA_NL], b_lfree[DA_NL], b_sfull[2], b_sfree[2],
        b_pfull[2], b_odone[2], b_next;
    __shared__ int wsum[DA_THREADS / 32], last_unit;
    __shared__ DenseShare shares[2];
    __shared__ uint32_t tmem_base;
    const uint32_t raw = umma::smem_u32(dyn);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* sm = dyn + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto sa = [&](const void* x) { return umma::smem_u32(x); };
    float* red = reinterpret_cast<float*>(sm + DA_RED);
    float* m_run = reinterpret_cast<float*>(sm + DA_MISC);
    float* fac = m_run + DA_H;
    int* qexp = reinterpret_cast<int*>(fac + DA_H);
    int* flag = qexp + DA_H;
    unsigned int* wmaxs = reinterpret_cast<unsigned int*>(flag + 4);
    if (tid == 0) {
        for (int i = 0; i < DA_NL; ++i) {
            umma::mbar_init(sa(&b_lhalf[i]), DA_LOADERS / 32);
            umma::mbar_init(sa(&b_lfull[i]), DA_LOADERS / 32);
            umma::mbar_init(sa(&b_lfree[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(sa(&b_sfull[i]), 2);
            umma::mbar_init(sa(&b_sfree[i]), DA_SMW);
            umma::mbar_init(sa(&b_pfull[i]), DA_SMW);
            umma::mbar_init(sa(&b_odone[i]), 2);
        }
        umma::mbar_init(sa(&b_next), 1 + DA_LOADERS / 32);
        umma::fence_mbar_init();
        wmaxs[0] = wmaxs[1] = 0u;
    }
    if (warp == DA_LOADW - 1) umma::tmem_alloc(sa(&tmem_base), DAT_COLS);
    pdl_wait();                  // q, the positions and the window may come from the preceding kernel
    pdl_launch_next();

    // ---- this block's units: a sum over the items' units, each thread taking consecutive items (two at most)
    const int per = (a.n_items + DA_THREADS - 1) / DA_THREADS;
    const int i0 = min(tid * per, a.n_items), ni = min(per, a.n_items - i0);
    DenseWork w[2];
    int units[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (k < ni) {
            w[k] = da_work(a, i0 + k);
            units[k] = w[k].tiles() + w[k].win();
        }
    int upto = units[0] + units[1];
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) wsum[warp] = upto;
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i * per * 32 < a.n_items; ++i) {                     // warps that have items
        const int v = wsum[i];
        if (i < warp) before += v;
        total += v;
    }
    const DenseParts pt(total, (int)gridDim.x);
    const int u0 = pt.start(blockIdx.x), u1 = pt.start(blockIdx.x + 1);
    const int first = before + upto - units[0] - units[1];               // this thread's first unit
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int u = u0, s = first + (k > 0 ? units[0] : 0), item = i0 + k;
        if (k < ni && u0 < u1 && s <= u0 && u0 < s + units[k])
            if (!da_part(a, w[k], u, u1, s, item, &shares[0])) da_next(a, u, u1, s, item, &shares[0]);
    }
    if (tid == 0) last_unit = u1;
    if (tid == 0 && u0 >= u1) shares[0].rows = -1;
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = tmem_base;
    // where the shares of every item are, for the kernel that joins them: the last block, which has least to do
    if (blockIdx.x == gridDim.x - 1)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (k < ni) {
                const int s = first + (k > 0 ? units[0] : 0), ws = s + w[k].tiles();
                DenseItem it{0, 0, -1, -1};
                if (ws > s) it.b0 = pt.block_of(s), it.n_fp4 = pt.block_of(ws - 1) - it.b0 + 1;
                if (w[k].win() > 0) it.w0 = pt.block_of(ws);
                if (w[k].win() > DA_WIN) it.w1 = pt.block_of(ws + DA_WIN);
                if (it.w1 == it.w0) it.w1 = -1;
                a.items[i0 + k] = it;
            }
    bool ok = true;
    const int lt = tid - DA_LOADW * 32;
    int q_item = -1;                                         // the item whose queries are staged
    uint32_t tb = 0;                                         // tiles done so far: the rings go on from share to share

    // The loaders go from share to share by themselves, held by the buffers alone; the other warps meet.  Phase k of
    // b_next says that the share after share k is known.  A loader warp arrives on it too, once it has seen phase
    // k - 1: warps 0-11 could otherwise go through share k + 1's hand-over before a delayed loader has looked, and
    // its wait, which knows a phase by its parity alone, would meet a barrier two phases on.
    if (warp >= DA_LOADW && lane == 0) umma::mbar_arrive(sa(&b_next));
    for (uint32_t k = 0; shares[k & 1].rows >= 0; ++k) {
        const uint32_t cur = k & 1;
        const DenseShare& S = shares[cur];
        const int rows = S.rows, T = (rows + DA_TILE - 1) / DA_TILE;
        const bool window = S.window;
        unsigned int* wmax = wmaxs + cur;

        // FP4 rows: a tile is 64 rows x 16 units of 32 dims (16 bytes of codes, 2 of scales)
        const uint8_t* codes = a.codes + S.row * (D_LAT / 2);
        const uint8_t* scales = a.scales + S.row * (D_LAT / 16);
        constexpr int NU = DA_TILE * 16 / DA_LOADERS;
        // unit u: a warp takes 4 rows x 8 units, so that a load touches whole 128-byte lines and the
        // 8 threads of a quarter warp write different bank groups; units below 512 hold dims 0-255
        auto unit_rc = [&](int i, int& r, int& c) {
            const int qq = (lt >> 5) + 8 * i;
            r = 4 * (qq & 15) + (lane & 3);
            c = 8 * (qq >> 4) + (lane >> 2);
        };
        uint4 cw[NU];
        uint32_t sc[NU];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                int r, c;
                unit_rc(i, r, c);
                cw[i] = make_uint4(0, 0, 0, 0);      // rows past the end expand to zeros
                sc[i] = 0u;
                const int j = t * DA_TILE + r;
                if (j < rows) {
                    cw[i] = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)j * (D_LAT / 2)) + c);
                    sc[i] = __ldg(reinterpret_cast<const uint16_t*>(scales + (int64_t)j * (D_LAT / 16)) + c);
                }
            }
        };
        if (warp < DA_LOADW) {
            if (k > 0) {             // the share before is done with Q, O and the running max
                umma::fence_before();
                umma::bar_named(3, DA_LOADW * 32);
                umma::fence_after();
            }
            if (tid < DA_H) m_run[tid] = -INFINITY;
        }
        // Q: heads h0 .. h0+63 (zero rows past n_heads), bf16 -> fp16 slabs, by warps 0-11; a head whose largest
        // magnitude lies outside [2^-10, 2^15) is scaled by a power of two on the way
        if (q_item != S.item && warp < DA_LOADW) {
            const uint4* qsrc = reinterpret_cast<const uint4*>(a.q + (S.gq * a.n_heads + S.h0) * D_LAT);
            const int nh = min(DA_H, a.n_heads - S.h0);
            // (a loop: unrolled over all heads it waits for its own code)
#pragma unroll 1
            for (int h0 = warp; h0 < nh; h0 += 2 * DA_LOADW) {
                uint4 qv[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int h = h0 + DA_LOADW * r;
                    if (h < nh) {
                        qv[r][0] = qsrc[h * 64 + lane];
                        qv[r][1] = qsrc[h * 64 + 32 + lane];
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int h = h0 + DA_LOADW * r;
                    if (h >= nh) break;
                    const uint32_t mx = __reduce_max_sync(0xffffffffu, max(bf16_absmax8(qv[r][0]), bf16_absmax8(qv[r][1])));
                    const int e = f16_range_exp(mx);
                    const float d = pow2f(-e);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int c = lane + 32 * hh;
                        *reinterpret_cast<uint4*>(sm + DA_SQ + (c >> 3) * DA_QSLAB + da_swz(h, c & 7)) =
                            bf16x8_to_f16x8(qv[r][hh], d);
                    }
                    if (lane == 0) qexp[h] = e;
                }
            }
#pragma unroll 1
            for (int i = nh * 64 + tid; i < DA_H * 64; i += DA_LOADW * 32) {
                *reinterpret_cast<uint4*>(sm + DA_SQ + ((i & 63) >> 3) * DA_QSLAB + da_swz(i >> 6, i & 7)) = make_uint4(0, 0, 0, 0);
                qexp[i >> 6] = 0;
            }
            umma::fence_proxy_async();
        }
        q_item = S.item;
        if (warp < DA_LOADW) umma::bar_named(3, DA_LOADW * 32);
        if (tid == DA_LOADW * 32 - 1) {          // the last warp that has nothing to do yet
            wmaxs[cur ^ 1] = 0u;
            da_next(a, S.u, last_unit, S.start, S.next_item, &shares[cur ^ 1]);
            umma::mbar_arrive(sa(&b_next));
        }
        __syncwarp();

        if (warp >= DA_LOADW) {
            if (window) {
                // ================= window rows: bf16, at most two tiles, so every tile has a buffer.  They are converted
                // as they are while their largest magnitude is found, and once more where it asks for a scale.
                const uint4* src = reinterpret_cast<const uint4*>(a.swa + S.row * D_LAT);
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t;
                    if (tg >= DA_NL) ok = ok && umma::mbar_wait_fast(sa(&b_lfree[tg % DA_NL]), (tg / DA_NL - 1) & 1);
                }
                uint32_t mx = 0u;
                auto convert = [&](float d) {
#pragma unroll 1
                    for (int v0 = lt; v0 < T * DA_TILE * 64; v0 += 8 * DA_LOADERS) {
                        uint4 x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int v = v0 + i * DA_LOADERS;
                            x[i] = make_uint4(0, 0, 0, 0);
                            if (v < rows * 64) x[i] = src[v];
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int v = v0 + i * DA_LOADERS, t = v >> 12, r = (v >> 6) & 63, c = v & 63;
                            mx = max(mx, bf16_absmax8(x[i]));
                            *reinterpret_cast<uint4*>(sm + DA_SL + ((tb + t) % DA_NL) * DA_LBUF + (c >> 3) * DA_LSLAB + da_swz(r, c & 7)) =
                                bf16x8_to_f16x8(x[i], d);
                        }
                    }
                };
                convert(1.0f);
                mx = __reduce_max_sync(0xffffffffu, mx);
                if (lane == 0) atomicMax(wmax, mx);
                umma::bar_named(2, DA_LOADERS);
                const int e = f16_range_exp(*reinterpret_cast<volatile unsigned int*>(wmax));
                if (e != 0) convert(pow2f(-e));
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    for (int t = 0; t < T; ++t) {
                        umma::mbar_arrive(sa(&b_lhalf[(tb + t) % DA_NL]));
                        umma::mbar_arrive(sa(&b_lfull[(tb + t) % DA_NL]));
                    }
            } else {
                // ================= FP4 rows
                for (int t = 0; t < T; ++t) {
                    const uint32_t tg = tb + t, buf = tg % DA_NL;
                    uint8_t* L = sm + DA_SL + buf * DA_LBUF;
                    fetch(t);
                    if (lt < DA_TILE && (t + 1) * DA_TILE + lt < rows) {
                        const int64_t j = (t + 1) * DA_TILE + lt;
                        umma::prefetch_l2(codes + j * (D_LAT / 2));
                        umma::prefetch_l2(codes + j * (D_LAT / 2) + 128);
                        if ((lt & 3) == 0) umma::prefetch_l2(scales + j * (D_LAT / 16));
                    }
                    if (tg >= DA_NL) ok = ok && umma::mbar_wait_fast(sa(&b_lfree[buf]), (tg / DA_NL - 1) & 1);
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
                        for (int k = 0; k < 4; ++k) {
                            const int cc = c * 4 + k;
                            *reinterpret_cast<uint4*>(L + (cc >> 3) * DA_LSLAB + da_swz(r, cc & 7)) =
                                e2m1x8_scaled(words[k], (k >> 1) ? s_hi : s_lo);
                        }
                    }
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(sa(&b_lfull[buf]));
                }
            }
        } else if (warp == DA_MMA1 || warp == DA_MMA1 + 1) {
            // ================= scores of tile t once its dims are expanded and the softmax has read tile t-2's.
            // The whole warp walks the tiles, so that descriptors and addresses stay in uniform registers (one
            // lane alone moves them there for every MMA: 110 to 140 clocks each); one elected lane issues.
            const int half = warp - DA_MMA1;
            const uint32_t id = umma::idesc_f16(64, DA_TILE, 0, 0);
            const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
            const uint64_t qd = umma::desc(base + DA_SQ, 16, 1024, umma::LAYOUT_SW128);
            unsigned long long* ready = half == 0 ? b_lhalf : b_lfull;
            for (int t = 0; t < T; ++t) {
                const uint32_t tg = tb + t, lb = tg % DA_NL, sb = tg & 1;
                ok = ok && umma::mbar_wait_fast(sa(&ready[lb]), (tg / DA_NL) & 1);
                if (tg >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_sfree[sb]), ((tg >> 1) - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                umma::fence_after();
                const uint64_t ld = umma::desc(base + DA_SL + lb * DA_LBUF, 16, 1024, umma::LAYOUT_SW128);
                if (umma::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk) {
                        const int ks = 16 * half + kk;
                        const uint64_t off = (uint64_t)(((ks >> 2) * DA_LSLAB + (ks & 3) * 32) >> 4);
                        umma::mma_f16(tm + DAT_S + 64 * (2 * sb + half), qd + off, ld + off, id, kk > 0);
                    }
                    umma::commit(sa(&b_sfull[sb]));
                }
                __syncwarp();
            }
        } else if (warp == DA_MMA2 || warp == DA_MMA2 + 1) {
            // ================= values of tile t once P is written; completion frees the L and P buffers
            const int half = warp - DA_MMA2;
            const int n16 = min(DA_H, (a.n_heads - S.h0 + 15) & ~15);        // heads that are there, in MMA steps
            const uint32_t id = umma::idesc_f16(128, n16, 1, 0);
            const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
            for (int t = 0; t < T; ++t) {
                const uint32_t tg = tb + t, lb = tg % DA_NL, sb = tg & 1;
                ok = ok && umma::mbar_wait_fast(sa(&b_pfull[sb]), (tg >> 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                umma::fence_after();
                const uint64_t la = umma::desc(base + DA_SL + lb * DA_LBUF, DA_LSLAB, 1024, umma::LAYOUT_SW128);
                const uint64_t pb = umma::desc(base + DA_SP + sb * DA_PBUF, 16, 1024, umma::LAYOUT_SW128);
                if (umma::elect_one()) {
#pragma unroll
                    for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
                        for (int ks = 0; ks < DA_TILE / 16; ++ks) {
                            const int mt = 2 * half + m2;
                            umma::mma_f16(tm + DAT_O + 64 * mt, la + (uint64_t)((2 * mt * DA_LSLAB + ks * 2048) >> 4),
                                          pb + (uint64_t)((ks * 32) >> 4), id, (t > 0 || ks > 0) ? 1u : 0u);
                        }
                    umma::commit(sa(&b_lfree[lb]));
                    umma::commit(sa(&b_odone[sb]));
                }
                __syncwarp();
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
                const uint32_t tg = tb + t, sb = tg & 1;
                float x[16];
                ok = ok && umma::mbar_wait_fast(sa(&b_sfull[sb]), (tg >> 1) & 1);
                umma::fence_after();
                {
                    float x1[16];
                    umma::tmem_ld16x64b_x16(lane_base + DAT_S + 64 * (2 * sb) + 32 * half, x);
                    umma::tmem_ld16x64b_x16(lane_base + DAT_S + 64 * (2 * sb + 1) + 32 * half, x1);
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] += x1[i];
                }
                umma::fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(sa(&b_sfree[sb]));
                // the scores times scale and this head's and the window's powers of two (known once tile 0 is in)
                if (t == 0) {
                    if (window) ok = ok && umma::mbar_wait_fast(sa(&b_lfull[tg % DA_NL]), (tg / DA_NL) & 1);
                    mul = a.scale_log2e * pow2f(qexp[h]) *
                          (window ? pow2f(f16_range_exp(*reinterpret_cast<volatile unsigned int*>(wmax))) : 1.0f);
                }
                const float mh = m_run[h];
                const int left = rows - t * DA_TILE - 32 * half;     // valid keys of this half
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] *= mul;
                if (left < 32)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (par + 2 * i >= left) x[i] = -INFINITY;
                float mx = x[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[i]);
                if (umma::bar_red_or(1, DA_SMT, mx - mh > DA_TOP)) {
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    if (par == 0) red[half * DA_H + h] = mx;
                    umma::bar_named(1, DA_SMT);
                    if (half == 0) {
                        float f = 1.0f;
                        if (par == 0) {
                            const float mt = fmaxf(red[h], red[DA_H + h]), mo = m_run[h], mn = mt - DA_UP;
                            // (differences, exact where they matter: a sum with m would round away from it)
                            if (mt > -INFINITY && (mo == -INFINITY || mt - mo > DA_TOP)) {
                                f = mo == -INFINITY ? 0.0f : umma::ex2(mo - mn);
                                m_run[h] = mn;
                            }
                            fac[h] = f;
                        }
                        const unsigned any = __ballot_sync(0xffffffffu, f != 1.0f);
                        if (lane == 0) flag[qd] = any != 0;
                    }
                    if (t >= 1) ok = ok && umma::mbar_wait_fast(sa(&b_odone[sb ^ 1]), ((tg - 1) >> 1) & 1);   // O settled
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
                if (tg >= 2) ok = ok && umma::mbar_wait_fast(sa(&b_odone[sb]), ((tg >> 1) - 1) & 1);   // P buffer free
                const float m = m_run[h];
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] = umma::ex2_ftz(x[i] - m);              // 0 for a masked key; m is finite: a tile has a key
                    sum[i & 1] += x[i];
                }
                lsum += sum[0] + sum[1];
                // row h of P^T: trade half of the values with the lane of the other parity for 16 consecutive keys
                float rv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) rv[i] = __shfl_xor_sync(0xffffffffu, par ? x[i] : x[8 + i], 2);
                uint32_t p2[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) p2[j] = par ? f16x2_bits(rv[j], x[8 + j]) : f16x2_bits(x[j], rv[j]);
                uint8_t* P = sm + DA_SP + sb * DA_PBUF;
                *reinterpret_cast<uint4*>(P + da_swz(h, 4 * half + 2 * par)) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                *reinterpret_cast<uint4*>(P + da_swz(h, 4 * half + 2 * par + 1)) = make_uint4(p2[4], p2[5], p2[6], p2[7]);
                umma::fence_proxy_async();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(sa(&b_pfull[sb]));
            }
            lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
            if (par == 0) red[half * DA_H + h] = lsum;
            umma::bar_named(1, DA_SMT);
            if (tid < DA_H) a.part_ml[(int64_t)S.share * DA_H + tid] = make_float2(m_run[tid], red[tid] + red[DA_H + tid]);
            // ---- this share's O^T (the window's back on the common scale) to the workspace, [head][dim]
            const uint32_t tl = tb + T - 1;
            ok = ok && umma::mbar_wait_fast(sa(&b_odone[tl & 1]), (tl >> 1) & 1);
            umma::fence_after();
            const float up = window ? pow2f(f16_range_exp(*wmax)) : 1.0f;
            const int nh = min(DA_H, a.n_heads - S.h0);
#pragma unroll 1
            for (int mt = 2 * half; mt < 2 * half + 2; ++mt) {
                float* dst = a.part_o + (int64_t)S.share * DA_H * D_LAT + mt * 128 + qd * 32 + lane;
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
        tb += T;
        __syncwarp();                                        // the issuers' other lanes
        ok = umma::mbar_wait_fast(sa(&b_next), k & 1) && ok;
        __syncwarp();
        if (warp >= DA_LOADW && lane == 0) umma::mbar_arrive(sa(&b_next));
    }
    if (!ok) atomicExch(a.err, 1);
    umma::fence_before();
    __syncthreads();
    if (warp == DA_LOADW - 1) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, DAT_COLS);
    }
}

// Joins the shares of every query and head, four dims a thread: 128 threads per head (SPREAD 1, four heads
// per block), or four groups of 128 that take every fourth share and are added up in order (SPREAD 4).  Every
// warp finds the shares' factors for itself, 32 at a time, so that nothing waits but the groups' sum.
constexpr int DA_MAXS = DA_SMS + 2;              // shares of one query at most

template <typename TO, int SPREAD>
__global__ void __launch_bounds__(512) k_dense_combine(const float* part_o, const float2* part_ml,
                                                       const DenseItem* items, int n_items, int blocks,
                                                       int hgroups, int n_heads, int64_t query0, int n_rows,
                                                       TO* out, float* lse) {
    constexpr int NK = (DA_MAXS + 31) / 32;
    __shared__ float4 sums[SPREAD > 1 ? 3 : 1][128];
    __shared__ float factors[512 / 32][32 * NK];
    const int tid = threadIdx.x, lane = tid & 31, dim = tid & 127, group = SPREAD > 1 ? tid >> 7 : 0;
    const int row = SPREAD > 1 ? (int)blockIdx.x : (int)blockIdx.x * 4 + (tid >> 7);         // query of this pass, head
    const int ql = (int)((unsigned)row / (unsigned)n_heads);
    const int head = row - ql * n_heads, item = ql * hgroups + head / DA_H;
    float* fw = factors[tid >> 5];
    pdl_wait();
    if (SPREAD == 1 && row >= n_rows) return;
    const DenseItem it = *(items + item);
    const int n = it.n_fp4 + (it.w0 >= 0) + (it.w1 >= 0);
    auto share = [&](int s) {
        return (int64_t)item + (s < it.n_fp4 ? it.b0 + s : n_items + blocks - 1 + (s == it.n_fp4 ? it.w0 : it.w1));
    };
    // several shares' loads in flight at a time (past the end: the last one again, times nothing), the first of
    // them before the factors are known
    constexpr int NB = SPREAD > 1 ? 8 : 4;
    const float4* src = reinterpret_cast<const float4*>(part_o + (int64_t)(head % DA_H) * D_LAT) + dim;
    float4 x[NB];
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < NB; ++i) x[i] = src[share(min(s0 + i * SPREAD, n - 1)) * DA_H * (D_LAT / 4)];
    };
    if (n > 0) load(group);
    float fs[NK], ls[NK], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        fs[k] = -INFINITY, ls[k] = 0.0f;
        const int s = 32 * k + lane;
        if (s < n) {
            const float2 v = part_ml[share(s) * DA_H + head % DA_H];
            fs[k] = v.x, ls[k] = v.y;
            if (v.y != 0.0f) m = fmaxf(m, v.x);
        }
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int k = 0; k < NK; ++k)
        if (32 * k < n) {
            fs[k] = ls[k] != 0.0f ? exp2f(fs[k] - m) : 0.0f;
            l = fmaf(fs[k], ls[k], l);
            fw[32 * k + lane] = fs[k];
        }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    __syncwarp();
    float o[4] = {};
    for (int s0 = group; s0 < n;) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int s = s0 + i * SPREAD;
            const float f = s < n ? fw[s] : 0.0f;
            o[0] = fmaf(f, x[i].x, o[0]), o[1] = fmaf(f, x[i].y, o[1]);
            o[2] = fmaf(f, x[i].z, o[2]), o[3] = fmaf(f, x[i].w, o[3]);
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
    const int64_t at = query0 * n_heads + row;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    ElemVec<TO, 4> y;
    y.pack(o);
    y.store(out + at * D_LAT + 4 * dim);
    if (lse != nullptr && dim == 0) lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

namespace {
constexpr size_t DA_HEAD = 256;                                   // the error word and padding
constexpr int64_t DA_PASS = 1024;                                 // items of one pass at most: their shares stay below 300 MB

struct DensePlan {
    int hgroups, blocks;
    int64_t pass_queries;
    size_t items_bytes, o_bytes, ml_bytes;
};
DensePlan dense_plan(int64_t queries, int n_heads, int64_t capacity) {
    DensePlan p;
    p.hgroups = (n_heads + DA_H - 1) / DA_H;
    const int64_t units = (capacity + DA_TILE - 1) / DA_TILE + DA_NL * DA_WIN;       // of an item, at most
    p.pass_queries = std::min(queries, std::min(DA_PASS, 0x7fffffff / units) / p.hgroups);   // units are counted in 32 bits
    const int64_t items = p.pass_queries * p.hgroups;
    // one block per SM, fewer where even a full cache has fewer units
    p.blocks = (int)std::min<int64_t>(DA_SMS, items * units);
    const size_t rows = (size_t)2 * (items + p.blocks - 1) * DA_H;
    p.items_bytes = ((size_t)items * sizeof(DenseItem) + 255) / 256 * 256;
    p.o_bytes = rows * D_LAT * sizeof(float);
    p.ml_bytes = rows * sizeof(float2);
    return p;
}
}  // namespace

size_t dense_attn_ws(int batch, int n_q, int n_heads, int64_t capacity) {
    const DensePlan p = dense_plan((int64_t)batch * n_q, n_heads, capacity);
    return DA_HEAD + p.items_bytes + p.o_bytes + p.ml_bytes;
}

cudaError_t launch_dense_attn(const csa2_cache& c, const uint16_t* q, int n_q, int n_heads, const int64_t* q_pos,
                              const uint16_t* swa, const int64_t* swa_pos0, int swa_len, float scale, void* out,
                              int out_type, float* lse, void* ws, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_dense_attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DA_DYN);
    if (e != cudaSuccess) return e;
    const int64_t queries = (int64_t)c.batch * n_q;
    const DensePlan p = dense_plan(queries, n_heads, c.capacity);
    uint8_t* w = reinterpret_cast<uint8_t*>(ws) + DA_HEAD;
    DenseArgs a{c.lat_codes, c.lat_scales, c.capacity, c.ratio, q, n_q, n_heads, p.hgroups, q_pos, swa, swa_pos0, swa_len,
                scale * 1.4426950408889634f, 0, 0, reinterpret_cast<DenseItem*>(w),
                reinterpret_cast<float*>(w + p.items_bytes), reinterpret_cast<float2*>(w + p.items_bytes + p.o_bytes),
                reinterpret_cast<int*>(ws)};
    for (int64_t q0 = 0; q0 < queries; q0 += p.pass_queries) {
        const int64_t nq = std::min(p.pass_queries, queries - q0);
        a.query0 = q0;
        a.n_items = (int)(nq * p.hgroups);
        launch_k(k_dense_attn, dim3((unsigned)p.blocks), DA_THREADS, DA_DYN, st, a);
        auto join = [&](auto* y) {
            // few items: many shares each, so a block per head; else about (blocks + 2 items) / items of them
            using TO = std::remove_pointer_t<decltype(y)>;
            const int64_t rows = nq * n_heads;
            const bool spread = a.n_items * 8 <= p.blocks;
            launch_k(spread ? k_dense_combine<TO, 4> : k_dense_combine<TO, 1>, dim3((unsigned)(spread ? rows : (rows + 3) / 4)),
                     512, 0, st, a.part_o, a.part_ml, a.items, a.n_items, p.blocks, p.hgroups, n_heads, q0, (int)rows, y, lse);
        };
        if (out_type == CSA2_F32)
            join(reinterpret_cast<float*>(out));
        else if (out_type == CSA2_F16)
            join(reinterpret_cast<__half*>(out));
        else
            join(reinterpret_cast<__nv_bfloat16*>(out));
        note_launch(2);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace csa2
