// Before the attention of drafted trees: of every sequence the chains of its nodes, what each node attends to, and the rows
// that are not in the cache (the committed window rows, then the drafts) as fp16.  They are a few hundred KB that every item
// of the sequence reads, so they are converted once.
#include <algorithm>

#include "fp4_f16.cuh"
#include "tree.cuh"

namespace csa2 {

// The exponent e with which a row goes to fp16 as 2^-e of itself, from the bf16 bits of its largest magnitude: 0 while that lies in
// [2^-3, 2^5) or is 0, else what brings it into [2^2, 2^3), -100 at least.  So the rows are of one size within 2^8 wherever their
// exponents are not all the same, what a row loses is 2^-22 of its largest magnitude at most, and a weight times 2^e,
// which is what the value products take, is small only where the row's part of the output is.
__device__ __forceinline__ int tree_row_exp(uint32_t mx) {
    const int e = (int)(mx >> 7) - 127;
    return mx == 0u || (e >= -3 && e < 5) ? 0 : max(-100, e - 2);
}

// A row of 512 bf16 values, two pieces of 16 bytes a lane, to fp16; returns its exponent.
__device__ __forceinline__ int row_to_f16(const uint4* x, uint4* d0, uint4* d1, bool neg) {
    const int e = tree_row_exp(__reduce_max_sync(0xffffffffu, max(bf16_absmax8(x[0]), bf16_absmax8(x[1]))));
    const float d = neg ? -pow2f(-e) : pow2f(-e);
    *d0 = bf16x8_to_f16x8(x[0], d);
    *d1 = bf16x8_to_f16x8(x[1], d);
    return e;
}

// Blocks (sequence, group of 16 rows), `fill` more that write the rows of items that nobody works on, and others that convert
// the sequence's queries.  All but those find the chains for themselves (a thread a node), the first one writes the nodes'
// part; then a warp has two rows.
__global__ void __launch_bounds__(256) k_tree_prep(const __grid_constant__ TreeCall a, int fill) {
    __shared__ int parent[TREE_NODES], last_s, vis_s, offs[8];
    __shared__ long long hi_s;
    __shared__ uint32_t there[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, group = blockIdx.y, N = a.n_q;
    if (tid == 0) last_s = -1, vis_s = 0, hi_s = -1;
    if (tid < 4) there[tid] = 0u;
    pdl_wait();
    pdl_launch_next();
    if (group >= TREE_GROUPS + fill) {
        // four rows of the sequence's queries a warp at a time (those of nodes that are not there too: nobody reads them)
        const int rows = N * a.n_heads, warps = ((int)gridDim.y - TREE_GROUPS - fill) * 8;
        const int64_t r0 = (int64_t)b * rows;
        for (int r = (group - TREE_GROUPS - fill) * 8 + warp; r < rows; r += 4 * warps) {
            uint4 x[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i * warps < rows) {
                    const uint4* src = reinterpret_cast<const uint4*>(a.q + (r0 + r + i * warps) * D_LAT);
                    x[i][0] = src[lane], x[i][1] = src[32 + lane];
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (r + i * warps >= rows) break;
                const int64_t at = r0 + r + i * warps;
                uint4 *d0 = reinterpret_cast<uint4*>(a.t.q16 + at * D_LAT) + lane, *d1 = d0 + 32;
                if (a.q_tiles) {                         // slabs lane / 8 and 4 + lane / 8 of the row's tile
                    const int rr = r + i * warps;
                    uint8_t* tile = reinterpret_cast<uint8_t*>(a.t.q16) + ((int64_t)b * ((rows + 127) / 128) * 2 + (rr >> 6)) * 65536;
                    d0 = reinterpret_cast<uint4*>(tile + (lane >> 3) * 8192 + tree_swz(rr & 63, lane & 7)), d1 = d0 + 4 * 8192 / 16;
                }
                const int e = row_to_f16(x[i], d0, d1, a.neg_q);
                if (lane == 0) a.t.q_exps[at] = (int8_t)e;
            }
        }
        return;
    }
    int64_t p = 0;
    if (tid < N) {
        parent[tid] = a.parent[(int64_t)b * N + tid];
        p = a.q_pos[(int64_t)b * N + tid];
    }
    const int64_t s0 = a.swa_pos0 ? a.swa_pos0[b] : 0;
    __syncthreads();
    int len = 0;
    uint32_t anc[4] = {0u, 0u, 0u, 0u};              // the node and its ancestors
    if (tid < N) {
        int j = tid;
        while (j >= 0) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if ((j >> 5) == w) anc[w] |= 1u << (j & 31);
            ++len;
            const int up = parent[j];
            j = up >= -1 && up < j ? up : -2;
        }
        if (j != -1) len = 0;
        if (len > 0) {
            atomicOr(&there[warp], 1u << lane);
            atomicMax(&last_s, tid);
            // every child of the last committed token stands at the same position: the one after hi (if not, all blocks take the last)
            if (parent[tid] == -1) atomicMax(&hi_s, (long long)(p - len));
        }
    }
    __syncthreads();
    const int last = last_s;
    const int row_tiles = ((last + 1) * a.n_heads + 127) / 128;
    if (group >= TREE_GROUPS) {
        const int64_t r0 = (int64_t)row_tiles * 128, r1 = (int64_t)N * a.n_heads, base = (int64_t)b * r1;
        const int pieces = D_LAT * a.out_size / 16;
        uint4* o = reinterpret_cast<uint4*>(a.out) + base * pieces;
        const int64_t step = (int64_t)fill * 256, first = (int64_t)(group - TREE_GROUPS) * 256 + tid;
        for (int64_t i = r0 * pieces + first; i < r1 * pieces; i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr)
            for (int64_t i = r0 + first; i < r1; i += step) a.lse[base + i] = -INFINITY;
        return;
    }
    const int64_t hi0 = hi_s;
    const int64_t lo = max(max((int64_t)0, hi0 - (WINDOW - 2)), s0), hi = min(hi0, s0 + a.swa_len - 1);
    const int nw = last >= 0 && hi >= lo ? (int)(hi - lo + 1) : 0;       // at most 127
    const int n_rows = last >= 0 ? nw + last + 1 : 0;
    // ---- rows group * 16 + warp and 8 further as fp16
    if (group * 16 < n_rows) {
        uint4 x[2][2];
        bool off = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = group * 16 + warp + 8 * i, j = r - nw;
            const uint4* src = nullptr;
            if (j < 0)
                src = reinterpret_cast<const uint4*>(a.swa + ((int64_t)b * a.swa_len + (lo - s0) + r) * D_LAT);
            else if (r < n_rows && ((there[j >> 5] >> (j & 31)) & 1u))
                src = reinterpret_cast<const uint4*>(a.draft + ((int64_t)b * N + j) * D_LAT);
            x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (src != nullptr) x[i][0] = src[lane], x[i][1] = src[32 + lane];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = group * 16 + warp + 8 * i;
            if (r >= n_rows) break;
            uint4* dst = reinterpret_cast<uint4*>(a.t.rows16 + ((int64_t)b * a.t.row_stride + r) * D_LAT) + lane;
            const int e = row_to_f16(x[i], dst, dst + 32, false);
            if (lane == 0) a.t.exps[b * 256 + r] = (int8_t)e;
            off = off || e != 0;
        }
        if (lane == 0) offs[warp] = off;
    }
    if (group == 0 && tid < N) {
        int vis = 0;
        uint32_t m[8] = {};
        if (len > 0) {
            vis = (int)min(p >= WINDOW - 1 ? (p - (WINDOW - 1)) >> (a.ratio - 1) : (int64_t)0, (int64_t)a.capacity);
            atomicMax(&vis_s, vis);
            // committed rows c0 .. nw-1; with the chain no more than the window holds, wherever the positions are
            const int c0 = max((int)max((int64_t)0, min((int64_t)nw, p - (WINDOW - 1) - lo)), nw - (WINDOW - len));
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const int f = max(c0 - 32 * w, 0), e = min(nw - 32 * w, 32);
                if (f < e) m[w] = (e == 32 ? 0xffffffffu : (1u << e) - 1u) & ~((1u << f) - 1u);
#pragma unroll
                for (int v = 0; v < 4; ++v) {            // drafts: bit j of the chain at row nw + j
                    const int at = nw + 32 * v - 32 * w;
                    if (at >= 0 && at < 32) m[w] |= anc[v] << at;
                    if (at < 0 && at > -32) m[w] |= anc[v] >> -at;
                }
            }
        }
        a.t.vis[(int64_t)b * N + tid] = vis;
        uint4* mask = reinterpret_cast<uint4*>(a.t.mask + ((int64_t)b * N + tid) * 8);
        mask[0] = make_uint4(m[0], m[1], m[2], m[3]);
        mask[1] = make_uint4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    if (tid == 0) {
        if (group * 16 < n_rows) {
            int off = 0;
            for (int i = 0; i < 8; ++i) off |= offs[i];
            a.t.off[b * TREE_GROUPS + group] = off;
        }
        if (group == 0) a.t.seq[b] = TreeSeq{vis_s, n_rows, row_tiles, 0};
    }
}

namespace {
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
struct NodeParts {
    size_t seq, vis, mask, exps, off, rows, q, q_exps;
    NodeParts(int batch, int n_q, int q_rows)
        : seq(up256((size_t)batch * sizeof(TreeSeq))),
          vis(up256((size_t)batch * n_q * sizeof(int))),
          mask(up256((size_t)batch * n_q * 8 * sizeof(uint32_t))),
          exps((size_t)batch * 256),
          off(up256((size_t)batch * TREE_GROUPS * sizeof(int))),
          rows((size_t)batch * (WINDOW - 1 + n_q) * D_LAT * sizeof(uint16_t)),
          q((size_t)batch * q_rows * D_LAT * sizeof(uint16_t)),
          q_exps(up256((size_t)batch * q_rows)) {}
};
}  // namespace

size_t tree_nodes_bytes(int batch, int n_q, int q_rows) {
    const NodeParts p(batch, n_q, q_rows);
    return p.seq + p.vis + p.mask + p.exps + p.off + p.rows + p.q + p.q_exps;
}

uint8_t* tree_nodes_take(TreeNodes& t, int batch, int n_q, int q_rows, uint8_t* w) {
    const NodeParts p(batch, n_q, q_rows);
    t.seq = reinterpret_cast<TreeSeq*>(w), w += p.seq;
    t.vis = reinterpret_cast<int*>(w), w += p.vis;
    t.mask = reinterpret_cast<uint32_t*>(w), w += p.mask;
    t.exps = reinterpret_cast<int8_t*>(w), w += p.exps;
    t.off = reinterpret_cast<int*>(w), w += p.off;
    t.rows16 = reinterpret_cast<uint16_t*>(w), w += p.rows;
    t.row_stride = WINDOW - 1 + n_q;
    t.q16 = reinterpret_cast<uint16_t*>(w), w += p.q;
    t.q_exps = reinterpret_cast<int8_t*>(w), w += p.q_exps;
    return w;
}

cudaError_t launch_tree_prep(const TreeCall& c, cudaStream_t st) {
    const int rows = c.n_q * c.n_heads;
    const int fill = c.out ? std::min(16, (rows + 511) / 512) : 0;
    launch_k(k_tree_prep, dim3((unsigned)c.batch, (unsigned)(TREE_GROUPS + fill + (rows + 31) / 32)), 256, 0, st, c, fill);
    note_launch();
    return cudaGetLastError();
}

}  // namespace csa2
