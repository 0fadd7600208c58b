// Before the attention of drafted trees: of every sequence the chains of its nodes, what each node attends to, and the rows
// that are not in the cache (the committed window rows, then the drafts) as fp16.  They are a few hundred KB that every item
// of the sequence reads, so they are converted once.
#include <algorithm>

#include "fp4_f16.cuh"
#include "tree.cuh"

namespace csa2 {

// One block a sequence, and some that write the rows of items that nobody works on.  A thread has a node at first, then 16
// pieces of 16 bytes (at most 255 rows of 64 pieces): all loads in flight, their largest magnitude, the conversion.
__global__ void __launch_bounds__(1024) k_tree_prep(const __grid_constant__ TreeCall a) {
    __shared__ int parent[TREE_NODES], last_s, vis_s;
    __shared__ long long hi_s;
    __shared__ uint32_t there[4], mx_s;
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x, N = a.n_q;
    if (tid == 0) last_s = -1, vis_s = 0, mx_s = 0u, hi_s = -1;
    if (tid < 4) there[tid] = 0u;
    pdl_wait();
    pdl_launch_next();
    if (tid < N) parent[tid] = a.parent[(int64_t)b * N + tid];
    __syncthreads();
    int len = 0;
    uint32_t anc[4] = {0u, 0u, 0u, 0u};              // the node and its ancestors
    int64_t p = 0;
    if (tid < N) {
        p = a.q_pos[(int64_t)b * N + tid];
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
            atomicOr(&there[tid >> 5], 1u << lane);
            atomicMax(&last_s, tid);
        }
    }
    __syncthreads();
    const int last = last_s;
    const int row_tiles = ((last + 1) * a.n_heads + 127) / 128;
    if (blockIdx.y > 0) {
        const int64_t r0 = (int64_t)row_tiles * 128, r1 = (int64_t)N * a.n_heads, base = (int64_t)b * r1;
        const int pieces = D_LAT * a.out_size / 16;
        uint4* o = reinterpret_cast<uint4*>(a.out) + base * pieces;
        const int64_t step = (int64_t)(gridDim.y - 1) * 1024, first = (int64_t)(blockIdx.y - 1) * 1024 + tid;
        for (int64_t i = r0 * pieces + first; i < r1 * pieces; i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr)
            for (int64_t i = r0 + first; i < r1; i += step) a.lse[base + i] = -INFINITY;
        return;
    }
    // every child of the last committed token stands at the same position: the one after hi
    if (len > 0 && parent[tid] == -1) hi_s = p - len;
    __syncthreads();
    const int64_t s0 = a.swa_pos0 ? a.swa_pos0[b] : 0, hi0 = hi_s;
    const int64_t lo = max(max((int64_t)0, hi0 - (WINDOW - 2)), s0), hi = min(hi0, s0 + a.swa_len - 1);
    const int nw = last >= 0 && hi >= lo ? (int)(hi - lo + 1) : 0;       // at most 127
    const int n_rows = last >= 0 ? nw + last + 1 : 0;
    if (tid < N) {
        int vis = 0;
        uint32_t m[8] = {};
        if (len > 0) {
            vis = (int)min(p >= WINDOW - 1 ? (p - (WINDOW - 1)) >> (a.ratio - 1) : (int64_t)0, (int64_t)a.capacity);
            atomicMax(&vis_s, vis);
            const int c0 = (int)max((int64_t)0, min((int64_t)nw, p - (WINDOW - 1) - lo));        // committed rows c0 .. nw-1
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
    uint32_t mx = 0u;
    const uint4* win = reinterpret_cast<const uint4*>(a.swa + ((int64_t)b * a.swa_len + (lo - s0)) * D_LAT);
    const uint4* dr = reinterpret_cast<const uint4*>(a.draft + (int64_t)b * N * D_LAT);
    uint4 x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int v = tid + i * 1024, r = v >> 6, j = r - nw;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < nw)
            x[i] = win[v];
        else if (r < n_rows && ((there[j >> 5] >> (j & 31)) & 1u))
            x[i] = dr[v - nw * 64];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = max(mx, bf16_absmax8(x[i]));
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) atomicMax(&mx_s, mx);
    __syncthreads();
    const int e = f16_range_exp(mx_s);
    const float down = pow2f(-e);
    uint4* rows = reinterpret_cast<uint4*>(a.t.rows16 + (int64_t)b * a.t.row_stride * D_LAT);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int v = tid + i * 1024;
        if (v < n_rows * 64) rows[v] = bf16x8_to_f16x8(x[i], down);
    }
    if (tid == 0) a.t.seq[b] = TreeSeq{vis_s, n_rows, row_tiles, e};
}

namespace {
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
struct NodeParts {
    size_t seq, vis, mask, rows;
    NodeParts(int batch, int n_q)
        : seq(up256((size_t)batch * sizeof(TreeSeq))),
          vis(up256((size_t)batch * n_q * sizeof(int))),
          mask((size_t)batch * n_q * 8 * sizeof(uint32_t)),
          rows((size_t)batch * (WINDOW - 1 + n_q) * D_LAT * sizeof(uint16_t)) {
        mask = up256(mask);
    }
};
}  // namespace

size_t tree_nodes_bytes(int batch, int n_q) {
    const NodeParts p(batch, n_q);
    return p.seq + p.vis + p.mask + p.rows;
}

uint8_t* tree_nodes_take(TreeNodes& t, int batch, int n_q, uint8_t* w) {
    const NodeParts p(batch, n_q);
    t.seq = reinterpret_cast<TreeSeq*>(w), w += p.seq;
    t.vis = reinterpret_cast<int*>(w), w += p.vis;
    t.mask = reinterpret_cast<uint32_t*>(w), w += p.mask;
    t.rows16 = reinterpret_cast<uint16_t*>(w), w += p.rows;
    t.row_stride = WINDOW - 1 + n_q;
    return w;
}

cudaError_t launch_tree_prep(const TreeCall& c, cudaStream_t st) {
    const int zero = c.out_size == 0 ? 0 : std::min(16, (c.n_q * c.n_heads + 511) / 512);
    launch_k(k_tree_prep, dim3((unsigned)c.batch, (unsigned)(1 + zero)), 1024, 0, st, c);
    note_launch();
    return cudaGetLastError();
}

}  // namespace csa2
