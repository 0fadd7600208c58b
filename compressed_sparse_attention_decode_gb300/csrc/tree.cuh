// What both kernels of drafted trees (attn_tree.cu: every visible entry, attn_list.cu: index lists) take from k_tree_prep.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "fp4_f16.cuh"

namespace csa2 {

// what the nodes of a sequence attend to, all together
struct TreeSeq {
    int n_vis;                   // entries 0 .. n_vis-1
    int n_rows;                  // rows of rows16: the committed window rows, then the drafts up to the last node that is there
    int row_tiles;               // items of attn_tree.cu
    int pad;
};
constexpr int TREE_GROUPS = 16;  // of 16 rows each: at most 255 rows
// A call's parts of the workspace that k_tree_prep writes
struct TreeNodes {
    TreeSeq* seq;                // [batch]
    int* vis;                    // [batch][n_q] entries that a node sees
    uint32_t* mask;              // [batch][n_q][8] which of the n_rows rows, 128 at most; none for a node that is not there
    // fp16, row r a 2^-exps[r] of the window row or draft (tree_row_exp), zeros for drafts that are not there
    uint16_t* rows16;            // [batch][row_stride][512]
    int8_t* exps;                // [batch][256]
    int* off;                    // [batch][TREE_GROUPS] whether a row of the group has another exponent than 0
    int row_stride;
    // the queries as fp16, row r a 2^-q_exps[r] of q's (times -1 where neg_q)
    uint16_t* q16;               // [batch][n_q][n_heads][512], or q_tiles: [batch][64 rows][8 slabs of 64 dims][64][64], swizzled
    int8_t* q_exps;              // [batch][n_q][n_heads]
};
// Whether any of a sequence's rows has another exponent than 0 (a whole warp calls it)
__device__ __forceinline__ bool tree_scaled(const TreeNodes& t, int b, int n_rows) {
    const int lane = threadIdx.x & 31;
    return __any_sync(0xffffffffu, lane * 16 < n_rows && t.off[b * TREE_GROUPS + lane] != 0);
}
// |scale| 2^e times a score, -200 <= e <= 252, in steps that leave fp32's range only where the whole does
__device__ __forceinline__ float tree_score(float x, float scale, int e) {
    return x * scale * pow2f(e >> 1) * pow2f(e - (e >> 1));
}
struct TreeCall {
    int batch, capacity, ratio, n_q, n_heads;
    const int64_t* q_pos;
    const int32_t* parent;
    const uint16_t* draft;
    const uint16_t* swa;
    const int64_t* swa_pos0;
    int swa_len;
    TreeNodes t;
    const uint16_t* q;
    bool neg_q, q_tiles;
    void* out;                   // or NULL: rows of attn_tree.cu's items that nobody works on are written by k_tree_prep
    float* lse;
    int out_size;                // bytes of an element
};
// rows of q16 that a sequence has
inline int tree_q_rows(int n_q, int n_heads, bool q_tiles) { return q_tiles ? (n_q * n_heads + 127) / 128 * 128 : n_q * n_heads; }
// Sequences of a pass: 65,536 rows at most (of one sequence 16,384), whose fp16 queries are 64 MB
inline int tree_pass(int batch, int q_rows) { return std::min(batch, (1 << 16) / q_rows); }
// a workspace's bytes for a pass, and its pointers from byte w on (returns the first byte after it)
size_t tree_nodes_bytes(int batch, int n_q, int q_rows);
uint8_t* tree_nodes_take(TreeNodes& t, int batch, int n_q, int q_rows, uint8_t* w);
// byte of 16-byte chunk `chunk` of row `row` of a 128-byte swizzled slab
__device__ __forceinline__ uint32_t tree_swz(uint32_t row, uint32_t chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }
cudaError_t launch_tree_prep(const TreeCall& c, cudaStream_t st);

// 16 bytes from global to shared memory, zeros where `there` is false
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace csa2
