// Attention of a tree of drafted tokens over the FP4 cache: what csa2_dense_attn and csa2_sparse_attn compute for
// queries in a row, for the nodes of a tree whose own rows are not in the cache yet ("DeepSeek-v4.1 Flash:
// KVキャッシュ圧縮の限界を押し広げる" §1.1: one 512-dim latent, key and value of every head; §2.3.1: the top-k entries
// and the local window).  Node i at raw position p, with the chain of its `len` last tokens that are drafted (itself
// and its ancestors), attends to
//     the entries 0 .. floor((p - 127) / ratio) - 1, or those that its index list names;
//     the committed window rows of positions max(0, p - 127) .. p - len;
//     the draft rows of its chain (at most 128, so that they always lie in the window).
//
// One block of 8 warps a node and 8 heads, a warp a head: 32 rows at a time as fp32 in shared memory, an online
// softmax with 16 of the output's dims a lane.
#include "common.cuh"
#include "elem.cuh"

namespace csa2 {

constexpr int TS_TILE = 32, TS_HEADS = 8;

struct TreeArgs {
    const uint8_t *codes, *scales;
    int capacity, ratio;
    const uint16_t* q;
    int n_q, n_heads;
    const int64_t* q_pos;
    const int32_t* parent;
    const uint16_t* draft;
    const int32_t* idx;
    int k;                       // < 0: every visible entry
    const uint16_t* swa;
    const int64_t* swa_pos0;
    int swa_len;
    float scale;
    float* lse;
};

template <typename TO>
__global__ void __launch_bounds__(256) k_tree_attn_simt(const __grid_constant__ TreeArgs a, TO* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    extern __shared__ float sm[];
    float* qs = sm;                                  // [8][512]
    float* tile = qs + TS_HEADS * D_LAT;             // [32][512]
    __shared__ int chain[128], there[TS_TILE], len_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h0 = blockIdx.x * TS_HEADS, i = blockIdx.y, b = blockIdx.z, h = h0 + warp;
    const int64_t gq = (int64_t)b * a.n_q + i;
    if (tid == 0) {
        int n = 0, j = i;
        const int32_t* parent = a.parent + (int64_t)b * a.n_q;
        while (j >= 0) {
            chain[n++] = j;
            const int up = parent[j];
            j = up >= -1 && up < j ? up : -2;
        }
        len_s = j == -1 ? n : 0;
    }
    for (int v = tid; v < TS_HEADS * D_LAT; v += 256)
        qs[v] = h0 + v / D_LAT < a.n_heads ? bf16_bits_to_f32(a.q[(gq * a.n_heads + h0) * D_LAT + v]) : 0.0f;
    __syncthreads();
    const int len = len_s;
    const int64_t p = a.q_pos[gq], s0 = a.swa_pos0 ? a.swa_pos0[b] : 0;
    const int64_t vis = p >= WINDOW - 1 ? (p - (WINDOW - 1)) >> (a.ratio - 1) : 0;
    const int n4 = len == 0 ? 0 : a.k >= 0 ? a.k : (int)min(vis, (int64_t)a.capacity);
    const int64_t lo = max(max((int64_t)0, p - (WINDOW - 1)), s0), hi = min(p - len, s0 + a.swa_len - 1);
    const int nw = len > 0 && hi >= lo ? (int)(hi - lo + 1) : 0;
    const int64_t n = (int64_t)n4 + nw + len;
    float m = -INFINITY, l = 0.0f, o[16] = {};
    for (int64_t t = 0; t < n; t += TS_TILE) {
        __syncthreads();
        const int r = tid >> 3, part = tid & 7;                          // 8 threads a row, 64 dims each
        const int64_t s = t + r;
        float* dst = tile + r * D_LAT + part * 64;
        const uint16_t* src = nullptr;
        bool ok = false;
        if (s < n4) {
            const int64_t j = a.k >= 0 ? (int64_t)a.idx[gq * a.k + s] : s;
            ok = j >= 0 && j < a.capacity;
            if (ok) {
                const int64_t row = (int64_t)b * a.capacity + j;
                for (int g = 0; g < 4; ++g) {
                    const uint32_t c0 = reinterpret_cast<const uint32_t*>(a.codes + row * (D_LAT / 2) + part * 32)[2 * g];
                    const uint32_t c1 = reinterpret_cast<const uint32_t*>(a.codes + row * (D_LAT / 2) + part * 32)[2 * g + 1];
                    const float f = e4m3_to_f32(a.scales[row * (D_LAT / 16) + part * 4 + g]);
                    for (int e = 0; e < 16; ++e) {
                        const uint32_t code = ((e < 8 ? c0 : c1) >> (4 * (e & 7))) & 15u, mag = code & 7u;
                        const float v = mag < 2 ? 0.5f * mag : (float)(1u << ((mag >> 1) - 1)) * ((mag & 1) ? 1.5f : 1.0f);
                        dst[16 * g + e] = (code & 8u ? -v : v) * f;
                    }
                }
            }
        } else if (s < n4 + nw) {
            src = a.swa + ((int64_t)b * a.swa_len + (lo - s0) + (s - n4)) * D_LAT;
        } else if (s < n) {
            src = a.draft + ((int64_t)b * a.n_q + chain[s - n4 - nw]) * D_LAT;
        }
        if (src != nullptr) {
            ok = true;
            for (int e = 0; e < 64; ++e) dst[e] = bf16_bits_to_f32(src[part * 64 + e]);
        }
        if (part == 0) there[r] = ok;
        __syncthreads();
        if (h < a.n_heads)
            for (int k = 0; k < TS_TILE; ++k) {
                if (!there[k]) continue;
                const float* row = tile + k * D_LAT;
                float dot = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) dot = fmaf(qs[warp * D_LAT + lane + 32 * e], row[lane + 32 * e], dot);
                for (int w = 16; w; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
                const float x = dot * a.scale;
                if (x > m) {
                    const float f = expf(m - x);
                    l *= f, m = x;
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= f;
                }
                const float w = expf(x - m);
                l += w;
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = fmaf(w, row[lane + 32 * e], o[e]);
            }
    }
    if (h >= a.n_heads) return;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) out[(gq * a.n_heads + h) * D_LAT + lane + 32 * e] = from_f32<TO>(o[e] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[gq * a.n_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

size_t tree_attn_ws(int, int, int, int, int64_t) { return 256; }

cudaError_t launch_tree_attn(const csa2_cache& c, const uint16_t* q, int n_q, int n_heads, const int64_t* q_pos,
                             const int32_t* parent, const uint16_t* draft, const int32_t* idx, int k, const uint16_t* swa,
                             const int64_t* swa_pos0, int swa_len, float scale, void* out, int out_type, float* lse, void*,
                             cudaStream_t st) {
    const TreeArgs a{c.lat_codes, c.lat_scales, c.capacity, c.ratio, q, n_q, n_heads, q_pos, parent, draft, idx, k,
                     swa, swa_pos0, swa_len, scale, lse};
    const size_t smem = (TS_HEADS + TS_TILE) * D_LAT * sizeof(float);
    auto go = [&](auto* y) {
        const auto kern = k_tree_attn_simt<std::remove_pointer_t<decltype(y)>>;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        launch_k(kern, dim3((n_heads + TS_HEADS - 1) / TS_HEADS, n_q, c.batch), 256, smem, st, a, y);
        note_launch();
        return cudaGetLastError();
    };
    return out_type == CSA2_F32   ? go(reinterpret_cast<float*>(out))
           : out_type == CSA2_F16 ? go(reinterpret_cast<__half*>(out))
                                  : go(reinterpret_cast<__nv_bfloat16*>(out));
}

}  // namespace csa2
