// Per-head RMS norm with the position rotation in the same pass, for the query
// heads and the key rows of a step.  For a head row x of d values at raw
// position p:
//     v_j = x_j * rsqrt(mean_i x_i^2 + eps) * w_j        (or v = x without the norm)
//     the last d_rot values of v, as d_rot/2 pairs (a_i, b_i), are turned by the
//     angle p * f_i:  a' = a cos - b sin, b' = a sin + b cos   (back: -angle)
// Sums, norm and rotation are in fp32; the result is rounded once.
//
// Bound: memory, each row read and written once.  A row belongs to L lanes (the
// power of two that covers it in 8-value pieces, a whole warp from 256 values on),
// each with the same columns of every row: the weights stay in registers, the sum
// of squares is L-lane shuffles, and shared memory holds the angles alone (and,
// where the two values of a pair lie in different lanes, one row's rotated values
// per slot).  A block takes consecutive rows (tokens x heads) of one set and computes
// the cosines and sines of its tokens once: with 64 heads of 512 and 64 rotated
// values that is 32 angles for 64 rows.  The next row's loads are issued before
// this row's sum is complete.
//
// Angles.  p * f in turns, modulo one, as a 64-bit fraction: f / 2pi in units of
// 2^-64 turns (a 24-bit mantissa times a 64-bit 1/2pi), times p modulo 2^64.  Exact
// to about |p| 2^-64 turns, so positions past 2^24 lose nothing, and no 64-bit
// floating point is used (its rate is low on this GPU).
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"

namespace csa2 {

constexpr int NR_THREADS = 256;

struct NrRows {                              // one of the two row sets of a call
    const void* x;
    void* y;
    const float* w;
    int64_t x_tok, x_head, y_tok, y_head;    // strides in elements
    int heads;
};

// f / 2pi modulo one turn, in units of 2^-64 turns (f finite)
__device__ __forceinline__ unsigned long long nr_turns(float f) {
    const uint32_t b = __float_as_uint(f);
    const uint32_t e8 = (b >> 23) & 255u;
    const unsigned long long m = (b & 0x7fffffu) | (e8 ? 0x800000u : 0u);
    const int e = e8 ? (int)e8 : 1;          // f = m * 2^(e - 150)
    // floor(2^66 / 2pi); m * INV is m / 2pi in units of 2^-66
    const unsigned long long INV = 0xa2f9836e4e441529ull;
    unsigned long long lo = m * INV, hi = __umul64hi(m, INV), r;
    const int s = 152 - e;                   // units of 2^-64 turns: m * INV * 2^-s
    if (s <= 0)
        r = s > -64 ? lo << -s : 0ull;
    else if (s < 64)
        r = (lo >> s) | (hi << (64 - s));
    else
        r = s < 128 ? hi >> (s - 64) : 0ull;
    return (b >> 31) ? 0ull - r : r;
}

// VEC consecutive elements per access, up to NCH accesses per lane and row.  Blocks below `q_blocks`
// take query rows, the others key rows: a block's rows share their weights.
template <typename TX, int VEC, int NCH>
__global__ void __launch_bounds__(NR_THREADS, VEC > 1 && VEC * NCH <= 16 ? 4 : VEC * NCH <= 16 ? 2 : 1)
    k_norm_rope(NrRows q, NrRows k, int64_t n_tok, unsigned q_blocks, int rows_per_block, int lanes, int d, int d_rot,
                int table, const int64_t* __restrict__ pos, const float* __restrict__ inv_freq, float eps, int norm,
                int halves, int inverse, int y_type) {
    extern __shared__ float2 cs[];           // [tokens of this block][d_rot / 2] (cos, sin); row buffers
    const bool isq = blockIdx.x < q_blocks;
    const NrRows R = isq ? q : k;
    const int heads = R.heads, half = d_rot / 2, keep = d - d_rot;
    const int64_t n_rows = n_tok * heads;
    const int64_t r0 = (int64_t)(isq ? blockIdx.x : blockIdx.x - q_blocks) * rows_per_block;
    const int nr = (int)min((int64_t)rows_per_block, n_rows - r0);
    const int64_t t0 = r0 / heads;
    const int h0 = (int)(r0 - t0 * heads);
    const int nt = (h0 + nr - 1) / heads + 1;
    const int sub = threadIdx.x & (lanes - 1);               // lane within the row
    const int slots = NR_THREADS / lanes, slot = threadIdx.x / lanes;
    const bool swap = VEC == 1 || halves;                    // a pair's two values lie in different lanes
    float* buf = reinterpret_cast<float*>(cs + table) + slot * d_rot;
    constexpr bool WREG = VEC > 1;                           // weights in registers (else read as they are used)
    float w[WREG ? NCH : 1][VEC];
    if (WREG && R.w != nullptr) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int j = (sub + c * lanes) * VEC + e;
                w[c][e] = j < d ? __ldg(R.w + j) : 0.0f;
            }
    }
    pdl_wait();                              // x and the positions may come from the preceding kernel

    ElemVec<TX, VEC> v[NCH];                 // this lane's columns of row i of the block
    auto load = [&](int i) {
        const int t = (h0 + i) / heads, h = h0 + i - t * heads;
        const TX* x = reinterpret_cast<const TX*>(R.x) + (t0 + t) * R.x_tok + h * R.x_head;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (j < d) v[c].load(x + j);
        }
    };
    if (slot < nr) load(slot);               // in flight while the angles are computed
    for (int i = threadIdx.x; i < nt * half; i += NR_THREADS) {
        const int t = i / half, c = i - t * half;
        const float f = __ldg(inv_freq + c);
        const unsigned long long a = nr_turns(f) * (unsigned long long)pos[t0 + t];
        float s, co;
        sincospif((float)(long long)a * 0x1p-63f, &s, &co);      // half turns in [-1, 1)
        if (!isfinite(f)) s = co = __int_as_float(0x7fc00000);
        cs[i] = make_float2(co, inverse ? -s : s);
    }
    __syncthreads();

    for (int i0 = 0; i0 < nr; i0 += slots) {                 // the same trip count for every lane of a warp
        const int i = i0 + slot;
        const bool live = i < nr;
        float a[NCH][VEC], ss = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                a[c][e] = live && (sub + c * lanes) * VEC < d ? v[c].get(e) : 0.0f;
                ss = fmaf(a[c][e], a[c][e], ss);
            }
        const int t = live ? (h0 + i) / heads : 0, h = live ? h0 + i - t * heads : 0;
        __syncwarp();                                        // every load of a row before its stores: y may be x
        if (i + slots < nr) load(i + slots);                 // the next row, while this one's sum goes round
        float r = 1.0f;
        if (norm) {
            for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(ss / (float)d + eps);
        }
        const float2* tab = cs + t * half;
        const int64_t y0 = (t0 + t) * R.y_tok + h * R.y_head;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                a[c][e] *= r;
                if (R.w != nullptr) a[c][e] *= WREG ? w[WREG ? c : 0][e] : (j + e < d ? __ldg(R.w + j + e) : 0.0f);
            }
            if (swap && live && j < d && j >= keep)
#pragma unroll
                for (int e = 0; e < VEC; ++e) buf[j - keep + e] = a[c][e];
        }
        if (swap) __syncwarp();
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (!live || j >= d) continue;
            if (j >= keep) {
                const int u = j - keep;
                if (!swap) {
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2) {
                        const float2 z = tab[(u + e) >> 1];
                        const float p0 = a[c][e], p1 = a[c][e + 1];
                        a[c][e] = p0 * z.x - p1 * z.y;
                        a[c][e + 1] = p0 * z.y + p1 * z.x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int ue = u + e;
                        const bool first = halves ? ue < half : !(ue & 1);
                        const float p = buf[halves ? (first ? ue + half : ue - half) : (ue ^ 1)];
                        const float2 z = tab[halves ? (first ? ue : ue - half) : ue >> 1];
                        a[c][e] = first ? a[c][e] * z.x - p * z.y : p * z.y + a[c][e] * z.x;
                    }
                }
            }
            if (y_type == CSA2_BF16) {
                ElemVec<__nv_bfloat16, VEC> o;
                o.pack(a[c]);
                o.store(reinterpret_cast<__nv_bfloat16*>(R.y) + y0 + j);
            } else if (y_type == CSA2_F16) {
                ElemVec<__half, VEC> o;
                o.pack(a[c]);
                o.store(reinterpret_cast<__half*>(R.y) + y0 + j);
            } else {
                ElemVec<float, VEC> o;
                o.pack(a[c]);
                o.store(reinterpret_cast<float*>(R.y) + y0 + j);
            }
        }
        if (swap) __syncwarp();                              // the row buffer is read before the next row writes it
    }
    // The attention stages its queries and window rows before it waits for the kernel before it, and
    // this kernel writes those: it never lets its successor start early, and its rows are visible to
    // the whole GPU before its blocks end.
    __threadfence();
}

namespace {

template <typename TX, int VEC, int NCH>
cudaError_t nr_launch(const NrRows& q, const NrRows& k, int64_t n_tok, int d, int d_rot, const int64_t* pos,
                      const float* inv_freq, float eps, int norm, int halves, int inverse, int y_type, cudaStream_t st) {
    int lanes = 1;
    while (lanes < 32 && lanes * VEC < d) lanes *= 2;
    const int slots = NR_THREADS / lanes;
    const int64_t n_rows = n_tok * (q.heads + k.heads);
    // Rows per block: one round of slots until the grid fills the GPU several times over, then more
    // rounds, which share the block's angles and weights, while the angles stay within 16 KB
    const int few = std::min(q.heads ? q.heads : k.heads, k.heads ? k.heads : q.heads);
    int rounds = 1;
    auto table = [&](int r) { return (int)(((r * slots - 1) / few + 2) * (d_rot / 2)); };
    while (rounds < 8 && n_rows / ((int64_t)slots * rounds * 2) >= 152 * 8 && table(rounds * 2) <= 2048) rounds *= 2;
    const int rpb = rounds * slots;
    const int64_t qb = (n_tok * q.heads + rpb - 1) / rpb, kb = (n_tok * k.heads + rpb - 1) / rpb;
    if (qb + kb > 0x7fffffff) return cudaErrorInvalidConfiguration;
    // the angles, and one row's rotated values per slot where a pair's values lie in different lanes
    const size_t smem = table(rounds) * sizeof(float2) + (VEC == 1 || halves ? (size_t)slots * d_rot * sizeof(float) : 0);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_norm_rope<TX, VEC, NCH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    launch_k(k_norm_rope<TX, VEC, NCH>, dim3((unsigned)(qb + kb)), NR_THREADS, smem, st, q, k, n_tok, (unsigned)qb, rpb,
             lanes, d, d_rot, table(rounds), pos, inv_freq, eps, norm, halves, inverse, y_type);
    note_launch();
    return cudaGetLastError();
}

// vec: the widest access that pointers, strides, sizes and the rotation's boundaries allow
template <typename TX, typename... A>
cudaError_t nr_pick(int vec, int d, A... a) {
    if (vec == 8) return d <= 256 ? nr_launch<TX, 8, 1>(a...) : d <= 512 ? nr_launch<TX, 8, 2>(a...) : nr_launch<TX, 8, 4>(a...);
    if (vec == 4) return d <= 512 ? nr_launch<TX, 4, 4>(a...) : nr_launch<TX, 4, 8>(a...);
    return d <= 128 ? nr_launch<TX, 1, 4>(a...) : d <= 512 ? nr_launch<TX, 1, 16>(a...) : nr_launch<TX, 1, 32>(a...);
}

}  // namespace

cudaError_t launch_norm_rope(const csa2_head_rows* q, const csa2_head_rows* k, int x_type, int y_type, int n_tok, int d,
                             int d_rot, const int64_t* pos, const float* inv_freq, float eps, int flags,
                             cudaStream_t st) {
    const int norm = !(flags & CSA2_ROPE_NO_NORM), halves = !!(flags & CSA2_ROPE_HALVES),
              inverse = !!(flags & CSA2_ROPE_INVERSE);
    const int xs = x_type == CSA2_F32 ? 4 : 2, ys = y_type == CSA2_F32 ? 4 : 2;
    NrRows rows[2] = {};
    int vec = 8;
    const csa2_head_rows* in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        if (!in[i] || in[i]->n_heads == 0) continue;
        const csa2_head_rows& r = *in[i];
        rows[i] = NrRows{r.x, r.y, r.weight, r.x_tok, r.x_head, r.y_tok, r.y_head, r.n_heads};
        for (int v = 8; v >= 4; v /= 2) {
            // an access of v elements moves min(16, v * size) aligned bytes at a time
            const int xb = v * xs < 16 ? v * xs : 16, yb = v * ys < 16 ? v * ys : 16;
            const bool fits = reinterpret_cast<uintptr_t>(r.x) % xb == 0 && reinterpret_cast<uintptr_t>(r.y) % yb == 0 &&
                              r.x_tok * xs % xb == 0 && r.x_head * xs % xb == 0 && r.y_tok * ys % yb == 0 &&
                              r.y_head * ys % yb == 0 && d % v == 0 && d_rot % v == 0 && (!halves || d_rot / 2 % v == 0);
            if (!fits && vec >= v) vec = v == 8 ? 4 : 1;
        }
    }
    const auto pick = [&](auto tx) {
        return nr_pick<decltype(tx)>(vec, d, rows[0], rows[1], (int64_t)n_tok, d, d_rot, pos, inv_freq, eps, norm, halves,
                                     inverse, y_type, st);
    };
    if (x_type == CSA2_BF16) return pick(__nv_bfloat16());
    if (x_type == CSA2_F16) return pick(__half());
    return pick(0.0f);
}

}  // namespace csa2
