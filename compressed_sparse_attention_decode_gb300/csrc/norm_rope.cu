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
// this row's sum is complete.  Measured: 4,096 tokens of 64 + 1 rows of 512 in bf16, 90 us,
// 6.0 TB/s (0.90 of a plain copy); a single token's 65 rows 2.8 us, which is the launch and one
// row's chain of loads.
//
// Angles.  p * f in turns, modulo one, as a 64-bit fraction: f / 2pi in units of
// 2^-64 turns (a 24-bit mantissa times a 64-bit 1/2pi), times p modulo 2^64.  Exact
// to |p| (1 + |f| / 4) 2^-64 turns, so positions past 2^24 lose nothing, and no 64-bit
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

// (a0, a1) = (a0 b0, a1 b1) in one packed instruction
__device__ __forceinline__ void mul2_rn(float& a0, float& a1, float b0, float b1) {
    asm("{\n .reg .b64 ra, rb;\n mov.b64 ra, {%0, %1};\n mov.b64 rb, {%2, %3};\n mul.rn.f32x2 ra, ra, rb;\n"
        " mov.b64 {%0, %1}, ra;\n}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

struct NrArgs {
    NrRows set[2];                           // queries, keys
    int64_t n_tok;
    unsigned q_blocks;                       // blocks below take query rows, the others key rows
    int rows_per_block[2], lanes, d, d_rot, table;
    const int64_t* pos;
    const float* inv_freq;
    float eps, inv_d;
    int norm, halves, inverse, y_type, x_wide, y_wide;
};

// VEC consecutive elements per access, NCH accesses per lane and row (up to NCH unless FULL).  SWAP: a
// pair's two values lie in different lanes and meet in a row buffer.  Rows whose alignment does not hold for
// wide accesses are read or written an element at a time (never FULL).  Issue slots are what this kernel
// runs out of first (a 1 KB row is 45 clocks of its SM's share of HBM), so sizes are compile-time where
// the common shapes allow and the products go two at a time.
template <typename TX, int VEC, int NCH, bool SWAP, bool FULL>
__global__ void __launch_bounds__(NR_THREADS, VEC * NCH > 16 ? 1 : VEC == 1 ? 2 : SWAP ? 3 : 4)
    k_norm_rope(const NrArgs g) {
    extern __shared__ __align__(16) float2 cs[];     // [tokens of this block][d_rot / 2] (cos, sin); row buffers
    const bool isq = blockIdx.x < g.q_blocks;
    const NrRows R = g.set[isq ? 0 : 1];
    const int heads = R.heads, d = g.d, d_rot = g.d_rot, half = d_rot / 2, keep = d - d_rot;
    const int lanes = FULL && NCH > 1 ? 32 : g.lanes;
    const int rpb = g.rows_per_block[isq ? 0 : 1];
    const int64_t r0 = (int64_t)(isq ? blockIdx.x : blockIdx.x - g.q_blocks) * rpb;
    const int nr = (int)min((int64_t)rpb, g.n_tok * heads - r0);
    const int64_t t0 = r0 / heads;
    const int h0 = (int)(r0 - t0 * heads);
    const int nt = (h0 + nr - 1) / heads + 1;
    const int sub = threadIdx.x & (lanes - 1);               // lane within the row
    const int slots = NR_THREADS / lanes, slot = threadIdx.x / lanes;
    float* buf = reinterpret_cast<float*>(cs + g.table) + slot * d_rot;
    pdl_wait();                              // x, the weights and the positions may come from the preceding kernel

    // Row i of the block is head h of its token t.  Slots past the last row repeat it and store nothing.
    const int last = nr - 1;
    int i = slot, t = (h0 + min(i, last)) / heads, h = h0 + min(i, last) - t * heads;
    const int dt = slots / heads, dh = slots - dt * heads;   // a step of `slots` rows
    const TX* x0 = reinterpret_cast<const TX*>(R.x) + t0 * R.x_tok;
    ElemVec<TX, VEC> v[NCH];                 // this lane's columns
    auto load = [&](int t, int h) {
        const TX* x = x0 + t * R.x_tok + h * R.x_head;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (FULL || (j < d && g.x_wide))
                v[c].load(x + j);
            else if (j < d)
                v[c].load_each(x + j);
            else
#pragma unroll
                for (int k = 0; k < ElemVec<TX, VEC>::WORDS; ++k) v[c].w[k] = 0u;
        }
    };
    load(t, h);                              // in flight while the angles are computed
    constexpr bool WREG = VEC > 1;                           // weights in registers (else read as they are used)
    float w[WREG ? NCH : 1][VEC];
    if (WREG) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int j = (sub + c * lanes) * VEC + e;
                w[c][e] = R.w == nullptr ? 1.0f : FULL || j < d ? R.w[j] : 0.0f;
            }
    }
    for (int k = threadIdx.x; k < nt * half; k += NR_THREADS) {
        const int tt = k / half, c = k - tt * half;
        const float f = g.inv_freq[c];
        const unsigned long long a = nr_turns(f) * (unsigned long long)g.pos[t0 + tt];
        float s, co;
        sincospif((float)(long long)a * 0x1p-63f, &s, &co);      // half turns in [-1, 1)
        if (!isfinite(f)) s = co = __int_as_float(0x7fc00000);
        cs[k] = make_float2(co, g.inverse ? -s : s);
    }
    __syncthreads();

    for (int i0 = 0; i0 < nr; i0 += slots, i += slots) {     // the same trip count for every lane of a warp
        const bool live = i <= last;
        const int ct = t, ch = h;
        float a[NCH][VEC], ss[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) a[c][e] = v[c].get(e);
            if (VEC == 1)
                ss[0] = fmaf(a[c][0], a[c][0], ss[0]);
            else
#pragma unroll
                for (int e = 0; e + 1 < VEC; e += 2) fma2_rn(ss[0], ss[1], a[c][e], a[c][e + 1], a[c][e], a[c][e + 1]);
        }
        __syncwarp();                                        // every load of a row before its stores: y may be x
        if (i + slots <= last) {                             // the next row, while this one's sum goes round
            t += dt, h += dh;
            if (h >= heads) h -= heads, ++t;
            load(t, h);
        }
        float r = 1.0f;
        if (g.norm) {
            float sum = ss[0] + ss[1];
            for (int o = lanes >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r = rsqrtf(fmaf(sum, g.inv_d, g.eps));
        }
        const float2* tab = cs + ct * half;
        const int64_t y0 = (t0 + ct) * R.y_tok + ch * R.y_head;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (VEC == 1) {
                a[c][0] *= r;
                if (R.w != nullptr && j < d) a[c][0] *= R.w[j];
            } else {
#pragma unroll
                for (int e = 0; e + 1 < VEC; e += 2) {
                    float w0 = w[WREG ? c : 0][e], w1 = w[WREG ? c : 0][VEC > 1 ? e + 1 : e];
                    mul2_rn(w0, w1, r, r);
                    mul2_rn(a[c][e], a[c][VEC > 1 ? e + 1 : e], w0, w1);
                }
            }
            if (SWAP && live && (FULL || j < d) && j >= keep) {
                if constexpr (VEC == 1)
                    buf[j - keep] = a[c][0];
                else
#pragma unroll
                    for (int e = 0; e < VEC; e += 4)
                        *reinterpret_cast<float4*>(buf + j - keep + e) = make_float4(a[c][e], a[c][e + 1], a[c][e + 2], a[c][e + 3]);
            }
        }
        if (SWAP) __syncwarp();
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (!live || !(FULL || j < d)) continue;
            if (j >= keep) {
                const int u = j - keep;
                if (!SWAP) {
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2) {
                        const float2 z = tab[(u + e) >> 1];
                        const float p0 = a[c][e], p1 = a[c][e + 1];
                        a[c][e] = p0 * z.x - p1 * z.y;
                        a[c][e + 1] = p0 * z.y + p1 * z.x;
                    }
                } else if (VEC == 1) {
                    const bool first = g.halves ? u < half : !(u & 1);
                    const float p = buf[g.halves ? (first ? u + half : u - half) : (u ^ 1)];
                    const float2 z = tab[g.halves ? (first ? u : u - half) : u >> 1];
                    a[c][0] = first ? a[c][0] * z.x - p * z.y : p * z.y + a[c][0] * z.x;
                } else {                                     // halves: a whole access lies on one side
                    const bool first = u < half;
                    const float* p = buf + (first ? u + half : u - half);
                    const float4* z = reinterpret_cast<const float4*>(tab + (first ? u : u - half));
#pragma unroll
                    for (int e = 0; e + 3 < VEC; e += 4) {
                        const float4 q4 = *reinterpret_cast<const float4*>(p + e);
                        const float4 z0 = z[e / 2], z1 = z[e / 2 + 1];
                        const float pp[4] = {q4.x, q4.y, q4.z, q4.w}, cc[4] = {z0.x, z0.z, z1.x, z1.z},
                                    sn[4] = {z0.y, z0.w, z1.y, z1.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[c][e + i] = first ? a[c][e + i] * cc[i] - pp[i] * sn[i] : pp[i] * sn[i] + a[c][e + i] * cc[i];
                    }
                }
            }
            const auto put = [&](const auto& o, auto* p) {
                if (FULL || g.y_wide)
                    o.store(p);
                else
                    o.store_each(p);
            };
            if (g.y_type == CSA2_BF16) {
                ElemVec<__nv_bfloat16, VEC> o;
                o.pack(a[c]);
                put(o, reinterpret_cast<__nv_bfloat16*>(R.y) + y0 + j);
            } else if (g.y_type == CSA2_F16) {
                ElemVec<__half, VEC> o;
                o.pack(a[c]);
                put(o, reinterpret_cast<__half*>(R.y) + y0 + j);
            } else {
                ElemVec<float, VEC> o;
                o.pack(a[c]);
                put(o, reinterpret_cast<float*>(R.y) + y0 + j);
            }
        }
        if (SWAP) __syncwarp();                              // the row buffer is read before the next row writes it
    }
    // The attention stages its queries and window rows before it waits for the kernel before it, and
    // this kernel writes those: it never lets its successor start early, and its rows are visible to
    // the whole GPU before its blocks end (one fence for all threads, ordered after their stores by the
    // block's barrier).
    __syncthreads();
    if (threadIdx.x == 0) __threadfence();
}

namespace {

template <typename TX, int VEC, int NCH>
cudaError_t nr_launch(const NrRows& q, const NrRows& k, int64_t n_tok, int d, int d_rot, const int64_t* pos,
                      const float* inv_freq, float eps, int norm, int halves, int inverse, int y_type, int x_wide, int y_wide,
                      cudaStream_t st) {
    int lanes = 1;
    while (lanes < 32 && lanes * VEC < d) lanes *= 2;
    const int slots = NR_THREADS / lanes;
    const int64_t n_rows = n_tok * (q.heads + k.heads);
    // Rows per block: one round of slots until the grid fills the GPU several times over, then more
    // rounds, which share the block's angles and weights (4,096 tokens x 64 heads of 512: 105 us with four
    // rounds, 92 with sixteen, 90 with thirty-two), while a set's angles stay within 16 KB
    auto table = [&](int heads, int r) { return heads == 0 ? 0 : (int)(((r * slots - 1) / heads + 2) * (d_rot / 2)); };
    int rounds[2] = {1, 1}, cs = 0;
    const int heads[2] = {q.heads, k.heads};
    for (int i = 0; i < 2; ++i) {
        while (rounds[i] < 32 && n_rows / ((int64_t)slots * rounds[i] * 2) >= 152 * 3 && table(heads[i], rounds[i] * 2) <= 2048)
            rounds[i] *= 2;
        cs = std::max(cs, table(heads[i], rounds[i]));
    }
    cs = (cs + 1) & ~1;                          // the row buffers start on 16 bytes
    const int rq = rounds[0] * slots, rk = rounds[1] * slots;
    const int64_t qb = (n_tok * q.heads + rq - 1) / rq, kb = (n_tok * k.heads + rk - 1) / rk;
    if (qb + kb > 0x7fffffff) return cudaErrorInvalidConfiguration;
    // the angles, and one row's rotated values per slot where a pair's values lie in different lanes
    const bool swap = VEC == 1 || halves, full = VEC == 8 && NCH <= 2 && d == lanes * VEC * NCH && x_wide && y_wide;
    const size_t smem = cs * sizeof(float2) + (swap ? (size_t)slots * d_rot * sizeof(float) : 0);
    const NrArgs a{{q, k}, n_tok, (unsigned)qb, {rq, rk}, lanes, d, d_rot, cs, pos, inv_freq, eps, 1.0f / (float)d,
                   norm, halves, inverse, y_type, x_wide, y_wide};
    void (*kern)(NrArgs) = k_norm_rope<TX, VEC, NCH, true, false>;
    if constexpr (VEC > 1) {
        constexpr bool F = VEC == 8 && NCH <= 2;
        kern = swap ? (full ? k_norm_rope<TX, VEC, NCH, true, F> : k_norm_rope<TX, VEC, NCH, true, false>)
                    : (full ? k_norm_rope<TX, VEC, NCH, false, F> : k_norm_rope<TX, VEC, NCH, false, false>);
    }
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    launch_k(kern, dim3((unsigned)(qb + kb)), NR_THREADS, smem, st, a);
    note_launch();
    return cudaGetLastError();
}

// vec: the widest piece that the sizes and the rotation's boundaries allow
template <typename TX, typename... A>
cudaError_t nr_pick(int vec, int d, A... a) {
    if (vec == 8) return d <= 256 ? nr_launch<TX, 8, 1>(a...) : d <= 512 ? nr_launch<TX, 8, 2>(a...) : nr_launch<TX, 8, 4>(a...);
    if (vec == 4) return d <= 128 ? nr_launch<TX, 4, 1>(a...) : d <= 512 ? nr_launch<TX, 4, 4>(a...) : nr_launch<TX, 4, 8>(a...);
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
    int vec = 1, x_wide = 1, y_wide = 1;
    for (int v = 8; v >= 4 && vec == 1; v /= 2)
        if (d % v == 0 && d_rot % v == 0 && (!halves || d_rot / 2 % v == 0)) vec = v;
    // a piece moves min(16, vec * size) aligned bytes at a time
    const int xb = std::min(16, vec * xs), yb = std::min(16, vec * ys);
    const csa2_head_rows* in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        if (!in[i] || in[i]->n_heads == 0) continue;
        const csa2_head_rows& r = *in[i];
        rows[i] = NrRows{r.x, r.y, r.weight, r.x_tok, r.x_head, r.y_tok, r.y_head, r.n_heads};
        x_wide &= reinterpret_cast<uintptr_t>(r.x) % xb == 0 && r.x_tok * xs % xb == 0 && r.x_head * xs % xb == 0;
        y_wide &= reinterpret_cast<uintptr_t>(r.y) % yb == 0 && r.y_tok * ys % yb == 0 && r.y_head * ys % yb == 0;
    }
    const auto pick = [&](auto tx) {
        return nr_pick<decltype(tx)>(vec, d, rows[0], rows[1], (int64_t)n_tok, d, d_rot, pos, inv_freq, eps, norm, halves,
                                     inverse, y_type, x_wide, y_wide, st);
    };
    if (x_type == CSA2_BF16) return pick(__nv_bfloat16());
    if (x_type == CSA2_F16) return pick(__half());
    return pick(0.0f);
}

}  // namespace csa2
