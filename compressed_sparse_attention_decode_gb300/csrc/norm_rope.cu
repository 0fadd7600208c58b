// Per-head RMS norm with the position rotation in the same pass, for the query
// heads and the key rows of a step.  For a head row x of d values at raw
// position p:
//     v_j = x_j * rsqrt(mean_i x_i^2 + eps) * w_j        (or v = x without the norm)
//     the last d_rot values of v, as d_rot/2 pairs (a_i, b_i), are turned by the
//     angle p * f_i:  a' = a cos - b sin, b' = a sin + b cos   (back: -angle)
// Sums, norm and rotation are in fp32; the result is rounded once.
//
// Bound: memory, each row read and written once.  A row belongs to L lanes (the
// power of two that covers it in 16-byte pieces, a whole warp from 256 values
// on), each with the same columns of every row, so the sum of squares is L-lane
// shuffles and nothing goes through shared memory but the angles.  A block takes
// consecutive rows (tokens x heads) and computes the cosines and sines of its
// tokens once: with 64 heads of 512 and 64 rotated values that is 32 angles for
// 64 rows.
//
// Angles.  p * f in turns, modulo one, as a 64-bit fraction: f / 2pi in units of
// 2^-64 turns (a 24-bit mantissa times a 64-bit 1/2pi), times p modulo 2^64.  Exact
// to about |p| 2^-64 turns, so positions past 2^24 lose nothing, and no 64-bit
// floating point is used (its rate is low on this GPU).
#include <cmath>

#include "common.cuh"
#include "elem.cuh"

namespace csa2 {

constexpr int NR_THREADS = 256;

struct NrRows {                              // one of the two row sets of a call
    const void* x;
    void* y;
    const float* w;
    int64_t x_tok, x_head, y_tok, y_head;    // strides in elements
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

// VEC consecutive elements per access, up to NCH accesses per lane and row
template <typename TX, typename TY, int VEC, int NCH>
__global__ void __launch_bounds__(NR_THREADS) k_norm_rope(NrRows q, NrRows k, int hq, int hk, int64_t n_rows,
                                                          int rows_per_block, int lanes, int d, int d_rot,
                                                          const int64_t* __restrict__ pos,
                                                          const float* __restrict__ inv_freq, float eps, int norm,
                                                          int halves, int inverse) {
    extern __shared__ float2 cs[];           // [tokens of this block][d_rot / 2] (cos, sin)
    pdl_wait();                              // x and the positions may come from the preceding kernel
    const int rows_tok = hq + hk, half = d_rot / 2;
    const int64_t r0 = (int64_t)blockIdx.x * rows_per_block;
    const int nr = (int)min((int64_t)rows_per_block, n_rows - r0);
    const int64_t t0 = r0 / rows_tok;
    const int h0 = (int)(r0 - t0 * rows_tok);
    const int nt = (h0 + nr - 1) / rows_tok + 1;
    for (int i = threadIdx.x; i < nt * half; i += NR_THREADS) {
        const int t = i / half, c = i - t * half;
        const float f = inv_freq[c];
        const unsigned long long a = nr_turns(f) * (unsigned long long)pos[t0 + t];
        float s, co;
        sincospif((float)(long long)a * 0x1p-63f, &s, &co);      // half turns in [-1, 1)
        if (!isfinite(f)) s = co = __int_as_float(0x7fc00000);
        cs[i] = make_float2(co, inverse ? -s : s);
    }
    __syncthreads();

    const int sub = threadIdx.x & (lanes - 1);               // lane within the row
    const int slots = NR_THREADS / lanes, slot = threadIdx.x / lanes;
    const int keep = d - d_rot;
    for (int i0 = 0; i0 < nr; i0 += slots) {                 // the same trip count for every lane of a warp
        const int i = i0 + slot;
        const bool live = i < nr;
        const int t = live ? (h0 + i) / rows_tok : 0;
        const int h = live ? h0 + i - t * rows_tok : 0;
        const bool isq = h < hq;
        const NrRows& R = isq ? q : k;
        const int hh = isq ? h : h - hq;
        const TX* x = reinterpret_cast<const TX*>(R.x) + (t0 + t) * R.x_tok + hh * R.x_head;
        TY* y = reinterpret_cast<TY*>(R.y) + (t0 + t) * R.y_tok + hh * R.y_head;
        const float* w = R.w;

        ElemVec<TX, VEC> v[NCH], other[NCH];                 // the columns and, where needed, their partners
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (live && j < d) {
                v[c].load(x + j);
                if (j >= keep && (VEC == 1 || halves)) {
                    const int u = j - keep;
                    other[c].load(x + keep + (halves ? (u < half ? u + half : u - half) : (u ^ 1)));
                }
            }
        }
        float r = 1.0f;
        if (norm) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int j = (sub + c * lanes) * VEC;
                if (live && j < d)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss = fmaf(v[c].get(e), v[c].get(e), ss);
            }
            for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(ss / (float)d + eps);
        }
        __syncwarp();                                        // every load of the row before its stores: y may be x
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (sub + c * lanes) * VEC;
            if (!live || j >= d) continue;
            float a[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) a[e] = v[c].get(e) * r;
            if (w != nullptr)
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[e] *= __ldg(w + j + e);
            if (j >= keep) {
                const int u = j - keep;
                const float2* tab = cs + t * half;
                if (VEC > 1 && !halves) {
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2) {
                        const float2 z = tab[(u + e) >> 1];
                        const float p0 = a[e], p1 = a[e + 1];
                        a[e] = p0 * z.x - p1 * z.y;
                        a[e + 1] = p0 * z.y + p1 * z.x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int ue = u + e;
                        const bool first = halves ? ue < half : !(ue & 1);
                        const int up = halves ? (first ? ue + half : ue - half) : (ue ^ 1);
                        const float2 z = tab[halves ? (first ? ue : ue - half) : ue >> 1];
                        float b = other[c].get(e) * r;
                        if (w != nullptr) b *= __ldg(w + keep + up);
                        a[e] = first ? a[e] * z.x - b * z.y : b * z.y + a[e] * z.x;
                    }
                }
            }
            ElemVec<TY, VEC> o;
#pragma unroll
            for (int i2 = 0; i2 < ElemVec<TY, VEC>::WORDS; ++i2) o.w[i2] = 0u;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o.set(e, a[e]);
            o.store(y + j);
        }
    }
    // The attention stages its queries and window rows before it waits for the kernel before it, and
    // this kernel writes those: it never lets its successor start early, and its rows are visible to
    // the whole GPU before its blocks end.
    __threadfence();
}

namespace {

template <typename TX, typename TY, int VEC, int NCH>
cudaError_t nr_launch(const NrRows& q, const NrRows& k, int hq, int hk, int64_t n_tok, int d, int d_rot,
                      const int64_t* pos, const float* inv_freq, float eps, int norm, int halves, int inverse,
                      cudaStream_t st) {
    int lanes = 1;
    while (lanes < 32 && lanes * VEC < d) lanes *= 2;
    const int slots = NR_THREADS / lanes, rows_tok = hq + hk;
    const int64_t n_rows = n_tok * rows_tok;
    // Rows per block: one round of slots until the grid fills the GPU several times over, then more
    // rounds, which share the block's angles, while the angles stay within 32 KB
    int rounds = 1;
    auto table = [&](int r) { return ((size_t)(r * slots - 1) / rows_tok + 2) * (d_rot / 2) * sizeof(float2); };
    while (rounds < 8 && n_rows / ((int64_t)slots * rounds * 2) >= 152 * 8 && table(rounds * 2) <= 32768) rounds *= 2;
    const int rpb = rounds * slots;
    const int64_t blocks = (n_rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    launch_k(k_norm_rope<TX, TY, VEC, NCH>, dim3((unsigned)blocks), NR_THREADS, table(rounds), st, q, k, hq, hk, n_rows, rpb,
             lanes, d, d_rot, pos, inv_freq, eps, norm, halves, inverse);
    note_launch();
    return cudaGetLastError();
}

// the widest access that pointers, strides, sizes and the rotation's boundaries allow
template <typename TX, typename TY, typename... A>
cudaError_t nr_pick(int vec, int d, A... a) {
    if (vec == 8) return d <= 512 ? nr_launch<TX, TY, 8, 2>(a...) : nr_launch<TX, TY, 8, 4>(a...);
    if (vec == 4) return nr_launch<TX, TY, 4, 8>(a...);
    return nr_launch<TX, TY, 1, 32>(a...);
}

template <typename TX, typename... A>
cudaError_t nr_pick_y(int y_type, A... a) {
    if (y_type == CSA2_BF16) return nr_pick<TX, __nv_bfloat16>(a...);
    if (y_type == CSA2_F16) return nr_pick<TX, __half>(a...);
    return nr_pick<TX, float>(a...);
}

}  // namespace

cudaError_t launch_norm_rope(const csa2_head_rows* q, const csa2_head_rows* k, int x_type, int y_type, int n_tok, int d,
                             int d_rot, const int64_t* pos, const float* inv_freq, float eps, int flags,
                             cudaStream_t st) {
    const int norm = !(flags & CSA2_ROPE_NO_NORM), halves = !!(flags & CSA2_ROPE_HALVES),
              inverse = !!(flags & CSA2_ROPE_INVERSE);
    const int xs = x_type == CSA2_F32 ? 4 : 2, ys = y_type == CSA2_F32 ? 4 : 2;
    NrRows rows[2] = {};
    int heads[2] = {0, 0}, vec = 8;
    const csa2_head_rows* in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        if (!in[i] || in[i]->n_heads == 0) continue;
        const csa2_head_rows& r = *in[i];
        rows[i] = NrRows{r.x, r.y, r.weight, r.x_tok, r.x_head, r.y_tok, r.y_head};
        heads[i] = r.n_heads;
        for (int v = 8; v >= 4; v /= 2) {
            // an access of v elements moves min(16, v * size) aligned bytes at a time
            const int xb = v * xs < 16 ? v * xs : 16, yb = v * ys < 16 ? v * ys : 16;
            const bool fits = reinterpret_cast<uintptr_t>(r.x) % xb == 0 && reinterpret_cast<uintptr_t>(r.y) % yb == 0 &&
                              r.x_tok * xs % xb == 0 && r.x_head * xs % xb == 0 && r.y_tok * ys % yb == 0 &&
                              r.y_head * ys % yb == 0 && d % v == 0 && d_rot % v == 0 && (!halves || d_rot / 2 % v == 0);
            if (!fits && vec >= v) vec = v == 8 ? 4 : 1;
        }
    }
    if (x_type == CSA2_BF16)
        return nr_pick_y<__nv_bfloat16>(y_type, vec, d, rows[0], rows[1], heads[0], heads[1], (int64_t)n_tok, d, d_rot, pos,
                                        inv_freq, eps, norm, halves, inverse, st);
    if (x_type == CSA2_F16)
        return nr_pick_y<__half>(y_type, vec, d, rows[0], rows[1], heads[0], heads[1], (int64_t)n_tok, d, d_rot, pos,
                                 inv_freq, eps, norm, halves, inverse, st);
    return nr_pick_y<float>(y_type, vec, d, rows[0], rows[1], heads[0], heads[1], (int64_t)n_tok, d, d_rot, pos, inv_freq,
                            eps, norm, halves, inverse, st);
}

}  // namespace csa2
