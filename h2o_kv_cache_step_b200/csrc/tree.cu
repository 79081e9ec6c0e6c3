// tree.cu -- attention of a tree of drafted tokens over the cache, on the CUDA
// cores (fp32 contexts, and small calls of bf16 ones; the arithmetic is fp32 for
// either element type).
//
// Row i of sequence b sees the n valid cache slots and the nodes on its path to
// the root, itself included:
//   O_i = sum_j p_ij v_j,  p_ij = exp(s_ij - LSE_i),  s_ij = q_i . k_j / sqrt(d),
//   LSE_i = log sum_j exp(s_ij).
// A node whose path does not end in a root (parent -1) is absent: O = 0,
// LSE = -inf.
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "operators.h"
#include "vec.cuh"

namespace h2o {
namespace {

constexpr int kWarps = 8;
constexpr int kTreeMinKeys = 96;  // keys that repay a CTA of their own

// One CTA per kRows query rows of one KV group (row = head-in-group * T + i), four
// where that still gives every SM a CTA (each key is then read once for four rows),
// one otherwise (latency: 6.2 us against 10.1 at 24 nodes, 201 slots, 4 / 2
// heads). Eight lanes share a key (d / 8 columns each), so a warp takes four keys and
// the CTA 32 at a time, straight from global memory into registers; every lane
// group keeps its own running maximum, sum and output, merged at the end.
// Where the rows are few (`slice` < n + T) the keys are divided among CTAs, `slice`
// each: a CTA leaves its unnormalised rows, maxima (NaN: the node is absent) and
// sums, and the last one of its rows to arrive merges them, in order. One token over
// 2048 slots is bound by latency: the loads, two exchanges through shared memory and
// the merge's way through L2 (10.9 us on the device, 12.7 on the tensor cores).
struct TreeSplit {
    int slice;        // keys per CTA, a multiple of 32
    int parts;        // CTAs per kRows rows
    float* o;         // [rows / kRows][parts][kRows][D]
    float2* ml;       // [rows / kRows][parts][kRows]
    unsigned* count;  // [rows / kRows], zero
};

template <typename E, int D, int kRows>
__global__ void __launch_bounds__(kWarps * 32)
tree_simt_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v,
                 const int32_t* __restrict__ parent, const E* __restrict__ Kc, const E* __restrict__ Vc,
                 E* __restrict__ out, float* __restrict__ lse, int Hq, int Hkv, int C, int T, int n, int blocks_per_group,
                 float scale_log2, const TreeSplit split) {
    constexpr int Q4 = D / 32;  // float4 per lane and row
    __shared__ int up[kTreeMaxT];
    __shared__ int last;
    __shared__ uint32_t mask[kRows][kTreeMaskWords];
    __shared__ int present[kRows];
    __shared__ __align__(16) float part[kWarps][kRows][D];  // stored to as float4
    __shared__ float part_m[kWarps][kRows], part_l[kWarps][kRows];
    const int G = Hq / Hkv, R = G * T;
    const int unit = blockIdx.x / split.parts, piece = blockIdx.x % split.parts;
    const int bg = unit / blocks_per_group, r0 = (unit % blocks_per_group) * kRows;
    const int total = n + T, lo = piece * split.slice, hi = min(total, lo + split.slice);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane >> 3, l8 = lane & 7;
    const size_t row0 = (size_t)bg * R + r0;  // [B,Hq,T] rows of a group are contiguous

    griddep_wait();  // the work before is complete; what follows may set up
    griddep_launch_dependents();
    // the path of each row's node to the root: parents have smaller indices, so
    // the walk ends
    if (hi > n) {
        for (int i = threadIdx.x; i < T; i += kWarps * 32) up[i] = parent[(size_t)(bg / Hkv) * T + i];
        __syncthreads();
    }
    if (threadIdx.x < kRows) {
        const int r = threadIdx.x;
        for (int w = 0; w < kTreeMaskWords; ++w) mask[r][w] = 0;
        int at = hi <= n ? -1 : r0 + r < R ? (r0 + r) % T : -2;
        while (at >= 0) {
            mask[r][at >> 5] |= 1u << (at & 31);
            const int u = up[at];
            at = u == -1 ? -1 : (u >= 0 && u < at) ? u : -2;
        }
        present[r] = at == -1;
    }
    float4 qr[kRows][Q4], acc[kRows][Q4];
    float m[kRows], l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        const size_t row = row0 + min(r, R - 1 - r0);
#pragma unroll
        for (int c = 0; c < Q4; ++c) {
            qr[r][c] = load4(q + row * D + 32 * c + 4 * l8);
            acc[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __syncthreads();

#pragma unroll 2
    for (int u0 = lo + warp * 4; u0 < hi; u0 += kWarps * 4) {
        const int u = u0 + sub;
        const bool in = u < hi;
        const int uu = in ? u : hi - 1;
        const E* kp = uu < n ? Kc + ((size_t)bg * C + uu) * D : k + ((size_t)bg * T + (uu - n)) * D;
        const E* vp = uu < n ? Vc + ((size_t)bg * C + uu) * D : v + ((size_t)bg * T + (uu - n)) * D;
        float4 kk[Q4], vv[Q4];
#pragma unroll
        for (int c = 0; c < Q4; ++c) kk[c] = load4(kp + 32 * c + 4 * l8);
#pragma unroll
        for (int c = 0; c < Q4; ++c) vv[c] = load4(vp + 32 * c + 4 * l8);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < Q4; ++c)
                s = fmaf(qr[r][c].x, kk[c].x, fmaf(qr[r][c].y, kk[c].y, fmaf(qr[r][c].z, kk[c].z, fmaf(qr[r][c].w, kk[c].w, s))));
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            // a key the row does not see touches nothing, whatever it holds
            const bool vis = in && (u < n || ((mask[r][(u - n) >> 5] >> ((u - n) & 31)) & 1u));
            s *= scale_log2;
            const float mn = fmaxf(m[r], s);
            if (vis && !(s == mn && mn == -INFINITY)) {
                const float a = exp2f(m[r] - mn), p = exp2f(s - mn);
                l[r] = fmaf(l[r], a, p);
                m[r] = mn;
#pragma unroll
                for (int c = 0; c < Q4; ++c) {
                    acc[r][c].x = fmaf(p, vv[c].x, acc[r][c].x * a);
                    acc[r][c].y = fmaf(p, vv[c].y, acc[r][c].y * a);
                    acc[r][c].z = fmaf(p, vv[c].z, acc[r][c].z * a);
                    acc[r][c].w = fmaf(p, vv[c].w, acc[r][c].w * a);
                }
            }
        }
    }
    // merge the four lane groups of a warp, then the warps
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float M = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 8));
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
        const float w = m[r] == -INFINITY && l[r] == 0.f ? 0.f : exp2f(m[r] - M);
        float L = l[r] * w;
        L += __shfl_xor_sync(0xffffffffu, L, 8);
        L += __shfl_xor_sync(0xffffffffu, L, 16);
#pragma unroll
        for (int c = 0; c < Q4; ++c) {
            float x[4] = {acc[r][c].x * w, acc[r][c].y * w, acc[r][c].z * w, acc[r][c].w * w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] += __shfl_xor_sync(0xffffffffu, x[e], 8);
                x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
            }
            if (sub == 0) *reinterpret_cast<float4*>(&part[warp][r][32 * c + 4 * l8]) = make_float4(x[0], x[1], x[2], x[3]);
        }
        if (lane == 0) {
            part_m[warp][r] = M;
            part_l[warp][r] = L;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * D; e += kWarps * 32) {
        const int r = e / D, x = e % D;
        if (r0 + r >= R) continue;
        float M = -INFINITY, L = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_m[w][r]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = part_m[w][r] == -INFINITY && part_l[w][r] == 0.f ? 0.f : exp2f(part_m[w][r] - M);
            L = fmaf(part_l[w][r], f, L);
            o = fmaf(part[w][r][x], f, o);
        }
        if (split.parts > 1) {
            const size_t at = ((size_t)unit * split.parts + piece) * kRows + r;
            split.o[at * D + x] = o;
            if (x == 0) split.ml[at] = make_float2(present[r] ? M : __uint_as_float(0x7fffffffu), L);
        } else {
            out[(row0 + r) * D + x] = from_f32<E>(present[r] ? o / L : 0.f);
            if (x == 0) lse[row0 + r] = present[r] ? (M + log2f(L)) * kLn2 : -INFINITY;
        }
    }
    if (split.parts == 1) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomicAdd(split.count + unit, 1u) == (unsigned)split.parts - 1;
        if (last) split.count[unit] = 0;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // kGroups threads share four columns of a row, every kGroups-th part each, and meet
    // in shared memory
    constexpr int kItems = kRows * (D / 4), kGroups = kItems * kWarps <= kWarps * 32 ? kWarps : kWarps * 32 / kItems;
    const int item = threadIdx.x % kItems, g = threadIdx.x / kItems, r = item / (D / 4), c4 = item % (D / 4);
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool absent = false;
    if (g < kGroups && r0 + r < R) {
#pragma unroll 8
        for (int p = g; p < split.parts; p += kGroups) {
            const size_t at = ((size_t)unit * split.parts + p) * kRows + r;
            const float2 ml = split.ml[at];
            const float4 x = load4(split.o + at * D + 4 * c4);
            absent |= ml.x != ml.x;
            const float Mn = fmaxf(M, ml.x), ms = Mn == -INFINITY ? 0.f : Mn;
            const float a = exp2f(M - ms), w = exp2f(ml.x - ms);
            M = Mn;
            L = fmaf(L, a, ml.y * w);
            o = fma4(w, x, scale4(o, a));
        }
    }
    if (g < kGroups) {
        store4(&part[g][r][4 * c4], o);
        if (c4 == 0) {
            part_m[g][r] = absent ? __uint_as_float(0x7fffffffu) : M;
            part_l[g][r] = L;
        }
    }
    __syncthreads();
    if (g != 0 || r0 + r >= R) return;
    M = -INFINITY;
    absent = false;
#pragma unroll
    for (int p = 0; p < kGroups; ++p) {
        absent |= part_m[p][r] != part_m[p][r];
        M = fmaxf(M, part_m[p][r]);
    }
    const float ms = M == -INFINITY ? 0.f : M;
    L = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kGroups; ++p) {
        const float w = exp2f(part_m[p][r] - ms);
        L = fmaf(part_l[p][r], w, L);
        o = fma4(w, load4(&part[p][r][4 * c4]), o);
    }
    store4(out + (row0 + r) * D + 4 * c4, absent ? make_float4(0.f, 0.f, 0.f, 0.f) : scale4(o, 1.f / L));
    if (c4 == 0) lse[row0 + r] = absent ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <typename E, int D, int kRows>
cudaError_t tree_simt_rows(const TreeArgs& a) {
    const int R = a.Hq / a.Hkv * a.T, per = (R + kRows - 1) / kRows, units = a.B * a.Hkv * per, total = a.n + a.T;
    TreeSplit s{};
    // as many CTAs as SMs, if each gets kTreeMinKeys keys
    s.parts = std::max(1, std::min(a.num_sms / units, total / kTreeMinKeys));
    s.slice = ((total + s.parts - 1) / s.parts + 31) / 32 * 32;
    s.parts = (total + s.slice - 1) / s.slice;
    s.o = a.part;
    s.ml = reinterpret_cast<float2*>(a.part + (size_t)a.num_sms * kRows * D);
    s.count = a.count;
    return launch_ex(true, tree_simt_kernel<E, D, kRows>, dim3((unsigned)(units * s.parts)), dim3(kWarps * 32), 0, a.stream,
                     (const E*)a.q, (const E*)a.k, (const E*)a.v, a.parent, (const E*)a.Kc, (const E*)a.Vc, (E*)a.out, a.lse,
                     a.Hq, a.Hkv, a.C, a.T, a.n, per, kLog2e / sqrtf((float)D), s);
}

// Four rows a CTA while that gives every SM a CTA, by rows or by slices of the keys.
template <typename E, int D>
cudaError_t tree_simt_typed(const TreeArgs& a) {
    const long long fours = (long long)a.B * a.Hkv * ((a.Hq / a.Hkv * a.T + 3) / 4);
    const long long ctas = fours * std::max(1, (a.n + a.T) / kTreeMinKeys);
    return ctas >= a.num_sms ? tree_simt_rows<E, D, 4>(a) : tree_simt_rows<E, D, 1>(a);
}

}  // namespace

size_t tree_simt_part_floats(int num_sms, int d) { return (size_t)num_sms * 4 * (d + 2); }

cudaError_t launch_tree_simt(const TreeArgs& a) {
    if (a.dtype == 1) return a.d == 64 ? tree_simt_typed<float, 64>(a) : tree_simt_typed<float, 128>(a);
    return a.d == 64 ? tree_simt_typed<__nv_bfloat16, 64>(a) : tree_simt_typed<__nv_bfloat16, 128>(a);
}

}  // namespace h2o
