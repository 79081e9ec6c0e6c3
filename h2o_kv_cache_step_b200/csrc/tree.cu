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
// heads; 5.1 since four keys per lane group are in flight). Eight lanes share a key (d / 8 columns each), so a warp takes four keys and
// the CTA 32 at a time, straight from global memory into registers; every lane
// group keeps its own running maximum, sum and output, merged at the end.
// Where the rows are few (`slice` < n + T) the keys are divided among CTAs, `slice`
// each: a CTA leaves its unnormalised rows, maxima (NaN: the node is absent) and
// sums, and the last one of its rows to arrive merges them, in order. One token over
// 2048 slots is bound by latency: the loads, two exchanges through shared memory and
// the merge's way through L2 (8.2 us on the device, 10.5 with the loads of two keys in
// flight per lane group instead of four; 11.9 a pass on the tensor cores, 8.0 here).
struct TreeSplit {
    int slice;        // keys per CTA, a multiple of 32
    int parts;        // CTAs per kRows rows
    float* o;         // [rows / kRows][parts][kRows][D]
    float2* ml;       // [rows / kRows][parts][kRows]
    unsigned* count;  // [rows / kRows], zero
};

// A key's or a query's channels as eight lanes hold them, 16 bytes at a time: value i
// of lane l8 is channel 8 kVec (i / kVec) + kVec l8 + i % kVec.
template <typename E>
constexpr int kVec = 16 / (int)sizeof(E);

template <typename E, int N>
__device__ __forceinline__ void load_lane(const E* row, int l8, uint4 (&w)[N]) {
#pragma unroll
    for (int c = 0; c < N; ++c) w[c] = *reinterpret_cast<const uint4*>(row + 8 * kVec<E> * c + kVec<E> * l8);
}
template <int N>
__device__ __forceinline__ void expand(const uint4 (&w)[N], float (&f)[4 * N], float) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
        f[4 * c] = __uint_as_float(w[c].x);
        f[4 * c + 1] = __uint_as_float(w[c].y);
        f[4 * c + 2] = __uint_as_float(w[c].z);
        f[4 * c + 3] = __uint_as_float(w[c].w);
    }
}
template <int N>
__device__ __forceinline__ void expand(const uint4 (&w)[N], float (&f)[8 * N], __nv_bfloat16) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[8 * c + 2 * j] = __uint_as_float(u[j] << 16);
            f[8 * c + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
}
// The channel of the first of four values: values 4 j .. 4 j + 3 of lane l8 are
// kept at 4 (8 j + l8) of a row in shared memory (no two lanes in a bank) and of
// the parts; `four` counts those.
template <typename E>
__device__ __forceinline__ int channel(int four) {
    const int i = 4 * (four >> 3), l8 = four & 7;
    return 8 * kVec<E> * (i / kVec<E>) + kVec<E> * l8 + i % kVec<E>;
}

// Adds one; what the CTA wrote before its barrier is visible to whoever counts after.
__device__ __forceinline__ unsigned count_acq_rel(unsigned* count) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
    return old;
}

template <typename E, int D, int kRows>
__global__ void __launch_bounds__(kWarps * 32)
tree_simt_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v,
                 const int32_t* __restrict__ parent, const E* __restrict__ Kc, const E* __restrict__ Vc,
                 E* __restrict__ out, float* __restrict__ lse, int Hq, int Hkv, int C, int T, int n, int blocks_per_group,
                 float scale_log2, const TreeSplit split) {
    constexpr int kLane = D / 8;                         // values per lane and row
    constexpr int kLoads = kLane / kVec<E>;              // 16-byte loads of them
    constexpr int kBatch = sizeof(E) == 4 && kRows == 4 ? 2 : 4;  // keys in flight per lane group
    constexpr int kStride = kWarps * 4;                  // keys of the CTA at a time
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
    uint4 kw[kBatch][kLoads], vw[kBatch][kLoads];
    // the keys u0 + kStride b + sub; past the slice its last one, not used
    auto load = [&](int u0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int u = min(u0 + kStride * b + sub, hi - 1);
            const size_t at = u < n ? ((size_t)bg * C + u) * D : ((size_t)bg * T + (u - n)) * D;
            load_lane((u < n ? Kc : k) + at, l8, kw[b]);
            load_lane((u < n ? Vc : v) + at, l8, vw[b]);
        }
    };
    int u0 = lo + warp * 4;
    if (u0 < hi) load(u0);
    // the path of each row's node to the root: parents have smaller indices, so
    // the walk ends
    if (hi > n) {
        for (int i = threadIdx.x; i < T; i += kWarps * 32) up[i] = parent[(size_t)(bg / Hkv) * T + i];
        __syncthreads();
    }
    float qf[kRows][kLane], acc[kRows][kLane];
    float m[kRows], l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        uint4 w[kLoads];
        load_lane(q + (row0 + min(r, R - 1 - r0)) * D, l8, w);
        expand(w, qf[r], E());
#pragma unroll
        for (int i = 0; i < kLane; ++i) acc[r][i] = 0.f;
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
    __syncthreads();

    while (u0 < hi) {
        float s[kRows][kBatch];
        uint32_t vis[kBatch];  // rows that see the key
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int u = u0 + kStride * b + sub;
            float kf[kLane];
            expand(kw[b], kf, E());
            vis[b] = 0;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < kLane; ++i) x = fmaf(qf[r][i], kf[i], x);
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                const bool see = u < hi && (u < n || ((mask[r][(u - n) >> 5] >> ((u - n) & 31)) & 1u));
                vis[b] |= (uint32_t)see << r;
                s[r][b] = see ? x * scale_log2 : -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float mn = m[r];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) mn = fmaxf(mn, s[r][b]);
            const float ms = mn == -INFINITY ? 0.f : mn, a = exp2f(m[r] - ms);
            m[r] = mn;
            l[r] *= a;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                s[r][b] = exp2f(s[r][b] - ms);
                l[r] += s[r][b];
            }
#pragma unroll
            for (int i = 0; i < kLane; ++i) acc[r][i] *= a;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            float vf[kLane];
            expand(vw[b], vf, E());
            if (vis[b] == (1u << kRows) - 1) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int i = 0; i < kLane; ++i) acc[r][i] = fmaf(s[r][b], vf[i], acc[r][i]);
            } else {  // a key the row does not see touches nothing, whatever it holds
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (vis[b] >> r & 1u)
#pragma unroll
                        for (int i = 0; i < kLane; ++i) acc[r][i] = fmaf(s[r][b], vf[i], acc[r][i]);
            }
        }
        u0 += kStride * kBatch;
        if (u0 < hi) load(u0);
    }
    // merge the four lane groups of a warp: each ends with a quarter of the rows' values
    float x[kRows * kLane];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float M = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 8));
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
        const float w = m[r] == -INFINITY && l[r] == 0.f ? 0.f : exp2f(m[r] - M);
        float L = l[r] * w;
        L += __shfl_xor_sync(0xffffffffu, L, 8);
        L += __shfl_xor_sync(0xffffffffu, L, 16);
#pragma unroll
        for (int i = 0; i < kLane; ++i) x[r * kLane + i] = acc[r][i] * w;
        if (lane == 0) {
            part_m[warp][r] = M;
            part_l[warp][r] = L;
        }
    }
    constexpr int kHalf = kRows * kLane / 2, kQuarter = kHalf / 2;
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
        const float send = sub & 2 ? x[i] : x[kHalf + i], keep = sub & 2 ? x[kHalf + i] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
#pragma unroll
    for (int i = 0; i < kQuarter; ++i) {
        const float send = sub & 1 ? x[i] : x[kQuarter + i], keep = sub & 1 ? x[kQuarter + i] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
    }
    {
        const int r = kRows == 1 ? 0 : sub, i0 = kRows == 1 ? sub * kQuarter : 0;  // value 0 of the quarter
        static_assert(kRows == 1 || kRows == 4, "a quarter is a row or a part of the only one");
        float* dst = &part[warp][r][32 * (i0 / 4) + 4 * l8 + i0 % 4];
        if constexpr (kQuarter == 2) {
            *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
        } else {
#pragma unroll
            for (int j = 0; j < kQuarter / 4; ++j)
                *reinterpret_cast<float4*>(dst + 32 * j) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        }
    }
    __syncthreads();
    // merge the warps, four values per thread
    constexpr int kItems = kRows * (D / 4);
    const int item = threadIdx.x % kItems, g = threadIdx.x / kItems, r = item / (D / 4), c4 = item % (D / 4);
    if (g == 0 && r0 + r < R) {
        float M = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = part_m[w][r] == -INFINITY && part_l[w][r] == 0.f ? 0.f : exp2f(part_m[w][r] - M);
            L = fmaf(part_l[w][r], f, L);
            o = fma4(f, load4(&part[w][r][4 * c4]), o);
        }
        if (split.parts > 1) {
            const size_t at = ((size_t)unit * split.parts + piece) * kRows + r;
            store4(split.o + at * D + 4 * c4, o);
            if (c4 == 0) split.ml[at] = make_float2(present[r] ? M : __uint_as_float(0x7fffffffu), L);
        } else {
            store4(out + (row0 + r) * D + channel<E>(c4),
                   present[r] ? make_float4(o.x / L, o.y / L, o.z / L, o.w / L) : make_float4(0.f, 0.f, 0.f, 0.f));
            if (c4 == 0) lse[row0 + r] = present[r] ? (M + log2f(L)) * kLn2 : -INFINITY;
        }
    }
    if (split.parts == 1) return;
    __syncthreads();  // the CTA's part is written, and released with the count
    if (threadIdx.x == 0) {
        last = count_acq_rel(split.count + unit) == (unsigned)split.parts - 1;
        if (last) split.count[unit] = 0;
    }
    __syncthreads();
    if (!last) return;
    // kGroups threads share four columns of a row, every kGroups-th part each, and meet
    // in shared memory
    constexpr int kGroups = kItems * kWarps <= kWarps * 32 ? kWarps : kWarps * 32 / kItems;
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
    store4(out + (row0 + r) * D + channel<E>(c4), absent ? make_float4(0.f, 0.f, 0.f, 0.f) : scale4(o, 1.f / L));
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
