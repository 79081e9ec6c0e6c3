// ckpt_backward.cu -- backward of a step's attention at the values an 8-bit
// checkpoint stands for, on the CUDA cores (fp32 contexts; fp32 arithmetic).
//
// Row i of a head sees the n cache slots and the chunk tokens t <= i. With
//   s_ij = q_i . k_j / sqrt(d),  p_ij = exp(s_ij) / sum_j exp(s_ij),
//   dp_ij = dO_i . v_j,          D_i = sum_j p_ij dp_ij,
//   ds_ij = p_ij (dp_ij - D_i):
//   dq_i = sum_j ds_ij k_j / sqrt(d), dk_j = sum_i ds_ij q_i / sqrt(d),
//   dv_j = sum_i p_ij dO_i,
// sums over i running over every query head of the key's KV head. The softmax
// statistics are recomputed: the restored keys are not the ones the forward
// saw, so its log-sum-exp would not normalise these weights.
#include <math.h>

#include "kernels.h"
#include "operators.h"
#include "vec.cuh"

namespace h2o {
namespace {

constexpr int kWarps = 8, kStride = kWarps * 4;  // keys or rows of a CTA at a time
// dq: query rows per CTA, and dk, dv: keys per CTA, in registers: two where that still
// gives every SM two CTAs, one otherwise (64 rows, 320 keys, 4 / 2 heads: dq 9.6 us with
// two and 8.0 with one, dk and dv 6.3 and 8.1). A lane group then has two or four keys
// (rows) in flight (one at a time, and so: 15.4 and 14.2 us a pass at 64 rows, 256
// slots, 4 / 2 heads, d = 64; 2748 and 2120 at 256 rows, 2048 slots, 32 / 8 heads, d = 128).
// Bound by latencies, of loads from L2 and of the three exchanges that close a dot
// product: in large steps the registers leave two warps to a scheduler, which issue in 46
// (dq) and 40 % (dk, dv) of the cycles, and the fp32 pipe is busy in 33 and 24 % (64
// rows, 1024 slots, 32 / 8 heads, d = 128: 160 and 192 us, where the eight products of d
// per pair would take 59 at the pipe's full rate).

__device__ __forceinline__ float sum8(float x) {  // over the eight lanes of a key or row
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 4);
}
__device__ __forceinline__ float sum_subs(float x) {  // over a warp's four lane groups
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
__device__ __forceinline__ float4 sum_subs(float4 a) {
    return make_float4(sum_subs(a.x), sum_subs(a.y), sum_subs(a.z), sum_subs(a.w));
}

// dq of kRows rows of one KV group (row = head-in-group * T + i), and their
// statistics. One pass over the keys with a running maximum, keeping
// A = sum e dp k, Z = sum e k, sum e dp and sum e (e = exp(s - max)):
// dq = (A - D Z) / (sum e sqrt(d)). Eight lanes share a key.
template <int D, int kRows>
__global__ void __launch_bounds__(kWarps * 32, kRows * D <= 128 ? 2 : 1)
ckpt_dq_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                    const float* __restrict__ K, const float* __restrict__ V, const float* __restrict__ dout,
                    float* __restrict__ dq, float4* __restrict__ stats, int G, int T, int n, int pitch,
                    int blocks_per_group, float scale_log2, float scale) {
    griddep_wait();  // the restored values are there
    griddep_launch_dependents();
    constexpr int Q4 = D / 32;
    constexpr int kBatch = kRows * D > 64 ? 2 : 4;
    __shared__ float4 part[2][kWarps][kRows][D / 4];
    __shared__ float part_s[kWarps][kRows][3];  // maximum, sum e, sum e dp
    const int R = G * T;
    const size_t bg = blockIdx.x / blocks_per_group;
    const int r0 = (blockIdx.x % blocks_per_group) * kRows;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane >> 3, l8 = lane & 7;
    const size_t row0 = bg * R + r0;
    float4 qr[kRows][Q4], dr[kRows][Q4], A[kRows][Q4], Z[kRows][Q4];
    float m[kRows], l[kRows], w[kRows];
    int tok[kRows], last = 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int rr = min(r0 + r, R - 1);
        tok[r] = rr % T;
        last = max(last, tok[r]);
        m[r] = -INFINITY;
        l[r] = w[r] = 0.f;
#pragma unroll
        for (int c = 0; c < Q4; ++c) {
            qr[r][c] = load4(q + (bg * R + rr) * D + 32 * c + 4 * l8);
            dr[r][c] = load4(dout + (bg * R + rr) * D + 32 * c + 4 * l8);
            A[r][c] = Z[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    const int total = n + last + 1;
    for (int u0 = warp * 4; u0 < total; u0 += kStride * kBatch) {
        float4 kk[kBatch][Q4], vv[kBatch][Q4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int u = min(u0 + kStride * b + sub, total - 1);
            const size_t at = u < n ? (bg * pitch + u) * D : (bg * T + (u - n)) * D;
            const float *kp = (u < n ? K : k) + at, *vp = (u < n ? V : v) + at;
#pragma unroll
            for (int c = 0; c < Q4; ++c) kk[b][c] = load4(kp + 32 * c + 4 * l8);
#pragma unroll
            for (int c = 0; c < Q4; ++c) vv[b][c] = load4(vp + 32 * c + 4 * l8);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float s[kBatch], dp[kBatch];
            bool see[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                s[b] = dp[b] = 0.f;
#pragma unroll
                for (int c = 0; c < Q4; ++c) {
                    s[b] = dot4(qr[r][c], kk[b][c], s[b]);
                    dp[b] = dot4(dr[r][c], vv[b][c], dp[b]);
                }
                const int u = u0 + kStride * b + sub;
                see[b] = u < total && u - n <= tok[r];
                s[b] = sum8(s[b]);
                s[b] = see[b] ? s[b] * scale_log2 : -INFINITY;
                dp[b] = sum8(dp[b]);
            }
            float mn = m[r];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) mn = fmaxf(mn, s[b]);
            const float ms = mn == -INFINITY ? 0.f : mn, a = exp2f(m[r] - ms);
            m[r] = mn;
            l[r] *= a;
            w[r] *= a;
#pragma unroll
            for (int c = 0; c < Q4; ++c) {
                A[r][c] = scale4(A[r][c], a);
                Z[r][c] = scale4(Z[r][c], a);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (see[b]) {
                    const float e = exp2f(s[b] - ms), ed = e * dp[b];
                    l[r] += e;
                    w[r] += ed;
#pragma unroll
                    for (int c = 0; c < Q4; ++c) {
                        A[r][c] = fma4(ed, kk[b][c], A[r][c]);
                        Z[r][c] = fma4(e, kk[b][c], Z[r][c]);
                    }
                }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float M = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 8));
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
        const float f = m[r] == -INFINITY ? 0.f : exp2f(m[r] - M);
#pragma unroll
        for (int c = 0; c < Q4; ++c) {
            const float4 a = sum_subs(scale4(A[r][c], f)), z = sum_subs(scale4(Z[r][c], f));
            if (sub == 0) {
                part[0][warp][r][8 * c + l8] = a;
                part[1][warp][r][8 * c + l8] = z;
            }
        }
        const float ls = sum_subs(l[r] * f), ws = sum_subs(w[r] * f);
        if (lane == 0) {
            part_s[warp][r][0] = M;
            part_s[warp][r][1] = ls;
            part_s[warp][r][2] = ws;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * (D / 4); e += kWarps * 32) {
        const int r = e / (D / 4), x = e % (D / 4);
        if (r0 + r >= R) continue;
        float M = -INFINITY, L = 0.f, W = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), z = a;
        for (int i = 0; i < kWarps; ++i) M = fmaxf(M, part_s[i][r][0]);
        for (int i = 0; i < kWarps; ++i) {
            const float f = part_s[i][r][0] == -INFINITY ? 0.f : exp2f(part_s[i][r][0] - M);
            L = fmaf(part_s[i][r][1], f, L);
            W = fmaf(part_s[i][r][2], f, W);
            a = fma4(f, part[0][i][r][x], a);
            z = fma4(f, part[1][i][r][x], z);
        }
        const float Dr = W / L, g = scale / L;
        // D z is rounded on its own, so that a row that sees one key gets exactly zero
        store4(dq + (row0 + r) * D + 4 * x,
               make_float4((a.x - __fmul_rn(Dr, z.x)) * g, (a.y - __fmul_rn(Dr, z.y)) * g,
                           (a.z - __fmul_rn(Dr, z.z)) * g, (a.w - __fmul_rn(Dr, z.w)) * g));
        if (x == 0) stats[row0 + r] = make_float4(M, 1.f / L, Dr, 0.f);
    }
}

// dk and dv of kKeys keys of one KV group: key u < C is cache slot u (zero
// gradients from n on), u >= C is chunk token u - C. Eight lanes share a query
// row, the CTA takes 32 rows at a time.
template <int D, int kKeys>
__global__ void __launch_bounds__(kWarps * 32, D == 64 ? 2 : 1)
ckpt_dkdv_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                      const float* __restrict__ K, const float* __restrict__ V, const float* __restrict__ dout,
                      const float4* __restrict__ stats, float* __restrict__ dK, float* __restrict__ dV,
                      float* __restrict__ dk, float* __restrict__ dv, int G, int C, int T, int n, int pitch,
                      int blocks_per_group, float scale_log2, float scale) {
    griddep_wait();  // the statistics are there
    constexpr int Q4 = D / 32;
    constexpr int kBatch = kKeys * D > 64 ? 2 : 4;
    __shared__ float4 part[2][kWarps][kKeys][D / 4];
    const int R = G * T;
    const size_t bg = blockIdx.x / blocks_per_group;
    const int u0 = (blockIdx.x % blocks_per_group) * kKeys;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane >> 3, l8 = lane & 7;
    float4 kr[kKeys][Q4], vr[kKeys][Q4], gk[kKeys][Q4], gv[kKeys][Q4];
    int from[kKeys];  // first row token that sees the key (T: none)
    int first = T;
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
        const int u = u0 + j;
        const bool cache = u < C;
        from[j] = cache ? (u < n ? 0 : T) : (u < C + T ? u - C : T);
        first = min(first, from[j]);
        const float* kp = cache ? K + (bg * pitch + u) * D : k + (bg * T + (u - C)) * D;
        const float* vp = cache ? V + (bg * pitch + u) * D : v + (bg * T + (u - C)) * D;
#pragma unroll
        for (int c = 0; c < Q4; ++c) {
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            gk[j][c] = gv[j][c] = zero;
            kr[j][c] = from[j] < T ? load4(kp + 32 * c + 4 * l8) : zero;
            vr[j][c] = from[j] < T ? load4(vp + 32 * c + 4 * l8) : zero;
        }
    }
    const int span = T - first;  // rows of each head from `first` on
    for (int x0 = warp * 4; x0 < G * span; x0 += kStride * kBatch) {
        float4 qq[kBatch][Q4], dd[kBatch][Q4], st[kBatch];
        int tok[kBatch];  // -1: no row
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int x = min(x0 + kStride * b + sub, G * span - 1), head = x / span, i = first + x - head * span;
            const size_t row = bg * R + (size_t)head * T + i;
            tok[b] = x0 + kStride * b + sub < G * span ? i : -1;
#pragma unroll
            for (int c = 0; c < Q4; ++c) qq[b][c] = load4(q + row * D + 32 * c + 4 * l8);
#pragma unroll
            for (int c = 0; c < Q4; ++c) dd[b][c] = load4(dout + row * D + 32 * c + 4 * l8);
            st[b] = stats[row];
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                float s = 0.f, dp = 0.f;
#pragma unroll
                for (int c = 0; c < Q4; ++c) {
                    s = dot4(qq[b][c], kr[j][c], s);
                    dp = dot4(dd[b][c], vr[j][c], dp);
                }
                s = sum8(s) * scale_log2;
                dp = sum8(dp);
                if (tok[b] >= from[j]) {
                    const float p = exp2f(s - st[b].x) * st[b].y, ds = p * (dp - st[b].z);
#pragma unroll
                    for (int c = 0; c < Q4; ++c) {
                        gv[j][c] = fma4(p, dd[b][c], gv[j][c]);
                        gk[j][c] = fma4(ds, qq[b][c], gk[j][c]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kKeys; ++j)
#pragma unroll
        for (int c = 0; c < Q4; ++c) {
            const float4 a = sum_subs(gk[j][c]), b = sum_subs(gv[j][c]);
            if (sub == 0) {
                part[0][warp][j][8 * c + l8] = a;
                part[1][warp][j][8 * c + l8] = b;
            }
        }
    __syncthreads();
    for (int e = threadIdx.x; e < kKeys * (D / 4); e += kWarps * 32) {
        const int j = e / (D / 4), x = e % (D / 4), u = u0 + j;
        if (u >= C + T) continue;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        for (int i = 0; i < kWarps; ++i) {
            a = add4(a, part[0][i][j][x]);
            b = add4(b, part[1][i][j][x]);
        }
        float* ka = u < C ? dK + (bg * C + u) * D : dk + (bg * T + (u - C)) * D;
        float* va = u < C ? dV + (bg * C + u) * D : dv + (bg * T + (u - C)) * D;
        store4(ka + 4 * x, scale4(a, scale));
        store4(va + 4 * x, b);
    }
}

template <int D, int kRows>
cudaError_t dq_launch(const CkptBwdArgs& a, float scale) {
    const int G = a.Hq / a.Hkv, per = (G * a.T + kRows - 1) / kRows;
    return launch_ex(true, ckpt_dq_simt_kernel<D, kRows>, dim3((unsigned)(a.B * a.Hkv * per)), dim3(kWarps * 32), 0,
                     a.stream, (const float*)a.q, (const float*)a.k, (const float*)a.v, (const float*)a.K,
                     (const float*)a.V, (const float*)a.dout, (float*)a.dq, reinterpret_cast<float4*>(a.stats), G, a.T,
                     a.n, a.pitch, per, kLog2e * scale, scale);
}

template <int D, int kKeys>
cudaError_t dkdv_launch(const CkptBwdArgs& a, float scale) {
    const int G = a.Hq / a.Hkv, per = (a.C + a.T + kKeys - 1) / kKeys;
    return launch_ex(true, ckpt_dkdv_simt_kernel<D, kKeys>, dim3((unsigned)(a.B * a.Hkv * per)), dim3(kWarps * 32), 0,
                     a.stream, (const float*)a.q, (const float*)a.k, (const float*)a.v, (const float*)a.K,
                     (const float*)a.V, (const float*)a.dout, reinterpret_cast<const float4*>(a.stats), (float*)a.dK,
                     (float*)a.dV, (float*)a.dk, (float*)a.dv, G, a.C, a.T, a.n, a.pitch, per, kLog2e * scale, scale);
}

template <int D>
cudaError_t backward_width(const CkptBwdArgs& a) {
    const float scale = 1.f / sqrtf((float)D);
    const long long ctas = 4ll * a.num_sms;
    const cudaError_t e = (long long)a.B * a.Hq * a.T >= ctas ? dq_launch<D, 2>(a, scale) : dq_launch<D, 1>(a, scale);
    if (e != cudaSuccess) return e;
    return (long long)a.B * a.Hkv * (a.C + a.T) >= ctas ? dkdv_launch<D, 2>(a, scale) : dkdv_launch<D, 1>(a, scale);
}

}  // namespace

cudaError_t launch_ckpt_backward_simt(const CkptBwdArgs& a) {
    return a.d == 64 ? backward_width<64>(a) : backward_width<128>(a);
}

}  // namespace h2o
