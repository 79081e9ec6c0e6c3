// ckpt_backward_tc.cu -- tensor-core (tcgen05 + TMEM + TMA) kernels of the
// backward of a step's attention at the values an 8-bit checkpoint stands for
// (bf16; the formulas are ckpt_backward.cu's).
//
// ckpt_dq_tc_kernel    one CTA per (128-row query tile, head), two passes over
//     the tile's key blocks. The first computes S = Q K^T and dP = dO V^T and
//     keeps each row's running maximum m, sum l = sum e and w = sum e dp
//     (e = 2^(s - m)); then LSE = m + log2 l and D = w / l, in fp32. The second
//     recomputes both products, writes dS = P (dP - D) as bf16 over S in TMEM
//     and accumulates dQ += dS K with dS as the A operand from TMEM.
// ckpt_dkdv_tc_kernel  one CTA per (KV head, 128-key block), one key per TMEM
//     lane: per 128-row query tile of the KV head, S^T = K Q^T and
//     dP^T = V dO^T; P^T and dS^T go back over them as bf16 and are the A
//     operands of dV += P^T dO and dK += dS^T Q.
//
// Bound by the tensor core: 5 products of 2 d per visible (row, key) in the
// first kernel, 4 in the second. An operand pair from shared memory needs
// 128 bytes a clock at the MMA's full rate, all there is, so P and dS stay in
// TMEM (64 bytes a clock), and they never cross shared memory. Ten warps: a TMA
// loader, an MMA issuer and two warpgroups that share every tile, one half of
// its columns each. The issue order keeps the tensor core on a product that
// does not wait for the exponentials in progress: dV(t), S(t+1) while dS(t) is
// computed, dK(t), dP(t+1) while P(t+1) is.
//
// Rows past the end of a head or cache arrive as zeros (3-D tensor maps), so
// nothing of another head enters a tile. P and dS are rounded to bf16, the MMA's
// operand type; statistics and gradients accumulate in fp32.
#include <cuda.h>
#include <math.h>

#include "operators.h"
#include "tc.h"
#include "tc_ptx.cuh"

namespace h2o {
namespace {

using tc::desc_kmajor_sw128;
using tc::desc_mnmajor_sw128;
using tc::ex2;
using tc::fence_after_sync;
using tc::fence_before_sync;

constexpr int kThreads = 320;   // loader, MMA issuer, two warpgroups
constexpr int kConsumers = 256;
constexpr int kMaxCluster = 4;

struct CkptTcParams {
    int B, Hq, Hkv, T, C, n;
    int n_mblk;  // 128-row query tiles per head
    int nbc;     // cache key blocks = ceil(n / 128)
    int nbC;     // 128-slot blocks of the whole cache
    float scale_log2, scale;
    float* nL2;  // [B*Hq][128 * n_mblk]: -(log2-domain LSE) per row, -inf in padding rows
    float* D;    // [B*Hq][128 * n_mblk], 0 in padding rows
    __nv_bfloat16* dq;
    __nv_bfloat16* dK;
    __nv_bfloat16* dV;
    __nv_bfloat16* dk;
    __nv_bfloat16* dv;
    WaitBound wb;
};

// 64 accumulator columns of this thread's lane, times mul, as 128 bytes of bf16.
__device__ __forceinline__ void store_acc64(uint32_t taddr, __nv_bfloat16* dst, float mul, bool in) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t o[32];
        tc::tmem_ld32(taddr + 32 * c, o);
        tc::tmem_ld_wait();
        tc::reg_fence(o);
        if (in) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
                *reinterpret_cast<uint4*>(dst + 32 * c + e) =
                    make_uint4(tc::pack_bf16(__uint_as_float(o[e]) * mul, __uint_as_float(o[e + 1]) * mul),
                               tc::pack_bf16(__uint_as_float(o[e + 2]) * mul, __uint_as_float(o[e + 3]) * mul),
                               tc::pack_bf16(__uint_as_float(o[e + 4]) * mul, __uint_as_float(o[e + 5]) * mul),
                               tc::pack_bf16(__uint_as_float(o[e + 6]) * mul, __uint_as_float(o[e + 7]) * mul));
        }
    }
}

// ============================================================================
// dQ and the rows' statistics
// ============================================================================
template <int D>
struct DqCfg {
    static constexpr int HALF = 128 * 128;  // 128 rows x 64 bf16
    static constexpr int TILE = 128 * D * 2;
    static constexpr int RING = 5;          // K / V slots, loaded K0, V0, K1, V1, ...
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_DO = TILE;
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_ST = OFF_RING + RING * TILE;  // [3][128] floats
    static constexpr int OFF_BAR = OFF_ST + 3 * 128 * 4;
    static constexpr int NBAR = 24;
    static constexpr int SMEM_RAW = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int SMEM = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;  // one CTA (512 TMEM columns) per SM
    static constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(128, 128, false);
    static constexpr uint32_t IDESC_G = tc::idesc_bf16_f32(128, D, true);
};
static_assert(DqCfg<128>::SMEM_RAW <= 232448, "dQ kernel shared memory exceeds the per-CTA limit");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
ckpt_dq_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                  const __grid_constant__ CUtensorMap map_kc, const __grid_constant__ CUtensorMap map_vc,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const CkptTcParams p) {
    using Cfg = DqCfg<D>;
    constexpr int RING = Cfg::RING;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* q_full = bars;                  // Q and dO tiles
    uint64_t* ring_full = bars + 1;           // [RING]
    uint64_t* ring_empty = ring_full + RING;  // [RING]
    uint64_t* sd_full = ring_empty + RING;    // [2] pass 1: S and dP of a buffer
    uint64_t* sd_free = sd_full + 2;          // [2] pass 1, 8 arrivals: in registers
    uint64_t* s_full = sd_free + 2;           // [2] pass 2: S of a buffer
    uint64_t* dp_full = s_full + 2;           // pass 2: dP
    uint64_t* ds_full = dp_full + 1;          // pass 2, 8 arrivals: dS over S, dP in registers
    uint64_t* drain = ds_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per_mblk = p.B * p.Hq;
    const int mblk = p.n_mblk - 1 - (int)(blockIdx.x / per_mblk);  // most key blocks first
    const int bh = blockIdx.x % per_mblk;
    const int bg = bh / (p.Hq / p.Hkv);
    const int m0 = mblk * 128;
    const int nb = p.nbc + mblk + 1;  // key blocks per pass: cache, then chunk 0..mblk

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < RING; ++s) {
            mbar_init(ring_full + s, 1);
            mbar_init(ring_empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sd_full + b, 1);
            mbar_init(sd_free + b, 8);
            mbar_init(s_full + b, 1);
        }
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;  // S of the two buffers at 0 and 128, dP at 256 (and 384 in pass 1), dQ at 384
    const uint32_t sbase = smem_u32(smem);

    if (warp == 0) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, 2 * Cfg::TILE);
            for (int hh = 0; hh < D / 64; ++hh) {
                tc::tma_load_3d(smem + Cfg::OFF_Q + hh * Cfg::HALF, &map_q, 64 * hh, m0, bh, q_full);
                tc::tma_load_3d(smem + Cfg::OFF_DO + hh * Cfg::HALF, &map_do, 64 * hh, m0, bh, q_full);
            }
            int L = 0;
            bool ok = true;
            for (int it = 0; ok && it < 2 * nb; ++it) {
                const int j = it % nb;
                const bool cache = j < p.nbc;
                const int row = 128 * (cache ? j : j - p.nbc);
                for (int kv = 0; kv < 2; ++kv, ++L) {
                    const int slot = L % RING;
                    if (!(ok = wait_bar(ring_empty + slot, ((L / RING) & 1) ^ 1, p.wb, kDevTimeoutSlotWait, abort_flag)))
                        break;
                    const CUtensorMap* map = kv ? (cache ? &map_vc : &map_v) : (cache ? &map_kc : &map_k);
                    mbar_arrive_expect_tx(ring_full + slot, Cfg::TILE);
                    for (int hh = 0; hh < D / 64; ++hh)
                        tc::tma_load_3d(smem + Cfg::OFF_RING + slot * Cfg::TILE + hh * Cfg::HALF, map, 64 * hh, row, bg,
                                        ring_full + slot);
                }
            }
            // every load issued here has landed before the CTA may exit
            wait_bar(q_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag);
            for (int s = 0; s < RING; ++s) {
                const int uses = L / RING + (s < L % RING ? 1 : 0);
                if (uses) wait_bar(ring_full + s, (uses - 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint64_t dQd = desc_kmajor_sw128(sbase + Cfg::OFF_Q);
        const uint64_t dOd = desc_kmajor_sw128(sbase + Cfg::OFF_DO);
        const uint64_t dRingK = desc_kmajor_sw128(sbase + Cfg::OFF_RING);
        const uint64_t dRingN = desc_mnmajor_sw128(sbase + Cfg::OFF_RING, Cfg::HALF);
        auto wait_ring = [&](int l) {
            return warp_wait(ring_full + l % RING, (l / RING) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
        };
        // D = A B^T over d, both from shared memory, K-major
        auto issue_ss = [&](uint32_t acc, uint64_t a, int slot) {
            const uint64_t b = dRingK + (uint64_t)((slot * Cfg::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * Cfg::HALF + (kk & 3) * 32) >> 4;
                tc::mma_bf16_ss_warp(acc, a + off, b + off, Cfg::IDESC_S, kk > 0);
            }
        };
        bool ok = warp_wait(q_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag);
        // pass 1: S and dP of block t into buffer t & 1
        for (int t = 0; ok && t < nb; ++t) {
            const int b = t & 1, ks = 2 * t, vs = 2 * t + 1;
            ok = (t < 2 || warp_wait(sd_free + b, ((t >> 1) - 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag)) && wait_ring(ks);
            if (!ok) break;
            fence_after_sync();
            issue_ss(tmem + 128 * b, dQd, ks % RING);
            tc::mma_commit_warp(ring_empty + ks % RING);
            if (!(ok = wait_ring(vs))) break;
            issue_ss(tmem + 256 + 128 * b, dOd, vs % RING);
            tc::mma_commit_warp(sd_full + b);
            tc::mma_commit_warp(ring_empty + vs % RING);
        }
        // pass 2: S(t) and then dS(t) in buffer t & 1, one dP, dQ
        for (int b = 0; b < 2 && b < nb; ++b)  // both buffers read
            ok = ok && warp_wait(sd_free + b, ((nb - 1 - b) >> 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag);
        fence_after_sync();
        const int L0 = 2 * nb;
        auto issue_s = [&](int t) {  // needs buffer t & 1 free, or read by products issued before
            const int l = L0 + 2 * t;
            if (!wait_ring(l)) return false;
            issue_ss(tmem + 128 * (t & 1), dQd, l % RING);
            tc::mma_commit_warp(s_full + (t & 1));
            return true;
        };
        auto issue_dp = [&](int t) {
            const int l = L0 + 2 * t + 1;
            if (!wait_ring(l)) return false;
            issue_ss(tmem + 256, dOd, l % RING);
            tc::mma_commit_warp(dp_full);
            tc::mma_commit_warp(ring_empty + l % RING);
            return true;
        };
        ok = ok && issue_s(0) && issue_dp(0) && (nb < 2 || issue_s(1));
        for (int t = 0; ok && t < nb; ++t) {
            if (!(ok = warp_wait(ds_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            if (t + 1 < nb && !(ok = issue_dp(t + 1))) break;
            const int ks = (L0 + 2 * t) % RING;
            const uint64_t b = dRingN + (uint64_t)((ks * Cfg::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 keys at a time; the keys' halves at columns 0 and 64
                tc::mma_bf16_ts_warp(tmem + 384, tmem + 128 * (t & 1) + 64 * (kk >> 2) + 8 * (kk & 3),
                                     b + (uint64_t)((kk * 16 * 128) >> 4), Cfg::IDESC_G, (t > 0 || kk > 0) ? 1u : 0u);
            tc::mma_commit_warp(ring_empty + ks);
            if (t + 2 < nb) ok = issue_s(t + 2);
        }
        // all MMAs issued here complete before TMEM can be released
        tc::mma_commit_warp(drain);
        __syncwarp();
        warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
    } else {
        // ---------------------------------------------------------- row warpgroups
        const int wg = (warp - 2) >> 2;  // columns 64 wg .. 64 wg + 63
        const int quad = warp & 3;
        const int r = quad * 32 + lane;  // row inside the tile = TMEM lane
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16) + 64 * wg;
        float* st = reinterpret_cast<float*>(smem + Cfg::OFF_ST);
        // visible columns of this row's half in block j: e < limit
        auto limit_of = [&](int j) { return (j < p.nbc ? p.n - 128 * j : m0 + r - 128 * (j - p.nbc) + 1) - 64 * wg; };
        float m = -INFINITY, l = 0.f, w = 0.f;
        bool ok = true;
        for (int t = 0; t < nb; ++t) {
            const int b = t & 1;
            if (!(ok = warp_wait(sd_full + b, (t >> 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t s[2][32], dp[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tl + 128 * b + 32 * c, s[c]);
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tl + 256 + 128 * b + 32 * c, dp[c]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tc::reg_fence(s[c]);
                tc::reg_fence(dp[c]);
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(sd_free + b);
            const int limit = limit_of(t);
            if (limit < 64) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e >= limit) s[e >> 5][e & 31] = __float_as_uint(-INFINITY);
            }
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                mx0 = tc::max3(mx0, __uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1]));
                mx1 = tc::max3(mx1, __uint_as_float(s[e >> 5][(e & 31) + 2]), __uint_as_float(s[e >> 5][(e & 31) + 3]));
            }
            const float mn = fmaxf(m, fmaxf(mx0, mx1) * p.scale_log2);
            const float ms = mn == -INFINITY ? 0.f : mn;  // no visible key in this half yet
            const float a = ex2(m - ms);
            m = mn;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-ms, -ms);
            float2 l2 = make_float2(0.f, 0.f), w2 = l2;
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
                const float2 x = tc::ffma2(
                    make_float2(__uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1])), sc2, nm2);
                const float2 pe = make_float2(ex2(x.x), ex2(x.y));
                l2 = tc::fadd2(l2, pe);
                w2 = tc::ffma2(pe, make_float2(__uint_as_float(dp[e >> 5][e & 31]), __uint_as_float(dp[e >> 5][(e & 31) + 1])), w2);
            }
            l = fmaf(l, a, l2.x + l2.y);
            w = fmaf(w, a, w2.x + w2.y);
        }
        // the two halves of a row meet: the second hands over its m, l and w, the
        // first gives back -LSE and D
        const bool row_ok = m0 + r < p.T;
        float nL2, Dr;
        if (wg == 1) {
            st[r] = m;
            st[128 + r] = l;
            st[256 + r] = w;
            tc::named_sync(1, kConsumers);
            tc::named_sync(2, kConsumers);
            nL2 = st[r];
            Dr = st[128 + r];
        } else {
            tc::named_sync(1, kConsumers);
            const float M = fmaxf(m, st[r]);
            const float a0 = ex2(m - M), a1 = ex2(st[r] - M);
            const float L = l * a0 + st[128 + r] * a1;
            nL2 = -(M + log2f(L));
            Dr = (w * a0 + st[256 + r] * a1) / L;
            st[r] = nL2;
            st[128 + r] = Dr;
            tc::named_sync(2, kConsumers);
            const size_t at = ((size_t)bh * p.n_mblk + mblk) * 128 + r;
            p.nL2[at] = row_ok ? nL2 : -INFINITY;
            p.D[at] = row_ok ? Dr : 0.f;
        }
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nL2, nL2), nd2 = make_float2(-Dr, -Dr);
        for (int t = 0; ok && t < nb; ++t) {
            const uint32_t tS = tl + 128 * (t & 1);
            if (!(ok = warp_wait(s_full + (t & 1), (t >> 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t s[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tS + 32 * c, s[c]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::reg_fence(s[c]);
            const int limit = limit_of(t);
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
                const float2 x = tc::ffma2(
                    make_float2(__uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1])), sc2, nl2);
                s[e >> 5][e & 31] = __float_as_uint(ex2(x.x));
                s[e >> 5][(e & 31) + 1] = __float_as_uint(ex2(x.y));
            }
            if (limit < 64) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e >= limit) s[e >> 5][e & 31] = 0u;
            }
            if (!(ok = warp_wait(dp_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t dp[32];
                tc::tmem_ld32(tl + 256 + 32 * c, dp);
                tc::tmem_ld_wait();
                tc::reg_fence(dp);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 y = tc::fadd2(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), nd2);
                    pk[16 * c + (e >> 1)] = tc::pack_bf16(__uint_as_float(s[c][e]) * y.x, __uint_as_float(s[c][e + 1]) * y.y);
                }
            }
            tc::tmem_st32(tS, pk);
            tc::tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        if (ok && warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag)) {
            fence_after_sync();
            if (64 * wg < D)
                store_acc64(tl + 384, p.dq + ((size_t)bh * p.T + m0 + r) * D + 64 * wg, p.scale, row_ok);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ============================================================================
// dK, dV
// ============================================================================
template <int D>
struct DkvCfg {
    static constexpr int HALF = 128 * 128;
    static constexpr int TILE = 128 * D * 2;
    static constexpr int STAGES = 2;             // query tiles: Q, dO and their rows' statistics
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = TILE;
    static constexpr int OFF_T = 2 * TILE;       // [STAGES][Q, dO]
    static constexpr int OFF_ROW = OFF_T + STAGES * 2 * TILE;  // [STAGES][2][128] floats: -LSE and D
    static constexpr int OFF_BAR = OFF_ROW + STAGES * 2 * 128 * 4;
    static constexpr int NBAR = 16;
    static constexpr int SMEM_RAW = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int SMEM = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;
    static constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(128, 128, false);
    static constexpr uint32_t IDESC_G = tc::idesc_bf16_f32(128, D, true);
};
static_assert(DkvCfg<128>::SMEM_RAW <= 232448, "dK/dV kernel shared memory exceeds the per-CTA limit");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
ckpt_dkdv_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                    const __grid_constant__ CUtensorMap map_kc, const __grid_constant__ CUtensorMap map_vc,
                    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const CkptTcParams p) {
    using Cfg = DkvCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* kv_full = bars;
    uint64_t* t_full = bars + 1;   // [2] a query tile has landed
    uint64_t* t_empty = bars + 3;  // [2] its MMAs have completed
    uint64_t* s_full = bars + 5;   // S^T
    uint64_t* p_full = bars + 6;   // 8 arrivals: P^T over S^T
    uint64_t* dp_full = bars + 7;  // dP^T
    uint64_t* ds_full = bars + 8;  // 8 arrivals: dS^T over dP^T
    uint64_t* drain = bars + 9;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int G = p.Hq / p.Hkv;
    const int groups = p.B * p.Hkv;
    // blocks in decreasing work: cache blocks (all rows see them), chunk blocks,
    // blocks of empty slots (zeros)
    const int rank = tc::cluster_rank(), ranks = tc::cluster_size();  // the cluster's CTAs share a key block
    const int unit = blockIdx.x / ranks;
    const int kb = unit / groups, bg = unit % groups;
    if (kb >= p.nbc + p.n_mblk) {
        const int s0 = 128 * (kb - p.n_mblk);
        const size_t at = ((size_t)bg * p.C + s0) * D;
        const int vecs = min(128, p.C - s0) * D / 8;
        for (int e = rank * kThreads + threadIdx.x; e < vecs; e += ranks * kThreads) {
            reinterpret_cast<uint4*>(p.dK + at)[e] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(p.dV + at)[e] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const bool cache = kb < p.nbc;
    const int t0 = cache ? 0 : 128 * (kb - p.nbc);  // first chunk token of the block
    const int m_first = t0 / 128;                   // query tiles before it see none of a chunk block
    const int per_head = p.n_mblk - m_first;
    // query tiles of the KV head, heads one after the other; this CTA's are
    // first .. first + ntiles - 1
    const int first = G * per_head * rank / ranks, ntiles = G * per_head * (rank + 1) / ranks - first;

    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(t_full + s, 1);
            mbar_init(t_empty + s, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(p_full, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;  // S^T at 0, dP^T at 128, dV at 256, dK at 256 + D
    const uint32_t sbase = smem_u32(smem);

    if (warp == 0) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            const int krow = cache ? 128 * kb : t0;
            mbar_arrive_expect_tx(kv_full, 2 * Cfg::TILE);
            for (int hh = 0; hh < D / 64; ++hh) {
                tc::tma_load_3d(smem + Cfg::OFF_K + hh * Cfg::HALF, cache ? &map_kc : &map_k, 64 * hh, krow, bg, kv_full);
                tc::tma_load_3d(smem + Cfg::OFF_V + hh * Cfg::HALF, cache ? &map_vc : &map_v, 64 * hh, krow, bg, kv_full);
            }
            int t = 0;
            for (; t < ntiles; ++t) {
                const int s = t & 1;
                if (!wait_bar(t_empty + s, ((t >> 1) & 1) ^ 1, p.wb, kDevTimeoutSlotWait, abort_flag)) break;
                const int bh = bg * G + (first + t) / per_head, m = m_first + (first + t) % per_head;
                uint8_t* dst = smem + Cfg::OFF_T + s * 2 * Cfg::TILE;
                uint8_t* rows = smem + Cfg::OFF_ROW + s * 1024;
                mbar_arrive_expect_tx(t_full + s, 2 * Cfg::TILE + 1024);
                for (int x = 0; x < D / 64; ++x) {
                    tc::tma_load_3d(dst + x * Cfg::HALF, &map_q, 64 * x, 128 * m, bh, t_full + s);
                    tc::tma_load_3d(dst + Cfg::TILE + x * Cfg::HALF, &map_do, 64 * x, 128 * m, bh, t_full + s);
                }
                const size_t at = ((size_t)bh * p.n_mblk + m) * 128;
                tc::bulk_load(rows, p.nL2 + at, 512, t_full + s);
                tc::bulk_load(rows + 512, p.D + at, 512, t_full + s);
            }
            wait_bar(kv_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag);
            for (int s = 0; s < 2; ++s) {
                const int uses = (t - s + 1) / 2;
                if (uses > 0) wait_bar(t_full + s, (uses - 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint64_t dK = desc_kmajor_sw128(sbase + Cfg::OFF_K);
        const uint64_t dV = desc_kmajor_sw128(sbase + Cfg::OFF_V);
        const uint64_t dTk = desc_kmajor_sw128(sbase + Cfg::OFF_T);
        const uint64_t dTn = desc_mnmajor_sw128(sbase + Cfg::OFF_T, Cfg::HALF);
        auto issue_ss = [&](uint32_t acc, uint64_t a, uint64_t b) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * Cfg::HALF + (kk & 3) * 32) >> 4;
                tc::mma_bf16_ss_warp(acc, a + off, b + off, Cfg::IDESC_S, kk > 0);
            }
        };
        auto issue_ts = [&](uint32_t acc, uint32_t a, uint64_t b, bool first) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 rows at a time; the rows' halves at columns 0 and 64
                tc::mma_bf16_ts_warp(acc, a + 64 * (kk >> 2) + 8 * (kk & 3), b + (uint64_t)((kk * 16 * 128) >> 4),
                                     Cfg::IDESC_G, (!first || kk > 0) ? 1u : 0u);
        };
        constexpr uint64_t kStage = (2 * Cfg::TILE) >> 4, kDO = Cfg::TILE >> 4;
        bool ok = ntiles > 0 && warp_wait(kv_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag) &&
                  warp_wait(t_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag);
        if (ok) {
            issue_ss(tmem, dK, dTk);
            tc::mma_commit_warp(s_full);
            issue_ss(tmem + 128, dV, dTk + kDO);
            tc::mma_commit_warp(dp_full);
        }
        for (int t = 0; ok && t < ntiles; ++t) {
            const uint64_t at = (t & 1) * kStage, next = kStage - at;
            if (!(ok = warp_wait(p_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            issue_ts(tmem + 256, tmem, dTn + at + kDO, t == 0);  // dV += P^T dO
            if (t + 1 < ntiles) {
                if (!(ok = warp_wait(t_full + ((t + 1) & 1), ((t + 1) >> 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag))) break;
                issue_ss(tmem, dK, dTk + next);
                tc::mma_commit_warp(s_full);
            }
            if (!(ok = warp_wait(ds_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            issue_ts(tmem + 256 + D, tmem + 128, dTn + at, t == 0);  // dK += dS^T Q
            tc::mma_commit_warp(t_empty + (t & 1));
            if (t + 1 < ntiles) {
                issue_ss(tmem + 128, dV, dTk + next + kDO);
                tc::mma_commit_warp(dp_full);
            }
        }
        tc::mma_commit_warp(drain);
        __syncwarp();
        warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
    } else {
        // ---------------------------------------------------------- key warpgroups
        const int wg = (warp - 2) >> 2;  // rows 64 wg .. 64 wg + 63 of a tile
        const int quad = warp & 3;
        const int kr = quad * 32 + lane;  // key inside the block = TMEM lane
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tl = tmem + lane_off + 64 * wg;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        for (int t = 0; t < ntiles; ++t) {
            // the rows' statistics came with the tile
            const float* rows = reinterpret_cast<const float*>(smem + Cfg::OFF_ROW + (t & 1) * 1024) + 64 * wg;
            if (!(ok = warp_wait(t_full + (t & 1), (t >> 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag) &&
                       warp_wait(s_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag)))
                break;
            fence_after_sync();
            uint32_t s[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tl + 32 * c, s[c]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::reg_fence(s[c]);
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                const float4 nl = *reinterpret_cast<const float4*>(rows + e);
                uint32_t* x = &s[e >> 5][e & 31];
                const float2 a = tc::ffma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, make_float2(nl.x, nl.y));
                const float2 b = tc::ffma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), sc2, make_float2(nl.z, nl.w));
                x[0] = __float_as_uint(ex2(a.x));
                x[1] = __float_as_uint(ex2(a.y));
                x[2] = __float_as_uint(ex2(b.x));
                x[3] = __float_as_uint(ex2(b.y));
            }
            // the diagonal tile: row c sees key kr if c >= kr
            if (!cache && (first + t) % per_head == 0) {
                const int lo = kr - 64 * wg;
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e < lo) s[e >> 5][e & 31] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 64; e += 2)
                pk[e >> 1] = tc::pack_bf16(__uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1]));
            tc::tmem_st32(tl, pk);
            tc::tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            if (!(ok = warp_wait(dp_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t dp[32];
                tc::tmem_ld32(tl + 128 + 32 * c, dp);
                tc::tmem_ld_wait();
                tc::reg_fence(dp);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 dr = *reinterpret_cast<const float4*>(rows + 128 + 32 * c + e);
                    pk[16 * c + (e >> 1)] =
                        tc::pack_bf16(__uint_as_float(s[c][e]) * (__uint_as_float(dp[e]) - dr.x),
                                      __uint_as_float(s[c][e + 1]) * (__uint_as_float(dp[e + 1]) - dr.y));
                    pk[16 * c + (e >> 1) + 1] =
                        tc::pack_bf16(__uint_as_float(s[c][e + 2]) * (__uint_as_float(dp[e + 2]) - dr.z),
                                      __uint_as_float(s[c][e + 3]) * (__uint_as_float(dp[e + 3]) - dr.w));
                }
            }
            tc::tmem_st32(tl + 128, pk);
            tc::tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        if (ok && warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag)) {
            fence_after_sync();
            // into shared memory, where the query tiles were: dV by the first warpgroup,
            // dK by the second; 16-byte chunks of a row are permuted by the row, so that
            // neither these stores nor the loads below meet in a bank
            float* acc = reinterpret_cast<float*>(smem + Cfg::OFF_T) + (wg * 128 + kr) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc::tmem_ld32(tmem + lane_off + 256 + wg * D + c, o);
                tc::tmem_ld_wait();
                tc::reg_fence(o);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4*>(acc + (((c + e) / 4) ^ (kr & (D / 4 - 1))) * 4) =
                        ntiles ? make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    fence_before_sync();
    __syncwarp();
    tc::cluster_sync();
    if (warp == 1) {
        fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
    // each CTA adds up its share of the keys over the cluster, in the order of its
    // CTAs; slots n.. of the last cache block get zeros
    const int key0 = cache ? 128 * kb : t0, keys = min(128, (cache ? p.C : p.T) - key0);
    const int k0 = 128 * rank / ranks, k1 = min(keys, 128 * (rank + 1) / ranks);
    for (int e = threadIdx.x; e < 2 * (k1 - k0) * (D / 4); e += kThreads) {
        const int c4 = e % (D / 4), k = k0 + e / (D / 4) % (k1 - k0), part = e / (D / 4) / (k1 - k0);
        const uint32_t at = sbase + Cfg::OFF_T + ((part * 128 + k) * D + (c4 ^ (k & (D / 4 - 1))) * 4) * 4;
        float4 a = tc::cluster_load4(at, 0);
        for (int q = 1; q < ranks; ++q) {
            const float4 x = tc::cluster_load4(at, q);
            a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
        }
        const float mul = part ? p.scale : 1.f;
        uint2 h = make_uint2(tc::pack_bf16(a.x * mul, a.y * mul), tc::pack_bf16(a.z * mul, a.w * mul));
        if (cache && key0 + k >= p.n) h = make_uint2(0, 0);
        __nv_bfloat16* base = part ? (cache ? p.dK : p.dk) : (cache ? p.dV : p.dv);
        *reinterpret_cast<uint2*>(base + ((size_t)bg * (cache ? p.C : p.T) + key0 + k) * D + 4 * c4) = h;
    }
    tc::cluster_sync();  // no CTA leaves while another reads its sums
}

// CTAs per key block of the dK / dV kernel. A block's query tiles are divided among
// a cluster when there are few blocks, or when whole blocks leave SMs idle at the
// end. The estimate, in tiles: what an SM has to do, half of a CTA's tiles as the
// unevenness of the last round, and kCtaTiles for what every CTA does besides.
int cluster_for(int groups, int G, int n_mblk, int nbc, int num_sms) {
    constexpr double kCtaTiles = 2.0;
    const double units = (double)groups * (nbc + n_mblk);
    const double sum = (double)groups * G * n_mblk * (nbc + 0.5 * (n_mblk + 1));
    const double most = G * n_mblk;
    double best = 0;
    int s_best = 1;
    for (int s = 1; s <= kMaxCluster && s <= most; ++s) {
        const double ctas = units * s;
        const double t = ctas <= num_sms ? most / s + kCtaTiles : sum / num_sms + 0.5 * most / s + kCtaTiles * ctas / num_sms;
        if (s == 1 || t < best) {
            best = t;
            s_best = s;
        }
    }
    return s_best;
}

template <int D>
cudaError_t backward_launch(const CkptBwdArgs& a) {
    if (cudaError_t e = ensure_smem_limit(ckpt_dq_tc_kernel<D>, DqCfg<D>::SMEM); e != cudaSuccess) return e;
    if (cudaError_t e = ensure_smem_limit(ckpt_dkdv_tc_kernel<D>, DkvCfg<D>::SMEM); e != cudaSuccess) return e;
    CUtensorMap mq, mdo, mkc, mvc, mk, mv;
    const uint64_t heads = (uint64_t)a.B * a.Hq, groups = (uint64_t)a.B * a.Hkv;
    const uint64_t rows = a.n > 0 ? a.n : 1;  // an empty cache is never loaded from
    if (!tc_make_map3(&mq, a.q, a.T, heads, a.T, D, 128) || !tc_make_map3(&mdo, a.dout, a.T, heads, a.T, D, 128) ||
        !tc_make_map3(&mkc, a.K, rows, groups, a.pitch, D, 128) || !tc_make_map3(&mvc, a.V, rows, groups, a.pitch, D, 128) ||
        !tc_make_map3(&mk, a.k, a.T, groups, a.T, D, 128) || !tc_make_map3(&mv, a.v, a.T, groups, a.T, D, 128))
        return cudaErrorInvalidValue;
    CkptTcParams p;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.T = a.T;
    p.C = a.C;
    p.n = a.n;
    p.n_mblk = (a.T + 127) / 128;
    p.nbc = (a.n + 127) / 128;
    p.nbC = (a.C + 127) / 128;
    p.scale = 1.f / sqrtf((float)D);
    p.scale_log2 = kLog2e * p.scale;
    p.nL2 = a.stats;
    p.D = a.stats + heads * p.n_mblk * 128;
    p.dq = static_cast<__nv_bfloat16*>(a.dq);
    p.dK = static_cast<__nv_bfloat16*>(a.dK);
    p.dV = static_cast<__nv_bfloat16*>(a.dV);
    p.dk = static_cast<__nv_bfloat16*>(a.dk);
    p.dv = static_cast<__nv_bfloat16*>(a.dv);
    p.wb = a.wb;
    cudaError_t e = launch_ex(false, ckpt_dq_tc_kernel<D>, dim3((unsigned)(p.n_mblk * heads)), dim3(kThreads),
                              DqCfg<D>::SMEM, a.stream, mq, mdo, mkc, mvc, mk, mv, p);
    if (e != cudaSuccess) return e;
    const int ranks = cluster_for((int)groups, a.Hq / a.Hkv, p.n_mblk, p.nbc, a.num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.nbC + p.n_mblk) * groups * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = DkvCfg<D>::SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ckpt_dkdv_tc_kernel<D>, mq, mdo, mkc, mvc, mk, mv, p);
}

}  // namespace

cudaError_t launch_ckpt_backward_tc(const CkptBwdArgs& a) {
    return a.d == 64 ? backward_launch<64>(a) : backward_launch<128>(a);
}

}  // namespace h2o
