// ckpt_backward_tc.cu -- tensor-core (tcgen05 + TMEM + TMA) kernels of the
// backward of a step's attention at the values an 8-bit checkpoint stands for
// (bf16; the formulas are ckpt_backward.cu's).
//
// The query rows of a KV head, R = G T of them (row = head-in-group * T + token),
// are cut into 128-row tiles whatever their heads, so that short chunks fill them;
// the keys into 128-key blocks, the cache's and the chunk's.
//
// ckpt_stats_tc_kernel  one CTA per query tile: S = Q K^T and dP = dO V^T per key
//     block, and each row's running maximum m, sum l = sum e and w = sum e dp
//     (e = 2^(s - m)); then LSE = m + log2 l and D = w / l, in fp32.
// ckpt_grad_tc_kernel   two kinds of CTA in one grid:
//     dQ, one CTA per query tile: the two products again, dS = P (dP - D) over S in
//     TMEM as a bf16 pair hi + lo, and dQ += hi K + lo K with them as A operands from
//     TMEM.
//     dK and dV, one CTA, or a cluster, per (KV head, 128-key block), one key per TMEM
//     lane: per query tile of the KV head, S^T = K Q^T and dP^T = V dO^T; P^T and dS^T
//     go back over them as bf16 pairs and are the A operands of dV += P^T dO and
//     dK += dS^T Q.
// With pairs (16 bits) a gradient's error is that of its own rounding to bf16, whatever
// the size of the step. With one bf16 per weight it is, in 2-norm over heavy-hitter keys,
// 1.7 times that for dq, whose terms cancel (sum_j ds_j = 0, and keys have much in
// common), and 1.2 to 1.7 times for dk and dv. The second products of dq cost 18 us of
// 121 at T=1024 C=2048, those of dk and dv 216 against 200 us a pass with the inputs in
// L2 and 251 against 226 without.
// Where query tiles are few, their key blocks are divided among several CTAs: the last
// one of a tile adds up the statistics, and ckpt_dq_combine_kernel the parts of dQ, in
// order.
//
// Bound by the tensor core: 2 products of 2 d per visible (row, key) for the
// statistics, 4 for dQ and 6 for dK and dV, a pair's two one after the other over the
// same operand (all hi before all lo: 225 us a pass for 216). An operand pair from shared
// memory needs 128 bytes a clock at the MMA's full rate, all there is, so P and dS stay
// in TMEM (64 bytes a clock), and they never cross shared memory. A TMA loader, an MMA
// issuer and four warpgroups that share every tile, 32 of its columns each (two with
// 64: 202 us a pass at T=1024 C=2048 d=128 and 49 at B=2 T=333 C=1000 d=64; four: 197
// and 47; one bf16 per weight of dk and dv). The issue order keeps the tensor core on a
// product that does not wait for the exponentials in progress: dV(t), S(t+1) while dS(t)
// is computed, dK(t), dP(t+1) while P(t+1) is.
//
// Times of a pass are taken with the inputs in L2 and the clock not yet held down by
// power, unless they say otherwise; with inputs that change from pass to pass
// T=1024 C=2048 takes 251 us where it takes 216 so.
//
// Rows past the end of a KV head or cache arrive as zeros (3-D tensor maps), so
// nothing of another head enters a tile. Statistics and gradients accumulate in fp32.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "operators.h"
#include "tc_operators.cuh"

namespace h2o {
namespace {

using tc::desc_kmajor_sw128;
using tc::desc_mnmajor_sw128;
using tc::ex2;
using tc::fence_after_sync;
using tc::fence_before_sync;

constexpr int kGroups = 4;  // warpgroups that share a tile, 32 of its columns each
constexpr int kConsumers = 128 * kGroups, kThreads = 64 + kConsumers;  // and a loader and an MMA issuer
constexpr int kArrivals = kConsumers / 32;
constexpr int kMaxCluster = 4;

struct CkptTcParams {
    int B, Hq, Hkv, T, C, n;
    int R;       // query rows per KV head
    int tiles;   // 128-row query tiles per KV head
    int n_mblk;  // chunk key blocks = ceil(T / 128)
    int nbc;     // cache key blocks = ceil(n / 128)
    int nbC;     // 128-slot blocks of the whole cache
    int parts;   // CTAs per query tile, in both passes
    int dkdv_ctas, dq_ctas;  // of the gradients' grid
    float scale_log2, scale;
    float* nL2;     // [B*Hkv][128 * tiles]: -(log2-domain LSE) per row, -inf in padding rows
    float* D;       // [B*Hkv][128 * tiles], 0 in padding rows
    float4* stat;   // parts > 1: [parts][B*Hkv][128 * tiles]: m, l, w of a part
    unsigned* count;  // parts > 1: [B*Hkv * tiles], zero
    float4* part;   // parts > 1: [parts][B*Hkv * tiles][D / 4][128]: four columns of dQ
    __nv_bfloat16* dq;
    __nv_bfloat16* dK;
    __nv_bfloat16* dV;
    __nv_bfloat16* dk;
    __nv_bfloat16* dv;
    WaitBound wb;
};

// Chunk key blocks that some row of a query tile sees (at least one).
__device__ __forceinline__ int chunk_blocks(const CkptTcParams& p, int tile) {
    const int r0 = 128 * tile, r1 = min(p.R, r0 + 128) - 1;
    return (r1 / p.T > r0 / p.T ? p.T - 1 : r1 % p.T) / 128 + 1;
}

// What rounding to the packed bf16 `hi` left of 32 values, as bf16, to 16 columns.
__device__ __forceinline__ void store_rest(uint32_t taddr, const uint32_t (&x)[32], const uint32_t (&hi)[16]) {
    uint32_t lo[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const uint32_t h = hi[e >> 1];
        lo[e >> 1] = tc::pack_bf16(__uint_as_float(x[e]) - __uint_as_float(h << 16),
                                   __uint_as_float(x[e + 1]) - __uint_as_float(h & 0xffff0000u));
    }
    tc::tmem_st16(taddr, lo);
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
    static constexpr int OFF_BAR = OFF_RING + RING * TILE;
    static constexpr int NBAR = 24;
    static constexpr int SMEM_RAW = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int SMEM = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;  // one CTA (512 TMEM columns) per SM
    static constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(128, 128, false);
    static constexpr uint32_t IDESC_G = tc::idesc_bf16_f32(128, D, true);
};
static_assert(DqCfg<128>::SMEM_RAW <= 232448, "dQ kernel shared memory exceeds the per-CTA limit");

// One CTA (number `cta`) of the first pass (kPass 1) or the second (kPass 2).
template <int D, int kPass>
__device__ __forceinline__ void dq_cta(const CUtensorMap& map_q, const CUtensorMap& map_do, const CUtensorMap& map_kc,
                                       const CUtensorMap& map_vc, const CUtensorMap& map_k, const CUtensorMap& map_v,
                                       const CkptTcParams& p, int cta) {
    using Cfg = DqCfg<D>;
    constexpr int RING = Cfg::RING;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* q_full = bars;                  // Q and dO tiles
    uint64_t* ring_full = bars + 1;           // [RING]
    uint64_t* ring_empty = ring_full + RING;  // [RING]
    uint64_t* sd_full = ring_empty + RING;    // [2] pass 1: S and dP of a buffer
    uint64_t* sd_free = sd_full + 2;          // [2] pass 1, kArrivals: in registers
    uint64_t* s_full = sd_free + 2;           // [2] pass 2: S of a buffer
    uint64_t* dp_full = s_full + 2;           // pass 2: dP
    uint64_t* ds_full = dp_full + 1;          // pass 2, kArrivals: dS over S, dP in registers
    uint64_t* drain = ds_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int part = cta % p.parts, unit = cta / p.parts;
    const int groups = p.B * p.Hkv, bg = unit % groups;
    int tile = p.tiles - 1 - unit / groups;
    if (p.T % 128 == 0)  // the heads' last tiles first: they have the most key blocks
        tile = unit / groups % (p.tiles / p.n_mblk) * p.n_mblk + p.n_mblk - 1 - unit / groups / (p.tiles / p.n_mblk);
    const int m0 = tile * 128;
    const int all = p.nbc + chunk_blocks(p, tile);  // key blocks: cache, then chunk
    const int jb = all * part / p.parts, nb = all * (part + 1) / p.parts - jb;  // this CTA's
    constexpr bool pass1 = kPass == 1, pass2 = kPass == 2;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < RING; ++s) {
            mbar_init(ring_full + s, 1);
            mbar_init(ring_empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sd_full + b, 1);
            mbar_init(sd_free + b, kArrivals);
            mbar_init(s_full + b, 1);
        }
        mbar_init(dp_full, 1);
        mbar_init(ds_full, kArrivals);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    uint32_t tmem = 0;
    if (warp == 0) {
        // the loader has initialised the barriers and needs nothing else: its first loads
        // are on their way while the others set up
        __syncwarp();
        tc::named_arrive(4, kThreads);
    } else {
        if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
        fence_before_sync();
        tc::named_sync(4, kThreads);
        fence_after_sync();
        tmem = *tmem_slot;
    }
    griddep_wait();  // the kernel before has written what this one reads
    if (pass1 || p.parts > 1) griddep_launch_dependents();
     // S of the two buffers at 0 and 128, dP at 256 (and 384 in pass 1), dQ at 384
    const uint32_t sbase = smem_u32(smem);

    if (warp == 0) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, 2 * Cfg::TILE);
            for (int hh = 0; hh < D / 64; ++hh) {
                tc::tma_load_3d(smem + Cfg::OFF_Q + hh * Cfg::HALF, &map_q, 64 * hh, m0, bg, q_full);
                tc::tma_load_3d(smem + Cfg::OFF_DO + hh * Cfg::HALF, &map_do, 64 * hh, m0, bg, q_full);
            }
            int L = 0;
            bool ok = true;
            for (int it = 0; ok && it < nb; ++it) {
                const int j = jb + it;
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
        const int n1 = pass1 ? nb : 0, n2 = pass2 ? nb : 0;
        for (int t = 0; ok && t < n1; ++t) {
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
        auto issue_s = [&](int t) {  // needs buffer t & 1 free, or read by products issued before
            const int l = 2 * t;
            if (!wait_ring(l)) return false;
            issue_ss(tmem + 128 * (t & 1), dQd, l % RING);
            tc::mma_commit_warp(s_full + (t & 1));
            return true;
        };
        auto issue_dp = [&](int t) {
            const int l = 2 * t + 1;
            if (!wait_ring(l)) return false;
            issue_ss(tmem + 256, dOd, l % RING);
            tc::mma_commit_warp(dp_full);
            tc::mma_commit_warp(ring_empty + l % RING);
            return true;
        };
        ok = ok && (n2 < 1 || (issue_s(0) && issue_dp(0))) && (n2 < 2 || issue_s(1));
        for (int t = 0; ok && t < n2; ++t) {
            if (!(ok = warp_wait(ds_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            if (t + 1 < n2 && !(ok = issue_dp(t + 1))) break;
            const int ks = 2 * t % RING;
            const uint64_t b = dRingN + (uint64_t)((ks * Cfg::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 16 keys at a time; every 32 keys at their columns, hi and lo
                const uint32_t a = tmem + 128 * (t & 1) + 32 * (kk >> 1) + 8 * (kk & 1);
                const uint64_t bk = b + (uint64_t)((kk * 16 * 128) >> 4);
                tc::mma_bf16_ts_warp(tmem + 384, a, bk, Cfg::IDESC_G, (t > 0 || kk > 0) ? 1u : 0u);
                tc::mma_bf16_ts_warp(tmem + 384, a + 16, bk, Cfg::IDESC_G, 1u);
            }
            tc::mma_commit_warp(ring_empty + ks);
            if (t + 2 < n2) ok = issue_s(t + 2);
        }
        // all MMAs issued here complete before TMEM can be released
        tc::mma_commit_warp(drain);
        __syncwarp();
        warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
    } else {
        // ---------------------------------------------------------- row warpgroups
        const int wg = (warp - 2) >> 2;  // columns 32 wg .. 32 wg + 31
        const int quad = warp & 3;
        const int r = quad * 32 + lane;  // row inside the tile = TMEM lane
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16) + 32 * wg;
        const int token = (m0 + r) % p.T;
        // visible columns of this thread's in this CTA's block t: e < limit
        auto limit_of = [&](int t) {
            const int j = jb + t;
            return (j < p.nbc ? p.n - 128 * j : token - 128 * (j - p.nbc) + 1) - 32 * wg;
        };
        float m = -INFINITY, l = 0.f, w = 0.f;
        bool ok = true;
        for (int t = 0; pass1 && t < nb; ++t) {
            const int b = t & 1;
            if (!(ok = warp_wait(sd_full + b, (t >> 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t s[32], dp[32];
            tc::tmem_ld32(tl + 128 * b, s);
            tc::tmem_ld32(tl + 256 + 128 * b, dp);
            tc::tmem_ld_wait();
            tc::reg_fence(s);
            tc::reg_fence(dp);
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(sd_free + b);
            const int limit = limit_of(t);
            if (limit < 32) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e >= limit) s[e] = __float_as_uint(-INFINITY);
            }
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                mx0 = tc::max3(mx0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                mx1 = tc::max3(mx1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
            }
            const float mn = fmaxf(m, fmaxf(mx0, mx1) * p.scale_log2);
            const float ms = mn == -INFINITY ? 0.f : mn;  // no visible key in these columns yet
            const float a = ex2(m - ms);
            m = mn;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-ms, -ms);
            float2 l2 = make_float2(0.f, 0.f), w2 = l2;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 x = tc::ffma2(
                    make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, nm2);
                const float2 pe = make_float2(ex2(x.x), ex2(x.y));
                l2 = tc::fadd2(l2, pe);
                w2 = tc::ffma2(pe, make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), w2);
            }
            l = fmaf(l, a, l2.x + l2.y);
            w = fmaf(w, a, w2.x + w2.y);
        }
        const bool row_ok = m0 + r < p.R;
        const size_t at = ((size_t)bg * p.tiles + tile) * 128 + r, all_rows = (size_t)groups * p.tiles * 128;
        if (pass1) {
            // the quarters of a row meet, in the ring: every key block has been multiplied
            float* st = reinterpret_cast<float*>(smem + Cfg::OFF_RING);  // [kGroups][3][128]
            st[384 * wg + r] = m;
            st[384 * wg + 128 + r] = l;
            st[384 * wg + 256 + r] = w;
            tc::named_sync(1, kConsumers);
            if (wg == 0) {
                float M = m;
#pragma unroll
                for (int g = 1; g < kGroups; ++g) M = fmaxf(M, st[384 * g + r]);
                float Ms = M == -INFINITY ? 0.f : M, L = 0.f, W = 0.f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float a = ex2(st[384 * g + r] - Ms);
                    L = fmaf(st[384 * g + 128 + r], a, L);
                    W = fmaf(st[384 * g + 256 + r], a, W);
                }
                bool mine = true;
                if (p.parts > 1) {
                    // the tile's last CTA adds up its parts, in order
                    p.stat[part * all_rows + at] = make_float4(M, L, W, 0.f);
                    __threadfence();
                    tc::named_sync(2, 128);
                    if (threadIdx.x == 64) {
                        const bool last = atomicAdd(p.count + unit, 1u) == (unsigned)p.parts - 1;
                        if (last) p.count[unit] = 0;
                        st[0] = last ? 1.f : 0.f;
                    }
                    tc::named_sync(2, 128);
                    mine = st[0] != 0.f;
                    if (mine) {
                        __threadfence();
                        M = -INFINITY;
                        for (int q = 0; q < p.parts; ++q) M = fmaxf(M, p.stat[q * all_rows + at].x);
                        Ms = M == -INFINITY ? 0.f : M;
                        L = W = 0.f;
                        for (int q = 0; q < p.parts; ++q) {
                            const float4 x = p.stat[q * all_rows + at];
                            const float a = ex2(x.x - Ms);
                            L = fmaf(x.y, a, L);
                            W = fmaf(x.z, a, W);
                        }
                    }
                }
                if (mine) {
                    p.nL2[at] = row_ok ? -(M + log2f(L)) : -INFINITY;
                    p.D[at] = row_ok ? W / L : 0.f;
                }
            }
        }
        const float nL2 = pass2 ? p.nL2[at] : 0.f, Dr = pass2 ? p.D[at] : 0.f;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nL2, nL2), nd2 = make_float2(-Dr, -Dr);
        for (int t = 0; pass2 && ok && t < nb; ++t) {
            const uint32_t tS = tl + 128 * (t & 1);
            if (!(ok = warp_wait(s_full + (t & 1), (t >> 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t s[32];
            tc::tmem_ld32(tS, s);
            tc::tmem_ld_wait();
            tc::reg_fence(s);
            const int limit = limit_of(t);
            if (limit < 32) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e >= limit) s[e] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 x = tc::ffma2(
                    make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, nl2);
                s[e] = __float_as_uint(ex2(x.x));
                s[e + 1] = __float_as_uint(ex2(x.y));
            }
            if (!(ok = warp_wait(dp_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t dp[32], hi[16], lo[16];
            tc::tmem_ld32(tl + 256, dp);
            tc::tmem_ld_wait();
            tc::reg_fence(dp);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 y = tc::fadd2(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), nd2);
                const float a = __uint_as_float(s[e]) * y.x, b = __uint_as_float(s[e + 1]) * y.y;
                const uint32_t h = tc::pack_bf16(a, b);
                hi[e >> 1] = h;
                lo[e >> 1] = tc::pack_bf16(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
            }
            tc::tmem_st16(tS, hi);
            tc::tmem_st16(tS + 16, lo);
            tc::tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        if (ok) ok = warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
        fence_after_sync();
        // dQ: this thread has D / 4 columns of its row. A part goes to memory as it is,
        // rows next to each other; the whole goes through shared memory (the key ring is
        // done with), 16-byte chunks permuted by the row so that no bank is met twice
        constexpr int kCols = D / kGroups;
        const int col0 = kCols * wg;
        float* acc = reinterpret_cast<float*>(smem + Cfg::OFF_RING);
        if (pass2 && ok) {
            uint32_t o[kCols];
            const uint32_t tQ = tmem + ((uint32_t)(quad * 32) << 16) + 384 + col0;
            if constexpr (kCols == 32)
                tc::tmem_ld32(tQ, o);
            else
                tc::tmem_ld16(tQ, o);
            tc::tmem_ld_wait();
            tc::reg_fence(o);
            float4* dst = p.part + ((((size_t)part * groups + bg) * p.tiles + tile) * (D / 4) + col0 / 4) * 128 + r;
#pragma unroll
            for (int e = 0; e < kCols; e += 4) {
                const float4 x = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                             __uint_as_float(o[e + 3]));
                if (p.parts > 1)
                    dst[e / 4 * 128] = x;
                else
                    *reinterpret_cast<float4*>(acc + r * D + (((col0 + e) / 4) ^ (r & (D / 4 - 1))) * 4) = x;
            }
        }
        if (pass2 && p.parts == 1) {
            tc::named_sync(1, kConsumers);
            const int rows = min(128, p.R - m0);
            for (int e = threadIdx.x - 64; e < rows * (D / 4); e += kConsumers) {
                const int rr = e / (D / 4), c4 = e % (D / 4);
                const float4 x = *reinterpret_cast<const float4*>(acc + rr * D + (c4 ^ (rr & (D / 4 - 1))) * 4);
                *reinterpret_cast<uint2*>(p.dq + ((size_t)bg * p.R + m0 + rr) * D + 4 * c4) =
                    make_uint2(tc::pack_bf16(x.x * p.scale, x.y * p.scale), tc::pack_bf16(x.z * p.scale, x.w * p.scale));
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// dQ of a row from the parts of its tile, in order; one thread per four columns,
// neighbouring lanes neighbouring rows, as the parts lie.
template <int D>
__global__ void __launch_bounds__(256) ckpt_dq_combine_kernel(const CkptTcParams p) {
    griddep_wait();
    const int r = threadIdx.x % 32 + 32 * (blockIdx.x % 4), unit = blockIdx.x / 4;  // KV head and tile
    const int row = unit % p.tiles * 128 + r;
    if (row >= p.R) return;
    for (int c4 = threadIdx.x / 32; c4 < D / 4; c4 += 8) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int q = 0; q < p.parts; ++q) {
            const float4 x = p.part[(((size_t)q * p.B * p.Hkv * p.tiles + unit) * (D / 4) + c4) * 128 + r];
            a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
        }
        *reinterpret_cast<uint2*>(p.dq + ((size_t)(unit / p.tiles) * p.R + row) * D + 4 * c4) =
            make_uint2(tc::pack_bf16(a.x * p.scale, a.y * p.scale), tc::pack_bf16(a.z * p.scale, a.w * p.scale));
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

// One CTA (number `cta`), or its cluster.
template <int D>
__device__ __forceinline__ void dkdv_cta(const CUtensorMap& map_q, const CUtensorMap& map_do, const CUtensorMap& map_kc,
                                         const CUtensorMap& map_vc, const CUtensorMap& map_k, const CUtensorMap& map_v,
                                         const CkptTcParams& p, int cta) {
    using Cfg = DkvCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* kv_full = bars;
    uint64_t* t_full = bars + 1;   // [2] a query tile has landed
    uint64_t* t_empty = bars + 3;  // [2] its MMAs have completed
    uint64_t* s_full = bars + 5;   // S^T
    uint64_t* p_full = bars + 6;   // kArrivals: P^T over S^T
    uint64_t* dp_full = bars + 7;  // dP^T
    uint64_t* ds_full = bars + 8;  // kArrivals: dS^T over dP^T
    uint64_t* drain = bars + 9;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int groups = p.B * p.Hkv;
    // blocks in decreasing work: cache blocks (all rows see them), chunk blocks,
    // blocks of empty slots (zeros)
    const int rank = tc::cluster_rank(), ranks = tc::cluster_size();  // the cluster's CTAs share a key block
    const int unit = cta / ranks;
    const int kb = unit / groups, bg = unit % groups;
    if (kb >= p.nbc + p.n_mblk) {
        griddep_wait();  // who used dK and dV before is done with them
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
    // this CTA's query tiles: of those of the KV head that see a key of the block,
    // every ranks-th one; next() gives the one after `tile` (p.tiles: none)
    auto next = [&](int tile, int steps) {
        if (t0 == 0) return min(tile + steps, p.tiles);
        while (steps > 0 && ++tile < p.tiles) steps -= 128 * (chunk_blocks(p, tile) - 1) >= t0;
        return tile;
    };
    const int first = next(-1, rank + 1);
    const bool any = first < p.tiles;

    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(t_full + s, 1);
            mbar_init(t_empty + s, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(p_full, kArrivals);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, kArrivals);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    uint32_t tmem = 0;
    if (warp == 0) {
        // the loader has initialised the barriers and needs nothing else: its first loads
        // are on their way while the others set up
        __syncwarp();
        tc::named_arrive(4, kThreads);
    } else {
        if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
        fence_before_sync();
        tc::named_sync(4, kThreads);
        fence_after_sync();
        tmem = *tmem_slot;
    }
    griddep_wait();  // the kernel before has written what this one reads
    if (p.parts > 1) griddep_launch_dependents();
     // S^T at 0, dP^T at 128, dV at 256, dK at 256 + D
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
            for (int tile = first; tile < p.tiles; tile = next(tile, ranks), ++t) {
                const int s = t & 1;
                if (!wait_bar(t_empty + s, ((t >> 1) & 1) ^ 1, p.wb, kDevTimeoutSlotWait, abort_flag)) break;
                uint8_t* dst = smem + Cfg::OFF_T + s * 2 * Cfg::TILE;
                uint8_t* rows = smem + Cfg::OFF_ROW + s * 1024;
                mbar_arrive_expect_tx(t_full + s, 2 * Cfg::TILE + 1024);
                for (int x = 0; x < D / 64; ++x) {
                    tc::tma_load_3d(dst + x * Cfg::HALF, &map_q, 64 * x, 128 * tile, bg, t_full + s);
                    tc::tma_load_3d(dst + Cfg::TILE + x * Cfg::HALF, &map_do, 64 * x, 128 * tile, bg, t_full + s);
                }
                const size_t at = ((size_t)bg * p.tiles + tile) * 128;
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
            for (int kk = 0; kk < 8; ++kk) {  // 16 rows at a time; every 32 rows at their columns, hi and lo
                const uint32_t ak = a + 32 * (kk >> 1) + 8 * (kk & 1);
                const uint64_t bk = b + (uint64_t)((kk * 16 * 128) >> 4);
                tc::mma_bf16_ts_warp(acc, ak, bk, Cfg::IDESC_G, (!first || kk > 0) ? 1u : 0u);
                tc::mma_bf16_ts_warp(acc, ak + 16, bk, Cfg::IDESC_G, 1u);
            }
        };
        constexpr uint64_t kStage = (2 * Cfg::TILE) >> 4, kDO = Cfg::TILE >> 4;
        bool ok = any && warp_wait(kv_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag) &&
                  warp_wait(t_full, 0, p.wb, kDevTimeoutTmaWait, abort_flag);
        if (ok) {
            issue_ss(tmem, dK, dTk);
            tc::mma_commit_warp(s_full);
            issue_ss(tmem + 128, dV, dTk + kDO);
            tc::mma_commit_warp(dp_full);
        }
        int t = 0;
        for (int tile = first, after; ok && tile < p.tiles; tile = after, ++t) {
            after = next(tile, ranks);
            const bool more = after < p.tiles;
            const uint64_t at = (t & 1) * kStage, ahead = kStage - at;
            if (!(ok = warp_wait(p_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            issue_ts(tmem + 256, tmem, dTn + at + kDO, t == 0);  // dV += P^T dO
            if (more) {
                if (!(ok = warp_wait(t_full + ((t + 1) & 1), ((t + 1) >> 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag))) break;
                issue_ss(tmem, dK, dTk + ahead);
                tc::mma_commit_warp(s_full);
            }
            if (!(ok = warp_wait(ds_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            issue_ts(tmem + 256 + D, tmem + 128, dTn + at, t == 0);  // dK += dS^T Q
            tc::mma_commit_warp(t_empty + (t & 1));
            if (more) {
                issue_ss(tmem + 128, dV, dTk + ahead + kDO);
                tc::mma_commit_warp(dp_full);
            }
        }
        tc::mma_commit_warp(drain);
        __syncwarp();
        warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
    } else {
        // ---------------------------------------------------------- key warpgroups
        const int wg = (warp - 2) >> 2;  // rows 32 wg .. 32 wg + 31 of a tile
        const int quad = warp & 3;
        const int kr = quad * 32 + lane;  // key inside the block = TMEM lane
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tl = tmem + lane_off + 32 * wg;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        int t = 0;
        for (int tile = first; tile < p.tiles; tile = next(tile, ranks), ++t) {
            // the rows' statistics came with the tile
            const float* rows = reinterpret_cast<const float*>(smem + Cfg::OFF_ROW + (t & 1) * 1024) + 32 * wg;
            if (!(ok = warp_wait(t_full + (t & 1), (t >> 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag) &&
                       warp_wait(s_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag)))
                break;
            fence_after_sync();
            uint32_t s[32];
            tc::tmem_ld32(tl, s);
            tc::tmem_ld_wait();
            tc::reg_fence(s);
            // a chunk key is seen by the tokens from its own on: unless every row of the
            // tile is one, each is compared (a tile may hold the end of one head and the
            // start of another, or several heads)
            if (!cache) {
                const int i0 = 128 * tile % p.T;
                if (i0 + 127 >= p.T || i0 < t0 + 127) {
                    uint32_t vis = 0;
                    for (int c = -((i0 + 32 * wg) % p.T); c < 32; c += p.T) {  // a head starts at column c
                        const int lo = max(c + t0 + kr, 0), hi = min(c + p.T, 32);
                        if (lo < hi) vis |= (~0u >> (32 - (hi - lo))) << lo;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((vis >> e) & 1u)) s[e] = __float_as_uint(-INFINITY);
                }
            }
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 nl = *reinterpret_cast<const float4*>(rows + e);
                uint32_t* x = &s[e];
                const float2 a = tc::ffma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, make_float2(nl.x, nl.y));
                const float2 b = tc::ffma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), sc2, make_float2(nl.z, nl.w));
                const float2 pa = make_float2(ex2(a.x), ex2(a.y)), pb = make_float2(ex2(b.x), ex2(b.y));
                x[0] = __float_as_uint(pa.x);
                x[1] = __float_as_uint(pa.y);
                x[2] = __float_as_uint(pb.x);
                x[3] = __float_as_uint(pb.y);
                pk[e >> 1] = tc::pack_bf16(pa.x, pa.y);
                pk[(e >> 1) + 1] = tc::pack_bf16(pb.x, pb.y);
            }
            tc::tmem_st16(tl, pk);
            store_rest(tl + 16, s, pk);
            tc::tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            if (!(ok = warp_wait(dp_full, t & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
            fence_after_sync();
            uint32_t dp[32];
            tc::tmem_ld32(tl + 128, dp);
            tc::tmem_ld_wait();
            tc::reg_fence(dp);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 dr = *reinterpret_cast<const float4*>(rows + 128 + e);
                const float d4[4] = {dr.x, dr.y, dr.z, dr.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    s[e + x] = __float_as_uint(__uint_as_float(s[e + x]) * (__uint_as_float(dp[e + x]) - d4[x]));
                pk[e >> 1] = tc::pack_bf16(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                pk[(e >> 1) + 1] = tc::pack_bf16(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
            }
            tc::tmem_st16(tl + 128, pk);
            store_rest(tl + 144, s, pk);
            tc::tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        if (ok && warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag)) {
            fence_after_sync();
            // into shared memory, where the query tiles were: dV by the first two warpgroups,
            // dK by the others, half of the columns each; 16-byte chunks of a row are permuted by the row, so that
            // neither these stores nor the loads below meet in a bank
            float* acc = reinterpret_cast<float*>(smem + Cfg::OFF_T) + (wg / 2 * 128 + kr) * D;
#pragma unroll 1
            for (int c = wg % 2 * (D / 2); c < (wg % 2 + 1) * (D / 2); c += 32) {
                uint32_t o[32];
                tc::tmem_ld32(tmem + lane_off + 256 + wg / 2 * D + c, o);
                tc::tmem_ld_wait();
                tc::reg_fence(o);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4*>(acc + (((c + e) / 4) ^ (kr & (D / 4 - 1))) * 4) =
                        any ? make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_uint4(0, 0, 0, 0);
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
    const int k0 = 128 * rank / ranks, mine = min(keys, 128 * (rank + 1) / ranks) - k0;
    constexpr int kLanes = D / 4, kPerWarp = 32 / kLanes;  // lanes per row, rows per warp
    const int c4 = lane % kLanes;
#pragma unroll 4
    for (int i = warp * kPerWarp + lane / kLanes; i < 2 * mine; i += kThreads / 32 * kPerWarp) {
        const int part = i >= mine, k = k0 + i - (part ? mine : 0);
        const uint32_t at = Cfg::OFF_T + ((part * 128 + k) * D + (c4 ^ (k & (kLanes - 1))) * 4) * 4;
        float4 a;
        if (ranks == 1) {
            a = *reinterpret_cast<const float4*>(smem + at);
        } else {
            a = tc::cluster_load4(sbase + at, 0);
            for (int q = 1; q < ranks; ++q) {
                const float4 x = tc::cluster_load4(sbase + at, q);
                a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
            }
        }
        const float mul = part ? p.scale : 1.f;
        uint2 h = make_uint2(tc::pack_bf16(a.x * mul, a.y * mul), tc::pack_bf16(a.z * mul, a.w * mul));
        if (cache && key0 + k >= p.n) h = make_uint2(0, 0);
        __nv_bfloat16* base = part ? (cache ? p.dK : p.dk) : (cache ? p.dV : p.dv);
        *reinterpret_cast<uint2*>(base + ((size_t)bg * (cache ? p.C : p.T) + key0 + k) * D + 4 * c4) = h;
    }
    if (ranks > 1) tc::cluster_sync();  // no CTA leaves while another reads its sums
}

// First pass: the rows' statistics.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
ckpt_stats_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                     const __grid_constant__ CUtensorMap map_kc, const __grid_constant__ CUtensorMap map_vc,
                     const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const CkptTcParams p) {
    dq_cta<D, 1>(map_q, map_do, map_kc, map_vc, map_k, map_v, p, blockIdx.x);
}

// The gradients: dK and dV by the first CTAs, dQ by the rest, in one grid, so that
// each fills the SMs the other leaves idle (one after the other, with the first pass
// inside dQ's kernel: 242 us a pass at T=1024 C=2048 d=128 and 55 at B=2 T=333 C=1000
// d=64, against 202 and 52, one bf16 per weight of dk and dv). The longer CTAs, dK and
// dV's, go first (the other way round: 218 us).
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
ckpt_grad_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                    const __grid_constant__ CUtensorMap map_kc, const __grid_constant__ CUtensorMap map_vc,
                    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const CkptTcParams p) {
    const int cta = blockIdx.x - p.dkdv_ctas;
    if (cta < 0)
        dkdv_cta<D>(map_q, map_do, map_kc, map_vc, map_k, map_v, p, blockIdx.x);
    else if (cta < p.dq_ctas)  // the rest fills the last cluster
        dq_cta<D, 2>(map_q, map_do, map_kc, map_vc, map_k, map_v, p, cta);
}

// CTAs per key block for dK and dV: a block's query tiles are divided among a cluster
// when whole blocks would make a long tail. The estimate, in tiles (a query tile of a
// key block, and a key block of a query tile, take about as long): the longest CTA if
// all fit at once, else what an SM has to do, half of the longest CTA as the
// unevenness of the last round, and kCtaTiles for what every CTA does besides.
// Measured, clusters of 1, 2, 3 and 4: 216, 230, 261, 276 us a pass at T=1024 C=2048
// d=128 (192 blocks of up to 32 tiles), 104, 122, 142, 149 at T=512, 59, 62, 74, 84 at
// T=384 C=1024; 68, 46, 52, 53 with changing inputs at B=2 T=333 C=1000 d=64, eight query
// heads to a KV head (40 blocks of 21).
int cluster_for(int groups, int tiles, int n_mblk, int nbc, int parts, int num_sms) {
    constexpr double kCtaTiles = 6.0;
    const double sum = 2.0 * groups * tiles * (nbc + 0.5 * (n_mblk + 1));
    const int blocks = (nbc + n_mblk + parts - 1) / parts;
    double best = 0;
    int s_best = 1;
    for (int s = 1; s <= kMaxCluster && s <= tiles; ++s) {
        const double ctas = (double)groups * ((nbc + n_mblk) * s + tiles * parts), most = std::max((tiles + s - 1) / s, blocks);
        const double t = ctas <= num_sms ? most + kCtaTiles : sum / num_sms + 0.5 * most + kCtaTiles * ctas / num_sms;
        if (s == 1 || t < best) {
            best = t;
            s_best = s;
        }
    }
    return s_best;
}

int dq_tiles(int Hq, int Hkv, int T) { return (Hq / Hkv * T + 127) / 128; }

// CTAs per query tile of the dQ kernel: more than one only when the tiles fill less
// than half of the SMs and have blocks enough to repay two more launches.
int dq_parts(int groups, int tiles, int blocks, int num_sms) {
    const int units = groups * tiles;
    if (2 * units > num_sms || blocks < 8) return 1;
    return std::min(num_sms / units, blocks / 2);
}

template <int D>
cudaError_t backward_launch(const CkptBwdArgs& a) {
    constexpr int kGradSmem = std::max(DqCfg<D>::SMEM, DkvCfg<D>::SMEM);
    if (cudaError_t e = ensure_smem_limit(ckpt_stats_tc_kernel<D>, DqCfg<D>::SMEM); e != cudaSuccess) return e;
    if (cudaError_t e = ensure_smem_limit(ckpt_grad_tc_kernel<D>, kGradSmem); e != cudaSuccess) return e;
    CUtensorMap mq, mdo, mkc, mvc, mk, mv;
    const uint64_t groups = (uint64_t)a.B * a.Hkv;
    const int R = a.Hq / a.Hkv * a.T;
    const uint64_t rows = a.n > 0 ? a.n : 1;  // an empty cache is never loaded from
    if (!tc_make_map3(&mq, a.q, R, groups, R, D, 128) || !tc_make_map3(&mdo, a.dout, R, groups, R, D, 128) ||
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
    p.R = R;
    p.tiles = dq_tiles(a.Hq, a.Hkv, a.T);
    p.n_mblk = (a.T + 127) / 128;
    p.nbc = (a.n + 127) / 128;
    p.nbC = (a.C + 127) / 128;
    p.scale = 1.f / sqrtf((float)D);
    p.scale_log2 = kLog2e * p.scale;
    p.parts = dq_parts((int)groups, p.tiles, p.nbc + 1, a.num_sms);
    const size_t table = groups * p.tiles * 128;
    p.nL2 = a.stats;
    p.D = p.nL2 + table;
    p.stat = reinterpret_cast<float4*>(p.D + table);
    p.part = p.stat + table * p.parts;
    p.dq = static_cast<__nv_bfloat16*>(a.dq);
    p.dK = static_cast<__nv_bfloat16*>(a.dK);
    p.dV = static_cast<__nv_bfloat16*>(a.dV);
    p.dk = static_cast<__nv_bfloat16*>(a.dk);
    p.dv = static_cast<__nv_bfloat16*>(a.dv);
    p.wb = a.wb;
    p.count = a.count;
    const int ranks = cluster_for((int)groups, p.tiles, p.n_mblk, p.nbc, p.parts, a.num_sms);
    p.dkdv_ctas = (int)((p.nbC + p.n_mblk) * groups * ranks);
    p.dq_ctas = (int)(p.tiles * groups * p.parts);
    cudaError_t e = launch_ex(true, ckpt_stats_tc_kernel<D>, dim3((unsigned)p.dq_ctas), dim3(kThreads), DqCfg<D>::SMEM, a.stream,
                              mq, mdo, mkc, mvc, mk, mv, p);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.dkdv_ctas + (p.dq_ctas + ranks - 1) / ranks * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kGradSmem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, ckpt_grad_tc_kernel<D>, mq, mdo, mkc, mvc, mk, mv, p);
    if (e != cudaSuccess || p.parts == 1) return e;
    return launch_ex(true, ckpt_dq_combine_kernel<D>, dim3((unsigned)(p.tiles * groups * 4)), dim3(256), 0, a.stream, p);
}

}  // namespace

size_t ckpt_stats_floats(const CkptBwdArgs& a) {
    const int groups = a.B * a.Hkv, tiles = dq_tiles(a.Hq, a.Hkv, a.T);
    // parts exist where they and the tiles are at most num_sms
    return std::max((size_t)a.B * a.Hq * a.T * 4, (size_t)groups * tiles * 128 * 2) + (size_t)a.num_sms * 128 * (4 + a.d);
}

cudaError_t launch_ckpt_backward_tc(const CkptBwdArgs& a) {
    return a.d == 64 ? backward_launch<64>(a) : backward_launch<128>(a);
}

}  // namespace h2o
