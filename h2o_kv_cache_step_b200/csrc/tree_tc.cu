// tree_tc.cu -- tensor-core (tcgen05 + TMEM + TMA) attention of a tree of drafted
// tokens over the cache (bf16; the formulas are tree.cu's).
//
// The query rows of a KV head, R = G T of them (row = head-in-group * T + node),
// are cut into 128-row tiles and the keys into 128-key blocks: the cache's first,
// the drafted nodes' last. A unit is a pair of tiles with all blocks of its KV
// head. The blocks of all units form one line that is divided evenly over the
// SMs, one CTA each, so a CTA works on the end of one unit, whole units, and the
// start of another; a part of a unit leaves its unnormalised output, maximum and
// sum in fp32, and tree_combine_kernel merges the parts in order. Where it costs no
// more blocks, a unit's CTAs are a cluster, keep their parts in shared memory and merge
// them there.
//
// Per block and tile: S = Q K^T in TMEM; two threads per row take 64 columns each
// into registers, exchange their maxima, and write P = 2^(s - m) back over S as
// bf16, the A operand of O += P V (also in TMEM). The running maximum m moves, and
// O is rescaled, only when it grows by more than 2^16. A tile's products wait for
// its softmax, so two tiles share a CTA and every K and V block: one's products
// run during the other's softmax. Twenty warps: a TMA loader, an MMA issuer, two
// softmax warpgroups per tile and two warps for the masks.
//
// A row's visible nodes are a bit mask of its ancestors, built in shared memory by
// pointer jumping (each round a node takes the mask of the node it points to and
// points where that one does: 8 rounds for 256 nodes), by warps of their own while
// the cache's blocks are worked on. Keys outside the mask get
// weight zero; a NaN or an infinity in a drafted v is zeroed in shared memory,
// because zero times it is not zero, and at the end added to its column of the rows
// that see it.
// Rows past the end of a cache, of the nodes or of a KV head's queries arrive as
// zeros (3-D tensor maps).
//
// P is rounded to bf16, the MMA's operand type, as in the step that commits the accepted
// path and whose rows these are compared with; maxima, sums and outputs stay in fp32
// until the end. The output's error against 64 bits is then 1.4 times that of its own
// rounding. P as a bf16 pair makes it 1.0, for one more product per tile and block, which
// the tensor core has no room for: 37.9 us a pass at T=61 B=4 C=4096 and 108 at T=256
// C=16384, against 32.7 and 87.5.
//
// Times of a pass are taken with inputs that change from pass to pass, others with the
// inputs in L2 and the clock not yet held down by power (T=256 C=16384: 86.6 and 81.8).
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

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

// P may exceed 1 by up to 2^16 before the running maximum moves: bf16 has fp32's
// exponents, and O and the sum are fp32.
constexpr float kRescale = 16.f;
constexpr int kUnitRows = 256;
constexpr int kMaxCluster = 8;

template <int D>
struct TreeCfg {
    static constexpr int HALF = 128 * 128;  // 128 rows x 64 bf16
    static constexpr int TILE = 128 * D * 2;
    static constexpr int RING = 4;          // K / V slots, loaded K0, V0, K1, V1, ...
    static constexpr int OFF_Q = 0;         // [2 tiles]
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_MASK = OFF_RING + RING * TILE;                  // [256][8] words
    static constexpr int OFF_PTR = OFF_MASK + kTreeMaxT * kTreeMaskWords * 4;  // [256]
    static constexpr int OFF_BAD = OFF_PTR + kTreeMaxT * 4;                  // word
    static constexpr int OFF_MAX = OFF_BAD + 32;                             // [2 tiles][2 blocks][2 halves][128] floats
    static constexpr int OFF_BAR = OFF_MAX + 2 * 2 * 2 * 128 * 4;
    static constexpr int NBAR = 28;
    static constexpr int SMEM_RAW = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int SMEM = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;  // one CTA (512 TMEM columns) per SM
    static constexpr int THREADS = 640;
    static constexpr uint32_t IDESC_QK = tc::idesc_bf16_f32(128, 128, false);
    static constexpr uint32_t IDESC_PV = tc::idesc_bf16_f32(128, D, true);
};
static_assert(TreeCfg<128>::SMEM_RAW <= 232448, "tree attention shared memory exceeds the per-CTA limit");

// CTA c's share of the line: runs of `run` blocks (the whole line, or one unit) are
// divided among k CTAs each, q blocks a CTA, one more for the first `extra`.
struct Split {
    int run, k, q, extra;
    __host__ __device__ int first(int c) const {
        const int i = c % k;
        return c / k * run + i * q + (i < extra ? i : extra);
    }
    __host__ __device__ int owner(int w) const {
        const int r = w % run, big = extra * (q + 1);
        return w / run * k + (r < big ? r / (q + 1) : extra + (r - big) / q);
    }
};

struct TreeParams {
    int Hkv, T, n, R;   // R: query rows per KV head
    int pairs;          // units per KV head
    int nbc, nb;        // cache blocks, blocks per unit
    Split split;        // of the blocks of all units
    float scale_log2;
    const int32_t* parent;
    const __nv_bfloat16* v;  // of the nodes
    __nv_bfloat16* out;
    float* lse;
    float4* part_o;  // [2 CTAs][D / 4][256]: four columns of a row together, rows next to each other
    unsigned* count; // [KV heads], zero: CTAs that have left their part (nullptr: merged by a kernel of its own)
    float2* part_ml; // [2 CTAs][256]: log2-domain maximum (NaN: the row's node is absent) and sum
    int cluster;     // > 0: a unit's CTAs, a cluster of as many, merge it in shared memory
    WaitBound wb;
};

// A CTA's next run of blocks of one unit.
struct Segment {
    int bg, m0, rows;   // KV head, first row, rows of the unit
    int j0, j1;         // blocks
    bool hasB, whole, first;
};
__device__ __forceinline__ Segment segment(const TreeParams& p, int w, int w0, int w1) {
    Segment s;
    const int unit = w / p.nb;
    s.j0 = w - unit * p.nb;
    s.j1 = min(p.nb, s.j0 + (w1 - w));
    s.bg = unit / p.pairs;
    s.m0 = unit % p.pairs * kUnitRows;
    s.rows = min(kUnitRows, p.R - s.m0);
    s.hasB = s.rows > 128;
    s.whole = s.j0 == 0 && s.j1 == p.nb;
    s.first = w == w0;
    return s;
}

// Four columns of a row of KV head bg from the parts that the CTAs left: with the
// parts' maxima m and sums l, M = max m, L = sum l 2^(m - M),
// O = sum 2^(m - M) O_part / L, in the order of the parts.
template <int D>
__device__ __forceinline__ void merge_row(const TreeParams& p, unsigned bg, int row, int col4) {
    const int b0 = (int)(bg * p.pairs + row / kUnitRows) * p.nb;
    const int c0 = p.split.owner(b0), c1 = p.split.owner(b0 + p.nb - 1);
    if (c0 == c1) return;  // written whole
    // where CTA c left its part: the unit is the first one of every CTA but, it may be, c0
    const bool second = p.split.first(c0) < b0;
    auto part = [&](int c) { return (size_t)(2 * c + (c == c0 && second ? 1 : 0)); };
    const int r = row % kUnitRows;
    constexpr int kBatch = 9;  // parts in flight: one after the other they cost an L2 latency each
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool absent = false;
    for (int c = c0; c <= c1; c += kBatch) {
        float2 ml[kBatch];
        float4 o[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const size_t at = part(min(c + u, c1));
            ml[u] = p.part_ml[at * kUnitRows + r];
            o[u] = p.part_o[(at * (D / 4) + col4) * kUnitRows + r];
        }
        float Mn = M;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            absent |= ml[u].x != ml[u].x;
            Mn = fmaxf(Mn, ml[u].x);
        }
        const float ms = Mn == -INFINITY ? 0.f : Mn, a = ex2(M - ms);
        M = Mn;
        L *= a;
        acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (c + u > c1) continue;
            const float w = ex2(ml[u].x - ms);
            L = fmaf(ml[u].y, w, L);
            acc.x = fmaf(o[u].x, w, acc.x);
            acc.y = fmaf(o[u].y, w, acc.y);
            acc.z = fmaf(o[u].z, w, acc.z);
            acc.w = fmaf(o[u].w, w, acc.w);
        }
    }
    const float inv = 1.f / L;
    uint2 h = make_uint2(tc::pack_bf16(acc.x * inv, acc.y * inv), tc::pack_bf16(acc.z * inv, acc.w * inv));
    if (absent) h = make_uint2(0, 0);
    const size_t at = (size_t)bg * p.R + row;
    *reinterpret_cast<uint2*>(p.out + at * D + 4 * col4) = h;
    if (col4 == 0) p.lse[at] = absent ? -INFINITY : (M + log2f(L)) * kLn2;
}

// The same for a unit whose parts lie in the shared memory of a cluster: each CTA merges
// its share of the rows. `acc`, `ml`: shared addresses of a part's rows and of their
// maxima and sums.
template <int D>
__device__ __forceinline__ void merge_cluster(const TreeParams& p, const Segment& s, uint32_t acc, uint32_t ml) {
    constexpr int kLanes = D / 4, kPerWarp = 32 / kLanes;  // lanes per row, rows per warp
    const int rank = tc::cluster_rank(), warp = threadIdx.x / 32, lane = threadIdx.x % 32, c4 = lane % kLanes;
    const int end = s.rows * (rank + 1) / p.cluster;
    for (int r = s.rows * rank / p.cluster + warp * kPerWarp + lane / kLanes; r < end; r += TreeCfg<D>::THREADS / 32 * kPerWarp) {
        float2 x[kMaxCluster];
        float4 o[kMaxCluster];
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            if (q >= p.cluster) break;
            const float4 s4 = tc::cluster_load4(ml + 16 * r, q);
            x[q] = make_float2(s4.x, s4.y);
            o[q] = tc::cluster_load4(acc + (r * D + (c4 ^ (r & (kLanes - 1))) * 4) * 4, q);
        }
        float M = -INFINITY, L = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        bool absent = false;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            if (q >= p.cluster) break;
            absent |= x[q].x != x[q].x;
            M = fmaxf(M, x[q].x);
        }
        const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            if (q >= p.cluster) break;
            const float w = ex2(x[q].x - ms);
            L = fmaf(x[q].y, w, L);
            a = make_float4(fmaf(o[q].x, w, a.x), fmaf(o[q].y, w, a.y), fmaf(o[q].z, w, a.z), fmaf(o[q].w, w, a.w));
        }
        const float inv = 1.f / L;
        uint2 out = make_uint2(tc::pack_bf16(a.x * inv, a.y * inv), tc::pack_bf16(a.z * inv, a.w * inv));
        if (absent) out = make_uint2(0, 0);
        const size_t at = (size_t)s.bg * p.R + s.m0 + r;
        *reinterpret_cast<uint2*>(p.out + at * D + 4 * c4) = out;
        if (c4 == 0) p.lse[at] = absent ? -INFINITY : (M + log2f(L)) * kLn2;
    }
}

// What is not finite in v of the nodes that a row sees, of a CTA's segments, added to the
// row's output or part of it (weights are positive, so it is what the values' weighted
// sum comes to). Rare: a CTA that met such a value does this once its outputs are
// stored. `acc`: where a cluster's part lies.
template <int D>
__device__ __noinline__ void add_not_finite(const TreeParams& p, int w0, int w1, float* acc) {
    for (int w = w0; w < w1;) {
        const Segment s = segment(p, w, w0, w1);
        w += s.j1 - s.j0;
        const int lo = 128 * (s.j0 - p.nbc), hi = 128 * (s.j1 - p.nbc);  // its nodes
        if (hi <= 0) continue;
        const int32_t* parent = p.parent + (size_t)(s.bg / p.Hkv) * p.T;
        for (int e = threadIdx.x; e < s.rows * D; e += TreeCfg<D>::THREADS) {
            const int r = e / D, col = e % D;
            float sum = 0.f;
            bool any = false;
            int u = (s.m0 + r) % p.T;
            while (u >= 0) {
                const float x = __bfloat162float(p.v[((size_t)s.bg * p.T + u) * D + col]);
                if (u >= lo && u < hi && !isfinite(x)) {
                    sum += x;
                    any = true;
                }
                const int up = parent[u];
                u = up == -1 ? -1 : (up >= 0 && up < u) ? up : -2;
            }
            if (!any || u != -1) continue;  // an absent node's row stays zero
            if (p.cluster) {
                acc[r * D + ((col / 4) ^ (r & (D / 4 - 1))) * 4 + col % 4] += sum;
            } else if (s.whole) {
                __nv_bfloat16* out = p.out + ((size_t)s.bg * p.R + s.m0 + r) * D + col;
                *out = __float2bfloat16_rn(__bfloat162float(*out) + sum);
            } else {
                const size_t part = 2 * blockIdx.x + (s.first ? 0 : 1);
                reinterpret_cast<float*>(p.part_o + (part * (D / 4) + col / 4) * kUnitRows + r)[col % 4] += sum;
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kc,
               const __grid_constant__ CUtensorMap map_vc, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TreeParams p) {
    using Cfg = TreeCfg<D>;
    constexpr int RING = Cfg::RING;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* q_full = bars;
    uint64_t* q_empty = bars + 1;              // the segment's products have read Q
    uint64_t* ring_full = bars + 2;            // [RING]
    uint64_t* ring_empty = ring_full + RING;   // [RING]
    uint64_t* s_full = ring_empty + RING;      // [2 tiles]; O of the blocks before is complete too
    uint64_t* p_full = s_full + 2;             // [2 tiles], 8 arrivals: P over S, O rescaled
    uint64_t* o_full = p_full + 2;             // [2 tiles]: O of a segment
    uint64_t* v_ok = o_full + 2;               // [2], 4 arrivals: a node block's V is finite
    uint64_t* mask_full = v_ok + 2;            // 2 arrivals: the masks of a segment's nodes
    uint64_t* mask_free = mask_full + 1;       // 16 arrivals: no longer needed
    uint64_t* drain = mask_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int w0 = p.split.first(blockIdx.x), w1 = p.split.first(blockIdx.x + 1);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < RING; ++s) {
            mbar_init(ring_full + s, 1);
            mbar_init(ring_empty + s, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + t, 1);
            mbar_init(p_full + t, 8);
            mbar_init(o_full + t, 1);
            mbar_init(v_ok + t, 4);
        }
        mbar_init(mask_full, 2);
        mbar_init(mask_free, 16);
        mbar_init(drain, 1);
        *abort_flag = 0;
        *reinterpret_cast<uint32_t*>(smem + Cfg::OFF_BAD) = 0;
        fence_mbar_init();
    }
    uint32_t tmem = 0;  // tile X: S at 256 X, O at 256 X + 128
    if (warp == 0) {
        // the loader has initialised the barriers and needs nothing else: its first loads
        // are on their way while the others set up
        __syncwarp();
        tc::named_arrive(4, Cfg::THREADS);
    } else {
        if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
        fence_before_sync();
        tc::named_sync(4, Cfg::THREADS);
        fence_after_sync();
        tmem = *tmem_slot;
    }
    const uint32_t sbase = smem_u32(smem);
    griddep_wait();  // the work before is complete; what follows may set up
    griddep_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            int L = 0, q = 0;
            bool ok = true;
            for (int w = w0; ok && w < w1; ++q) {
                const Segment s = segment(p, w, w0, w1);
                w += s.j1 - s.j0;
                if (!(ok = wait_bar(q_empty, (q & 1) ^ 1, p.wb, kDevTimeoutSlotWait, abort_flag))) break;
                mbar_arrive_expect_tx(q_full, Cfg::TILE * (s.hasB ? 2 : 1));
                for (int x = 0; x < (s.hasB ? 2 : 1); ++x)
                    for (int hh = 0; hh < D / 64; ++hh)
                        tc::tma_load_3d(smem + Cfg::OFF_Q + x * Cfg::TILE + hh * Cfg::HALF, &map_q, 64 * hh, s.m0 + 128 * x, s.bg,
                                        q_full);
                for (int j = s.j0; ok && j < s.j1; ++j) {
                    const bool cache = j < p.nbc;
                    const int row = 128 * (cache ? j : j - p.nbc);
                    for (int kv = 0; kv < 2; ++kv, ++L) {
                        const int slot = L % RING;
                        if (!(ok = wait_bar(ring_empty + slot, ((L / RING) & 1) ^ 1, p.wb, kDevTimeoutSlotWait, abort_flag)))
                            break;
                        const CUtensorMap* map = kv ? (cache ? &map_vc : &map_v) : (cache ? &map_kc : &map_k);
                        mbar_arrive_expect_tx(ring_full + slot, Cfg::TILE);
                        for (int hh = 0; hh < D / 64; ++hh)
                            tc::tma_load_3d(smem + Cfg::OFF_RING + slot * Cfg::TILE + hh * Cfg::HALF, map, 64 * hh, row, s.bg,
                                            ring_full + slot);
                    }
                }
                if (!ok) ++q;  // its Q load was issued
                if (!ok) break;
            }
            // every load issued here has landed before the CTA may exit
            if (q) wait_bar(q_full, (q - 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
            for (int s = 0; s < RING; ++s) {
                const int uses = L / RING + (s < L % RING ? 1 : 0);
                if (uses) wait_bar(ring_full + s, (uses - 1) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
            }
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMA issuer
        // One warp for both tiles, so that the tensor core takes a tile's PV(j) and
        // QK(j + 1) together and then the other's: the two stay out of step, one in its
        // softmax while the other has the tensor core. With an issuer per tile their
        // products interleave, both wait and then both take exponentials (98 us at 256
        // nodes and 16384 slots, against 83 then).
        const uint64_t dQ = desc_kmajor_sw128(sbase + Cfg::OFF_Q);
        const uint64_t dRingK = desc_kmajor_sw128(sbase + Cfg::OFF_RING);
        const uint64_t dRingV = desc_mnmajor_sw128(sbase + Cfg::OFF_RING, Cfg::HALF);
        int L = 0, q = 0, tb = 0, blocks[2] = {0, 0};  // ring loads, segments, node blocks, blocks of a tile
        auto wait_ring = [&](int& slot) {
            slot = L % RING;
            const bool r = warp_wait(ring_full + slot, (L / RING) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
            ++L;
            return r;
        };
        auto issue_qk = [&](int X, int slot) {
            const uint64_t a = dQ + (uint64_t)((X * Cfg::TILE) >> 4), b = dRingK + (uint64_t)((slot * Cfg::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * Cfg::HALF + (kk & 3) * 32) >> 4;
                tc::mma_bf16_ss_warp(tmem + 256 * X, a + off, b + off, Cfg::IDESC_QK, kk > 0);
            }
            tc::mma_commit_warp(s_full + X);
        };
        auto issue_pv = [&](int X, int slot, bool first) {
            const uint32_t tS = tmem + 256 * X;
            const uint64_t b = dRingV + (uint64_t)((slot * Cfg::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 keys per instruction; the keys' halves at columns 0 and 64
                tc::mma_bf16_ts_warp(tS + 128, tS + 64 * (kk >> 2) + 8 * (kk & 3), b + (uint64_t)((kk * 16 * 128) >> 4),
                                     Cfg::IDESC_PV, (!first || kk > 0) ? 1u : 0u);
        };
        bool ok = true;
        for (int w = w0; ok && w < w1; ++q) {
            const Segment s = segment(p, w, w0, w1);
            w += s.j1 - s.j0;
            const int tiles = s.hasB ? 2 : 1;
            int ks = 0, vs = 0;
            if (!(ok = warp_wait(q_full, q & 1, p.wb, kDevTimeoutTmaWait, abort_flag) && wait_ring(ks))) break;
            fence_after_sync();
            for (int X = 0; X < tiles; ++X) issue_qk(X, ks);
            tc::mma_commit_warp(ring_empty + ks);
            for (int j = s.j0; j < s.j1; ++j) {
                const bool more = j + 1 < s.j1;
                ok = wait_ring(vs);
                if (ok && j >= p.nbc) {
                    ok = warp_wait(v_ok + (tb & 1), (tb >> 1) & 1, p.wb, kDevTimeoutMmaWait, abort_flag);
                    ++tb;
                }
                if (ok && more) ok = wait_ring(ks);
                for (int X = 0; ok && X < tiles; ++X) {
                    if (!(ok = warp_wait(p_full + X, blocks[X] & 1, p.wb, kDevTimeoutMmaWait, abort_flag))) break;
                    ++blocks[X];
                    fence_after_sync();
                    issue_pv(X, vs, j == s.j0);
                    // S: the softmax took its last row out before it handed P over, and the
                    // product that reads that P is ahead of this one
                    if (more) issue_qk(X, ks);
                    else tc::mma_commit_warp(o_full + X);
                }
                if (!ok) break;
                tc::mma_commit_warp(ring_empty + vs);
                if (more) tc::mma_commit_warp(ring_empty + ks);
            }
            if (ok) tc::mma_commit_warp(q_empty);
        }
        // all MMAs issued here complete before TMEM can be released
        tc::mma_commit_warp(drain);
        __syncwarp();
        warp_wait(drain, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
    } else if (warp >= 18) {
        // ------------------------------------------------------------ node masks
        // (a give-up goes on without waiting: both warps join every barrier)
        const int t = threadIdx.x - 18 * 32;  // nodes t, t + 64, t + 128, t + 192
        uint32_t* mask = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MASK);
        int* ptr = reinterpret_cast<int*>(smem + Cfg::OFF_PTR);
        int built = 0;
        bool ok = true;
        for (int w = w0; w < w1;) {
            const Segment s = segment(p, w, w0, w1);
            w += s.j1 - s.j0;
            if (s.j1 <= p.nbc) continue;
            uint32_t mw[4][kTreeMaskWords];
            int to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = t + 64 * u;
                to[u] = -2;
                if (i < p.T) {
                    const int up = p.parent[(size_t)(s.bg / p.Hkv) * p.T + i];
                    to[u] = up == -1 ? -1 : (up >= 0 && up < i) ? up : -2;
                }
#pragma unroll
                for (int k = 0; k < kTreeMaskWords; ++k) mw[u][k] = (i >> 5) == k ? 1u << (i & 31) : 0u;
            }
            if (ok) ok = warp_wait(mask_free, (built & 1) ^ 1, p.wb, kDevTimeoutSlotWait, abort_flag);
            ++built;
            for (int span = 1;; span *= 2) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = t + 64 * u;
                    if (i >= p.T) continue;
                    ptr[i] = to[u];
                    uint4* own = reinterpret_cast<uint4*>(mask + i * kTreeMaskWords);
                    own[0] = make_uint4(mw[u][0], mw[u][1], mw[u][2], mw[u][3]);
                    own[1] = make_uint4(mw[u][4], mw[u][5], mw[u][6], mw[u][7]);
                }
                tc::named_sync(3, 64);
                if (span >= p.T) break;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (to[u] < 0) continue;
                    const uint4* from = reinterpret_cast<const uint4*>(mask + to[u] * kTreeMaskWords);
                    const uint4 a = from[0], e = from[1];
                    mw[u][0] |= a.x;
                    mw[u][1] |= a.y;
                    mw[u][2] |= a.z;
                    mw[u][3] |= a.w;
                    mw[u][4] |= e.x;
                    mw[u][5] |= e.y;
                    mw[u][6] |= e.z;
                    mw[u][7] |= e.w;
                    to[u] = ptr[to[u]];
                }
                tc::named_sync(3, 64);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(mask_full);
        }
    } else {
        // -------------------------------------------------------------- softmax
        // A warp that gives up a wait goes on without waiting: every warp joins every
        // named barrier.
        const int X = warp < 10 ? 0 : 1, h = (warp - 2) >> 2 & 1;  // tile, half of the columns
        const int quad = warp & 3;
        const int r = quad * 32 + lane;  // row inside the tile = TMEM lane
        const uint32_t tX = tmem + 256 * X + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = tX + 64 * h, tO = tX + 128 + h * (D / 2);  // this thread's columns of S (and P) and O
        const uint32_t* mask = reinterpret_cast<const uint32_t*>(smem + Cfg::OFF_MASK);
        const int* ptr = reinterpret_cast<const int*>(smem + Cfg::OFF_PTR);
        float* xmax = reinterpret_cast<float*>(smem + Cfg::OFF_MAX) + X * 512 + r;
        int L = 0, c = 0, tb = 0, done = 0, masks = 0;  // ring loads, blocks of this tile, node blocks, segments of this tile, with nodes
        bool ok = true;
        for (int w = w0; w < w1;) {
            const Segment s = segment(p, w, w0, w1);
            w += s.j1 - s.j0;
            const int tree_blocks = max(0, s.j1 - max(s.j0, p.nbc));
            if (X == 1 && !s.hasB) {
                L += 2 * (s.j1 - s.j0);
                tb += tree_blocks;
                masks += tree_blocks > 0;
                continue;
            }
            const int row = s.m0 + 128 * X + r;                  // of the KV head
            const bool busy = s.m0 + 128 * X + 32 * quad < p.R;  // the warp has rows
            const int node = row % p.T;
            bool absent = false;
            float m = -INFINITY, l = 0.f;
            for (int j = s.j0; j < s.j1; ++j, ++c, L += 2) {
                uint32_t vis[2] = {~0u, ~0u};  // of this thread's columns
                const bool nodes = j >= p.nbc, masked = nodes || p.n - 128 * j < 128;
                if (nodes && X == 0 && h == 0) {
                    // V of the nodes: what is not finite becomes zero
                    const int slot = (L + 1) % RING;
                    if (ok) ok = warp_wait(ring_full + slot, ((L + 1) / RING) & 1, p.wb, kDevTimeoutTmaWait, abort_flag);
                    uint8_t* vt = smem + Cfg::OFF_RING + slot * Cfg::TILE + r * 128;
                    uint32_t over = 0;
#pragma unroll 4
                    for (int x = 0; x < D / 8; ++x) {
                        const uint4 v4 = *reinterpret_cast<const uint4*>(vt + (x >> 3) * Cfg::HALF + (((x & 7) ^ (r & 7)) << 4));
                        const uint32_t u[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            over |= (uint32_t)((u[k] & 0x7f80u) == 0x7f80u) | (uint32_t)((u[k] & 0x7f800000u) == 0x7f800000u);
                    }
                    if (over) {
#pragma unroll 1
                        for (int x = 0; x < D / 2; ++x) {
                            uint32_t* u = reinterpret_cast<uint32_t*>(vt + (x >> 5) * Cfg::HALF) + (x & 31);
                            if ((*u & 0x7f80u) == 0x7f80u) *u &= 0xffff0000u;
                            if ((*u & 0x7f800000u) == 0x7f800000u) *u &= 0xffffu;
                        }
                        *reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_BAD) = 1;
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_ok + (tb & 1));
                }
                if (ok) ok = warp_wait(s_full + X, c & 1, p.wb, kDevTimeoutMmaWait, abort_flag);
                if (nodes) {
                    if (ok) ok = warp_wait(mask_full, masks & 1, p.wb, kDevTimeoutSlotWait, abort_flag);
                    absent = ptr[node] != -1;
                    const uint32_t* mk = mask + node * kTreeMaskWords + 4 * (j - p.nbc);
                    vis[0] = mk[2 * h];
                    vis[1] = mk[2 * h + 1];
                    ++tb;
                } else if (masked) {
                    const int limit = p.n - 128 * j - 64 * h;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        vis[k] = limit >= 32 * k + 32 ? ~0u : limit <= 32 * k ? 0u : (1u << (limit - 32 * k)) - 1;
                }
                fence_after_sync();
                float* xm = xmax + (c & 1) * 256;
                if (!busy) {  // P of rows that nobody reads: whatever S holds
                    tc::named_sync(1 + X, 256);
                    if (lane == 0) mbar_arrive(p_full + X);
                    continue;
                }
                uint32_t v[2][32];
                tc::tmem_ld32(tS, v[0]);
                tc::tmem_ld32(tS + 32, v[1]);
                tc::tmem_ld_wait();
                tc::reg_fence(v[0]);
                tc::reg_fence(v[1]);
                if (masked) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((vis[k] >> e) & 1u)) v[k][e] = __float_as_uint(-INFINITY);
                }
                float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        mx0 = tc::max3(mx0, __uint_as_float(v[k][e]), __uint_as_float(v[k][e + 1]));
                        mx1 = tc::max3(mx1, __uint_as_float(v[k][e + 2]), __uint_as_float(v[k][e + 3]));
                    }
                mx0 = fmaxf(mx0, mx1);
                xm[128 * h] = mx0;
                tc::named_sync(1 + X, 256);
                const float m_new = fmaxf(m, fmaxf(mx0, xm[128 - 128 * h]) * p.scale_log2);
                const bool resc = m_new > m + kRescale;
                const float m_use = resc ? m_new : m;
                const float alpha = resc ? ex2(m - m_use) : 1.f;
                if (j > s.j0 && __any_sync(0xffffffffu, resc)) {
                    // O of the blocks before is complete: their products were issued before
                    // this S, and the next one waits for this P
#pragma unroll 1
                    for (int x = 0; x < D / 2; x += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16(tO + x, o);
                        tc::tmem_ld_wait();
                        tc::reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc::tmem_st16(tO + x, o);
                    }
                }
                const float ms = m_use == -INFINITY ? 0.f : m_use;  // the row sees no key yet
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-ms, -ms);
                float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // a NaN or +inf score makes its P and the sum NaN
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float2 x = tc::ffma2(make_float2(__uint_as_float(v[k][e]), __uint_as_float(v[k][e + 1])), sc2, nm2);
                        const float2 y = tc::ffma2(make_float2(__uint_as_float(v[k][e + 2]), __uint_as_float(v[k][e + 3])), sc2, nm2);
                        const float2 a = make_float2(ex2(x.x), ex2(x.y)), b = make_float2(ex2(y.x), ex2(y.y));
                        acc0 = tc::fadd2(acc0, a);
                        acc1 = tc::fadd2(acc1, b);
                        pk[e >> 1] = tc::pack_bf16(a.x, a.y);
                        pk[(e >> 1) + 1] = tc::pack_bf16(b.x, b.y);
                    }
                    tc::tmem_st16(tS + 16 * k, pk);
                }
                tc::tmem_st_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + X);
                l = fmaf(l, alpha, (acc0.x + acc0.y) + (acc1.x + acc1.y));
                m = m_use;
            }
            if (tree_blocks) {
                ++masks;
                __syncwarp();
                if (lane == 0) {  // for the tile that sits out, too
                    mbar_arrive(mask_free);
                    if (!s.hasB) mbar_arrive(mask_free);
                }
            }
            // ---------------------------------------------------------- epilogue
            // the halves' sums meet, in the buffer that the last block's maxima are not in
            float* xl = xmax + (c & 1) * 256;
            xl[128 * h] = l;
            tc::named_sync(1 + X, 256);
            l += xl[128 - 128 * h];
            tc::named_sync(1 + X, 256);
            if (ok) ok = warp_wait(o_full + X, done++ & 1, p.wb, kDevTimeoutMmaWait, abort_flag);
            // the other tile's products too: what follows overwrites their operands
            if (p.cluster && s.hasB && ok) ok = warp_wait(o_full + 1 - X, 0, p.wb, kDevTimeoutMmaWait, abort_flag);
            fence_after_sync();
            if (p.cluster) {
                if (busy && ok) {
                    // to shared memory, 16-byte chunks of a row permuted by the row, so that
                    // neither these stores nor the merge's loads meet in a bank
                    float* acc = reinterpret_cast<float*>(smem + Cfg::OFF_RING) + (128 * X + r) * D;
#pragma unroll 1
                    for (int x = 0; x < D / 2; x += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16(tO + x, o);
                        tc::tmem_ld_wait();
                        tc::reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const int chunk = (h * (D / 2) + x + e) / 4;
                            *reinterpret_cast<uint4*>(acc + (chunk ^ (r & (D / 4 - 1))) * 4) =
                                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                    if (h == 0)
                        reinterpret_cast<float4*>(smem + Cfg::OFF_Q)[128 * X + r] =
                            make_float4(absent ? __uint_as_float(0x7fffffffu) : m, l, 0.f, 0.f);
                }
            } else if (busy && ok) {
                const float nan = __uint_as_float(0x7fffffffu);
                const bool row_ok = row < p.R;
                const size_t part = 2 * blockIdx.x + (s.first ? 0 : 1);
                const size_t at = (size_t)s.bg * p.R + row;
                const float f = s.whole ? 1.f / l : 1.f;
#pragma unroll 1
                for (int x = 0; x < D / 2; x += 16) {
                    uint32_t o[16];
                    tc::tmem_ld16(tO + x, o);
                    tc::tmem_ld_wait();
                    tc::reg_fence(o);
                    if (!row_ok) continue;
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    const int col = h * (D / 2) + x;
                    if (!s.whole) {
                        float4* dst = p.part_o + (part * (D / 4) + col / 4) * kUnitRows + 128 * X + r;
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            dst[(e >> 2) * kUnitRows] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                    __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = absent ? 0u : tc::pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                        uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + col);
                        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                if (row_ok && h == 0) {
                    if (!s.whole)
                        p.part_ml[part * kUnitRows + 128 * X + r] = make_float2(absent ? nan : m, l);
                    else
                        p.lse[at] = absent ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            }
            fence_before_sync();
        }
    }
    fence_before_sync();
    __syncthreads();
    if (*reinterpret_cast<const volatile uint32_t*>(smem + Cfg::OFF_BAD)) {
        add_not_finite<D>(p, w0, w1, reinterpret_cast<float*>(smem + Cfg::OFF_RING));
        __syncthreads();
    }
    if (p.cluster) {
        __syncwarp();
        tc::cluster_sync();
    }
    if (warp == 1) {
        fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
    if (p.cluster) {
        merge_cluster<D>(p, segment(p, w0, w0, w1), sbase + Cfg::OFF_RING, sbase + Cfg::OFF_Q);
        tc::cluster_sync();  // no CTA leaves while another reads its part
    } else if (p.count && w1 - w0 < p.nb) {
        // few rows: the unit's last CTA merges, which spares a launch
        const unsigned bg = w0 / p.nb;  // a unit per KV head
        unsigned* flag = reinterpret_cast<unsigned*>(smem + Cfg::OFF_MAX);
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            const unsigned before = atomicAdd(p.count + bg, 1u);
            *flag = before == (unsigned)p.split.k - 1;
            if (*flag) p.count[bg] = 0;
        }
        __syncthreads();
        if (*flag) {
            __threadfence();
            for (int e = threadIdx.x; e < p.R * (D / 4); e += Cfg::THREADS) merge_row<D>(p, bg, e % p.R, e / p.R);
        }
    }
}

// Merges the units that were divided, but those that their last CTA merged. One
// thread per four columns of a row; a block takes 1024 / D consecutive rows,
// neighbouring lanes neighbouring rows, as the parts lie.
template <int D>
__global__ void __launch_bounds__(256)
tree_combine_kernel(const TreeParams p, unsigned rows) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr unsigned kRows = 1024 / D;
    const unsigned g = blockIdx.x * kRows + threadIdx.x % kRows;
    if (g < rows) merge_row<D>(p, g / (unsigned)p.R, (int)(g % (unsigned)p.R), threadIdx.x / kRows);
}

// Clusters of k CTAs that can be on the device at once (an SM takes one CTA, and a
// cluster stays inside one part of the device).
template <int D>
cudaError_t clusters_at_once(int k, int* clusters) {
    static std::mutex mu;
    static std::map<std::pair<int, int>, int> known;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    const auto at = known.find({dev, k});
    if (at != known.end()) {
        *clusters = at->second;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(k);
    cfg.blockDim = dim3(TreeCfg<D>::THREADS);
    cfg.dynamicSmemBytes = TreeCfg<D>::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = k;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaError_t e = cudaOccupancyMaxActiveClusters(clusters, tree_tc_kernel<D>, &cfg); e != cudaSuccess) return e;
    known[{dev, k}] = *clusters;
    return cudaSuccess;
}

template <int D>
cudaError_t tree_launch(const TreeArgs& a) {
    using Cfg = TreeCfg<D>;
    if (cudaError_t e = ensure_smem_limit(tree_tc_kernel<D>, Cfg::SMEM); e != cudaSuccess) return e;
    CUtensorMap mq, mkc, mvc, mk, mv;
    const uint64_t groups = (uint64_t)a.B * a.Hkv;
    const int R = a.Hq / a.Hkv * a.T;
    const uint64_t n = a.n > 0 ? a.n : 1;  // an empty cache is never loaded from
    if (!tc_make_map3(&mq, a.q, R, groups, R, D, 128) || !tc_make_map3(&mkc, a.Kc, n, groups, a.C, D, 128) ||
        !tc_make_map3(&mvc, a.Vc, n, groups, a.C, D, 128) || !tc_make_map3(&mk, a.k, a.T, groups, a.T, D, 128) ||
        !tc_make_map3(&mv, a.v, a.T, groups, a.T, D, 128))
        return cudaErrorInvalidValue;
    TreeParams p;
    p.Hkv = a.Hkv;
    p.T = a.T;
    p.n = a.n;
    p.R = R;
    p.pairs = (R + kUnitRows - 1) / kUnitRows;
    p.nbc = (a.n + 127) / 128;
    p.nb = p.nbc + (a.T + 127) / 128;
    const long long total = (long long)groups * p.pairs * p.nb;
    if (total >= 1ll << 31) return cudaErrorInvalidValue;  // a cache of this many blocks does not fit the card
    // The line is divided evenly, or every unit among the same number of CTAs: then
    // fewer CTAs may work, but each leaves one part where most leave two; or among a
    // cluster, whose CTAs merge their parts in shared memory. A part that goes through
    // memory costs about as much as kPartBlocks blocks (its stores, and the merge of it).
    // Measured, evenly, by unit, by clusters, 32 / 8 heads, d = 128 unless given: 41.2,
    // 37.1 and 32.7 us a pass at T=61 B=4 C=4096; 91.4, 91.0 and 86.6 at T=256 C=16384.
    // With inputs in L2: 28.6, 24.5 and 22.7 at T=100 B=2 C=2048; 40.4, 30.6 and 30.6 at
    // T=256 C=8192, 16 / 4 heads; 44.1, 40.1 and 40.2 at T=128 C=16384, d = 64.
    constexpr int kPartBlocks = 2;
    const int units = (int)(total / p.nb), most = std::min(a.num_sms / units, p.nb);
    int k = 0, cost = (int)((total + a.num_sms - 1) / a.num_sms) + 2 * kPartBlocks;  // 0: evenly
    if (most >= 1 && (p.nb + most - 1) / most + kPartBlocks <= cost) {
        k = most;
        cost = (p.nb + most - 1) / most + kPartBlocks * (most > 1);
    }
    p.cluster = 0;
    for (int c = std::min(most, kMaxCluster); c > 1 && (p.nb + c - 1) / c <= cost; --c) {
        int fit = 0;  // all at once, or the last clusters would wait for the first
        if (cudaError_t e = clusters_at_once<D>(c, &fit); e != cudaSuccess) return e;
        if (units > fit) continue;
        k = p.cluster = c;
        break;
    }
    const bool by_unit = k > 0;
    const int ctas = by_unit ? units * k : (int)std::min<long long>(a.num_sms, total);
    p.split.run = by_unit ? p.nb : (int)total;
    p.split.k = by_unit ? k : ctas;
    p.split.q = p.split.run / p.split.k;
    p.split.extra = p.split.run % p.split.k;
    p.scale_log2 = kLog2e / sqrtf((float)D);
    p.parent = a.parent;
    p.v = static_cast<const __nv_bfloat16*>(a.v);
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.part_o = reinterpret_cast<float4*>(a.part);
    p.part_ml = reinterpret_cast<float2*>(a.part + (size_t)2 * a.num_sms * kUnitRows * D);
    p.wb = a.wb;
    // Up to kMergeRows rows per KV head are merged by the unit's last CTA, where that is
    // shorter than a kernel's launch. Measured, by the CTA and by a kernel, inputs in L2:
    // 4 rows, C = 9000: 17.5 us and 18.0, C = 16384: 24.0 and 24.3; 8 rows, C = 9000: 17.4
    // and 18.2; 32 rows, C = 16384: 26.2 to 30.4 and 25.3 to 30.0 (d = 64: 21.4 and 22.6);
    // 48 rows: 31.6 and 27.5; 64 rows, d = 64: 24.3 and 23.6.
    constexpr int kMergeRows = 32;
    p.count = by_unit && R <= kMergeRows && !p.cluster ? a.count : nullptr;
    if (p.cluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(Cfg::THREADS);
        cfg.dynamicSmemBytes = Cfg::SMEM;
        cfg.stream = a.stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = k;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, tree_tc_kernel<D>, mq, mkc, mvc, mk, mv, p);
    }
    cudaError_t e = launch_ex(true, tree_tc_kernel<D>, dim3(ctas), dim3(Cfg::THREADS), Cfg::SMEM, a.stream, mq, mkc, mvc, mk, mv, p);
    if (e != cudaSuccess) return e;
    bool divided = false;
    for (int c = 1; c < ctas && !divided; ++c) divided = p.split.first(c) % p.nb != 0;
    if (!divided || p.count) return cudaSuccess;
    const unsigned rows = (unsigned)(groups * R);  // a [B,Hq,T,d] tensor of 2^32 rows does not fit the card
    return launch_ex(true, tree_combine_kernel<D>, dim3((rows + 1024 / D - 1) / (1024 / D)), dim3(256), 0, a.stream, p, rows);
}

}  // namespace

size_t tree_part_floats(int num_sms, int d) { return (size_t)2 * num_sms * kUnitRows * (d + 2); }

cudaError_t launch_tree_tc(const TreeArgs& a) { return a.d == 64 ? tree_launch<64>(a) : tree_launch<128>(a); }

}  // namespace h2o
