// checkpoint.cu -- a step's inputs kept in 8 bits, and the gradient of the cache
// carried through the eviction.
//
// Record: with a = max |x| over 32 consecutive channels of a row,
//   code = rint(127 x / a) (ties to even), scale = a / 127 rounded to fp32,
// and the value it stands for is code * scale, rounded to the element type. A
// group of zeros has scale 0; a group with a NaN or an infinity has scale NaN
// and stands for NaNs. The quotient decides the code, so it is taken where its
// rounding cannot move it across a border k + 1/2: 127 x is exact in fp32 for a
// bf16 x, and 254 x - (2k + 1) a is a whole number of units of the last place of
// two 8-bit significands, so an fp32 quotient (24 bits) falls on the real
// quotient's side; fp32 inputs take the quotient in 64 bits for the same reason.
//
// Both directions are bound by memory: each value is read and written once.
#include <math.h>

#include "operators.h"
#include "vec.cuh"

namespace h2o {
namespace {

constexpr int kThreads = 256;

// The five sections of a record in order, as row counts and first rows.
struct Sections {
    unsigned long long end[5];  // first row after the section (record rows)
    int block_end[5];           // first block after the section
};

__device__ __forceinline__ int section_of(const Sections& s, int block) {
    int k = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) k += block >= s.block_end[i];
    return k;
}

struct CkptPtrs {
    void* x[5];
};

template <typename E>
struct Chunk;  // 16 bytes of values
template <>
struct Chunk<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float code(float x, float a) { return (float)rint(127.0 * (double)x / (double)a); }
};
template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    // 127 x would overflow from 2^121 on: there both sides are scaled down first
    static __device__ __forceinline__ float code(float x, float a) {
        const float f = a >= 0x1p120f ? 0x1p-8f : 1.f;
        return rintf(__fdiv_rn(127.f * (x * f), a * f));
    }
};

// Each thread codes 16 bytes of values; the threads of a group of 32 channels
// are neighbours in a warp.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
ckpt_save_kernel(CkptPtrs src, int8_t* __restrict__ codes, float* __restrict__ scales, Sections sec, int n, int pitch) {
    constexpr int N = Chunk<E>::N, PER_ROW = D / N, LANES = kCkptGroup / N;
    const int s = section_of(sec, blockIdx.x);
    const unsigned long long first = s ? sec.end[s - 1] : 0;
    const unsigned long long at = (unsigned long long)(blockIdx.x - (s ? sec.block_end[s - 1] : 0)) * kThreads + threadIdx.x;
    const unsigned long long row = at / PER_ROW;
    const int x = (int)(at % PER_ROW) * N;
    const bool in = row < sec.end[s] - first;
    const unsigned long long from = s < 3 ? row : row / n * pitch + row % n;
    float f[N];
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in) w = *reinterpret_cast<const uint4*>(static_cast<const E*>(src.x[s]) + from * D + x);
    Chunk<E>::unpack(w, f);
    // the largest magnitude by bits: a NaN is above infinity, infinity above all else
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!in) return;
    const float a = __uint_as_float(top);
    const bool coded = top > 0 && top < 0x7f800000u;
    uint32_t packed[N / 4] = {};
    if (coded) {
#pragma unroll
        for (int i = 0; i < N; ++i) packed[i >> 2] |= ((uint32_t)(int)Chunk<E>::code(f[i], a) & 0xffu) << (8 * (i & 3));
    }
    const unsigned long long to = first + row;
    uint32_t* dst = reinterpret_cast<uint32_t*>(codes + to * D + x);
    if (N == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[N / 4 - 1]);
    else
        *dst = packed[0];
    if (x % kCkptGroup == 0)
        scales[to * (D / kCkptGroup) + x / kCkptGroup] = coded || top == 0 ? __fdiv_rn(a, 127.f) : __uint_as_float(0x7fffffffu);
}

template <typename E>
__device__ __forceinline__ void store8(E* p, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Each thread restores 8 values. K and V rows are counted over the pitch: the
// rows of empty slots get zeros.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
ckpt_restore_kernel(CkptPtrs dst, const int8_t* __restrict__ codes, const float* __restrict__ scales, Sections sec,
                    Sections out, int n, int pitch) {
    const int s = section_of(out, blockIdx.x);
    if (dst.x[s] == nullptr) return;
    const unsigned long long at = (unsigned long long)(blockIdx.x - (s ? out.block_end[s - 1] : 0)) * kThreads + threadIdx.x;
    const unsigned long long row = at / (D / 8);
    const int x = (int)(at % (D / 8)) * 8;
    if (row >= out.end[s]) return;
    unsigned long long from = (s ? sec.end[s - 1] : 0) + row;
    bool valid = true;
    if (s >= 3) {
        const unsigned long long slot = row % pitch;
        valid = slot < (unsigned long long)n;
        from = sec.end[s - 1] + row / pitch * n + slot;
    }
    float f[8] = {};
    if (valid) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + from * D + x);
        const float sc = scales[from * (D / kCkptGroup) + x / kCkptGroup];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3))) * sc;
    }
    store8(static_cast<E*>(dst.x[s]) + row * D + x, f);
}

int blocks_for(unsigned long long rows, int per_row) { return (int)((rows * per_row + kThreads - 1) / kThreads); }

Sections sections(const CkptArgs& a, int per_row) {
    const unsigned long long rows[5] = {(unsigned long long)a.B * a.Hq * a.T, (unsigned long long)a.B * a.Hkv * a.T,
                                        (unsigned long long)a.B * a.Hkv * a.T, (unsigned long long)a.B * a.Hkv * a.n,
                                        (unsigned long long)a.B * a.Hkv * a.n};
    Sections s;
    unsigned long long r = 0;
    int blk = 0;
    for (int i = 0; i < 5; ++i) {
        s.end[i] = r += rows[i];
        s.block_end[i] = blk += blocks_for(rows[i], per_row);
    }
    return s;
}

CkptPtrs pointers(const CkptArgs& a) { return CkptPtrs{{a.q, a.k, a.v, a.K, a.V}}; }

template <typename E, int D>
cudaError_t save_typed(const CkptArgs& a) {
    const Sections sec = sections(a, D / Chunk<E>::N);
    ckpt_save_kernel<E, D><<<sec.block_end[4], kThreads, 0, a.stream>>>(pointers(a), a.codes, a.scales, sec, a.n, a.pitch);
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t restore_typed(const CkptArgs& a) {
    const Sections sec = sections(a, D / 8);
    Sections out = sec;  // rows written per section, and its blocks
    int blk = 0;
    const unsigned long long rows[5] = {(unsigned long long)a.B * a.Hq * a.T, (unsigned long long)a.B * a.Hkv * a.T,
                                        (unsigned long long)a.B * a.Hkv * a.T, (unsigned long long)a.B * a.Hkv * a.pitch,
                                        (unsigned long long)a.B * a.Hkv * a.pitch};
    for (int i = 0; i < 5; ++i) {
        out.end[i] = rows[i];
        out.block_end[i] = blk += blocks_for(rows[i], D / 8);
    }
    ckpt_restore_kernel<E, D><<<blk, kThreads, 0, a.stream>>>(pointers(a), a.codes, a.scales, sec, out, a.n, a.pitch);
    return cudaGetLastError();
}

// ============================================================================
// gradient carry
// ============================================================================
// With slot[t] the slot that chunk token t was written to (-1: dropped), and g
// the gradient of the cache after the step:
//   g_before[s] = d[s] + (no token was written to s ? g[s] : 0)   (s < n, else 0)
//   g_chunk[t]  = d_chunk[t] + (slot[t] >= 0 ? g[slot[t]] : 0)
// in fp32, the chunk's sums rounded once to the element type. Bound by memory:
// each row of g is read once, by its slot or by its token.
constexpr int kCarryRows = 32;  // slots or tokens per block

template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
carry_kernel(const int32_t* __restrict__ token_slot, const E* __restrict__ dK, const E* __restrict__ dV,
             const E* __restrict__ dk, const E* __restrict__ dv, const float* __restrict__ gK_next,
             const float* __restrict__ gV_next, float* __restrict__ gK, float* __restrict__ gV, E* __restrict__ gk,
             E* __restrict__ gv, int C, int T, int n, int slot_blocks, int token_blocks) {
    __shared__ int taken[kCarryRows];
    const int per = slot_blocks + token_blocks;
    const size_t bg = blockIdx.x / per;
    const int blk = blockIdx.x % per;
    const int32_t* slots = token_slot + bg * T;
    constexpr int PER_ROW = D / 4;
    if (blk < slot_blocks) {
        const int s0 = blk * kCarryRows;
        if (threadIdx.x < kCarryRows) taken[threadIdx.x] = 0;
        __syncthreads();
        for (int t = threadIdx.x; t < T; t += kThreads) {
            const int s = slots[t];
            if (s >= s0 && s < s0 + kCarryRows && s < C) taken[s - s0] = 1;
        }
        __syncthreads();
        const int rows = min(kCarryRows, C - s0);
        for (int e = threadIdx.x; e < rows * PER_ROW; e += kThreads) {
            const int s = s0 + e / PER_ROW;
            const size_t off = (bg * C + s) * D + 4 * (e % PER_ROW);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
            if (s < n) {
                a = load4(dK + off);
                c = load4(dV + off);
                if (gK_next && !taken[s - s0]) {
                    a = add4(a, load4(gK_next + off));
                    c = add4(c, load4(gV_next + off));
                }
            }
            store4(gK + off, a);
            store4(gV + off, c);
        }
    } else {
        const int t0 = (blk - slot_blocks) * kCarryRows;
        const int rows = min(kCarryRows, T - t0);
        for (int e = threadIdx.x; e < rows * PER_ROW; e += kThreads) {
            const int t = t0 + e / PER_ROW, x = 4 * (e % PER_ROW);
            const size_t off = (bg * T + t) * D + x;
            const int s = slots[t];
            float4 a = load4(dk + off), c = load4(dv + off);
            if (gK_next && s >= 0 && s < C) {
                a = add4(a, load4(gK_next + (bg * C + s) * D + x));
                c = add4(c, load4(gV_next + (bg * C + s) * D + x));
            }
            store4(gk + off, a);
            store4(gv + off, c);
        }
    }
}

template <typename E, int D>
cudaError_t carry_typed(const CarryArgs& a) {
    const int sb = (a.C + kCarryRows - 1) / kCarryRows, tb = (a.T + kCarryRows - 1) / kCarryRows;
    carry_kernel<E, D><<<(unsigned)(a.B * a.Hkv * (sb + tb)), kThreads, 0, a.stream>>>(
        a.token_slot, (const E*)a.dK, (const E*)a.dV, (const E*)a.dk, (const E*)a.dv, a.gK_next, a.gV_next, a.gK, a.gV,
        (E*)a.gk, (E*)a.gv, a.C, a.T, a.n, sb, tb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt_save(const CkptArgs& a) {
    if (a.dtype == 1) return a.d == 64 ? save_typed<float, 64>(a) : save_typed<float, 128>(a);
    return a.d == 64 ? save_typed<__nv_bfloat16, 64>(a) : save_typed<__nv_bfloat16, 128>(a);
}

cudaError_t launch_ckpt_restore(const CkptArgs& a) {
    if (a.dtype == 1) return a.d == 64 ? restore_typed<float, 64>(a) : restore_typed<float, 128>(a);
    return a.d == 64 ? restore_typed<__nv_bfloat16, 64>(a) : restore_typed<__nv_bfloat16, 128>(a);
}

cudaError_t launch_carry(const CarryArgs& a) {
    if (a.dtype == 1) return a.d == 64 ? carry_typed<float, 64>(a) : carry_typed<float, 128>(a);
    return a.d == 64 ? carry_typed<__nv_bfloat16, 64>(a) : carry_typed<__nv_bfloat16, 128>(a);
}

}  // namespace h2o
