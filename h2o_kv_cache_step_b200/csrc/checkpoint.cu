// checkpoint.cu -- a step's inputs kept in 8 bits, and the gradient of the cache
// carried through the eviction.
//
// Record: with a = max |x| over 32 consecutive channels of a row,
//   code = rint(127 x / a) (ties to even), scale = a / 127 rounded to fp32 (down for
//   fp32's largest value, whose 127 scale would round to infinity),
// and the value it stands for is code * scale, rounded to the element type. A
// group of zeros has scale 0; a group with a NaN or an infinity has scale NaN
// and stands for NaNs.
//
// The code follows the real quotient without a division per value. With p-bit
// significands (8 for bf16, 24 for fp32), 254 x - (2k + 1) a is a whole number
// of units of x's last place, so a quotient that is not on a border k + 1/2
// keeps a relative distance of 2^-(8 + p) from it; x times the rounded 127 / a
// is within 2^-20 of it in fp32 and 2^-52 in 64 bits, so its nearest whole number
// is the code. What is left are the borders, (2k + 1) a = 254 x:
//   bf16, in fp32: 127 is prime, so it divides 2k + 1 (then k = 63 and x = a / 2)
//   or a's significand (then that is 127 times a power of two, and 127 / a is
//   exact). With 127 / a taken two units too large, the first lands just above 63.5
//   and goes to 64, the even one; the second takes the exact power of two. One
//   multiply-add and its rounding give the code. Groups near the ends of fp32's range
//   are moved by a power of two, which leaves quotients alone: 1 / a has to be a normal
//   number, or it is off by more than the two units.
//   fp32, in 64 bits: the remainder 127 x - code a is exact, is +-a / 2 on a
//   border, and an odd code then moves to its even neighbour.
//
// Both directions are bound by memory: each value is read and written once. A thread
// of the save takes 16 values twice, so that finding its place costs less next to them
// (once, twice, four times: 51.9, 48.5, 56.3 us for a batch of four chunks of 2048
// tokens and caches of 4096 slots, 262 MB; the floor is 40.0), a thread of the restore
// once (43.1 us; twice 46.3).
#include <math.h>

#include "kernels.h"
#include "operators.h"
#include "vec.cuh"

namespace h2o {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;  // values per thread at a time; two threads share a group of 32
constexpr int kSaveIter = 2, kRestoreIter = 1;  // times
static_assert(kCkptGroup == 2 * kPer, "a group is a pair of threads");
constexpr float kMaxScale = 0x1.020406p+121f;  // 127 times the next value is infinite in fp32

// The five sections of a record (q, k, v, K, V): `outer` runs of `rows` rows in
// the record, and of `pitch` rows in the tensors (rows past `rows` are empty).
struct Section {
    void* x;
    unsigned long long code_row;  // first row in the record
    unsigned long long rows, pitch;
    int blocks;      // per run
    int block_end;   // first block after the section
};
struct Sections {
    Section s[5];
};

// Where a thread works: its section, its first row there and its channel. Its other
// rows are kRows<D> further each.
template <int D>
constexpr int kRows = kThreads * kPer / D;

struct Place {
    void* x;
    unsigned long long code, row;  // row in the record, row in the tensor
    int col;
    long long in, valid;  // rows from here to the end of the run in the tensor, in the record
};

template <int D, int kIter>
__device__ __forceinline__ Place place(const Sections& sec) {
    int k = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) k += (int)blockIdx.x >= sec.s[i].block_end;
    const Section& s = sec.s[k];
    const unsigned blk = blockIdx.x - (k ? sec.s[k - 1].block_end : 0), run = blk / (unsigned)s.blocks;
    const unsigned long long r = (unsigned long long)(blk - run * s.blocks) * (kRows<D> * kIter) + threadIdx.x / (D / kPer);
    Place p;
    p.x = s.x;
    p.col = threadIdx.x % (D / kPer) * kPer;
    p.in = (long long)(s.pitch - r);
    p.valid = (long long)(s.rows - r);
    p.code = s.code_row + run * s.rows + r;
    p.row = run * s.pitch + r;
    return p;
}

__device__ __forceinline__ void load16(const float* x, float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = reinterpret_cast<const float4*>(x)[i];
        f[4 * i] = w.x;
        f[4 * i + 1] = w.y;
        f[4 * i + 2] = w.z;
        f[4 * i + 3] = w.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* x, float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 w = reinterpret_cast<const uint4*>(x)[i];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
            f[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void store16(float* x, const float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(x)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* x, const float (&f)[kPer]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&t);
        }
        reinterpret_cast<uint4*>(x)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The codes of 16 values of a group whose largest magnitude is a (finite, > 0),
// in the low bytes of c. Adding 1.5 * 2^23 rounds to a whole number, ties to
// even, and leaves it in the low bits.
__device__ __forceinline__ void codes16(float (&f)[kPer], float a, uint32_t (&c)[kPer], __nv_bfloat16) {
    if (a < 0x1p-100f || a >= 0x1p100f) {  // 127 / a stays in range, 1 / a normal (24 bits)
        const float by = a < 1.f ? 0x1p60f : 0x1p-60f;
        a *= by;
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] *= by;
    }
    const uint32_t bits = __float_as_uint(a);
    const float over = __uint_as_float(__float_as_uint(127.f * __frcp_rn(a)) + 2);
    // a = 127 * 2^(e - 133), e its exponent field
    const float r = (bits & 0x7fffffu) == 0x7e0000u ? __uint_as_float((260u - (bits >> 23)) << 23) : over;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = __float_as_uint(fmaf(f[i], r, 12582912.f));
}
__device__ __forceinline__ void codes16(float (&f)[kPer], float a, uint32_t (&c)[kPer], float) {
    const double b = a, r = 1.0 / b, half = 0.5 * b;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const double x = 127.0 * f[i];
        double q = rint(x * r);
        const double rem = fma(-q, b, x);
        if (fabs(rem) == half && ((int)q & 1)) q += rem > 0.0 ? 1.0 : -1.0;
        c[i] = (uint32_t)(int)q;
    }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
ckpt_save_kernel(const __grid_constant__ Sections sec, int8_t* __restrict__ codes, float* __restrict__ scales) {
    constexpr int kIter = kSaveIter;
    const Place p = place<D, kIter>(sec);
    const E* src = static_cast<const E*>(p.x) + p.row * D + p.col;
    griddep_wait();  // the work before is complete; what follows may set up
    griddep_launch_dependents();
    float all[kIter][kPer] = {};
#pragma unroll
    for (int it = 0; it < kIter; ++it)
        if (it * kRows<D> < p.valid) load16(src + it * kRows<D> * D, all[it]);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const bool valid = it * kRows<D> < p.valid;
        float(&f)[kPer] = all[it];
        // the largest magnitude by bits: a NaN is above infinity, infinity above all else
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (!valid) continue;
        const float a = __uint_as_float(top);
        const bool coded = top > 0 && top < 0x7f800000u;
        uint32_t c[kPer] = {};
        if (coded) codes16(f, a, c, E());
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
        const unsigned long long at = (p.code + it * kRows<D>) * D + p.col;
        *reinterpret_cast<uint4*>(codes + at) = make_uint4(w[0], w[1], w[2], w[3]);
        if (p.col % kCkptGroup == 0)
            scales[at / kCkptGroup] =
                coded || top == 0 ? fminf(__fdiv_rn(a, 127.f), kMaxScale) : __uint_as_float(0x7fffffffu);
    }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
ckpt_restore_kernel(const __grid_constant__ Sections sec, const int8_t* __restrict__ codes, const float* __restrict__ scales) {
    constexpr int kIter = kRestoreIter;
    const Place p = place<D, kIter>(sec);
    griddep_wait();  // the work before is complete; what follows may set up
    griddep_launch_dependents();
    if (p.x == nullptr) return;
    E* dst = static_cast<E*>(p.x) + p.row * D + p.col;
    uint4 w[kIter];
    float sc[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        w[it] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        sc[it] = 0.f;
        if (it * kRows<D> >= p.valid) continue;
        const unsigned long long at = (p.code + it * kRows<D>) * D + p.col;
        const uint4 x = *reinterpret_cast<const uint4*>(codes + at);
        w[it] = make_uint4(x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u);
        sc[it] = scales[at / kCkptGroup];
    }
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        if (it * kRows<D> >= p.in) continue;
        const uint32_t u[4] = {w[it].x, w[it].y, w[it].z, w[it].w};
        float f[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i)  // code + 128 as the last byte of 2^23's float, less 2^23 + 128
            f[i] = (__uint_as_float(__byte_perm(u[i >> 2], 0x4b000000u, 0x7440 + (i & 3))) - 8388736.f) * sc[it];
        store16(dst + it * kRows<D> * D, f);
    }
}

// The save visits the rows of the record, the restore those of the tensors.
Sections sections(const CkptArgs& a, bool restore) {
    const unsigned long long groups = (unsigned long long)a.B * a.Hkv;
    const unsigned long long per = kThreads * kPer / a.d * (restore ? kRestoreIter : kSaveIter);
    void* x[5] = {a.q, a.k, a.v, a.K, a.V};
    Sections out;
    unsigned long long row = 0;
    int blk = 0;
    for (int i = 0; i < 5; ++i) {
        Section& s = out.s[i];
        const bool cache = i >= 3;
        const unsigned long long outer = cache ? groups : 1;
        s.x = x[i];
        s.code_row = row;
        s.rows = cache ? a.n : (i ? groups : (unsigned long long)a.B * a.Hq) * a.T;
        s.pitch = cache ? a.pitch : s.rows;
        const unsigned long long visited = restore ? s.pitch : s.rows;
        s.blocks = (int)((visited + per - 1) / per);
        row += outer * s.rows;
        s.block_end = blk += (int)outer * s.blocks;
    }
    return out;
}

template <typename E, int D>
cudaError_t save_typed(const CkptArgs& a) {
    const Sections sec = sections(a, false);
    return launch_ex(true, ckpt_save_kernel<E, D>, dim3(sec.s[4].block_end), dim3(kThreads), 0, a.stream, sec, a.codes, a.scales);
}

template <typename E, int D>
cudaError_t restore_typed(const CkptArgs& a) {
    const Sections sec = sections(a, true);
    return launch_ex(true, ckpt_restore_kernel<E, D>, dim3(sec.s[4].block_end), dim3(kThreads), 0, a.stream, sec,
                     (const int8_t*)a.codes, (const float*)a.scales);
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
    griddep_wait();  // the work before is complete; what follows may set up
    griddep_launch_dependents();
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
    return launch_ex(
        true, carry_kernel<E, D>, dim3((unsigned)(a.B * a.Hkv * (sb + tb))), dim3(kThreads), 0, a.stream,
        a.token_slot, (const E*)a.dK, (const E*)a.dV, (const E*)a.dk, (const E*)a.dv, a.gK_next, a.gV_next, a.gK, a.gV,
        (E*)a.gk, (E*)a.gv, a.C, a.T, a.n, sb, tb);
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
