// operators.h -- launch interface of the operators that stand next to the H2O
// step: tree attention over the cache, the 8-bit step checkpoint, the backward
// from one, and the gradient carried through the eviction.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace h2o {

constexpr int kTreeMaxT = 256;                   // drafted nodes per sequence
constexpr int kTreeMaskWords = kTreeMaxT / 32;   // ancestor bits of a node
constexpr int kCkptGroup = 32;                   // channels that share one scale

// Tree attention: every drafted node attends to the n valid cache slots, to its
// ancestors and to itself; the cache is only read. Device pointers.
struct TreeArgs {
    int B, Hq, Hkv, d, C, T;
    int n;                  // valid cache slots (prefix 0..n-1)
    int dtype;              // 0 = bf16, 1 = fp32
    const void* q;          // [B,Hq,T,d]
    const void* k;          // [B,Hkv,T,d]
    const void* v;          // [B,Hkv,T,d]
    const int32_t* parent;  // [B,T]: -1 = root, 0..i-1 = that node, else absent
    const void* Kc;         // [B,Hkv,C,d]
    const void* Vc;         // [B,Hkv,C,d]
    void* out;              // [B,Hq,T,d]
    float* lse;             // [B,Hq,T]
    float* part;            // workspace of tree_part_floats() floats (CUDA cores: tree_simt_part_floats())
    unsigned* count;        // workspace of max(B * Hkv, num_sms) words, zero between calls
    WaitBound wb;
    cudaStream_t stream;
    int num_sms;
};
cudaError_t launch_tree_simt(const TreeArgs& a);
cudaError_t launch_tree_tc(const TreeArgs& a);  // bf16
size_t tree_part_floats(int num_sms, int d);
size_t tree_simt_part_floats(int num_sms, int d);
// bf16: up to so many products of a query and a key channel take the CUDA cores, where
// the tensor-core kernel's way through TMEM costs more than the arithmetic; more where a
// KV head has few rows, which read each key once or twice. Measured, us a pass, CUDA
// cores / tensor cores, millions of products: 4 or 8 rows: 8.4: 8.0 / 11.9, 16.8:
// 11.1 / 12.0, 30.7: 15.1 / 15.9, 33.6: 16.8 / 15.8; 12 to 64 rows: 3.8: 6.6 / 7.8, 8.5:
// 9.9 / 9.6 (d = 64: 11.6 / 8.1), 16.8: 12.3 / 10.5.
constexpr int kTreeFewRows = 8;
constexpr long long kTreeSimtProductsFew = 30ll << 20, kTreeSimtProducts = 8ll << 20;

// 8-bit record of a step's inputs: codes of q, k, v (the chunk) and of the n
// valid slots of K and V, row after row, then their scales in the same order.
struct CkptArgs {
    int B, Hq, Hkv, d, T, n;
    int dtype;
    int8_t* codes;      // [rows][d]
    float* scales;      // [rows][d / kCkptGroup]
    void* q;            // values: read by the save, written by the restore
    void* k;
    void* v;
    void* K;            // [B,Hkv,pitch,d]
    void* V;
    int pitch;          // slots per (sequence, KV head) of K and V (>= n)
    cudaStream_t stream;
};
// Rows of a record (d codes and d / kCkptGroup scales each).
inline size_t ckpt_rows(int B, int Hq, int Hkv, int T, int n) {
    return (size_t)B * ((size_t)Hq * T + 2 * (size_t)Hkv * T + 2 * (size_t)Hkv * n);
}
inline size_t ckpt_bytes(int B, int Hq, int Hkv, int d, int T, int n) {
    return ckpt_rows(B, Hq, Hkv, T, n) * (d + d / kCkptGroup * sizeof(float));
}
cudaError_t launch_ckpt_save(const CkptArgs& a);
// Writes the values for which a pointer is given; slots n..pitch-1 get zeros.
cudaError_t launch_ckpt_restore(const CkptArgs& a);

// Backward of a step's attention at restored values, its softmax statistics
// recomputed. Device pointers; gradients in the element type.
struct CkptBwdArgs {
    int B, Hq, Hkv, d, C, T;
    int n;              // valid cache slots of the record
    int dtype;          // 0 = bf16, 1 = fp32
    const void* q;      // [B,Hq,T,d]
    const void* k;      // [B,Hkv,T,d]
    const void* v;      // [B,Hkv,T,d]
    const void* K;      // [B,Hkv,pitch,d]
    const void* V;      // [B,Hkv,pitch,d]
    int pitch;
    const void* dout;   // [B,Hq,T,d]
    void* dq;           // [B,Hq,T,d]
    void* dK;           // [B,Hkv,C,d] (zero in slots n..C-1)
    void* dV;
    void* dk;           // [B,Hkv,T,d]
    void* dv;
    float* stats;       // workspace of ckpt_stats_floats() floats
    unsigned* count;    // num_sms words, zero between calls
    WaitBound wb;
    cudaStream_t stream;
    int num_sms;
};
// Floats of the workspace for the rows' statistics (and, on the tensor cores, the
// parts of divided query tiles); needs the sizes and num_sms of a, enough for any
// smaller T and n.
size_t ckpt_stats_floats(const CkptBwdArgs& a);
cudaError_t launch_ckpt_backward_simt(const CkptBwdArgs& a);  // fp32
cudaError_t launch_ckpt_backward_tc(const CkptBwdArgs& a);  // bf16

// Gradient of the cache after a step handed back through the eviction.
struct CarryArgs {
    int B, Hkv, d, C, T, n;
    int dtype;                  // of dK, dV, dk, dv, gk, gv
    const int32_t* token_slot;  // [B,Hkv,T]
    const void* dK;             // [B,Hkv,C,d]
    const void* dV;
    const void* dk;             // [B,Hkv,T,d]
    const void* dv;
    const float* gK_next;       // [B,Hkv,C,d], or nullptr (no later step)
    const float* gV_next;
    float* gK;                  // [B,Hkv,C,d]
    float* gV;
    void* gk;                   // [B,Hkv,T,d]
    void* gv;
    cudaStream_t stream;
};
cudaError_t launch_carry(const CarryArgs& a);

}  // namespace h2o
