// context.h -- the context behind the C ABI's handle, and the helpers its entry
// points share: error reporting, the device guard and the argument checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <vector>

#include "../../include/h2o.h"
#include "kernels.h"

struct h2o_ctx {
    int B, Hq, Hkv, d, C, dtype, tmax;
    int policy = 0;  // H2O_POLICY_SUM
    int device;
    int num_sms;
    int64_t P, n;
    size_t elem;
    // cache
    void* Kc = nullptr;
    void* Vc = nullptr;
    float* scores = nullptr;
    int32_t* pos = nullptr;
    // workspace (capacity tmax tokens)
    float* lse = nullptr;
    float* cand_score = nullptr;
    int32_t* cand_pos = nullptr;
    uint8_t* cand_kept = nullptr;
    int32_t* token_slot = nullptr;
    float* partials = nullptr;
    size_t partial_elems = 0;
    float* nlse2 = nullptr;
    int rows_pad = 0;
    // insert-always workspace (allocated when the policy is first selected):
    // compact K/V of the kept entries, their slots, scores and positions
    void* ins_K = nullptr;
    void* ins_V = nullptr;
    int32_t* ins_slot = nullptr;
    float* ins_score = nullptr;
    int32_t* ins_pos = nullptr;
    // backward workspace (allocated on the first h2o_backward): dO . O and the
    // log2-domain LSE per flattened group row, [2][groups][bwd_rows_pad]
    float* bwd_rows = nullptr;
    int bwd_rows_pad = 0;
    // split SDPA workspace (grown on demand when a step splits its units)
    float* sdpa_part = nullptr;
    size_t sdpa_part_elems = 0;
    // decode-path workspace (chunks of up to kDecodeMaxT tokens)
    float* dec_part = nullptr;
    float* dec_logits = nullptr;
    float* dec_lse2 = nullptr;
    // host staging for h2o_step_host
    void* stage = nullptr;
    size_t stage_bytes = 0;
    // pipelined host path (h2o_step_host_async): two staging slots, an upload
    // and a download stream, and per-slot events
    void* aslot[2] = {nullptr, nullptr};
    size_t aslot_bytes = 0;
    cudaStream_t s_in = nullptr, s_out = nullptr;
    cudaEvent_t ev_in[2] = {nullptr, nullptr};    // slot's inputs uploaded
    cudaEvent_t ev_step[2] = {nullptr, nullptr};  // step reading the slot done
    cudaEvent_t ev_out[2] = {nullptr, nullptr};   // slot's output downloaded
    long long achunks = 0;
    // error word (host-mapped)
    int* err_host = nullptr;
    int* err_dev = nullptr;
    unsigned long long wait_ns;
    int poisoned = 0;
    // last step
    int last_T = 0, last_n = 0;
    bool use_tc = false;
    // tree attention and checkpoint workspaces (allocated on first use; an
    // outgrown one is kept until the context goes, because a captured graph
    // may hold its address)
    float* tree_part = nullptr;
    unsigned* tree_count = nullptr;
    void* ckpt_ws = nullptr;
    size_t ckpt_ws_bytes = 0;
    std::vector<void*> retired;
    std::mutex workspaces;  // held by the calls that use them: two threads' calls are queued one after the other
    // per-kernel profiling
    bool prof_on = false;
    int prof_max_steps = 0, prof_steps = 0;
    std::vector<cudaEvent_t> prof_ev;      // (kMaxStepKernels + 1) per step
    std::vector<h2o::LaunchLog> prof_logs;
    char err[512];
};

namespace h2o {

inline int fail(h2o_ctx* c, int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    if (c) {
        snprintf(c->err, sizeof(c->err), "%s", buf);
    } else {
        set_thread_error_message(buf);
    }
    return code;
}

// The status reports the error, so the runtime's own record of it goes: the launchers
// end in cudaGetLastError(), and the next call of this thread would fail with an
// allocation that this one could not make. (What breaks the CUDA context stays.)
inline int cuda_fail(h2o_ctx* c, cudaError_t e, const char* what) {
    cudaGetLastError();
    return fail(c, e == cudaErrorMemoryAllocation ? H2O_ERR_OOM : H2O_ERR_CUDA, "%s: %s (%s)", what,
                cudaGetErrorString(e), cudaGetErrorName(e));
}

#define H2O_TRY(ctx, expr, what)                        \
    do {                                                \
        cudaError_t e_ = (expr);                        \
        if (e_ != cudaSuccess) return cuda_fail(ctx, e_, what); \
    } while (0)

// Makes the context's device current for the lifetime of the object.
struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) {
            changed = cudaSetDevice(dev) == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_ctx(h2o_ctx* c) {
    if (!c) return fail(nullptr, H2O_ERR_ARG, "null context");
    if (c->poisoned) return fail(c, H2O_ERR_POISONED, "context poisoned by an earlier device error");
    const int word = *(volatile int*)c->err_host;
    if (word != kDevOk) {
        c->poisoned = 1;
        return fail(c, H2O_ERR_TIMEOUT, "a kernel stopped after a bounded wait ran out (device code %d)",
                    word);
    }
    return H2O_OK;
}

}  // namespace h2o
