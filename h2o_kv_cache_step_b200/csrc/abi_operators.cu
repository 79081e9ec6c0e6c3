// abi_operators.cu -- C ABI of the operators next to the step (declared in
// include/h2o.h): tree attention, 8-bit step checkpoints, the backward from
// one, and the gradient carried through the eviction.
//
// The host checks the arguments, keeps the workspaces and launches; a workspace
// that has to grow is kept until the context is destroyed, because a captured
// graph may hold its address.
#include <algorithm>
#include <exception>
#include <mutex>

#include "context.h"
#include "operators.h"

using namespace h2o;

namespace {

bool overlap(const void* a, const void* b, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bytes && y < x + bytes;
}

bool capturing(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(s, &st) == cudaSuccess && st != cudaStreamCaptureStatusNone;
}

// Counters at the start of the checkpoint workspace, one per SM, zero between calls.
size_t ckpt_count_bytes(const h2o_ctx* c) { return (sizeof(unsigned) * c->num_sms + 255) & ~(size_t)255; }

// The checkpoint workspace, at least `bytes` large. An outgrown one is replaced by one
// of twice its size, if the card has that much, so that calls that grow step by step
// allocate rarely and what is kept of them is less than the one in use.
int checkpoint_workspace(h2o_ctx* c, size_t bytes, cudaStream_t s) {
    if (bytes <= c->ckpt_ws_bytes) return H2O_OK;
    if (capturing(s))
        return fail(c, H2O_ERR_UNSUPPORTED, "the workspace has to be allocated outside a capture: make the call once before");
    c->retired.reserve(c->retired.size() + 1);
    void* p = nullptr;
    size_t got = std::max(bytes, 2 * c->ckpt_ws_bytes);
    cudaError_t e = cudaMalloc(&p, got);
    if (e == cudaErrorMemoryAllocation && got > bytes) {
        cudaGetLastError();
        e = cudaMalloc(&p, got = bytes);
    }
    if (e != cudaSuccess) return cuda_fail(c, e, "cudaMalloc(checkpoint workspace)");
    e = cudaMemset(p, 0, ckpt_count_bytes(c));
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        cudaFree(p);
        return cuda_fail(c, e, "clearing the checkpoint workspace");
    }
    if (c->ckpt_ws) c->retired.push_back(c->ckpt_ws);  // room reserved above
    c->ckpt_ws = p;
    c->ckpt_ws_bytes = got;
    return H2O_OK;
}

int check_chunk(h2o_ctx* c, int T) {
    if (T < 1) return fail(c, H2O_ERR_ARG, "T must be >= 1 (got %d)", T);
    if ((long long)c->C + T > (1ll << 30)) return fail(c, H2O_ERR_UNSUPPORTED, "C + T too large");
    return H2O_OK;
}

int check_slots(h2o_ctx* c, int n) {
    if (n < 0 || n > c->C) return fail(c, H2O_ERR_ARG, "need 0 <= n <= C (got n = %d, C = %d)", n, c->C);
    return H2O_OK;
}

int check_record(h2o_ctx* c, const void* ckpt, size_t bytes, int T, int n) {
    int rc = check_chunk(c, T);
    if (rc == H2O_OK) rc = check_slots(c, n);
    if (rc != H2O_OK) return rc;
    if (!ckpt) return fail(c, H2O_ERR_ARG, "ckpt must be non-NULL");
    if (!aligned16(ckpt)) return fail(c, H2O_ERR_ALIGN, "ckpt must be 16-byte aligned");
    const size_t need = ckpt_bytes(c->B, c->Hq, c->Hkv, c->d, T, n);
    if (bytes < need)
        return fail(c, H2O_ERR_ARG, "the record of T = %d tokens and n = %d slots takes %zu bytes (got %zu)", T, n, need, bytes);
    return H2O_OK;
}

CkptArgs ckpt_args(const h2o_ctx* c, const void* ckpt, int T, int n, cudaStream_t s) {
    CkptArgs a{};
    a.B = c->B;
    a.Hq = c->Hq;
    a.Hkv = c->Hkv;
    a.d = c->d;
    a.T = T;
    a.n = n;
    a.dtype = c->dtype;
    a.codes = static_cast<int8_t*>(const_cast<void*>(ckpt));
    a.scales = reinterpret_cast<float*>(a.codes + ckpt_rows(c->B, c->Hq, c->Hkv, T, n) * c->d);
    a.pitch = c->C;
    a.stream = s;
    return a;
}

// Nothing the host code below throws (a container that finds no memory) leaves a C
// entry.
int thrown(h2o_ctx* c, const std::exception& e) { return fail(c, H2O_ERR_OOM, "host: %s", e.what()); }

}  // namespace

extern "C" {

int h2o_tree_attend(h2o_ctx* c, const void* q, const void* k, const void* v, const int32_t* parent, void* out,
                    float* lse, int T, void* stream) try {
    int rc = check_ctx(c);
    if (rc != H2O_OK) return rc;
    if (T < 1) return fail(c, H2O_ERR_ARG, "T must be >= 1 (got %d)", T);
    if (T > kTreeMaxT) return fail(c, H2O_ERR_UNSUPPORTED, "a tree has at most %d nodes per sequence (got %d)", kTreeMaxT, T);
    if (c->policy == H2O_POLICY_INSERT_ALWAYS)
        return fail(c, H2O_ERR_UNSUPPORTED,
                    "under insert-always the number of accepted tokens decides which slots a row may see");
    if (!q || !k || !v || !parent || !out || !lse)
        return fail(c, H2O_ERR_ARG, "q, k, v, parent, out, lse must be non-NULL");
    for (const void* p : {q, k, v, (const void*)out})
        if (!aligned16(p)) return fail(c, H2O_ERR_ALIGN, "q, k, v, out must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(parent) & 3) || (reinterpret_cast<uintptr_t>(lse) & 3))
        return fail(c, H2O_ERR_ALIGN, "parent and lse must be 4-byte aligned");
    DeviceGuard g(c->device);
    const std::lock_guard<std::mutex> lock(c->workspaces);
    if (!c->tree_part) {
        if (capturing((cudaStream_t)stream))
            return fail(c, H2O_ERR_UNSUPPORTED, "the workspace has to be allocated outside a capture: make the call once before");
        const size_t words = std::max((size_t)c->B * c->Hkv, (size_t)c->num_sms);
        if (!c->tree_count) {
            unsigned* count = nullptr;
            H2O_TRY(c, cudaMalloc(&count, sizeof(unsigned) * words), "cudaMalloc(tree workspace)");
            cudaError_t e = cudaMemset(count, 0, sizeof(unsigned) * words);
            if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
            if (e != cudaSuccess) {
                cudaFree(count);
                return cuda_fail(c, e, "clearing the tree workspace");
            }
            c->tree_count = count;
        }
        const size_t floats = c->use_tc ? tree_part_floats(c->num_sms, c->d) : tree_simt_part_floats(c->num_sms, c->d);
        H2O_TRY(c, cudaMalloc(&c->tree_part, sizeof(float) * floats), "cudaMalloc(tree workspace)");
    }
    TreeArgs a{};
    a.B = c->B;
    a.Hq = c->Hq;
    a.Hkv = c->Hkv;
    a.d = c->d;
    a.C = c->C;
    a.T = T;
    a.n = (int)c->n;
    a.dtype = c->dtype;
    a.q = q;
    a.k = k;
    a.v = v;
    a.parent = parent;
    a.Kc = c->Kc;
    a.Vc = c->Vc;
    a.out = out;
    a.lse = lse;
    a.part = c->tree_part;
    a.count = c->tree_count;
    a.wb.err_word = c->err_dev;
    a.wb.ns = c->wait_ns;
    a.stream = (cudaStream_t)stream;
    a.num_sms = c->num_sms;
    const long long simt = c->Hq / c->Hkv * T <= kTreeFewRows ? kTreeSimtProductsFew : kTreeSimtProducts;
    const bool tc = c->use_tc && (long long)c->B * c->Hq * T * (c->n + T) * c->d > simt;
    H2O_TRY(c, tc ? launch_tree_tc(a) : launch_tree_simt(a), "launch tree attention");
    return H2O_OK;
} catch (const std::exception& e) {
    return thrown(c, e);
}

int h2o_checkpoint_bytes(const h2o_ctx* c, int T, int n, size_t* bytes) {
    if (!c) return fail(nullptr, H2O_ERR_ARG, "null context");
    h2o_ctx* m = const_cast<h2o_ctx*>(c);
    if (!bytes) return fail(m, H2O_ERR_ARG, "bytes is NULL");
    int rc = check_chunk(m, T);
    if (rc == H2O_OK) rc = check_slots(m, n);
    if (rc != H2O_OK) return rc;
    *bytes = ckpt_bytes(c->B, c->Hq, c->Hkv, c->d, T, n);
    return H2O_OK;
}

int h2o_checkpoint_save(h2o_ctx* c, const void* q, const void* k, const void* v, int T, void* ckpt, size_t bytes,
                        void* stream) try {
    int rc = check_ctx(c);
    if (rc != H2O_OK) return rc;
    if (c->policy == H2O_POLICY_INSERT_ALWAYS)
        return fail(c, H2O_ERR_UNSUPPORTED, "under insert-always a step does not attend to the cache it starts from");
    rc = check_record(c, ckpt, bytes, T, (int)c->n);
    if (rc != H2O_OK) return rc;
    if (!q || !k || !v) return fail(c, H2O_ERR_ARG, "q, k, v must be non-NULL");
    for (const void* p : {q, k, v})
        if (!aligned16(p)) return fail(c, H2O_ERR_ALIGN, "q, k, v must be 16-byte aligned");
    DeviceGuard g(c->device);
    CkptArgs a = ckpt_args(c, ckpt, T, (int)c->n, (cudaStream_t)stream);
    a.q = const_cast<void*>(q);
    a.k = const_cast<void*>(k);
    a.v = const_cast<void*>(v);
    a.K = c->Kc;
    a.V = c->Vc;
    H2O_TRY(c, launch_ckpt_save(a), "launch checkpoint save");
    return H2O_OK;
} catch (const std::exception& e) {
    return thrown(c, e);
}

int h2o_checkpoint_restore(h2o_ctx* c, const void* ckpt, size_t bytes, int T, int n, void* q, void* k, void* v,
                           void* K, void* V, void* stream) try {
    int rc = check_ctx(c);
    if (rc == H2O_OK) rc = check_record(c, ckpt, bytes, T, n);
    if (rc != H2O_OK) return rc;
    if (!q && !k && !v && !K && !V) return fail(c, H2O_ERR_ARG, "nothing to restore: every pointer is NULL");
    for (const void* p : {q, k, v, K, V})
        if (p && !aligned16(p)) return fail(c, H2O_ERR_ALIGN, "q, k, v, K, V must be 16-byte aligned");
    DeviceGuard g(c->device);
    CkptArgs a = ckpt_args(c, ckpt, T, n, (cudaStream_t)stream);
    a.q = q;
    a.k = k;
    a.v = v;
    a.K = K;
    a.V = V;
    H2O_TRY(c, launch_ckpt_restore(a), "launch checkpoint restore");
    return H2O_OK;
} catch (const std::exception& e) {
    return thrown(c, e);
}

int h2o_checkpoint_backward(h2o_ctx* c, const void* ckpt, size_t bytes, int T, int n, const void* dout, void* dq,
                            void* dK, void* dV, void* dk, void* dv, void* stream) try {
    int rc = check_ctx(c);
    if (rc == H2O_OK) rc = check_record(c, ckpt, bytes, T, n);
    if (rc != H2O_OK) return rc;
    if (!dout || !dq || !dK || !dV || !dk || !dv)
        return fail(c, H2O_ERR_ARG, "every pointer argument must be non-NULL");
    for (const void* p : {dout, (const void*)dq, (const void*)dK, (const void*)dV, (const void*)dk, (const void*)dv})
        if (!aligned16(p)) return fail(c, H2O_ERR_ALIGN, "every pointer argument must be 16-byte aligned");
    if (c->dtype == H2O_BF16 && !c->use_tc)
        return fail(c, H2O_ERR_UNSUPPORTED, "the bf16 backward runs on the tensor cores, which need the driver's tensor maps");
    DeviceGuard g(c->device);
    cudaStream_t s = (cudaStream_t)stream;
    CkptBwdArgs a{};
    a.B = c->B;
    a.Hq = c->Hq;
    a.Hkv = c->Hkv;
    a.d = c->d;
    a.C = c->C;
    a.T = T;
    a.n = n;
    a.dtype = c->dtype;
    a.num_sms = c->num_sms;
    // workspace: the restored step and the statistics of its rows, for C slots and the
    // context's chunk length, so that a run of steps over a filling cache allocates once
    CkptBwdArgs most = a;
    most.T = std::max(T, c->tmax);
    most.n = c->C;
    const size_t groups = (size_t)c->B * c->Hkv;
    const size_t nq = (size_t)c->B * c->Hq * most.T * c->d, nk = groups * most.T * c->d, nK = groups * c->C * c->d;
    size_t end = ckpt_count_bytes(c);
    auto take = [&](size_t b) {
        const size_t at = end;
        end += (b + 255) & ~(size_t)255;
        return at;
    };
    const size_t oq = take(nq * c->elem), ok = take(nk * c->elem), ov = take(nk * c->elem);
    const size_t oK = take(nK * c->elem), oV = take(nK * c->elem), os = take(sizeof(float) * ckpt_stats_floats(most));
    const std::lock_guard<std::mutex> lock(c->workspaces);
    rc = checkpoint_workspace(c, end, s);
    if (rc != H2O_OK) return rc;
    char* w = static_cast<char*>(c->ckpt_ws);
    const int pitch = std::max(n, 1);

    CkptArgs r = ckpt_args(c, ckpt, T, n, s);
    r.q = w + oq;
    r.k = w + ok;
    r.v = w + ov;
    r.K = w + oK;
    r.V = w + oV;
    r.pitch = pitch;
    H2O_TRY(c, launch_ckpt_restore(r), "launch checkpoint restore");

    a.q = r.q;
    a.k = r.k;
    a.v = r.v;
    a.K = r.K;
    a.V = r.V;
    a.pitch = pitch;
    a.dout = dout;
    a.dq = dq;
    a.dK = dK;
    a.dV = dV;
    a.dk = dk;
    a.dv = dv;
    a.stats = reinterpret_cast<float*>(w + os);
    a.count = static_cast<unsigned*>(c->ckpt_ws);
    a.wb.err_word = c->err_dev;
    a.wb.ns = c->wait_ns;
    a.stream = s;
    H2O_TRY(c, c->use_tc ? launch_ckpt_backward_tc(a) : launch_ckpt_backward_simt(a), "launch checkpoint backward");
    return H2O_OK;
} catch (const std::exception& e) {
    return thrown(c, e);
}

int h2o_carry_grad(h2o_ctx* c, const int32_t* token_slot, int T, int n, const void* dK, const void* dV, const void* dk,
                   const void* dv, const float* gK_next, const float* gV_next, float* gK, float* gV, void* gk, void* gv,
                   void* stream) try {
    int rc = check_ctx(c);
    if (rc == H2O_OK) rc = check_chunk(c, T);
    if (rc == H2O_OK) rc = check_slots(c, n);
    if (rc != H2O_OK) return rc;
    if (!token_slot || !dK || !dV || !dk || !dv || !gK || !gV || !gk || !gv)
        return fail(c, H2O_ERR_ARG, "every pointer argument but gK_next and gV_next must be non-NULL");
    if (!gK_next != !gV_next) return fail(c, H2O_ERR_ARG, "gK_next and gV_next are given together or not at all");
    for (const void* p : {dK, dV, dk, dv, (const void*)gK_next, (const void*)gV_next, (const void*)gK, (const void*)gV,
                          (const void*)gk, (const void*)gv})
        if (!aligned16(p)) return fail(c, H2O_ERR_ALIGN, "every gradient pointer must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(token_slot) & 3) return fail(c, H2O_ERR_ALIGN, "token_slot must be 4-byte aligned");
    const size_t bytes = sizeof(float) * (size_t)c->B * c->Hkv * c->C * c->d;
    for (const float* x : {gK_next, gV_next})
        for (const float* y : {gK, gV})
            if (x && overlap(x, y, bytes))
                return fail(c, H2O_ERR_ARG, "gK and gV must not overlap gK_next and gV_next: tokens and slots read them apart");
    DeviceGuard g(c->device);
    CarryArgs a{};
    a.B = c->B;
    a.Hkv = c->Hkv;
    a.d = c->d;
    a.C = c->C;
    a.T = T;
    a.n = n;
    a.dtype = c->dtype;
    a.token_slot = token_slot;
    a.dK = dK;
    a.dV = dV;
    a.dk = dk;
    a.dv = dv;
    a.gK_next = gK_next;
    a.gV_next = gV_next;
    a.gK = gK;
    a.gV = gV;
    a.gk = gk;
    a.gv = gv;
    a.stream = (cudaStream_t)stream;
    H2O_TRY(c, launch_carry(a), "launch gradient carry");
    return H2O_OK;
} catch (const std::exception& e) {
    return thrown(c, e);
}

}  // extern "C"
