// api_int8.cu -- the C ABI of scored routing and the int8 layer (include/moe.h):
// argument checks, workspace carving and launch sequences.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "expert_int8.cuh"
#include "int8_rows.cuh"
#include "route_scored.cuh"

namespace moe {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 27;  // T * k
constexpr int kMaxWidth = 131072;               // 127 * 127 * width < 2^31

bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
bool ok_opt(const void* p) { return p == nullptr || aligned16(p); }

int check_counts(const moe_shape& s) {
    if (s.T < 0 || s.E <= 0 || s.k <= 0 || s.k > s.E) return MOE_ERR_INVALID_ARG;
    if (s.E > kScoredMaxE || s.k > kScoredMaxK) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)s.T * s.k > kMaxRows) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_width(int n) {
    if (n <= 0) return MOE_ERR_INVALID_ARG;
    return n % 16 != 0 || n > kMaxWidth ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_shape(const moe_shape& s) {
    if (s.d <= 0 || s.d_ff <= 0) return MOE_ERR_INVALID_ARG;
    int rc = check_counts(s);
    if (rc == MOE_OK) rc = check_width(s.d);
    if (rc == MOE_OK) rc = check_width(s.d_ff);
    return rc;
}

int check_scoring(const moe_shape& s, const moe_scoring& r) {
    const int rc = check_counts(s);
    if (rc) return rc;
    if (r.score != MOE_SCORE_SOFTMAX && r.score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (r.n_group < 1 || s.E % r.n_group != 0) return MOE_ERR_INVALID_ARG;
    if (r.n_group > kScoredMaxGroups) return MOE_ERR_UNSUPPORTED;
    if (r.topk_group < 1 || r.topk_group > r.n_group) return MOE_ERR_INVALID_ARG;
    if (r.group_top < 1 || r.group_top > 2) return MOE_ERR_INVALID_ARG;
    if (s.k > r.topk_group * (s.E / r.n_group)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(r.scale)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

bool logits_type_ok(int t) { return t == MOE_LOGITS_F32 || t == MOE_LOGITS_BF16; }

// Workspace of moe_forward_int8: the experts' (with what has to be zeroed) first.
struct Layout {
    size_t idx, gate, offsets, perm, inv, xs, xq, o, total;
};

Layout layout(const moe_shape& s) {
    const size_t T = (size_t)s.T, R = T * s.k;
    Layout L{};
    size_t off = int8_workspace(s).total;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    L.idx = take(R * 4);
    L.gate = take(R * 4);
    L.offsets = take((size_t)(s.E + 1) * 4);
    L.perm = take(R * 4);
    L.inv = take(R * 4);
    L.xs = take(R * 4);
    L.xq = take(R * s.d);
    L.o = take(R * s.d * 2);
    L.total = off;
    return L;
}

template <typename T>
T* at(void* base, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

int experts(const moe_shape& s, const int8_t* xq, const float* xs, const int32_t* offsets,
            const Int8Experts& w, void* o, void* ws, size_t ws_bytes, int stall_after,
            uint64_t timeout_ns, cudaStream_t st) {
    const int rc = check_shape(s);
    if (rc || s.T == 0) return rc;
    if (!ok_ptr(xq) || !ok_ptr(xs) || !ok_ptr(offsets) || !ok_ptr(w.W1) || !ok_ptr(w.s1) ||
        !ok_ptr(w.W3) || !ok_ptr(w.s3) || !ok_ptr(w.W2) || !ok_ptr(w.s2) || !ok_ptr(o) ||
        !ok_ptr(ws))
        return MOE_ERR_INVALID_ARG;
    const Int8Workspace L = int8_workspace(s);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if (cudaMemsetAsync(ws, 0, L.zero_bytes, st) != cudaSuccess) return MOE_ERR_CUDA;
    return expert_products_int8(s, xq, xs, offsets, w, o, ws, static_cast<int*>(ws), timeout_ns,
                                stall_after, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_check_scoring(moe_shape s, moe_scoring r) { return check_scoring(s, r); }

int moe_check_shape_int8(moe_shape s) { return check_shape(s); }

int moe_route_scored(moe_shape s, moe_scoring r, const void* logits, int logits_type,
                     const float* bias, const uint8_t* mask, int32_t* idx, float* gate,
                     void* stream) {
    const int rc = check_scoring(s, r);
    if (rc) return rc;
    if (!logits_type_ok(logits_type)) return MOE_ERR_INVALID_ARG;
    if (s.T == 0) return MOE_OK;
    if (!ok_ptr(logits) || !ok_opt(bias) || !ok_opt(mask) || !ok_ptr(idx) || !ok_ptr(gate))
        return MOE_ERR_INVALID_ARG;
    return launch_route_scored(s, r, logits, logits_type == MOE_LOGITS_BF16, bias, mask, idx, gate,
                               static_cast<cudaStream_t>(stream));
}

int moe_route_scored_backward(moe_shape s, moe_scoring r, const void* logits, int logits_type,
                              const int32_t* idx, const float* dgate, void* dlogits,
                              void* stream) {
    const int rc = check_scoring(s, r);
    if (rc) return rc;
    if (!logits_type_ok(logits_type)) return MOE_ERR_INVALID_ARG;
    if (s.T == 0) return MOE_OK;
    if (!ok_ptr(logits) || !ok_ptr(idx) || !ok_ptr(dgate) || !ok_ptr(dlogits))
        return MOE_ERR_INVALID_ARG;
    return launch_route_scored_backward(s, r, logits, logits_type == MOE_LOGITS_BF16, idx, dgate,
                                        dlogits, static_cast<cudaStream_t>(stream));
}

int moe_quantize_weights_int8(int E, int K, int N, const void* W, int8_t* Wq, float* scale,
                              void* stream) {
    if (E < 1) return MOE_ERR_INVALID_ARG;
    if (E > kScoredMaxE) return MOE_ERR_UNSUPPORTED;
    if (const int rc = check_width(K)) return rc;
    if (const int rc = check_width(N)) return rc;
    if (!ok_ptr(W) || !ok_ptr(Wq) || !ok_ptr(scale)) return MOE_ERR_INVALID_ARG;
    return launch_quantize_weights(E, K, N, W, Wq, scale, static_cast<cudaStream_t>(stream));
}

int moe_dispatch_int8(moe_shape s, const int32_t* idx, const void* x, int32_t* offsets,
                      int32_t* perm_tok, int32_t* inv, int8_t* xq, float* xs, void* stream) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!ok_ptr(offsets)) return MOE_ERR_INVALID_ARG;
    if (s.T > 0 && (!ok_ptr(idx) || !ok_ptr(x) || !ok_ptr(perm_tok) || !ok_ptr(inv) ||
                    !ok_ptr(xq) || !ok_ptr(xs)))
        return MOE_ERR_INVALID_ARG;
    return launch_dispatch_quantize(s, idx, x, offsets, perm_tok, inv, xq, xs, nullptr, 0,
                                    static_cast<cudaStream_t>(stream));
}

size_t moe_expert_swiglu_int8_workspace_bytes(moe_shape s) {
    return check_shape(s) ? 0 : int8_workspace(s).total;
}

int moe_expert_swiglu_int8(moe_shape s, const int8_t* xq, const float* xs,
                           const int32_t* offsets, const int8_t* W1q, const float* s1,
                           const int8_t* W3q, const float* s3, const int8_t* W2q,
                           const float* s2, void* o, void* ws, size_t ws_bytes, void* stream) {
    return experts(s, xq, xs, offsets, Int8Experts{W1q, s1, W3q, s3, W2q, s2}, o, ws, ws_bytes, -1,
                   kDefaultWaitTimeoutNs, static_cast<cudaStream_t>(stream));
}

int moe_expert_swiglu_int8_stall_test(moe_shape s, const int8_t* xq, const float* xs,
                                      const int32_t* offsets, const int8_t* W1q,
                                      const float* s1, const int8_t* W3q, const float* s3,
                                      const int8_t* W2q, const float* s2, void* o, void* ws,
                                      size_t ws_bytes, int stall_after, uint64_t timeout_ns,
                                      void* stream) {
    if (stall_after < 0) return MOE_ERR_INVALID_ARG;
    if (timeout_ns < 1000 || timeout_ns > kDefaultWaitTimeoutNs) return MOE_ERR_INVALID_ARG;
    return experts(s, xq, xs, offsets, Int8Experts{W1q, s1, W3q, s3, W2q, s2}, o, ws, ws_bytes,
                   stall_after, timeout_ns, static_cast<cudaStream_t>(stream));
}

int moe_combine_bf16(moe_shape s, const void* o, const int32_t* inv, const float* gate, void* y,
                     void* stream) {
    const int rc = check_shape(s);
    if (rc || s.T == 0) return rc;
    if (!ok_ptr(o) || !ok_ptr(inv) || !ok_ptr(gate) || !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
    return launch_combine_bf16(s, o, inv, gate, y, static_cast<cudaStream_t>(stream));
}

size_t moe_forward_int8_workspace_bytes(moe_shape s) {
    return check_shape(s) ? 0 : layout(s).total;
}

int moe_forward_int8(moe_shape s, const void* x, const void* logits, int logits_type,
                     moe_scoring r, const float* route_bias, const uint8_t* mask,
                     const int8_t* W1q, const float* s1, const int8_t* W3q, const float* s3,
                     const int8_t* W2q, const float* s2, void* y, int32_t* idx_out,
                     float* gate_out, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_shape(s);
    if (rc == MOE_OK) rc = check_scoring(s, r);
    if (rc) return rc;
    if (!logits_type_ok(logits_type)) return MOE_ERR_INVALID_ARG;
    if (s.T == 0) return MOE_OK;
    if (!ok_ptr(x) || !ok_ptr(logits) || !ok_opt(route_bias) || !ok_opt(mask) || !ok_ptr(W1q) ||
        !ok_ptr(s1) || !ok_ptr(W3q) || !ok_ptr(s3) || !ok_ptr(W2q) || !ok_ptr(s2) || !ok_ptr(y) ||
        !ok_opt(idx_out) || !ok_opt(gate_out) || !ok_ptr(ws))
        return MOE_ERR_INVALID_ARG;
    const Layout L = layout(s);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t* idx = idx_out ? idx_out : at<int32_t>(ws, L.idx);
    float* gate = gate_out ? gate_out : at<float>(ws, L.gate);
    int32_t* offsets = at<int32_t>(ws, L.offsets);
    int32_t* inv = at<int32_t>(ws, L.inv);
    int8_t* xq = at<int8_t>(ws, L.xq);
    float* xs = at<float>(ws, L.xs);
    void* o = at<void>(ws, L.o);
    rc = launch_route_scored(s, r, logits, logits_type == MOE_LOGITS_BF16, route_bias, mask, idx,
                             gate, st);
    if (rc) return rc;
    // the row kernel also clears the status word and the tile counters
    rc = launch_dispatch_quantize(s, idx, x, offsets, at<int32_t>(ws, L.perm), inv, xq, xs,
                                  static_cast<uint32_t*>(ws),
                                  (int64_t)(int8_workspace(s).zero_bytes / 4), st);
    if (rc) return rc;
    rc = expert_products_int8(s, xq, xs, offsets, Int8Experts{W1q, s1, W3q, s3, W2q, s2}, o, ws,
                              static_cast<int*>(ws), kDefaultWaitTimeoutNs, -1, st);
    if (rc) return rc;
    return launch_combine_bf16(s, o, inv, gate, y, st);
}

}  // extern "C"
