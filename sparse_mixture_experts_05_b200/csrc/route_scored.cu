// route_scored.cu -- scored routing and its gradient: float logits, and the choice of the
// logits' type.  The kernels are in route_scored_kernels.cuh; route_scored_bf16.cu compiles
// them for bf16 logits (two files, because together they compile for minutes).
#include "route_scored_kernels.cuh"

namespace moe {

namespace scored {
extern template int route_for<__nv_bfloat16>(const moe_shape&, const moe_scoring&, const void*,
                                             const float*, const uint8_t*, int32_t*, float*,
                                             cudaStream_t);
extern template int backward_for<__nv_bfloat16>(const moe_shape&, const moe_scoring&, const void*,
                                                const int32_t*, const float*, void*, cudaStream_t);
}  // namespace scored

int launch_route_scored(const moe_shape& s, const moe_scoring& r, const void* logits,
                        bool logits_bf16, const float* bias, const uint8_t* mask, int32_t* idx,
                        float* gate, cudaStream_t stream) {
    return logits_bf16
               ? scored::route_for<__nv_bfloat16>(s, r, logits, bias, mask, idx, gate, stream)
               : scored::route_for<float>(s, r, logits, bias, mask, idx, gate, stream);
}

int launch_route_scored_backward(const moe_shape& s, const moe_scoring& r, const void* logits,
                                 bool logits_bf16, const int32_t* idx, const float* dgate,
                                 void* dlogits, cudaStream_t stream) {
    return logits_bf16
               ? scored::backward_for<__nv_bfloat16>(s, r, logits, idx, dgate, dlogits, stream)
               : scored::backward_for<float>(s, r, logits, idx, dgate, dlogits, stream);
}

}  // namespace moe
