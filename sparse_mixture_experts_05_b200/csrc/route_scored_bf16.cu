// route_scored_bf16.cu -- scored routing and its gradient for bf16 logits.
#include "route_scored_kernels.cuh"

namespace moe {
namespace scored {

template int route_for<__nv_bfloat16>(const moe_shape&, const moe_scoring&, const void*,
                                      const float*, const uint8_t*, int32_t*, float*, cudaStream_t);
template int backward_for<__nv_bfloat16>(const moe_shape&, const moe_scoring&, const void*,
                                         const int32_t*, const float*, void*, cudaStream_t);

}  // namespace scored
}  // namespace moe
