// route_scored.cuh -- scored routing and its gradient (route_scored.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

constexpr int kScoredMaxE = 512;
constexpr int kScoredMaxK = 16;
constexpr int kScoredMaxGroups = 32;

// Arguments of the kernels that are the same for every row; checked by the caller.
int launch_route_scored(const moe_shape& s, const moe_scoring& r, const void* logits,
                        bool logits_bf16, const float* bias, const uint8_t* mask, int32_t* idx,
                        float* gate, cudaStream_t stream);

int launch_route_scored_backward(const moe_shape& s, const moe_scoring& r, const void* logits,
                                 bool logits_bf16, const int32_t* idx, const float* dgate,
                                 void* dlogits, cudaStream_t stream);

}  // namespace moe
