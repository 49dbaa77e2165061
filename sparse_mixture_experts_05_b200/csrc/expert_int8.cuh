// expert_int8.cuh -- host entry of the experts' int8 products (expert_int8.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

struct Int8Experts {
    const int8_t* W1;
    const float* s1;
    const int8_t* W3;
    const float* s3;
    const int8_t* W2;
    const float* s2;
};

// Scratch of the two products: `zero_bytes` from its start (status word and tile
// counters) must be zero at launch.
struct Int8Workspace {
    size_t zero_bytes, cnt1, cnt2, part, hs, hq, h, total;
};
Int8Workspace int8_workspace(const moe_shape& s);

// x rows -> h (bf16) -> hq, hs -> o (bf16) over the expert groups of `offsets`.
// `err` is the device status word; `stall_after` >= 0 makes the producers stop
// after that many pipeline stages (test of the bounded waits).
int expert_products_int8(const moe_shape& s, const int8_t* xq, const float* xs,
                         const int32_t* offsets, const Int8Experts& w, void* o, void* ws, int* err,
                         uint64_t timeout_ns, int stall_after, cudaStream_t stream);

}  // namespace moe
