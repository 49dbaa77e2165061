// int8_rows.cuh -- row kernels of the int8 layer (int8_rows.cu): per-expert token
// lists for many experts, quantised rows and channels, combine of bf16 outputs.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

// offsets, perm_tok and inv of moe_dispatch for up to 512 experts and 16 slots, and the
// rows of x quantised: xq[inv[t, s]], xs[inv[t, s]] for every slot s with a row.
// Zeroes `zero_words` 32-bit words at `zero` on the way (may be none).
int launch_dispatch_quantize(const moe_shape& s, const int32_t* idx, const void* x,
                             int32_t* offsets, int32_t* perm_tok, int32_t* inv, int8_t* xq,
                             float* xs, uint32_t* zero, int64_t zero_words, cudaStream_t stream);

// hq[r], hs[r] = row r of h [max_rows, cols] quantised, for r < *n_rows.
int launch_quantize_rows(const void* h, int max_rows, int cols, const int32_t* n_rows, int8_t* hq,
                         float* hs, cudaStream_t stream);

int launch_quantize_weights(int E, int K, int N, const void* W, int8_t* Wq, float* scale,
                            cudaStream_t stream);

int launch_combine_bf16(const moe_shape& s, const void* o, const int32_t* inv, const float* gate,
                        void* y, cudaStream_t stream);

}  // namespace moe
