// What sv_policy.cu and sv_preference.cu share with each other.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/specverify.h"

namespace sv {

// The sizes, types, temperature and rows that the entry points over a row's
// token check alike; `grad` may be the logits themselves.
bool rows_ok(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits, const void* grad, float temperature);

// sv_token_logp without its checks; lse may be null.  `kept`, or null, takes what a
// gradient needs of a row later (.x to .z) and what the rounding of its logp left
// (.w), for sums of many.  `followed`: the next kernel on the stream waits for this
// one itself.
cudaError_t launch_token_logp(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                              float temperature, float* logp, float* entropy, float* lse, float4* kept, bool followed,
                              cudaStream_t s);
// The gradient from `kept`, d_rows rows with one d_logp, behind a kernel that is so
// followed.
cudaError_t launch_kept_grad(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                             const float4* kept, const float* d_logp, int d_rows, float temperature, void* grad,
                             cudaStream_t s);

}  // namespace sv
