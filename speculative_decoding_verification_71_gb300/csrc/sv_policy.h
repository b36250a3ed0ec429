// What sv_policy.cu and sv_preference.cu share with each other.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/specverify.h"

namespace sv {

// The sizes, types, temperature and rows that the entry points over a row's
// token check alike; `grad` may be the logits themselves.
bool rows_ok(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits, const void* grad, float temperature);

// sv_token_logp and sv_token_logp_grad without their checks.  `followed`: the next
// kernel on the stream waits for this one itself; `dependent`: the kernel before
// is so followed.  `d_rows` rows share a d_logp.  logp_rest, or null, takes what
// the rounding of logp left, for sums of many.
cudaError_t launch_token_logp(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                              float temperature, float* logp, float* entropy, float* lse, float* logp_rest, bool followed, cudaStream_t s);
cudaError_t launch_token_grad(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                              const float* logp, const float* lse, const float* entropy, const float* d_logp, int d_rows,
                              const float* d_entropy, float temperature, void* grad, bool dependent, cudaStream_t s);

}  // namespace sv
