// loss[b] = w_b * sum_t row_loss[b, t], what the losses over logit rows end with.
#pragma once

#include "sv_device.cuh"

namespace sv {
namespace {

// In 64 bits and a fixed order: by a warp, by all warps of a CTA where
// positions are many (one rollout of 4096: 3 us, by one thread 300).
constexpr int kRowSumThreads = 256, kRowSumWarps = kRowSumThreads / 32;
constexpr int kRowSumMany = 256;
__global__ void __launch_bounds__(kRowSumThreads) row_sum_kernel(int n_seq, int t_len, const float* row_loss,
                                                                 const float* weights, float* loss) {
  __shared__ double parts[kRowSumWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool many = t_len > kRowSumMany;
  const int b = many ? blockIdx.x : static_cast<int>(blockIdx.x) * kRowSumWarps + warp;
  const int step = many ? kRowSumThreads : 32;
  grid_dependency_wait();
  double s = 0.0;
  if (b < n_seq) {
    const float* row = row_loss + static_cast<long long>(b) * t_len;
#pragma unroll 8
    for (int t = many ? static_cast<int>(threadIdx.x) : lane; t < t_len; t += step) s += static_cast<double>(row[t]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (many) {
    if (lane == 0) parts[warp] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < kRowSumWarps; ++w) s += parts[w];
  }
  if (b < n_seq && (many ? threadIdx.x == 0 : lane == 0)) loss[b] = static_cast<float>(static_cast<double>(weights[b]) * s);
}

// Launched behind the rows' kernel, which may let it take its place early.
inline cudaError_t launch_row_sum(int n_seq, int t_len, const float* row_loss, const float* weights, float* loss,
                                  cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(t_len > kRowSumMany ? n_seq : (n_seq + kRowSumWarps - 1) / kRowSumWarps));
  cfg.blockDim = dim3(kRowSumThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, row_sum_kernel, n_seq, t_len, row_loss, weights, loss);
}

}  // namespace
}  // namespace sv
