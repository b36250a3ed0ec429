// A loss of pairs of sequences, one preferred to the other, and its gradient in
// the logits, for sm_103a.
//
// With s_b the sum (or the mean) of a sequence's log-probabilities, a pair's
// h = (s_c - s_r) - (ref_c - ref_r) and m = beta h, the loss is
//   sigmoid  (1 - e) log(1 + e^-m) + e log(1 + e^m),  e the smoothing;
//   hinge    max(0, 1 - m);
//   ipo      (h - 1 / (2 beta))^2.
// Its derivative in a token's log-probability is that in h, with the other sign
// for the rejected sequence, divided by the tokens for the mean; from there on
// the gradient is that of sv_token.cuh.
//
// Three launches: the rows' log-probabilities, a CTA a pair, the rows' gradients, each
// launched before the one before it has ended.  A row is read twice, the second time
// from L2 where the pairs are few; 16 padded pairs of up to 64 rows of 128256 bf16 take
// 186 us, 5.1 TB/s of what crosses HBM.  One cooperative kernel that kept a pair's two
// readings together was slower (190 to 237 us): the pair's sums go round between them.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_device.cuh"
#include "sv_policy.h"

namespace sv {
namespace {

struct PairParams {
  const int* tokens;           // [2 n_pair, t_len]
  const float* logp;           // [2 n_pair, t_len]
  const float4* kept;          // [2 n_pair, t_len]: .w is what the rounding of logp left
  const float* ref;            // [2 n_pair]
  const float* weights;        // [n_pair]
  float *margin, *loss;        // [n_pair]
  float* d_logp;               // [2 n_pair], of each token of a sequence, or null
  int t_len, kind, average;
  float beta, smoothing;
};

constexpr int kPairThreads = 256, kPairWarps = kPairThreads / 32;

// log(1 + e^x) and 1 / (1 + e^-x).  The sums and h are taken in 64 bits, what
// follows, a few float32 steps of a float32 output, in 32: with 64-bit exponentials
// in every thread a pair took 14 us, in one thread the whole call 2 us more (23.6 for
// 21.7, which brought the loss from 2e-7 to 6e-8 of itself).
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.f, 1.f + expf(-x)); }

__global__ void __launch_bounds__(kPairThreads) pair_kernel(const __grid_constant__ PairParams P) {
  __shared__ double sums[2][kPairWarps];
  __shared__ int counts[2][kPairWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long i = blockIdx.x;
  grid_dependents_launch();      // (the gradient's rows wait for the end of this grid)
  grid_dependency_wait();
  for (int q = 0; q < 2; ++q) {
    const long long at = (2 * i + q) * P.t_len;
    double s = 0.0;
    int n = 0;
    for (int t = tid; t < P.t_len; t += kPairThreads) {
      s += static_cast<double>(P.logp[at + t]) + static_cast<double>(P.kept[at + t].w);
      n += P.tokens[at + t] >= 0;
    }
    s = warp_sum(s);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sums[q][warp] = s, counts[q][warp] = n;
  }
  __syncthreads();
  if (tid) return;
  double s[2] = {0.0, 0.0};
  int n[2] = {0, 0};
  for (int w = 0; w < kPairWarps; ++w)
    for (int q = 0; q < 2; ++q) s[q] += sums[q][w], n[q] += counts[q][w];
  float per[2] = {1.f, 1.f};
  if (P.average)
    for (int q = 0; q < 2; ++q)
      if (n[q] > 1) {
        s[q] /= n[q];
        per[q] = __fdiv_rn(1.f, static_cast<float>(n[q]));
      }
  const double h = (s[0] - s[1]) - (static_cast<double>(P.ref[2 * i]) - static_cast<double>(P.ref[2 * i + 1]));
  const float m = static_cast<float>(P.beta * h), e = P.smoothing, w = P.weights[i];
  float loss, slope;
  if (P.kind == SV_PREF_SIGMOID) {
    loss = (1.f - e) * softplus(-m);
    slope = -(1.f - e) * sigmoid(-m);
    if (e > 0.f) {
      loss = __fmaf_rn(e, softplus(m), loss);
      slope = __fmaf_rn(e, sigmoid(m), slope);
    }
    slope *= P.beta;
  } else if (P.kind == SV_PREF_HINGE) {
    const double room = 1.0 - P.beta * h;
    loss = room > 0.0 ? static_cast<float>(room) : m == m ? 0.f : m;
    slope = room > 0.0 ? -P.beta : m == m ? 0.f : m;
  } else {
    const double off = h - 0.5 / P.beta;
    loss = static_cast<float>(off * off);
    slope = static_cast<float>(2.0 * off);
  }
  P.margin[i] = m;
  P.loss[i] = w * loss;
  if (P.d_logp)
    for (int q = 0; q < 2; ++q) P.d_logp[2 * i + q] = (q ? -w : w) * slope * per[q];
}

}  // namespace
}  // namespace sv

extern "C" size_t sv_preference_work(int n_pair, int t_len) {
  // four floats of each row and each sequence's derivative
  return n_pair < 1 || t_len < 1 ? 0 : static_cast<size_t>(n_pair) * 2 * (4 * static_cast<size_t>(t_len) + 1);
}

extern "C" sv_status sv_preference_loss(int n_pair, int t_len, int V, sv_dtype dtype, const void* logits,
                                        const int32_t* tokens, const float* ref_logp, const float* weights,
                                        float temperature, float beta, int kind, float smoothing, int average,
                                        float* logp, float* margin, float* loss, void* grad, float* work,
                                        sv_stream_t stream) {
  using namespace sv;
  if (n_pair < 1 || n_pair > (1 << 27) || !tokens || !ref_logp || !weights || !logp || !margin || !loss || !work)
    return SV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(work) % 16) return SV_ERR_INVALID_ARG;
  if (!(beta > 0.f) || !std::isfinite(beta)) return SV_ERR_INVALID_ARG;
  if (kind != SV_PREF_SIGMOID && kind != SV_PREF_HINGE && kind != SV_PREF_IPO) return SV_ERR_INVALID_ARG;
  if (!(smoothing >= 0.f && smoothing < 0.5f) || (smoothing != 0.f && kind != SV_PREF_SIGMOID)) return SV_ERR_INVALID_ARG;
  if (average != 0 && average != 1) return SV_ERR_INVALID_ARG;
  const int n_seq = 2 * n_pair;
  if (!rows_ok(n_seq, t_len, V, dtype, logits, grad, temperature)) return SV_ERR_INVALID_ARG;
  NvtxRange range("sv_preference_loss");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rows = n_seq * t_len;
  float4* kept = reinterpret_cast<float4*>(work);
  float* d_logp = grad ? work + 4 * static_cast<size_t>(rows) : nullptr;
  if (launch_token_logp(rows, V, dtype, logits, tokens, temperature, logp, nullptr, nullptr, kept, true, s) != cudaSuccess)
    return SV_ERR_CUDA;
  const PairParams p{tokens, logp, kept, ref_logp, weights, margin, loss, d_logp, t_len, kind, average, beta, smoothing};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(n_pair));
  cfg.blockDim = dim3(kPairThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, pair_kernel, p) != cudaSuccess) return SV_ERR_CUDA;
  if (grad && launch_kept_grad(rows, V, dtype, logits, tokens, kept, d_logp, t_len, temperature, grad, s) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}
