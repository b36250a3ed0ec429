// Log-probabilities of a rollout's tokens, their gradient in the logits, and
// the clipped policy loss with its gradient, for sm_103a.
//
// The row's sums and the form of the gradient are those of sv_token.cuh.  With
// A the advantage, r = exp(log p(x) - log p_old(x)) and d = log p_ref(x) - log p(x)
// a row's loss is
//   -min(r A, clip(r, 1 - low, 1 + high) A)    (where A < 0 and `dual` is given, at most -dual A)
//   + kl (e^d - d - 1) - entropy H,
// and its derivative in log p(x) is -r A where the unclipped term is the smaller
// one (0 otherwise) plus kl (1 - e^d), that in H is -entropy.
//
// A CTA takes a row and reads it once for the sums and, for the gradient, again.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_kd.h"
#include "sv_rowsum.cuh"
#include "sv_token.cuh"

namespace sv {
namespace {

constexpr int kTokMaxRow = 1 << 20;        // bytes of a row

struct PolicyArgs {
  const float* advantages;     // [rows] or [rows / t_len]
  const float* weights;        // [rows / t_len]
  const float* old_logp;       // [rows] or null
  const float* ref_logp;       // [rows] or null
  int per_token;
  float low, high, dual, kl, entropy;
};

struct RowParams {
  const unsigned char* logits; // [rows, V]
  const int* tokens;           // [rows]
  float *logp, *entropy, *lse; // [rows]; entropy and lse or null
  float* row_loss;             // [rows]: a policy's loss; null for the log-probabilities alone
  unsigned char* grad;         // [rows, V] or null
  int t_len, V;
  int same_shift;              // logits and grad lie alike: 16-byte stores
  float c2, inv_T;             // log2(e) / T, 1 / T
  PolicyArgs policy;
};

// (e^d - d - 1), without cancellation where d is small.
__device__ __forceinline__ float kl_term(float d) {
  if (d == INFINITY) return d;             // a token that the policy cannot say
  if (!(fabsf(d) <= 0.125f)) return __fsub_rn(expm1f(d), d);
  // d^2 (1/2 + d/6 + ... + d^4/720): the next term is below 2e-9 of it
  float s = __fmaf_rn(d, 1.f / 720.f, 1.f / 120.f);
  s = __fmaf_rn(d, s, 1.f / 24.f);
  s = __fmaf_rn(d, s, 1.f / 6.f);
  s = __fmaf_rn(d, s, 0.5f);
  return d * d * s;
}

// A row's loss and its derivative in the token's log-probability.
__device__ __forceinline__ void policy_row(const PolicyArgs& P, float A, float old_logp, float ref_logp, const TokRow& R,
                                           float& loss, float& slope) {
  const float r = P.old_logp ? expf(__fsub_rn(R.logp, old_logp)) : 1.f;
  const float low = 1.f - P.low, high = 1.f + P.high;
  const float gained = r * A, held = (r < low ? low : r > high ? high : r) * A;
  float gain = gained <= held ? gained : held;
  slope = gained <= held ? -gained : 0.f;
  if (!(gained == gained)) gain = slope = NAN;
  if (P.dual > 0.f && A < 0.f && gain < P.dual * A) {
    gain = P.dual * A;
    slope = 0.f;
  }
  loss = -gain;
  if (P.ref_logp) {
    const float d = __fsub_rn(ref_logp, R.logp);
    loss = __fmaf_rn(P.kl, kl_term(d), loss);
    slope = __fmaf_rn(-P.kl, expm1f(d), slope);
  }
  if (P.entropy != 0.f) loss = __fmaf_rn(-P.entropy, R.H, loss);
}

constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;

template <int ELT>
__device__ __forceinline__ void zero_row(unsigned char* grad, int V, int shift, int nvec, int same_shift) {
  for (int v = threadIdx.x; v < nvec; v += blockDim.x)
    store_edge<ELT>(grad, V, v * Vec<ELT>::N - shift, same_shift, make_uint4(0, 0, 0, 0));
}

template <int ELT, bool ENT>
__device__ __forceinline__ void write_gradient(const unsigned char* row, unsigned char* grad, int V, int shift, int nvec,
                                               int same_shift, int x, const TokGrad& G, float c2) {
  constexpr int N = Vec<ELT>::N;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const uint4 w = load_row_vec<ELT>(row, V, shift, v);
    store_edge<ELT>(grad, V, v * N - shift, same_shift, tok_vec_grad<ELT, ENT>(w, G, c2, x + shift - v * N));
  }
}

template <int ELT, bool ENT, bool GRAD>
__global__ void __launch_bounds__(kRowThreads) token_row_kernel(const __grid_constant__ RowParams P) {
  constexpr int N = Vec<ELT>::N;
  __shared__ TokPart parts[kRowWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x;
  const unsigned char* row = P.logits + r * P.V * ELT;
  unsigned char* grad = GRAD ? P.grad + r * P.V * ELT : nullptr;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  if (P.row_loss) grid_dependents_launch();   // the sum of the rows may take its place on an SM
  const int x = P.tokens[r];
  if (x < 0) {
    if (tid == 0) {
      P.logp[r] = 0.f;
      if (P.entropy) P.entropy[r] = 0.f;
      if (P.lse) P.lse[r] = -INFINITY;
      if (P.row_loss) P.row_loss[r] = 0.f;
    }
    if (GRAD) zero_row<ELT>(grad, P.V, shift, nvec, P.same_shift);
    return;
  }
  const float zx = x < P.V ? load_elem<ELT>(row, x) : NAN;
  TokSum<ELT, ENT> sum;
  for (int v = tid; v < nvec; v += kRowThreads) {
    uint4 w[1] = {load_row_vec<ELT>(row, P.V, shift, v)};
    tok_take_out<ELT>(w[0], x + shift - v * N);
    sum.add(w, P.c2);
  }
  TokPart part = tok_join<ENT>(sum.part(), P.c2);
  if (lane == 0) parts[warp] = part;
  __syncthreads();
  part = tok_join<ENT>(lane < kRowWarps ? parts[lane] : tok_none(), P.c2);
  const TokRow R = tok_row<ENT>(part, zx, P.inv_T);
  float loss = 0.f, slope = 0.f;
  if (P.row_loss) {
    const PolicyArgs& a = P.policy;
    policy_row(a, a.advantages[a.per_token ? r : r / P.t_len], a.old_logp ? a.old_logp[r] : 0.f,
               a.ref_logp ? a.ref_logp[r] : 0.f, R, loss, slope);
  }
  if (tid == 0) {
    P.logp[r] = R.logp;
    if (ENT && P.entropy) P.entropy[r] = R.H;
    if (P.lse) P.lse[r] = R.lse;
    if (P.row_loss) P.row_loss[r] = loss;
  }
  if (GRAD) {
    const float w = P.policy.weights[r / P.t_len];
    const TokGrad G = tok_grad(R, w * slope, ENT ? -P.policy.entropy * w : 0.f, P.inv_T);
    __syncthreads();             // (in place: every thread has read the row)
    write_gradient<ELT, ENT>(row, grad, P.V, shift, nvec, P.same_shift, x, G, P.c2);
  }
}

struct GradParams {
  const unsigned char* logits;
  const int* tokens;
  const float *logp, *lse, *entropy, *d_logp, *d_entropy;   // [rows]; the entropies or null
  unsigned char* grad;
  int V, same_shift;
  float c2, inv_T;
};

template <int ELT, bool ENT>
__global__ void __launch_bounds__(kRowThreads) token_grad_kernel(const __grid_constant__ GradParams P) {
  const long long r = blockIdx.x;
  const unsigned char* row = P.logits + r * P.V * ELT;
  unsigned char* grad = P.grad + r * P.V * ELT;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  const int x = P.tokens[r];
  TokGrad G;
  G.none();
  if (x >= 0) {
    const float zx = x < P.V ? load_elem<ELT>(row, x) : NAN;
    G = tok_grad_from(zx, x < P.V ? P.logp[r] : NAN, P.lse[r], ENT ? P.entropy[r] : 0.f, P.d_logp[r],
                      ENT ? P.d_entropy[r] : 0.f, P.inv_T);
  }
  __syncthreads();               // (in place: every thread has the token's logit)
  if (G.zero()) zero_row<ELT>(grad, P.V, shift, nvec, P.same_shift);
  else write_gradient<ELT, ENT>(row, grad, P.V, shift, nvec, P.same_shift, x, G, P.c2);
}

template <int ELT>
cudaError_t launch_rows(const RowParams& p, int rows, bool ent, cudaStream_t s) {
  const unsigned n = static_cast<unsigned>(rows);
  if (p.grad) {
    if (ent) token_row_kernel<ELT, true, true><<<n, kRowThreads, 0, s>>>(p);
    else token_row_kernel<ELT, false, true><<<n, kRowThreads, 0, s>>>(p);
  } else {
    if (ent) token_row_kernel<ELT, true, false><<<n, kRowThreads, 0, s>>>(p);
    else token_row_kernel<ELT, false, false><<<n, kRowThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

// The sizes, types, temperature and rows that every entry point here checks
// alike; `grad` may be the logits themselves.
bool rows_ok(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits, const void* grad, float temperature) {
  if (n_seq < 1 || t_len < 1 || V < 1 || static_cast<long long>(n_seq) * t_len > (1LL << 28)) return false;
  if (dtype != SV_F32 && dtype != SV_BF16) return false;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return false;
  if (!(1.4426950408889634 / static_cast<double>(temperature) < 1e30) || !(1.f / temperature > 0.f)) return false;
  const int elt = dtype == SV_F32 ? 4 : 2;
  if (!logits || static_cast<long long>(V) * elt > kTokMaxRow) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(logits), g = reinterpret_cast<uintptr_t>(grad);
  if (a % elt || g % elt) return false;
  const uintptr_t bytes = static_cast<uintptr_t>(n_seq) * t_len * V * elt;
  return !(grad && a != g && a < g + bytes && g < a + bytes);
}

RowParams row_params(int t_len, int V, const void* logits, const int32_t* tokens, float temperature, void* grad) {
  RowParams p{};
  p.logits = static_cast<const unsigned char*>(logits);
  p.tokens = tokens;
  p.grad = static_cast<unsigned char*>(grad);
  p.t_len = t_len;
  p.V = V;
  p.same_shift = reinterpret_cast<uintptr_t>(logits) % 16 == reinterpret_cast<uintptr_t>(grad) % 16;
  p.c2 = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
  p.inv_T = 1.f / temperature;
  return p;
}

}  // namespace
}  // namespace sv

extern "C" sv_status sv_token_logp(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits,
                                   const int32_t* tokens, float temperature, float* logp, float* entropy, float* lse,
                                   sv_stream_t stream) {
  using namespace sv;
  if (!rows_ok(n_seq, t_len, V, dtype, logits, nullptr, temperature) || !tokens || !logp || !lse)
    return SV_ERR_INVALID_ARG;
  RowParams p = row_params(t_len, V, logits, tokens, temperature, nullptr);
  p.logp = logp;
  p.entropy = entropy;
  p.lse = lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_token_logp");
  const cudaError_t e = dtype == SV_BF16 ? launch_rows<2>(p, n_seq * t_len, entropy != nullptr, s)
                                         : launch_rows<4>(p, n_seq * t_len, entropy != nullptr, s);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status sv_token_logp_grad(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits,
                                        const int32_t* tokens, const float* logp, const float* lse,
                                        const float* entropy, const float* d_logp, const float* d_entropy,
                                        float temperature, void* grad, sv_stream_t stream) {
  using namespace sv;
  if (!rows_ok(n_seq, t_len, V, dtype, logits, grad, temperature) || !tokens || !logp || !lse || !d_logp || !grad)
    return SV_ERR_INVALID_ARG;
  if (!entropy != !d_entropy) return SV_ERR_INVALID_ARG;
  const RowParams q = row_params(t_len, V, logits, tokens, temperature, grad);
  const GradParams p{q.logits, tokens, logp, lse, entropy, d_logp, d_entropy, q.grad, V, q.same_shift, q.c2, q.inv_T};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_token_logp_grad");
  const unsigned n = static_cast<unsigned>(n_seq) * static_cast<unsigned>(t_len);
  if (dtype == SV_BF16) {
    if (entropy) token_grad_kernel<2, true><<<n, kRowThreads, 0, s>>>(p);
    else token_grad_kernel<2, false><<<n, kRowThreads, 0, s>>>(p);
  } else {
    if (entropy) token_grad_kernel<4, true><<<n, kRowThreads, 0, s>>>(p);
    else token_grad_kernel<4, false><<<n, kRowThreads, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status sv_policy_loss(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits,
                                    const int32_t* tokens, const float* advantages, int per_token,
                                    const float* weights, const float* old_logp, const float* ref_logp,
                                    float temperature, float clip_low, float clip_high, float dual_clip,
                                    float kl_coef, float entropy_coef, float* logp, float* entropy, float* row_loss,
                                    float* loss, void* grad, sv_stream_t stream) {
  using namespace sv;
  if (!rows_ok(n_seq, t_len, V, dtype, logits, grad, temperature)) return SV_ERR_INVALID_ARG;
  if (!tokens || !advantages || !weights || !logp || !row_loss || !loss) return SV_ERR_INVALID_ARG;
  if (per_token != 0 && per_token != 1) return SV_ERR_INVALID_ARG;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !std::isfinite(clip_high)) return SV_ERR_INVALID_ARG;
  if (!(dual_clip == 0.f || dual_clip > 1.f) || !std::isfinite(dual_clip)) return SV_ERR_INVALID_ARG;
  if (!std::isfinite(kl_coef) || !std::isfinite(entropy_coef) || (kl_coef != 0.f && !ref_logp)) return SV_ERR_INVALID_ARG;
  RowParams p = row_params(t_len, V, logits, tokens, temperature, grad);
  p.logp = logp;
  p.entropy = entropy;
  p.row_loss = row_loss;
  p.policy = PolicyArgs{advantages, weights, old_logp, kl_coef != 0.f ? ref_logp : nullptr, per_token,
                        clip_low, clip_high, dual_clip, kl_coef, entropy_coef};
  const bool ent = entropy || entropy_coef != 0.f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_policy_loss");
  const int rows = n_seq * t_len;
  const cudaError_t e = dtype == SV_BF16 ? launch_rows<2>(p, rows, ent, s) : launch_rows<4>(p, rows, ent, s);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  return launch_row_sum(n_seq, t_len, row_loss, weights, loss, s) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
