// Distillation of the drafter from a teacher's top log-probabilities: the
// loss and its gradient in the draft logits, for sm_103a.
//
// A row's list holds ids x_j and log p_j; with q = softmax(z / T) of the draft
// row, w the rollout's weight, P = sum p_j and Q = sum q(x_j):
//   tail    r = 1 - P;  KL = sum p_j (log p_j - log q(x_j)) + r (log r - log(1 - Q))
//           dL/dz(x_j) = w (q(x_j) - p_j) / T,  dL/dz(x) = w q(x) (1 - r / (1 - Q)) / T else
//   renorm  the same with p_j / P in place of p_j and r = 0.
// 1 - Q would cancel where the drafter is sure, so the row is summed apart:
// the tokens that are not listed against their own maximum M,
// S = sum 2^((z - M) c) with c = log2(e) / T, the listed ones from their own
// logits.  So with E = 2^((z - M) c) the gradient of an unlisted token is one multiply,
// E * w / T * (1 / Z - r / S), Z the row's whole sum scaled alike.
//
// A CTA takes a row: it marks the listed tokens in a shared-memory bitmap and
// gathers their logits, streams the row for (M, S), and streams it again for
// the gradient; then the listed tokens' own gradients are stored over it.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kTlThreads = 512;
constexpr int kTlWarps = kTlThreads / 32;
constexpr int kTlMaxV = 524288;
// a tail mass below this is rounding: float32 log-probabilities tell no less
constexpr float kTlComplete = 1.f / 1048576.f;

struct TopLossParams {
  const int* ids;              // [rows, K]
  const float* logp;           // [rows, K]
  const unsigned char* draft;  // [rows, V]
  const float* weights;        // [rows / t_len]
  float* row_kl;               // [rows]
  unsigned char* grad;         // [rows, V] or null
  int t_len, V, K;
  int renorm;
  int same_shift;              // draft and grad lie alike: 16-byte stores
  float c2, T, inv_T;
};

struct TlShared {
  float wm[kTlWarps], ws[kTlWarps];
  float red[4][kTlWarps];
  int bad, used;
};

// The sum (or maximum) of a value over the CTA, the same in every thread, in
// a fixed order.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, x) : v + x;
  }
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = slot[0];
  for (int w = 1; w < kTlWarps; ++w) r = MAX ? fmaxf(r, slot[w]) : r + slot[w];
  __syncthreads();
  return r;
}

template <int ELT>
__device__ __forceinline__ void fill_row(unsigned char* out, int V, float value) {
  for (int t = threadIdx.x; t < V; t += kTlThreads) Vec<ELT>::store_rounded(out, t, value);
}

template <int ELT>
__global__ void __launch_bounds__(kTlThreads) toploss_kernel(const TopLossParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  extern __shared__ uint32_t bitmap[];   // [V / 32 + 2], from 8 tokens before the row on
  __shared__ TlShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x;
  const unsigned char* row = P.draft + r * P.V * ELT;
  unsigned char* grad = P.grad ? P.grad + r * P.V * ELT : nullptr;

  // ---- the list: thread j holds entry j
  int id = -1;
  float lp = -INFINITY;
  if (tid < P.K) {
    id = P.ids[r * P.K + tid];
    lp = P.logp[r * P.K + tid];
  }
  const int words = (P.V + 8 + 31) / 32 + 1;
  for (int w = tid; w < words; w += kTlThreads) bitmap[w] = 0;
  if (tid == 0) sh.bad = 0, sh.used = 0;
  __syncthreads();
  float zj = -INFINITY;
  if (lp != lp || lp == INFINITY || id >= P.V) sh.bad = 1;
  if (id >= P.V) id = -1;
  if (id >= 0) {
    sh.used = 1;
    const int u = id + 8;
    if (atomicOr(&bitmap[u >> 5], 1u << (u & 31)) & (1u << (u & 31))) sh.bad = 1;   // listed twice
    zj = load_elem<ELT>(row, id);
    if (zj != zj || zj == INFINITY) sh.bad = 1;
  }
  __syncthreads();
  if (!sh.bad && !sh.used) {   // no list: no loss
    if (tid == 0) P.row_kl[r] = 0.f;
    if (grad) fill_row<ELT>(grad, P.V, 0.f);
    return;
  }

  // ---- the unlisted tokens: running maximum and sum
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  float m = -INFINITY, base = 0.f, s = 0.f;
  for (int v = tid; v < nvec; v += kTlThreads) {
    float z[N];
    VT::unpack(load_row_vec<ELT>(row, P.V, shift, v), z);
    const uint32_t in_list = bits_at<N>(bitmap, v * N - shift + 8);
    if (in_list) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if ((in_list >> e) & 1u) z[e] = -INFINITY;
    }
    float vm = z[0];
#pragma unroll
    for (int e = 1; e < N; ++e) vm = fmaxf(vm, z[e]);
    if (vm > m) {
      s = m == -INFINITY ? 0.f : s * fast_exp2(__fmul_rn(__fsub_rn(m, vm), P.c2));
      m = base = vm;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) s += fast_exp2(__fmul_rn(__fsub_rn(z[e], base), P.c2));
  }
  if (s != s) m = NAN;
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmax_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  float ws = m > -INFINITY ? s * fast_exp2(__fmul_rn(__fsub_rn(m, wm), P.c2)) : 0.f;
  ws = warp_sum(ws);
  if (lane == 0) sh.wm[warp] = wm, sh.ws[warp] = ws;
  __syncthreads();
  float M = -INFINITY, S = 0.f;
  for (int w = 0; w < kTlWarps; ++w) M = fmax_nan(M, sh.wm[w]);
  for (int w = 0; w < kTlWarps; ++w)
    if (sh.wm[w] > -INFINITY) S += sh.ws[w] * fast_exp2(__fmul_rn(__fsub_rn(sh.wm[w], M), P.c2));

  // ---- the listed tokens, and the whole row against Ma = max(M, Ml)
  const float Ml = cta_reduce<true>(zj, sh.red[0]);
  const float Ma = fmaxf(M, Ml);
  const bool valid = !sh.bad && M == M && M < INFINITY && S == S && Ma > -INFINITY;
  // the listed tokens carry most of Z: full-precision exponentials for them
  const float lj = __fdiv_rn(__fsub_rn(zj, Ma), P.T);
  const float ej = zj > -INFINITY ? expf(lj) : 0.f;
  const float Sl = cta_reduce<false>(ej, sh.red[1]);
  const float lt = __fdiv_rn(__fsub_rn(M, Ma), P.T);
  const float ft = M > -INFINITY ? expf(lt) : 0.f;
  const float Z = __fadd_rn(__fmul_rn(S, ft), Sl), LZ = logf(Z);
  float p = id >= 0 ? expf(lp) : 0.f;
  const float mass = cta_reduce<false>(p, sh.red[2]);
  float rest = 0.f;
  if (P.renorm) {
    lp = mass > 0.f ? __fsub_rn(lp, logf(mass)) : -INFINITY;
    p = mass > 0.f ? __fdiv_rn(p, mass) : 0.f;
  } else {
    rest = __fsub_rn(1.f, mass);
    if (rest < kTlComplete) rest = 0.f;
  }
  float term = 0.f;
  if (p > 0.f) term = __fmul_rn(p, __fsub_rn(lp, __fsub_rn(lj, LZ)));
  float kl = cta_reduce<false>(term, sh.red[3]);
  if (rest > 0.f)
    kl = S > 0.f ? kl + rest * (logf(rest) - __fsub_rn(__fadd_rn(lt, logf(S)), LZ)) : INFINITY;
  if (tid == 0) P.row_kl[r] = valid ? kl : NAN;
  if (!grad) return;
  if (!valid) {
    fill_row<ELT>(grad, P.V, NAN);
    return;
  }

  // ---- the gradient
  const float scale = P.weights[r / P.t_len] * P.inv_T;
  const float tail_base = M > -INFINITY ? M : 0.f;
  const float a = scale * __fsub_rn(__fdiv_rn(ft, Z), S > 0.f ? __fdiv_rn(rest, S) : 0.f);
  for (int v = tid; v < nvec; v += kTlThreads) {
    float z[N];
    VT::unpack(load_row_vec<ELT>(row, P.V, shift, v), z);
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = a * fast_exp2(__fmul_rn(__fsub_rn(z[e], tail_base), P.c2));
    const int t0 = v * N - shift;
    if (P.same_shift && t0 >= 0 && t0 <= P.V - N) {
      store_vec16(grad + static_cast<long long>(t0) * ELT, VT::pack(z));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (t0 + e >= 0 && t0 + e < P.V) VT::store_rounded(grad, t0 + e, z[e]);
    }
  }
  __syncthreads();   // the listed tokens' stores come after
  if (id >= 0) VT::store_rounded(grad, id, scale * __fsub_rn(__fdiv_rn(ej, Z), p));
}

// loss[b] = w_b * sum_t row_kl[b, t], in position order.
__global__ void toploss_sum_kernel(int n_seq, int t_len, const float* row_kl, const float* weights, float* loss) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= n_seq) return;
  double s = 0.0;
  for (int t = 0; t < t_len; ++t) s += static_cast<double>(row_kl[static_cast<long long>(b) * t_len + t]);
  loss[b] = static_cast<float>(static_cast<double>(weights[b]) * s);
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_kd_top_loss(int n_seq, int t_len, int V, sv_dtype dtype, int K, const int32_t* ids,
                                      const float* logp, const void* draft_logits, const float* weights,
                                      float temperature, int mode, float* row_kl, float* loss, void* grad,
                                      sv_stream_t stream) {
  using namespace sv;
  if (n_seq < 1 || t_len < 1 || V < 1 || V > kTlMaxV || K < 1 || K > SV_KD_TOP_MAX) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(n_seq) * t_len > (1LL << 30)) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (mode != SV_KD_TOP_TAIL && mode != SV_KD_TOP_RENORM) return SV_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SV_ERR_INVALID_ARG;
  if (!ids || !logp || !draft_logits || !weights || !row_kl || !loss) return SV_ERR_INVALID_ARG;
  const int elt = dtype == SV_F32 ? 4 : 2;
  const uintptr_t a = reinterpret_cast<uintptr_t>(draft_logits), g = reinterpret_cast<uintptr_t>(grad);
  if (a % elt || g % elt) return SV_ERR_INVALID_ARG;
  const uintptr_t bytes = static_cast<uintptr_t>(n_seq) * t_len * V * elt;
  if (grad && a < g + bytes && g < a + bytes) return SV_ERR_INVALID_ARG;
  const double c2 = 1.4426950408889634 / static_cast<double>(temperature);
  if (!(c2 < 1e30)) return SV_ERR_INVALID_ARG;
  TopLossParams p{ids, logp, static_cast<const unsigned char*>(draft_logits), weights, row_kl,
                  static_cast<unsigned char*>(grad), t_len, V, K, mode == SV_KD_TOP_RENORM, (a % 16) == (g % 16),
                  static_cast<float>(c2), temperature, 1.f / temperature};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("spec_kd_top_loss");
  const int rows = n_seq * t_len, smem = 4 * ((V + 8 + 31) / 32 + 1);
  auto launch = [&](auto kernel) {
    if (smem > 48 * 1024 - static_cast<int>(sizeof(TlShared)) &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (kTlMaxV / 32 + 4)) != cudaSuccess)
      return SV_ERR_CUDA;
    kernel<<<rows, kTlThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  };
  const sv_status st = elt == 2 ? launch(toploss_kernel<2>) : launch(toploss_kernel<4>);
  if (st != SV_OK) return st;
  toploss_sum_kernel<<<(n_seq + 127) / 128, 128, 0, s>>>(n_seq, t_len, row_kl, weights, loss);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
