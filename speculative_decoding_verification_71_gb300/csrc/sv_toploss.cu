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
// A row goes to a cluster of up to 8 CTAs and stays in their registers: every
// thread loads its vectors of the row once, the cluster exchanges each part's
// (M, S) of the unlisted tokens and the same of the listed ones through
// distributed shared memory, and the gradient is stored from the registers.
// Each logit crosses HBM once and each gradient once, with no second read.
// The listed tokens are marked in a bitmap of the part and gathered by a
// thread each, which stores their gradients after the row's.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kTlMaxRow = 1 << 20;        // bytes of a row
constexpr int kTlMaxCtas = 8;
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

// A part's sums: the unlisted tokens' about their maximum m, the listed ones'
// about theirs.
struct alignas(16) TlPart {
  float m, s, ml, sl;
};

// What the whole row comes to.
struct TlRow {
  float a, base;               // an unlisted token's gradient is a 2^((z - base) c)
  float Ma, Z, LZ, mass;       // the row's maximum, its sum about it and the logarithm, P
  float kl;                    // the unlisted tokens' term
  int valid;
};

template <int WARPS>
struct TlShared {
  TlPart part[kTlMaxCtas];     // the cluster's CTAs'
  TlPart warp[WARPS];
  float mass[WARPS];           // the warps' parts of P
  float term[WARPS];           // ... of the listed tokens' divergence
  float kl[kTlMaxCtas];        // (first CTA) the CTAs' parts of it
  TlRow row;
};

__device__ __forceinline__ void tl_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void tl_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The parts of all lanes on their common maxima, the same in every lane and in
// a fixed order; a NaN among the sums stays.
__device__ __forceinline__ TlPart tl_combine(const TlPart& p, float c2, float inv_T) {
  TlPart r;
  r.m = from_ordered_key(__reduce_max_sync(0xffffffffu, ordered_key(p.m)));
  r.ml = from_ordered_key(__reduce_max_sync(0xffffffffu, ordered_key(p.ml)));
  // (a NaN sum with its maximum at -inf is kept too)
  r.s = warp_sum(p.m > -INFINITY ? p.s * fast_exp2(__fmul_rn(__fsub_rn(p.m, r.m), c2)) : p.s);
  r.sl = warp_sum(p.ml > -INFINITY ? p.sl * expf(__fmul_rn(__fsub_rn(p.ml, r.ml), inv_T)) : p.sl);
  return r;
}

// A vector with -inf in the places of `bits`.
template <int ELT>
__device__ __noinline__ uint4 with_neg_inf(uint4 w, uint32_t bits) {
  constexpr int N = Vec<ELT>::N;
  float z[N];
  Vec<ELT>::unpack(w, z);
#pragma unroll
  for (int e = 0; e < N; ++e)
    if ((bits >> e) & 1u) z[e] = -INFINITY;
  return Vec<ELT>::pack(z);
}

// A vector's gradients where it may reach past its row, or the rows lie unlike.
template <int ELT>
__device__ __noinline__ void store_edge(unsigned char* grad, int V, int t0, int same_shift, const float (&g)[Vec<ELT>::N]) {
  constexpr int N = Vec<ELT>::N;
  if (same_shift && t0 >= 0 && t0 <= V - N) {
    store_vec16(grad + static_cast<long long>(t0) * ELT, Vec<ELT>::pack(g));
    return;
  }
  for (int e = 0; e < N; ++e)
    if (t0 + e >= 0 && t0 + e < V) Vec<ELT>::store_rounded(grad, t0 + e, g[e]);
}

// NV vectors of the row per thread, in registers throughout.
template <int ELT, int THREADS, int NV, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) toploss_kernel(const __grid_constant__ TopLossParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N, kWarps = THREADS / 32;
  __shared__ TlShared<kWarps> sh;
  __shared__ alignas(16) uint32_t listed_words[(THREADS * NV + 15) / 16 * 4];
  uint8_t* listed = reinterpret_cast<uint8_t*>(listed_words);   // a bit per token of a vector: listed
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster_ctas(), rank = cluster_rank();
  const long long r = blockIdx.x / ctas;
  const unsigned char* row = P.draft + r * P.V * ELT;
  unsigned char* grad = P.grad ? P.grad + r * P.V * ELT : nullptr;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  const int per = (nvec + ctas - 1) / ctas;
  const int v0 = min(nvec, rank * per), v1 = min(nvec, v0 + per);
  const int t_first = v0 * N - shift;      // token of the part's first element
  // whether the part is of whole vectors only
  const bool whole = t_first >= 0 && v1 * N - shift <= P.V;
  const int n = v1 - v0 - tid;             // this thread's vectors: q THREADS < n

  // ---- the list: thread j holds entries j and j + THREADS
  constexpr int kE = (SV_KD_TOP_MAX + THREADS - 1) / THREADS;
  int id[kE];
  float lp[kE];
  bool bad = false, any = false;
#pragma unroll
  for (int k = 0; k < kE; ++k) {
    const int j = tid + k * THREADS;
    id[k] = j < P.K ? P.ids[r * P.K + j] : -1;
    lp[k] = j < P.K ? P.logp[r * P.K + j] : -INFINITY;
  }
  for (int w = tid; w < (per + 15) / 16; w += THREADS) reinterpret_cast<uint4*>(listed_words)[w] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < kE; ++k) {
    bad |= lp[k] != lp[k] || lp[k] == INFINITY || id[k] >= P.V;
    if (id[k] >= P.V) id[k] = -1;
    any |= id[k] >= 0;
  }
  // a row without a list is not read and has no loss
  if (!__syncthreads_or(any || bad)) {
    if (rank == 0 && tid == 0) P.row_kl[r] = 0.f;
    if (grad)
      for (int v = v0 + tid; v < v1; v += THREADS) {
        const int t0 = v * N - shift;
        if (P.same_shift && t0 >= 0 && t0 <= P.V - N) {
          store_vec16(grad + static_cast<long long>(t0) * ELT, make_uint4(0, 0, 0, 0));
        } else {
          for (int e = 0; e < N; ++e)
            if (t0 + e >= 0 && t0 + e < P.V) VT::store_rounded(grad, t0 + e, 0.f);
        }
      }
    return;
  }
  uint4 w[NV];
  if (whole) {
    const unsigned char* at = row + (static_cast<long long>(v0 + tid) * N - shift) * ELT;
#pragma unroll
    for (int q = 0; q < NV; ++q) w[q] = q * THREADS < n ? load_vec16(at + q * THREADS * 16) : VT::neg_inf();
  } else {
#pragma unroll
    for (int q = 0; q < NV; ++q)
      w[q] = q * THREADS < n ? load_row_vec<ELT>(row, P.V, shift, v0 + q * THREADS + tid) : VT::neg_inf();
  }
  bool mine[kE];
  float zj[kE];
#pragma unroll
  for (int k = 0; k < kE; ++k) {
    const int at = id[k] - t_first;        // the entry's place in the part
    mine[k] = id[k] >= 0 && at >= 0 && at < (v1 - v0) * N;
    zj[k] = -INFINITY;
    if (mine[k]) {
      const int bit = at / N * 8 + at % N;
      bad |= (atomicOr(&listed_words[bit >> 5], 1u << (bit & 31)) >> (bit & 31)) & 1u;   // listed twice
      zj[k] = load_elem<ELT>(row, id[k]);
      bad |= zj[k] != zj[k] || zj[k] == INFINITY;
    }
  }
  float p[kE], mass = 0.f;
#pragma unroll
  for (int k = 0; k < kE; ++k) mass += p[k] = id[k] >= 0 ? expf(lp[k]) : 0.f;
  __syncthreads();

  // ---- the part's sums
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const uint32_t in = q * THREADS < n ? listed[q * THREADS + tid] : 0u;
    if (in) w[q] = with_neg_inf<ELT>(w[q], in);   // out of the unlisted tokens' sum
  }
  const float m = VT::vmax(w);             // NaN is passed over here and kept by the sum
  const float mb = m > -INFINITY ? m : 0.f;
  const f2 cc = pack2(P.c2, P.c2), mm = pack2(mb, mb);
  f2 s2 = 0ull, s3 = 0ull;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    f2 z[N / 2];
    VT::pairs(w[q], z);
#pragma unroll
    for (int i = 0; i < N / 2; i += 2) {
      s2 = add2(s2, exp2_2(mul2(sub2(z[i], mm), cc)));
      s3 = add2(s3, exp2_2(mul2(sub2(z[i + 1], mm), cc)));
    }
  }
  float s, s_hi;
  unpack2(add2(s2, s3), s, s_hi);
  TlPart part{m, s + s_hi, zj[0], zj[0] > -INFINITY ? 1.f : 0.f};
#pragma unroll
  for (int k = 1; k < kE; ++k) {
    const float top = fmaxf(part.ml, zj[k]);
    if (top > -INFINITY)
      part.sl = (part.ml > -INFINITY ? part.sl * expf(__fmul_rn(__fsub_rn(part.ml, top), P.inv_T)) : 0.f) +
                (zj[k] > -INFINITY ? expf(__fmul_rn(__fsub_rn(zj[k], top), P.inv_T)) : 0.f);
    part.ml = top;
  }
  if (bad) part.s = NAN;
  part = tl_combine(part, P.c2, P.inv_T);
  mass = warp_sum(mass);
  if (lane == 0) sh.warp[warp] = part, sh.mass[warp] = mass;
  __syncthreads();
  const TlPart none{-INFINITY, 0.f, -INFINITY, 0.f};
  if (warp == 0) {
    part = tl_combine(lane < kWarps ? sh.warp[lane] : none, P.c2, P.inv_T);
    if (ctas == 1) {
      if (lane == 0) sh.part[0] = part;
    } else if (lane < ctas) {              // to every CTA of the cluster
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                   :: "r"(peer(&sh.part[rank], lane)), "f"(part.m), "f"(part.s), "f"(part.ml), "f"(part.sl) : "memory");
    }
  }
  if (ctas > 1) {
    tl_arrive();
    tl_wait();
  } else {
    __syncwarp();
  }

  // ---- the row against Ma = max(M, Ml); Z its whole sum
  const float scale = grad ? P.weights[r / P.t_len] * P.inv_T : 0.f;
  if (warp == 0) {
    part = tl_combine(lane < ctas ? sh.part[lane] : none, P.c2, P.inv_T);
    mass = warp_sum(lane < kWarps ? sh.mass[lane] : 0.f);
    TlRow R;
    R.Ma = fmaxf(part.m, part.ml);
    R.valid = part.s == part.s && R.Ma > -INFINITY && R.Ma < INFINITY;
    // the listed tokens carry most of Z: full-precision exponentials for them
    const float lt = __fmul_rn(__fsub_rn(part.m, R.Ma), P.inv_T);
    const float ft = part.m > -INFINITY ? expf(lt) : 0.f;
    const float fl = part.ml > -INFINITY ? expf(__fmul_rn(__fsub_rn(part.ml, R.Ma), P.inv_T)) : 0.f;
    R.Z = __fadd_rn(__fmul_rn(part.s, ft), __fmul_rn(part.sl, fl));
    R.LZ = logf(R.Z);
    R.mass = mass;
    float rest = P.renorm ? 0.f : __fsub_rn(1.f, mass);
    if (rest < kTlComplete) rest = 0.f;
    R.a = R.valid ? scale * __fsub_rn(__fdiv_rn(ft, R.Z), part.s > 0.f ? __fdiv_rn(rest, part.s) : 0.f) : NAN;
    R.base = part.m > -INFINITY ? part.m : 0.f;
    R.kl = 0.f;
    if (rest > 0.f) R.kl = part.s > 0.f ? rest * (logf(rest) - __fsub_rn(__fadd_rn(lt, logf(part.s)), R.LZ)) : INFINITY;
    if (lane == 0) sh.row = R;
  }
  __syncthreads();
  const TlRow R = sh.row;

  // ---- the gradient
  if (grad) {
    const f2 bb = pack2(R.base, R.base), aa = pack2(R.a, R.a);
    auto gradient = [&](const uint4& x, float (&g)[N]) {
      f2 z[N / 2];
      VT::pairs(x, z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) unpack2(mul2(aa, exp2_2(mul2(sub2(z[i], bb), cc))), g[2 * i], g[2 * i + 1]);
    };
    if (whole && P.same_shift) {
      unsigned char* at = grad + (static_cast<long long>(v0 + tid) * N - shift) * ELT;
#pragma unroll
      for (int q = 0; q < NV; ++q)
        if (q * THREADS < n) {
          float g[N];
          gradient(w[q], g);
          store_vec16(at + q * THREADS * 16, VT::pack(g));
        }
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q)
        if (q * THREADS < n) {
          float g[N];
          gradient(w[q], g);
          store_edge<ELT>(grad, P.V, (v0 + q * THREADS + tid) * N - shift, P.same_shift, g);
        }
    }
  }

  // ---- the listed tokens: their gradients after the row's, and the divergence
  float term = 0.f, ej[kE];
#pragma unroll
  for (int k = 0; k < kE; ++k) {
    const float lj = __fmul_rn(__fsub_rn(zj[k], R.Ma), P.inv_T);
    ej[k] = zj[k] > -INFINITY ? __fdiv_rn(expf(lj), R.Z) : 0.f;
    if (P.renorm) {
      lp[k] = R.mass > 0.f ? __fsub_rn(lp[k], logf(R.mass)) : -INFINITY;
      p[k] = R.mass > 0.f ? __fdiv_rn(p[k], R.mass) : 0.f;
    }
    if (mine[k] && p[k] > 0.f) term += __fmul_rn(p[k], __fsub_rn(lp[k], __fsub_rn(lj, R.LZ)));
  }
  term = warp_sum(term);
  if (lane == 0) sh.term[warp] = term;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kE; ++k)
    if (grad && mine[k]) VT::store_rounded(grad, id[k], R.valid ? scale * __fsub_rn(ej[k], p[k]) : NAN);
  if (tid == 0) {
    term = 0.f;
    for (int c = 0; c < kWarps; ++c) term += sh.term[c];
    asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(peer(&sh.kl[rank], 0)), "f"(term) : "memory");
  }
  if (ctas > 1) {
    tl_arrive();
    if (rank != 0) return;                 // the first CTA's memory is written, and waits
    tl_wait();
  }
  if (tid == 0) {
    float kl = R.kl;
    for (int c = 0; c < ctas; ++c) kl += sh.kl[c];
    P.row_kl[r] = R.valid ? kl : NAN;
  }
}

// loss[b] = w_b * sum_t row_kl[b, t], in position order.
__global__ void toploss_sum_kernel(int n_seq, int t_len, const float* row_kl, const float* weights, float* loss) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= n_seq) return;
  double s = 0.0;
  for (int t = 0; t < t_len; ++t) s += static_cast<double>(row_kl[static_cast<long long>(b) * t_len + t]);
  loss[b] = static_cast<float>(static_cast<double>(weights[b]) * s);
}

template <int ELT, int THREADS, int NV, int CTAS>
cudaError_t launch_parts(const TopLossParams& p, int rows, int nvec, cudaStream_t s) {
  const int cluster = (nvec + THREADS * NV - 1) / (THREADS * NV);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, toploss_kernel<ELT, THREADS, NV, CTAS>, p);
}

template <int ELT>
cudaError_t launch_toploss(const TopLossParams& p, int rows, cudaStream_t s) {
  // the vectors of a row that lies anyhow on its 16-byte boundaries
  const int nvec = (p.V + 2 * Vec<ELT>::N - 2) / Vec<ELT>::N;
  if (nvec <= 128 * 4) return launch_parts<ELT, 128, 4, 8>(p, rows, nvec, s);
  if (nvec <= kTlMaxCtas * 128 * 20) return launch_parts<ELT, 128, 20, 4>(p, rows, nvec, s);
  if (nvec <= kTlMaxCtas * 256 * 20) return launch_parts<ELT, 256, 20, 2>(p, rows, nvec, s);
  return launch_parts<ELT, 256, 33, 1>(p, rows, nvec, s);
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_kd_top_loss(int n_seq, int t_len, int V, sv_dtype dtype, int K, const int32_t* ids,
                                      const float* logp, const void* draft_logits, const float* weights,
                                      float temperature, int mode, float* row_kl, float* loss, void* grad,
                                      sv_stream_t stream) {
  using namespace sv;
  if (n_seq < 1 || t_len < 1 || V < 1 || K < 1 || K > SV_KD_TOP_MAX) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(n_seq) * t_len > (1LL << 28)) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (mode != SV_KD_TOP_TAIL && mode != SV_KD_TOP_RENORM) return SV_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SV_ERR_INVALID_ARG;
  if (!ids || !logp || !draft_logits || !weights || !row_kl || !loss) return SV_ERR_INVALID_ARG;
  const int elt = dtype == SV_F32 ? 4 : 2;
  if (static_cast<long long>(V) * elt > kTlMaxRow) return SV_ERR_INVALID_ARG;
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
  const int rows = n_seq * t_len;
  const cudaError_t e = elt == 2 ? launch_toploss<2>(p, rows, s) : launch_toploss<4>(p, rows, s);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  toploss_sum_kernel<<<(n_seq + 127) / 128, 128, 0, s>>>(n_seq, t_len, row_kl, weights, loss);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
