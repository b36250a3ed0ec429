// The K most likely tokens of teacher rows as log-probabilities, with the
// row's log-sum-exp, for sm_103a.
//
// For a row z and a temperature T, with c = log2(e) / T, M = max z and
// S = sum_x 2^((z(x) - M) c):
//   lse = M / T + ln S,  logp(x) = (z(x) - M) / T - ln S.
// Differences are taken before the scale: a likely token's logp keeps its
// digits whatever the row's level, and a row of the type's lowest values
// does not overflow.  The K tokens are those with the largest z, ties
// to the lower id; a token of probability 0 (z = -inf) is never listed.
//
// A CTA takes a row.  The list comes from a radix selection on the values'
// order-preserving 32-bit keys, eight bits a pass, then of the tokens that
// tie with the last one those of the lowest ids.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kTopThreads = 512;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kTopMaxK = SV_KD_TOP_MAX;

struct TopParams {
  const unsigned char* rows;   // [n_seq, t_len, V]
  const int* n_rows;           // [n_seq] or null: t_len
  int* ids;                    // [n_seq * t_len, K]
  float* logp;                 // [n_seq * t_len, K]
  float* lse;                  // [n_seq * t_len]
  int t_len, V, K;
  float c2;                    // log2(e) / T
  float T;
};

constexpr uint32_t kKeyNegInf = 0x007fffffu;   // top_key(-inf)

// Larger for a larger value; -0 and 0 are one value.
__device__ __forceinline__ uint32_t top_key(float z) {
  const uint32_t u = __float_as_uint(__fadd_rn(z, 0.f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct TopShared {
  float wm[kTopWarps], ws[kTopWarps];
  unsigned int hist[256];
  unsigned int warp_n[kTopWarps];
  unsigned int n_found;
  uint32_t prefix;
  int remaining;
  unsigned long long list[kTopMaxK];
};

template <int ELT>
__global__ void __launch_bounds__(kTopThreads) top_kernel(const TopParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  __shared__ TopShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x;
  const unsigned char* row = P.rows + r * P.V * ELT;
  int* ids = P.ids + r * P.K;
  float* logp = P.logp + r * P.K;
  if (P.n_rows && static_cast<int>(r % P.t_len) >= P.n_rows[r / P.t_len]) {
    for (int j = tid; j < P.K; j += kTopThreads) ids[j] = -1, logp[j] = -INFINITY;
    if (tid == 0) P.lse[r] = -INFINITY;
    return;
  }
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);

  // ---- M and S: per thread a running maximum and the sum against it
  float m = -INFINITY, base = 0.f, s = 0.f;
  unsigned finite = 0;
  for (int v = tid; v < nvec; v += kTopThreads) {
    float z[N];
    VT::unpack(load_row_vec<ELT>(row, P.V, shift, v), z);
    float vm = z[0];
#pragma unroll
    for (int e = 1; e < N; ++e) vm = fmaxf(vm, z[e]);
    if (vm > m) {
      s = m == -INFINITY ? 0.f : s * fast_exp2(__fmul_rn(__fsub_rn(m, vm), P.c2));
      m = base = vm;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      s += fast_exp2(__fmul_rn(__fsub_rn(z[e], base), P.c2));
      finite += z[e] > -INFINITY;
    }
  }
  if (s != s) m = NAN;   // a NaN is carried by the maximum
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmax_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  float ws = m > -INFINITY ? s * fast_exp2(__fmul_rn(__fsub_rn(m, wm), P.c2)) : 0.f;
  ws = warp_sum(ws);
  finite = __reduce_add_sync(0xffffffffu, finite);
  if (lane == 0) sh.wm[warp] = wm, sh.ws[warp] = ws, sh.warp_n[warp] = finite;
  if (tid == 0) sh.n_found = 0, sh.prefix = 0;
  __syncthreads();
  float M = -INFINITY, S = 0.f;
  unsigned n_finite = 0;
  for (int w = 0; w < kTopWarps; ++w) M = fmax_nan(M, sh.wm[w]), n_finite += sh.warp_n[w];
  for (int w = 0; w < kTopWarps; ++w)
    if (sh.wm[w] > -INFINITY) S += sh.ws[w] * fast_exp2(__fmul_rn(__fsub_rn(sh.wm[w], M), P.c2));
  if (!(S > 0.f) || !isfinite(S) || !isfinite(M)) {   // NaN, +inf, or nothing but -inf
    for (int j = tid; j < P.K; j += kTopThreads) ids[j] = -1, logp[j] = NAN;
    if (tid == 0) P.lse[r] = M == -INFINITY ? -INFINITY : NAN;
    return;
  }

  // ---- the K-th largest key, most significant byte first
  int need = min(static_cast<unsigned>(P.K), n_finite);
  const int listed = need;
  uint32_t prefix = 0;
  for (int shift_bits = 24; shift_bits >= 0; shift_bits -= 8) {
    for (int i = tid; i < 256; i += kTopThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int v = tid; v < nvec; v += kTopThreads) {
      float z[N];
      VT::unpack(load_row_vec<ELT>(row, P.V, shift, v), z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t key = top_key(z[e]);
        if (key > kKeyNegInf && (shift_bits == 24 || (key >> (shift_bits + 8)) == (prefix >> (shift_bits + 8))))
          atomicAdd(&sh.hist[(key >> shift_bits) & 255u], 1u);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int left = need;
      int d = 255;
      for (; d > 0 && static_cast<int>(sh.hist[d]) < left; --d) left -= sh.hist[d];
      sh.prefix = prefix | (static_cast<uint32_t>(d) << shift_bits);
      sh.remaining = left;
    }
    __syncthreads();
    prefix = sh.prefix;
    need = sh.remaining;
  }
  // `need` of the tokens that tie with key `prefix`, and every larger one
  unsigned ties_before = 0;
  for (int v0 = 0; v0 < nvec; v0 += kTopThreads) {
    const int v = v0 + tid;
    float z[N];
    unsigned tie = 0;
    if (v < nvec) {
      VT::unpack(load_row_vec<ELT>(row, P.V, shift, v), z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t key = top_key(z[e]);
        const uint32_t id = static_cast<uint32_t>(v * N - shift + e);
        if (key > prefix) sh.list[atomicAdd(&sh.n_found, 1u)] = (static_cast<unsigned long long>(key) << 32) | ~id;
        else if (key == prefix && key > kKeyNegInf) tie |= 1u << e;
      }
    }
    // the ties of earlier threads: ids ascend with the thread
    const unsigned mine = __popc(tie);
    unsigned incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) sh.warp_n[warp] = incl;
    __syncthreads();
    unsigned at = ties_before + incl - mine, all = 0;
    for (int w = 0; w < kTopWarps; ++w) {
      if (w < warp) at += sh.warp_n[w];
      all += sh.warp_n[w];
    }
    for (int e = 0; e < N; ++e)
      if ((tie >> e) & 1u) {
        const uint32_t id = static_cast<uint32_t>(v * N - shift + e);
        if (at < static_cast<unsigned>(need))
          sh.list[listed - need + at] = (static_cast<unsigned long long>(prefix) << 32) | ~id;
        ++at;
      }
    ties_before += all;
  }
  __syncthreads();

  // ---- in order: each entry's place is the number of larger ones
  const float L = logf(S);
  for (int j = tid; j < P.K; j += kTopThreads) {
    if (j >= listed) {
      ids[j] = -1;
      logp[j] = -INFINITY;
      continue;
    }
    const unsigned long long mine = sh.list[j];
    int place = 0;
    for (int i = 0; i < listed; ++i) place += sh.list[i] > mine;
    const float z = key_value(static_cast<uint32_t>(mine >> 32));
    ids[place] = static_cast<int>(~static_cast<uint32_t>(mine));
    logp[place] = __fsub_rn(__fdiv_rn(__fsub_rn(z, M), P.T), L);
  }
  if (tid == 0) P.lse[r] = __fadd_rn(__fdiv_rn(M, P.T), L);
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_kd_top(int n_seq, int t_len, int V, sv_dtype dtype, const void* target_logits,
                                 const int32_t* n_rows, int K, float temperature, int32_t* ids, float* logp,
                                 float* lse, sv_stream_t stream) {
  using namespace sv;
  if (n_seq < 1 || t_len < 1 || V < 1 || K < 1 || K > SV_KD_TOP_MAX) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(n_seq) * t_len > (1LL << 30)) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SV_ERR_INVALID_ARG;
  if (!target_logits || !ids || !logp || !lse) return SV_ERR_INVALID_ARG;
  const int elt = dtype == SV_F32 ? 4 : 2;
  if (static_cast<long long>(V) * elt > (1LL << 30)) return SV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(target_logits) % elt) return SV_ERR_INVALID_ARG;
  const double c2 = 1.4426950408889634 / static_cast<double>(temperature);
  if (!(c2 < 1e30)) return SV_ERR_INVALID_ARG;
  TopParams p{static_cast<const unsigned char*>(target_logits), n_rows, ids, logp, lse, t_len, V, K,
              static_cast<float>(c2), temperature};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("spec_kd_top");
  const int ctas = n_seq * t_len;
  if (elt == 2) top_kernel<2><<<ctas, kTopThreads, 0, s>>>(p);
  else top_kernel<4><<<ctas, kTopThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
