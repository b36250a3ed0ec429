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
// A row goes to a cluster of 1 to 8 CTAs, each streaming its part of it once:
// running maxima and sums per thread for (M, S), and beside them the 16-byte
// vectors that can still hold a token of the list.  A token can be left out
// as soon as K others at or above some t are known and it is below t; t comes
// from the threads' running maxima: if q = K / 16 lanes of each of the 16
// warps have seen a value of at least t, K tokens have.  So t is the least of
// the warps' q-th largest lane maxima, and what passes is a few times K.  The
// warps publish their parts of t without a barrier but one, after the first
// tile (an older part is smaller and lets more through).  A vector whose
// maximum passes is kept whole, a ballot and one addition for a warp; its
// tokens are looked at once t is final (appending token by token while
// streaming: 116 us against @@ on 1024 ragged rows of 128256 bf16 logits,
// K = 64).
//
// The CTAs hand their tokens at or above t, and their M and S, to the
// cluster's first one and leave; it selects the K by radix and ranks them.
// Vectors that outgrow their buffer (rows of few distinct values, or masked
// with a finite value) are dropped, and the first CTA selects from the row
// itself.

#include <cuda_runtime.h>

#include <cfloat>
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
constexpr int kTopUnroll = 4;             // 16-byte vectors of a tile per thread
constexpr int kTopTile = kTopThreads * kTopUnroll;
constexpr int kTopFewRows = 1216;         // CTAs below which a row is split
constexpr int kTopVecs = 2048;            // vectors a CTA can hold: more than a part that
                                          // leaves threads idle has
constexpr int kTopPush = 512;             // tokens that a CTA hands on at most
constexpr int kTopCap = 8 * kTopPush;     // tokens to select from

struct TopParams {
  const unsigned char* rows;   // [n_seq, t_len, V]
  const int* n_rows;           // [n_seq] or null: t_len
  int* ids;                    // [n_seq * t_len, K]
  float* logp;                 // [n_seq * t_len, K]
  float* lse;                  // [n_seq * t_len]
  int t_len, V, K;
  float c2;                    // log2(e) / T
  float T;
  int quota;                   // ceil(K / warps)
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

typedef unsigned long long key64;   // key and id: larger for a larger value, then a lower id
__device__ __forceinline__ key64 top_entry(uint32_t key, uint32_t id) { return (static_cast<key64>(key) << 32) | ~id; }

struct TopShared {
  float wm[kTopWarps], ws[kTopWarps];     // the warps' maxima and sums
  volatile float wt[kTopWarps];           // the warps' parts of t
  unsigned int hist[256];
  unsigned int warp_n[kTopWarps];
  unsigned int n_vecs;                    // vectors kept (may pass kTopVecs)
  unsigned int n_tokens;                  // tokens to select from (may pass kTopCap)
  unsigned int n_list;
  unsigned int base;                      // where this CTA's tokens go in the first one's
  unsigned int lost;                      // (first CTA) some CTA's vectors outgrew its buffer
  float M[8], S[8];                       // (first CTA) the CTAs' parts
  int digit, left;
  key64 list[kTopMaxK];
};
constexpr int kTopVecsAt = (static_cast<int>(sizeof(TopShared)) + 15) / 16 * 16;
constexpr int kTopIdsAt = kTopVecsAt + kTopVecs * 16;
constexpr int kTopTokensAt = kTopIdsAt + kTopVecs * 4;
constexpr int kTopSmem = kTopTokensAt + kTopCap * static_cast<int>(sizeof(key64));

// All threads of the cluster: arrive (what they wrote before is visible to
// those that wait after), and wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Shared variables of the cluster's first CTA.
__device__ __forceinline__ unsigned int first_add(unsigned int* p, unsigned int v) {
  unsigned int old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(peer(p, 0)), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void first_store(float* p, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(peer(p, 0)), "f"(v) : "memory");
}
__device__ __forceinline__ void first_store(key64* p, key64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(peer(p, 0)), "l"(v) : "memory");
}

// The warp's lanes' values in descending order.
__device__ __forceinline__ float warp_sort(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, v, o);
      const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
      v = keep_max ? fmaxf(v, x) : fminf(v, x);
    }
  return v;
}

// The bin, from the top, in which the running count of hist reaches `left`
// (1 <= left <= total), and what is left of `left` in it: by warp 0.
__device__ __forceinline__ void find_bin(TopShared& sh, int left) {
  const int lane = threadIdx.x;
  if (lane < 32) {
    unsigned int h[8], sum = 0;    // lane 0 has the eight highest bins
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += h[i] = sh.hist[255 - (lane * 8 + i)];
    unsigned int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned int up = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += up;
    }
    before -= sum;
    if (before < static_cast<unsigned>(left) && before + sum >= static_cast<unsigned>(left)) {
      int i = 0;
      for (; i < 7 && before + h[i] < static_cast<unsigned>(left); ++i) before += h[i];
      sh.digit = 255 - (lane * 8 + i);
      sh.left = left - static_cast<int>(before);
    }
  }
}

// The n_list largest of n distinct entries (n_list <= n), into sh.list in any
// order.
__device__ __forceinline__ void select_entries(TopShared& sh, const key64* cand, int n, int n_list) {
  const int tid = threadIdx.x;
  key64 prefix = 0;     // the digits of the n_list-th largest so far, the rest zero
  if (n > n_list) {
    int left = n_list;
    for (int shift = 56; shift >= 0; shift -= 8) {
      if (tid < 256) sh.hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kTopThreads) {
        const key64 k = cand[i];
        if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      find_bin(sh, left);
      __syncthreads();
      prefix |= static_cast<key64>(sh.digit) << shift;
      left = sh.left;
      if (static_cast<unsigned>(left) == sh.hist[sh.digit]) break;   // the whole bin
    }
  }
  for (int i = tid; i < n; i += kTopThreads)
    if (cand[i] >= prefix) sh.list[atomicAdd(&sh.n_list, 1u)] = cand[i];
  __syncthreads();
}

// The n_list largest tokens of a row (of which at least n_list are above
// -inf) from the row itself, into sh.list in any order: a radix selection on
// the values, then of the tokens that tie with the last one the lowest ids.
template <int ELT>
__device__ __noinline__ void select_from_row(TopShared& sh, const unsigned char* row, int V, int n_list) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(V, shift);
  int need = n_list;
  uint32_t prefix = 0;
  for (int bits = 24; bits >= 0; bits -= 8) {
    if (tid < 256) sh.hist[tid] = 0;
    __syncthreads();
    for (int v = tid; v < nvec; v += kTopThreads) {
      float z[N];
      VT::unpack(load_row_vec<ELT>(row, V, shift, v), z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t key = top_key(z[e]);
        if (key > kKeyNegInf && (bits == 24 || (key >> (bits + 8)) == (prefix >> (bits + 8))))
          atomicAdd(&sh.hist[(key >> bits) & 255u], 1u);
      }
    }
    __syncthreads();
    find_bin(sh, need);
    __syncthreads();
    prefix |= static_cast<uint32_t>(sh.digit) << bits;
    need = sh.left;
  }
  // `need` of the tokens that tie with key `prefix`, and every larger one
  unsigned ties_before = 0;
  for (int v0 = 0; v0 < nvec; v0 += kTopThreads) {
    const int v = v0 + tid;
    float z[N];
    unsigned tie = 0;
    if (v < nvec) {
      VT::unpack(load_row_vec<ELT>(row, V, shift, v), z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t key = top_key(z[e]);
        if (key > prefix) sh.list[atomicAdd(&sh.n_list, 1u)] = top_entry(key, static_cast<uint32_t>(v * N - shift + e));
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
        if (at < static_cast<unsigned>(need))
          sh.list[n_list - need + at] = top_entry(prefix, static_cast<uint32_t>(v * N - shift + e));
        ++at;
      }
    ties_before += all;
  }
  __syncthreads();
}

template <int ELT>
__global__ void __launch_bounds__(kTopThreads, 2) top_kernel(const TopParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  extern __shared__ __align__(16) unsigned char smem[];
  TopShared& sh = *reinterpret_cast<TopShared*>(smem);
  uint4* vecs = reinterpret_cast<uint4*>(smem + kTopVecsAt);
  int* vec_at = reinterpret_cast<int*>(smem + kTopIdsAt);
  key64* tokens = reinterpret_cast<key64*>(smem + kTopTokensAt);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster_ctas(), rank = cluster_rank();
  const long long r = blockIdx.x / ctas;
  const unsigned char* row = P.rows + r * P.V * ELT;
  int* ids = P.ids + r * P.K;
  float* logp = P.logp + r * P.K;
  if (P.n_rows && static_cast<int>(r % P.t_len) >= P.n_rows[r / P.t_len]) {   // the whole cluster
    if (rank == 0) {
      for (int j = tid; j < P.K; j += kTopThreads) ids[j] = -1, logp[j] = -INFINITY;
      if (tid == 0) P.lse[r] = -INFINITY;
    }
    return;
  }
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  const int part = (nvec + ctas - 1) / ctas;
  const int v0 = min(nvec, rank * part), v1 = min(nvec, v0 + part);

  auto load = [&](uint4 (&w)[kTopUnroll], int base) {
    // inside the part and away from the row's first and last vector
    if (base >= v0 + 1 && base + kTopTile < v1) {
      const unsigned char* at = row + (static_cast<long long>(base + tid) * N - shift) * ELT;
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) w[q] = load_vec16(at + q * kTopThreads * 16);
    } else {
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) {
        const int v = base + q * kTopThreads + tid;
        w[q] = v < v1 ? load_row_vec<ELT>(row, P.V, shift, v) : VT::neg_inf();
      }
    }
  };

  float m = -INFINITY, t = -FLT_MAX;   // below t nothing is a candidate, nor is -inf
  f2 s2 = 0ull;
  const f2 cc = pack2(P.c2, P.c2);
  uint4 w[kTopUnroll];
  load(w, v0);
  if (tid == 0) sh.n_vecs = sh.n_tokens = sh.n_list = sh.lost = 0;
  if (ctas > 1) {
    __syncthreads();
    cluster_arrive();                  // the counters are set
  }
  int tile = 0;
  for (int base = v0; base < v1; base += kTopTile, ++tile) {
    uint4 next[kTopUnroll];
    if (base + kTopTile < v1) load(next, base + kTopTile);
    const float vm = VT::vmax(w);        // NaN is passed over here and kept by the sum
    if (vm > m) {
      if (m > -INFINITY) {
        const float f = fast_exp2(__fmul_rn(__fsub_rn(m, vm), P.c2));
        s2 = mul2(s2, pack2(f, f));
      }
      m = vm;
    }
    const float mb = m > -INFINITY ? m : 0.f;
    const f2 mm = pack2(mb, mb);
#pragma unroll
    for (int q = 0; q < kTopUnroll; ++q) {
      f2 z[N / 2];
      VT::pairs(w[q], z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) s2 = add2(s2, exp2_2(mul2(sub2(z[i], mm), cc)));
    }
    // ---- t: after the first tile, and each time the tiles seen have doubled
    if ((tile & (tile + 1)) == 0) {
      const float part_t = __shfl_sync(0xffffffffu, warp_sort(m, lane), P.quota - 1);
      if (lane == 0) sh.wt[warp] = part_t;
      if (tile == 0) __syncthreads();
    }
    const float seen = sh.wt[lane & (kTopWarps - 1)];
    t = fmaxf(from_ordered_key(__reduce_min_sync(0xffffffffu, ordered_key(seen))), -FLT_MAX);
    if (__any_sync(0xffffffffu, vm >= t)) {
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) {
        const uint4 one[1] = {w[q]};
        const bool keep = VT::vmax(one) >= t;
        const unsigned who = __ballot_sync(0xffffffffu, keep);
        if (!who) continue;
        unsigned at = 0;
        if (lane == 0) at = atomicAdd(&sh.n_vecs, __popc(who));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
        if (keep && at < kTopVecs) {
          vecs[at] = w[q];
          vec_at[at] = base + q * kTopThreads + tid;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kTopUnroll; ++q) w[q] = next[q];
  }

  // ---- this CTA's M, S and t
  float s, s_hi;
  unpack2(s2, s, s_hi);
  s += s_hi;
  const float part_t = __shfl_sync(0xffffffffu, warp_sort(m, lane), P.quota - 1);
  if (s != s) m = NAN;   // a NaN is carried by the maximum
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmax_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  float ws = m > -INFINITY ? s * fast_exp2(__fmul_rn(__fsub_rn(m, wm), P.c2)) : 0.f;
  ws = warp_sum(ws);
  if (lane == 0) sh.wm[warp] = wm, sh.ws[warp] = ws, sh.wt[warp] = part_t;
  __syncthreads();
  if (ctas > 1) cluster_wait();        // the first CTA's counters are set
  if (warp == 0) {
    const bool in = lane < kTopWarps;
    const float lm = in ? sh.wm[lane] : -INFINITY;
    float M = lm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmax_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float S = warp_sum(lm > -INFINITY ? sh.ws[lane] * fast_exp2(__fmul_rn(__fsub_rn(lm, M), P.c2)) : 0.f);
    if (lane == 0) {
      first_store(&sh.M[rank], M);
      first_store(&sh.S[rank], S);
    }
  }
  {
    const float seen = sh.wt[lane & (kTopWarps - 1)];
    t = fmaxf(from_ordered_key(__reduce_min_sync(0xffffffffu, ordered_key(seen))), -FLT_MAX);
  }
  // ---- the kept vectors' tokens at or above t
  const bool whole = sh.n_vecs <= kTopVecs;
  const int n_vecs = static_cast<int>(whole ? sh.n_vecs : 0u);
  for (int i = tid; i < n_vecs; i += kTopThreads) {
    float z[N];
    VT::unpack(vecs[i], z);
    const int t0 = vec_at[i] * N - shift;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (z[e] >= t) {
        const unsigned at = atomicAdd(&sh.n_tokens, 1u);
        if (at < kTopCap) tokens[at] = top_entry(top_key(z[e]), static_cast<uint32_t>(t0 + e));
      }
  }
  if (rank != 0) {
    __syncthreads();
    // at most kTopPush: where there are more, the K largest
    unsigned n = sh.n_tokens;
    const key64* from = tokens;
    if (n > kTopPush && n <= kTopCap) {
      select_entries(sh, tokens, static_cast<int>(n), P.K);
      from = sh.list;
      n = P.K;
    }
    if (tid == 0) {
      const bool lost = !whole || n > kTopCap;
      if (lost) first_add(&sh.lost, 1u);
      sh.base = first_add(&sh.n_tokens, lost ? 0u : n);
      if (lost) sh.n_tokens = 0;
    }
    __syncthreads();
    if (sh.n_tokens)
      for (unsigned i = tid; i < n; i += kTopThreads)
        if (sh.base + i < kTopCap) first_store(&tokens[sh.base + i], from[i]);
    cluster_arrive();                  // and leave
    return;
  }
  if (tid == 0 && !whole) atomicAdd(&sh.lost, 1u);
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }

  // ---- the row's M and S
  float M = -INFINITY, S = 0.f;
  for (int c = 0; c < ctas; ++c) M = fmax_nan(M, sh.M[c]);
  for (int c = 0; c < ctas; ++c)
    if (sh.M[c] > -INFINITY) S += sh.S[c] * fast_exp2(__fmul_rn(__fsub_rn(sh.M[c], M), P.c2));
  const bool valid = S > 0.f && isfinite(S) && isfinite(M);   // not NaN, +inf, or nothing but -inf
  int listed = 0;
  if (valid) {
    if (!sh.lost && sh.n_tokens <= kTopCap) {
      const int n = static_cast<int>(sh.n_tokens);
      listed = min(P.K, n);
      select_entries(sh, tokens, n, listed);
    } else {
      // more candidates than the buffers hold: K of them at least
      listed = P.K;
      select_from_row<ELT>(sh, row, P.V, listed);
    }
  }
  // ---- in order: each entry's place is the number of larger ones
  const float L = logf(S);
  for (int j = tid; j < P.K; j += kTopThreads) {
    if (j >= listed) {
      ids[j] = -1;
      logp[j] = valid ? -INFINITY : NAN;
      continue;
    }
    const key64 mine = sh.list[j];
    int place = 0;
    for (int i = 0; i < listed; ++i) place += sh.list[i] > mine;
    const float z = key_value(static_cast<uint32_t>(mine >> 32));
    ids[place] = static_cast<int>(~static_cast<uint32_t>(mine));
    logp[place] = __fsub_rn(__fdiv_rn(__fsub_rn(z, M), P.T), L);
  }
  if (tid == 0) P.lse[r] = valid ? __fadd_rn(__fdiv_rn(M, P.T), L) : M == -INFINITY ? -INFINITY : NAN;
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_kd_top(int n_seq, int t_len, int V, sv_dtype dtype, const void* target_logits,
                                 const int32_t* n_rows, int K, float temperature, int32_t* ids, float* logp,
                                 float* lse, sv_stream_t stream) {
  using namespace sv;
  if (n_seq < 1 || t_len < 1 || V < 1 || K < 1 || K > SV_KD_TOP_MAX) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(n_seq) * t_len > (1LL << 28)) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SV_ERR_INVALID_ARG;
  if (!target_logits || !ids || !logp || !lse) return SV_ERR_INVALID_ARG;
  const int elt = dtype == SV_F32 ? 4 : 2;
  if (static_cast<long long>(V) * elt > (1LL << 30)) return SV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(target_logits) % elt) return SV_ERR_INVALID_ARG;
  const double c2 = 1.4426950408889634 / static_cast<double>(temperature);
  if (!(c2 < 1e30)) return SV_ERR_INVALID_ARG;
  TopParams p{static_cast<const unsigned char*>(target_logits), n_rows, ids, logp, lse, t_len, V, K,
              static_cast<float>(c2), temperature, (K + kTopWarps - 1) / kTopWarps};
  // as many CTAs to a row as leave each two tiles, until there are enough of them
  const int rows = n_seq * t_len, nvec = V / (16 / elt);
  int cluster = 1;
  while (cluster < 8 && static_cast<long long>(rows) * cluster < kTopFewRows && nvec / (2 * cluster) >= 2 * kTopTile) cluster *= 2;
  NvtxRange range("spec_kd_top");
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
  cfg.blockDim = dim3(kTopThreads);
  cfg.dynamicSmemBytes = kTopSmem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // 105 KB a CTA: more than the 48 KB that need no asking
  const void* fn = elt == 2 ? reinterpret_cast<const void*>(&top_kernel<2>) : reinterpret_cast<const void*>(&top_kernel<4>);
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopSmem) != cudaSuccess) return SV_ERR_CUDA;
  const cudaError_t e = elt == 2 ? cudaLaunchKernelEx(&cfg, top_kernel<2>, p) : cudaLaunchKernelEx(&cfg, top_kernel<4>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
