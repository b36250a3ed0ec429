// The K most likely tokens of teacher rows as log-probabilities, with the
// row's log-sum-exp, for sm_103a.
//
// For a row z and a temperature T, with c = log2(e) / T, M = max z,
// K0 = fl(M c) and S = sum_x 2^(z(x) c - K0) (one fused multiply-add a term):
//   L = ln S + ln 2 (K0 - M c) = ln sum_x e^((z(x) - M) / T),
//   lse = M / T + L,  logp(x) = (z(x) - M) / T - L,
// K0 - M c exactly (a fused multiply-add again), so that a likely token's logp
// keeps its digits.  That holds while K0 - M c, half a unit in K0's last place
// at most, is small beside the exponent's range: the largest term is 2^(M c -
// K0).  So K0 is kept within +-2^24 (top_base), and a row whose M c lies
// outside (one forced to 1e10, or masked whole with -1e30) takes its sum again,
// of 2^((z - M) c) with the difference first, L = ln S (sum_again).  Taking the
// difference first everywhere would cost an instruction a pair of logits.
// The K tokens are those with the largest z, ties
// to the lower id; a token of probability 0 (z = -inf) is never listed.
//
// A row goes to a cluster of 1 to 8 CTAs, each streaming its part of it once:
// running maxima and sums per thread for (M, S), and beside them what can
// still hold a token of the list.  A token can be left out as soon as K others
// at or above some t are known and it is below t; t comes from the threads'
// maxima: if q = K / 8 values of at least t are among the largest that the lanes
// of each of the 8 warps have seen in a tile, K tokens have.  So t is the least
// of the warps' q-th largest, and what passes is a few times K.  The warps publish
// their parts of t without a barrier but one, after the first tile (an older
// part is smaller and lets more through).  A thread whose four vectors of a
// tile hold a value of at least t notes them, with one ballot and one addition
// a warp, and their largest value; once t is final, those that still pass are
// read again, from L2, and their tokens at or above t kept.
// On 1024 ragged rows of 128256 bf16 logits, K = 64: 44 us; appending token by
// token while streaming 116 us.  A row that takes its sum again, 24 us for 9.
//
// The CTAs hand their tokens at or above t, and their M and S, to the
// cluster's first one and leave; it sorts them, after a selection by
// histogram where they are many: every warp sorts 32, and each of these looks
// its rank up in the other warps' lists (one barrier for a bitonic sort's
// twelve; 1024 ragged rows went from 50 to 47 us with it and with a vector's
// tokens counted before they are placed).  Notes or tokens that outgrow their
// buffer (rows of few distinct values, or masked with a finite value) are
// dropped, and the first CTA selects from the row itself.

#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kTopMaxK = SV_KD_TOP_MAX;
constexpr int kTopSms = 152;
constexpr int kTopUnroll = 4;             // 16-byte vectors of a tile per thread
constexpr int kTopTile = kTopThreads * kTopUnroll;
constexpr int kTopLeft = 768;             // noted places that hold a token at or above the final t
constexpr int kTopEdge = 128;             // entries that share the last one's bin, told apart by counting
constexpr int kTopCount = 256;            // tokens sorted; of more the K are selected first

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
  int push;                    // tokens that a CTA hands on at most (>= K)
  // sizes of a CTA's buffers
  int places;                  // (thread, tile) places noted: more than a part that leaves threads idle has
  int held;                    // ... with their values
  int cap;                     // tokens to sort or to select from
};

typedef unsigned long long key64;   // key and id: larger for a larger value, then a lower id
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // top_key(-inf)

// Larger for a larger value; -0 and 0 are one value.
__device__ __forceinline__ uint32_t top_key(float z) {
  const uint32_t u = __float_as_uint(__fadd_rn(z, 0.f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ key64 top_entry(uint32_t key, uint32_t id) { return (static_cast<key64>(key) << 32) | ~id; }

// What a CTA keeps in shared memory: no more than it needs, for what that
// leaves is L1, and loads in flight need its lines (54 KB a CTA in place of
// 43: 215 us against 207 on 4096 rows of 128256 bf16 logits, K = 64).
struct TopShared {
  float wm[kTopWarps], ws[kTopWarps];   // the warps' maxima and sums
  volatile int wt[kTopWarps];           // the warps' parts of t, as ordered keys
  unsigned int hist[256];
  unsigned int warp_n[kTopWarps];
  unsigned int n_places;                // places noted (may pass `places`)
  unsigned int n_left;                  // ... that hold a token at or above the final t (may pass kTopLeft)
  unsigned int n_tokens;                // tokens to select from (may pass `cap`)
  unsigned int n_list;
  unsigned int base;                    // where this CTA's tokens go in the first one's
  unsigned int lost;                    // (first CTA) some CTA's tokens outgrew its buffers
  float M[8], S[8], t[8];               // (first CTA) the CTAs' parts
  int digit, left;
  unsigned int n_edge;
  key64 edge[kTopEdge];
  key64 list[kTopMaxK];
  int lefts[kTopLeft];                  // the places that hold a token at or above the final t
};
// and, as large as the call needs them:
//   key64 tokens[cap]
//   uint4 held[kTopUnroll][held]
//   int places[places]      a thread's first vector of a tile; ~ of a row's end
//   float tops[places]      ... and the largest value of its vectors
constexpr int kTopBuffersAt = (static_cast<int>(sizeof(TopShared)) + 15) / 16 * 16;

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

// Element e of a vector, e not known to the compiler.
template <int ELT>
__device__ __forceinline__ float element_of(const uint4& v, int e) {
  const int w = ELT == 4 ? e : e >> 1;
  const uint32_t lo = w & 1 ? v.y : v.x, hi = w & 1 ? v.w : v.z, x = w & 2 ? hi : lo;
  return __uint_as_float(ELT == 4 ? x : e & 1 ? x & 0xffff0000u : x << 16);
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

// A value that at least `quota` tokens seen by the warp's lanes reach, from the
// lanes' largest tile maxima m1 and, where half the lanes would not be enough
// to tell, their second largest m2.
__device__ __forceinline__ float quota_of(float m1, float m2, int quota, int lane) {
  if (quota <= 4) {
    int key = ordered_key(m1), top = 0;
    for (int i = 0; i < quota; ++i) {   // the largest leaves, one lane at a time
      top = __reduce_max_sync(0xffffffffu, key);
      const unsigned who = __ballot_sync(0xffffffffu, key == top);
      if (lane == __ffs(who) - 1) key = static_cast<int>(0x80000000u);
    }
    return from_ordered_key(top);
  }
  float v = warp_sort(m1, lane);
  if (quota > 16) {   // the upper half of both, in order again
    v = fmaxf(v, __shfl_sync(0xffffffffu, warp_sort(m2, lane), 31 - lane));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, v, o);
      v = lane & o ? fminf(v, x) : fmaxf(v, x);
    }
  }
  return __shfl_sync(0xffffffffu, v, quota - 1);
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

// The n_list largest of n distinct entries (n_list <= n <= cap), all of
// keys from `least` on, into sh.list in any order.  One histogram of 256 bins
// spread over the keys' own range; then what falls into the bin of the
// n_list-th largest is told apart by counting.  Where that bin is too full to
// count (values that tie), radix passes from the entries' most significant
// byte on.
__device__ __noinline__ void select_entries(TopShared& sh, const key64* cand, int n, int n_list, uint32_t least,
                                               uint32_t most) {
  const int tid = threadIdx.x;
  if (n == n_list) {
    for (int i = tid; i < n; i += kTopThreads) sh.list[i] = cand[i];
    __syncthreads();
    return;
  }
  const int coarse = max(0, 24 - __clz(most - least));   // (most - least) >> coarse < 256
  auto bin = [&](key64 k) { return (static_cast<uint32_t>(k >> 32) - least) >> coarse; };
  if (tid < 256) sh.hist[tid] = 0;
  if (tid == 0) sh.n_list = sh.n_edge = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kTopThreads) atomicAdd(&sh.hist[bin(cand[i])], 1u);
  __syncthreads();
  find_bin(sh, n_list);
  __syncthreads();
  const uint32_t edge = sh.digit;
  int left = sh.left;
  if (sh.hist[edge] <= kTopEdge) {
    for (int i = tid; i < n; i += kTopThreads) {
      const key64 k = cand[i];
      if (bin(k) > edge) sh.list[atomicAdd(&sh.n_list, 1u)] = k;
      if (bin(k) == edge) sh.edge[atomicAdd(&sh.n_edge, 1u)] = k;
    }
    __syncthreads();
    const int n_edge = static_cast<int>(sh.n_edge);
    if (tid < n_edge) {
      const key64 mine = sh.edge[tid];
      int larger = 0;
      for (int i = 0; i < n_edge; ++i) larger += sh.edge[i] > mine;
      if (larger < left) sh.list[n_list - left + larger] = mine;
    }
    __syncthreads();
    return;
  }
  key64 prefix = 0;     // the digits of the n_list-th largest so far, the rest zero
  left = n_list;
  for (int shift = 56; shift >= 0; shift -= 8) {
    __syncthreads();
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
  for (int i = tid; i < n; i += kTopThreads)
    if (cand[i] >= prefix) sh.list[atomicAdd(&sh.n_list, 1u)] = cand[i];
  __syncthreads();
}

// The key of the n_list-th largest value of a row, and how many of the tokens
// that have it are needed: radix, most significant byte first.
template <int ELT>
__device__ __noinline__ void select_value(TopShared& sh, const unsigned char* row, int V, int n_list, int& need,
                                          uint32_t& prefix) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  const int tid = threadIdx.x;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(V, shift);
  need = n_list;
  prefix = 0;
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
}

// The n_list largest tokens of a row from the row itself, into sh.list in any
// order; at least n_list of its tokens reach t (which is above -inf).  Those
// above t, and where they are fewer of those that tie with t the lowest ids,
// which a row of few values or one masked with a finite value has at its very
// front.  Where more are above t than `tokens` holds, a radix selection on the
// values first.
template <int ELT>
__device__ __noinline__ void select_from_row(TopShared& sh, const unsigned char* row, int V, int n_list, float t, float M,
                                             key64* tokens, int cap) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(V, shift);
  __syncthreads();
  if (tid == 0) sh.n_tokens = sh.n_list = 0;
  __syncthreads();
  for (int v = tid; v < nvec; v += kTopThreads) {
    const uint4 one[1] = {load_row_vec<ELT>(row, V, shift, v)};
    if (!(VT::vmax(one) > t)) continue;
    float z[N];
    VT::unpack(one[0], z);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (z[e] > t) {
        const unsigned at = atomicAdd(&sh.n_tokens, 1u);
        if (at < static_cast<unsigned>(cap)) tokens[at] = top_entry(top_key(z[e]), static_cast<uint32_t>(v * N - shift + e));
      }
  }
  __syncthreads();
  const int above = static_cast<int>(min(sh.n_tokens, 0x7fffffffu));
  if (above >= n_list && above <= cap) {
    select_entries(sh, tokens, above, n_list, top_key(t), top_key(M));
    return;
  }
  int need = n_list - above;
  uint32_t prefix = top_key(t);
  if (above < n_list) {
    for (int i = tid; i < above; i += kTopThreads) sh.list[i] = tokens[i];
  } else {
    select_value<ELT>(sh, row, V, n_list, need, prefix);
  }
  // `need` of the tokens that tie with key `prefix` (and, after a selection,
  // every larger one)
  const bool larger = above >= n_list;
  unsigned ties_before = 0;
  for (int v0 = 0; v0 < nvec && (larger || ties_before < static_cast<unsigned>(need)); v0 += kTopThreads) {
    const int v = v0 + tid;
    float z[N];
    unsigned tie = 0;
    if (v < nvec) {
      VT::unpack(load_row_vec<ELT>(row, V, shift, v), z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t key = top_key(z[e]);
        if (larger && key > prefix) sh.list[atomicAdd(&sh.n_list, 1u)] = top_entry(key, static_cast<uint32_t>(v * N - shift + e));
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

// The base of a sum of maximum m: fl(m c), but within +-kTopFar.  There a term is
// at most 2^(1/2).  Below -kTopFar the terms vanish against a row whose maximum is
// above; past kTopFar a sum may be +inf, but then this and every later base is
// kTopFar, so it is only ever scaled by 1, and NaN comes from NaN alone.
constexpr float kTopFar = 16777216.f;
__device__ __forceinline__ float top_base(float m, float c) {
  return fminf(fmaxf(__fmul_rn(m, c), -kTopFar), kTopFar);
}
// ... which is not fl(m c): the sum about it says nothing of a row with this maximum.
__device__ __forceinline__ bool top_far(float m, float c) { return !(fabsf(__fmul_rn(m, c)) < kTopFar); }

// S of a row whose M c is far, as 2^((z - M) c).
template <int ELT>
__device__ __noinline__ float sum_again(TopShared& sh, const unsigned char* row, int V, float M, float c) {
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(V, shift);
  float s = 0.f;
  for (int v = threadIdx.x; v < nvec; v += kTopThreads) {
    float z[Vec<ELT>::N];
    Vec<ELT>::unpack(load_row_vec<ELT>(row, V, shift, v), z);
    float part = 0.f;
    for (int e = 0; e < Vec<ELT>::N; ++e) part += fast_exp2(__fmul_rn(__fsub_rn(z[e], M), c));
    s += part;
  }
  s = warp_sum(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.ws[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int w = 0; w < kTopWarps; ++w) s += sh.ws[w];
  return s;
}

template <int ELT>
__global__ void __launch_bounds__(kTopThreads, 4) top_kernel(const __grid_constant__ TopParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  extern __shared__ __align__(16) unsigned char smem[];
  TopShared& sh = *reinterpret_cast<TopShared*>(smem);
  key64* tokens = reinterpret_cast<key64*>(smem + kTopBuffersAt);
  uint4* held = reinterpret_cast<uint4*>(tokens + P.cap);
  int* places = reinterpret_cast<int*>(held + kTopUnroll * P.held);
  float* tops = reinterpret_cast<float*>(places + P.places);
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
  int v0 = min(nvec, rank * part), v1 = min(nvec, v0 + part);
  if (tid == 0) sh.n_places = sh.n_left = sh.n_tokens = sh.n_list = sh.lost = 0;
  if (tid < kTopWarps) sh.wt[tid] = ordered_key(-FLT_MAX);
  __syncthreads();
  if (ctas > 1) cluster_arrive();      // the counters are set

  float m = -INFINITY, m2 = -INFINITY, k0 = 0.f;
  float t = -FLT_MAX;                  // below t nothing is a candidate, nor is -inf
  f2 s2 = 0ull;
  const f2 cc = pack2(P.c2, P.c2);
  const unsigned below = (1u << lane) - 1u;
  // A thread's vectors of a tile, the first of them vector `at`.
  auto take = [&](const uint4 (&w)[kTopUnroll], int at, bool publish, bool barrier) {
    const float vm = VT::vmax(w);        // NaN is passed over here and kept by the sum
    m2 = fmaxf(m2, fminf(m, vm));
    // The first tile has no second maximum but within itself: 384 bf16 rows of
    // 6937, K=255: 13 us, without it 40 us (t is low and the buffers overflow).
    if (barrier && P.quota > 16) {
      float most = -INFINITY;
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) {
        const uint4 one[1] = {w[q]};
        const float x = VT::vmax(one);
        m2 = fmaxf(m2, fminf(most, x));
        most = fmaxf(most, x);
      }
    }
    // (a base that follows only where terms would pass 2^24 is 1 % faster, but
    // the largest terms' exponents then lose four bits)
    if (vm > m) {
      const float kn = top_base(vm, P.c2);
      const float f = m > -INFINITY ? fast_exp2(__fsub_rn(k0, kn)) : 0.f;
      s2 = mul2(s2, pack2(f, f));
      m = vm;
      k0 = kn;
    }
    const f2 nk = pack2(-k0, -k0);
#pragma unroll
    for (int q = 0; q < kTopUnroll; ++q) {
      f2 z[N / 2];
      VT::pairs(w[q], z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) s2 = add2(s2, exp2_2(fma2(z[i], cc, nk)));
    }
    if (publish) {
      const float part_t = quota_of(m, m2, P.quota, lane);
      if (lane == 0) sh.wt[warp] = ordered_key(fmaxf(part_t, -FLT_MAX));
      if (barrier) __syncthreads();
    }
    t = from_ordered_key(__reduce_min_sync(0xffffffffu, sh.wt[lane & (kTopWarps - 1)]));
    const unsigned who = __ballot_sync(0xffffffffu, vm >= t);
    if (who) {
      int note = 0;
      if (lane == 0) note = static_cast<int>(atomicAdd(&sh.n_places, __popc(who)));
      note = __shfl_sync(0xffffffffu, note, 0) + __popc(who & below);
      if (vm >= t && note < P.places) {
        places[note] = at;
        tops[note] = vm;
        if (note < P.held) {
#pragma unroll
          for (int q = 0; q < kTopUnroll; ++q) held[q * P.held + note] = w[q];
        }
      }
    }
  };

  // ---- a first tile of the row's ends where they are not whole vectors (two
  // threads, in the CTAs that have them, padded with -inf), then full tiles,
  // the next one's loads ahead, then the rest
  const bool head = shift != 0 && v0 == 0, tail = v1 == nvec && (P.V + shift) % N != 0 && v1 > v0;
  const int ends = head || tail;
  int place = v0 + head + tid;
  uint4 a[kTopUnroll], b[kTopUnroll];
  if (ends) {
#pragma unroll
    for (int q = 0; q < kTopUnroll; ++q) a[q] = VT::neg_inf();
    if (tid == 0 && head) a[0] = load_row_vec<ELT>(row, P.V, shift, 0), place = ~0;
    if (tid == 1 && tail && nvec > head) a[0] = load_row_vec<ELT>(row, P.V, shift, nvec - 1), place = ~(nvec - 1);
    v0 += head;
    v1 -= tail;
  }
  const unsigned char* at = row + (static_cast<long long>(v0 + tid) * N - shift) * ELT;
  int left = v1 - v0;                    // vectors not yet loaded
  auto load = [&](uint4 (&w)[kTopUnroll]) {
    if (left >= kTopTile) {
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) w[q] = load_vec16(at + q * kTopThreads * 16);
    } else {
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q)
        w[q] = tid + q * kTopThreads < left ? load_vec16(at + q * kTopThreads * 16) : VT::neg_inf();
    }
    at += kTopTile * 16;
    left -= kTopTile;
  };
  // t is published after the first full tile (with a barrier) and each time
  // the tiles taken have doubled
  int tiles = -ends;                     // taken, not counting the ends
  if (!ends) load(a);
  for (;;) {
    const bool more = left > 0;
    if (more) load(b);
    take(a, place, tiles >= 0 && (tiles & (tiles + 1)) == 0, tiles == 0);
    if (++tiles == 0) place = v0 + tid;
    else place += kTopTile;
    if (!more) break;
    const bool again = left > 0;
    if (again) load(a);
    take(b, place, (tiles & (tiles + 1)) == 0, tiles == 0);
    ++tiles;
    place += kTopTile;
    if (!again) break;
  }

  // ---- this CTA's t, M and S
  float s, s_hi;
  unpack2(s2, s, s_hi);
  s += s_hi;
  if (tiles & (tiles - 1)) {             // tiles taken since t was published
    const float part_t = quota_of(m, m2, P.quota, lane);
    if (lane == 0) sh.wt[warp] = ordered_key(fmaxf(part_t, -FLT_MAX));
  }
  // a NaN is carried by the maximum
  float wm = from_ordered_key(__reduce_max_sync(0xffffffffu, ordered_key(m)));
  if (__any_sync(0xffffffffu, s != s)) wm = NAN;
  const float ws = warp_sum(m > -INFINITY ? s * fast_exp2(__fsub_rn(k0, top_base(wm, P.c2))) : 0.f);
  if (lane == 0) sh.wm[warp] = wm, sh.ws[warp] = ws;
  __syncthreads();
  if (ctas > 1) cluster_wait();        // the first CTA's counters are set
  t = from_ordered_key(__reduce_min_sync(0xffffffffu, sh.wt[lane & (kTopWarps - 1)]));
  if (warp == kTopWarps - 1) {         // the warp with the fewest notes to look at
    const bool in = lane < kTopWarps;
    const float lm = in ? sh.wm[lane] : -INFINITY;
    float M = lm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmax_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float S = warp_sum(lm > -INFINITY ? sh.ws[lane] * fast_exp2(__fsub_rn(top_base(lm, P.c2), top_base(M, P.c2))) : 0.f);
    if (lane == 0) {
      first_store(&sh.M[rank], M);
      first_store(&sh.S[rank], S);
      first_store(&sh.t[rank], t);
    }
  }
  // ---- the noted vectors' tokens at or above t: the places that still hold
  // one, and those again
  bool whole = static_cast<int>(sh.n_places) <= P.places;
  int n_left = static_cast<int>(whole ? sh.n_places : 0u);
  const bool few = n_left <= kTopThreads;   // one to a thread
  if (!few) {
    for (int i = tid; i < n_left; i += kTopThreads)
      if (tops[i] >= t) {
        const unsigned k = atomicAdd(&sh.n_left, 1u);
        if (k < kTopLeft) sh.lefts[k] = i;
      }
    __syncthreads();
    whole = sh.n_left <= kTopLeft;
    n_left = static_cast<int>(whole ? sh.n_left : 0u);
  }
  for (int j = tid; j < n_left; j += kTopThreads) {
    const int i = few ? j : sh.lefts[j];
    if (few && tops[i] < t) continue;
    const int noted = places[i], first = noted < 0 ? ~noted : noted;
    uint4 w[kTopUnroll];
    if (i < P.held) {
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) w[q] = held[q * P.held + i];
    } else {
#pragma unroll
      for (int q = 0; q < kTopUnroll; ++q) {
        const int v = first + q * kTopThreads;
        w[q] = noted >= 0 && v < v1 ? load_vec16(row + (static_cast<long long>(v) * N - shift) * ELT) : VT::neg_inf();
      }
      if (noted < 0) w[0] = load_row_vec<ELT>(row, P.V, shift, first);
    }
    unsigned in = 0;                     // the vectors with a token at or above t
#pragma unroll
    for (int q = 0; q < kTopUnroll; ++q) {
      const uint4 one[1] = {w[q]};
      in |= static_cast<unsigned>(VT::vmax(one) >= t) << q;
    }
    for (; in; in &= in - 1) {
      const int q = __ffs(in) - 1;
      const uint4 one = q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3];
      float z[N];
      VT::unpack(one, z);
      unsigned hits = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) hits |= static_cast<unsigned>(z[e] >= t) << e;
      unsigned at = atomicAdd(&sh.n_tokens, static_cast<unsigned>(__popc(hits)));
      const int t0 = (first + q * kTopThreads) * N - shift;
      for (; hits; hits &= hits - 1, ++at) {
        const int e = __ffs(hits) - 1;
        if (at < static_cast<unsigned>(P.cap)) tokens[at] = top_entry(top_key(element_of<ELT>(one, e)), static_cast<uint32_t>(t0 + e));
      }
    }
  }
  if (rank != 0) {
    __syncthreads();
    // at most P.push: where there are more, the K largest
    unsigned n = sh.n_tokens;
    const key64* from = tokens;
    if (n > static_cast<unsigned>(P.push) && n <= static_cast<unsigned>(P.cap)) {
      select_entries(sh, tokens, static_cast<int>(n), P.K, top_key(t), 0xffffffffu);
      from = sh.list;
      n = P.K;
    }
    if (tid == 0) {
      const bool lost = !whole || n > static_cast<unsigned>(P.cap);
      if (lost) first_add(&sh.lost, 1u);
      sh.base = first_add(&sh.n_tokens, lost ? 0u : n);
      if (lost) sh.n_tokens = 0;
    }
    __syncthreads();
    if (sh.n_tokens)
      for (unsigned i = tid; i < n; i += kTopThreads)
        if (sh.base + i < static_cast<unsigned>(P.cap)) first_store(&tokens[sh.base + i], from[i]);
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
  float M = sh.M[0], S = sh.S[0], t_min = sh.t[0], t_max = sh.t[0];
  if (ctas > 1) {
    for (int c = 1; c < ctas; ++c) M = fmax_nan(M, sh.M[c]), t_min = fminf(t_min, sh.t[c]), t_max = fmaxf(t_max, sh.t[c]);
    S = 0.f;
    for (int c = 0; c < ctas; ++c)
      if (sh.M[c] > -INFINITY) S += sh.S[c] * fast_exp2(__fsub_rn(top_base(sh.M[c], P.c2), top_base(M, P.c2)));
  }
  const bool far = top_far(M, P.c2);
  if (far && isfinite(M)) S = sum_again<ELT>(sh, row, P.V, M, P.c2);
  const bool valid = S > 0.f && isfinite(S) && isfinite(M);   // not NaN, +inf, or nothing but -inf
  // ln S and ln 2 (K0 - M c)
  const float K0 = __fmul_rn(M, P.c2), residue = far ? 0.f : -__fmaf_rn(M, P.c2, -K0);
  const float L = __fmaf_rn(0.6931471805599453f, residue, logf(S));
  int listed = 0, n_ranked = 0;        // entries of the list, and those that are ranked for it
  const key64* from = tokens;
  if (valid) {
    const bool fits = !sh.lost && sh.n_tokens <= static_cast<unsigned>(P.cap);
    n_ranked = static_cast<int>(sh.n_tokens);
    listed = fits ? min(P.K, n_ranked) : P.K;
    if (!fits || n_ranked > kTopCount) {
      // more candidates than the buffers hold are K of them at least
      if (fits) select_entries(sh, tokens, n_ranked, listed, top_key(t_min), top_key(M));
      else select_from_row<ELT>(sh, row, P.V, listed, t_max, M, tokens, P.cap);
      from = sh.list;
      n_ranked = listed;
    }
  }
  // ---- in order: of a few, four neighbours count the larger ones of an entry;
  // of more every warp sorts 32, an entry a thread, and looks each up in the
  // other warps' lists
  static_assert(kTopThreads >= kTopCount && kTopThreads >= kTopMaxK, "an entry a thread");
  key64 mine;
  int to = tid;
  if (n_ranked <= kTopThreads / 4) {
    mine = from[min(tid >> 2, max(n_ranked, 1) - 1)];
    to = 0;
    for (int i = tid & 3; i < n_ranked; i += 4) to += from[i] > mine;
    to += __shfl_xor_sync(0xffffffffu, to, 1);
    to += __shfl_xor_sync(0xffffffffu, to, 2);
    if ((tid & 3) || (tid >> 2) >= n_ranked) to = kTopMaxK;
  } else {
    mine = tid < n_ranked ? from[tid] : 0;   // (0 is less than any)
    const int lists = (n_ranked + 31) / 32;
    if (warp < lists) {
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
          const key64 other = __shfl_xor_sync(0xffffffffu, mine, o);
          const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
          mine = (mine > other) == keep_max ? mine : other;
        }
    }
    __syncthreads();                       // `from` may be the list
    sh.list[tid] = mine;
    __syncthreads();
    to = kTopMaxK;
    if (mine != 0) {
      to = lane;
      for (int w0 = 0; w0 < lists; w0 += 4) {
        int larger[4] = {0, 0, 0, 0};
#pragma unroll
        for (int step = 16; step > 0; step >>= 1)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (sh.list[(w0 + q) * 32 + larger[q] + step - 1] > mine) larger[q] += step;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          larger[q] += sh.list[(w0 + q) * 32 + larger[q]] > mine;
          if (w0 + q != warp) to += larger[q];
        }
      }
    }
  }
  if (to < listed) {
    const float z = key_value(static_cast<uint32_t>(mine >> 32));
    ids[to] = static_cast<int>(~static_cast<uint32_t>(mine));
    // (the lowest values below a maximum of 1e32 and more: a difference past the
    // range, of which a T above 1 may leave a number)
    const float d = __fsub_rn(z, M);
    const float at = d > -INFINITY ? __fdiv_rn(d, P.T) : __fsub_rn(__fdiv_rn(z, P.T), __fdiv_rn(M, P.T));
    logp[to] = __fsub_rn(at, L);
  }
  for (int j = listed + tid; j < P.K; j += kTopThreads) ids[j] = -1, logp[j] = valid ? -INFINITY : NAN;
  if (tid == 0) P.lse[r] = valid ? __fadd_rn(__fdiv_rn(M, P.T), L) : M == -INFINITY ? -INFINITY : NAN;
}

template <int ELT>
cudaError_t launch_top(TopParams p, int rows, cudaStream_t s) {
  // A row is split only where there are few, as each part has its own first
  // tile, in which little is known of t, and its own end; half a tile at least
  // to each part.  The parts of long lists cost more to join, so only long rows
  // are split for them, and where the SMs have about a row each, two CTAs to a
  // row are for long rows alone.  In us, split and whole, bf16:
  //   16 rows of  32000: K=64  8.6 and  8.4, K=128 14.9 and 11.1
  //   16 rows of  64000: K=64  9.1 and 11.4, K=128 15.4 and 13.8
  //   16 rows of 128256: K=64 11.2 and 15.9, K=128 16.5 and 18.9, K=256 20.8 and 21.2
  //  140 rows of  64000: K=64 14.7 and 12.0, K=128 19.0 and 14.5
  //  140 rows of 128256: K=64 18.0 and 19.4, K=128 23.8 and 22.3
  //  140 rows of 262144: K=64 24.8 and 31.3, K=128 32.7 and 34.6
  const int nvec = p.V / Vec<ELT>::N, most = p.K > 128 ? 4 : 8;
  const int least = rows > kTopSms / 2 ? (p.K > 64 ? 20 : 12) : p.K > 64 ? 12 : 4;   // tiles
  int cluster = 1;
  while (cluster < most && static_cast<long long>(rows) * 2 * cluster <= 2 * kTopSms && nvec >= least * kTopTile &&
         nvec / (2 * cluster) >= kTopTile / 2)
    cluster *= 2;
  // long lists note more, which is read again; short ones keep it all
  p.places = p.K > 64 ? 1792 : 1024;
  // a long row notes as many again each time its length doubles (384 fp32 rows
  // of 262144, K=256: 79 us, with 1792 places 203 us as they run out; 2 % more
  // at 100000 where they do not, as the rows' loads have less L1)
  if (nvec / cluster > 20 * kTopTile) p.places += p.K > 64 ? 1280 : 512;
  p.held = p.K > 64 ? 0 : 256;
  p.cap = cluster > 1 ? 1792 : p.K > 64 ? 1280 : 768;
  const int smem = kTopBuffersAt + p.cap * 8 + p.held * kTopUnroll * 16 + p.places * 8;
  // long rows split in two take more than the 48 KB that need no asking
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(top_kernel<ELT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
  cfg.blockDim = dim3(kTopThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, top_kernel<ELT>, p);
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
              static_cast<float>(c2), temperature, (K + kTopWarps - 1) / kTopWarps, K > 128 ? 256 : 192};
  const int rows = n_seq * t_len;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("spec_kd_top");
  const cudaError_t e = elt == 2 ? launch_top<2>(p, rows, st) : launch_top<4>(p, rows, st);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
