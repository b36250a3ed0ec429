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
// Short rows take a CTA each and stay in its registers.  Longer ones go to
// clusters of 1 to 8 CTAs, two CTAs to an SM, row c + i * clusters to cluster
// c; each CTA takes a part of the row.  A producer warp streams it through a
// ring of three 32 KB slots, 8 consumer warps sum it and, for the
// gradient, take it a second time from L2, where it was a few microseconds
// before.  The ring runs ahead over the end of a row, and the SM's other CTA
// fills what is left of the gap while a row's numbers are put together.  A
// marking warp stands between producer and consumers: it puts -inf in the
// listed tokens' places of a slot, so that the consumers need not look for
// them (a look at a byte a vector was an eighth of their instructions).  Every
// CTA gathers the listed tokens' logits itself, a thread each, so the CTAs of
// a cluster exchange nothing but their (M, S), through distributed shared
// memory; the listed tokens' gradients are stored after the row's.
//
// Every wait has a limit.  A consumer warp whose wait for a slot expires touches
// no barrier of the ring again: its sums and gradients are NaN from there on, so
// that every later row of its cluster is, and the row itself is set to NaN at the
// end (its numbers may have been put together before).  The CTAs of a cluster go
// on exchanging parts.  The producer, which then waits in vain for the slots'
// release, leaves last, when its copies have landed: none is to reach shared
// memory that a later CTA owns.
//
// 4096 rows of 151936 bf16 logits with their gradients: 460 us, 5.4 TB/s of
// each logit read and each gradient written once; the loss alone 189 us, 6.6
// TB/s.  With one CTA to a row the rows at work do not stay in L2 (452 MB read
// for 311 MB of rows) and the gradients take 523 us.  Kept in the registers of
// a cluster's CTAs in place of read twice: 742 us, each CTA idle while the
// row's numbers go round.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_kd.h"
#include "sv_rowsum.cuh"
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
  float c2, inv_T;             // log2(e) / T, 1 / T
  long long wait_limit_ns;     // of a consumer's wait for a slot
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

// p (m - z) / T where (z - m) / T is past the range (the type's lowest value for
// a mask, at a T below 1 or under a maximum of 1e32): p may bring it back.
__device__ __forceinline__ float tl_far(float p, float m, float z, float inv_T) {
  if (!(z > -INFINITY)) return INFINITY;
  const float s = __fmul_rn(p, inv_T), d = __fsub_rn(m, z);
  return d < INFINITY ? __fmul_rn(s, d) : __fsub_rn(__fmul_rn(s, m), __fmul_rn(s, z));
}

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

// The row's numbers from its combined part: Ma = max(M, Ml), Z its whole sum.
__device__ __forceinline__ TlRow tl_row(const TlPart& part, double mass, float scale, const TopLossParams& P) {
  TlRow R;
  R.Ma = fmaxf(part.m, part.ml);
  R.valid = part.s == part.s && R.Ma > -INFINITY && R.Ma < INFINITY;
  // the listed tokens carry most of Z: full-precision exponentials for them
  const float lt = __fmul_rn(__fsub_rn(part.m, R.Ma), P.inv_T);
  const float ft = part.m > -INFINITY ? expf(lt) : 0.f;
  const float fl = part.ml > -INFINITY ? expf(__fmul_rn(__fsub_rn(part.ml, R.Ma), P.inv_T)) : 0.f;
  const float tail = __fmul_rn(part.s, ft);   // of Z
  R.Z = __fadd_rn(tail, __fmul_rn(part.sl, fl));
  R.LZ = logf(R.Z);
  R.mass = static_cast<float>(mass);
  float rest = P.renorm ? 0.f : static_cast<float>(1.0 - mass);
  if (rest < kTlComplete) rest = 0.f;
  R.a = R.valid ? scale * __fsub_rn(__fdiv_rn(ft, R.Z), part.s > 0.f ? __fdiv_rn(rest, part.s) : 0.f) : NAN;
  R.base = part.m > -INFINITY ? part.m : 0.f;
  // r (log r - log(1 - Q)), the logarithm of one ratio where 1 - Q can be
  // written: r and 1 - Q are alike, and their logarithms' roundings are not
  R.kl = 0.f;
  if (rest > 0.f)
    R.kl = tail > 1e-30f         ? rest * logf(__fdiv_rn(__fmul_rn(rest, R.Z), tail))
           : !(part.s > 0.f)     ? INFINITY
           : lt > -INFINITY      ? rest * (logf(rest) - __fsub_rn(__fadd_rn(lt, logf(part.s)), R.LZ))
                                 : tl_far(rest, R.Ma, part.m, P.inv_T);
  return R;
}

// Whether `x` holds for any of the `threads` threads at barrier 1.
__device__ __forceinline__ bool tl_any(bool x, int threads) {
  int any;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.red.or.pred q, 1, %2, p;\n\t"
               "selp.s32 %0, 1, 0, q;\n\t}" : "=r"(any) : "r"(static_cast<int>(x)), "r"(threads) : "memory");
  return any != 0;
}

constexpr int kTrWarps = 8;                           // consumer warps
constexpr int kTrConsumers = kTrWarps * 32;
constexpr int kTrThreads = kTrConsumers + 64;         // + the producer and the marking warp
constexpr int kTrCtas = 2;                            // to an SM
constexpr int kTrSlots = 3;
constexpr int kTrPerLane = 8;                         // vectors per lane and slot
constexpr int kTrSlotVecs = kTrConsumers * kTrPerLane;
constexpr int kTrHash = 1024;                         // places for a row's listed ids

constexpr int kTrGrid = 152 * kTrCtas;                // CTAs that fit at once
constexpr long long kTrInL2 = 72LL << 20;             // bytes of rows at work that L2 keeps
constexpr int kTrMinPart = 16 * 1024;                 // a part's bytes where a row is split for want of rows
// A CTA's parts come within two expired waits for its slots.
constexpr long long kTrJoinLimitNs = 4 * kDrainLimitNs;
constexpr int kTrNoRow = 0x7fffffff;

struct TrShared {
  uint64_t full[kTrSlots], ready[kTrSlots], empty[kTrSlots];
  uint64_t joined[2];            // the cluster's parts of a row are here, by row parity as what follows
  uint4 part[2][kTlMaxCtas];     // the CTAs' (M, S)
  TlPart warp[2][kTrWarps];      // the warps' parts
  double mass[2][kTrWarps];      // P in 64 bits: 1 - P keeps what the log-probabilities have
  float term[2][kTrWarps];
  TlRow row[2];
  int failed;                    // the first row in which a wait expired, or kTrNoRow
  int ids[kTrHash];              // open addressing; -1: empty
};
constexpr int kTrRingAt = (static_cast<int>(sizeof(TrShared)) + 127) / 128 * 128;
constexpr int kTrSmem = kTrRingAt + kTrSlots * kTrSlotVecs * 16;
static_assert(kTrCtas * (kTrSmem + 1024) <= 228 * 1024, "the CTAs must fit on an SM");
static_assert(kTrConsumers >= SV_KD_TOP_MAX, "a thread for each entry of the list");

// Enters an id; its place, or -1 if it is there already.
__device__ __forceinline__ int tr_enter(int* ids, int id) {
  for (unsigned at = static_cast<unsigned>(id) * 2654435761u >> 22;; at = (at + 1) % kTrHash) {
    const int there = atomicCAS(&ids[at], -1, id);
    if (there == -1) return static_cast<int>(at);
    if (there == id) return -1;
  }
}
__device__ __forceinline__ bool tr_listed(const int* ids, int id) {
  for (unsigned at = static_cast<unsigned>(id) * 2654435761u >> 22; ids[at] != -1; at = (at + 1) % kTrHash)
    if (ids[at] == id) return true;
  return false;
}

// A CTA's part of a row's whole vectors: the place of its first one, which of
// the row's vectors that is, and their number (the row's ends are taken apart).
struct TrRow {
  const unsigned char* at;
  int first, n;
  template <int ELT>
  __device__ __forceinline__ static TrRow of(const TopLossParams& P, long long r, int ctas, int rank) {
    constexpr int N = Vec<ELT>::N;
    const unsigned char* row = P.draft + r * P.V * ELT;
    const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
    const int head = shift ? 1 : 0;
    const int all = nvec - head - ((P.V + shift) % N && nvec > head ? 1 : 0);
    const int per = (all + ctas - 1) / ctas;
    TrRow t;
    t.first = head + min(all, rank * per);
    t.n = min(all, rank * per + per) - min(all, rank * per);
    t.at = row + (static_cast<long long>(t.first) * N - shift) * ELT;
    return t;
  }
};

// mbar_wait_bounded for a limit above 0.
__device__ __forceinline__ bool tr_wait(uint64_t* bar, uint32_t parity, long long limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (static_cast<long long>(global_ns() - t0) >= limit_ns) return false;
  return true;
}

// NaN in place of this thread's gradients of a part.
template <int ELT>
__device__ __noinline__ void tr_nan_gradient(unsigned char* grad, int V, int first, int n, int shift, int same_shift) {
  const uint32_t x = 0x7fc07fc0u;   // in either type
  for (int v = threadIdx.x; v < n; v += kTrConsumers)
    store_edge<ELT>(grad, V, (first + v) * Vec<ELT>::N - shift, same_shift, make_uint4(x, x, x, x));
}

// Whether a row has a list, and whether anything is wrong with it, by one warp.
__device__ __forceinline__ bool tr_has_list(const TopLossParams& P, long long r, int lane) {
  bool any = false;
  for (int j = lane; j < P.K; j += 32) {
    const float lp = P.logp[r * P.K + j];
    any |= P.ids[r * P.K + j] >= 0 || lp != lp || lp == INFINITY;
  }
  return __any_sync(0xffffffffu, any);
}

template <int ELT, bool GRAD>
__global__ void __launch_bounds__(kTrThreads, kTrCtas) toploss_kernel(const __grid_constant__ TopLossParams P, int rows) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  extern __shared__ __align__(1024) unsigned char smem[];
  TrShared& sh = *reinterpret_cast<TrShared*>(smem);
  unsigned char* ring = smem + kTrRingAt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster_ctas(), rank = cluster_rank();
  const int cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas;
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) mbar_init(&sh.joined[b], 1);
    for (int s = 0; s < kTrSlots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.ready[s], 1);
      mbar_init(&sh.empty[s], kTrWarps + 1);
    }
    sh.failed = kTrNoRow;
    fence_mbar_init();
  }
  for (int w = tid; w < kTrHash; w += kTrThreads) sh.ids[w] = -1;
  if (ctas > 1) cluster_sync();   // the others' barriers are set up too
  else __syncthreads();
  grid_dependents_launch();       // the sum of the rows may take its place on an SM

  if (warp == kTrWarps) {
    // ---- the producer: every row with a list once, for the gradient twice
    const uint64_t first_out = evict_first_policy();
    unsigned q = 0;
    bool given_up = false;
    for (long long r = cluster; r < rows && !given_up; r += clusters) {
      if (!tr_has_list(P, r, lane)) continue;
      const TrRow row = TrRow::of<ELT>(P, r, ctas, rank);
      for (int pass = 0; pass < (GRAD ? 2 : 1) && !given_up; ++pass)
        for (int v = 0; v < row.n; v += kTrSlotVecs, ++q) {
          const int s = q % kTrSlots;
          int ok = 1;
          if (lane == 0) ok = mbar_wait_bounded(&sh.empty[s], ((q / kTrSlots) & 1) ^ 1, kDrainLimitNs) ? 1 : 0;
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            given_up = true;             // as a consumer or the marking warp has
            break;
          }
          if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(min(kTrSlotVecs, row.n - v)) * 16u;
            const unsigned char* src = row.at + static_cast<long long>(v) * 16;
            mbar_expect_tx(&sh.full[s], bytes);
            // the last read of a row marks its lines first out of L2
            if (GRAD && pass == 0) bulk_load(ring + s * kTrSlotVecs * 16, src, bytes, &sh.full[s]);
            else bulk_load_hint(ring + s * kTrSlotVecs * 16, src, bytes, &sh.full[s], first_out);
          }
        }
    }
    // the last copy of every slot has landed, whether it was waited for or not
    if (lane == 0)
      for (unsigned i = q > kTrSlots ? q - kTrSlots : 0; i < q; ++i)
        mbar_wait_bounded(&sh.full[i % kTrSlots], (i / kTrSlots) & 1u, kDrainLimitNs);
    return;
  }

  if (warp == kTrWarps + 1) {
    // ---- the marking warp: the listed tokens out of the first pass's slots
    unsigned q = 0;
    for (long long r = cluster; r < rows; r += clusters) {
      if (!tr_has_list(P, r, lane)) continue;
      const TrRow row = TrRow::of<ELT>(P, r, ctas, rank);
      const int t_first = static_cast<int>((row.at - (P.draft + r * P.V * ELT)) / ELT);   // the first slot's first token
      int at[SV_KD_TOP_MAX / 32];
#pragma unroll
      for (int k = 0; k < SV_KD_TOP_MAX / 32; ++k) {
        const int j = k * 32 + lane, id = j < P.K ? P.ids[r * P.K + j] : -1;
        at[k] = id >= 0 && id < P.V ? id - t_first : -1;
      }
      for (int pass = 0; pass < (GRAD ? 2 : 1); ++pass)
        for (int v = 0; v < row.n; v += kTrSlotVecs, ++q) {
          const int s = q % kTrSlots;
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[s], (q / kTrSlots) & 1u, kDrainLimitNs))) return;
          if (pass == 0) {
            unsigned char* slot = ring + s * kTrSlotVecs * 16;
            const unsigned n = static_cast<unsigned>(min(kTrSlotVecs, row.n - v)) * N;
#pragma unroll
            for (int k = 0; k < SV_KD_TOP_MAX / 32; ++k) {
              const int in = at[k] - v * N;
              if (at[k] >= 0 && static_cast<unsigned>(in) < n) VT::store_scalar(slot, in, -INFINITY);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the slot is filled again
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.ready[s]);
            mbar_arrive(&sh.empty[s]);
          }
        }
    }
    return;
  }

  // ---- the consumers
  const f2 cc = pack2(P.c2, P.c2);
  unsigned q = 0;
  // a wait of this warp has expired: what it adds is NaN (a limit of 0, at which
  // every wait expires, is looked at here once: at each wait it took 1 % of rows
  // of 40 KB)
  bool dead = P.wait_limit_ns <= 0;
  bool alone = false;            // (warp 0) the others' parts did not come
  int turn = 0, alone_turn = 0;
  // this lane's vectors of the slot, -inf past the row's; the slot is released
  // as soon as they are in registers.  After an expired wait they are whatever
  // lies there, and the caller makes NaN of it once a row (at each slot it took
  // 2 % of rows of 64 KB).
  auto take = [&](uint4 (&w)[kTrPerLane], int n, bool marked) {
    const int s = q % kTrSlots;
    const uint32_t phase = (q / kTrSlots) & 1u;
    bool ok = !dead && tr_wait(&sh.full[s], phase, P.wait_limit_ns);
    if (marked) ok = ok && tr_wait(&sh.ready[s], phase, P.wait_limit_ns);
    dead = !__all_sync(0xffffffffu, ok);
    const uint4* src = reinterpret_cast<const uint4*>(ring + s * kTrSlotVecs * 16) + tid;
    if (n >= kTrSlotVecs) {
#pragma unroll
      for (int k = 0; k < kTrPerLane; ++k) w[k] = src[k * kTrConsumers];
    } else {
#pragma unroll
      for (int k = 0; k < kTrPerLane; ++k) w[k] = tid + k * kTrConsumers < n ? src[k * kTrConsumers] : VT::neg_inf();
    }
    __syncwarp();
    if (lane == 0 && !dead) mbar_arrive(&sh.empty[s]);
    ++q;
  };
  // the next row's list is loaded while this one is at work
  int next_id = -1;
  float next_lp = -INFINITY, next_weight = 0.f;
  auto load_list = [&](long long r) {
    if (r >= rows) return;
    if (tid < P.K) {
      next_id = P.ids[r * P.K + tid];
      next_lp = P.logp[r * P.K + tid];
    }
    if (GRAD) next_weight = P.weights[r / P.t_len];
  };
  load_list(cluster);
  for (long long r = cluster; r < rows; r += clusters) {
    unsigned char* grad = GRAD ? P.grad + r * P.V * ELT : nullptr;
    const unsigned char* start = P.draft + r * P.V * ELT;
    const int shift = row_shift<ELT>(start), nvec = row_vecs<ELT>(P.V, shift);
    // ---- the list: thread j holds entry j
    int id = next_id;
    float lp = next_lp;
    const float weight = GRAD ? next_weight : 0.f;
    load_list(r + clusters);
    bool bad = lp != lp || lp == INFINITY || id >= P.V;
    if (id >= P.V) id = -1;
    if (!tl_any(id >= 0 || bad, kTrConsumers)) {         // no list: no loss
      if (tid == 0 && rank == 0) P.row_kl[r] = 0.f;
      if (GRAD)
        for (int v = rank * kTrConsumers + tid; v < nvec; v += ctas * kTrConsumers) {
          const int t0 = v * N - shift;
          if (P.same_shift && t0 >= 0 && t0 <= P.V - N) {
            store_vec16(grad + static_cast<long long>(t0) * ELT, make_uint4(0, 0, 0, 0));
          } else {
            for (int e = 0; e < N; ++e)
              if (t0 + e >= 0 && t0 + e < P.V) VT::store_rounded(grad, t0 + e, 0.f);
          }
        }
      continue;
    }
    const int par = turn & 1, phase = turn >> 1 & 1;
    ++turn;                                // rows with a list
    float zj = -INFINITY, p = 0.f;
    int place = -1;
    if (id >= 0) {
      place = tr_enter(sh.ids, id);
      bad |= place < 0;                    // listed twice
      zj = load_elem<ELT>(start, id);
      p = expf(lp);
    }
    const TrRow row = TrRow::of<ELT>(P, r, ctas, rank);
    named_barrier_sync(1, kTrConsumers);

    // ---- the unlisted tokens: running maximum and sum per lane
    float m = -INFINITY;
    f2 s2 = 0ull, s3 = 0ull;
    auto add = [&](const auto& w) {        // an array of vectors
      const float vm = VT::vmax(w);        // NaN is passed over here and kept by the sum
      if (vm > m) {
        const float f = m > -INFINITY ? fast_exp2(__fmul_rn(__fsub_rn(m, vm), P.c2)) : 0.f;
        s2 = mul2(s2, pack2(f, f));
        s3 = mul2(s3, pack2(f, f));
        m = vm;
      }
      const float mb = m > -INFINITY ? m : 0.f;
      const f2 mm = pack2(mb, mb);
#pragma unroll
      for (const uint4& x : w) {
        f2 z[N / 2];
        VT::pairs(x, z);
#pragma unroll
        for (int i = 0; i < N / 2; i += 2) {
          s2 = add2(s2, exp2_2(mul2(sub2(z[i], mm), cc)));
          s3 = add2(s3, exp2_2(mul2(sub2(z[i + 1], mm), cc)));
        }
      }
    };
    // the row's ends, where they are not whole vectors, by two threads of the
    // first CTA
    int end = -1;
    if (rank == 0 && tid == 0 && shift) end = 0;
    if (rank == 0 && tid == 1 && (P.V + shift) % N && nvec > (shift ? 1 : 0)) end = nvec - 1;
    uint4 end_vec = VT::neg_inf();
    if (end >= 0) end_vec = load_row_vec<ELT>(start, P.V, shift, end);
    for (int v = 0; v < row.n; v += kTrSlotVecs) {
      uint4 w[kTrPerLane];
      take(w, row.n - v, true);
      if (row.n - v > kTrSlotVecs / 2) {
        add(w);
      } else {   // a last slot of half the vectors at most (10000 rows of 20000: 2 % less than as a whole one)
        uint4 half[kTrPerLane / 2];
#pragma unroll
        for (int k = 0; k < kTrPerLane / 2; ++k) half[k] = w[k];
        add(half);
      }
    }
    if (end >= 0) {
      uint32_t in = 0;
      for (int e = 0; e < N; ++e) {
        const int t = end * N - shift + e;
        if (t >= 0 && t < P.V) in |= static_cast<uint32_t>(tr_listed(sh.ids, t)) << e;
      }
      const uint4 one[1] = {with_neg_inf<ELT>(end_vec, in)};
      add(one);
    }
    bad |= zj != zj || zj == INFINITY;
    float s, s_hi;
    unpack2(add2(s2, s3), s, s_hi);
    TlPart part{m, s + s_hi, zj, zj > -INFINITY ? 1.f : 0.f};
    if (bad || dead) part.s = NAN;
    part = tl_combine(part, P.c2, P.inv_T);
    double mass = warp * 32 < P.K ? warp_sum(static_cast<double>(p)) : 0.0;
    if (lane == 0) sh.warp[par][warp] = part, sh.mass[par][warp] = mass;
    named_barrier_sync(1, kTrConsumers);
    if (place >= 0) sh.ids[place] = -1;

    // ---- the row's numbers, by one warp for all
    const float scale = weight * P.inv_T;
    if (warp == 0) {
      const TlPart none{-INFINITY, 0.f, -INFINITY, 0.f};
      part = tl_combine(lane < kTrWarps ? sh.warp[par][lane] : none, P.c2, P.inv_T);
      if (ctas > 1) {
        TlPart other = none;
        if (!alone) {
          if (lane == 0) mbar_expect_tx(&sh.joined[par], static_cast<uint32_t>(ctas) * 16u);
          if (lane < ctas)
            st_async(peer(&sh.part[par][rank], lane), make_uint4(__float_as_uint(part.m), __float_as_uint(part.s), 0u, 0u),
                     peer(&sh.joined[par], lane));
          alone = !__all_sync(0xffffffffu, mbar_wait_bounded(&sh.joined[par], static_cast<uint32_t>(phase), kTrJoinLimitNs));
          if (alone && lane == 0) {
            // another CTA may still get here and on to the next row, where it
            // waits in vain: what it sends until then is waited for at the end
            mbar_expect_tx(&sh.joined[par ^ 1], static_cast<uint32_t>(ctas) * 16u);
            atomicMin(&sh.failed, static_cast<int>(r));
          }
          if (alone) alone_turn = turn - 1;
          if (lane < ctas && !alone) {
            const uint4 x = sh.part[par][lane];
            other.m = __uint_as_float(x.x);
            other.s = __uint_as_float(x.y);
          }
        }
        other = tl_combine(other, P.c2, P.inv_T);
        part.m = other.m;
        part.s = alone ? NAN : other.s;
      }
      mass = sh.mass[par][lane % kTrWarps];
#pragma unroll
      for (int o = kTrWarps / 2; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
      const TlRow mine = tl_row(part, mass, scale, P);
      if (lane == 0) sh.row[par] = mine;
    }
    named_barrier_sync(1, kTrConsumers);
    const TlRow R = sh.row[par];

    // ---- the gradient
    if (GRAD) {
      const f2 bb = pack2(R.base, R.base), aa = pack2(R.a, R.a);
      auto gradient = [&](const uint4& x) {
        f2 z[N / 2];
        float g[N];
        VT::pairs(x, z);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) unpack2(mul2(aa, exp2_2(mul2(sub2(z[i], bb), cc))), g[2 * i], g[2 * i + 1]);
        return VT::pack(g);
      };
      unsigned char* out = grad + (static_cast<long long>(row.first) * N - shift) * ELT;
      for (int v = 0; v < row.n; v += kTrSlotVecs) {
        uint4 w[kTrPerLane];
        take(w, row.n - v, false);
        unsigned char* at = out + static_cast<long long>(v + tid) * 16;
        if (P.same_shift && row.n - v >= kTrSlotVecs) {
#pragma unroll
          for (int k = 0; k < kTrPerLane; ++k) store_vec16(at + k * kTrConsumers * 16, gradient(w[k]));
        } else {
#pragma unroll
          for (int k = 0; k < kTrPerLane; ++k)
            if (v + tid + k * kTrConsumers < row.n)
              store_edge<ELT>(grad, P.V, (row.first + v + tid + k * kTrConsumers) * N - shift, P.same_shift, gradient(w[k]));
        }
      }
      if (end >= 0) store_edge<ELT>(grad, P.V, end * N - shift, P.same_shift, gradient(end_vec));
      if (dead) tr_nan_gradient<ELT>(grad, P.V, row.first, row.n, shift, P.same_shift);
    }
    if (dead && lane == 0) atomicMin(&sh.failed, static_cast<int>(r));

    // ---- the listed tokens: their gradients after the row's, and the divergence
    const float lj = __fmul_rn(__fsub_rn(zj, R.Ma), P.inv_T);
    if (P.renorm) {
      lp = R.mass > 0.f ? __fsub_rn(lp, logf(R.mass)) : -INFINITY;
      p = R.mass > 0.f ? __fdiv_rn(p, R.mass) : 0.f;
    }
    float term = 0.f;
    if (id >= 0 && p > 0.f)
      term = lj > -INFINITY ? __fmul_rn(p, __fsub_rn(lp, __fsub_rn(lj, R.LZ))) : tl_far(p, R.Ma, zj, P.inv_T);
    term = warp_sum(term);
    if (lane == 0) sh.term[par][warp] = term;
    named_barrier_sync(1, kTrConsumers);
    const bool valid = R.valid && !dead;
    const int in_row = id + shift, v_id = in_row / N - row.first;   // the entry's vector, in this part or not
    const bool at_end = rank == 0 && ((shift && in_row < N) || (in_row / N == nvec - 1 && (P.V + shift) % N));
    if (GRAD && id >= 0 && ((v_id >= 0 && v_id < row.n) || at_end)) {
      const float qj = zj > -INFINITY ? __fdiv_rn(expf(lj), R.Z) : 0.f;
      VT::store_rounded(grad, id, valid ? scale * __fsub_rn(qj, p) : NAN);
    }
    if (tid == 0 && rank == 0) {
      float kl = R.kl;
      for (int w = 0; w < kTrWarps; ++w) kl += sh.term[par][w];
      P.row_kl[r] = valid ? kl : NAN;
    }
  }
  if (ctas > 1) {
    cluster_sync();              // nothing will be sent to a CTA that has left, nor is it on its way:
    if (alone)
      for (int t = alone_turn; t < alone_turn + 2; ++t)
        mbar_wait_bounded(&sh.joined[t & 1], static_cast<uint32_t>(t >> 1 & 1), kDrainLimitNs);
  } else {
    named_barrier_sync(1, kTrConsumers);
  }
  // the row in which a wait expired, its divergence perhaps stored before
  if (tid == 0 && sh.failed != kTrNoRow) P.row_kl[sh.failed] = NAN;
}

// ---- short rows: a CTA to a row, which stays in its registers
//
// What a streamed row costs besides its bytes (the ring's hand-overs, five
// barriers and a list among two CTAs an SM, 5 us) is more than a short row's
// time on the wire; here twice the CTAs work at once and the row is read once.
// Bound by its instructions: the list and the row's numbers cost as much as
// 8000 logits (with every warp working out the row's numbers for itself 50000
// rows of 4000 took 391 us where they take 359, with lists of 64).  Eight
// vectors of bf16 with the gradient spill 48 bytes at three CTAs an SM.
constexpr int kTsThreads = 256, kTsWarps = kTsThreads / 32;
static_assert(kTsThreads >= SV_KD_TOP_MAX && kTsWarps == kTrWarps, "a thread for each entry of the list");

template <int ELT, int U, bool GRAD>
__global__ void __launch_bounds__(kTsThreads, U > 4 ? 3 : 4) toploss_short_kernel(const __grid_constant__ TopLossParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  __shared__ uint32_t listed[kTsThreads * U * N / 32];   // a bit for each place of the row's vectors
  __shared__ TlPart parts[kTsWarps];
  __shared__ double masses[kTsWarps];
  __shared__ float terms[kTsWarps];
  __shared__ TlRow total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long r = blockIdx.x;
  unsigned char* grad = GRAD ? P.grad + r * P.V * ELT : nullptr;
  const unsigned char* row = P.draft + r * P.V * ELT;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  // ---- every load goes out at once; thread j holds entry j of the list
  int id = -1;
  float lp = -INFINITY;
  if (tid < P.K) {
    id = P.ids[r * P.K + tid];
    lp = P.logp[r * P.K + tid];
  }
  const float weight = GRAD ? P.weights[r / P.t_len] : 0.f;
  uint4 w[U];
#pragma unroll
  for (int k = 0; k < U; ++k)
    w[k] = tid + k * kTsThreads < nvec ? load_row_vec<ELT>(row, P.V, shift, tid + k * kTsThreads) : VT::neg_inf();
  for (int i = tid; i < kTsThreads * U * N / 32; i += kTsThreads) listed[i] = 0;
  grid_dependents_launch();
  bool bad = lp != lp || lp == INFINITY || id >= P.V;
  if (id >= P.V) id = -1;
  if (!__syncthreads_or(id >= 0 || bad)) {             // no list: no loss
    if (tid == 0) P.row_kl[r] = 0.f;
    if (GRAD)
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (tid + k * kTsThreads < nvec)
          store_edge<ELT>(grad, P.V, (tid + k * kTsThreads) * N - shift, P.same_shift, make_uint4(0, 0, 0, 0));
    return;
  }
  float zj = -INFINITY, p = 0.f;
  if (id >= 0) {
    const uint32_t bit = 1u << ((id + shift) & 31);
    bad |= (atomicOr(&listed[(id + shift) >> 5], bit) & bit) != 0;   // listed twice
    zj = load_elem<ELT>(row, id);
    p = expf(lp);
  }
  __syncthreads();

  // ---- the unlisted tokens' maximum and sum
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int at = (tid + k * kTsThreads) * N;
    const uint32_t in = (listed[at >> 5] >> (at & 31)) & ((1u << N) - 1u);
    if (in) w[k] = with_neg_inf<ELT>(w[k], in);
  }
  const f2 cc = pack2(P.c2, P.c2);
  const float m = VT::vmax(w);             // NaN is passed over here and kept by the sum
  const float mb = m > -INFINITY ? m : 0.f;
  const f2 mm = pack2(mb, mb);
  f2 s2 = 0ull, s3 = 0ull;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    f2 z[N / 2];
    VT::pairs(w[k], z);
#pragma unroll
    for (int i = 0; i < N / 2; i += 2) {
      s2 = add2(s2, exp2_2(mul2(sub2(z[i], mm), cc)));
      s3 = add2(s3, exp2_2(mul2(sub2(z[i + 1], mm), cc)));
    }
  }
  bad |= zj != zj || zj == INFINITY;
  float s, s_hi;
  unpack2(add2(s2, s3), s, s_hi);
  TlPart part{m, s + s_hi, zj, zj > -INFINITY ? 1.f : 0.f};
  if (bad) part.s = NAN;
  part = tl_combine(part, P.c2, P.inv_T);
  double mass = warp * 32 < P.K ? warp_sum(static_cast<double>(p)) : 0.0;
  if (lane == 0) parts[warp] = part, masses[warp] = mass;
  __syncthreads();

  // ---- the row's numbers, by one warp for all
  const float scale = weight * P.inv_T;
  if (warp == 0) {
    const TlPart none{-INFINITY, 0.f, -INFINITY, 0.f};
    part = tl_combine(lane < kTsWarps ? parts[lane] : none, P.c2, P.inv_T);
    mass = masses[lane % kTsWarps];
#pragma unroll
    for (int o = kTsWarps / 2; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    const TlRow mine = tl_row(part, mass, scale, P);
    if (lane == 0) total = mine;
  }
  __syncthreads();
  const TlRow R = total;

  // ---- the gradient, the listed tokens' after the others'
  if (GRAD) {
    const f2 bb = pack2(R.base, R.base), aa = pack2(R.a, R.a);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      f2 z[N / 2];
      float g[N];
      VT::pairs(w[k], z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) unpack2(mul2(aa, exp2_2(mul2(sub2(z[i], bb), cc))), g[2 * i], g[2 * i + 1]);
      const int v = tid + k * kTsThreads, t0 = v * N - shift;
      if (P.same_shift && t0 >= 0 && t0 <= P.V - N) store_vec16(grad + static_cast<long long>(t0) * ELT, VT::pack(g));
      else if (v < nvec) store_edge<ELT>(grad, P.V, t0, P.same_shift, VT::pack(g));
    }
  }
  const float lj = __fmul_rn(__fsub_rn(zj, R.Ma), P.inv_T);
  if (P.renorm) {
    lp = R.mass > 0.f ? __fsub_rn(lp, logf(R.mass)) : -INFINITY;
    p = R.mass > 0.f ? __fdiv_rn(p, R.mass) : 0.f;
  }
  float term = 0.f;
  if (id >= 0 && p > 0.f)
    term = lj > -INFINITY ? __fmul_rn(p, __fsub_rn(lp, __fsub_rn(lj, R.LZ))) : tl_far(p, R.Ma, zj, P.inv_T);
  term = warp_sum(term);
  if (lane == 0) terms[warp] = term;
  __syncthreads();
  if (GRAD && id >= 0) {
    const float qj = zj > -INFINITY ? __fdiv_rn(expf(lj), R.Z) : 0.f;
    VT::store_rounded(grad, id, R.valid ? scale * __fsub_rn(qj, p) : NAN);
  }
  if (tid == 0) {
    float kl = R.kl;
    for (int i = 0; i < kTsWarps; ++i) kl += terms[i];
    P.row_kl[r] = R.valid ? kl : NAN;
  }
}

template <int ELT>
cudaError_t launch_toploss(const TopLossParams& p, int rows, cudaStream_t s) {
  // Few rows: as many CTAs to a row as give the SMs work (a row of 128256 bf16
  // logits: 16.6 us with one, 8.7 us with eight).  Many rows with a gradient:
  // two where the rows at work would not stay in L2 for their second reading
  // (more than two wait for one another longer than that saves: 888 us with
  // four).
  const long long row_bytes = static_cast<long long>(p.V) * ELT;
  // Rows that fit in a CTA's registers, up to 32 KB, the lists' bits with them
  // (two vectors more for a row off the 16-byte boundary): 50000 bf16 rows of
  // 4000 logits with gradients 359 us, streamed 790; 25000 of 8000 256 and 427;
  // 12500 of 16000 249 and 263; 16 of 16000 8.6 and 9.2.
  const int vecs = static_cast<int>(row_bytes / 16) + 2;
  if (vecs <= 8 * kTsThreads) {
    auto launch = [&](auto kernel) {
      kernel<<<static_cast<unsigned>(rows), kTsThreads, 0, s>>>(p);
      return cudaGetLastError();
    };
#define SV_LAUNCH(U) (p.grad ? launch(toploss_short_kernel<ELT, U, true>) : launch(toploss_short_kernel<ELT, U, false>))
    return vecs <= 2 * kTsThreads ? SV_LAUNCH(2) : vecs <= 4 * kTsThreads ? SV_LAUNCH(4) : SV_LAUNCH(8);
#undef SV_LAUNCH
  }
  int cluster = 1;
  while (cluster < kTlMaxCtas && rows * 2 * cluster <= kTrGrid && row_bytes / (2 * cluster) >= kTrMinPart) cluster *= 2;
  if (cluster == 1 && p.grad && (rows < kTrGrid ? rows : kTrGrid) * row_bytes > kTrInL2) cluster = 2;
  const void* fn = p.grad ? reinterpret_cast<const void*>(&toploss_kernel<ELT, true>)
                          : reinterpret_cast<const void*>(&toploss_kernel<ELT, false>);
  // the shared-memory limit, raised once per instance and device
  static std::atomic<unsigned long long> raised[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ULL << (dev & 63);
  if (dev >= 64 || !(raised[p.grad != nullptr].load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTrSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised[p.grad != nullptr].fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  const int clusters = kTrGrid / cluster;
  cfg.gridDim = dim3(static_cast<unsigned>((rows < clusters ? rows : clusters) * cluster));
  cfg.blockDim = dim3(kTrThreads);
  cfg.dynamicSmemBytes = kTrSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return p.grad ? cudaLaunchKernelEx(&cfg, toploss_kernel<ELT, true>, p, rows)
                : cudaLaunchKernelEx(&cfg, toploss_kernel<ELT, false>, p, rows);
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
                  static_cast<float>(c2), 1.f / temperature, kd_wait_limit_ns()};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("spec_kd_top_loss");
  const int rows = n_seq * t_len;
  const cudaError_t e = elt == 2 ? launch_toploss<2>(p, rows, s) : launch_toploss<4>(p, rows, s);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  if (launch_row_sum(n_seq, t_len, row_kl, weights, loss, s) != cudaSuccess) return SV_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
