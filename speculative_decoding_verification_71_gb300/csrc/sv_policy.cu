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
// Short rows stay in the registers of a few warps, long ones in the shared memory
// of a cluster, so that each is read once.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_kd.h"
#include "sv_policy.h"
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
  float4* kept;                // [rows]: base, 1 / Z, 1 - p(x), what logp's rounding left (tok_kept), or null
  float* row_loss;             // [rows]: a policy's loss; null for the log-probabilities alone
  unsigned char* grad;         // [rows, V] or null
  int t_len, V;
  int same_shift;              // logits and grad lie alike: 16-byte stores
  int followed;                // by a kernel that waits for this one: it may take its place on an SM early
  float c2, inv_T;             // log2(e) / T, 1 / T
  float inv_T_rest;            // what 1 / T's rounding left
  long long wait_limit_ns;     // of a wait for staged logits
  PolicyArgs policy;
};

// (e^d - d - 1) from e^d - 1, without cancellation where d is small.
__device__ __forceinline__ float kl_term(float d, float up) {
  if (d == INFINITY) return d;             // a token that the policy cannot say
  if (!(fabsf(d) <= 0.125f)) return __fsub_rn(up, d);
  // d^2 (1/2 + d/6 + ... + d^4/720): the next term is below 1.3e-8 of it
  float s = __fmaf_rn(d, 1.f / 720.f, 1.f / 120.f);
  s = __fmaf_rn(d, s, 1.f / 24.f);
  s = __fmaf_rn(d, s, 1.f / 6.f);
  s = __fmaf_rn(d, s, 0.5f);
  return d * d * s;
}

// What a row's loss needs besides its logits.
struct PolicyRow {
  float A, old_logp, ref_logp, weight;
  __device__ __forceinline__ static PolicyRow of(const PolicyArgs& P, int r, int t_len) {
    const int b = static_cast<unsigned>(r) / static_cast<unsigned>(t_len);
    return PolicyRow{P.advantages[P.per_token ? r : b], P.old_logp ? P.old_logp[r] : 0.f,
                     P.ref_logp ? P.ref_logp[r] : 0.f, P.weights[b]};
  }
};

// A row's loss and its derivative in the token's log-probability.
template <bool ENT>
__device__ __forceinline__ void policy_row(const PolicyArgs& P, const PolicyRow& row, const TokRow& R, float& loss,
                                           float& slope) {
  const float A = row.A;
  const float up_old = P.old_logp ? __fadd_rn(__fsub_rn(R.logp, row.old_logp), R.logp_rest) : 0.f;
  const float r = P.old_logp ? expf(up_old) : 1.f;
  const float low = 1.f - P.low, high = 1.f + P.high;
  float gained = r * A;
  if (r == INFINITY && up_old < INFINITY) {   // past the range where the product need not be
    const float half = expf(0.5f * up_old);
    gained = A == 0.f ? A : half * A * half;
  }
  const float held = (r < low ? low : r > high ? high : r) * A;
  float gain = gained <= held ? gained : held;
  slope = gained <= held ? -gained : 0.f;
  if (!(gained == gained)) gain = slope = NAN;
  if (P.dual > 0.f && A < 0.f && gain < P.dual * A) {
    gain = P.dual * A;
    slope = 0.f;
  }
  loss = R.valid ? -gain : NAN;
  if (P.ref_logp) {
    const float d = __fsub_rn(__fsub_rn(row.ref_logp, R.logp), R.logp_rest), up = expm1f(d);
    if (up == INFINITY && d < INFINITY) {     // likewise
      const float half = expf(0.5f * d), pull = P.kl * half * half;
      loss += pull;
      slope -= pull;
    } else {
      loss = __fmaf_rn(P.kl, kl_term(d, up), loss);
      slope = __fmaf_rn(-P.kl, up, slope);
    }
  }
  if (ENT) loss = __fmaf_rn(-P.entropy, R.entropy(), loss);
}

// Zeros in a row's place, by `threads` threads of which this is `tid`.
template <int ELT>
__device__ __forceinline__ void zero_row(unsigned char* grad, int V, int tid, int threads) {
  const int shift = row_shift<ELT>(grad), nvec = row_vecs<ELT>(V, shift);
  for (int v = tid; v < nvec; v += threads) store_edge<ELT>(grad, V, v * Vec<ELT>::N - shift, 1, make_uint4(0, 0, 0, 0));
}

// ---- short rows: in the registers of one, two or four warps
//
// A warp holds 8 KB of a row, 16 vectors a lane, and asks for them all at once;
// sixteen warps an SM keep 128 KB on their way.  A row is read once, its warps meet
// at one barrier, and no CTA waits for another.  Bound by instructions: what a row's
// numbers take beside its logits, by every warp of its own.  50000 rows of 4000 bf16
// logits with the policy loss's gradient: 153 us, 5.2 TB/s; 200000 of 1000: 325 us, 2.5
// TB/s (a CTA to a row, read twice: 385 and 1253 us).
constexpr int kShThreads = 128, kShWarps = kShThreads / 32, kShPerLane = 16, kShChunk = 4;
constexpr int kShPerSm = 4;                                 // CTAs
constexpr int kShMaxVecs = kShWarps * 32 * kShPerLane;      // of a row

template <int ELT, bool ENT, bool GRAD, int G>
__global__ void __launch_bounds__(kShThreads, kShPerSm) token_short_kernel(const __grid_constant__ RowParams P, int rows) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N, kGroups = kShWarps / G;
  __shared__ TokPart parts[2][kShWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / G, sub = warp % G, tid = sub * 32 + lane;
  if (P.followed) grid_dependents_launch();
  const int stride = static_cast<int>(gridDim.x) * kGroups;
  int par = 0, r = static_cast<int>(blockIdx.x) * kGroups + group;
  int x_next = r < rows ? P.tokens[r] : -1;
  for (; r < rows; r += stride) {
    const int x_row = x_next;
    x_next = r + stride < rows ? P.tokens[r + stride] : -1;
    const unsigned long long at_row = static_cast<unsigned long long>(r) * (static_cast<unsigned>(P.V) * ELT);
    const unsigned char* row = P.logits + at_row;
    unsigned char* grad = GRAD ? P.grad + at_row : nullptr;
    if (x_row < 0) {
      if (tid == 0) {
        P.logp[r] = 0.f;
        if (P.entropy) P.entropy[r] = 0.f;
        if (P.lse) P.lse[r] = -INFINITY;
        if (P.kept) P.kept[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (P.row_loss) P.row_loss[r] = 0.f;
      }
      if (GRAD) zero_row<ELT>(grad, P.V, tid, G * 32);
      continue;
    }
    const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
    const uint32_t zx_bits = load_bits<ELT>(row, min(x_row, P.V - 1));
    uint4 w[kShPerLane];
#pragma unroll
    for (int c = 0; c < kShPerLane; c += kShChunk) {
      const int v0 = c * G * 32, v1 = (c + kShChunk) * G * 32;       // the chunk's vectors, of all the row's warps
      if (v0 * N - shift >= 0 && v1 * N - shift <= P.V) {
        const unsigned char* at = row + (static_cast<long long>(v0 + tid) * N - shift) * ELT;
#pragma unroll
        for (int k = 0; k < kShChunk; ++k) w[c + k] = load_vec16(at + k * G * 512);
      } else if (v0 < nvec) {
#pragma unroll
        for (int k = 0; k < kShChunk; ++k)
          w[c + k] = v0 + k * G * 32 + tid < nvec ? load_row_vec<ELT>(row, P.V, shift, v0 + k * G * 32 + tid) : VT::neg_inf();
      }
    }
    PolicyRow mine{};
    if (P.row_loss) mine = PolicyRow::of(P.policy, r, P.t_len);
    const int x = x_row < P.V ? x_row : -(1 << 30), x_vec = (x + shift) / N;
    const float zx = x_row < P.V ? value_of<ELT>(zx_bits) : NAN;
    TokSum<ELT, ENT> sum(zx);
#pragma unroll
    for (int c = 0; c < kShPerLane; c += kShChunk) {
      if (c * G * 32 < nvec) {
        uint4 some[kShChunk];
#pragma unroll
        for (int k = 0; k < kShChunk; ++k) {
          some[k] = w[c + k];
          if ((c + k) * G * 32 + tid == x_vec) tok_take_out<ELT>(some[k], x + shift - x_vec * N);
        }
        sum.add(some, P.c2);
      }
    }
    TokPart part = sum.part();
    if (zx != zx) part.s = NAN;
    part = tok_join<ENT>(part, P.c2);
    if (G > 1) {
      if (lane == 0) parts[par][warp] = part;
      named_barrier_sync(1 + group, G * 32);
      part = tok_join<ENT>(lane < G ? parts[par][group * G + lane] : tok_none(), P.c2);
      par ^= 1;   // only here: the next row's barrier lies between these reads and the writes to the same place
    }
    const TokRow R = tok_row<ENT>(part, zx, TokTemp{P.inv_T, P.inv_T_rest});
    float loss = 0.f, slope = 0.f;
    if (P.row_loss) policy_row<ENT>(P.policy, mine, R, loss, slope);
    if (tid == 0) {
      P.logp[r] = R.logp;
      if (ENT && P.entropy) P.entropy[r] = R.entropy();
      if (P.lse) P.lse[r] = R.lse(P.inv_T);
      if (P.kept) P.kept[r] = tok_kept(R);
      if (P.row_loss) P.row_loss[r] = loss;
    }
    if (GRAD) {
      const TokGrad D = tok_grad<ENT>(R, mine.weight * slope, ENT ? -P.policy.entropy * mine.weight : 0.f, P.inv_T);
#pragma unroll
      for (int c = 0; c < kShPerLane; c += kShChunk) {
        const int v0 = c * G * 32, v1 = (c + kShChunk) * G * 32;
        if (P.same_shift && v0 * N - shift >= 0 && v1 * N - shift <= P.V) {
          unsigned char* at = grad + (static_cast<long long>(v0 + tid) * N - shift) * ELT;
#pragma unroll
          for (int k = 0; k < kShChunk; ++k) store_vec16(at + k * G * 512, tok_vec_grad<ELT, ENT>(w[c + k], D, P.c2));
        } else if (v0 < nvec) {
#pragma unroll
          for (int k = 0; k < kShChunk; ++k)
            if (v0 + k * G * 32 + tid < nvec)
              store_edge<ELT>(grad, P.V, (v0 + k * G * 32 + tid) * N - shift, P.same_shift, tok_vec_grad<ELT, ENT>(w[c + k], D, P.c2));
        }
      }
      // the token's own after its vector's, by the same thread
      if (x_vec >= 0 && x >= 0 && x_vec % (G * 32) == tid) VT::store_rounded(grad, x, D.at_token);
    }
  }
}

// ---- long rows: streamed through shared memory, where they stay for the gradient
//
// A row goes to a cluster of 1 to 8 CTAs, a part to each.  A producer warp streams
// the part through a ring of 16 KB slots, worker warps sum it as it lands, and a
// warp of its own puts the row's numbers together from their sums (and through
// distributed shared memory from the other CTAs'), so that the workers need not:
// with every warp working them out a row cost each 1780 instructions besides its
// logits.  For the gradient the slots keep the row: the workers read them a second
// time once the numbers are there, and give them back to the producer one by one.
// Meanwhile they sum the next row, where two parts fit the ring.  So every logit
// crosses HBM once and every gradient value once, and neither the loads nor the
// workers stop at a row's end.  That takes an SM's shared memory.  Without a
// gradient a slot is given back as soon as it is read, and two CTAs share an SM.
//
// Rows with a token are dealt to the clusters in turn, whatever lies between them
// (a batch of padded rollouts dealt by row number keeps some clusters a third
// longer at work): every CTA counts the tokens of a window of rows and lists its
// own.  Rows without one are zero-filled by single CTAs in between.
//
// 4096 rows of 151936 bf16 logits: log-probabilities 186 us, 6.7 TB/s; with the policy
// loss's gradient 418 us, 6.0 TB/s of each logit read and each gradient written once.
// Bound there by instructions (17 a logit over both passes, half of them beside the
// arithmetic) and by eight SMs that clusters of four leave idle.
//
// Every wait has a limit.  A worker thread whose wait for a slot expires touches the
// ring no more: its sums and gradients are NaN from there on, and so are all later
// rows of its cluster.  A CTA whose cluster does not answer takes the row and all
// later ones as NaN.  The producer, which then waits in vain for slots, leaves
// last, when its copies have landed.
template <bool GRAD>
struct Rg {
  static constexpr int kWorkers = GRAD ? 16 : 8;
  static constexpr int kPerLane = 32 / kWorkers;             // vectors per lane and slot
  static constexpr int kWork = kWorkers * 32, kThreads = kWork + 64;   // + the producer's and the row's warp
  static constexpr int kSlotVecs = kWork * kPerLane, kSlotBytes = kSlotVecs * 16;
  static constexpr int kSlots = GRAD ? 14 : 6;
  static constexpr int kPerSm = GRAD ? 1 : 2;                // CTAs
};
constexpr int kRgSlotVecs = 1024, kRgSlotBytes = kRgSlotVecs * 16;
constexpr int kRgMaxWorkers = 16, kRgMaxSlots = 14;
constexpr int kRgMaxCtas = 8;
constexpr int kRgWindow = 8192;                             // rows whose tokens are looked at together
constexpr int kRgLive = 448, kRgDead = 64;                  // of which a cluster, a CTA gets so many at most
constexpr int kRgSms = 152;
constexpr int kRgMinPart = 16 * 1024;                       // and where a row is split for want of rows
constexpr long long kRgJoinLimitNs = 4 * kDrainLimitNs;     // a CTA's part comes within an expired wait
constexpr long long kRgRowLimitNs = 2 * kRgJoinLimitNs;     // and a row's numbers within that one
constexpr int kRgNoRow = 0x7fffffff;
static_assert(Rg<true>::kSlotBytes == kRgSlotBytes && Rg<false>::kSlotBytes == kRgSlotBytes, "slots");
static_assert((kTokMaxRow / kRgSlotBytes + 5) / 6 < Rg<true>::kSlots, "the longest row fits a cluster of 6");

struct RgShared {
  uint64_t full[kRgMaxSlots], empty[kRgMaxSlots];
  uint64_t summed[2];            // the workers' sums of a row are here, by row parity as what follows
  uint64_t joined[2];            // the CTAs' are
  uint64_t ready[2];             // what the gradient takes is (without one: the sums have been read)
  uint4 part[2][kRgMaxCtas];     // the CTAs' sums
  TokPart warp[2][kRgMaxWorkers];
  TokGrad grad[2];
  int counts[kRgMaxWorkers];     // rows with and without a token in a warp's strip of the window
  int failed;                    // the first row in which the cluster did not answer, or kRgNoRow
  unsigned short live[kRgLive], dead[kRgDead];
};
constexpr int kRgRingAt = (static_cast<int>(sizeof(RgShared)) + 127) / 128 * 128;
template <bool GRAD>
constexpr int rg_smem() { return kRgRingAt + Rg<GRAD>::kSlots * kRgSlotBytes; }
static_assert(rg_smem<true>() <= 227 * 1024 && 2 * (rg_smem<false>() + 1024) <= 228 * 1024, "an SM's shared memory");

// A CTA's part of a row's whole vectors: which of the row's vectors is its first,
// and their number (the row's ends are taken apart).
struct RgPart {
  int first, n, shift, nvec;
  template <int ELT>
  __device__ __forceinline__ static RgPart of(const unsigned char* row, int V, int per, int rank) {
    constexpr int N = Vec<ELT>::N;
    RgPart t;
    t.shift = row_shift<ELT>(row);
    t.nvec = row_vecs<ELT>(V, t.shift);
    const int head = t.shift ? 1 : 0;
    const int all = t.nvec - head - ((V + t.shift) % N && t.nvec > head ? 1 : 0);
    const int from = min(all, rank * per);
    t.first = head + from;
    t.n = min(all, rank * per + per) - from;
    return t;
  }
  // of the first vector, in bytes from the row's start on
  __device__ __forceinline__ int offset(int elt) const { return first * 16 - shift * elt; }
  // the token that this thread takes of the row's ends, of whole vectors no part, or -1
  template <int ELT>
  __device__ __forceinline__ int end(int V, int rank, int tid) const {
    constexpr int N = Vec<ELT>::N;
    const int e = tid & 31;
    if (rank || tid >= 64 || e >= N) return -1;
    if (tid < 32) return shift && e < N - shift ? e : -1;
    const int over = (V + shift) % N;    // of the last vector's places
    return e < over ? V - over + e : -1;
  }
};

// A vector of one value, the others -inf.
template <int ELT>
__device__ __forceinline__ uint4 rg_one(uint32_t bits) {
  uint4 w = Vec<ELT>::neg_inf();
  w.x = ELT == 4 ? bits : (w.x & 0xffff0000u) | bits;
  return w;
}

// A wait of at most `limit_ns`, the warp parked meanwhile.
__device__ __noinline__ bool rg_wait_longer(uint64_t* bar, uint32_t parity, long long limit_ns) {
  const unsigned long long t0 = global_ns();
  while (!mbar_park(bar, parity, 20000))
    if (static_cast<long long>(global_ns() - t0) >= limit_ns) return false;
  return true;
}
__device__ __forceinline__ bool rg_wait(uint64_t* bar, uint32_t parity, long long limit_ns) {
  return mbar_try_wait(bar, parity) || rg_wait_longer(bar, parity, limit_ns);
}

// How many of the numbers from `from`, which is below `of`, to `to` are `own` modulo `of`.
__device__ __forceinline__ int rg_own(unsigned from, unsigned to, unsigned own, unsigned of) {
  return static_cast<int>((to > own ? (to - own + of - 1) / of : 0u) - (from > own ? 1u : 0u));
}

// `window`: rows whose tokens are looked at together; `per`: vectors of a CTA's
// part at most; `ahead`: two parts fit the ring.
template <int ELT, bool ENT, bool GRAD>
__global__ void __launch_bounds__(Rg<GRAD>::kThreads, Rg<GRAD>::kPerSm)
    token_ring_kernel(const __grid_constant__ RowParams P, int rows, int window, int per, int ahead) {
  using VT = Vec<ELT>;
  using R_ = Rg<GRAD>;
  constexpr int N = VT::N, kSlots = R_::kSlots, kWorkers = R_::kWorkers, kWork = R_::kWork, U = R_::kPerLane;
  extern __shared__ __align__(1024) unsigned char smem[];
  RgShared& sh = *reinterpret_cast<RgShared*>(smem);
  unsigned char* ring = smem + kRgRingAt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster_ctas(), rank = cluster_rank();
  const int cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kWorkers);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.summed[b], kWorkers);
      mbar_init(&sh.joined[b], 1);
      mbar_init(&sh.ready[b], 1);
    }
    sh.failed = kRgNoRow;
    fence_mbar_init();
  }
  if (ctas > 1) cluster_sync();   // the others' barriers are set up too
  else __syncthreads();
  if (P.followed) grid_dependents_launch();

  // rows of whole vectors lie alike, so one part stands for all
  const unsigned row_bytes = static_cast<unsigned>(P.V) * ELT;
  const bool alike = row_bytes % 16 == 0;
  RgPart t = RgPart::of<ELT>(P.logits, P.V, per, rank);
  auto row_at = [&](long long w, int i) {      // byte offset of row i of this cluster's
    return static_cast<unsigned long long>(static_cast<unsigned>(w) + sh.live[i]) * row_bytes;
  };

  // every role's place in the ring, and the parity of that slot's copies
  int slot = 0;
  uint32_t round = 0;
  auto step = [&](int& s, uint32_t& odd) {
    if (++s == kSlots) s = 0, odd ^= 1;
  };
  unsigned copies = 0;            // (producer)
  unsigned turn = 0;              // rows with a token
  // a wait of this thread has expired (at a limit of 0, looked at here once, every
  // one has); the producer has given up
  bool dead = P.wait_limit_ns <= 0 && warp < kWorkers;
  bool alone = false;             // (the row's warp) the cluster did not answer
  unsigned alone_turn = 0;
  unsigned turn_live = 0, turn_dead = 0;   // whose the next rows are
  for (long long w0 = 0; w0 < rows; w0 += window) {
    // ---- which rows of the window are this cluster's, and this CTA's to fill
    const int in_window = static_cast<int>(rows - w0 < window ? rows - w0 : window);
    const int words = (in_window + kWork - 1) / kWork;      // 32 rows each, a lane for each
    uint32_t live_bits = 0, dead_bits = 0;
    if (warp < kWorkers)
      for (int j = 0; j < words; ++j) {
        const int at = (warp * words + j) * 32 + lane;
        const bool in = at < in_window, has = in && P.tokens[w0 + at] >= 0;
        const uint32_t l = __ballot_sync(0xffffffffu, has), d = __ballot_sync(0xffffffffu, in && !has);
        if (lane == j) live_bits = l, dead_bits = d;
      }
    const int mine = __popc(live_bits) | __popc(dead_bits) << 16;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    __syncthreads();              // the last window's lists have been read
    if (lane == 31 && warp < kWorkers) sh.counts[warp] = upto;
    __syncthreads();
    const int count = lane < kWorkers ? sh.counts[lane] : 0;
    const int total = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(count)));
    const int before = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(lane < warp ? count : 0))) + upto - mine;
    // row k of those with a token (from `turn_live` on, modulo the clusters) is
    // cluster k % clusters's, and likewise for the CTAs and the others
    for (int j = 0; j < words; ++j) {
      const uint32_t l = __shfl_sync(0xffffffffu, live_bits, j), d = __shfl_sync(0xffffffffu, dead_bits, j);
      const int from = __shfl_sync(0xffffffffu, before, j), at = (warp * words + j) * 32 + lane;
      const uint32_t lower = (1u << lane) - 1u;
      const bool has = l >> lane & 1u;
      if (has || (d >> lane & 1u)) {
        const unsigned k = (has ? turn_live + (from & 0xffff) : turn_dead + (from >> 16)) + __popc((has ? l : d) & lower);
        const unsigned of = has ? clusters : gridDim.x, own = has ? cluster : blockIdx.x;
        if (k % of == own) {
          const unsigned place = k / of - (own < (has ? turn_live : turn_dead) ? 1u : 0u);
          (has ? sh.live : sh.dead)[place] = static_cast<unsigned short>(at);
          if (!has) {
            const long long r = w0 + at;
            P.logp[r] = 0.f;
            if (P.entropy) P.entropy[r] = 0.f;
            if (P.lse) P.lse[r] = -INFINITY;
            if (P.kept) P.kept[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (P.row_loss) P.row_loss[r] = 0.f;
          }
        }
      }
    }
    const int n_live = rg_own(turn_live, turn_live + (total & 0xffff), cluster, clusters);
    const int n_dead = rg_own(turn_dead, turn_dead + (total >> 16), blockIdx.x, gridDim.x);
    turn_live = (turn_live + (total & 0xffff)) % clusters;
    turn_dead = (turn_dead + (total >> 16)) % gridDim.x;
    __syncthreads();

    if (warp == kWorkers) {
      // ---- the producer
      for (int i = 0; i < n_live && !dead; ++i) {
        const unsigned char* row = P.logits + row_at(w0, i);
        if (!alike) t = RgPart::of<ELT>(row, P.V, per, rank);
        const unsigned char* from = row + t.offset(ELT);
        for (int v = 0; v < t.n && !dead; v += kRgSlotVecs) {
          int ok = 1;
          if (lane == 0) ok = rg_wait(&sh.empty[slot], round ^ 1, kDrainLimitNs) ? 1 : 0;
          dead = !__shfl_sync(0xffffffffu, ok, 0);
          if (dead) break;        // as a worker has
          if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(min(kRgSlotVecs, t.n - v)) * 16u;
            mbar_expect_tx(&sh.full[slot], bytes);
            bulk_load(ring + slot * kRgSlotBytes, from + v * 16, bytes, &sh.full[slot]);
          }
          ++copies;
          step(slot, round);
        }
      }
      continue;
    }

    if (warp == kWorkers + 1) {
      // ---- the row's warp: the next row's token and logit are loaded while it waits
      int x = n_live ? P.tokens[w0 + sh.live[0]] : 0;
      float zx = n_live && x < P.V ? load_elem<ELT>(P.logits + (w0 + sh.live[0]) * P.V * ELT, x) : NAN;
      for (int i = 0; i < n_live; ++i, ++turn) {
        const long long r = w0 + sh.live[i], r_next = i + 1 < n_live ? w0 + sh.live[i + 1] : r;
        const int par = turn & 1;
        const uint32_t phase = turn >> 1 & 1;
        PolicyRow mine_row{};
        if (P.row_loss) mine_row = PolicyRow::of(P.policy, static_cast<int>(r), P.t_len);
        const int x_next = P.tokens[r_next];
        bool here = __all_sync(0xffffffffu, rg_wait(&sh.summed[par], phase, kRgRowLimitNs));
        const float zx_next = x_next < P.V ? load_elem<ELT>(P.logits + r_next * P.V * ELT, x_next) : NAN;
        TokPart part = tok_join<ENT>(lane < kWorkers ? sh.warp[par][lane] : tok_none(), P.c2);
        if (!GRAD && lane == 0) mbar_arrive(&sh.ready[par]);   // the row after the next may take the sums' place
        // (the token's logit is part of what the others wait for: in place they may write over it afterwards)
        if (!here || zx != zx) part.s = NAN;
        if (ctas > 1) {
          TokPart other = tok_none();
          if (!alone) {
            if (lane == 0) mbar_expect_tx(&sh.joined[par], static_cast<uint32_t>(ctas) * 16u);
            if (lane < ctas)
              st_async(peer(&sh.part[par][rank], lane),
                       make_uint4(__float_as_uint(part.m), __float_as_uint(part.s), __float_as_uint(part.a), 0u),
                       peer(&sh.joined[par], lane));
            alone = !__all_sync(0xffffffffu, rg_wait(&sh.joined[par], phase, kRgJoinLimitNs));
            if (alone) {
              // another CTA may still get here and on to the next row, where it
              // waits in vain: what it sends until then is waited for at the end
              if (lane == 0) mbar_expect_tx(&sh.joined[par ^ 1], static_cast<uint32_t>(ctas) * 16u);
              alone_turn = turn;
            } else if (lane < ctas) {
              const uint4 y = sh.part[par][lane];
              other = TokPart{__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z)};
            }
          }
          part = tok_join<ENT>(other, P.c2);
          here = !alone;
        }
        if (!here) {
          part.s = NAN;
          if (lane == 0) atomicMin(&sh.failed, static_cast<int>(r));
        }
        const TokRow row = tok_row<ENT>(part, zx, TokTemp{P.inv_T, P.inv_T_rest});
        float loss = 0.f, slope = 0.f;
        if (P.row_loss) policy_row<ENT>(P.policy, mine_row, row, loss, slope);
        if (GRAD) {
          const TokGrad G = tok_grad<ENT>(row, mine_row.weight * slope, ENT ? -P.policy.entropy * mine_row.weight : 0.f, P.inv_T);
          if (lane == 0) {
            sh.grad[par] = G;
            mbar_arrive(&sh.ready[par]);
          }
        }
        if (lane == 0 && rank == 0) {
          P.logp[r] = row.logp;
          if (ENT && P.entropy) P.entropy[r] = row.entropy();
          if (P.lse) P.lse[r] = row.lse(P.inv_T);
          if (P.kept) P.kept[r] = tok_kept(row);
          if (P.row_loss) P.row_loss[r] = loss;
        }
        x = x_next;
        zx = zx_next;
      }
      continue;
    }

    // ---- the workers: row i summed, and the gradient of the row before (of row i
    // itself where two do not fit)
    int kept_slot = slot;         // where the row begins whose gradient is next
    int filled = 0;
    uint32_t end_next = 0u, end_kept = 0u;   // this thread's logit at the ends of the row summed last and of the one before
    int x_next = n_live ? P.tokens[w0 + sh.live[0]] : 0, x_before = 0;
    uint32_t zx_next = n_live ? load_bits<ELT>(P.logits + row_at(w0, 0), min(x_next, P.V - 1)) : 0u;
    const unsigned first_turn = turn;
    for (int i = 0; i < n_live + (GRAD ? ahead : 0); ++i) {
      int x_now = x_next;
      if (i < n_live) {
        const unsigned char* row = P.logits + row_at(w0, i);
        if (!alike) t = RgPart::of<ELT>(row, P.V, per, rank);
        const int x = x_now < P.V ? x_now : -(1 << 30);
        if (i + 1 < n_live) x_next = P.tokens[w0 + sh.live[i + 1]];
        // where x lies from the part's first vector on; the slot in which this thread reads it
        const int x_vec = (x + t.shift) / N - t.first;
        const int x_at = x_vec >= 0 && x_vec < t.n && x_vec % kWork == tid ? x_vec / kRgSlotVecs : -1;
        const int end = t.end<ELT>(P.V, rank, tid);
        const uint32_t end_now = end >= 0 ? load_bits<ELT>(row, end) : 0u;
        TokSum<ELT, ENT> sum(value_of<ELT>(zx_next));
        // (after an expired wait the vectors are whatever lies there, which is made
        // NaN once a row)
        const int slots = (t.n + kRgSlotVecs - 1) / kRgSlotVecs;
        auto take = [&](uint4* w, int v) {
          const int n = t.n - v * kRgSlotVecs;
          unsigned char* at = ring + slot * kRgSlotBytes;
          if (!dead) dead = !rg_wait(&sh.full[slot], round, P.wait_limit_ns);
          if (v == x_at) {        // out of the sum: this thread reads what it writes here
            VT::store_scalar(at, (x_vec - v * kRgSlotVecs) * N + (x + t.shift) % N, -INFINITY);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the slot is filled again
          }
          const uint4* src = reinterpret_cast<const uint4*>(at) + tid;
          if (n >= kRgSlotVecs) {
#pragma unroll
            for (int k = 0; k < U; ++k) w[k] = src[k * kWork];
          } else {
#pragma unroll
            for (int k = 0; k < U; ++k) w[k] = tid + k * kWork < n ? src[k * kWork] : VT::neg_inf();
          }
          if (!GRAD) {
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(&sh.empty[slot]);
          }
          step(slot, round);
        };
        // two slots at a time, which halves what a sum costs beside its logits (1024 rows
        // of 151936 bf16 with the gradient: 115 us, one at a time 125)
        int v = 0;
        for (; v + 1 < slots; v += 2) {
          uint4 w[2 * U];
          take(w, v);
          take(w + U, v + 1);
          sum.add(w, P.c2);
        }
        if (v < slots) {
          uint4 w[U];
          take(w, v);
          sum.add(w, P.c2);
        }
        if (end >= 0 && end != x) {
          const uint4 one[1] = {rg_one<ELT>(end_now)};
          sum.add(one, P.c2);
        }
        end_kept = end_next;
        end_next = end_now;
        TokPart part = sum.part();
        if (dead) part.s = NAN;
        part = tok_join<ENT>(part, P.c2);
        const unsigned at_turn = first_turn + static_cast<unsigned>(i);
        const int par = at_turn & 1;
        // (for the gradient the workers have waited for that row's numbers)
        if (!GRAD && at_turn >= 2 && !rg_wait(&sh.ready[par], (at_turn >> 1 & 1) ^ 1, kRgRowLimitNs)) dead = true;
        if (lane == 0) {
          sh.warp[par][warp] = part;
          mbar_arrive(&sh.summed[par]);
        }
        if (i + 1 < n_live) zx_next = load_bits<ELT>(P.logits + row_at(w0, i + 1), min(x_next, P.V - 1));
      }
      if (GRAD && i >= ahead) {
        const long long r = w0 + sh.live[i - ahead];
        const unsigned at_turn = first_turn + static_cast<unsigned>(i - ahead);
        const unsigned long long at_row = row_at(w0, i - ahead);
        if (!alike) t = RgPart::of<ELT>(P.logits + at_row, P.V, per, rank);
        unsigned char* grad = P.grad + at_row;
        const int x_row = ahead ? x_before : x_now;
        const int x = x_row < P.V ? x_row : -(1 << 30), x_vec = (x + t.shift) / N - t.first;
        const int end = t.end<ELT>(P.V, rank, tid);
        const uint32_t end_bits = ahead && i < n_live ? end_kept : end_next;   // (nothing was summed after the last row)
        const bool here = rg_wait(&sh.ready[at_turn & 1], at_turn >> 1 & 1, kRgRowLimitNs);
        TokGrad G = sh.grad[at_turn & 1];
        if (!here) {
          atomicMin(&sh.failed, static_cast<int>(r));
          dead = true;
        }
        if (dead) G.alpha = G.at_token = NAN;
        unsigned char* out = grad + t.offset(ELT) + tid * 16;
        auto give = [&](int v, auto full) {
          const int n = t.n - v * kRgSlotVecs;
          const uint4* src = reinterpret_cast<const uint4*>(ring + kept_slot * kRgSlotBytes) + tid;
          uint4 w[U];
#pragma unroll
          for (int k = 0; k < U; ++k) w[k] = decltype(full)::value || tid + k * kWork < n ? src[k * kWork] : VT::neg_inf();
          __syncwarp();
          if (lane == 0 && !dead) mbar_arrive(&sh.empty[kept_slot]);
          if (++kept_slot == kSlots) kept_slot = 0;
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const uint4 d = tok_vec_grad<ELT, ENT>(w[k], G, P.c2);
            if (decltype(full)::value) store_vec16(out + k * kWork * 16, d);
            else if (tid + k * kWork < n)
              store_edge<ELT>(grad, P.V, (t.first + v * kRgSlotVecs + tid + k * kWork) * N - t.shift, P.same_shift, d);
          }
          out += kRgSlotBytes;
        };
        const int whole = P.same_shift ? t.n / kRgSlotVecs : 0;
        for (int v = 0; v < whole; ++v) give(v, std::true_type());
        for (int v = whole; v * kRgSlotVecs < t.n; ++v) give(v, std::false_type());
        if (end >= 0) {
          float d[N];
          VT::unpack(tok_vec_grad<ELT, ENT>(rg_one<ELT>(end_bits), G, P.c2), d);
          VT::store_rounded(grad, end, end == x ? G.at_token : d[0]);
        }
        // the token's own after its vector's, by the same thread
        if (x_vec >= 0 && x_vec < t.n && x_vec % kWork == tid) VT::store_rounded(grad, x, G.at_token);
        // rows without a token, as many as there are for each row with one
        for (; static_cast<long long>(filled) * n_live < static_cast<long long>(i + 1 - ahead) * n_dead; ++filled) {
          zero_row<ELT>(P.grad + static_cast<unsigned long long>(w0 + sh.dead[filled]) * row_bytes, P.V, tid, kWork);
        }
      }
      x_before = x_now;
    }
    turn += static_cast<unsigned>(n_live);
    if (GRAD)
      for (; filled < n_dead; ++filled) {
        zero_row<ELT>(P.grad + static_cast<unsigned long long>(w0 + sh.dead[filled]) * row_bytes, P.V, tid, kWork);
      }
  }
  // ---- no copy is left in flight, and nothing on its way to a CTA that has left
  if (warp == kWorkers && lane == 0)
    for (unsigned k = copies > kSlots ? copies - kSlots : 0; k < copies; ++k)
      rg_wait(&sh.full[k % kSlots], k / kSlots & 1, kDrainLimitNs);
  if (ctas > 1) {
    cluster_sync();
    if (alone)
      for (unsigned k = alone_turn; k < alone_turn + 2; ++k) rg_wait(&sh.joined[k & 1], k >> 1 & 1, kDrainLimitNs);
  } else {
    __syncthreads();
  }
  // a row that the others may have put together before
  if (tid == 0 && sh.failed != kRgNoRow) {
    P.logp[sh.failed] = NAN;
    if (P.entropy) P.entropy[sh.failed] = NAN;
    if (P.lse) P.lse[sh.failed] = NAN;
    if (P.row_loss) P.row_loss[sh.failed] = NAN;
  }
}

// ---- the gradient from what token_logp gave: a stream of 32 KB pieces
//
// A row's pieces go to as many CTAs, up to eight, each with all its loads in flight
// at once; four CTAs an SM hide each other's chain of two trips to memory (the
// row's numbers, then its token's logit).  In place the token's logit may be
// overwritten by another piece's CTA, so there the row's CTAs are a cluster, which
// goes on when all of them have it (what the preference loss keeps of a row has no
// need of that logit).  4096 rows of 151936 bf16: 384 us, 6.5 TB/s;
// 50000 of 4000 259 us, 3.1 TB/s.
struct GradParams {
  const unsigned char* logits;
  const int* tokens;
  const float *logp, *lse, *entropy, *d_logp, *d_entropy;   // [rows]; the entropies or null
  const float4* kept;          // [rows]: in place of logp and lse, or null
  unsigned char* grad;
  int V, same_shift;
  int d_rows;                  // rows that share a d_logp
  int in_place;                // and the token's logit is read
  float c2, inv_T, T;
};
constexpr int kGrThreads = 256, kGrPerThread = 8, kGrVecs = kGrThreads * kGrPerThread;
constexpr int kGrMaxParts = 8;

template <int ELT, bool ENT>
__global__ void __launch_bounds__(kGrThreads, 4) token_grad_kernel(const __grid_constant__ GradParams P, int parts, int per) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  const int tid = threadIdx.x;
  // the last rows first: token_logp, just before, has left them in L2
  const int r = static_cast<int>(gridDim.x / parts - 1 - blockIdx.x / parts), part = static_cast<int>(blockIdx.x) % parts;
  const unsigned long long at_row = static_cast<unsigned long long>(r) * (static_cast<unsigned>(P.V) * ELT);
  const unsigned char* row = P.logits + at_row;
  unsigned char* grad = P.grad + at_row;
  const int shift = row_shift<ELT>(row), nvec = row_vecs<ELT>(P.V, shift);
  const int x = P.tokens[r];
  grid_dependency_wait();      // (the rows' numbers may be a kernel's before this one; the logits and tokens are not)
  TokGrad G;
  G.none();
  if (x >= 0 && P.kept) {
    G = tok_grad_kept(P.kept[r], P.d_logp[static_cast<unsigned>(r) / static_cast<unsigned>(P.d_rows)], P.inv_T);
  } else if (x >= 0) {
    const uint32_t zx = load_bits<ELT>(row, min(x, P.V - 1));
    G = tok_grad_from(value_of<ELT>(zx), x < P.V ? P.logp[r] : NAN, P.lse[r], ENT ? P.entropy[r] : 0.f,
                      P.d_logp[r], ENT ? P.d_entropy[r] : 0.f, P.T, P.inv_T, P.c2);
  }
  if (P.in_place) {
    if (parts > 1) cluster_sync();
    else __syncthreads();
  }
  const int to = min(nvec, (part + 1) * per);
  const bool zero = G.zero();
  for (int v0 = part * per; v0 < to; v0 += kGrVecs) {
    const int v = v0 + tid, n = to - v0;
    // pieces of whole vectors go without a look at each
    const bool whole = n >= kGrVecs && P.same_shift && v0 * N - shift >= 0 && (v0 + kGrVecs) * N - shift <= P.V;
    if (whole) {
      const long long at = (static_cast<long long>(v) * N - shift) * ELT;
      if (zero) {
#pragma unroll
        for (int k = 0; k < kGrPerThread; ++k) store_vec16(grad + at + k * kGrThreads * 16, make_uint4(0, 0, 0, 0));
      } else {
        uint4 w[kGrPerThread];
#pragma unroll
        for (int k = 0; k < kGrPerThread; ++k) w[k] = load_vec16(row + at + k * kGrThreads * 16);
#pragma unroll
        for (int k = 0; k < kGrPerThread; ++k) store_vec16(grad + at + k * kGrThreads * 16, tok_vec_grad<ELT, ENT>(w[k], G, P.c2));
      }
    } else {
      uint4 w[kGrPerThread];
#pragma unroll
      for (int k = 0; k < kGrPerThread; ++k)
        w[k] = !zero && tid + k * kGrThreads < n ? load_row_vec<ELT>(row, P.V, shift, v + k * kGrThreads) : VT::neg_inf();
#pragma unroll
      for (int k = 0; k < kGrPerThread; ++k)
        if (tid + k * kGrThreads < n)
          store_edge<ELT>(grad, P.V, (v + k * kGrThreads) * N - shift, P.same_shift,
                          zero ? make_uint4(0, 0, 0, 0) : tok_vec_grad<ELT, ENT>(w[k], G, P.c2));
    }
    // the token's own after its vector's, by the same thread
    const int x_vec = x >= 0 && x < P.V ? (x + shift) / N - v0 : -1;
    if (!zero && x_vec >= 0 && x_vec < min(n, kGrVecs) && x_vec % kGrThreads == tid) VT::store_rounded(grad, x, G.at_token);
  }
}

template <int ELT, bool ENT>
cudaError_t launch_grad(const GradParams& p, int rows, bool dependent, cudaStream_t s) {
  const int nvec = (p.V + 2 * Vec<ELT>::N - 2) / Vec<ELT>::N;      // of a row off the 16-byte boundary
  const int parts = std::min(kGrMaxParts, (nvec + kGrVecs - 1) / kGrVecs), per = (nvec + parts - 1) / parts;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  if (dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (p.in_place && parts > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kGrThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, token_grad_kernel<ELT, ENT>, p, parts, per);
}

// Clusters of `ctas` of the ring kernel that fit at once, asked for once per
// instance, size and device.
template <int ELT, bool ENT, bool GRAD>
cudaError_t ring_clusters(int ctas, int* fit) {
  static std::atomic<int> known[64][kRgMaxCtas + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*fit = known[dev][ctas].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  const void* fn = reinterpret_cast<const void*>(&token_ring_kernel<ELT, ENT, GRAD>);
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, rg_smem<GRAD>());
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(Rg<GRAD>::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(rg_smem<GRAD>());
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(fit, fn, &cfg);
  if (e != cudaSuccess) return e;
  if (*fit < 1) return cudaErrorInvalidConfiguration;
  if (dev < 64) known[dev][ctas].store(*fit, std::memory_order_release);
  return cudaSuccess;
}

template <int ELT, bool ENT, bool GRAD>
cudaError_t launch_ring(const RowParams& p, int rows, cudaStream_t s) {
  const long long row_bytes = static_cast<long long>(p.V) * ELT;
  // For the gradient a CTA's part of a row stays in its ring.  Clusters of 1, 2, 4
  // and 6 leave 0, 0, 8 and 14 of the SMs idle.  In bf16, where the workers are as
  // busy as the memory, the smallest of them that fits two parts, so that one row is
  // summed while the other's gradient is written (1024 rows of 151936: 115 us, of
  // 128256 102 us; with one part 124 and 108); in float32 the smallest that fits one
  // (1024 rows of 50001: 83 us, with two parts 86; 4096 of 100003 552 and 616; 512 of
  // 50001 the other way, 51 and 48).
  const int slots = static_cast<int>((row_bytes + kRgSlotBytes - 1) / kRgSlotBytes), kept = Rg<GRAD>::kSlots - 1;
  auto fits = [&](int ctas, int most) { return (slots + ctas - 1) / ctas <= most; };
  int ctas = 1;
  if (GRAD) {
    const int most = ELT == 2 ? Rg<GRAD>::kSlots / 2 : kept;
    ctas = fits(1, most) ? 1 : fits(2, most) ? 2 : fits(4, kept) ? 4 : 6;
  }
  // few rows: as many CTAs to a row as give the SMs work
  const int room = kRgSms * Rg<GRAD>::kPerSm;
  while (ctas < kRgMaxCtas && static_cast<long long>(rows) * 2 * ctas <= room && row_bytes / (2 * ctas) >= kRgMinPart) ctas *= 2;
  if (ctas > kRgMaxCtas) ctas = kRgMaxCtas;
  int fit = 0;
  cudaError_t e = ring_clusters<ELT, ENT, GRAD>(ctas, &fit);
  if (e != cudaSuccess) return e;
  const int clusters = rows < fit ? rows : fit;
  const long long window = std::min<long long>(kRgWindow, std::min<long long>(static_cast<long long>(kRgLive) * clusters,
                                                                              static_cast<long long>(kRgDead) * clusters * ctas));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ctas));
  cfg.blockDim = dim3(Rg<GRAD>::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(rg_smem<GRAD>());
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int per = (p.V / Vec<ELT>::N + ctas - 1) / ctas;
  const int ahead = 2 * ((per + kRgSlotVecs - 1) / kRgSlotVecs) <= Rg<GRAD>::kSlots;
  return cudaLaunchKernelEx(&cfg, token_ring_kernel<ELT, ENT, GRAD>, p, rows, static_cast<int>(window), per, ahead);
}

template <int ELT, bool ENT, bool GRAD>
cudaError_t launch_rows(const RowParams& p, int rows, cudaStream_t s) {
  const int nvec = (p.V + 2 * Vec<ELT>::N - 2) / Vec<ELT>::N;      // of a row off the 16-byte boundary
  if (nvec > kShMaxVecs) return launch_ring<ELT, ENT, GRAD>(p, rows, s);
  // as few warps to a row as hold it; four where rows are few
  const int grid = kRgSms * kShPerSm;
  const int warps = nvec > 2 * 32 * kShPerLane || rows <= grid ? 4 : nvec > 32 * kShPerLane ? 2 : 1;
  const unsigned ctas = static_cast<unsigned>(std::min<long long>(grid, (static_cast<long long>(rows) * warps + kShWarps - 1) / kShWarps));
  if (warps == 4) token_short_kernel<ELT, ENT, GRAD, 4><<<ctas, kShThreads, 0, s>>>(p, rows);
  else if (warps == 2) token_short_kernel<ELT, ENT, GRAD, 2><<<ctas, kShThreads, 0, s>>>(p, rows);
  else token_short_kernel<ELT, ENT, GRAD, 1><<<ctas, kShThreads, 0, s>>>(p, rows);
  return cudaGetLastError();
}

template <int ELT>
cudaError_t launch_rows(const RowParams& p, int rows, bool ent, cudaStream_t s) {
  if (p.grad) return ent ? launch_rows<ELT, true, true>(p, rows, s) : launch_rows<ELT, false, true>(p, rows, s);
  return ent ? launch_rows<ELT, true, false>(p, rows, s) : launch_rows<ELT, false, false>(p, rows, s);
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
  p.inv_T_rest = static_cast<float>(1.0 / static_cast<double>(temperature) - static_cast<double>(p.inv_T));
  p.wait_limit_ns = kd_wait_limit_ns();
  return p;
}

}  // namespace

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

cudaError_t launch_token_logp(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                              float temperature, float* logp, float* entropy, float* lse, float4* kept, bool followed, cudaStream_t s) {
  RowParams p = row_params(1, V, logits, tokens, temperature, nullptr);
  p.logp = logp;
  p.entropy = entropy;
  p.lse = lse;
  p.kept = kept;
  p.followed = followed;
  return dtype == SV_BF16 ? launch_rows<2>(p, rows, entropy != nullptr, s) : launch_rows<4>(p, rows, entropy != nullptr, s);
}

cudaError_t launch_token_grad(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                              const float* logp, const float* lse, const float* entropy, const float* d_logp,
                              const float* d_entropy, float temperature, void* grad, cudaStream_t s) {
  const RowParams q = row_params(1, V, logits, tokens, temperature, grad);
  const GradParams p{q.logits, tokens, logp, lse, entropy, d_logp, d_entropy, nullptr, q.grad, V, q.same_shift, 1,
                     grad == logits, q.c2, q.inv_T, temperature};
  if (dtype == SV_BF16) return entropy ? launch_grad<2, true>(p, rows, false, s) : launch_grad<2, false>(p, rows, false, s);
  return entropy ? launch_grad<4, true>(p, rows, false, s) : launch_grad<4, false>(p, rows, false, s);
}

cudaError_t launch_kept_grad(int rows, int V, sv_dtype dtype, const void* logits, const int32_t* tokens,
                             const float4* kept, const float* d_logp, int d_rows, float temperature, void* grad,
                             cudaStream_t s) {
  const RowParams q = row_params(1, V, logits, tokens, temperature, grad);
  const GradParams p{q.logits, tokens, nullptr, nullptr, nullptr, d_logp, nullptr, kept, q.grad, V, q.same_shift, d_rows,
                     0, q.c2, q.inv_T, temperature};
  return dtype == SV_BF16 ? launch_grad<2, false>(p, rows, true, s) : launch_grad<4, false>(p, rows, true, s);
}

}  // namespace sv

extern "C" sv_status sv_token_logp(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits,
                                   const int32_t* tokens, float temperature, float* logp, float* entropy, float* lse,
                                   sv_stream_t stream) {
  using namespace sv;
  if (!rows_ok(n_seq, t_len, V, dtype, logits, nullptr, temperature) || !tokens || !logp || !lse)
    return SV_ERR_INVALID_ARG;
  NvtxRange range("sv_token_logp");
  return launch_token_logp(n_seq * t_len, V, dtype, logits, tokens, temperature, logp, entropy, lse, nullptr, false,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status sv_token_logp_grad(int n_seq, int t_len, int V, sv_dtype dtype, const void* logits,
                                        const int32_t* tokens, const float* logp, const float* lse,
                                        const float* entropy, const float* d_logp, const float* d_entropy,
                                        float temperature, void* grad, sv_stream_t stream) {
  using namespace sv;
  if (!rows_ok(n_seq, t_len, V, dtype, logits, grad, temperature) || !tokens || !logp || !lse || !d_logp || !grad)
    return SV_ERR_INVALID_ARG;
  if (!entropy != !d_entropy) return SV_ERR_INVALID_ARG;
  NvtxRange range("sv_token_logp_grad");
  return launch_token_grad(n_seq * t_len, V, dtype, logits, tokens, logp, lse, entropy, d_logp, d_entropy, temperature,
                           grad, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
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
  p.followed = 1;
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
