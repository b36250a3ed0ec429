// Penalties for repeated tokens, biases and grammar masks on logit rows, for
// sm_103a.
//
// Row i of sequence b is scored after the sequence's history and its drafts
// x_0 .. x_{i-1}.  With n(v) the times v was generated (history after the
// prompt, and those drafts) and seen(v) whether it was generated or stands in
// the prompt:
//   z <- z / r if z > 0 else z r          where seen(v)       (repetition)
//   z <- z - f n(v) - p                   where n(v) > 0      (frequency, presence)
//   z <- z + bias(v);  z <- -inf where the row's mask has bit v clear
// in fp32, rounded once to the logits' type.
//
// A CTA takes one slice of the vocabulary of one sequence and, where there are
// CTAs enough, all its rows, else a few of them.  It counts the history's
// tokens of its slice into a shared-memory table (an integer word per token, so
// the order of the additions cannot show) and marks them in a bitmap.  Two
// passes over the slice's rows follow:
//   - the mask and the copy, 16 bytes at a time and without a look at the
//     table (a vector that is masked altogether is written without being
//     read; in place, only what the mask forbids is touched); its first loads
//     are under way while the history is counted;
//   - the tokens of the bitmap, a thread for each token of each row.
// On 256 sequences of up to four rows of 128256 bf16 logits with histories of
// up to 4096 tokens: 70 us (4.7 TB/s of what has to be read and written), the
// copy alone 53 us.  Bound by the chain of short phases that each CTA goes
// through besides its copy (count, list, correct: they move little, and grow
// with the distinct tokens, from 57 us at histories of 64 tokens to 71 us at
// 4096).  Every load whose address is known goes out before the first barrier
// (74 us with the drafts' and numbers' loads behind it); the grid has a
// dimension for each of a CTA's coordinates, as dividing one index apart took
// 0.4 us a wave.  Measured the other way: looking the table up while streaming
// 193 us (nearly every warp holds some repeated token and runs the rule for one
// or two of its lanes); listing the tokens while counting them 105 us, marking
// each with its first addition's result 72.2, finding them in the table
// afterwards 78; a slice of many tokens row by row through the rule, without a
// list, 94 (its one CTA outlasts the rest); one history for a cluster's CTAs,
// with additions into each other's tables, 110 us (3.6 cycles an addition and
// SM); persistent CTAs 149 us (rows differ too much); slices of interleaved
// blocks, which share out a vocabulary's frequent first tokens evenly, 80 to
// 95 us (more instructions for each token counted).

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kLgThreads = 256;
// Resident CTAs per SM: with 3 the ragged rows take 77 us, with 5 94, as registers
// spill (at 4 only the masked kernels of four vectors do, 40 bytes).
constexpr int kLgCtas = 4;
constexpr int kLgEnough = 912, kLgMost = 2432;   // CTAs: one and a half times those resident, and four times
constexpr int kLgMaxDrafts = 32;
// A table word: in the prompt, among the drafts, the last bias's entry + 1
// and the times generated in the history.
constexpr uint32_t kLgPrompt = 1u << 31, kLgDraft = 1u << 30;
constexpr int kLgBiasShift = 20;
constexpr uint32_t kLgBias = (kLgDraft - 1) >> kLgBiasShift << kLgBiasShift;   // 10 bits
constexpr uint32_t kLgCount = (1u << kLgBiasShift) - 1;
constexpr int kLgPad = 8;                 // tokens before the slice that a shifted row's vectors reach

struct LogitsParams {
  const unsigned char* logits;   // [B, R, V]
  unsigned char* out;            // [B, R, V], may be `logits`
  const int* history;            // [B, .] rows of `history_stride`
  const int* prompt_len;         // [B] or null: 0
  const int* history_len;        // [B] or null: history_max
  const int* tokens;             // [B, k]
  const int* draft_len;          // [B] or null: every row
  const float* repetition;       // [B] or null: 1
  const float* presence;         // [B] or null: 0
  const float* frequency;        // [B] or null: 0
  const int* bias_ids;           // [B, n_bias]
  const float* bias_values;      // [B, n_bias]
  const int* mask;               // [B, R, ceil(V / 32)]
  long long history_stride;
  int history_max;
  int B, R, V, k, n_bias;
  int group_rows;                // rows that a CTA takes
  int parts;                     // passes of 256 U vectors that a slice takes per row
  int list_max;                  // tokens that a table can hold at most
  int history_vec;               // history rows lie on 16 bytes
  int table;                     // there is something to look up: history, drafts or biases
  int same_shift;                // logits and out lie alike: rows go as 16-byte vectors
};

// Words of the bitmap over a table of `span` tokens: whole 16-byte units.
__host__ __device__ constexpr int lg_bitmap_words(int span) { return (span + 127) / 128 * 4; }

// Element by element a where the bit is set, else b: bit copies, so that a
// value that stays keeps its bits (a conversion would not keep a NaN's).
template <int ELT>
__device__ __forceinline__ uint4 select(uint32_t bits, uint4 a, uint4 b) {
  auto word = [&](int i, uint32_t x, uint32_t y) {
    uint32_t keep;
    if (ELT == 4) keep = 0u - ((bits >> i) & 1u);
    else keep = ((bits >> (2 * i)) & 1u) * 0xffffu + ((bits >> (2 * i + 1)) & 1u) * 0xffff0000u;
    return (x & keep) | (y & ~keep);
  };
  return make_uint4(word(0, a.x, b.x), word(1, a.y, b.y), word(2, a.z, b.z), word(3, a.w, b.w));
}

__device__ __forceinline__ bool mask_allows(const int* mask, int t) {
  return !mask || ((static_cast<uint32_t>(mask[t >> 5]) >> (t & 31)) & 1u);
}

// The mask and the copy for a vector that reaches past its row, or of a row
// that lies unlike in logits and out: element by element.
template <int ELT>
__device__ __noinline__ void edge_vector(const unsigned char* in, unsigned char* out, const int* mask, int t0,
                                         int V) {
  using VT = Vec<ELT>;
  for (int t = max(t0, 0); t < min(t0 + VT::N, V); ++t) {
    unsigned char* o = out + static_cast<long long>(t) * ELT;
    if (!mask_allows(mask, t)) VT::store_rounded(o, 0, -INFINITY);
    else if (in != out) VT::store_scalar(o, 0, load_elem<ELT>(in, t));   // the very bits
  }
}

// A thread's vectors of one pass over a row: what the mask says of them and,
// where they have to be read, their values.
template <int ELT, int U, bool MASK>
struct RowPart {
  uint4 w[U];
  uint32_t allowed[MASK ? U : 1];

  static constexpr int N = Vec<ELT>::N;
  static constexpr int kTokens = kLgThreads * U * N;
  static constexpr uint32_t kAll = (1u << N) - 1u;

  // Token of vector q of a pass from token s on.
  __device__ __forceinline__ static int token(int q, int s) {
    return s + (static_cast<int>(threadIdx.x) + q * kLgThreads) * N;
  }
  // s: first token of the pass less the row's shift.  A pass inside its row
  // needs no look at the row's ends.
  __device__ __forceinline__ static bool inside(const LogitsParams& P, int s) {
    return P.same_shift && s >= 0 && s <= P.V - kTokens;
  }
  __device__ __forceinline__ static bool whole(const LogitsParams& P, int t0) {
    return P.same_shift && t0 >= 0 && t0 <= P.V - N;
  }

  // The mask's bits for the pass; its vectors are loaded by them later.
  __device__ __forceinline__ void load_mask(const LogitsParams& P, long long r, int s0) {
    if (!MASK) return;
    const int s = s0 - row_shift<ELT>(P.logits + r * P.V * ELT);
    const int* mask = P.mask + r * ((P.V + 31) / 32);
    const bool all = inside(P, s);
#pragma unroll
    for (int q = 0; q < U; ++q) allowed[q] = all || whole(P, token(q, s)) ? bits_at<N>(mask, token(q, s)) : 0u;
  }
  __device__ __forceinline__ void load(const LogitsParams& P, long long r, int s0, bool in_place) {
    const unsigned char* in = P.logits + r * P.V * ELT;
    const int s = s0 - row_shift<ELT>(in);
    const unsigned char* at = in + static_cast<long long>(token(0, s)) * ELT;
    if (MASK) {
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (allowed[q] && !(in_place && allowed[q] == kAll)) w[q] = load_vec16(at + q * kLgThreads * 16);
    } else if (inside(P, s)) {
#pragma unroll
      for (int q = 0; q < U; ++q) w[q] = load_vec16(at + q * kLgThreads * 16);
    } else {
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (whole(P, token(q, s))) w[q] = load_vec16(at + q * kLgThreads * 16);
    }
  }
  __device__ __forceinline__ void store(const LogitsParams& P, long long r, int s0, bool in_place) const {
    const unsigned char* in = P.logits + r * P.V * ELT;
    unsigned char* out = P.out + r * P.V * ELT;
    const int s = s0 - row_shift<ELT>(in);
    unsigned char* at = out + static_cast<long long>(token(0, s)) * ELT;
    if (inside(P, s)) {
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (!(MASK && in_place && allowed[q] == kAll)) store_vec16(at + q * kLgThreads * 16, masked(q));
      return;
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (whole(P, token(q, s))) {
        if (!(MASK && in_place && allowed[q] == kAll)) store_vec16(at + q * kLgThreads * 16, masked(q));
      } else if (token(q, s) < P.V) {
        edge_vector<ELT>(in, out, MASK ? P.mask + r * ((P.V + 31) / 32) : nullptr, token(q, s), P.V);
      }
    }
  }
  __device__ __forceinline__ uint4 masked(int q) const {
    if (!MASK || allowed[MASK ? q : 0] == kAll) return w[q];
    if (!allowed[MASK ? q : 0]) return Vec<ELT>::neg_inf();
    return select<ELT>(allowed[MASK ? q : 0], w[q], Vec<ELT>::neg_inf());
  }
};

// A batch of history tokens, 4 kLgAhead per thread: entries
// lg_entry(j0, q) .. + 3; -1 from `end` on.
constexpr int kLgAhead = 4;
constexpr int kLgBatch = kLgThreads * 4 * kLgAhead;
__device__ __forceinline__ int lg_entry(int j0, int q) { return j0 + (static_cast<int>(threadIdx.x) + q * kLgThreads) * 4; }
__device__ __forceinline__ void load_history(const int* h, int j0, int end, int vec, int4 (&t)[kLgAhead]) {
#pragma unroll
  for (int q = 0; q < kLgAhead; ++q) {
    const int j = lg_entry(j0, q);
    if (j >= end) {
      t[q] = make_int4(-1, -1, -1, -1);
    } else if (vec && j + 3 < end) {
      t[q] = *reinterpret_cast<const int4*>(h + j);
    } else {
      t[q].x = j < end ? h[j] : -1;
      t[q].y = j + 1 < end ? h[j + 1] : -1;
      t[q].z = j + 2 < end ? h[j + 2] : -1;
      t[q].w = j + 3 < end ? h[j + 3] : -1;
    }
  }
}

// A token of the table in one row: what its correction reads.
struct LogitsFix {
  uint32_t word;     // the table's
  float z, bias;
  bool mine;

  template <int ELT>
  __device__ __forceinline__ void load(const LogitsParams& P, long long r, int s0, int n_slice, uint32_t w, int u, int b) {
    const unsigned char* row = P.logits + r * P.V * ELT;
    const int t = s0 - kLgPad + u;
    word = w;
    // the copy of the row's tokens from s0 - shift on is this CTA's; its
    // neighbour marks the few before s0 too
    mine = static_cast<unsigned>(u - kLgPad + row_shift<ELT>(row)) < static_cast<unsigned>(n_slice) &&
           mask_allows(P.mask ? P.mask + r * ((P.V + 31) / 32) : nullptr, t);
    z = load_elem<ELT>(row, t);
    if (word & kLgBias) bias = P.bias_values[static_cast<long long>(b) * P.n_bias + ((word & kLgBias) >> kLgBiasShift) - 1];
  }
};

// U vectors of a row per thread and pass.
template <int ELT, int U, bool MASK>
__global__ void __launch_bounds__(kLgThreads, kLgCtas) logits_kernel(const __grid_constant__ LogitsParams P) {
  using VT = Vec<ELT>;
  constexpr int kPart = kLgThreads * U * VT::N;    // tokens of a pass
  const int n_slice = kPart * P.parts;             // ... of the slice
  const int span = n_slice + kLgPad;               // ... of the table
  const int n_bitmap = lg_bitmap_words(span);
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int drafts[kLgMaxDrafts];
  __shared__ int n_listed;
  __shared__ float numbers[3];                     // repetition, presence, frequency
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem);
  uint32_t* touched = tab + span;                                  // bitmap over the table
  uint16_t* list = reinterpret_cast<uint16_t*>(touched + n_bitmap);   // [list_max]
  const int tid = threadIdx.x;
  // slice-major: a vocabulary's first tokens are its most frequent, so the
  // slices with the most to look up go first
  const int b = blockIdx.x, s0 = static_cast<int>(blockIdx.z) * n_slice, first = s0 - kLgPad;
  const int i0 = static_cast<int>(blockIdx.y) * P.group_rows;   // this CTA's first row
  const long long r0 = static_cast<long long>(b) * P.R + i0;
  const bool in_place = P.logits == P.out;
  const bool copies = MASK || !in_place;

  // ---- every load whose address is known goes out at once
  const int kb = P.draft_len ? P.draft_len[b] : P.k;
  const int* h = P.history + b * P.history_stride;
  int4 t[kLgAhead];
  int len = 0, plen = 0;
  if (P.history) {
    len = P.history_len ? P.history_len[b] : P.history_max;
    plen = P.prompt_len ? P.prompt_len[b] : 0;
    load_history(h, 0, P.history_max, P.history_vec, t);
  }
  int draft = -1;                                  // thread j has draft j
  float number = 0.f;                              // and one of the sequence's numbers
  if (P.table) {
    if (P.tokens && tid < P.k) draft = P.tokens[static_cast<long long>(b) * P.k + tid];
    if (tid == 0) number = P.repetition ? P.repetition[b] : 1.f;
    if (tid == 1) number = P.presence ? P.presence[b] : 0.f;
    if (tid == 2) number = P.frequency ? P.frequency[b] : 0.f;
  }
  RowPart<ELT, U, MASK> part;
  if (copies) {
    part.load_mask(P, r0, s0);
    part.load(P, r0, s0, in_place);
  }

  // ---- the table of the slice's tokens
  int n_fixes = 0;
  if (P.table) {
    uint4* zero = reinterpret_cast<uint4*>(smem);
    for (int w = tid; w < (span + n_bitmap) / 4; w += kLgThreads) zero[w] = make_uint4(0, 0, 0, 0);
    if (tid == 0) n_listed = 0;
    __syncthreads();                             // waits for none of the loads
  }
  if (kb < 0 || kb > P.k) return;                // the verifier reports it
  const int rows = min(P.group_rows, (P.draft_len ? min(P.R, kb + (P.R - P.k)) : P.R) - i0);
  if (rows <= 0) return;
  const int n_drafts = P.tokens ? kb : 0;
  LogitsFix fix;                                 // this thread's first (token, row) pair
  if (P.table) {
    auto touch = [&](int u) { atomicOr(&touched[u >> 5], 1u << (u & 31)); };
    // a token's place in this CTA's table, or -1
    auto place = [&](int x) {
      const int u = x - first;
      return x >= 0 && x < P.V && static_cast<unsigned>(u) < static_cast<unsigned>(span) ? u : -1;
    };
    if (P.n_bias) {   // the largest entry wins a token's word, before anything is added to it
      const int* ids = P.bias_ids + static_cast<long long>(b) * P.n_bias;
      for (int j = tid; j < P.n_bias; j += kLgThreads) {
        const int u = place(ids[j]);
        if (u >= 0) atomicMax(&tab[u], static_cast<uint32_t>(j + 1) << kLgBiasShift), touch(u);
      }
      __syncthreads();
    }
    if (tid < 3) numbers[tid] = number;
    if (tid < n_drafts) {
      drafts[tid] = draft;
      const int u = place(draft);
      if (u >= 0) atomicOr(&tab[u], kLgDraft), touch(u);
    }
    if (P.history) {
      len = min(len, P.history_max);
      // places of the tokens in [0, V) from `base` on: unsigned, so that what
      // lies before the slice, a -1 or any other id out of range is past them
      const int base = max(0, first), skipped = base - first;
      const uint32_t count = static_cast<uint32_t>(max(0, min(span - skipped, P.V - base)));
      uint32_t* const words = tab + skipped;
      auto add = [&](int x) {
        const uint32_t u = static_cast<uint32_t>(x) - static_cast<uint32_t>(base);
        if (u < count) atomicAdd(&words[u], 1u);
        if (u < count) touch(static_cast<int>(u) + skipped);
      };
      auto add_prompt = [&](int x) {
        const uint32_t u = static_cast<uint32_t>(x) - static_cast<uint32_t>(base);
        if (u < count) atomicOr(&words[u], kLgPrompt);
        if (u < count) touch(static_cast<int>(u) + skipped);
      };
      for (int j0 = 0; j0 < len; j0 += kLgBatch) {
        if (j0 > 0) load_history(h, j0, len, P.history_vec, t);
#pragma unroll
        for (int q = 0; q < kLgAhead; ++q) {
          const int j = lg_entry(j0, q);
          if (j >= len) break;
          if (j >= plen && j + 3 < len) {
            add(t[q].x); add(t[q].y); add(t[q].z); add(t[q].w);
          } else if (j + 3 < plen && j + 3 < len) {
            add_prompt(t[q].x); add_prompt(t[q].y); add_prompt(t[q].z); add_prompt(t[q].w);
          } else {
            for (int e = 0; e < 4 && j + e < len; ++e) {
              const int x = e == 0 ? t[q].x : e == 1 ? t[q].y : e == 2 ? t[q].z : t[q].w;
              if (j + e < plen) add_prompt(x);
              else add(x);
            }
          }
        }
      }
    }
    __syncthreads();
    // the list of the tokens that the table holds
    for (int w = tid; w < n_bitmap; w += kLgThreads) {
      uint32_t bits = touched[w];
      if (!bits) continue;
      int at = atomicAdd(&n_listed, __popc(bits));
      for (; bits; bits &= bits - 1) list[at++] = static_cast<uint16_t>(w * 32 + __ffs(bits) - 1);
    }
    __syncthreads();
    n_fixes = n_listed * rows;
    if (tid < n_fixes) {   // what it reads arrives during the copy
      const int i = tid / n_listed, u = list[tid - i * n_listed];
      fix.load<ELT>(P, r0 + i, s0, n_slice, tab[u], u, b);
    }
  }

  // ---- the mask and the copy: a pass's logits are loaded a pass ahead, its
  // mask two
  if (copies) {
    const int passes = rows * P.parts;
    int i = 0, q = 0;                // the pass two ahead of the one stored
    auto next = [&] {
      if (++q == P.parts) q = 0, ++i;
    };
    next();
    int at_row = 0, at_s = s0;
    RowPart<ELT, U, MASK> ahead;
    if (passes > 1) ahead.load_mask(P, r0 + i, s0 + q * kPart);
    for (int pass = 0; pass < passes; ++pass) {
      const int row_ahead = i, s_ahead = s0 + q * kPart;
      if (pass + 1 < passes) ahead.load(P, r0 + row_ahead, s_ahead, in_place);
      next();
      RowPart<ELT, U, MASK> after;
      if (MASK && pass + 2 < passes) after.load_mask(P, r0 + i, s0 + q * kPart);
      part.store(P, r0 + at_row, at_s, in_place);
      part = ahead;
      if (MASK) {
#pragma unroll
        for (int k = 0; k < U; ++k) ahead.allowed[MASK ? k : 0] = after.allowed[MASK ? k : 0];
      }
      at_row = row_ahead;
      at_s = s_ahead;
    }
  }
  if (n_fixes == 0) return;

  // ---- the tokens of the table, their stores after the copy's: a thread for
  // each token of each row, row by row, so that a warp's tokens are neighbours
  // where a slice holds many (48 sequences of eight rows with histories of
  // 16384: 68.5 us, with a token's rows side by side 70.2)
  __syncthreads();
  auto correct = [&](const LogitsFix& f, int j) {
    const int i = j / n_listed, u = list[j - i * n_listed];
    if (!f.mine) return;
    int n = static_cast<int>(f.word & kLgCount);
    if (f.word & kLgDraft)
      for (int d = 0; d < min(i0 + i, n_drafts); ++d) n += drafts[d] == first + u;
    const bool seen = n > 0 || (f.word & kLgPrompt);
    if (!seen && !(f.word & kLgBias)) return;   // drafted only later
    float z = f.z;
    if (seen) z = z > 0.f ? __fdiv_rn(z, numbers[0]) : __fmul_rn(z, numbers[0]);
    if (n > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(numbers[2], static_cast<float>(n))), numbers[1]);
    if (f.word & kLgBias) z = __fadd_rn(z, f.bias);
    VT::store_rounded(P.out + ((r0 + i) * P.V + first + u) * ELT, 0, z);
  };
  if (tid < n_fixes) correct(fix, tid);
  // more than a thread each: four at a time, so that their loads overlap
  constexpr int kMore = 4;
  for (int j0 = kLgThreads + tid; j0 < n_fixes; j0 += kLgThreads * kMore) {
    LogitsFix more[kMore];
#pragma unroll
    for (int q = 0; q < kMore; ++q) {
      const int j = min(j0 + q * kLgThreads, n_fixes - 1), i = j / n_listed, u = list[j - i * n_listed];
      more[q].load<ELT>(P, r0 + i, s0, n_slice, tab[u], u, b);
    }
#pragma unroll
    for (int q = 0; q < kMore; ++q)
      if (j0 + q * kLgThreads < n_fixes) correct(more[q], j0 + q * kLgThreads);
  }
}

int logits_smem(int n_tokens, int list_max) {
  const int span = n_tokens + kLgPad;
  return 4 * (span + lg_bitmap_words(span)) + (list_max + 1) / 2 * 4;
}

}  // namespace
}  // namespace sv

extern "C" sv_status sv_process_logits(int B, int R, int V, sv_dtype dtype, const void* logits, void* out,
                                       int history_max, long long history_stride, const int32_t* history,
                                       const int32_t* prompt_len, const int32_t* history_len, int k,
                                       const int32_t* tokens, const int32_t* draft_len, const float* repetition,
                                       const float* presence, const float* frequency, int n_bias,
                                       const int32_t* bias_ids, const float* bias_values, const int32_t* mask,
                                       sv_stream_t stream) {
  using namespace sv;
  if (B < 1 || R < 1 || V < 1 || k < 0 || k >= kLgMaxDrafts || n_bias < 0 || n_bias > SV_MAX_BIASES || history_max < 0) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (!logits || !out || (n_bias && (!bias_ids || !bias_values)) || (history_max && !history)) return SV_ERR_INVALID_ARG;
  if ((tokens || draft_len) && R != k && R != k + 1) return SV_ERR_INVALID_ARG;
  if (history_max > static_cast<int>(kLgCount) || (history_max && history_stride < history_max)) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * R > (1LL << 30)) return SV_ERR_INVALID_ARG;
  const int elt = dtype == SV_F32 ? 4 : 2;
  if (static_cast<long long>(V) * elt > (1LL << 30) - (1 << 16)) return SV_ERR_INVALID_ARG;   // 65535 slices
  const uintptr_t a = reinterpret_cast<uintptr_t>(logits), o = reinterpret_cast<uintptr_t>(out);
  const uintptr_t bytes = static_cast<uintptr_t>(B) * R * V * elt;
  if (a % elt || o % elt) return SV_ERR_INVALID_ARG;
  if (a != o && a < o + bytes && o < a + bytes) return SV_ERR_INVALID_ARG;   // neither in place nor apart

  LogitsParams p{};
  p.logits = static_cast<const unsigned char*>(logits);
  p.out = static_cast<unsigned char*>(out);
  p.history = history_max ? history : nullptr;
  p.prompt_len = prompt_len;
  p.history_len = history_len;
  p.tokens = k ? tokens : nullptr;
  p.draft_len = draft_len;
  p.repetition = repetition;
  p.presence = presence;
  p.frequency = frequency;
  p.bias_ids = bias_ids;
  p.bias_values = bias_values;
  p.mask = mask;
  p.history_stride = history_stride;
  p.history_max = history_max;
  p.B = B; p.R = R; p.V = V; p.k = k; p.n_bias = n_bias;
  const bool penalties = repetition || presence || frequency;
  if (!penalties) p.history = nullptr, p.tokens = nullptr;   // counts that nothing asks for
  p.table = p.history || p.tokens || n_bias;
  p.same_shift = (a % 16) == (o % 16);

  // Slices as large as give the SMs enough CTAs with two rows to a CTA: a
  // history is read once a CTA, and a slice of frequent tokens, which has the
  // most to correct, is shared out by its rows.  256 rows of 32000 with
  // histories of 4096: 15.4 us at 1024 CTAs, with half the slice 19.4; 14
  // sequences of 8 rows of 42896 and 16384: 22 us at 336, 19.8 at 1176.
  // Then CTAs take fewer rows, down to two, up to kLgMost CTAs (48 sequences of
  // 8 rows of 100003 fp32 logits: 67.6 us with 4, with 8 79.8), and one as long
  // as all fit on the SMs twice (33 sequences of 4 rows of 9951: 6.8 us, with
  // 2 rows 8.4; 64 of 8 of 32000, which would not: 19.1 and 16.4).
  const int n = elt == 2 ? 8 : 4;
  int unroll = 1;
  auto slices = [&](int u) { return (V + n - 1 + kLgThreads * u * n - 1) / (kLgThreads * u * n); };
  while (unroll < 4 && static_cast<long long>(B) * slices(2 * unroll) * ((R + 1) / 2) >= kLgEnough) unroll *= 2;
  // fp32 slices of as many tokens as bf16's, as the history is read once a
  // slice; but not where the corrections of a slice of frequent tokens would
  // outlast the rest.  512 sequences of one row with histories of 16384: 156 us
  // against 187; 192 of two 91 and 103; 256 of four with 4096 117 and 123, with
  // 16384 180 and 153; 96 of eight with 2048 89 and 82, with 16384 137 and 108
  const bool few = R <= 2 || (R <= 4 && history_max <= 8192);
  p.parts = elt == 4 && unroll == 4 && p.history && few && static_cast<long long>(B) * slices(8) >= kLgEnough ? 2 : 1;
  const long long slice_ctas = static_cast<long long>(B) * slices(unroll * p.parts);
  int groups = 1;
  while (groups < (R + 1) / 2 && slice_ctas * (groups + 1) <= kLgMost) ++groups;
  while (groups < R && slice_ctas * (groups + 1) <= kLgMost / 2) ++groups;
  p.group_rows = (R + groups - 1) / groups;
  const dim3 grid(B, (R + p.group_rows - 1) / p.group_rows, slices(unroll * p.parts));
  const int n_tokens = kLgThreads * unroll * n * p.parts;
  const long long held = (p.history ? history_max : 0LL) + (p.tokens ? k : 0) + n_bias;
  p.list_max = static_cast<int>(held < n_tokens + kLgPad ? held : n_tokens + kLgPad);
  p.history_vec = reinterpret_cast<uintptr_t>(history) % 16 == 0 && (history_stride % 4 == 0 || B == 1);
  const int smem = p.table ? logits_smem(n_tokens, p.list_max) : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_process_logits");
  auto launch = [&](auto kernel) {
    // up to 50 KB a CTA: above the 48 KB that need no asking
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess)
      return SV_ERR_CUDA;
    kernel<<<grid, kLgThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  };
#define SV_LAUNCH(ELT, U) (mask ? launch(logits_kernel<ELT, U, true>) : launch(logits_kernel<ELT, U, false>))
  if (elt == 2) return unroll == 4 ? SV_LAUNCH(2, 4) : unroll == 2 ? SV_LAUNCH(2, 2) : SV_LAUNCH(2, 1);
  return unroll == 4 ? SV_LAUNCH(4, 4) : unroll == 2 ? SV_LAUNCH(4, 2) : SV_LAUNCH(4, 1);
#undef SV_LAUNCH
}
