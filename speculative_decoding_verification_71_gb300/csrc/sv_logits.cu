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
// A CTA takes one slice of the vocabulary of one sequence and all its rows.
// It counts the history's tokens of its slice into a shared-memory table (an
// integer word per token, so the order of the additions cannot show) and
// marks them in a bitmap.  Two passes over the slice's rows follow:
//   - the mask and the copy, 16 bytes at a time and without a look at the
//     table (a vector that is masked altogether is written without being
//     read; in place, only what the mask forbids is touched); its first loads
//     are under way while the history is counted;
//   - the tokens of the bitmap, a thread for each token of each row.
// Looking the table up while streaming cost more than the stream: nearly
// every warp holds some repeated token, and ran the rule for one or two of
// its lanes (193 us against 106 on 256 sequences of up to four rows of
// 128256 bf16 logits, histories of up to 4096 tokens).  The counting is
// without a result that a thread would wait for and without a branch per
// token: listing the tokens while counting them, or sharing the history among
// a cluster's CTAs with additions into each other's tables (3.6 cycles an
// addition and SM), took 105 and 110 us against @@.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kLgThreads = 256;
constexpr int kLgCtas = 4;                // resident per SM
constexpr int kLgMaxDrafts = 32;
constexpr uint32_t kLgPrompt = 1u << 31;  // table word: in the prompt
constexpr uint32_t kLgDraft = 1u << 30;   // ... among the drafts
constexpr uint32_t kLgBias = 1u << 29;    // ... has a bias
constexpr uint32_t kLgCount = kLgBias - 1;    // ... times generated in the history
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
  int table;                     // there is something to look up: history, drafts or biases
  int same_shift;                // logits and out lie alike: rows go as 16-byte vectors
};

// Words of the bitmap over a table of `span` tokens: whole 16-byte units.
#define SV_LG_BITMAP_WORDS(span) (((span) + 127) / 128 * 4)

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

// A thread's vectors of one row's slice: what the mask says of them and, where
// they have to be read, their values.
template <int ELT, int U>
struct RowPart {
  uint4 w[U];
  uint32_t allowed[U];

  static constexpr int N = Vec<ELT>::N;
  static constexpr uint32_t kAll = (1u << N) - 1u;

  __device__ __forceinline__ static int token(int q, int s0, int shift) {
    return s0 - shift + (static_cast<int>(threadIdx.x) + q * kLgThreads) * N;
  }
  __device__ __forceinline__ void load(const LogitsParams& P, long long r, int s0, bool in_place) {
    const unsigned char* in = P.logits + r * P.V * ELT;
    const int* mask = P.mask ? P.mask + r * ((P.V + 31) / 32) : nullptr;
    const int shift = row_shift<ELT>(in);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int t0 = token(q, s0, shift);
      const bool whole = P.same_shift && t0 >= 0 && t0 <= P.V - N;
      allowed[q] = mask && whole ? bits_at<N>(mask, t0) : kAll;
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int t0 = token(q, s0, shift);
      const bool whole = P.same_shift && t0 >= 0 && t0 <= P.V - N;
      if (whole && allowed[q] && !(in_place && allowed[q] == kAll)) w[q] = load_vec16(in + static_cast<long long>(t0) * ELT);
    }
  }
  __device__ __forceinline__ void store(const LogitsParams& P, long long r, int s0, bool in_place) const {
    const unsigned char* in = P.logits + r * P.V * ELT;
    unsigned char* out = P.out + r * P.V * ELT;
    const int shift = row_shift<ELT>(in);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int t0 = token(q, s0, shift);
      if (P.same_shift && t0 >= 0 && t0 <= P.V - N) {
        if (in_place && allowed[q] == kAll) continue;
        uint4 res = w[q];
        if (allowed[q] != kAll)
          res = allowed[q] ? select<ELT>(allowed[q], res, Vec<ELT>::neg_inf()) : Vec<ELT>::neg_inf();
        store_vec16(out + static_cast<long long>(t0) * ELT, res);
      } else if (t0 < P.V) {
        edge_vector<ELT>(in, out, P.mask ? P.mask + r * ((P.V + 31) / 32) : nullptr, t0, P.V);
      }
    }
  }
};

// A batch of history tokens, kLgAhead per thread from entry j0 + thread on;
// -1 past history_max.
constexpr int kLgAhead = 8;
__device__ __forceinline__ void load_history(const int* h, int j0, int end, int (&t)[kLgAhead]) {
#pragma unroll
  for (int q = 0; q < kLgAhead; ++q) {
    const int j = j0 + static_cast<int>(threadIdx.x) + q * kLgThreads;
    t[q] = j < end ? h[j] : -1;
  }
}

// U vectors of a row per thread: slices of 256 U vectors.
template <int ELT, int U>
__global__ void __launch_bounds__(kLgThreads, kLgCtas) logits_kernel(const __grid_constant__ LogitsParams P) {
  using VT = Vec<ELT>;
  constexpr int kSlice = kLgThreads * U * VT::N;   // tokens
  constexpr int span = kSlice + kLgPad;            // tokens the table covers
  constexpr int kBitmap = SV_LG_BITMAP_WORDS(span);
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int drafts[kLgMaxDrafts];
  __shared__ int n_listed;
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem);
  uint32_t* touched = tab + span;                                  // bitmap over the table
  int* slot = reinterpret_cast<int*>(touched + kBitmap);           // biases: last entry + 1, with biases only
  uint16_t* list = reinterpret_cast<uint16_t*>(slot + (P.n_bias ? span : 0));
  const int tid = threadIdx.x;
  // slice-major: a vocabulary's first tokens are its most frequent, so the
  // slices with the most to look up go first
  const int b = blockIdx.x % P.B, s0 = blockIdx.x / P.B * kSlice, first = s0 - kLgPad;
  const long long r0 = static_cast<long long>(b) * P.R;
  const bool in_place = P.logits == P.out;
  const bool copies = !in_place || P.mask;

  // ---- every load whose address is known goes out at once
  const int kb = P.draft_len ? P.draft_len[b] : P.k;
  const int* h = P.history + b * P.history_stride;
  int t[kLgAhead];
  int len = 0, plen = 0;
  if (P.history) {
    len = P.history_len ? P.history_len[b] : P.history_max;
    plen = P.prompt_len ? P.prompt_len[b] : 0;
    load_history(h, 0, P.history_max, t);
  }
  RowPart<ELT, U> part;
  if (copies) part.load(P, r0, s0, in_place);

  // ---- the table of the slice's tokens
  int n_fixes = 0;
  if (P.table) {
    uint4* zero = reinterpret_cast<uint4*>(smem);
    for (int w = tid; w < (span + kBitmap + (P.n_bias ? span : 0)) / 4; w += kLgThreads) zero[w] = make_uint4(0, 0, 0, 0);
    if (tid == 0) n_listed = 0;
  }
  if (kb < 0 || kb > P.k) return;                // the verifier reports it
  const int rows = P.draft_len ? min(P.R, kb + (P.R - P.k)) : P.R;
  const int n_drafts = P.tokens ? kb : 0;
  int fix_u = -1;                                // this thread's first (token, row) pair
  float fix_z = 0.f;
  if (P.table) {
    if (tid < n_drafts) drafts[tid] = P.tokens[static_cast<long long>(b) * P.k + tid];
    __syncthreads();
    auto touch = [&](int u) { atomicOr(&touched[u >> 5], 1u << (u & 31)); };
    if (P.history) {
      len = min(len, P.history_max);
      const int end = min(span, P.V - first);    // places of tokens in [0, V)
      const int start = max(0, -first);
      for (int j0 = 0; j0 < len; j0 += kLgThreads * kLgAhead) {
        int ahead[kLgAhead];
        load_history(h, j0 + kLgThreads * kLgAhead, len, ahead);
#pragma unroll
        for (int q = 0; q < kLgAhead; ++q) {
          const int j = j0 + tid + q * kLgThreads;
          const int u = t[q] < 0 ? -1 : t[q] - first;
          const bool in = u >= start && u < end && j < len;
          if (in && j >= plen) atomicAdd(&tab[u], 1u);
          if (in && j < plen) atomicOr(&tab[u], kLgPrompt);
          if (in) touch(u);
          t[q] = ahead[q];
        }
      }
    }
    // a token's place in this CTA's table, or -1
    auto place = [&](int x) {
      const int u = x - first;
      return x >= 0 && x < P.V && static_cast<unsigned>(u) < static_cast<unsigned>(span) ? u : -1;
    };
    auto mark = [&](int u, uint32_t flag) {
      atomicOr(&tab[u], flag);
      touch(u);
    };
    if (tid < n_drafts) {
      const int u = place(drafts[tid]);
      if (u >= 0) mark(u, kLgDraft);
    }
    // the last bias of a token counts: the largest entry wins the token's word
    const int* ids = P.bias_ids + static_cast<long long>(b) * P.n_bias;
    for (int j = tid; j < P.n_bias; j += kLgThreads) {
      const int u = place(ids[j]);
      if (u >= 0) atomicMax(&slot[u], j + 1), mark(u, kLgBias);
    }
    __syncthreads();
    // the list of the tokens that the table holds
    for (int w = tid; w < kBitmap; w += kLgThreads) {
      uint32_t bits = touched[w];
      if (!bits) continue;
      int at = atomicAdd(&n_listed, __popc(bits));
      for (; bits; bits &= bits - 1) list[at++] = static_cast<uint16_t>(w * 32 + __ffs(bits) - 1);
    }
    __syncthreads();
    n_fixes = n_listed * rows;
    if (tid < n_fixes) {   // its logit arrives during the copy
      fix_u = list[tid / rows];
      const int x = min(max(first + fix_u, 0), P.V - 1);
      fix_z = load_elem<ELT>(P.logits + (r0 + tid % rows) * P.V * ELT, x);
    }
  }

  // ---- the mask and the copy, a row ahead
  for (int i = 0; copies && i < rows; ++i) {
    RowPart<ELT, U> ahead;
    if (i + 1 < rows) ahead.load(P, r0 + i + 1, s0, in_place);
    part.store(P, r0 + i, s0, in_place);
    part = ahead;
  }
  if (n_fixes == 0) return;

  // ---- the tokens of the table, their stores after the copy's: a thread for
  // each token of each row
  __syncthreads();
  const float rep = P.repetition ? P.repetition[b] : 1.f, pres = P.presence ? P.presence[b] : 0.f,
              freq = P.frequency ? P.frequency[b] : 0.f;
  const int mask_words = (P.V + 31) / 32;
  for (int j = tid; j < n_fixes; j += kLgThreads) {
    const bool have = j == tid;
    const int i = j % rows, u = have ? fix_u : list[j / rows], x = first + u;
    const uint32_t c = tab[u];
    int n = static_cast<int>(c & kLgCount);
    if (c & kLgDraft)
      for (int d = 0; d < min(i, n_drafts); ++d) n += drafts[d] == x;
    const bool seen = n > 0 || (c & kLgPrompt);
    if (!seen && !(c & kLgBias)) continue;   // drafted only later
    // the copy of the row's tokens from s0 - shift on is this CTA's; its
    // neighbour marks the few before s0 too
    const long long r = r0 + i;
    const unsigned char* rowp = P.logits + r * P.V * ELT;
    if (static_cast<unsigned>(u - kLgPad + row_shift<ELT>(rowp)) >= static_cast<unsigned>(kSlice)) continue;
    if (!mask_allows(P.mask ? P.mask + r * mask_words : nullptr, x)) continue;
    float z = have ? fix_z : load_elem<ELT>(rowp, x);
    if (seen) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
    if (n > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, static_cast<float>(n))), pres);
    if (c & kLgBias) z = __fadd_rn(z, P.bias_values[static_cast<long long>(b) * P.n_bias + slot[u] - 1]);
    VT::store_rounded(P.out + (r * P.V + x) * ELT, 0, z);
  }
}

int logits_smem(int n_tokens, bool table, bool with_bias) {
  const int span = n_tokens + kLgPad;
  return table ? span * (with_bias ? 10 : 6) + 4 * SV_LG_BITMAP_WORDS(span) : 0;
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
  if (B < 1 || R < 1 || V < 1 || k < 0 || k >= kLgMaxDrafts || n_bias < 0 || history_max < 0) return SV_ERR_INVALID_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
  if (!logits || !out || (n_bias && (!bias_ids || !bias_values)) || (history_max && !history)) return SV_ERR_INVALID_ARG;
  if ((tokens || draft_len) && R != k && R != k + 1) return SV_ERR_INVALID_ARG;
  if (history_max >= (1 << 29) || (history_max && history_stride < history_max)) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * R > (1LL << 30)) return SV_ERR_INVALID_ARG;
  const int elt = dtype == SV_F32 ? 4 : 2;
  if (static_cast<long long>(V) * elt > (1LL << 30)) return SV_ERR_INVALID_ARG;
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

  // the largest slices that still give every SM several CTAs
  const int n = elt == 2 ? 8 : 4;
  int unroll = 1;
  auto slices = [&](int u) { return (V + n - 1 + kLgThreads * u * n - 1) / (kLgThreads * u * n); };
  const int most = n_bias ? 2 : 4;   // with biases the table is twice as large (34 KB at most)
  while (unroll < most && static_cast<long long>(B) * slices(2 * unroll) >= 1216) unroll *= 2;
  const long long ctas = static_cast<long long>(B) * slices(unroll);
  if (ctas > 0x7fffffffLL) return SV_ERR_INVALID_ARG;
  const int smem = logits_smem(kLgThreads * unroll * n, p.table, n_bias > 0);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_process_logits");
  auto launch = [&](auto kernel) {
    // up to 50 KB a CTA: above the 48 KB that need no asking
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess)
      return SV_ERR_CUDA;
    kernel<<<static_cast<unsigned>(ctas), kLgThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  };
  if (elt == 2)
    return unroll == 4 ? launch(logits_kernel<2, 4>) : unroll == 2 ? launch(logits_kernel<2, 2>) : launch(logits_kernel<2, 1>);
  return unroll == 4 ? launch(logits_kernel<4, 4>) : unroll == 2 ? launch(logits_kernel<4, 2>) : launch(logits_kernel<4, 1>);
}
