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
// integer word per token, so the order of the atomics cannot show) and lists
// the tokens that the table holds.  Then two passes over the slice's rows:
//   - the mask and the copy, 16 bytes at a time and without a look at the
//     table (a vector that is masked altogether is written without being
//     read; in place, only what the mask forbids is touched);
//   - the listed tokens, a thread each, through all rows: the count grows by
//     one after every draft of the token.
// Looking the table up while streaming cost more than the stream: nearly
// every warp holds some repeated token, and ran the rule for one or two of
// its lanes (193 us against 106 on 256 sequences of up to four rows of
// 128256 bf16 logits, histories of up to 4096 tokens).

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kLgThreads = 256;
constexpr int kLgUnroll = 4;              // vectors in flight per thread
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
  int lg_vecs;                   // log2 of the vectors of a slice
  int n_slices;
  int table;                     // there is something to look up: history, drafts or biases
  int same_shift;                // logits and out lie alike: rows go as 16-byte vectors
};

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

template <int ELT>
__global__ void __launch_bounds__(kLgThreads, 4) logits_kernel(const __grid_constant__ LogitsParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  constexpr uint32_t kAll = (1u << N) - 1u;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int drafts[kLgMaxDrafts];
  __shared__ int n_listed;
  const int b = blockIdx.x / P.n_slices, slice = blockIdx.x % P.n_slices;
  const int nv = 1 << P.lg_vecs;
  const int span = nv * N + kLgPad;          // tokens the table covers
  const int s0 = slice * nv * N, first = s0 - kLgPad;
  const int tid = threadIdx.x;

  int rows = P.R, n_drafts = P.k;
  if (P.draft_len) {
    const int kb = P.draft_len[b];
    if (kb < 0 || kb > P.k) return;          // the verifier reports it
    rows = min(P.R, kb + (P.R - P.k));
    n_drafts = kb;
  }
  if (!P.tokens) n_drafts = 0;

  // ---- the table of the slice's tokens, and the list of those it holds
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem);
  float* bias = reinterpret_cast<float*>(tab + span);                        // with biases only
  uint16_t* list = reinterpret_cast<uint16_t*>(tab + span * (P.n_bias ? 2 : 1));
  if (P.table) {
    uint4* zero = reinterpret_cast<uint4*>(smem);
    for (int w = tid; w < span * (P.n_bias ? 2 : 1) / 4; w += kLgThreads) zero[w] = make_uint4(0, 0, 0, 0);
    if (tid < n_drafts) drafts[tid] = P.tokens[static_cast<long long>(b) * P.k + tid];
    if (tid == 0) n_listed = 0;
    __syncthreads();
    // a token's place in the table, or -1
    auto place = [&](int t) {
      const int u = t - first;
      return t >= 0 && t < P.V && static_cast<unsigned>(u) < static_cast<unsigned>(span) ? u : -1;
    };
    // the one whose operation found the word empty lists it
    auto note = [&](int u, uint32_t before) {
      if (before == 0) list[atomicAdd(&n_listed, 1)] = static_cast<uint16_t>(u);
    };
    if (P.history) {
      const int* h = P.history + b * P.history_stride;
      const int len = min(P.history_len ? max(P.history_len[b], 0) : P.history_max, P.history_max);
      const int plen = P.prompt_len ? P.prompt_len[b] : 0;
      constexpr int kAhead = 8;              // loads in flight per thread
      for (int j0 = tid; j0 < len; j0 += kLgThreads * kAhead) {
        int t[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) t[q] = j0 + q * kLgThreads < len ? h[j0 + q * kLgThreads] : -1;
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          const int u = place(t[q]);
          if (u < 0) continue;
          note(u, j0 + q * kLgThreads < plen ? atomicOr(&tab[u], kLgPrompt) : atomicAdd(&tab[u], 1u));
        }
      }
    }
    if (tid < n_drafts) {
      const int u = place(drafts[tid]);
      if (u >= 0) note(u, atomicOr(&tab[u], kLgDraft));
    }
    if (P.n_bias) {
      // the last entry of a token counts: the largest index + 1 wins the
      // token's word, which then takes the winner's value
      const int* ids = P.bias_ids + static_cast<long long>(b) * P.n_bias;
      int* slot = reinterpret_cast<int*>(bias);
      for (int j = tid; j < P.n_bias; j += kLgThreads) {
        const int u = place(ids[j]);
        if (u >= 0) atomicMax(&slot[u], j + 1), note(u, atomicOr(&tab[u], kLgBias));
      }
    }
  }

  // ---- the mask and the copy
  const bool in_place = P.logits == P.out;
  const int mask_words = (P.V + 31) / 32;
  const long long r0 = static_cast<long long>(b) * P.R;
  const int items = in_place && !P.mask ? 0 : rows << P.lg_vecs;
  for (int it = tid; it < items; it += kLgThreads * kLgUnroll) {
    uint4 w[kLgUnroll];
    uint32_t allowed[kLgUnroll];
    int t0[kLgUnroll];
    bool whole[kLgUnroll];
#pragma unroll
    for (int q = 0; q < kLgUnroll; ++q) {
      const int item = it + q * kLgThreads;
      const bool in = item < items;
      const long long r = r0 + (item >> P.lg_vecs);
      const unsigned char* rowp = P.logits + r * P.V * ELT;
      t0[q] = in ? s0 - row_shift<ELT>(rowp) + (item & (nv - 1)) * N : P.V;
      whole[q] = in && P.same_shift && t0[q] >= 0 && t0[q] <= P.V - N;
      allowed[q] = whole[q] && P.mask ? bits_at<N>(P.mask + r * mask_words, t0[q]) : kAll;
    }
#pragma unroll
    for (int q = 0; q < kLgUnroll; ++q) {
      const long long r = r0 + ((it + q * kLgThreads) >> P.lg_vecs);
      if (whole[q] && allowed[q] && !(in_place && allowed[q] == kAll))
        w[q] = load_vec16(P.logits + (r * P.V + t0[q]) * ELT);
    }
#pragma unroll
    for (int q = 0; q < kLgUnroll; ++q) {
      const long long r = r0 + ((it + q * kLgThreads) >> P.lg_vecs);
      if (whole[q]) {
        if (in_place && allowed[q] == kAll) continue;
        store_vec16(P.out + (r * P.V + t0[q]) * ELT,
                    allowed[q] == kAll ? w[q] : allowed[q] ? select<ELT>(allowed[q], w[q], VT::neg_inf()) : VT::neg_inf());
      } else if (t0[q] < P.V) {
        edge_vector<ELT>(P.logits + r * P.V * ELT, P.out + r * P.V * ELT, P.mask ? P.mask + r * mask_words : nullptr,
                         t0[q], P.V);
      }
    }
  }
  if (!P.table) return;

  // ---- the listed tokens, their stores after the copy's
  __syncthreads();
  const float rep = P.repetition ? P.repetition[b] : 1.f, pres = P.presence ? P.presence[b] : 0.f,
              freq = P.frequency ? P.frequency[b] : 0.f;
  for (int j = tid; j < n_listed; j += kLgThreads) {
    const int u = list[j], t = first + u;
    const uint32_t c = tab[u];
    int n = static_cast<int>(c & kLgCount);
    float add = 0.f;
    if (c & kLgBias) {
      const int at = reinterpret_cast<const int*>(bias)[u];
      add = P.bias_values[static_cast<long long>(b) * P.n_bias + at - 1];
    }
    for (int i = 0; i < rows; ++i) {
      if (i > 0 && (c & kLgDraft) && i <= n_drafts) n += drafts[i - 1] == t;
      const bool seen = n > 0 || (c & kLgPrompt);
      if (!seen && !(c & kLgBias)) continue;   // drafted only later
      // the copy of the row's tokens from s0 - shift on is this CTA's; the
      // others' neighbour lists them too
      const long long r = r0 + i;
      const unsigned char* rowp = P.logits + r * P.V * ELT;
      if (static_cast<unsigned>(u - kLgPad + row_shift<ELT>(rowp)) >= static_cast<unsigned>(nv * N)) continue;
      if (P.mask && !mask_allows(P.mask + r * mask_words, t)) continue;
      float z = load_elem<ELT>(rowp, t);
      if (seen) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
      if (n > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, static_cast<float>(n))), pres);
      if (c & kLgBias) z = __fadd_rn(z, add);
      VT::store_rounded(P.out + (r * P.V + t) * ELT, 0, z);
    }
  }
}

int logits_smem(int n_tokens, bool table, bool with_bias) {
  return table ? (n_tokens + kLgPad) * (with_bias ? 10 : 6) : 0;
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

  const int n = elt == 2 ? 8 : 4;
  int lg = 7;   // slices of 128 vectors
  while (lg < 10 && static_cast<long long>(B) * ((V + (n << (lg + 1)) - 1) / (n << (lg + 1))) >= 1216) ++lg;
  p.lg_vecs = lg;
  p.n_slices = (V + n - 1 + (n << lg) - 1) / (n << lg);
  const long long ctas = static_cast<long long>(B) * p.n_slices;
  if (ctas > 0x7fffffffLL) return SV_ERR_INVALID_ARG;
  const int smem = logits_smem(n << lg, p.table, n_bias > 0);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_process_logits");
  auto launch = [&](auto kernel) {
    // up to 82 KB a CTA: above the 48 KB that need no asking
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024) != cudaSuccess)
      return SV_ERR_CUDA;
    kernel<<<static_cast<unsigned>(ctas), kLgThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  };
  return elt == 2 ? launch(logits_kernel<2>) : launch(logits_kernel<4>);
}
