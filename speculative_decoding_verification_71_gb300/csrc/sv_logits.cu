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
// integer word per token, so the order of the atomics cannot show), marks
// what the table holds in a bitmap, and streams the slice of every row
// through registers: a vector whose bitmap and mask say that nothing happens
// to it is copied as it is (in place: neither read nor written), one that is
// masked altogether is written without being read.  Drafts are counted by
// comparison where the table marks a token as drafted, so all rows of the
// slice are independent work.

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

template <int ELT>
struct LogitsSlice {
  using VT = Vec<ELT>;

  const LogitsParams& P;
  const uint32_t* tab;       // [kLgPad + slice]
  const float* bias;         // [kLgPad + slice] or null
  const uint32_t* touched;   // bitmap over the same range
  const int* drafts;
  int s0;                    // first token of the slice
  float rep, pres, freq;

  // What happens to token t of row i; false if nothing does (a token drafted
  // only later).
  __device__ __forceinline__ bool rule(float& z, int t, int i) const {
    const int u = t - s0 + kLgPad;
    const uint32_t c = tab[u];
    int n = static_cast<int>(c & kLgCount);
    if (c & kLgDraft)
      for (int j = 0; j < i; ++j) n += drafts[j] == t;
    const bool seen = n > 0 || (c & kLgPrompt);
    if (seen) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
    if (n > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, static_cast<float>(n))), pres);
    if (c & kLgBias) z = __fadd_rn(z, bias[u]);
    return seen || (c & kLgBias);
  }
  __device__ __forceinline__ bool is_touched(int t) const {
    const int u = t - s0 + kLgPad;
    return P.table && ((touched[u >> 5] >> (u & 31)) & 1u);
  }
  // One element, for a row's ends and for rows that lie unlike.
  __device__ __forceinline__ void element(const unsigned char* in, unsigned char* out, const int* mask, int t,
                                          int i) const {
    unsigned char* o = out + static_cast<long long>(t) * ELT;
    if (mask && !((static_cast<uint32_t>(mask[t >> 5]) >> (t & 31)) & 1u)) {
      VT::store_rounded(o, 0, -INFINITY);
      return;
    }
    const bool hit = is_touched(t);
    if (!hit && in == out) return;
    float z = load_elem<ELT>(in, t);
    if (hit && rule(z, t, i)) VT::store_rounded(o, 0, z);
    else VT::store_scalar(o, 0, z);   // the very bits
  }
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

template <int ELT>
__global__ void __launch_bounds__(kLgThreads) logits_kernel(const LogitsParams P) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int drafts[kLgMaxDrafts];
  const int b = blockIdx.x / P.n_slices, slice = blockIdx.x % P.n_slices;
  const int nv = 1 << P.lg_vecs;
  const int span = nv * N + kLgPad;          // tokens the table covers
  const int s0 = slice * nv * N, first = s0 - kLgPad;
  const int tid = threadIdx.x;

  int rows = P.R;
  int n_drafts = 0;
  if (P.draft_len) {
    const int kb = P.draft_len[b];
    if (kb < 0 || kb > P.k) return;          // the verifier reports it
    rows = min(P.R, kb + (P.R - P.k));
    n_drafts = kb;
  } else {
    n_drafts = P.k;
  }
  if (!P.tokens) n_drafts = 0;

  uint32_t* tab = reinterpret_cast<uint32_t*>(smem);
  uint32_t* touched = tab + span;
  float* bias = P.n_bias ? reinterpret_cast<float*>(touched + (span + 31) / 32 + 1) : nullptr;
  if (P.table) {
    const int words = span + (span + 31) / 32 + 1 + (P.n_bias ? span : 0);
    for (int w = tid; w < words; w += kLgThreads) tab[w] = 0;
    if (tid < n_drafts) drafts[tid] = P.tokens[static_cast<long long>(b) * P.k + tid];
    __syncthreads();
    auto touch = [&](int u) { atomicOr(&touched[u >> 5], 1u << (u & 31)); };
    if (P.history) {
      const int* h = P.history + b * P.history_stride;
      const int len = min(P.history_len ? max(P.history_len[b], 0) : P.history_max, P.history_max);
      const int plen = P.prompt_len ? P.prompt_len[b] : 0;
#pragma unroll 8
      for (int j = tid; j < len; j += kLgThreads) {
        const int t = h[j];
        const int u = t - first;
        if (t >= 0 && t < P.V && static_cast<unsigned>(u) < static_cast<unsigned>(span)) {
          if (j < plen) atomicOr(&tab[u], kLgPrompt);
          else atomicAdd(&tab[u], 1u);
          touch(u);
        }
      }
    }
    if (tid < n_drafts) {
      const int t = drafts[tid], u = t - first;
      if (t >= 0 && t < P.V && static_cast<unsigned>(u) < static_cast<unsigned>(span)) {
        atomicOr(&tab[u], kLgDraft);
        touch(u);
      }
    }
    if (P.n_bias) {
      // the last entry of a token counts: the largest index + 1 wins the
      // token's word, which then takes the winner's value
      const int* ids = P.bias_ids + static_cast<long long>(b) * P.n_bias;
      const float* vals = P.bias_values + static_cast<long long>(b) * P.n_bias;
      int* slot = reinterpret_cast<int*>(bias);
      for (int j = tid; j < P.n_bias; j += kLgThreads) {
        const int t = ids[j], u = t - first;
        if (t >= 0 && t < P.V && static_cast<unsigned>(u) < static_cast<unsigned>(span)) {
          atomicMax(&slot[u], j + 1);
          touch(u);
        }
      }
      __syncthreads();
      for (int u = tid; u < span; u += kLgThreads) {
        const int j = slot[u];
        if (j) bias[u] = vals[j - 1], tab[u] |= kLgBias;
      }
    }
    __syncthreads();
  }

  LogitsSlice<ELT> S{P, tab, bias, touched, drafts, s0,
                     P.repetition ? P.repetition[b] : 1.f,
                     P.presence ? P.presence[b] : 0.f, P.frequency ? P.frequency[b] : 0.f};
  const bool in_place = P.logits == P.out;
  const int mask_words = (P.V + 31) / 32;
  const int items = rows << P.lg_vecs;
  for (int it = tid; it < items; it += kLgThreads * kLgUnroll) {
    uint4 w[kLgUnroll];
    uint32_t allowed[kLgUnroll], hit[kLgUnroll];
    int t0[kLgUnroll], row[kLgUnroll];
    bool whole[kLgUnroll];
#pragma unroll
    for (int q = 0; q < kLgUnroll; ++q) {
      const int item = it + q * kLgThreads;
      const bool in = item < items;
      row[q] = item >> P.lg_vecs;
      const long long r = static_cast<long long>(b) * P.R + row[q];
      const unsigned char* rowp = P.logits + r * P.V * ELT;
      t0[q] = in ? s0 - row_shift<ELT>(rowp) + (item & (nv - 1)) * N : P.V;
      whole[q] = in && P.same_shift && t0[q] >= 0 && t0[q] <= P.V - N;
      allowed[q] = (1u << N) - 1u;
      hit[q] = 0;
      if (whole[q]) {
        if (P.mask) allowed[q] = bits_at<N>(P.mask + r * mask_words, t0[q]);
        if (P.table) hit[q] = bits_at<N>(touched, t0[q] - first);
        if (allowed[q] && !(in_place && allowed[q] == (1u << N) - 1u && !hit[q]))
          w[q] = load_vec16(rowp + static_cast<long long>(t0[q]) * ELT);
      }
    }
#pragma unroll
    for (int q = 0; q < kLgUnroll; ++q) {
      const long long r = static_cast<long long>(b) * P.R + row[q];
      unsigned char* outp = P.out + r * P.V * ELT;
      if (whole[q]) {
        const bool plain = allowed[q] == (1u << N) - 1u && !hit[q];
        if (plain && in_place) continue;
        uint4 res = w[q];
        if (!allowed[q]) {
          res = VT::neg_inf();
        } else if (!plain) {
          if (hit[q] & allowed[q]) {
            float f[N];
            uint32_t done = 0;
            VT::unpack(w[q], f);
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (((hit[q] >> e) & 1u) && S.rule(f[e], t0[q] + e, row[q])) done |= 1u << e;
            res = select<ELT>(done, VT::pack(f), w[q]);
          }
          res = select<ELT>(allowed[q], res, VT::neg_inf());
        }
        store_vec16(outp + static_cast<long long>(t0[q]) * ELT, res);
      } else if (t0[q] < P.V) {
        const unsigned char* rowp = P.logits + r * P.V * ELT;
        const int* mask = P.mask ? P.mask + r * mask_words : nullptr;
        for (int e = 0; e < N; ++e)
          if (t0[q] + e >= 0 && t0[q] + e < P.V) S.element(rowp, outp, mask, t0[q] + e, row[q]);
      }
    }
  }
}

int logits_smem(int n_tokens, bool table, bool with_bias) {
  if (!table) return 0;
  const int span = n_tokens + kLgPad;
  return 4 * (span + (span + 31) / 32 + 1 + (with_bias ? span : 0));
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
    // up to 66 KB a CTA: above the 48 KB that need no asking
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024) != cudaSuccess)
      return SV_ERR_CUDA;
    kernel<<<static_cast<unsigned>(ctas), kLgThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  };
  return elt == 2 ? launch(logits_kernel<2>) : launch(logits_kernel<4>);
}
