// The norm of many gradients together, and their scaling to a largest norm,
// for sm_103a.
//
//   norm = sqrt(sum g^2) over every element of every tensor, or max |g|;
//   g <- g min(1, max_norm / (norm + 1e-6)).
//
// Bound by memory: one read for the norm, one more and a write for the scaling.
// Every tensor is cut into pieces of 32 KB at most on 16-byte boundaries of its
// memory, and piece b + i 608 of them all goes to CTA b (four an SM, fewer for few
// pieces), eight 16-byte loads a thread in flight.  The CTAs' sums go to `work` and every CTA of
// the second launch joins them again for itself, so there is no counter to reset
// and no order that changes.  The second launch takes the pieces backwards: the
// last ones are still in L2 then.
//
// 2.5 GB of bf16: the norm 349 us, 7.1 TB/s.  0.7 GB into scaled copies: 345 us, 6.1
// TB/s of two reads and a write.  2.5 GB in place, the norm exceeded: 1146 us, 6.6.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_rowvec.cuh"

namespace sv {
namespace {

constexpr int kClipThreads = 256, kClipWarps = kClipThreads / 32;
constexpr int kClipPerThread = 8;                             // vectors at most
constexpr int kClipGrid = SV_CLIP_WORK;    // CTAs, and their parts of the sum
constexpr int kClipFew = 64, kClipMany = 512;                 // tensors of a launch: its table is a kernel argument

// A sum of squares of 64 values in float32 outside these has lost or may lose
// some of them, and is taken again in 64 bits.  A thread joins the sums of all its
// pieces of a launch in float32: fewer than 2^21 of them (2^30 pieces over
// SV_CLIP_WORK CTAs), so below 2^117.
constexpr float kClipLow = 0x1p-100f, kClipHigh = 0x1p96f;
constexpr long long kClipMaxPieces = 1LL << 30;
static_assert(kClipMaxPieces / SV_CLIP_WORK < 1 << 21, "a thread's pieces");

template <int N>
struct ClipTable {
  const unsigned char* grad[N];
  unsigned char* out[N];
  long long size[N];
  int first[N + 1];                        // the tensor's first piece
  unsigned char wide[N];                   // bit 0: grad is float32, bit 1: out is
  int n;
  int kind;
  int per;                                 // a piece has this many vectors for each thread
};

struct ClipPart {
  double s;                                // of squares
  float hi, lo;                            // and what float32 sums came to, unrounded (a 64-bit addition a piece: 16 clocks of an SM)
  uint32_t top;                            // the largest |g| as bits: NaN is above infinity
};

__device__ __forceinline__ ClipPart clip_warp(ClipPart p) {
  p.s = warp_sum(p.s);
  p.top = __reduce_max_sync(0xffffffffu, p.top);
  return p;
}

// The parts of all threads, in a fixed order.
__device__ __forceinline__ ClipPart clip_block(ClipPart p) {
  __shared__ ClipPart parts[kClipWarps];
  p = clip_warp(p);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = p;
  __syncthreads();
  p = parts[0];
#pragma unroll
  for (int w = 1; w < kClipWarps; ++w) {
    p.s += parts[w].s;
    p.top = max(p.top, parts[w].top);
  }
  return p;
}

// A piece of a tensor: its vectors as sv_rowvec.cuh has them for a row.
template <int ELT>
struct ClipPieceOf {
  const unsigned char* grad;
  long long size, t0;                      // t0: the element where the piece begins, below 0 before the first
  int per;
  template <int N>
  __device__ __forceinline__ static ClipPieceOf of(const ClipTable<N>& T, int k, int piece) {
    ClipPieceOf p;
    p.grad = T.grad[k];
    p.size = T.size[k];
    p.per = T.per;
    p.t0 = static_cast<long long>(piece - T.first[k]) * (T.per * kClipThreads * Vec<ELT>::N) - row_shift<ELT>(p.grad);
    return p;
  }
  __device__ __forceinline__ bool whole() const { return t0 >= 0 && t0 + per * kClipThreads * Vec<ELT>::N <= size; }
  // this thread's vectors, zeros outside the tensor
  __device__ __forceinline__ void load(uint4 (&w)[kClipPerThread]) const {
    constexpr int N = Vec<ELT>::N;
    const long long t = t0 + threadIdx.x * N;
    if (whole()) {                         // they all go out at once
      const unsigned char* at = grad + t * ELT;
#pragma unroll
      for (int j = 0; j < kClipPerThread; ++j) w[j] = j < per ? load_vec16(at + j * kClipThreads * 16) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < kClipPerThread; ++j) w[j] = j < per ? load(t + j * kClipThreads * N) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ uint4 load(long long t) const {
    constexpr int N = Vec<ELT>::N;
    if (t >= 0 && t + N <= size) return load_vec16(grad + t * ELT);
    float f[N];
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = t + e >= 0 && t + e < size ? load_elem<ELT>(grad, t + e) : 0.f;
    return Vec<ELT>::pack(f);              // exact: the values are of the type
  }
};

// (a vector by value: by reference the thread's vectors went through memory, 575
// us where it is 350)
template <int ELT>
__device__ __noinline__ double clip_squares64(uint4 w) {
  float z[Vec<ELT>::N];
  Vec<ELT>::unpack(w, z);
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < Vec<ELT>::N; ++e) s = fma(static_cast<double>(z[e]), static_cast<double>(z[e]), s);
  return s;
}

template <int ELT, int N>
__device__ __forceinline__ void clip_add(const ClipTable<N>& T, int k, int piece, ClipPart& part) {
  using VT = Vec<ELT>;
  const ClipPieceOf<ELT> p = ClipPieceOf<ELT>::of(T, k, piece);
  uint4 w[kClipPerThread];
  p.load(w);
  if (T.kind == SV_NORM_L2) {
    f2 s0 = 0ull, s1 = 0ull;
#pragma unroll
    for (int j = 0; j < kClipPerThread; ++j) {
      f2 z[VT::N / 2];
      VT::pairs(w[j], z);
#pragma unroll
      for (int i = 0; i < VT::N / 2; i += 2) {
        s0 = fma2(z[i], z[i], s0);
        s1 = fma2(z[i + 1], z[i + 1], s1);
      }
    }
    float a, b;
    unpack2(add2(s0, s1), a, b);
    const float s = a + b;
    if (s >= kClipLow && s <= kClipHigh) {
      float e;
      two_sum(part.hi, s, part.hi, e);
      part.lo += e;
    } else {
#pragma unroll
      for (int j = 0; j < kClipPerThread; ++j)
        if (w[j].x | w[j].y | w[j].z | w[j].w) part.s += clip_squares64<ELT>(w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kClipPerThread; ++j) {
      const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ELT == 4) part.top = max(part.top, x[i] & 0x7fffffffu);
        else part.top = max(part.top, max((x[i] & 0x7fffu) << 16, x[i] & 0x7fff0000u));
      }
    }
  }
}

// The tensor of a piece.
template <int N>
__device__ __forceinline__ int clip_find(const ClipTable<N>& T, int piece) {
  int lo = 0, hi = T.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (T.first[mid] <= piece) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, 4) clip_norm_kernel(const __grid_constant__ ClipTable<N> T, double* work,
                                                                    int first) {
  grid_dependents_launch();
  ClipPart part{0.0, 0.f, 0.f, 0u};
  const int pieces = T.first[T.n];
  if (static_cast<int>(blockIdx.x) < pieces)
    for (int piece = blockIdx.x, k = clip_find(T, piece); piece < pieces; piece += gridDim.x) {
      while (piece >= T.first[k + 1]) ++k;
      if (T.wide[k] & 1) clip_add<4>(T, k, piece, part);
      else clip_add<2>(T, k, piece, part);
    }
  part.s += static_cast<double>(part.hi) + static_cast<double>(part.lo);
  part = clip_block(part);
  if (threadIdx.x == 0) {
    const double before = first ? 0.0 : work[blockIdx.x];
    const double top = static_cast<double>(__uint_as_float(part.top));
    work[blockIdx.x] = T.kind == SV_NORM_L2 ? before + part.s : top > before || top != top ? top : before;
  }
}

// The norm, the same in every CTA, and the factor that `max_norm` makes of it, which
// is rounded to float32 once: three roundings in turn would be common to all
// gradients.  By one thread (64-bit roots and divisions by all of them are
// microseconds); the others get it through shared memory.
struct ClipTotal {
  float norm, scale;
};
__device__ __forceinline__ ClipTotal clip_total(const double* work, int ctas, int kind, float max_norm) {
  __shared__ ClipTotal total;
  ClipPart part{0.0, 0.f, 0.f, 0u};
  for (int i = threadIdx.x; i < ctas; i += kClipThreads) {
    const double v = __ldcg(work + i);
    if (kind == SV_NORM_L2) part.s += v;
    else part.top = max(part.top, __float_as_uint(static_cast<float>(v)) & 0x7fffffffu);
  }
  part = clip_block(part);
  if (threadIdx.x == 0) {
    const double norm = kind == SV_NORM_L2 ? sqrt(part.s) : static_cast<double>(__uint_as_float(part.top));
    total.norm = static_cast<float>(norm);
    total.scale = 1.f;
    if (max_norm < INFINITY && total.norm < INFINITY)
      total.scale = fminf(static_cast<float>(static_cast<double>(max_norm) / (norm + 1e-6)), 1.f);
  }
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kClipThreads) clip_total_kernel(const double* work, int ctas, int kind, float* norm) {
  grid_dependency_wait();
  const ClipTotal total = clip_total(work, ctas, kind, INFINITY);
  if (threadIdx.x == 0) *norm = total.norm;
}

// Stores a vector as bfloat16 or as float32, whole.
template <int ELT, bool WIDE>
__device__ __forceinline__ void clip_store(unsigned char* at, const float (&z)[Vec<ELT>::N]) {
  if constexpr (!WIDE) {
    store_vec16(at, Vec<ELT>::pack(z));
  } else {
    if constexpr (ELT == 4) {
      store_vec16(at, Vec<4>::pack(z));
    } else {                               // a sector in one piece: two 16-byte stores a lane write each sector twice
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                   :: "l"(at), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7])
                   : "memory");
    }
  }
}

// A thread's vectors of a piece, scaled, to `out`; WIDE: that is float32.
template <int ELT, bool WIDE>
__device__ __forceinline__ void clip_write(const ClipPieceOf<ELT>& p, const uint4 (&w)[kClipPerThread], unsigned char* out,
                                           float scale) {
  constexpr int N = Vec<ELT>::N, OUT = WIDE ? 4 : 2, ALIGN = N * OUT;
  const long long t = p.t0 + threadIdx.x * N;
  unsigned char* at = out + t * OUT;
  const bool whole = p.whole() && reinterpret_cast<uintptr_t>(at) % ALIGN == 0;
#pragma unroll
  for (int j = 0; j < kClipPerThread; ++j, at += kClipThreads * N * OUT) {
    if (j >= p.per) break;
    float z[N];
    Vec<ELT>::unpack(w[j], z);
    // (a factor of 1 leaves denormals and infinities as they are)
    if (scale != 1.f) {
#pragma unroll
      for (int e = 0; e < N; ++e) z[e] = __fmul_rn(z[e], scale);
    }
    if (whole) {
      clip_store<ELT, WIDE>(at, z);
    } else {
      const long long tj = t + j * kClipThreads * N;
      if (tj >= 0 && tj + N <= p.size && reinterpret_cast<uintptr_t>(at) % ALIGN == 0) {
        clip_store<ELT, WIDE>(at, z);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (tj + e >= 0 && tj + e < p.size) Vec<OUT>::store_rounded(at, e, z[e]);
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void clip_fetch(const ClipTable<N>& T, int k, int piece, uint4 (&w)[kClipPerThread]) {
  if (T.wide[k] & 1) ClipPieceOf<4>::of(T, k, piece).load(w);
  else ClipPieceOf<2>::of(T, k, piece).load(w);
}

template <int N>
__device__ __forceinline__ void clip_scale(const ClipTable<N>& T, int k, int piece, const uint4 (&w)[kClipPerThread], float scale) {
  if (T.wide[k] & 1) clip_write<4, true>(ClipPieceOf<4>::of(T, k, piece), w, T.out[k], scale);
  else if (T.wide[k] & 2) clip_write<2, true>(ClipPieceOf<2>::of(T, k, piece), w, T.out[k], scale);
  else clip_write<2, false>(ClipPieceOf<2>::of(T, k, piece), w, T.out[k], scale);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, 4) clip_scale_kernel(const __grid_constant__ ClipTable<N> T, const double* work,
                                                                     float* norm, float max_norm, int in_place) {
  int piece = T.first[T.n] - 1 - static_cast<int>(blockIdx.x), k = 0;
  uint4 w[kClipPerThread];
  if (piece >= 0 && !in_place) {           // the gradients are there already: the first piece is on its way meanwhile
    k = clip_find(T, piece);
    clip_fetch(T, k, piece, w);
  }
  grid_dependency_wait();
  const ClipTotal total = clip_total(work, static_cast<int>(gridDim.x), T.kind, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total.norm;
  const float scale = total.scale;
  if (piece < 0 || (in_place && scale == 1.f)) return;
  if (in_place) {
    k = clip_find(T, piece);
    clip_fetch(T, k, piece, w);
  }
  while (true) {
    clip_scale(T, k, piece, w, scale);
    piece -= static_cast<int>(gridDim.x);
    if (piece < 0) break;
    while (piece < T.first[k]) --k;
    clip_fetch(T, k, piece, w);
  }
}

// What a call is about; its tensors go to the kernels in tables of N.
struct ClipCall {
  int n;
  const void* const* grads;
  const long long* sizes;
  const int* dtypes;
  int kind;
  float max_norm;
  void* const* outs;
  const int* out_dtypes;
  float* norm;
  double* work;
  cudaStream_t stream;
};

template <typename... Params, typename... Args>
cudaError_t clip_launch(void (*kernel)(Params...), int grid, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kClipThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

long long clip_pieces(const ClipCall& c, int i, int per) {
  const long long bytes = c.sizes[i] * (c.dtypes[i] == SV_F32 ? 4 : 2) +
                          static_cast<long long>(reinterpret_cast<uintptr_t>(c.grads[i]) % 16);
  const long long piece = static_cast<long long>(per) * kClipThreads * 16;
  return c.sizes[i] ? (bytes + piece - 1) / piece : 0;
}

// How many vectors of a piece each thread takes: what makes the CTA with the
// most pieces move the least, a piece's start counted as half a vector (48 MB of
// bf16, 3 pieces of 8 or 4 of 5: 12.2 and 11.8 us for the norm), and 64 CTAs as a
// vector (0.6 MB in five tensors: 6.4 us with a CTA a piece, 12.8 with 608).
int clip_per(const ClipCall& c, int first, int tensors) {
  int best = kClipPerThread;
  long long least = 0;
  for (int per = kClipPerThread; per >= 1; --per) {
    long long pieces = 0;
    for (int i = first; i < c.n && i < first + tensors; ++i) pieces += clip_pieces(c, i, per);
    const long long cost = (pieces + kClipGrid - 1) / kClipGrid * (2 * per + 1) + std::min<long long>(pieces, kClipGrid) / 32;
    if (per == kClipPerThread || cost < least) best = per, least = cost;
    if (pieces > 16LL * kClipGrid) break;     // nothing to win
  }
  return best;
}

template <int N>
cudaError_t clip_run_call(const ClipCall& c) {
  const bool scales = c.outs || c.max_norm < INFINITY;
  static thread_local ClipTable<N> t;
  int ctas = kClipGrid;
  for (int pass = 0; pass < (scales ? 2 : 1); ++pass)
    for (int first = 0; first < c.n || first == 0; first += N) {
      t.n = 0;
      t.kind = c.kind;
      t.per = clip_per(c, first, N);
      t.first[0] = 0;
      for (int i = first; i < c.n && i < first + N; ++i) {
        if (c.sizes[i] == 0) continue;
        const int k = t.n++, od = c.outs ? c.out_dtypes[i] : c.dtypes[i];
        t.grad[k] = static_cast<const unsigned char*>(c.grads[i]);
        t.out[k] = static_cast<unsigned char*>(c.outs ? c.outs[i] : const_cast<void*>(c.grads[i]));
        t.size[k] = c.sizes[i];
        t.wide[k] = static_cast<unsigned char>((c.dtypes[i] == SV_F32) | (od == SV_F32) << 1);
        t.first[k + 1] = t.first[k] + static_cast<int>(clip_pieces(c, i, t.per));
      }
      if (t.n == 0) {                        // the kernels look at one tensor at least
        t.n = 1;
        t.size[0] = 0;
        t.wide[0] = 0;
        t.first[1] = 0;
      }
      if (c.n <= N) ctas = std::max(1, std::min(kClipGrid, t.first[t.n]));
      cudaError_t e;
      if (pass == 0) {
        clip_norm_kernel<N><<<ctas, kClipThreads, 0, c.stream>>>(t, c.work, first == 0);
        e = cudaGetLastError();
      } else {
        e = clip_launch(clip_scale_kernel<N>, ctas, c.stream, t, static_cast<const double*>(c.work), c.norm,
                        c.max_norm, c.outs == nullptr ? 1 : 0);
      }
      if (e != cudaSuccess) return e;
    }
  if (scales) return cudaSuccess;
  return clip_launch(clip_total_kernel, 1, c.stream, static_cast<const double*>(c.work), ctas, c.kind, c.norm);
}

// Memory that a call reads or writes.
struct ClipRange {
  uintptr_t from, to;
  bool written;
};

// Whether anything written overlaps anything else.
bool clip_overlaps(ClipRange* r, int n) {
  std::sort(r, r + n, [](const ClipRange& a, const ClipRange& b) { return a.from < b.from; });
  uintptr_t end = 0, written_end = 0;      // of the ranges before this one
  for (int i = 0; i < n; ++i) {
    if (r[i].from < (r[i].written ? end : written_end)) return true;
    end = std::max(end, r[i].to);
    if (r[i].written) written_end = std::max(written_end, r[i].to);
  }
  return false;
}

}  // namespace
}  // namespace sv

extern "C" sv_status sv_clip_gradients(int n, const void* const* grads, const long long* sizes, const int* dtypes,
                                       int kind, float max_norm, void* const* outs, const int* out_dtypes, float* norm,
                                       double* work, sv_stream_t stream) {
  using namespace sv;
  if (n < 0 || (n > 0 && (!grads || !sizes || !dtypes)) || !norm || !work) return SV_ERR_INVALID_ARG;
  if (kind != SV_NORM_L2 && kind != SV_NORM_MAX) return SV_ERR_INVALID_ARG;
  if (!(max_norm > 0.f) || !outs != !out_dtypes) return SV_ERR_INVALID_ARG;
  const bool scales = outs || max_norm < INFINITY;
  long long pieces = 0;
  ClipRange* ranges = new (std::nothrow) ClipRange[2 * static_cast<size_t>(n) + 2];
  if (!ranges) return SV_ERR_CUDA;
  int used = 0;
  bool ok = true;
  auto range_of = [&](const void* p, long long size, int bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    ok = ok && at % bytes == 0;
    if (size > 0) ranges[used++] = ClipRange{at, at + static_cast<uintptr_t>(size) * bytes, written};
  };
  range_of(norm, 1, 4, true);
  range_of(work, SV_CLIP_WORK, 8, true);
  for (int i = 0; i < n && ok; ++i) {
    ok = sizes[i] >= 0 && sizes[i] < (1LL << 40) && (sizes[i] == 0 || grads[i]) &&
         (dtypes[i] == SV_F32 || dtypes[i] == SV_BF16);
    if (ok && outs)
      ok = (sizes[i] == 0 || outs[i]) && (out_dtypes[i] == SV_F32 || (out_dtypes[i] == SV_BF16 && dtypes[i] == SV_BF16));
    if (!ok) break;
    pieces += (sizes[i] * 4 + 16) / (kClipThreads * 16LL) + 1;
    const bool same = outs && outs[i] == grads[i] && out_dtypes[i] == dtypes[i];
    range_of(grads[i], sizes[i], dtypes[i] == SV_F32 ? 4 : 2, outs ? same : scales);
    if (outs && !same) range_of(outs[i], sizes[i], out_dtypes[i] == SV_F32 ? 4 : 2, true);
  }
  ok = ok && pieces < kClipMaxPieces && !clip_overlaps(ranges, used);
  delete[] ranges;
  if (!ok) return SV_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_clip_gradients");
  const ClipCall call{n, grads, sizes, dtypes, kind, max_norm, outs, out_dtypes, norm, work, s};
  const cudaError_t e = n <= kClipFew ? clip_run_call<kClipFew>(call) : clip_run_call<kClipMany>(call);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
