// The norm of many gradients together, and their scaling to a largest norm,
// for sm_103a.
//
//   norm = sqrt(sum g^2) over every element of every tensor, or max |g|;
//   g <- g min(1, max_norm / (norm + 1e-6)).

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/specverify.h"
#include "sv_internal.h"
#include "sv_device.cuh"

namespace sv {
namespace {

constexpr int kClipThreads = 512, kClipWarps = kClipThreads / 32;
constexpr int kClipTensors = 512;          // tensors of one launch
constexpr int kClipGrid = SV_CLIP_WORK;    // CTAs, and their parts of the sum

struct ClipTable {
  const void* grad[kClipTensors];
  void* out[kClipTensors];
  long long size[kClipTensors];
  unsigned char wide[kClipTensors];        // bit 0: grad is float32, bit 1: out is
  int n;
  int kind;
};

__device__ __forceinline__ float clip_load(const void* p, long long i, bool wide) {
  return wide ? static_cast<const float*>(p)[i]
              : __uint_as_float(static_cast<uint32_t>(static_cast<const unsigned short*>(p)[i]) << 16);
}

__device__ __forceinline__ double clip_join(double a, double b, int kind) {
  if (kind == SV_NORM_L2) return a + b;
  return a != a || b != b ? NAN : fmax(a, b);
}

__device__ __forceinline__ double clip_block(double v, int kind) {
  __shared__ double parts[kClipWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 16; o > 0; o >>= 1) v = clip_join(v, __shfl_xor_sync(0xffffffffu, v, o), kind);
  if (lane == 0) parts[warp] = v;
  __syncthreads();
  v = parts[0];
  for (int w = 1; w < kClipWarps; ++w) v = clip_join(v, parts[w], kind);
  return v;
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipTable T, double* work, int first) {
  double sum = 0.0;
  for (int k = 0; k < T.n; ++k)
    for (long long i = blockIdx.x * static_cast<long long>(kClipThreads) + threadIdx.x; i < T.size[k];
         i += static_cast<long long>(kClipGrid) * kClipThreads) {
      const double x = clip_load(T.grad[k], i, T.wide[k] & 1);
      sum = clip_join(sum, T.kind == SV_NORM_L2 ? x * x : fabs(x), T.kind);
    }
  sum = clip_block(sum, T.kind);
  if (threadIdx.x == 0) work[blockIdx.x] = first ? sum : clip_join(work[blockIdx.x], sum, T.kind);
}

__device__ __forceinline__ float clip_total(const double* work, int kind) {
  double v = 0.0;
  for (int i = threadIdx.x; i < kClipGrid; i += kClipThreads) v = clip_join(v, work[i], kind);
  v = clip_block(v, kind);
  return static_cast<float>(kind == SV_NORM_L2 ? sqrt(v) : v);
}

__global__ void __launch_bounds__(kClipThreads) clip_total_kernel(const double* work, int kind, float* norm) {
  const float v = clip_total(work, kind);
  if (threadIdx.x == 0) *norm = v;
}

__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipTable T, const float* norm,
                                                                  float max_norm, int in_place) {
  const float total = *norm;
  float scale = total < INFINITY ? fminf(__fdiv_rn(max_norm, __fadd_rn(total, 1e-6f)), 1.f) : 1.f;
  if (in_place && scale == 1.f) return;
  for (int k = 0; k < T.n; ++k)
    for (long long i = blockIdx.x * static_cast<long long>(kClipThreads) + threadIdx.x; i < T.size[k];
         i += static_cast<long long>(kClipGrid) * kClipThreads) {
      const float x = clip_load(T.grad[k], i, T.wide[k] & 1) * scale;
      if (T.wide[k] & 2) static_cast<float*>(T.out[k])[i] = x;
      else static_cast<__nv_bfloat16*>(T.out[k])[i] = __float2bfloat16_rn(x);
    }
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
  ClipRange* ranges = new (std::nothrow) ClipRange[2 * static_cast<size_t>(n) + 2];
  if (!ranges) return SV_ERR_INVALID_ARG;
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
    ok = sizes[i] >= 0 && sizes[i] < (1LL << 48) && (sizes[i] == 0 || grads[i]) &&
         (dtypes[i] == SV_F32 || dtypes[i] == SV_BF16);
    if (ok && outs)
      ok = (sizes[i] == 0 || outs[i]) && (out_dtypes[i] == SV_F32 || (out_dtypes[i] == SV_BF16 && dtypes[i] == SV_BF16));
    if (!ok) break;
    const bool same = outs && outs[i] == grads[i] && out_dtypes[i] == dtypes[i];
    range_of(grads[i], sizes[i], dtypes[i] == SV_F32 ? 4 : 2, outs ? same : scales);
    if (outs && !same) range_of(outs[i], sizes[i], out_dtypes[i] == SV_F32 ? 4 : 2, true);
  }
  ok = ok && !clip_overlaps(ranges, used);
  delete[] ranges;
  if (!ok) return SV_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NvtxRange range("sv_clip_gradients");
  ClipTable t;
  for (int pass = 0; pass < 2; ++pass) {
    for (int first = 0; first < n || first == 0; first += kClipTensors) {
      t.n = n - first < kClipTensors ? n - first : kClipTensors;
      t.kind = kind;
      for (int k = 0; k < t.n; ++k) {
        t.grad[k] = grads[first + k];
        t.out[k] = outs ? outs[first + k] : const_cast<void*>(grads[first + k]);
        t.size[k] = sizes[first + k];
        const int od = outs ? out_dtypes[first + k] : dtypes[first + k];
        t.wide[k] = static_cast<unsigned char>((dtypes[first + k] == SV_F32) | (od == SV_F32) << 1);
      }
      if (pass == 0) clip_norm_kernel<<<kClipGrid, kClipThreads, 0, s>>>(t, work, first == 0);
      else clip_scale_kernel<<<kClipGrid, kClipThreads, 0, s>>>(t, norm, max_norm, !outs);
    }
    if (pass == 0) clip_total_kernel<<<1, kClipThreads, 0, s>>>(work, kind, norm);
    if (!scales) break;
  }
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
