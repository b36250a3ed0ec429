// A row of logits as 16-byte vectors of global memory, whatever its first
// address: vector v of a row holds tokens N v - shift .. N v - shift + N - 1,
// shift being the distance of the row's first element from the 16-byte
// boundary before it.  So every vector of an odd vocabulary but a row's first
// and last is one aligned access, and those two go element by element.
#pragma once

#include "sv_device.cuh"

namespace sv {
namespace {

// Elements between p and the 16-byte boundary at or before it.
template <int ELT>
__device__ __forceinline__ int row_shift(const void* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / ELT);
}

template <int ELT>
__device__ __forceinline__ int row_vecs(int V, int shift) {
  constexpr int N = Vec<ELT>::N;
  return (V + shift + N - 1) / N;
}

__device__ __forceinline__ uint4 load_vec16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ void store_vec16(void* p, uint4 v) {
  asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};"
               :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Element t of a row, not through the read-only path (the row may be an
// output too): its bits, which are waited for only where their value is taken.
template <int ELT>
__device__ __forceinline__ uint32_t load_bits(const unsigned char* row, long long t) {
  if (ELT == 4) return *reinterpret_cast<const volatile uint32_t*>(row + t * 4);
  return *reinterpret_cast<const volatile unsigned short*>(row + t * 2);
}
template <int ELT>
__device__ __forceinline__ float value_of(uint32_t bits) {
  return __uint_as_float(ELT == 4 ? bits : bits << 16);
}
template <int ELT>
__device__ __forceinline__ float load_elem(const unsigned char* row, long long t) {
  return value_of<ELT>(load_bits<ELT>(row, t));
}

// Vector v of the row, -inf where it reaches past the row.
template <int ELT>
__device__ __forceinline__ uint4 load_row_vec(const unsigned char* row, int V, int shift, int v) {
  constexpr int N = Vec<ELT>::N;
  const int t0 = v * N - shift;
  if (t0 >= 0 && t0 <= V - N) return load_vec16(row + static_cast<long long>(t0) * ELT);
  float f[N];
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = (t0 + e >= 0 && t0 + e < V) ? load_elem<ELT>(row, t0 + e) : -INFINITY;
  return Vec<ELT>::pack(f);   // exact: the values are of the row's type
}

// A vector with -inf in the places of `bits`.
template <int ELT>
__device__ __noinline__ uint4 with_neg_inf(uint4 w, uint32_t bits) {
  constexpr int N = Vec<ELT>::N;
  float z[N];
  Vec<ELT>::unpack(w, z);
#pragma unroll
  for (int e = 0; e < N; ++e)
    if ((bits >> e) & 1u) z[e] = -INFINITY;
  return Vec<ELT>::pack(z);
}

// A vector's gradients where it may reach past its row, or the rows lie unlike.
template <int ELT>
__device__ __noinline__ void store_edge(unsigned char* grad, int V, int t0, int same_shift, uint4 g) {
  constexpr int N = Vec<ELT>::N;
  if (same_shift && t0 >= 0 && t0 <= V - N) {
    store_vec16(grad + static_cast<long long>(t0) * ELT, g);
    return;
  }
  float z[N];
  Vec<ELT>::unpack(g, z);
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (t0 + e >= 0 && t0 + e < V) Vec<ELT>::store_rounded(grad, t0 + e, z[e]);   // exact: of the type already
}

// N bits of a little-endian bit string from bit `at` on (at >= 0).  The word
// after the first is read only where the N bits reach into it.
template <int N, typename Word>
__device__ __forceinline__ uint32_t bits_at(const Word* words, int at) {
  const int o = at & 31;
  const uint32_t w0 = static_cast<uint32_t>(words[at >> 5]);
  const uint32_t w1 = o > 32 - N ? static_cast<uint32_t>(words[(at >> 5) + 1]) : 0u;
  return __funnelshift_r(w0, w1, o) & ((1u << N) - 1u);
}

}  // namespace
}  // namespace sv
