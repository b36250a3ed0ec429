// What the operators over a row of logits and its token share: the row's sums,
// the numbers that follow from them, and the gradient in the logits.
//
// With x the row's token, p = softmax(z / T) and H the entropy of p, a loss of
// log p(x) and H with derivatives g and h has
//   d/dz(v) = (g (1[v = x] - p(v)) - h p(v) (log p(v) + H)) / T.
// The tokens but x are summed apart from it, about a base m:
//   s = sum 2^t, a = sum 2^t t, t = (z - m) c, c = log2(e) / T,
// so that 1 - p(x) is never formed by a subtraction: a policy is sure of most of
// its tokens, and there log p(x) = -log(1 + s') and the gradient at x is
// g s' / Z, with s' the others' sum on x's scale.  For the other tokens
//   d/dz(v) = 2^t (alpha + gamma t) : one exponential, and one multiply-add where
// the entropy counts.
#pragma once

#include "sv_rowvec.cuh"

namespace sv {
namespace {

// t below this is taken as this where it is a factor beside 2^t = 0 (0 times
// -inf would be NaN).
constexpr float kTokFloor = -16384.f;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// A vector's values less `m`, as pairs.  bf16 values are subtracted from as they
// are (mixed-precision sub of sm_100 and later: exact widening, one rounding), a
// value an instruction where widening first takes one and a half.
template <int ELT>
__device__ __forceinline__ void tok_minus(const uint4& w, float m, f2 (&d)[Vec<ELT>::N / 2]) {
  if constexpr (ELT == 2) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tsub.rn.f32.bf16 %0, l, %3;\n\tsub.rn.f32.bf16 %1, h, %3;\n\t}"
          : "=f"(a), "=f"(b) : "r"(ws[i]), "f"(m));
      d[i] = pack2(a, b);
    }
  } else {
    Vec<ELT>::pairs(w, d);
    const f2 mm = pack2(m, m);
#pragma unroll
    for (f2& x : d) x = sub2(x, mm);
  }
}

struct TokPart {
  float m, s, a;
};
__device__ __forceinline__ TokPart tok_none() { return TokPart{-INFINITY, 0.f, 0.f}; }

// A thread's sums over vectors of a row, about the maximum so far, or the token's
// own logit while that is above it.  t is rounded to 2^-24 of itself, so what counts
// for the sum must not lie far from the base: about the token's logit alone, which
// saves half an instruction a value and a branch, the log-probabilities' errors had
// a deviation of 6e-7.

template <int ELT, bool ENT>
struct TokSum {
  float m;                       // -inf: none yet
  f2 s2 = 0ull, s3 = 0ull, a2 = 0ull, a3 = 0ull;
  __device__ __forceinline__ explicit TokSum(float base) : m(base > -INFINITY && base < INFINITY ? base : -INFINITY) {}

  template <int U>
  __device__ __forceinline__ void add(const uint4 (&w)[U], float c2) {
    const float vm = Vec<ELT>::vmax(w);  // NaN is passed over here and kept by the sum
    if (vm > m) {
      const float d = m > -INFINITY ? __fmul_rn(__fsub_rn(m, vm), c2) : kTokFloor;
      const float f = fast_exp2(d);
      const f2 ff = pack2(f, f);
      if (ENT) {
        const float dk = fmaxf(d, kTokFloor);
        const f2 dd = pack2(dk, dk);
        a2 = mul2(ff, fma2(s2, dd, a2));
        a3 = mul2(ff, fma2(s3, dd, a3));
      }
      s2 = mul2(s2, ff);
      s3 = mul2(s3, ff);
      m = vm;
    }
    // these vectors' sums by themselves: long runs of additions to one sum lose digits
    f2 l2 = 0ull, l3 = 0ull, b2 = 0ull, b3 = 0ull;
    about(w, m > -INFINITY ? m : 0.f, c2, l2, l3, b2, b3);
    s2 = add2(s2, l2);
    s3 = add2(s3, l3);
    if (ENT) {
      a2 = add2(a2, b2);
      a3 = add2(a3, b3);
    }
  }
  template <int U>
  __device__ __forceinline__ static void about(const uint4 (&w)[U], float base, float c2, f2& l2, f2& l3, f2& b2, f2& b3) {
    const f2 cc = pack2(c2, c2);
#pragma unroll
    for (const uint4& x : w) {
      f2 z[Vec<ELT>::N / 2];
      tok_minus<ELT>(x, base, z);
#pragma unroll
      for (int i = 0; i < Vec<ELT>::N / 2; i += 2) {
        const f2 t0 = mul2(z[i], cc), t1 = mul2(z[i + 1], cc);
        const f2 e0 = exp2_2(t0), e1 = exp2_2(t1);
        l2 = add2(l2, e0);
        l3 = add2(l3, e1);
        if (ENT) {
          b2 = fma2(e0, floored(t0), b2);
          b3 = fma2(e1, floored(t1), b3);
        }
      }
    }
  }
  __device__ __forceinline__ static f2 floored(f2 t) {
    float a, b;
    unpack2(t, a, b);
    return pack2(fmaxf(a, kTokFloor), fmaxf(b, kTokFloor));
  }
  __device__ __forceinline__ TokPart part() const {
    TokPart p{m, 0.f, 0.f};
    float hi;
    unpack2(add2(s2, s3), p.s, hi);
    p.s += hi;
    if (ENT) {
      unpack2(add2(a2, a3), p.a, hi);
      p.a += hi;
    }
    return p;
  }
};

// 2^((z - m) c) for z <= m, the product's rounding carried along.
__device__ __forceinline__ float tok_scale(float z, float m, float c2) {
  const float d = __fsub_rn(z, m), t = __fmul_rn(d, c2);
  const float f = fast_exp2(t);
  return t > kTokFloor ? __fmaf_rn(f, __fmul_rn(__fmaf_rn(d, c2, -t), kLn2), f) : 0.f;
}

// The lanes' parts on their largest base, the same in every lane and in a
// fixed order; a NaN among the sums stays (with its base at -inf too).
template <bool ENT>
__device__ __forceinline__ TokPart tok_join(const TokPart& p, float c2) {
  TokPart r;
  r.m = from_ordered_key(__reduce_max_sync(0xffffffffu, ordered_key(p.m)));
  const float f = p.m > -INFINITY ? tok_scale(p.m, r.m, c2) : 1.f;
  r.s = warp_sum(p.s * f);
  r.a = ENT ? warp_sum(f > 0.f && p.m > -INFINITY ? f * __fmaf_rn(p.s, __fmul_rn(__fsub_rn(p.m, r.m), c2), p.a) : 0.f) : 0.f;
  return r;
}

// log(Z + Z_rest) as a float and what its rounding leaves, for Z >= 1 and Z_rest
// within Z's rounding.  Of Z = 2^k f, f in [3/4, 3/2), log f is at most 0.41 and off
// by a step of 2^-25 at most, and k log 2 is taken as two numbers, so a sum of many
// logarithms does not gather their roundings (2^-22 each where Z is some thousands).
// Near Z = 1 the logarithm keeps the digits of Z - 1, which Z_rest completes (what
// Z_rest's square would add is below 2e-15): a nearly sure token's -log p.
__device__ __forceinline__ float tok_log(float Z, float Z_rest, float rZ, float& rest) {
  constexpr float kLn2Rest = static_cast<float>(0.69314718055994530942 - static_cast<double>(kLn2));
  const int at = __float_as_int(Z) - 0x3f400000;      // 3/4's bits
  const float k = static_cast<float>(at >> 23);
  const float f = __int_as_float(__float_as_int(Z) - (at & static_cast<int>(0xff800000)));
  const float hi = __fmul_rn(k, kLn2), lo = __fmaf_rn(k, kLn2Rest, __fmaf_rn(k, kLn2, -hi));
  float y, e;
  two_sum(hi, logf(f), y, e);
  e = __fadd_rn(e, __fmaf_rn(Z_rest, rZ, lo));
  const float whole = __fadd_rn(y, e);
  rest = __fadd_rn(__fsub_rn(y, whole), e);
  return whole;
}

// 1 / T, and what its rounding left: a common factor of all that is divided by T,
// which a sum over tokens would gather.
struct TokTemp {
  float inv, inv_rest;
};

// (z - m) / T for z <= m and what its roundings left, also where z - m passes the
// range and the quotient does not.
__device__ __forceinline__ float tok_below(float z, float m, TokTemp T, float& rest) {
  const float inv_T = T.inv;
  float d, e;
  two_sum(z, -m, d, e);
  const float q = __fmul_rn(d, inv_T);
  rest = __fmaf_rn(d, T.inv_rest, __fmaf_rn(e, inv_T, __fmaf_rn(d, inv_T, -q)));
  if (!(fabsf(rest) < 1.f)) rest = 0.f;    // (far below anything that counts)
  if (d > -INFINITY || !(z > -INFINITY)) return q;
  return __fsub_rn(__fmul_rn(z, inv_T), __fmul_rn(m, inv_T));
}

struct TokRow {
  float M, Z, rZ;      // a base that is no less than the token's logit, the sum about it, and 1 / Z
  float rest, px;      // 1 - p(x), p(x)
  float logp, log_Z;
  float logp_rest;     // what logp's rounding left
  float U;             // sum p (z - M) / T
  bool valid;
  __device__ __forceinline__ float entropy() const { return __fsub_rn(log_Z, U); }
  __device__ __forceinline__ float lse(float inv_T) const { return valid ? __fmaf_rn(M, inv_T, log_Z) : NAN; }
};

template <bool ENT>
__device__ __forceinline__ TokRow tok_row(const TokPart& part, float zx, TokTemp T) {
  TokRow R;
  const bool top = zx >= part.m;           // the token's logit is the base
  R.M = top ? zx : part.m;
  R.valid = part.s == part.s && zx == zx && R.M > -INFINITY && R.M < INFINITY;
  const float low = top ? part.m : zx;
  float d_rest = 0.f;
  const float d = low > -INFINITY ? tok_below(low, R.M, T, d_rest) : -INFINITY;
  float e = expf(d);
  e = __fmaf_rn(e, d_rest, e);
  const float rest = top ? __fmul_rn(part.s, e) : part.s, ex = top ? 1.f : e;
  float Z_rest, log_rest = 0.f;
  two_sum(rest, ex, R.Z, Z_rest);
  R.rZ = __fdiv_rn(1.f, R.Z);
  R.log_Z = tok_log(R.Z, Z_rest, R.rZ, log_rest);
  R.rest = __fmul_rn(rest, R.rZ);
  R.px = __fmul_rn(ex, R.rZ);
  float lp, lp_rest = 0.f;
  if (top) {
    lp = __fsub_rn(0.f, R.log_Z);
    lp_rest = -log_rest;
  } else if (!(d > -INFINITY)) {
    lp = d;
  } else {
    two_sum(d, -R.log_Z, lp, lp_rest);
    lp_rest = __fadd_rn(lp_rest, __fsub_rn(d_rest, log_rest));
    const float whole = __fadd_rn(lp, lp_rest);
    lp_rest = __fadd_rn(__fsub_rn(lp, whole), lp_rest);
    lp = whole;
  }
  R.logp = R.valid ? lp : NAN;
  R.logp_rest = lp_rest;
  R.U = 0.f;
  if (ENT) {
    float u = 0.f;
    if (e > 0.f) u = top ? __fmul_rn(e, __fmaf_rn(part.a, kLn2, part.s * d)) : __fmul_rn(e, d);
    if (!top) u = __fmaf_rn(part.a, kLn2, u);
    R.U = R.valid ? __fmul_rn(u, R.rZ) : NAN;
  }
  return R;
}

// The gradient of a row: 2^t (alpha + gamma t) with t = (z - base) c + k, and
// at the token itself.
struct TokGrad {
  float base, k, alpha, gamma, at_token;
  __device__ __forceinline__ void none() { base = k = alpha = gamma = at_token = 0.f; }
  __device__ __forceinline__ bool zero() const { return alpha == 0.f && gamma == 0.f && at_token == 0.f; }
};

// A derivative past the range has no gradient: NaN for the whole row.
__device__ __forceinline__ void tok_check(TokGrad& G, bool valid) {
  if (valid && fabsf(G.alpha) < INFINITY && fabsf(G.gamma) < INFINITY && fabsf(G.at_token) < INFINITY) return;
  G.alpha = G.at_token = NAN;
}

template <bool ENT>
__device__ __forceinline__ TokGrad tok_grad(const TokRow& R, float g, float h, float inv_T) {
  const float q = __fmul_rn(inv_T, R.rZ);
  TokGrad G;
  G.base = R.M;
  G.k = 0.f;
  G.alpha = __fmul_rn(q, ENT ? __fmaf_rn(h, R.U, -g) : -g);
  G.gamma = 0.f;
  float own = 0.f;
  if (ENT) {
    G.gamma = -h * kLn2 * q;
    if (R.px > 0.f) own = h * R.px * __fadd_rn(R.logp, R.entropy());
  }
  G.at_token = __fmul_rn(inv_T, __fmaf_rn(g, R.rest, -own));
  tok_check(G, R.valid);
  return G;
}

// What a gradient of log p(x) takes of a row later, and what the rounding of log
// p(x) left: no value of it is rounded at the level of the logits.
__device__ __forceinline__ float4 tok_kept(const TokRow& R) {
  return make_float4(R.M, R.valid ? R.rZ : NAN, R.rest, R.logp_rest);
}
__device__ __forceinline__ TokGrad tok_grad_kept(const float4& row, float g, float inv_T) {
  TokGrad G;
  G.base = row.x;
  G.k = G.gamma = 0.f;
  G.alpha = -g * __fmul_rn(inv_T, row.y);
  G.at_token = __fmul_rn(inv_T, g * row.z);
  tok_check(G, row.y == row.y);
  return G;
}

// The same from what token_logp gave for the row.  p(v) = e^((z(v) - b) / T) with b
// = z(x) - T log p(x), whose difference from the logits that count keeps its digits
// at any level, or b = T lse where the token is far below them.  b is a float and
// what that leaves, which k takes: an exponent near 0 has no rounding but those of
// log p(x) or lse themselves.
__device__ __forceinline__ TokGrad tok_grad_from(float zx, float logp, float lse, float H, float g, float h, float T,
                                                 float inv_T, float c2) {
  TokGrad G;
  const bool near_token = logp > -32.f;
  const float from = near_token ? zx : 0.f, y = near_token ? -logp : lse;
  const float up = __fmul_rn(y, T);
  float rest;
  two_sum(from, up, G.base, rest);
  G.k = -__fmul_rn(__fadd_rn(rest, __fmaf_rn(y, T, -up)), c2);
  if (!(fabsf(G.base) < INFINITY)) {      // T times it passes the range
    G.base = from;
    G.k = -__fmul_rn(y, kLog2e);
  }
  G.alpha = __fmul_rn(inv_T, __fmaf_rn(-h, H, -g));
  G.gamma = -h * kLn2 * inv_T;
  const float px = expf(logp);
  const float own = px > 0.f ? h * px * __fadd_rn(logp, H) : 0.f;
  G.at_token = __fmul_rn(inv_T, __fmaf_rn(g, -expm1f(logp), -own));
  tok_check(G, logp == logp && lse == lse);
  return G;
}

// A vector's gradients, as if none of it were the row's token.
template <int ELT, bool ENT>
__device__ __forceinline__ uint4 tok_vec_grad(const uint4& w, const TokGrad& G, float c2) {
  using VT = Vec<ELT>;
  constexpr int N = VT::N;
  const f2 cc = pack2(c2, c2), kk = pack2(G.k, G.k);
  const f2 aa = pack2(G.alpha, G.alpha), gg = pack2(G.gamma, G.gamma);
  f2 z[N / 2];
  float d[N];
  tok_minus<ELT>(w, G.base, z);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const f2 t = fma2(z[i], cc, kk);
    const f2 f = ENT ? fma2(TokSum<ELT, ENT>::floored(t), gg, aa) : aa;
    unpack2(mul2(exp2_2(t), f), d[2 * i], d[2 * i + 1]);
  }
  return VT::pack(d);
}

// A vector without the token at place x_at (which may lie outside).
template <int ELT>
__device__ __forceinline__ void tok_take_out(uint4& w, int x_at) {
  if (static_cast<unsigned>(x_at) < static_cast<unsigned>(Vec<ELT>::N)) w = with_neg_inf<ELT>(w, 1u << x_at);
}

}  // namespace
}  // namespace sv
