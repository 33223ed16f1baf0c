// fine_exp.cuh — 2^x to 2^-36 in fp32 arithmetic, and sums of such terms that
// keep it, for the places where a sum over the vocabulary is compared with a
// random number: between two of 10^5 tokens' borders lie 10^-5 of the total,
// and a sum of fp32 terms, off by 10^-8, would give another token once in a
// thousand draws.  (sm_103a does one fp64 operation for 64 fp32 ones.)
//
// A term is an unevaluated sum a + b + c, each below 1 / 90 of the one before:
//   x = d c - kappa as a pair (the product's error by FMA, c as two floats);
//   x = n + j / 32 + g, g = gh + gl, |g| <= 1 / 64 + 2^-24;
//   2^(j/32) = T_j 2^(delta_j), T_j the nearest fp32 number, delta_j taken into gl;
//   2^g - 1 = u + v:  u = gh ln 2 rounded, v its error, gl ln 2 and the Taylor
//   polynomial's terms of degree 2 to 4 (the remainder is below 2^-39);
//   a = T_j 2^n,   b = a u rounded,   c = its error + a v.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rl {
namespace {

constexpr int kPow = 32;  // powers in the table
__device__ constexpr float kPowT[kPow] = {
    0x1.000000p+0f, 0x1.059b0ep+0f, 0x1.0b5586p+0f, 0x1.11301ep+0f, 0x1.172b84p+0f, 0x1.1d4874p+0f, 0x1.2387a6p+0f,
    0x1.29e9e0p+0f, 0x1.306fe0p+0f, 0x1.371a74p+0f, 0x1.3dea64p+0f, 0x1.44e086p+0f, 0x1.4bfdaep+0f, 0x1.5342b6p+0f,
    0x1.5ab07ep+0f, 0x1.6247ecp+0f, 0x1.6a09e6p+0f, 0x1.71f75ep+0f, 0x1.7a1148p+0f, 0x1.82589ap+0f, 0x1.8ace54p+0f,
    0x1.93737cp+0f, 0x1.9c4918p+0f, 0x1.a5503cp+0f, 0x1.ae89fap+0f, 0x1.b7f770p+0f, 0x1.c199bep+0f, 0x1.cb720ep+0f,
    0x1.d5818ep+0f, 0x1.dfc974p+0f, 0x1.ea4afap+0f, 0x1.f50766p+0f};
// delta_j = j / 32 - log2 T_j
__device__ constexpr float kPowD[kPow] = {
    0.f, -0x1.23c062p-24f, 0x1.1ecccap-24f, -0x1.588ac2p-24f, -0x1.293ab8p-26f, -0x1.2e3b84p-24f, 0x1.2512a4p-24f,
    -0x1.af7176p-25f, 0x1.8bbfd2p-25f, -0x1.4d327cp-25f, 0x1.c0bec4p-25f, 0x1.bb86d2p-30f, -0x1.800eaep-25f,
    -0x1.46f4a0p-25f, -0x1.728d0ep-27f, -0x1.0712d2p-24f, 0x1.a82ebcp-26f, 0x1.1d0e32p-25f, -0x1.79b05ep-25f,
    -0x1.99e9aep-26f, 0x1.036b6ep-27f, -0x1.bd26f8p-25f, 0x1.2ec1d4p-27f, -0x1.81ea00p-25f, -0x1.6cd47cp-26f,
    -0x1.5db27ep-25f, -0x1.04ae88p-27f, -0x1.3b49d2p-27f, -0x1.2fc81cp-27f, -0x1.345598p-25f, 0x1.fda57cp-28f,
    -0x1.af2102p-27f};

struct Term {
  float a, b, c;
  __device__ __forceinline__ double value() const {
    return static_cast<double>(a) + (static_cast<double>(b) + static_cast<double>(c));
  }
};

// x + y = the sum returned + err, exactly
__device__ __forceinline__ float two_sum(float x, float y, float& err) {
  const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);
  err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, t)), __fsub_rn(y, t));
  return s;
}
// the same for |x| >= |y|
__device__ __forceinline__ float quick_two_sum(float x, float y, float& err) {
  const float s = __fadd_rn(x, y);
  err = __fsub_rn(y, __fsub_rn(s, x));
  return s;
}

// 2^((z - m) c - kappa), c = c_hi + c_lo.  z - m counts as at least dmin, so that what is
// below 2^-124 (and -inf) gives 2^-124, which no sum notices (is_zero() tells it from a
// weight), and as at most dmax, so that what is above 4 gives about 4.
struct FineExp {
  float m, c_hi, c_lo, kappa, dmin, dmax;

  // c: log2(e) / temperature, as two floats.  The frame: the terms are 2^(z c - k), kappa = k - m c.
  __device__ __forceinline__ void init(float c_hi_, float c_lo_, float unit, float m_, float kappa_) {
    c_hi = c_hi_;
    c_lo = c_lo_;
    m = m_;
    kappa = kappa_;
    dmin = -124.f * unit;  // unit: 1 / c
    dmax = 2.f * unit;
  }
  // kWide: z has 24 significant bits (16-bit numbers have 8 or 11).  kTop: z - m may be above dmax.
  template <bool kWide, bool kTop>
  __device__ __forceinline__ Term at(float z, const float* T, const float* delta) const {
    // the difference and its error r; of 16-bit numbers that is 0 unless |z| is far below |m|
    float r, d;
    if (kWide)
      d = two_sum(z, -m, r);
    else
      d = quick_two_sum(-m, z, r);
    r = d > dmin ? r : 0.f;
    d = fmaxf(d, dmin);
    if (kTop) {
      r = d < dmax ? r : 0.f;
      d = fminf(d, dmax);
    }
    const float x = __fmul_rn(d, c_hi);
    float gl = fmaf(r, c_hi, -kappa);
    gl = __fadd_rn(fmaf(d, c_hi, -x), fmaf(d, c_lo, gl));
    constexpr float kMagic = 393216.f;  // 1.5 2^18: its last place is 1 / 32
    const float t = __fadd_rn(x, kMagic);
    const int jn = __float_as_int(t) - __float_as_int(kMagic);
    const int j = jn & (kPow - 1);
    const float gh = __fsub_rn(x, __fsub_rn(t, kMagic));
    gl = __fadd_rn(gl, delta[j]);
    const float g = __fadd_rn(gh, gl);
    constexpr float kLn2Hi = 0x1.62e430p-1f, kLn2Lo = -0x1.05c610p-29f;
    const float u = __fmul_rn(gh, kLn2Hi);
    float v = fmaf(gl, kLn2Hi, fmaf(gh, kLn2Lo, fmaf(gh, kLn2Hi, -u)));
    float q = fmaf(g, 0x1.3b2ab6p-7f, 0x1.c6b08ep-5f);  // ln^4 2 / 24, ln^3 2 / 6
    q = fmaf(g, q, 0x1.ebfbe0p-3f);                      // ln^2 2 / 2
    v = fmaf(__fmul_rn(g, g), q, v);
    Term p;
    p.a = __int_as_float(__float_as_int(T[j]) + ((jn >> 5) << 23));
    p.b = __fmul_rn(p.a, u);
    p.c = fmaf(p.a, v, fmaf(p.a, u, -p.b));
    return p;
  }
  __device__ __forceinline__ bool is_zero(float z) const { return !(__fsub_rn(z, m) > dmin); }
};

// The difference of two terms; its sign is that of a + b + c.
__device__ __forceinline__ Term minus(const Term& p, const Term& q) {
  float e, f;
  Term d;
  d.a = two_sum(p.a, -q.a, e);
  d.b = two_sum(p.b, -q.b, f);
  d.c = __fadd_rn(__fadd_rn(e, f), __fsub_rn(p.c, q.c));
  return d;
}

// A sum of such terms, none above 1: hi and mid start at 1, so that the error
// of each addition to them is exact (the larger one comes first), and lo, which
// is small, takes those and the c.
struct FineSum {
  float hi, mid, lo;
  __device__ __forceinline__ void clear() {
    hi = mid = 1.f;
    lo = 0.f;
  }
  __device__ __forceinline__ void add(const Term& p) {
    float e, f;
    hi = quick_two_sum(hi, p.a, e);
    mid = quick_two_sum(mid, p.b, f);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(e, f), p.c));
  }
  __device__ __forceinline__ double value() const {
    return (static_cast<double>(hi) - 1.0) + ((static_cast<double>(mid) - 1.0) + static_cast<double>(lo));
  }
};

}  // namespace
}  // namespace rl
