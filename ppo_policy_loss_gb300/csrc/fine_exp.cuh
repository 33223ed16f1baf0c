// fine_exp.cuh — 2^x to 2^-41 in fp32 arithmetic, and sums of such terms that
// keep it, for the places where a sum over the vocabulary is compared with a
// random number: between two of 10^5 tokens' borders lie 10^-5 of the total,
// and a sum of fp32 terms, off by 10^-8, would give another token once in a
// thousand draws.  (sm_103a does one fp64 operation for 64 fp32 ones.)
//
// A term is an unevaluated sum a + b + c, each below 1 / 700 of the one before:
//   x = d c - kappa as a pair (the product's error by FMA, c as two floats);
//   x = n + j / 256 + g, g = gh + gl, |g| <= 1 / 512 + 2^-23;
//   2^(j/256) = T_j 2^(delta_j), T_j the nearest fp32 number, delta_j taken into gl;
//   2^g - 1 = u + v:  u = gh ln 2 rounded, v its error, gl ln 2 and the Taylor
//   polynomial's terms of degree 2 and 3 (the remainder is below 2^-42);
//   a = T_j 2^n,   b = a u rounded,   c = its error + a v.
// Everything is done for two numbers at a time (the packed fp32 instructions): an
// issue slot for two operations.  With 256 powers a term is 20 slots, and b so small that
// a difference of two b may be rounded; with 32 powers and scalars it was 45.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

namespace rl {
namespace {

constexpr int kPow = 256;  // powers in the table
// The bits of T_j = 2^(j/256), less j 2^15 (see FineExp::at), and of delta_j = j / 256 - log2 T_j.
__device__ const uint2 kPowers[kPow] = {
    {0x3f800000u, 0x00000000u}, {0x3f7fd8d8u, 0xb301f6f7u}, {0x3f7fb1edu, 0x33652774u}, {0x3f7f8b41u, 0xb386bd49u},
    {0x3f7f64d2u, 0xb20c09fbu}, {0x3f7f3ea1u, 0x33a032a6u}, {0x3f7f18afu, 0x333f7dfau}, {0x3f7ef2fcu, 0xb393a6abu},
    {0x3f7ecd87u, 0xb391e031u}, {0x3f7ea850u, 0x33a05659u}, {0x3f7e8359u, 0x335dad98u}, {0x3f7e5ea1u, 0x33803fccu},
    {0x3f7e3a29u, 0xb3287eefu}, {0x3f7e15f0u, 0xb355f73du}, {0x3f7df1f6u, 0x336f844eu}, {0x3f7dce3du, 0xb2d83ccbu},
    {0x3f7daac3u, 0x338f6665u}, {0x3f7d878au, 0x3301e4c2u}, {0x3f7d6491u, 0x337ba683u}, {0x3f7d41d9u, 0x328d6169u},
    {0x3f7d1f62u, 0xb39004abu}, {0x3f7cfd2bu, 0xb0304b57u}, {0x3f7cdb35u, 0x33adefaeu}, {0x3f7cb981u, 0x333fbe40u},
    {0x3f7c980fu, 0xb3ac4561u}, {0x3f7c76ddu, 0x33753b15u}, {0x3f7c55eeu, 0x31117b26u}, {0x3f7c3541u, 0xb36d2f99u},
    {0x3f7c14d5u, 0x339cdaeau}, {0x3f7bf4adu, 0xb38768b4u}, {0x3f7bd4c6u, 0x33380574u}, {0x3f7bb523u, 0xb37543acu},
    {0x3f7b95c2u, 0xb2949d5cu}, {0x3f7b76a4u, 0x330b01f8u}, {0x3f7b57cau, 0xb31cdd74u}, {0x3f7b3933u, 0xb3236d88u},
    {0x3f7b1adfu, 0x336f79fau}, {0x3f7afcd0u, 0xb32577b2u}, {0x3f7adf04u, 0x32a751ceu}, {0x3f7ac17du, 0xb36136f2u},
    {0x3f7aa43au, 0xb3971dc2u}, {0x3f7a873bu, 0xb1d62987u}, {0x3f7a6a81u, 0x3276353au}, {0x3f7a4e0cu, 0x32ad7cd8u},
    {0x3f7a31dcu, 0x332bd022u}, {0x3f7a15f2u, 0xb35727e8u}, {0x3f79fa4du, 0xb393d6fcu}, {0x3f79deedu, 0x32490c7du},
    {0x3f79c3d3u, 0x33928952u}, {0x3f79a900u, 0xb2b59b86u}, {0x3f798e72u, 0x339e3cd5u}, {0x3f79742cu, 0xb39595a6u},
    {0x3f795a2bu, 0x32ebfecfu}, {0x3f794072u, 0xb36da26du}, {0x3f7926ffu, 0x321c3d49u}, {0x3f790dd4u, 0xb34f75d5u},
    {0x3f78f4f0u, 0xb357b8bbu}, {0x3f78dc53u, 0x3306d89bu}, {0x3f78c3ffu, 0xb3956508u}, {0x3f78abf2u, 0xb3009252u},
    {0x3f78942du, 0x3307353bu}, {0x3f787cb1u, 0xb13eb171u}, {0x3f78657du, 0x33346241u}, {0x3f784e92u, 0x33510a8cu},
    {0x3f7837f0u, 0x3345dfe9u}, {0x3f782197u, 0x3386da22u}, {0x3f780b88u, 0xb28edaf9u}, {0x3f77f5c2u, 0xb2a72085u},
    {0x3f77e046u, 0xb382a804u}, {0x3f77cb13u, 0x3303f34au}, {0x3f77b62bu, 0xb1028d17u}, {0x3f77a18du, 0x325a97d9u},
    {0x3f778d3au, 0xb326993eu}, {0x3f777931u, 0x326c557eu}, {0x3f776573u, 0x33760705u}, {0x3f775201u, 0xb2abbd27u},
    {0x3f773edau, 0xb350a029u}, {0x3f772bfeu, 0xafb7676bu}, {0x3f77196eu, 0x326600b7u}, {0x3f77072au, 0x32b7bdc8u},
    {0x3f76f532u, 0x33605f62u}, {0x3f76e387u, 0xb183e4dfu}, {0x3f76d228u, 0x32accfdbu}, {0x3f76c116u, 0x327b1956u},
    {0x3f76b051u, 0x3210909bu}, {0x3f769fd9u, 0x3301071fu}, {0x3f768fafu, 0xb2f4822du}, {0x3f767fd2u, 0xb10c858bu},
    {0x3f767043u, 0x30ddc369u}, {0x3f766102u, 0x3240b014u}, {0x3f76520fu, 0x336d3baau}, {0x3f76436bu, 0x32ec2035u},
    {0x3f763516u, 0xb3385844u}, {0x3f76270fu, 0x31e1d029u}, {0x3f761958u, 0xb387a01cu}, {0x3f760befu, 0x333a208au},
    {0x3f75fed7u, 0xb3400757u}, {0x3f75f20eu, 0xb30c5d2du}, {0x3f75e595u, 0xb2d4bc77u}, {0x3f75d96cu, 0x32026513u},
    {0x3f75cd94u, 0xb325446eu}, {0x3f75c20cu, 0xb14d053du}, {0x3f75b6d5u, 0x3244da7bu}, {0x3f75abefu, 0x33100ab7u},
    {0x3f75a15bu, 0xb3237a50u}, {0x3f759718u, 0xb33fb6bdu}, {0x3f758d26u, 0x33339293u}, {0x3f758387u, 0xb21068acu},
    {0x3f757a3au, 0xb3201ca4u}, {0x3f75713fu, 0xb28d653au}, {0x3f756897u, 0xb3437d0bu}, {0x3f756041u, 0x3308a9fcu},
    {0x3f75583fu, 0xb2394687u}, {0x3f755090u, 0xb2939d1bu}, {0x3f754934u, 0x332f70b8u}, {0x3f75422du, 0xb3822f84u},
    {0x3f753b79u, 0xb32e1225u}, {0x3f753519u, 0x31682ea2u}, {0x3f752f0eu, 0xb2db35d6u}, {0x3f752957u, 0x32e39c3fu},
    {0x3f7523f6u, 0xb3838969u}, {0x3f751ee9u, 0xb24112f1u}, {0x3f751a32u, 0xb339ce38u}, {0x3f7515d0u, 0xb1a73992u},
    {0x3f7511c4u, 0x3219f2bau}, {0x3f750e0eu, 0x32e76df4u}, {0x3f750aafu, 0xb3400412u}, {0x3f7507a6u, 0xb36b5bdcu},
    {0x3f7504f3u, 0x32d4175eu}, {0x3f750298u, 0xb2b47248u}, {0x3f750094u, 0xb331d2bau}, {0x3f74fee7u, 0xb20c890eu},
    {0x3f74fd92u, 0xb268d5efu}, {0x3f74fc95u, 0xb2f66b2au}, {0x3f74fbf0u, 0xb2d697fau}, {0x3f74fba3u, 0x32debe04u},
    {0x3f74fbafu, 0x330e8719u}, {0x3f74fc14u, 0x32dc5fa4u}, {0x3f74fcd2u, 0x33095c3cu}, {0x3f74fdeau, 0xb320ebb4u},
    {0x3f74ff5bu, 0xb319e7dau}, {0x3f750126u, 0xb361d03bu}, {0x3f75034au, 0x3379606fu}, {0x3f7505cau, 0xb2e5b00cu},
    {0x3f7508a4u, 0xb33cd82fu}, {0x3f750bd8u, 0x331386b1u}, {0x3f750f68u, 0x31940d44u}, {0x3f751353u, 0x3239ee45u},
    {0x3f75179au, 0xb30e1902u}, {0x3f751c3cu, 0x328cebbfu}, {0x3f75213bu, 0xb334cf45u}, {0x3f752695u, 0x3353e690u},
    {0x3f752c4du, 0xb2ccf4d7u}, {0x3f753261u, 0xb19bc0ddu}, {0x3f7538d2u, 0x32bace05u}, {0x3f753fa1u, 0xb2fe3332u},
    {0x3f7546cdu, 0xb28f330eu}, {0x3f754e57u, 0xb2cd6714u}, {0x3f75563fu, 0xb2c26973u}, {0x3f755e85u, 0x32862cefu},
    {0x3f75672au, 0x3201b5b7u}, {0x3f75702eu, 0xb29a2877u}, {0x3f757991u, 0xb30a5384u}, {0x3f758353u, 0xb1e9a53cu},
    {0x3f758d75u, 0xb2ccce34u}, {0x3f7597f7u, 0xb369f17du}, {0x3f75a2d8u, 0x332a6376u}, {0x3f75ae1bu, 0xb3352958u},
    {0x3f75b9beu, 0xb35e937cu}, {0x3f75c5c1u, 0x3326225bu}, {0x3f75d226u, 0x332ba4efu}, {0x3f75deedu, 0xb2a0e592u},
    {0x3f75ec15u, 0xaff41909u}, {0x3f75f99fu, 0x32816306u}, {0x3f76078cu, 0xb35b333cu}, {0x3f7615dau, 0x333f8c9au},
    {0x3f76248cu, 0x321760eau}, {0x3f7633a1u, 0xb2bfa9b7u}, {0x3f764319u, 0xb2ae4806u}, {0x3f7652f4u, 0x33394340u},
    {0x3f766334u, 0xb283628bu}, {0x3f7673d7u, 0x333fb4dau}, {0x3f7684dfu, 0x332d4f6au}, {0x3f76964cu, 0x3076444cu},
    {0x3f76a81eu, 0xb340f500u}, {0x3f76ba54u, 0x33193b68u}, {0x3f76ccf1u, 0xb332b290u}, {0x3f76dff3u, 0xb32a5ccdu},
    {0x3f76f35bu, 0xb31202bdu}, {0x3f770729u, 0x3185cd8fu}, {0x3f771b5eu, 0xb017f78au}, {0x3f772ffau, 0xb29eaeb7u},
    {0x3f7744fdu, 0xb2b66a3eu}, {0x3f775a67u, 0x32a7feeau}, {0x3f777039u, 0x33026addu}, {0x3f778673u, 0x332b96efu},
    {0x3f779d16u, 0xb2d0d9b1u}, {0x3f77b421u, 0xb30b40e2u}, {0x3f77cb94u, 0x333ba6e7u}, {0x3f77e371u, 0x3305ed75u},
    {0x3f77fbb8u, 0xb32ed93fu}, {0x3f781468u, 0xb33978ffu}, {0x3f782d82u, 0xb34d5604u}, {0x3f784706u, 0xb2dfbb5fu},
    {0x3f7860f5u, 0xb350a709u}, {0x3f787b4eu, 0x325172f3u}, {0x3f789613u, 0xb25be0b3u}, {0x3f78b143u, 0x31847d93u},
    {0x3f78ccdfu, 0xb2025744u}, {0x3f78e8e7u, 0xb29dde47u}, {0x3f79055bu, 0xac1b4e5cu}, {0x3f79223cu, 0xb2b707b8u},
    {0x3f793f89u, 0x333a7c4du}, {0x3f795d44u, 0x32f741b0u}, {0x3f797b6du, 0xb31ad495u}, {0x3f799a03u, 0xb2dfe699u},
    {0x3f79b907u, 0xb21da4e9u}, {0x3f79d879u, 0x33390b2eu}, {0x3f79f85bu, 0xb30807a4u}, {0x3f7a18abu, 0xb26ce17fu},
    {0x3f7a396au, 0x32ff36a7u}, {0x3f7a5a99u, 0x330c0330u}, {0x3f7a7c38u, 0x32cbcf7fu}, {0x3f7a9e47u, 0x33083135u},
    {0x3f7ac0c7u, 0xb217e40eu}, {0x3f7ae3b7u, 0x32d2885fu}, {0x3f7b0719u, 0xb2e6a7f1u}, {0x3f7b2aecu, 0xb32ecfa7u},
    {0x3f7b4f30u, 0x32400cbbu}, {0x3f7b73e7u, 0xb2f2a989u}, {0x3f7b9910u, 0xb320e6a8u}, {0x3f7bbeabu, 0x324b016eu},
    {0x3f7be4bau, 0xb31a2accu}, {0x3f7c0b3bu, 0x33085677u}, {0x3f7c3231u, 0xb3073ee5u}, {0x3f7c599au, 0xb26ff5a0u},
    {0x3f7c8177u, 0x32b7d3e5u}, {0x3f7ca9c9u, 0x32560cceu}, {0x3f7cd290u, 0xb24c9fb7u}, {0x3f7cfbccu, 0xb2c61c7bu},
    {0x3f7d257du, 0x31fed2beu}, {0x3f7d4fa4u, 0x329bf546u}, {0x3f7d7a41u, 0x33228159u}, {0x3f7da555u, 0x31c870f2u},
    {0x3f7dd0dfu, 0x332b73bau}, {0x3f7dfce1u, 0xb21c6308u}, {0x3f7e295au, 0xb2cb7836u}, {0x3f7e564au, 0x32d1ae2bu},
    {0x3f7e83b3u, 0xb2579081u}, {0x3f7eb194u, 0xb29826b8u}, {0x3f7edfedu, 0x331fae17u}, {0x3f7f0ec0u, 0x31c86dfdu},
    {0x3f7f3e0cu, 0x319726b5u}, {0x3f7f6dd2u, 0xb2db5dc0u}, {0x3f7f9e11u, 0x33062615u}, {0x3f7fcecbu, 0x330134d5u}};

// x + y = the sum returned + err, exactly
__device__ __forceinline__ float two_sum(float x, float y, float& err) {
  const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);
  err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, t)), __fsub_rn(y, t));
  return s;
}

// A number of 48 bits as the sum of two floats, l at most half a last place of h.
struct Wide {
  float h, l;
  __device__ __forceinline__ Wide() {}
  __device__ __forceinline__ explicit Wide(float x) : h(x), l(0.f) {}
  // x + y, |x| >= |y|
  __device__ __forceinline__ Wide(float x, float y) {
    h = __fadd_rn(x, y);
    l = __fsub_rn(y, __fsub_rn(h, x));
  }
  __device__ __forceinline__ explicit operator float() const { return h; }
  __device__ __forceinline__ Wide operator-() const {
    Wide r;
    r.h = -h;
    r.l = -l;
    return r;
  }
};
__device__ __forceinline__ Wide operator+(const Wide& x, const Wide& y) {
  float e;
  const float s = two_sum(x.h, y.h, e);
  return Wide(s, __fadd_rn(e, __fadd_rn(x.l, y.l)));
}
__device__ __forceinline__ Wide operator-(const Wide& x, const Wide& y) { return x + (-y); }
__device__ __forceinline__ Wide& operator+=(Wide& x, const Wide& y) { return x = x + y; }
__device__ __forceinline__ Wide& operator-=(Wide& x, const Wide& y) { return x = x - y; }
__device__ __forceinline__ Wide operator*(const Wide& x, const Wide& y) {
  const float p = __fmul_rn(x.h, y.h);
  return Wide(p, __fadd_rn(fmaf(x.h, y.h, -p), fmaf(x.h, y.l, __fmul_rn(x.l, y.h))));
}
__device__ __forceinline__ bool operator>(const Wide& x, const Wide& y) { return x.h > y.h || (x.h == y.h && x.l > y.l); }
template <class N>
__device__ __forceinline__ N smaller(const N& x, const N& y) { return x > y ? y : x; }

// A warp's exchanges of plain and of wide numbers.
template <class N>
__device__ __forceinline__ N from_xor(const N& v, int o) {
  if constexpr (std::is_same<N, Wide>::value) {
    N r;
    r.h = __shfl_xor_sync(0xffffffffu, v.h, o);
    r.l = __shfl_xor_sync(0xffffffffu, v.l, o);
    return r;
  } else {
    return __shfl_xor_sync(0xffffffffu, v, o);
  }
}
template <class N>
__device__ __forceinline__ N from_below(const N& v, int o) {
  if constexpr (std::is_same<N, Wide>::value) {
    N r;
    r.h = __shfl_up_sync(0xffffffffu, v.h, o);
    r.l = __shfl_up_sync(0xffffffffu, v.l, o);
    return r;
  } else {
    return __shfl_up_sync(0xffffffffu, v, o);
  }
}
template <class N>
__device__ __forceinline__ N from_lane(const N& v, int src) {
  if constexpr (std::is_same<N, Wide>::value) {
    N r;
    r.h = __shfl_sync(0xffffffffu, v.h, src);
    r.l = __shfl_sync(0xffffffffu, v.l, src);
    return r;
  } else {
    return __shfl_sync(0xffffffffu, v, src);
  }
}

struct Term {
  float a, b, c;
  __device__ __forceinline__ Wide value() const {
    const Wide s(a, b);
    return Wide(s.h, __fadd_rn(s.l, c));
  }
};
struct Term2 {
  float2 a, b, c;
  __device__ __forceinline__ Term x() const { return Term{a.x, b.x, c.x}; }
  __device__ __forceinline__ Term y() const { return Term{a.y, b.y, c.y}; }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// Sums, differences and products of pairs, all as FMAs: the packed addition and product take
// twice as long to give their result, which counts where an SM has few warps.
__device__ __forceinline__ float2 add2(float2 x, float2 y) { return __ffma2_rn(x, both(1.f), y); }
__device__ __forceinline__ float2 sub2(float2 x, float2 y) { return __ffma2_rn(y, both(-1.f), x); }
__device__ __forceinline__ float2 mul2(float2 x, float2 y) { return __ffma2_rn(x, y, both(-0.f)); }

// the same for two numbers at a time
__device__ __forceinline__ float2 two_sum2(float2 x, float2 y, float2& err) {
  const float2 s = add2(x, y), t = sub2(s, x);
  err = add2(sub2(x, sub2(s, t)), sub2(y, t));
  return s;
}
// and for |x| >= |y|
__device__ __forceinline__ float2 quick_two_sum2(float2 x, float2 y, float2& err) {
  const float2 s = add2(x, y);
  err = sub2(y, sub2(s, x));
  return s;
}

// 2^((z - m) c - kappa), c = c_hi + c_lo.  z counts as at least zmin, so that what is
// below 2^-124 (and -inf) gives 2^-124, which no sum notices (is_zero() tells it from a
// weight), and as at most zmax, so that what is above 4 gives about 4.
// `far`: m is so large that zmin would be m itself; z - m is then formed first (exact
// where 2^((z - m) c) is not 0: z is within a factor of two of m).
struct FineExp {
  float c_hi, c_lo, kappa, off, m, zmin, zmax;

  // c: log2(e) / temperature, as two floats; unit: 1 / c.  The frame: the terms are 2^(z c - k),
  // kappa = k - m c.
  __device__ __forceinline__ void init(float c_hi_, float c_lo_, float unit, float m_, float kappa_, bool far) {
    c_hi = c_hi_;
    c_lo = c_lo_;
    off = far ? m_ : 0.f;
    m = far ? 0.f : m_;
    kappa = kappa_;
    zmin = fmaf(-124.f, unit, m);
    zmax = fmaf(2.f, unit, m);
  }
  // kWide: z has 24 significant bits (16-bit numbers have 8 or 11).  kTop: z may be above zmax.
  template <bool kWide, bool kTop>
  __device__ __forceinline__ Term2 at(float2 z, const uint2* powers) const {
    z = sub2(z, both(off));  // (a branch here would keep the pairs of a vector apart)
    z = make_float2(fmaxf(z.x, zmin), fmaxf(z.y, zmin));
    if (kTop) z = make_float2(fminf(z.x, zmax), fminf(z.y, zmax));
    // the difference and its error r; of 16-bit numbers that is 0 unless |z| is far below |m|
    float2 r, d;
    if (kWide)
      d = two_sum2(z, both(-m), r);
    else
      d = quick_two_sum2(both(-m), z, r);
    const float2 nx = mul2(d, both(-c_hi));
    float2 gl = __ffma2_rn(r, both(c_hi), both(-kappa));
    gl = add2(__ffma2_rn(d, both(c_hi), nx), __ffma2_rn(d, both(c_lo), gl));
    constexpr float kMagic = 49152.f;  // 1.5 2^15: its last place is 1 / 256, its bits from the 20th on only
    const float2 t = __ffma2_rn(d, both(c_hi), both(kMagic));
    const float2 gn = add2(nx, add2(t, both(-kMagic)));  // -gh
    const uint32_t t0 = __float_as_uint(t.x), t1 = __float_as_uint(t.y);
    const uint2 p0 = powers[t0 & (kPow - 1)], p1 = powers[t1 & (kPow - 1)];
    gl = add2(gl, make_float2(__uint_as_float(p0.y), __uint_as_float(p1.y)));
    const float2 g = sub2(gl, gn);
    constexpr float kLn2Hi = 0x1.62e430p-1f, kLn2Lo = -0x1.05c610p-29f;
    const float2 u = mul2(gn, both(-kLn2Hi));
    float2 v = __ffma2_rn(gn, both(-kLn2Hi), make_float2(-u.x, -u.y));
    v = __ffma2_rn(gn, both(-kLn2Lo), v);
    v = __ffma2_rn(gl, both(kLn2Hi), v);
    const float2 q = __ffma2_rn(g, both(0x1.c6b08ep-5f), both(0x1.ebfbe0p-3f));  // ln^3 2 / 6, ln^2 2 / 2
    v = __ffma2_rn(mul2(g, g), q, v);
    Term2 p;
    // the exponent n: t's bits are those of the magic number + 256 n + j
    p.a = make_float2(__uint_as_float(p0.x + (t0 << 15)), __uint_as_float(p1.x + (t1 << 15)));
    p.b = mul2(p.a, u);
    p.c = __ffma2_rn(p.a, v, __ffma2_rn(p.a, u, make_float2(-p.b.x, -p.b.y)));
    return p;
  }
  template <bool kWide, bool kTop>
  __device__ __forceinline__ Term at(float z, const uint2* powers) const {
    return at<kWide, kTop>(both(z), powers).x();
  }
  __device__ __forceinline__ bool is_zero(float z) const { return !(__fsub_rn(z, off) > zmin); }
};

// The differences of two terms, and 1 where they are positive, 0 elsewhere.  Of positive
// differences the first number is the larger one in a, or the two are so near that
// p.a - q.a is exact.
__device__ __forceinline__ Term2 above(const Term2& p, const Term2& q, float2& more) {
  float2 e;
  Term2 d;
  d.a = quick_two_sum2(p.a, make_float2(-q.a.x, -q.a.y), e);
  d.b = sub2(p.b, q.b);
  d.c = add2(e, sub2(p.c, q.c));
  const float2 s = add2(add2(d.a, d.b), d.c);
  more = make_float2(s.x > 0.f ? 1.f : 0.f, s.y > 0.f ? 1.f : 0.f);
  return d;
}

// A sum of such terms, none above 1: hi and mid start at 1, so that the error
// of each addition to them is exact (the larger one comes first), and lo, which
// is small, takes those and the c.
struct FineSum {
  float2 hi, mid, lo;
  __device__ __forceinline__ void clear() {
    hi = mid = both(1.f);
    lo = both(0.f);
  }
  __device__ __forceinline__ void add(const Term2& p) {
    float2 e, f;
    hi = quick_two_sum2(hi, p.a, e);
    mid = quick_two_sum2(mid, p.b, f);
    lo = add2(lo, add2(add2(e, f), p.c));
  }
  // the same times 1 or 0
  __device__ __forceinline__ void add(const Term2& p, float2 times) {
    const float2 h = __ffma2_rn(times, p.a, hi), m = __ffma2_rn(times, p.b, mid);
    const float2 e = __ffma2_rn(times, p.a, sub2(hi, h)), f = __ffma2_rn(times, p.b, sub2(mid, m));
    hi = h;
    mid = m;
    lo = add2(__ffma2_rn(times, p.c, lo), add2(e, f));
  }
  __device__ __forceinline__ Wide value() const {
    float e, f;
    const float s = two_sum(__fsub_rn(hi.x, 1.f), __fsub_rn(hi.y, 1.f), e);
    const float t = two_sum(__fsub_rn(mid.x, 1.f), __fsub_rn(mid.y, 1.f), f);
    float r;
    const float h = two_sum(s, t, r);
    return Wide(h, __fadd_rn(__fadd_rn(r, __fadd_rn(e, f)), __fadd_rn(lo.x, lo.y)));
  }
};

// log2 of a positive number, to 2^-38: the hardware's logarithm of its significand f, put right by
// what f 2^-log2(f) is above 1.
__device__ __forceinline__ Wide log2_wide(const Wide& s, const uint2* powers) {
  const int bits = __float_as_int(s.h), n = (bits >> 23) - 127;
  const float down = __int_as_float((127 - n) << 23);
  Wide f;
  f.h = __fmul_rn(s.h, down);
  f.l = __fmul_rn(s.l, down);
  const float y = __log2f(f.h);
  FineExp e;
  e.init(1.f, 0.f, 1.f, 0.f, 0.f, false);
  const Wide over = f * e.at<true, false>(-y, powers).value() - Wide(1.f);
  const float fix = __fmul_rn(over.h, fmaf(over.h, -0x1.715476p-1f, 0x1.715476p+0f));  // log2(e) (x - x^2 / 2)
  return Wide(static_cast<float>(n)) + Wide(y) + Wide(fix);
}

}  // namespace
}  // namespace rl
