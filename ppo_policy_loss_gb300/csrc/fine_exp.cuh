// fine_exp.cuh — e^y to 2^-39 (2^-41 in a row's own frame) in fp32 arithmetic, and sums of such terms that
// keep it, for the places where a sum over the vocabulary is compared with a
// random number: between two of 10^5 tokens' borders lie 10^-5 of the total,
// and a sum of fp32 terms, off by 10^-8, would give another token once in a
// thousand draws.  (sm_103a does one fp64 operation for 64 fp32 ones.)
//
// A term is an unevaluated sum a + b + c, each below 1 / 700 of the one before:
//   y = (z - m) / T - kappa as a pair yh + yl (1 / T as two floats; T = 1 takes no product);
//   yh = k ln 2 / 256 + gh with k whole: ln 2 / 256 as C1 + C2 + C3, C1 and C2 of 9 bits each, so
//   that both subtractions are exact (k has 15 bits, what is left at most 18);
//   gl = yl - k C3 + delta_j,   k = 256 n + j;
//   2^(j/256) = T_j e^(delta_j), T_j the nearest fp32 number;
//   e^g - 1 = gh + v,  v = gl + g^2 / 2 + g^3 / 6 with g = gh + gl, |g| <= ln 2 / 512 (what is left out
//   of the series is below 2^-42);
//   a = T_j 2^n,   b = a gh rounded,   c = its error + a v.
// (The table-driven exponential of P. T. P. Tang, ACM TOMS 15, 1989, with a constant split as W. J. Cody and W. Waite
// do, and the error-free sums of T. J. Dekker and D. E. Knuth; the table and the constants follow from these lines.)
// Everything is done for two numbers at a time (the packed fp32 instructions, an issue slot for
// two operations): 16 packed operations a pair with T = 1, 20 otherwise.  With 256 powers b is so small
// that a difference of two b may be rounded.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

namespace rl {
namespace {

constexpr int kPow = 256;  // powers in the table
// The bits of T_j, the fp32 number nearest to 2^(j/256), less j 2^15 (see FineExp::at), and of
// delta_j = j ln 2 / 256 - ln T_j.
__device__ const uint2 kPowers[kPow] = {
    {0x3f800000u, 0x00000000u}, {0x3f7fd8d8u, 0xb2b42b5au}, {0x3f7fb1edu, 0x331ed669u}, {0x3f7f8b41u, 0xb33ac9d8u},
    {0x3f7f64d2u, 0xb1c222a1u}, {0x3f7f3ea1u, 0x335e14d4u}, {0x3f7f18afu, 0x3304bb72u}, {0x3f7ef2fcu, 0xb34cb015u},
    {0x3f7ecd87u, 0xb34a3a0bu}, {0x3f7ea850u, 0x335e4651u}, {0x3f7e8359u, 0x3319a7d2u}, {0x3f7e5ea1u, 0x3331ca89u},
    {0x3f7e3a29u, 0xb2e995b7u}, {0x3f7e15f0u, 0xb3144f4du}, {0x3f7df1f6u, 0x33260539u}, {0x3f7dce3du, 0xb295e268u},
    {0x3f7daac3u, 0x3346cb6au}, {0x3f7d878au, 0x32b4121cu}, {0x3f7d6491u, 0x332e6e48u}, {0x3f7d41d9u, 0x3243feb8u},
    {0x3f7d1f62u, 0xb347a6d3u}, {0x3f7cfd2bu, 0xaff46553u}, {0x3f7cdb35u, 0x33712079u}, {0x3f7cb981u, 0x3304e7ffu},
    {0x3f7c980fu, 0xb36ed17fu}, {0x3f7c76ddu, 0x3329fb25u}, {0x3f7c55eeu, 0x30c9adf8u}, {0x3f7c3541u, 0xb324679eu},
    {0x3f7c14d5u, 0x33597287u}, {0x3f7bf4adu, 0xb33bb77cu}, {0x3f7bd4c6u, 0x32ff1b92u}, {0x3f7bb523u, 0xb32a0119u},
    {0x3f7b95c2u, 0xb24e0611u}, {0x3f7b76a4u, 0x32c0b4a0u}, {0x3f7b57cau, 0xb2d9760cu}, {0x3f7b3933u, 0xb2e28f22u},
    {0x3f7b1adfu, 0x3325fe11u}, {0x3f7afcd0u, 0xb2e56302u}, {0x3f7adf04u, 0x3267f443u}, {0x3f7ac17du, 0xb31c1b5du},
    {0x3f7aa43au, 0xb3517ddau}, {0x3f7a873bu, 0xb1947229u}, {0x3f7a6a81u, 0x322aa888u}, {0x3f7a4e0cu, 0x32708146u},
    {0x3f7a31dcu, 0x32ee2ef5u}, {0x3f7a15f2u, 0xb315227bu}, {0x3f79fa4du, 0xb34cf30fu}, {0x3f79deedu, 0x320b5b3du},
    {0x3f79c3d3u, 0x334b2481u}, {0x3f79a900u, 0xb27bc2efu}, {0x3f798e72u, 0x335b5d2bu}, {0x3f79742cu, 0xb34f5e44u},
    {0x3f795a2bu, 0x32a3945bu}, {0x3f794072u, 0xb324b736u}, {0x3f7926ffu, 0x31d89803u}, {0x3f790dd4u, 0xb30fcceeu},
    {0x3f78f4f0u, 0xb31586deu}, {0x3f78dc53u, 0x32baefb8u}, {0x3f78c3ffu, 0xb34f1adfu}, {0x3f78abf2u, 0xb2b23cf0u},
    {0x3f78942du, 0x32bb7020u}, {0x3f787cb1u, 0xb1042dacu}, {0x3f78657du, 0x32fa10a7u}, {0x3f784e92u, 0x3310e575u},
    {0x3f7837f0u, 0x33092801u}, {0x3f782197u, 0x333af1d7u}, {0x3f780b88u, 0xb2460a22u}, {0x3f77f5c2u, 0xb267aff1u},
    {0x3f77e046u, 0xb33520ccu}, {0x3f77cb13u, 0x32b6ec0au}, {0x3f77b62bu, 0xb0b4fb78u}, {0x3f77a18du, 0x32178469u},
    {0x3f778d3au, 0xb2e6f467u}, {0x3f777931u, 0x3223d070u}, {0x3f776573u, 0x332a8881u}, {0x3f775201u, 0xb26e14a5u},
    {0x3f773edau, 0xb3109bb7u}, {0x3f772bfeu, 0xaf7e407cu}, {0x3f77196eu, 0x321f6d01u}, {0x3f77072au, 0x327eb836u},
    {0x3f76f532u, 0x331b85f2u}, {0x3f76e387u, 0xb136d80cu}, {0x3f76d228u, 0x326f9177u}, {0x3f76c116u, 0x322e0c6du},
    {0x3f76b051u, 0x31c868d2u}, {0x3f769fd9u, 0x32b2dedbu}, {0x3f768fafu, 0xb2a97afau}, {0x3f767fd2u, 0xb0c2cdebu},
    {0x3f767043u, 0x3099b6f1u}, {0x3f766102u, 0x32058f9eu}, {0x3f76520fu, 0x33246ffbu}, {0x3f76436bu, 0x32a3ab81u},
    {0x3f763516u, 0xb2ff8e5fu}, {0x3f76270fu, 0x319c8590u}, {0x3f761958u, 0xb33c044bu}, {0x3f760befu, 0x33010373u},
    {0x3f75fed7u, 0xb3051aa9u}, {0x3f75f20eu, 0xb2c295f6u}, {0x3f75e595u, 0xb293751eu}, {0x3f75d96cu, 0x31b4c3ffu},
    {0x3f75cd94u, 0xb2e51bf0u}, {0x3f75c20cu, 0xb10e1bffu}, {0x3f75b6d5u, 0x320872cbu}, {0x3f75abefu, 0x32c7af35u},
    {0x3f75a15bu, 0xb2e2a0dbu}, {0x3f759718u, 0xb304e2cau}, {0x3f758d26u, 0x32f8f0c0u}, {0x3f758387u, 0xb1c83175u},
    {0x3f757a3au, 0xb2ddf652u}, {0x3f75713fu, 0xb2440403u}, {0x3f756897u, 0xb3078095u}, {0x3f756041u, 0x32bd74e0u},
    {0x3f75583fu, 0xb2006c56u}, {0x3f755090u, 0xb24ca2d3u}, {0x3f754934u, 0x32f33640u}, {0x3f75422du, 0xb33479bfu},
    {0x3f753b79u, 0xb2f15040u}, {0x3f753519u, 0x3120efb9u}, {0x3f752f0eu, 0xb297f1ebu}, {0x3f752957u, 0x329dc479u},
    {0x3f7523f6u, 0xb3365942u}, {0x3f751ee9u, 0xb205d425u}, {0x3f751a32u, 0xb300ca64u}, {0x3f7515d0u, 0xb167d2abu},
    {0x3f7511c4u, 0x31d56adfu}, {0x3f750e0eu, 0x32a06a2au}, {0x3f750aafu, 0xb3051864u}, {0x3f7507a6u, 0xb3232368u},
    {0x3f7504f3u, 0x329302aeu}, {0x3f750298u, 0xb27a26e0u}, {0x3f750094u, 0xb2f683e6u}, {0x3f74fee7u, 0xb1c2d2c9u},
    {0x3f74fd92u, 0xb22163afu}, {0x3f74fc95u, 0xb2aacdeau}, {0x3f74fbf0u, 0xb294beb8u}, {0x3f74fba3u, 0x329a64a7u},
    {0x3f74fbafu, 0x32c595dcu}, {0x3f74fc14u, 0x3298c058u}, {0x3f74fcd2u, 0x32be6bfbu}, {0x3f74fdeau, 0xb2df155fu},
    {0x3f74ff5bu, 0xb2d55bcbu}, {0x3f750126u, 0xb31c859cu}, {0x3f75034au, 0x332cdad1u}, {0x3f7505cau, 0xb29f3516u},
    {0x3f7508a4u, 0xb302e5a2u}, {0x3f750bd8u, 0x32cc83c1u}, {0x3f750f68u, 0x314d3e50u}, {0x3f751353u, 0x3200e09bu},
    {0x3f75179au, 0xb2c4fd3du}, {0x3f751c3cu, 0x32435b9bu}, {0x3f75213bu, 0xb2faa7c8u}, {0x3f752695u, 0x3312e0dau},
    {0x3f752c4du, 0xb28e10a1u}, {0x3f753261u, 0xb157eb87u}, {0x3f7538d2u, 0x32817bb3u}, {0x3f753fa1u, 0xb2b032b0u},
    {0x3f7546cdu, 0xb246843eu}, {0x3f754e57u, 0xb28e5fd0u}, {0x3f75563fu, 0xb286c18du}, {0x3f755e85u, 0x323a01bcu},
    {0x3f75672au, 0x31b3d0e5u}, {0x3f75702eu, 0xb255b55du}, {0x3f757991u, 0xb2bfc2c9u}, {0x3f758353u, 0xb1a1f360u},
    {0x3f758d75u, 0xb28df5d9u}, {0x3f7597f7u, 0xb322283bu}, {0x3f75a2d8u, 0x32ec356au}, {0x3f75ae1bu, 0xb2fb24a7u},
    {0x3f75b9beu, 0xb31a472bu}, {0x3f75c5c1u, 0x32e64f97u}, {0x3f75d226u, 0x32edf312u}, {0x3f75deedu, 0xb25f0cdfu},
    {0x3f75ec15u, 0xafa93219u}, {0x3f75f99fu, 0x32335e43u}, {0x3f76078cu, 0xb317f01eu}, {0x3f7615dau, 0x3304c595u},
    {0x3f76248cu, 0x31d1daf2u}, {0x3f7633a1u, 0xb284d9c3u}, {0x3f764319u, 0xb2719af1u}, {0x3f7652f4u, 0x33006a11u},
    {0x3f766334u, 0xb2362361u}, {0x3f7673d7u, 0x3304e17bu}, {0x3f7684dfu, 0x32f0424bu}, {0x3f76964cu, 0x302ab2fau},
    {0x3f76a81eu, 0xb305bf64u}, {0x3f76ba54u, 0x32d46cbcu}, {0x3f76ccf1u, 0xb2f7ba34u}, {0x3f76dff3u, 0xb2ec2c2eu},
    {0x3f76f35bu, 0xb2ca69efu}, {0x3f770729u, 0x31397d83u}, {0x3f771b5eu, 0xafd2abc1u}, {0x3f772ffau, 0xb25bfb0au},
    {0x3f7744fdu, 0xb27ce183u}, {0x3f775a67u, 0x3268e43eu}, {0x3f777039u, 0x32b4cc06u}, {0x3f778673u, 0x32eddfaau},
    {0x3f779d16u, 0xb290c398u}, {0x3f77b421u, 0xb2c10bd8u}, {0x3f77cb94u, 0x33021207u}, {0x3f77e371u, 0x32b9a9bcu},
    {0x3f77fbb8u, 0xb2f26443u}, {0x3f781468u, 0xb3008f51u}, {0x3f782d82u, 0xb30e53fcu}, {0x3f784706u, 0xb29b1443u},
    {0x3f7860f5u, 0xb310a07bu}, {0x3f787b4eu, 0x32112dd3u}, {0x3f789613u, 0xb218685au}, {0x3f78b143u, 0x3137abbeu},
    {0x3f78ccdfu, 0xb1b4b0dau}, {0x3f78e8e7u, 0xb25ada15u}, {0x3f79055bu, 0xabd74ccau}, {0x3f79223cu, 0xb27dbbd2u},
    {0x3f793f89u, 0x3301430eu}, {0x3f795d44u, 0x32ab629du}, {0x3f797b6du, 0xb2d6a3f8u}, {0x3f799a03u, 0xb29b323au},
    {0x3f79b907u, 0xb1da8a8fu}, {0x3f79d879u, 0x33004333u}, {0x3f79f85bu, 0xb2bc93d2u}, {0x3f7a18abu, 0xb224317cu},
    {0x3f7a396au, 0x32b0e688u}, {0x3f7a5a99u, 0x32c21936u}, {0x3f7a7c38u, 0x328d454cu}, {0x3f7a9e47u, 0x32bccd70u},
    {0x3f7ac0c7u, 0xb1d290beu}, {0x3f7ae3b7u, 0x3291ee1eu}, {0x3f7b0719u, 0xb29fe0eau}, {0x3f7b2aecu, 0xb2f256f7u},
    {0x3f7b4f30u, 0x32051e65u}, {0x3f7b73e7u, 0xb2a8335eu}, {0x3f7b9910u, 0xb2df0e5fu}, {0x3f7bbeabu, 0x320cb677u},
    {0x3f7be4bau, 0xb2d5b899u}, {0x3f7c0b3bu, 0x32bd0118u}, {0x3f7c3231u, 0xb2bb7d86u}, {0x3f7c599au, 0xb22653c5u},
    {0x3f7c8177u, 0x327ed6deu}, {0x3f7ca9c9u, 0x32145e40u}, {0x3f7cd290u, 0xb20dd5a0u}, {0x3f7cfbccu, 0xb28951fcu},
    {0x3f7d257du, 0x31b0a147u}, {0x3f7d4fa4u, 0x3258342fu}, {0x3f7d7a41u, 0x32e147b7u}, {0x3f7da555u, 0x318aef6cu},
    {0x3f7dd0dfu, 0x32edaedbu}, {0x3f7dfce1u, 0xb1d8cc57u}, {0x3f7e295au, 0xb28d08ccu}, {0x3f7e564au, 0x329156dfu},
    {0x3f7e83b3u, 0xb2156afcu}, {0x3f7eb194u, 0xb252ed29u}, {0x3f7edfedu, 0x32dd5d11u}, {0x3f7f0ec0u, 0x318aed60u},
    {0x3f7f3e0cu, 0x31518a42u}, {0x3f7f6dd2u, 0xb2980d96u}, {0x3f7f9e11u, 0x32b9f83cu}, {0x3f7fcecbu, 0x32b31e3au}};

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

constexpr float kFar = 0x1p20f;       // |m| / (T ln 2) beyond which m - 86 T is near m's own last place

// lse - ln_s - off / T as y / T + kappa, y a multiple of `step`.  (Next to a float so large that 100 is nothing, terms are 0
// or too large anyway.  Out of line: with it in the kernel 228 refused drafts took 164 us in place of 161.)
__device__ __noinline__ float2 beyond(float off, float T, double inv_t, float lse, float ln_h, float ln_l, float step) {
  double left = fma(-static_cast<double>(off), inv_t, static_cast<double>(lse)) - (static_cast<double>(ln_h) + static_cast<double>(ln_l));
  left = fmin(fmax(left, -100.0), 100.0);
  const float y = rintf(static_cast<float>(left) * T / step) * step;
  return make_float2(y, static_cast<float>(fma(-static_cast<double>(y), inv_t, left)));
}

// e^((z - m) / T - kappa).  z counts as at least zmin, so that what is
// below e^-86 (and -inf) gives e^-86, which no sum notices (is_zero() tells it from a
// weight), or another `low`, and as at most zmax, so that what is above 4 gives about 4.
// `far`: m is so large that zmin would be m itself; z - m is then formed first (exact
// where e^((z - m) / T) is not 0: z is within a factor of two of m).
struct FineExp {
  float r_hi, r_lo, kappa, off, m, zmin, zmax;

  // 1 / T as two floats; the frame: a number of the row's type, where the terms are 1.
  __device__ __forceinline__ void init(float r_hi_, float r_lo_, float T, float m_, bool far, float kappa_ = 0.f, float low = -86.f) {
    r_hi = r_hi_;
    r_lo = r_lo_;
    off = far ? m_ : 0.f;
    m = far ? 0.f : m_;
    kappa = kappa_;
    zmin = fmaf(low, T, m);
    zmax = fmaf(1.4f, T, m);
  }
  // e^(z / T - lse + ln_s).  m is the multiple of 2^-16 of T's power of two next to (lse - ln_s) T, so
  // that z - m is exact or has a float as its error, and |kappa| <= 2^-17: what is added to kappa in at()
  // is off by 2^-41 a step, 2^-39 in all.  (A coarser m leaves more in kappa, and a term good to 2^-23 kappa and to its
  // fourth power: steps of 2^-12 at every temperature gave 2^-35 at T = 1 and 2^-28 at 0.01.)  Where a float has no such digits,
  // from 2^8 T on, the nearest one is `off` and m what it leaves; z - off is exact where e^(z / T - lse) is above
  // e^-60, and the error that of the subtraction of off / T, |lse| 2^-52, where that is more.
  __device__ __forceinline__ void init_around(float r_hi_, float r_lo_, float T, double inv_t, float lse, const Wide& ln_s, float low) {
    const Wide k = Wide(lse) - ln_s;
    const int step_bits = (__float_as_int(T) & 0x7f800000) - (16 << 23);
    const float step = __int_as_float(step_bits), per_step = __int_as_float((254 << 23) - step_bits);
    float2 at = make_float2(k.h * T, 0.f);
    float far_off = 0.f;
    if (fabsf(at.x) < 0x1p24f * step) {
      at.x = rintf(at.x * per_step) * step;
      Wide r;
      r.h = r_hi_;
      r.l = r_lo_;
      at.y = (k - Wide(at.x) * r).h;
    } else {
      far_off = fminf(fmaxf(at.x, -0x1.fffffep127f), 0x1.fffffep127f);
      at = beyond(far_off, T, inv_t, lse, ln_s.h, ln_s.l, step);
    }
    init(r_hi_, r_lo_, T, at.x, false, at.y, low);
    off = far_off;
  }
  // kWide: z has 24 significant bits (16-bit numbers have 8 or 11).  kTop: z may be above zmax.  kUnit: T = 1.
  template <bool kWide, bool kTop, bool kUnit>
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
    float2 y, yl;
    if (kUnit) {
      y = d;
      yl = sub2(r, both(kappa));
    } else {
      y = mul2(d, both(r_hi));
      yl = add2(__ffma2_rn(d, both(r_hi), make_float2(-y.x, -y.y)), __ffma2_rn(d, both(r_lo), __ffma2_rn(r, both(r_hi), both(-kappa))));
    }
    constexpr float kMagic = 12582912.f;  // 1.5 2^23: its last place is 1, its bits from the 22nd on only
    const float2 t = __ffma2_rn(y, both(0x1.715476p+8f), both(kMagic));
    const float2 k = sub2(both(kMagic), t);  // -k
    const uint32_t t0 = __float_as_uint(t.x), t1 = __float_as_uint(t.y);
    const uint2 p0 = powers[t0 & (kPow - 1)], p1 = powers[t1 & (kPow - 1)];
    const float2 gh = __ffma2_rn(k, both(-0x1.bdp-21f), __ffma2_rn(k, both(0x1.63p-9f), y));
    const float2 gl = add2(__ffma2_rn(k, both(-0x1.05c610p-37f), yl), make_float2(__uint_as_float(p0.y), __uint_as_float(p1.y)));
    const float2 g = add2(gh, gl);
    const float2 v = __ffma2_rn(mul2(g, g), __ffma2_rn(g, both(0x1.555556p-3f), both(0.5f)), gl);
    Term2 p;
    // the exponent n: t's bits are those of the magic number + 256 n + j
    p.a = make_float2(__uint_as_float(p0.x + (t0 << 15)), __uint_as_float(p1.x + (t1 << 15)));
    p.b = mul2(p.a, gh);
    p.c = __ffma2_rn(p.a, v, __ffma2_rn(p.a, gh, make_float2(-p.b.x, -p.b.y)));
    return p;
  }
  template <bool kWide, bool kTop, bool kUnit>
  __device__ __forceinline__ Term at(float z, const uint2* powers) const {
    return at<kWide, kTop, kUnit>(both(z), powers).x();
  }
  __device__ __forceinline__ bool is_zero(float z) const { return !(__fsub_rn(z, off) > zmin); }
};

// The differences of two terms, 1 where they are positive, 0 elsewhere, and 1 where they are within
// `window` of q.  Of positive differences the first number is the larger one in a, or the two are so near that
// p.a - q.a is exact.
__device__ __forceinline__ Term2 above(const Term2& p, const Term2& q, float2& more, float window, float2& beside) {
  float2 e;
  Term2 d;
  d.a = quick_two_sum2(p.a, make_float2(-q.a.x, -q.a.y), e);
  d.b = sub2(p.b, q.b);
  d.c = add2(e, sub2(p.c, q.c));
  const float2 s = add2(add2(d.a, d.b), d.c), w = mul2(q.a, both(window));
  more = make_float2(s.x > 0.f ? 1.f : 0.f, s.y > 0.f ? 1.f : 0.f);
  beside = make_float2(fabsf(s.x) < w.x ? 1.f : 0.f, fabsf(s.y) < w.y ? 1.f : 0.f);
  return d;
}
__device__ __forceinline__ Term2 above(const Term2& p, const Term2& q, float2& more) {
  float2 beside;
  return above(p, q, more, 0.f, beside);
}

// A sum of such terms, none above half of `start`: hi and mid start there, so that the error
// of each addition to them is exact (the larger one comes first), and lo, which
// is small, takes those and the c.  What lo is rounded by is 2^-24 of it at each addition, always to the same side where terms are equal:
// settle(), after a few terms, leaves it 2^-24 of hi, and a start far above the terms would leave errors as large as theirs.  (One token and
// 151,935 equal ones of 2^-17 of it, in 8 parts: off by 2^-26 with a start of 1 and no settling, by 2^-34 with both, and a
// border by 2^-36.6; settling every other time 2^-36.1, every fourth 2^-34.2.  64 draws take 41.8 us, 40.8 without either.)
struct FineSum {
  float2 hi, mid, lo;
  __device__ __forceinline__ void clear(float start) {
    hi = mid = both(start);
    lo = both(0.f);
  }
  __device__ __forceinline__ void settle() {
    float2 e;
    hi = quick_two_sum2(hi, lo, e);
    lo = e;
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
  __device__ __forceinline__ Wide value(float start) const {
    float e, f;
    const float s = two_sum(__fsub_rn(hi.x, start), __fsub_rn(hi.y, start), e);
    const float t = two_sum(__fsub_rn(mid.x, start), __fsub_rn(mid.y, start), f);
    float r;
    const float h = two_sum(s, t, r);
    return Wide(h, __fadd_rn(__fadd_rn(r, __fadd_rn(e, f)), __fadd_rn(lo.x, lo.y)));
  }
};

// ln of a positive number, to 2^-38: the hardware's logarithm of its significand f, put right by
// what f e^-ln(f) is above 1.
__device__ __forceinline__ Wide ln_wide(const Wide& s, const uint2* powers) {
  const int bits = __float_as_int(s.h), n = (bits >> 23) - 127;
  const float down = __int_as_float((127 - n) << 23);
  Wide f, ln2;
  f.h = __fmul_rn(s.h, down);
  f.l = __fmul_rn(s.l, down);
  ln2.h = 0x1.62e430p-1f;
  ln2.l = -0x1.05c610p-29f;
  const float y = __logf(f.h);
  FineExp e;
  e.init(1.f, 0.f, 1.f, 0.f, false);
  const Wide over = f * e.at<true, false, true>(-y, powers).value() - Wide(1.f);
  const float fix = __fmul_rn(over.h, fmaf(over.h, -0.5f, 1.f));
  return Wide(static_cast<float>(n)) * ln2 + Wide(y) + Wide(fix);
}

}  // namespace
}  // namespace rl
