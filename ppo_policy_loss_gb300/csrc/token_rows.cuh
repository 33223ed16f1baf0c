// token_rows.cuh — building blocks of the token log-probability and
// distillation kernels (sm_103a): the 64-byte piece of a logits row that one
// thread takes at a time, its element formats, and the online softmax
// statistics whose sum leaves the maximum out.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "rl_device.cuh"
#include "rltoken.h"

namespace rl {
namespace {

// A piece: 64 consecutive bytes of a row, four 16-byte vectors.  Lanes of a
// warp take consecutive pieces, so that a piece's maximum is one key of the
// top-k search; from shared memory lane l takes its vectors in the order
// (j + l / 2) mod 4, which touches every bank once per 8 lanes.
constexpr int kPieceBytes = 64;
constexpr long long kMaxVocab = 1LL << 26;
// Rows of a masked batch.  A warp looks through the mask at 512 rows in 0.4 us, so
// 2^28 masked rows before a valid one take 0.2 s (the distillation, which also
// counts them, 0.5 s) while the consumers' wait for its first chunk runs: half
// of the wait's limit.
constexpr long long kMaxMaskedRows = 1LL << 28;

// Every logit counts as at least the format's floor where a maximum or an
// entropy is formed, so that -inf, and the large negative numbers that masks
// write, give 2^x = 0 and 0 * x = 0 instead of NaN.  That is exact while the
// row's maximum is far above the floor; a row whose maximum is at most kExact
// is taken again without the floor (needs_exact).  In any other row a floor
// element's term is 2^-x with x >= min(32768 - 16384, 65504 - 32768)
// log2(e) / 100 > 236: 0 in fp32.
constexpr float kMinTemperature = 0.01f, kMaxTemperature = 100.f;

__device__ __forceinline__ uint32_t pmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pmax_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Order keys: unsigned integers that compare as the values do, with -0 = +0,
// every NaN above +inf, and 0 below every value (an empty place).
__device__ __forceinline__ uint32_t order16(uint32_t b, uint32_t inf) {
  if ((b & 0x7fffu) > inf) return 0xffffu;
  if (b == 0x8000u) b = 0u;
  return (b & 0x8000u) ? (b ^ 0xffffu) : (b | 0x8000u);
}
__device__ __forceinline__ uint32_t unorder16(uint32_t k) { return (k & 0x8000u) ? (k & 0x7fffu) : (k ^ 0xffffu); }
__device__ __forceinline__ uint32_t order32(uint32_t b) {
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unorder32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Per format: elements per piece, the piece's raw maximum as a key and as a
// float, taking elements out of it, clamping a word at the floor, widening,
// and single elements.
template <int DT>
struct Fmt;

template <>
struct Fmt<RL_F32> {
  using Key = uint32_t;
  static constexpr int kBytes = 4, kPiece = 16, kVec = 4;
  static constexpr float kFloor = -32768.f, kExact = -16384.f;
  static constexpr uint32_t kNegInf2 = 0xff800000u;
  // of the piece at w[b .. b + 15]
  template <int N>
  __device__ static uint32_t raw_max(const uint32_t (&w)[N], int b) {
    float m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)  // four chains
      m[j] = max_nan(max_nan(__uint_as_float(w[b + j]), __uint_as_float(w[b + 4 + j])),
                     max_nan(__uint_as_float(w[b + 8 + j]), __uint_as_float(w[b + 12 + j])));
    return __float_as_uint(max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3])));
  }
  __device__ static float raw_value(uint32_t r) { return __uint_as_float(r); }
  __device__ static uint32_t clamp(uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), kFloor)); }
  // elements e .. 15 of the piece at w[b ..] become -inf
  template <int N>
  __device__ static void cut(uint32_t (&w)[N], int b, int e) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i >= e) w[b + i] = kNegInf2;
  }
  // element e of the piece becomes the floor
  template <int N>
  __device__ static void drop(uint32_t (&w)[N], int b, int e) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i == e) w[b + i] = __float_as_uint(kFloor);
  }
  // if `take`, the elements of value v become the floor; how many there were
  template <int N>
  __device__ static int drop_value(uint32_t (&w)[N], float v, bool take) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool hit = take && __uint_as_float(w[i]) == v;
      w[i] = hit ? __float_as_uint(kFloor) : w[i];
      n += hit;
    }
    return n;
  }
  template <int N>
  __device__ static void pair(const uint32_t (&w)[N], int i, float& a, float& b) {
    a = __uint_as_float(w[2 * i]);
    b = __uint_as_float(w[2 * i + 1]);
  }
  __device__ static float load(const unsigned char* row, long long i) { return reinterpret_cast<const float*>(row)[i]; }
  // elements of a vector that are not below thr (NaN is not), as bits; hit_elem: which element a bit is
  __device__ static uint32_t hits(const uint4& v, float thr) {
    return (!(__uint_as_float(v.x) < thr) ? 1u : 0u) | (!(__uint_as_float(v.y) < thr) ? 2u : 0u) |
           (!(__uint_as_float(v.z) < thr) ? 4u : 0u) | (!(__uint_as_float(v.w) < thr) ? 8u : 0u);
  }
  __device__ static int hit_elem(int bit) { return bit; }
  __device__ static uint32_t pick(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
  using Raw = uint32_t;
  __device__ static Raw load_raw(const unsigned char* row, long long i) { return reinterpret_cast<const Raw*>(row)[i]; }
  __device__ static uint32_t raw_order(Raw r) { return order32(r); }
  __device__ static uint32_t load_order(const unsigned char* row, long long i) { return raw_order(load_raw(row, i)); }
  __device__ static float order_value(uint32_t k) { return unorder32(k); }
  __device__ static uint32_t order_of(float v) { return order32(__float_as_uint(v)); }
  static constexpr uint32_t kOrderStep = 8u << 16;  // a few bf16 steps
  __device__ static float load_shared(const unsigned char* piece, int e) { return reinterpret_cast<const float*>(piece)[e]; }
  __device__ static void store(unsigned char* row, long long i, float v) { reinterpret_cast<float*>(row)[i] = v; }
  __device__ static void unpack(const uint4& w, float (&z)[kVec]) {
    z[0] = __uint_as_float(w.x);
    z[1] = __uint_as_float(w.y);
    z[2] = __uint_as_float(w.z);
    z[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 pack(const float (&z)[kVec]) {
    return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
  }
};

template <>
struct Fmt<RL_BF16> {
  using Key = uint16_t;
  static constexpr int kBytes = 2, kPiece = 32, kVec = 8;
  static constexpr float kFloor = -32768.f, kExact = -16384.f;
  static constexpr uint32_t kFloor2 = 0xC700C700u, kNegInf2 = 0xFF80FF80u;
  template <int N>
  __device__ static uint32_t raw_max(const uint32_t (&w)[N], int b) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)  // four chains
      c[j] = pmax_bf16x2(pmax_bf16x2(w[b + j], w[b + 4 + j]), pmax_bf16x2(w[b + 8 + j], w[b + 12 + j]));
    const uint32_t m = pmax_bf16x2(pmax_bf16x2(c[0], c[1]), pmax_bf16x2(c[2], c[3]));
    return pmax_bf16x2(m, (m >> 16) | (m << 16)) & 0xffffu;
  }
  __device__ static float raw_value(uint32_t r) { return __uint_as_float(r << 16); }
  __device__ static uint32_t clamp(uint32_t w) { return pmax_bf16x2(w, kFloor2); }
  template <int N>
  __device__ static void cut(uint32_t (&w)[N], int b, int e) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (2 * i >= e)
        w[b + i] = kNegInf2;
      else if (2 * i + 1 >= e)
        w[b + i] = (w[b + i] & 0xffffu) | (kNegInf2 & 0xffff0000u);
    }
  }
  template <int N>
  __device__ static void drop(uint32_t (&w)[N], int b, int e) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (2 * i == e) w[b + i] = (w[b + i] & 0xffff0000u) | (kFloor2 & 0xffffu);
      if (2 * i + 1 == e) w[b + i] = (w[b + i] & 0xffffu) | (kFloor2 & 0xffff0000u);
    }
  }
  template <int N>
  __device__ static int drop_value(uint32_t (&w)[N], float v, bool take) {
    const uint32_t on = take ? ~0u : 0u;
    const __nv_bfloat162 v2 = __float2bfloat162_rn(v);
    uint32_t n2 = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t hit = __heq2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), v2) & on;
      w[i] = (w[i] & ~hit) | (kFloor2 & hit);
      n2 += hit & 0x00010001u;
    }
    return static_cast<int>((n2 & 0xffffu) + (n2 >> 16));
  }
  template <int N>
  __device__ static void pair(const uint32_t (&w)[N], int i, float& a, float& b) {
    a = __uint_as_float(w[i] << 16);
    b = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ static float load(const unsigned char* row, long long i) {
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[i]) << 16);
  }
  __device__ static uint32_t hits(const uint4& v, float thr) {
    const __nv_bfloat162 t2 = __float2bfloat162_rn(thr);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t b = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b |= (__hgeu2_mask(*reinterpret_cast<const __nv_bfloat162*>(&u[j]), t2) & 0x00010001u) << j;
    return b;
  }
  __device__ static int hit_elem(int bit) { return 2 * (bit & 15) + (bit >> 4); }
  __device__ static uint32_t pick(const uint4& v, int i) {
    const uint32_t w = i < 4 ? (i < 2 ? v.x : v.y) : (i < 6 ? v.z : v.w);
    return (i & 1) ? w >> 16 : w & 0xffffu;
  }
  using Raw = uint16_t;
  __device__ static Raw load_raw(const unsigned char* row, long long i) { return reinterpret_cast<const Raw*>(row)[i]; }
  __device__ static uint32_t raw_order(Raw r) { return order16(r, 0x7f80u); }
  __device__ static uint32_t load_order(const unsigned char* row, long long i) { return raw_order(load_raw(row, i)); }
  __device__ static float order_value(uint32_t k) { return __uint_as_float(unorder16(k) << 16); }
  __device__ static uint32_t order_of(float v) { return order16(__float_as_uint(v) >> 16, 0x7f80u); }
  static constexpr uint32_t kOrderStep = 8u;
  __device__ static float load_shared(const unsigned char* piece, int e) { return load(piece, e); }
  __device__ static void store(unsigned char* row, long long i, float v) {
    reinterpret_cast<__nv_bfloat16*>(row)[i] = __float2bfloat16_rn(v);
  }
  __device__ static void unpack(const uint4& w, float (&z)[kVec]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      z[2 * k] = __uint_as_float(u[k] << 16);
      z[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float (&z)[kVec]) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __nv_bfloat162 h = __floats2bfloat162_rn(z[2 * k], z[2 * k + 1]);
      u[k] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

template <>
struct Fmt<RL_F16> {
  using Key = uint16_t;
  static constexpr int kBytes = 2, kPiece = 32, kVec = 8;
  static constexpr float kFloor = -65504.f, kExact = -32768.f;
  static constexpr uint32_t kFloor2 = 0xFBFFFBFFu, kNegInf2 = 0xFC00FC00u;
  template <int N>
  __device__ static uint32_t raw_max(const uint32_t (&w)[N], int b) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)  // four chains
      c[j] = pmax_f16x2(pmax_f16x2(w[b + j], w[b + 4 + j]), pmax_f16x2(w[b + 8 + j], w[b + 12 + j]));
    const uint32_t m = pmax_f16x2(pmax_f16x2(c[0], c[1]), pmax_f16x2(c[2], c[3]));
    return pmax_f16x2(m, (m >> 16) | (m << 16)) & 0xffffu;
  }
  __device__ static float half_bits(uint32_t r) { return __half2float(__ushort_as_half(static_cast<unsigned short>(r))); }
  __device__ static float raw_value(uint32_t r) { return half_bits(r); }
  __device__ static uint32_t clamp(uint32_t w) { return pmax_f16x2(w, kFloor2); }
  template <int N>
  __device__ static void cut(uint32_t (&w)[N], int b, int e) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (2 * i >= e)
        w[b + i] = kNegInf2;
      else if (2 * i + 1 >= e)
        w[b + i] = (w[b + i] & 0xffffu) | (kNegInf2 & 0xffff0000u);
    }
  }
  template <int N>
  __device__ static void drop(uint32_t (&w)[N], int b, int e) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (2 * i == e) w[b + i] = (w[b + i] & 0xffff0000u) | (kFloor2 & 0xffffu);
      if (2 * i + 1 == e) w[b + i] = (w[b + i] & 0xffffu) | (kFloor2 & 0xffff0000u);
    }
  }
  template <int N>
  __device__ static int drop_value(uint32_t (&w)[N], float v, bool take) {
    const uint32_t on = take ? ~0u : 0u;
    const __half2 v2 = __float2half2_rn(v);
    uint32_t n2 = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t hit = __heq2_mask(*reinterpret_cast<const __half2*>(&w[i]), v2) & on;
      w[i] = (w[i] & ~hit) | (kFloor2 & hit);
      n2 += hit & 0x00010001u;
    }
    return static_cast<int>((n2 & 0xffffu) + (n2 >> 16));
  }
  template <int N>
  __device__ static void pair(const uint32_t (&w)[N], int i, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    a = f.x;
    b = f.y;
  }
  __device__ static float load(const unsigned char* row, long long i) {
    return half_bits(reinterpret_cast<const uint16_t*>(row)[i]);
  }
  __device__ static uint32_t hits(const uint4& v, float thr) {
    const __half2 t2 = __float2half2_rn(thr);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t b = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b |= (__hgeu2_mask(*reinterpret_cast<const __half2*>(&u[j]), t2) & 0x00010001u) << j;
    return b;
  }
  __device__ static int hit_elem(int bit) { return 2 * (bit & 15) + (bit >> 4); }
  __device__ static uint32_t pick(const uint4& v, int i) {
    const uint32_t w = i < 4 ? (i < 2 ? v.x : v.y) : (i < 6 ? v.z : v.w);
    return (i & 1) ? w >> 16 : w & 0xffffu;
  }
  using Raw = uint16_t;
  __device__ static Raw load_raw(const unsigned char* row, long long i) { return reinterpret_cast<const Raw*>(row)[i]; }
  __device__ static uint32_t raw_order(Raw r) { return order16(r, 0x7c00u); }
  __device__ static uint32_t load_order(const unsigned char* row, long long i) { return raw_order(load_raw(row, i)); }
  __device__ static float order_value(uint32_t k) { return half_bits(unorder16(k)); }
  __device__ static uint32_t order_of(float v) { return order16(__half_as_ushort(__float2half_rn(v)), 0x7c00u); }
  static constexpr uint32_t kOrderStep = 32u;
  __device__ static float load_shared(const unsigned char* piece, int e) { return load(piece, e); }
  __device__ static void store(unsigned char* row, long long i, float v) {
    reinterpret_cast<__half*>(row)[i] = __float2half_rn(v);
  }
  __device__ static void unpack(const uint4& w, float (&z)[kVec]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
      z[2 * k] = f.x;
      z[2 * k + 1] = f.y;
    }
  }
  __device__ static uint4 pack(const float (&z)[kVec]) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __half2 h = __floats2half2_rn(z[2 * k], z[2 * k + 1]);
      u[k] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// ------------------------------------------------------------------ statistics
// Over a set of logits with maximum m: r = sum 2^x - 1 and t = sum 2^x x,
// x = (z - m) c with c = log2(e) / temperature.  Then
//   lse = m / temperature + log1p(r),   H = log1p(r) - ln 2 t / (1 + r).
// One of the maxima (its term is exactly 1) is left out of the sum, so r is a
// sum of small terms where one token holds nearly all the mass and log1p(r)
// keeps its relative precision.  An empty set is m = floor, r = -1, t = 0.
struct RowStats {
  float m, r, t;
};

__device__ __forceinline__ RowStats merge_row(RowStats a, RowStats b, float c) {
  if (b.m > a.m) {
    const RowStats x = a;
    a = b;
    b = x;
  }
  const float s = 1.f + b.r;
  if (s == 0.f) return a;  // empty (a NaN goes on and poisons)
  const float d = (a.m - b.m) * c;
  const float f = ex2_approx(-d);
  a.r = fmaf(f, s, a.r);
  a.t = fmaf(f, fmaf(-d, s, b.t), a.t);
  return a;
}

// A warp's running statistics: m is the warp's, r and t are spread over its
// lanes.  The terms are taken in the frame x' = z c + nm, nm = -m c rounded
// to fp32: one FMA an element, and the rounding that all terms of a frame
// share (2^rho, rho = -m c - nm) is put right once, when the frame ends.
// That holds for |m c| <= kFrame, where |rho| <= 1/2: every frame between the
// floor (65504 * 144.3 < kFrame at the lowest temperature) and such a maximum.
// A row with a larger maximum, or one of at most kExact, is taken again by
// differences to m.
constexpr float kFrame = 0x1p24f;
template <class F>
__device__ __forceinline__ bool needs_exact(float m, float c) {
  return !(m > F::kExact) || !(fabsf(m) * c <= kFrame);
}
struct WarpStats {
  float m, nm;
  float2 r[2], t[2];  // independent chains
  float own;  // lane 0: the maximum itself, where the set is not empty (else 0)
  bool low;   // -inf has been met: clamp what comes
};

template <class F>
__device__ __forceinline__ void warp_stats_init(WarpStats& a, float c) {
  a.m = F::kFloor;
  a.nm = -F::kFloor * c;
  a.r[0] = a.r[1] = make_float2(0.f, 0.f);
  a.t[0] = a.t[1] = make_float2(0.f, 0.f);
  a.own = 0.f;
}

// This lane's sums brought from the frame nm to the exact frame of m.  (Products
// that a sum takes are rounded: two builds of a caller give the same bits.)
__device__ __forceinline__ void end_frame(const WarpStats& a, float c, float& r, float& t) {
  const float rho = fmaf(-a.m, c, -a.nm);  // exact: the product's rounding error
  const float g = ex2_approx(rho);
  r = (a.r[0].x + a.r[0].y) + (a.r[1].x + a.r[1].y);
  t = __fmul_rn(fmaf(rho, r, (a.t[0].x + a.t[0].y) + (a.t[1].x + a.t[1].y)), g);
  r = __fmul_rn(r, g);
}

// One step: this lane's piece (raw words), of clamped maximum pm.  Warp-wide.
// -inf words add 0 to r, but NaN to t (0 * inf): they are looked for where
// `check` says so, and from then on the words are clamped at the floor first.
// A set without -inf gives the same bits either way: what the clamp changes is
// a term of 0 in the end (a row that needs_exact aside).
template <class F, bool kEntropy>
__device__ __forceinline__ void add_piece(WarpStats& a, uint32_t (&w)[16], float pm, float c, int lane, bool check) {
  float wm;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(wm) : "f"(pm));
  if (wm > a.m) {
    // the warp's maximum rises: the old frame ends, lane 0 takes the old
    // maximum back in, and the first lane that holds the new one drops it
    // (its other elements of that value are terms of exactly 1)
    float r, t;
    end_frame(a, c, r, t);
    const float d = (wm - a.m) * c;
    const float f = ex2_approx(-d);
    const float s = r + a.own;
    a.m = wm;
    a.nm = -wm * c;
    a.own = lane == 0 ? 1.f : 0.f;
    const uint32_t holders = __ballot_sync(0xffffffffu, pm == wm);
    const bool take = lane == __ffs(holders) - 1;
    const int n = F::template drop_value<16>(w, wm, take);
    // what goes on into the new frame: 2^-rho of it, x' = x - rho
    const float rho = fmaf(-wm, c, -a.nm), h = ex2_approx(-rho);
    const float kept = fmaf(f, s, take ? static_cast<float>(n - 1) : 0.f);
    a.r[0] = make_float2(h * kept, 0.f);
    a.r[1] = make_float2(0.f, 0.f);
    a.t[0] = make_float2(kEntropy ? h * fmaf(-rho, kept, f * fmaf(-d, s, t)) : 0.f, 0.f);
    a.t[1] = make_float2(0.f, 0.f);
  }
  if (kEntropy && check && !a.low) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) any = any || F::clamp(w[i]) != w[i];
    a.low = __any_sync(0xffffffffu, any);
  }
  if (kEntropy && a.low) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = F::clamp(w[i]);
  }
  const float2 c2 = make_float2(c, c), nm2 = make_float2(a.nm, a.nm);
#pragma unroll
  for (int i = 0; i < F::kPiece / 2; ++i) {
    float2 z;
    F::template pair<16>(w, i, z.x, z.y);
    const float2 x = __ffma2_rn(z, c2, nm2);
    const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    a.r[i & 1] = __fadd2_rn(a.r[i & 1], e);
    if (kEntropy) a.t[i & 1] = __ffma2_rn(e, x, a.t[i & 1]);
  }
}

// The sum of 2^x alone, over sets whose maximum need not be known: the frame
// is that of the maximum of the warp's first piece, and moves up only when a
// lane's sum passes kSumLimit.  The sum so far then goes along by 2^(nm' - nm),
// which its terms 2^(z c + nm) need to the bit; the last frame's rounding is
// put right at the end, as above.
constexpr float kSumLimit = 0x1p24f;
struct WarpSum {
  float m, nm;
  float2 r[2];  // independent chains
};
template <class F>
__device__ __forceinline__ float clamped_max(const uint32_t (&w)[16]) {
  float wm;
  const float pm = max_nan(F::raw_value(F::raw_max(w, 0)), F::kFloor);
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(wm) : "f"(pm));
  return wm;
}
template <class F>
__device__ __forceinline__ void sum_init(WarpSum& a, const uint32_t (&w)[16], float c) {
  a.m = clamped_max<F>(w);
  if (!(a.m >= F::kFloor)) a.m = F::kFloor;  // nothing but NaN
  a.nm = -a.m * c;
  a.r[0] = a.r[1] = make_float2(0.f, 0.f);
}
template <class F>
__device__ __forceinline__ void sum_piece(WarpSum& a, const uint32_t (&w)[16], float c) {
  const float2 r0 = a.r[0], r1 = a.r[1];
  const float2 c2 = make_float2(c, c);
  bool again = false;
#pragma unroll 1
  while (true) {
    const float2 nm2 = make_float2(a.nm, a.nm);
#pragma unroll
    for (int i = 0; i < F::kPiece / 2; ++i) {
      float2 z;
      F::template pair<16>(w, i, z.x, z.y);
      const float2 x = __ffma2_rn(z, c2, nm2);
      a.r[i & 1] = __fadd2_rn(a.r[i & 1], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
    }
    const float s = (a.r[0].x + a.r[0].y) + (a.r[1].x + a.r[1].y);
    if (again || !__any_sync(0xffffffffu, !(s < kSumLimit))) break;
    const float m = fmaxf(a.m, clamped_max<F>(w));
    const float nm = __fmul_rn(-m, c);  // rounded here, not fused into the difference
    const float f = ex2_approx(nm - a.nm);
    a.m = m;
    a.nm = nm;
    a.r[0] = make_float2(f * ((r0.x + r0.y) + (r1.x + r1.y)), 0.f);
    a.r[1] = make_float2(0.f, 0.f);
    again = true;  // (a NaN passes)
  }
}
template <class F>
__device__ __forceinline__ RowStats warp_sum_stats(const WarpSum& a, float c) {
  float r = (a.r[0].x + a.r[0].y) + (a.r[1].x + a.r[1].y);
  r *= ex2_approx(fmaf(-a.m, c, -a.nm));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return RowStats{a.m, r - 1.f, 0.f};
}

// The warp's statistics in every lane.
template <class F>
__device__ __forceinline__ RowStats warp_stats_sum(const WarpStats& a, float c) {
  float r, t;
  end_frame(a, c, r, t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r += __shfl_xor_sync(0xffffffffu, r, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  // nothing rose above the floor: no term was left out
  if (!(a.m > F::kFloor)) r -= 1.f;
  return RowStats{a.m, r, t};
}

// A lane's piece from shared memory.  Lanes take their four vectors in the
// order (j + sh) mod 4; sh = lane / 2 touches every bank once per 8 lanes, sh
// = 0 keeps the elements in order (a row's last, partly filled piece).
template <int N>
__device__ __forceinline__ void load_piece(uint32_t (&w)[N], int b, uint32_t at, int sh) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = ld_shared_v4(at + ((j + sh) & 3) * 16);
    w[b + 4 * j] = v.x;
    w[b + 4 * j + 1] = v.y;
    w[b + 4 * j + 2] = v.z;
    w[b + 4 * j + 3] = v.w;
  }
}

// ------------------------------------------------------------------ rows
// The valid (kValid) or the masked rows number first, first + stride, ... of the
// batch, so that every CTA gets the same share of them wherever the masked rows
// lie.  The mask is read 512 rows at a time; no mask: every row is valid.
// Whole warp.
template <bool kValid>
struct RowsOf {
  const unsigned char* mask;
  long long R;
  long long want;           // number of the next row among those
  long long base, before;   // first row of the window, such rows before it
  uint32_t bits, prefix;    // this lane's 16 rows, such rows of the window before them
  int total;                // such rows of the window
  __device__ RowsOf(const unsigned char* mask_, long long R_, long long first, int lane)
      : mask(mask_), R(R_), want(first), base(0), before(0), bits(0u), prefix(0u), total(0) {
    if (mask) load(lane);
  }
  __device__ __forceinline__ void load(int lane) {
    const long long r = base + lane * 16;
    bits = 0u;
    if (r + 16 <= R && ((reinterpret_cast<uintptr_t>(mask) + r) & 15) == 0) {
      const uint4 v = *reinterpret_cast<const uint4*>(mask + r);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) bits |= ((u[j] >> (8 * q)) & 0xffu) ? 1u << (4 * j + q) : 0u;
    } else {
      for (int q = 0; q < 16; ++q)
        if (r + q < R && mask[r + q]) bits |= 1u << q;
    }
    if (!kValid) bits = ~bits & (r + 16 <= R ? 0xffffu : r < R ? (1u << (R - r)) - 1u : 0u);
    const uint32_t n = __popc(bits);
    prefix = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, prefix, o);
      if (lane >= o) prefix += up;
    }
    total = __shfl_sync(0xffffffffu, prefix, 31);
    prefix -= n;
  }
  // the next row, -1 after the last
  __device__ __forceinline__ long long next(long long stride, int lane) {
    long long row = -1;
    if (!mask) {
      if (kValid && want < R) row = want;
    } else {
      while (want >= before + total && base + 512 < R) {
        before += total;
        base += 512;
        load(lane);
      }
      if (want < before + total) {
        const uint32_t at = static_cast<uint32_t>(want - before);
        const bool here = at >= prefix && at < prefix + __popc(bits);
        const uint32_t who = __ballot_sync(0xffffffffu, here);
        const uint32_t bit = here ? __fns(bits, 0, static_cast<int>(at - prefix) + 1) : 0u;
        const int l = __ffs(who) - 1;
        row = base + l * 16 + __shfl_sync(0xffffffffu, bit, l);
      }
    }
    want += stride;
    return row;
  }
  // row number n of them (in any order; forwards costs least)
  __device__ __forceinline__ long long at(long long n, int lane) {
    if (n >= R) return -1;
    if (mask && n < before) {
      base = before = 0;
      load(lane);
    }
    want = n;
    return next(0, lane);
  }
};

// ------------------------------------------------------------------ chunk ring
// Chunks of a row arrive by bulk copies in a ring of shared-memory slots: the
// producer (one lane) waits for a slot's release and issues the copy, the
// consumers wait for its arrival, in the same order of chunks.
template <int kSlots, int kChunk>
struct Ring {
  alignas(128) unsigned char data[kSlots][kChunk];
  unsigned long long full[kSlots], empty[kSlots];

  __device__ void init(int consumer_warps) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), consumer_warps);
    }
  }
  // producer: chunk number `it` of this CTA has a free slot; false once a wait has given up
  __device__ __forceinline__ bool reserve(uint32_t it, volatile int* abort) {
    const uint32_t slot = it % kSlots, round = it / kSlots;
    return round == 0 || wait_bounded<false>(smem_addr(&empty[slot]), (round - 1) & 1, abort);
  }
  __device__ __forceinline__ void fill(uint32_t it, const unsigned char* src, uint32_t bytes, uint64_t policy) {
    const uint32_t fb = smem_addr(&full[it % kSlots]);
    mbar_arrive_expect_tx(fb, bytes);
    bulk_load(smem_addr(data[it % kSlots]), src, bytes, fb, policy);
  }
  // producer: the `it` chunks issued so far have landed (before the CTA may exit)
  __device__ void drain(uint32_t it) {
    for (uint32_t k = it > kSlots ? it - kSlots : 0; k < it; ++k) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(smem_addr(&full[k % kSlots]), (k / kSlots) & 1) && global_ns() - t0 <= kWaitLimitNs) {
      }
    }
  }
  __device__ __forceinline__ uint32_t wait(uint32_t it, volatile int* abort) {
    const uint32_t slot = it % kSlots;
    wait_bounded<false>(smem_addr(&full[slot]), (it / kSlots) & 1, abort);
    return smem_addr(data[slot]);
  }
  // whole warp: the slot's bytes have been read
  __device__ __forceinline__ void release(uint32_t it, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&empty[it % kSlots]));
  }
};

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

__device__ __forceinline__ uint64_t policy_keep() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}
__device__ __forceinline__ uint64_t policy_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Host: the kernel's dynamic shared memory allowed, once per device (a bit of
// `allowed` each; nothing that can throw, for this runs below a C entry).
inline rl_status allow_smem(const void* fn, int dev, int smem, std::atomic<unsigned long long>& allowed) {
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (allowed.load(std::memory_order_acquire) & bit) return RL_OK;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return RL_ERR_CUDA;
  allowed.fetch_or(bit, std::memory_order_release);
  return RL_OK;
}

// Host: whether two matrices of R rows of `width` bytes, both with rows
// `row_bytes` apart, share any of them.
inline bool rows_overlap(const void* a, const void* b, long long R, long long row_bytes, long long width) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const uintptr_t d = x < y ? y - x : x - y, step = static_cast<uintptr_t>(row_bytes);
  const uintptr_t rows = static_cast<uintptr_t>(R), w = static_cast<uintptr_t>(width);
  // row j of the later one begins d % step past row j + d / step of the earlier one
  return (d / step < rows && d % step < w) || (d / step + 1 < rows && step - d % step < w);
}

}  // namespace
}  // namespace rl
