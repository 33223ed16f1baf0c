// quantize_rows.cu — rl_quantize_rows_int8: 8-bit codes of a matrix's rows and
// a scale for each (include/rlrollout.h).
//
// One pass over the data: a row stays in its threads' registers between the
// maximum and the rounding.  Bound by HBM: an element is 2 or 4 bytes in and 1 out.  Rows of more than
// kMaxThreads * kVecs vectors are read a second time, mostly from HBM again: 1.5 GB of bf16 rows of 16,384 take
// 430 us (5.2 TB/s of in and out), of 16,640 611 us (3.7), of 262,144 693 us; of fp32 rows of 8,192 346 us (5.4), of
// 16,384 435 us (4.3), of 262,144 640 us.
//
// The codes are those of the exact quotient x / s.  The candidate k, the low byte of
// x (1 / s) + 1.5 2^23, is within one of it, and e = x - k s is exact in one FMA
// (|k| >= 1: a multiple of s's last place below 2^24 of them; k = 0: x itself).  Where no
// |e| of a vector reaches s / 2, as in all but some 10^-4 of them, the candidates stand; else they
// are put right one by one.  So an element is one FMA, one subtraction, one FMA and a
// comparison, and no conversion (the unit for those is an eighth as fast), which HBM covers.
#include <cuda_runtime.h>

#include <cstdint>

#include "rlrollout.h"
#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kVecs = 4;            // 16-byte vectors that a thread keeps
constexpr int kMaxThreads = 512;    // of one row
constexpr int kBlock = 256;         // threads of a CTA of short rows
constexpr int kThreadsPerSm = 1280; // of 48 registers (a few words spilled: 82 us against 85 with 64 at 151,936 x 1024)
constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer

struct RowScale {
  float s, half, inv, up;  // the scale; with x up in the place of x: s up / 2 and 1 / (s up)
};

__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.s = __fdiv_rn(amax, 127.f);
  if (!(r.s < INFINITY)) r.s = __int_as_float(0x7fc00000);
  r.up = r.s < 0x1p-100f ? 0x1p80f : 1.f;  // (1 / s overflows for the smallest, and s / 2 has fewer digits)
  const float s = r.s * r.up;
  r.half = 0.5f * s;
  r.inv = r.s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
  return r;
}

// The codes of kN numbers, a byte each.
template <int kN>
__device__ __forceinline__ void codes_of(const float (&x)[kN], const RowScale& r, uint32_t (&w)[kN / 4]) {
  float z[kN], t[kN];
  bool again = r.up != 1.f;
  const float s = r.half + r.half;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    t[j] = fmaf(x[j], r.inv, kMagic);
    again = again || !(fabsf(fmaf(-__fsub_rn(t[j], kMagic), s, x[j])) < r.half);
  }
  if (again) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      z[j] = x[j] * r.up;
      t[j] = fmaf(z[j], r.inv, kMagic);
      float k = __fsub_rn(t[j], kMagic);
      const float e = fmaf(-k, s, z[j]);
      if (fabsf(e) >= r.half && (fabsf(e) > r.half || (__float_as_int(t[j]) & 1))) k += copysignf(1.f, e);
      k = fminf(fmaxf(k, -127.f), 127.f);  // (a scale of few digits may be too small)
      t[j] = r.s > 0.f ? __fadd_rn(k, kMagic) : kMagic;
    }
  }
#pragma unroll
  for (int j = 0; j < kN / 4; ++j)
    w[j] = __byte_perm(__byte_perm(__float_as_uint(t[4 * j]), __float_as_uint(t[4 * j + 1]), 0x0040),
                       __byte_perm(__float_as_uint(t[4 * j + 2]), __float_as_uint(t[4 * j + 3]), 0x0040), 0x5410);
}

// The vector at element i, zeros behind the row.
template <int DT>
__device__ __forceinline__ uint4 load_row(const unsigned char* row, long long i, long long D) {
  using F = Fmt<DT>;
  if (i + F::kVec <= D) return __ldcs(reinterpret_cast<const uint4*>(row + i * F::kBytes));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < F::kVec; ++j) {
    if (i + j < D) {
      const uint32_t x = F::load_raw(row, i + j);
      if (F::kBytes == 4)
        w[j & 3] = x;
      else
        w[j / 2 & 3] |= x << (16 * (j & 1));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest size of an element of vectors first .. first + kN - 1 (NaN if there is one).
template <int DT, int kN>
__device__ __forceinline__ float largest(const uint4 (&v)[kVecs], int first) {
  constexpr uint32_t sizes = DT == RL_F32 ? 0x7fffffffu : 0x7fff7fffu;
  uint32_t w[4 * kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    w[4 * j] = j < kN ? v[first + j].x & sizes : 0u;
    w[4 * j + 1] = j < kN ? v[first + j].y & sizes : 0u;
    w[4 * j + 2] = j < kN ? v[first + j].z & sizes : 0u;
    w[4 * j + 3] = j < kN ? v[first + j].w & sizes : 0u;
  }
  return Fmt<DT>::raw_value(Fmt<DT>::raw_max(w, 0));
}

template <int DT>
__device__ __forceinline__ void store_codes(signed char* row, long long i, long long D, const uint4& v, const RowScale& r) {
  using F = Fmt<DT>;
  if (i >= D) return;
  float z[F::kVec];
  F::unpack(v, z);
  uint32_t w[F::kVec / 4];
  codes_of<F::kVec>(z, r, w);
  if (i + F::kVec <= D) {
    if (F::kVec == 8)
      *reinterpret_cast<uint2*>(row + i) = make_uint2(w[0], w[F::kVec / 4 - 1]);
    else
      *reinterpret_cast<uint32_t*>(row + i) = w[0];
  } else {
#pragma unroll
    for (int j = 0; j < F::kVec; ++j)
      if (i + j < D) row[i + j] = static_cast<signed char>((w[j / 4] >> (8 * (j & 3))) & 0xffu);
  }
}

// TPR threads (a power of two of at least 32) take RPT rows at a time, kVecs vectors a thread in
// all: short rows several, so that as many loads are in flight.
template <int DT, int TPR, int RPT>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock, kThreadsPerSm / (TPR > kBlock ? TPR : kBlock))
quantize_rows_kernel(const unsigned char* __restrict__ x, long long R, long long D, long long row_bytes,
                     signed char* __restrict__ codes, long long ld_c, float* __restrict__ scale) {
  using F = Fmt<DT>;
  constexpr int kRows = TPR > kBlock ? 1 : kBlock / TPR;
  constexpr int kWarps = TPR / 32, kN = kVecs / RPT;
  constexpr long long kTurn = static_cast<long long>(kN) * TPR * F::kVec;  // elements of a row that the threads keep
  __shared__ float part[kRows][kWarps];
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const long long r0 = (static_cast<long long>(blockIdx.x) * kRows + g) * RPT;
  uint4 v[kVecs] = {};
#pragma unroll
  for (int k = 0; k < RPT; ++k)
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (r0 + k < R) v[k * kN + j] = load_row<DT>(x + (r0 + k) * row_bytes, (static_cast<long long>(j) * TPR + t) * F::kVec, D);
  float amax[RPT];
#pragma unroll
  for (int k = 0; k < RPT; ++k) amax[k] = largest<DT, kN>(v, k * kN);
  if (RPT == 1 && r0 < R) {
    for (long long base = kTurn; base < D; base += kTurn) {
      uint4 y[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j) y[j] = load_row<DT>(x + r0 * row_bytes, base + (static_cast<long long>(j) * TPR + t) * F::kVec, D);
      amax[0] = max_nan(amax[0], largest<DT, kVecs>(y, 0));
    }
  }
#pragma unroll
  for (int k = 0; k < RPT; ++k) asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(amax[k]) : "f"(amax[k]));
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) part[g][t / 32] = amax[0];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax[0] = max_nan(amax[0], part[g][w]);
  }
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const long long r = r0 + k;
    if (r >= R) return;
    const RowScale rs = row_scale(amax[k]);
    if (t == 0) scale[r] = rs.s;
    signed char* out = codes + r * ld_c;
#pragma unroll
    for (int j = 0; j < kN; ++j) store_codes<DT>(out, (static_cast<long long>(j) * TPR + t) * F::kVec, D, v[k * kN + j], rs);
    if (RPT == 1)
      for (long long i = kTurn + t * F::kVec; i < D; i += static_cast<long long>(TPR) * F::kVec)
        store_codes<DT>(out, i, D, load_row<DT>(x + r * row_bytes, i, D), rs);
  }
}

template <int DT, int TPR, int RPT>
void launch(const void* x, long long R, long long D, long long ld_x, signed char* codes, long long ld_c, float* scale,
            cudaStream_t stream) {
  static_assert(RPT == 1 || TPR == 32, "several rows are a warp's");
  constexpr int groups = TPR > kBlock ? 1 : kBlock / TPR, rows = groups * RPT;
  quantize_rows_kernel<DT, TPR, RPT><<<static_cast<unsigned>((R + rows - 1) / rows), groups * TPR, 0, stream>>>(
      static_cast<const unsigned char*>(x), R, D, ld_x * Fmt<DT>::kBytes, codes, ld_c, scale);
}

// as few threads as hold the row in their registers
template <int DT>
void launch_rows(const void* x, long long R, long long D, long long ld_x, signed char* codes, long long ld_c, float* scale,
                 cudaStream_t stream) {
  const long long vecs = (D + Fmt<DT>::kVec - 1) / Fmt<DT>::kVec;
  if (vecs <= 32)
    launch<DT, 32, 4>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 64)
    launch<DT, 32, 2>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 32 * kVecs)
    launch<DT, 32, 1>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 64 * kVecs)
    launch<DT, 64, 1>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 128 * kVecs)
    launch<DT, 128, 1>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 256 * kVecs)
    launch<DT, 256, 1>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else
    launch<DT, kMaxThreads, 1>(x, R, D, ld_x, codes, ld_c, scale, stream);
}

}  // namespace
}  // namespace rl

extern "C" rl_status rl_quantize_rows_int8(const void* x, rl_dtype dtype, long long R, long long D, long long ld_x,
                                           signed char* codes, long long ld_c, float* scale, void* stream) {
  using namespace rl;
  if (dtype != RL_F32 && dtype != RL_BF16 && dtype != RL_F16) return RL_ERR_DTYPE;
  const long long es = dtype == RL_F32 ? 4 : 2;
  if (R < 0 || R >= (1LL << 31) || D < 1 || D >= (1LL << 31) || ld_x < D || ld_c < D || ld_x >= (1LL << 40) ||
      ld_c >= (1LL << 40))
    return RL_ERR_SHAPE;
  if (R == 0) return RL_OK;
  if (!x || !codes || !scale) return RL_ERR_NULL;
  if (R > (1LL << 60) / (ld_x * es) || R > (1LL << 60) / ld_c) return RL_ERR_SHAPE;  // more than 64 bits address
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ca = reinterpret_cast<uintptr_t>(codes);
  if ((xa & 15) || (ca & 15) || ((ld_x * es) & 15) || (ld_c & 15) || (reinterpret_cast<uintptr_t>(scale) & 3)) return RL_ERR_ALIGN;
  const uintptr_t sa = reinterpret_cast<uintptr_t>(scale), x_end = xa + static_cast<uintptr_t>(((R - 1) * ld_x + D) * es),
                  c_end = ca + static_cast<uintptr_t>((R - 1) * ld_c + D), s_end = sa + static_cast<uintptr_t>(R * 4);
  if ((xa < c_end && ca < x_end) || (xa < s_end && sa < x_end) || (ca < s_end && sa < c_end)) return RL_ERR_ALIAS;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RL_F32)
    launch_rows<RL_F32>(x, R, D, ld_x, codes, ld_c, scale, s);
  else if (dtype == RL_BF16)
    launch_rows<RL_BF16>(x, R, D, ld_x, codes, ld_c, scale, s);
  else
    launch_rows<RL_F16>(x, R, D, ld_x, codes, ld_c, scale, s);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}
