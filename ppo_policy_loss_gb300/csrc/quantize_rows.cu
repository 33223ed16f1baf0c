// quantize_rows.cu — rl_quantize_rows_int8: 8-bit codes of a matrix's rows and
// a scale for each (include/rlrollout.h).
//
// One pass over the data: a row stays in its threads' registers between the
// maximum and the rounding (rows of more than kMaxThreads * kVecs vectors are read
// a second time, from L2).  Bound by HBM: an element is 2 or 4 bytes in and 1 out.
//
// The codes are those of the exact quotient x / s.  k = rint(x (1 / s)) is
// within one of it, and e = x - k s is exact in one FMA (|k| >= 1: a multiple
// of s's last place below 2^24 of them; k = 0: x itself), so 2 |e| against s
// says on which side of a half x lies.
#include <cuda_runtime.h>

#include <cstdint>

#include "rlrollout.h"
#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kVecs = 4;            // 16-byte vectors that a thread keeps
constexpr int kMaxThreads = 512;    // of one row
constexpr int kBlock = 256;         // threads of a CTA of short rows
constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer

struct RowScale {
  float s, s2, inv, up;  // the scale; what the codes are formed with: s2 = s up, inv = 1 / s2
};

__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.s = __fdiv_rn(amax, 127.f);
  if (!(r.s < INFINITY)) r.s = __int_as_float(0x7fc00000);
  r.up = r.s < 0x1p-100f ? 0x1p80f : 1.f;  // 1 / s overflows for the smallest
  r.s2 = r.s * r.up;
  r.inv = r.s > 0.f ? __fdiv_rn(1.f, r.s2) : 0.f;
  return r;
}

__device__ __forceinline__ int code_of(float x, const RowScale& r) {
  const float z = x * r.up;
  const float t = __fadd_rn(__fmul_rn(z, r.inv), kMagic);
  float k = __fsub_rn(t, kMagic);
  const float e = fmaf(-k, r.s2, z);
  const float e2 = fabsf(e + e);
  if (e2 >= r.s2 && (e2 > r.s2 || (__float_as_int(t) & 1))) k += copysignf(1.f, e);
  return static_cast<int>(fminf(fmaxf(k, -127.f), 127.f));
}

template <int DT>
__device__ __forceinline__ void load_vec(float (&z)[Fmt<DT>::kVec], const unsigned char* row, long long i, long long D) {
  using F = Fmt<DT>;
  if (i + F::kVec <= D) {
    F::unpack(*reinterpret_cast<const uint4*>(row + i * F::kBytes), z);
  } else {
#pragma unroll
    for (int j = 0; j < F::kVec; ++j) z[j] = i + j < D ? F::load(row, i + j) : 0.f;
  }
}

template <int DT>
__device__ __forceinline__ void store_codes(signed char* row, long long i, long long D, const float (&z)[Fmt<DT>::kVec],
                                            const RowScale& r) {
  using F = Fmt<DT>;
  uint32_t w[F::kVec / 4];
#pragma unroll
  for (int j = 0; j < F::kVec / 4; ++j) {
    w[j] = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) w[j] |= (static_cast<uint32_t>(code_of(z[4 * j + q], r)) & 0xffu) << (8 * q);
    if (!(r.s > 0.f)) w[j] = 0u;
  }
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

// TPR threads (a power of two of at least 32) take a row.
template <int DT, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
quantize_rows_kernel(const unsigned char* __restrict__ x, long long R, long long D, long long row_bytes,
                     signed char* __restrict__ codes, long long ld_c, float* __restrict__ scale) {
  using F = Fmt<DT>;
  constexpr int kRows = TPR > kBlock ? 1 : kBlock / TPR;
  constexpr int kWarps = TPR / 32;
  __shared__ float part[kRows][kWarps];
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const long long r = static_cast<long long>(blockIdx.x) * kRows + g;
  const bool here = r < R;
  const unsigned char* row = x + (here ? r : 0) * row_bytes;
  float z[kVecs][F::kVec];
  float amax = 0.f;
  if (here) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) load_vec<DT>(z[j], row, (static_cast<long long>(j) * TPR + t) * F::kVec, D);
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int q = 0; q < F::kVec; ++q) amax = max_nan(amax, fabsf(z[j][q]));
    for (long long i = (static_cast<long long>(kVecs) * TPR + t) * F::kVec; i < D; i += static_cast<long long>(TPR) * F::kVec) {
      float y[F::kVec];
      load_vec<DT>(y, row, i, D);
#pragma unroll
      for (int q = 0; q < F::kVec; ++q) amax = max_nan(amax, fabsf(y[q]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) part[g][t / 32] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = max_nan(amax, part[g][w]);
  }
  if (!here) return;
  const RowScale rs = row_scale(amax);
  if (t == 0) scale[r] = rs.s;
  signed char* out = codes + r * ld_c;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) store_codes<DT>(out, (static_cast<long long>(j) * TPR + t) * F::kVec, D, z[j], rs);
  for (long long i = (static_cast<long long>(kVecs) * TPR + t) * F::kVec; i < D; i += static_cast<long long>(TPR) * F::kVec) {
    float y[F::kVec];
    load_vec<DT>(y, row, i, D);
    store_codes<DT>(out, i, D, y, rs);
  }
}

template <int DT, int TPR>
void launch(const void* x, long long R, long long D, long long ld_x, signed char* codes, long long ld_c, float* scale,
            cudaStream_t stream) {
  constexpr int rows = TPR > kBlock ? 1 : kBlock / TPR;
  quantize_rows_kernel<DT, TPR><<<static_cast<unsigned>((R + rows - 1) / rows), rows * TPR, 0, stream>>>(
      static_cast<const unsigned char*>(x), R, D, ld_x * Fmt<DT>::kBytes, codes, ld_c, scale);
}

// as few threads as hold the row in their registers
template <int DT>
void launch_rows(const void* x, long long R, long long D, long long ld_x, signed char* codes, long long ld_c, float* scale,
                 cudaStream_t stream) {
  const long long vecs = (D + Fmt<DT>::kVec - 1) / Fmt<DT>::kVec;
  if (vecs <= 32 * kVecs)
    launch<DT, 32>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 64 * kVecs)
    launch<DT, 64>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 128 * kVecs)
    launch<DT, 128>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else if (vecs <= 256 * kVecs)
    launch<DT, 256>(x, R, D, ld_x, codes, ld_c, scale, stream);
  else
    launch<DT, kMaxThreads>(x, R, D, ld_x, codes, ld_c, scale, stream);
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
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ca = reinterpret_cast<uintptr_t>(codes);
  if ((xa & 15) || (ca & 15) || ((ld_x * es) & 15) || (ld_c & 15) || (reinterpret_cast<uintptr_t>(scale) & 3)) return RL_ERR_ALIGN;
  if (xa < ca + static_cast<uintptr_t>((R - 1) * ld_c + D) && ca < xa + static_cast<uintptr_t>(((R - 1) * ld_x + D) * es))
    return RL_ERR_ALIAS;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RL_F32)
    launch_rows<RL_F32>(x, R, D, ld_x, codes, ld_c, scale, s);
  else if (dtype == RL_BF16)
    launch_rows<RL_BF16>(x, R, D, ld_x, codes, ld_c, scale, s);
  else
    launch_rows<RL_F16>(x, R, D, ld_x, codes, ld_c, scale, s);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}
