// int8_logits.cu — rl_lmhead_logits_int8: the logits of an 8-bit LM head
// (include/rlrollout.h).
//
// Simple form: a CTA takes 64 tokens x 64 channels, 64 columns at a time in
// shared memory, and sums products of four codes at a time in 32-bit integers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rlrollout.h"

namespace rl {
namespace {

constexpr int kT = 64;       // tokens and channels of a tile, bytes of a step

template <class T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

template <class T>
__global__ void __launch_bounds__(256)
logits_int8_kernel(const signed char* __restrict__ h, long long ld_h, const float* __restrict__ sh,
                   const signed char* __restrict__ w, long long ld_w, const float* __restrict__ sw, long long R,
                   long long D, long long V, T* __restrict__ out, long long ld) {
  __shared__ int a[kT][kT / 4 + 1], b[kT][kT / 4 + 1];
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const long long v0 = static_cast<long long>(blockIdx.x) * kT, r0 = static_cast<long long>(blockIdx.y) * kT;
  int acc[4][4] = {};
  for (long long k = 0; k < D; k += kT) {
    for (int i = t; i < kT * kT / 4; i += 256) {
      const int row = i / (kT / 4), col = i % (kT / 4);
      int x = 0, y = 0;
      for (int j = 0; j < 4; ++j) {
        const long long d = k + col * 4 + j;
        if (d < D && r0 + row < R) x |= (h[(r0 + row) * ld_h + d] & 0xff) << (8 * j);
        if (d < D && v0 + row < V) y |= (w[(v0 + row) * ld_w + d] & 0xff) << (8 * j);
      }
      a[row][col] = x;
      b[row][col] = y;
    }
    __syncthreads();
    for (int c = 0; c < kT / 4; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a[ty * 4 + i][c], b[tx + 16 * j][c], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const long long r = r0 + ty * 4 + i, v = v0 + tx + 16 * j;
      if (r < R && v < V)
        out[r * ld + v] = rounded<T>(__fmul_rn(__fmul_rn(static_cast<float>(acc[i][j]), sh[r]), sw[v]));
    }
}

template <class T>
void launch(const signed char* h, long long ld_h, const float* sh, const signed char* w, long long ld_w, const float* sw,
            long long R, long long D, long long V, void* out, long long ld, cudaStream_t s) {
  for (long long r = 0; r < R; r += 65535LL * kT) {
    const long long n = R - r < 65535LL * kT ? R - r : 65535LL * kT;
    const dim3 grid(static_cast<unsigned>((V + kT - 1) / kT), static_cast<unsigned>((n + kT - 1) / kT));
    logits_int8_kernel<T><<<grid, 256, 0, s>>>(h + r * ld_h, ld_h, sh + r, w, ld_w, sw, n, D, V,
                                               static_cast<T*>(out) + r * ld, ld);
  }
}

bool shape_ok(long long R, long long D) { return R >= 0 && R < (1LL << 31) && D >= 1 && D <= RL_INT8_MAX_D; }

// Whether [x, x + nx) and [y, y + ny) share a byte.
bool overlap(const void* x, long long nx, const void* y, long long ny) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + static_cast<uintptr_t>(ny) && b < a + static_cast<uintptr_t>(nx);
}

}  // namespace
}  // namespace rl

extern "C" size_t rl_lmhead_int8_workspace_size(long long R, long long D) {
  using namespace rl;
  if (!shape_ok(R, D)) return 0;
  return (static_cast<size_t>(R) * static_cast<size_t>((D + 127) / 128 * 128) * 2 + 255) & ~size_t(255);
}

extern "C" rl_status rl_lmhead_logits_int8(const signed char* hidden, long long ld_h, const float* scale_h,
                                           const signed char* weight, long long ld_w, const float* scale_w,
                                           long long R, long long D, long long V, rl_dtype dtype, void* logits,
                                           long long ld, unsigned int* status_dev, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  using namespace rl;
  if (dtype != RL_F32 && dtype != RL_BF16 && dtype != RL_F16) return RL_ERR_DTYPE;
  const long long es = dtype == RL_F32 ? 4 : 2;
  if (!shape_ok(R, D) || V < 1 || V >= (1LL << 31) || ld_h < D || ld_w < D || ld < V || ld_h >= (1LL << 40) ||
      ld_w >= (1LL << 40) || ld >= (1LL << 40))
    return RL_ERR_SHAPE;
  if (R == 0) return RL_OK;
  if (!hidden || !weight || !scale_h || !scale_w || !logits) return RL_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(hidden) & 15) || (reinterpret_cast<uintptr_t>(weight) & 15) ||
      (reinterpret_cast<uintptr_t>(logits) & 15) || (reinterpret_cast<uintptr_t>(workspace) & 15) || (ld_h & 15) ||
      (ld_w & 15) || ((ld * es) & 15) || (reinterpret_cast<uintptr_t>(scale_h) & 3) ||
      (reinterpret_cast<uintptr_t>(scale_w) & 3))
    return RL_ERR_ALIGN;
  const long long out_bytes = ((R - 1) * ld + V) * es;
  if (overlap(logits, out_bytes, hidden, (R - 1) * ld_h + D) || overlap(logits, out_bytes, weight, (V - 1) * ld_w + D))
    return RL_ERR_ALIAS;
  if (!workspace || workspace_bytes < rl_lmhead_int8_workspace_size(R, D)) return RL_ERR_WORKSPACE;
  (void)status_dev;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RL_F32)
    launch<float>(hidden, ld_h, scale_h, weight, ld_w, scale_w, R, D, V, logits, ld, s);
  else if (dtype == RL_BF16)
    launch<__nv_bfloat16>(hidden, ld_h, scale_h, weight, ld_w, scale_w, R, D, V, logits, ld, s);
  else
    launch<__half>(hidden, ld_h, scale_h, weight, ld_w, scale_w, R, D, V, logits, ld, s);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}
