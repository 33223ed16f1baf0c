// int8_logits.cu — rl_lmhead_logits_int8: the logits of an 8-bit LM head
// (include/rlrollout.h) on the 5th-generation tensor cores (sm_103a).
//
// The tensor cores take 8-bit integers at a fraction of their 16-bit rate
// here, and fp16 holds every code exactly, every product of two codes has 15 bits,
// and a sum of 1024 such products is at most 2^24: fp32 accumulation is exact over
// 1024 columns.  So the codes are widened to fp16 on their way to the tensor
// cores, and sums over more columns are taken 1024 at a time and added in
// 32-bit integers.  HBM sees 8-bit weights only.
//
//   logits^T tile [128 channels x N tokens] = W[128 x D] . hidden[N x D]^T
//
//   * widen_kernel writes the tokens' codes as fp16 into the workspace (R D
//     elements, 1 to 2 us beside a product that reads V D bytes).
//   * warps 0 and 2: TMA producers of two rings: 8-bit weight tiles (128
//     channels x 128 columns, 16 KB) and fp16 token tiles (N x 128 columns).
//     Where all columns of a single token tile fit (small batches), they are loaded once and stay.
//   * warps 4-7 and 12-15, step by step in turn: one channel a thread.  A 128-byte row of codes from shared memory, widened
//     in registers (4 codes: one XOR, two byte permutes to 1024 + code + 128,
//     two fp16 subtractions), and stored to tensor memory: the A operand of
//     tcgen05.mma comes from there, so that widened weights cost no
//     shared-memory traffic, which the token tiles already keep busy.
//   * warp 1: tcgen05.mma.kind::f16, M = 128, K = 16, into one of two
//     accumulators of N columns.
//   * warps 8-11: epilogue, a channel a lane: scales, rounding, and stores of
//     32 neighbouring channels of a token at a time.
//   * N is a multiple of 16 up to 192 (2 accumulators of 192 columns and two widened tiles
//     of 64 fill the 512 columns of tensor memory); 128 where sums stay in the epilogue's registers (D > 1024).
//   * What bounds it.  Few tokens: HBM (1 token, 151,936 x 1024: 30 us, of which 6.7 us are launches, the
//     first tiles and the last stores; what more channels add runs at 6.7 TB/s).  Many: shared memory, at 128 bytes a
//     cycle.  A step writes the token tile (2 N cycles) and reads it (2 N), writes the weight tile (128) and
//     reads it (128): 1024 cycles at N = 192, of which the MMA needs 768 and a step takes 1044 (4096 tokens:
//     750 to 870 us, 1.47 to 1.7 PFLOP/s).  That is why weights are widened into tensor memory.
//   * Every mbarrier wait is bounded; on timeout the kernel raises an error
//     flag, waits for its own copies and tensor-core work, writes NaN for what it has
//     not finished, frees its tensor memory and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "rlrollout.h"
#include "tc_device.cuh"

namespace rl {
namespace {

constexpr int kM = 128;                   // channels of a tile
constexpr int kStepK = 128;               // columns of a weight tile
constexpr int kBlockK = 64;               // columns of a token tile (fp16: 128 bytes)
constexpr int kExactK = 1024;             // columns that fp32 sums exactly
constexpr int kChunkSteps = kExactK / kStepK;
constexpr int kMaxN = 192, kMaxNDeep = 128;
constexpr uint32_t kTileA = kM * kStepK;  // 16 KB
constexpr uint32_t kTmemAll = 512;        // columns: two accumulators of N, then widened tiles of 64
constexpr int kWideCols = kStepK / 2;
constexpr int kMaxA = 12, kMaxB = 48, kMaxWide = 4;  // ring slots, widened tiles
constexpr int kMaxDone = 8;
constexpr uint32_t kRingBytes = 222 * 1024;
constexpr int kWidenThreads = 256;

struct Bars {
  unsigned long long full_a[kMaxA], empty_a[kMaxA];
  unsigned long long full_b[kMaxB];
  unsigned long long wide_full[kMaxWide];
  unsigned long long done[kMaxDone];
  unsigned long long acc_full[2], acc_empty[2];
  unsigned long long drain;
  uint32_t tmem_base;
  int abort;
  alignas(16) float scale[2][kMaxN + 32];  // of the tokens of the epilogue's unit
};

static_assert((static_cast<int>(kTmemAll) - 2 * kMaxN) / kWideCols >= 2, "two widened tiles at least");
static_assert(kRingBytes + 1024 + sizeof(Bars) <= 232448, "rings and barriers fit the 227 KB a CTA may use");

struct IArgs {
  long long R, V, ld;
  int n_tt, n_vt, group;  // token tiles, channel tiles, token tiles of a unit group
  int N;                  // tokens of a tile
  int steps;              // tiles along D
  int slots_a, slots_b, slots_w, slots_d;
  int resident;           // the token tiles are loaded once
  uint32_t idesc;
  const float* scale_h;
  const float* scale_w;
  void* out;
  unsigned int* status;
};

// A place in a ring of n slots, and the parity of its present round.  (Counted, not
// divided: a division by n is a hundred cycles of the one lane that feeds the tensor cores.)
struct Place {
  uint32_t i = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++i == n) {
      i = 0;
      parity ^= 1;
    }
  }
};

__device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, tc_wait<false>(bar, parity, abort));
}
// A whole warp's wait; the outcome is warp-uniform.  (Every lane looks: a lane that
// waits by itself, with the others held at the next warp-wide instruction or at the end of
// its role, makes the scheduler change between the two: a tile took 5.4 us, not 3.4.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_on(bar, parity, abort);
}

// Both of two, the second looked at after the first: no lane takes what it saw of the second
// for an answer unless it had seen the first pass.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t bar1, uint32_t parity1, volatile int* abort) {
  const bool first = mbar_try_wait(bar, parity), second = mbar_try_wait(bar1, parity1);
  if (__all_sync(0xffffffffu, first && second)) return true;
  return warp_wait_on(bar, parity, abort) && warp_wait_on(bar1, parity1, abort);
}

// One lane of the warp issues.  (The whole warp runs the loop around it, so that the
// compiler sees warp-uniform operands: from a single lane's registers each operand takes a
// move to the uniform ones, and an instruction 110 cycles instead of 46.)
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// 32 consecutive columns of this thread's TMEM lane; tmem_wait_ld() before they are used.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 32 consecutive columns of this thread's TMEM lane, written.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four 8-bit codes as fp16 numbers, exactly: 0x6400 | u is 1024 + u.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;  // code + 128
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// The tokens' codes as fp16, rows ld_f elements apart: 16 codes a thread.
__global__ void __launch_bounds__(kWidenThreads)
widen_kernel(const signed char* h, long long ld_h, long long R, long long D, unsigned char* f, long long ld_f) {
  // The launch before may still be at work; behind the wait it is not, and what depends on this one
  // may start: its weight tiles load while the codes are widened.  (No __restrict__: a load that
  // counts as one of constants might be moved before the wait.)
  grid_dependency_wait();
  allow_dependents();
  const long long per_row = (D + 15) / 16;
  const long long i = static_cast<long long>(blockIdx.x) * kWidenThreads + threadIdx.x;
  if (i >= R * per_row) return;
  const long long r = i / per_row, c = (i - r * per_row) * 16;
  // (the stride is a multiple of 16: the columns behind D are the caller's, and multiplied by nothing)
  uint32_t w[4], o[8];
  if (c + 16 <= D) {
    const uint4 v = *reinterpret_cast<const uint4*>(h + r * ld_h + c);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + 4 * j + q < D) w[j] |= (static_cast<uint32_t>(h[r * ld_h + c + 4 * j + q]) & 0xffu) << (8 * q);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) widen4(w[j], o[2 * j], o[2 * j + 1]);
  uint4* p = reinterpret_cast<uint4*>(f + (r * ld_f + c) * 2);
  p[0] = make_uint4(o[0], o[1], o[2], o[3]);
  p[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <class T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// Where a lane writes what it holds of 32 tokens.  Neighbouring lanes hold neighbouring
// channels: of 16-bit logits, lanes 2i and 2i + 1 exchange halves, so that the even one
// writes both channels of the even tokens and the odd one those of the odd tokens.
template <class T>
struct Rows {
  T* p;
  long long ld;
  int odd;
  int width;  // channels that this lane writes of a token
  __device__ __forceinline__ Rows(T* out, long long v, long long V, long long ld_, int lane) : ld(ld_) {
    if (sizeof(T) == 2) {
      odd = lane & 1;
      const long long v0 = v - odd;
      width = v0 + 1 < V ? 2 : v0 < V ? 1 : 0;
      p = out + odd * ld + v0;
    } else {
      odd = 0;
      width = v < V;
      p = out + v;
    }
  }
  __device__ __forceinline__ void next(int tokens) { p += tokens * ld; }
};

__device__ __forceinline__ uint32_t pack2(float x, float y, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float x, float y, __half) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The scaled sums of 32 tokens (of which there are n), rounded and stored.  All words are
// formed before the first store, and those of whole tiles are stored without a branch.
__device__ __forceinline__ void store32(const uint32_t (&x)[32], const float* scale, float sw, int n, const Rows<float>& to) {
  float w[32];
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 s = *reinterpret_cast<const float4*>(scale + i);
    w[i] = __fmul_rn(__fmul_rn(__uint_as_float(x[i]), s.x), sw);
    w[i + 1] = __fmul_rn(__fmul_rn(__uint_as_float(x[i + 1]), s.y), sw);
    w[i + 2] = __fmul_rn(__fmul_rn(__uint_as_float(x[i + 2]), s.z), sw);
    w[i + 3] = __fmul_rn(__fmul_rn(__uint_as_float(x[i + 3]), s.w), sw);
  }
  float* p = to.p;
  if (__all_sync(0xffffffffu, to.width == 1) && n >= 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i, p += to.ld) *p = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i, p += to.ld)
      if (to.width && i < n) *p = w[i];
  }
}
template <class T>
__device__ __forceinline__ void store32(const uint32_t (&x)[32], const float* scale, float sw, int n, const Rows<T>& to) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 s = *reinterpret_cast<const float4*>(scale + i);
    w[i / 2] = pack2(__fmul_rn(__fmul_rn(__uint_as_float(x[i]), s.x), sw), __fmul_rn(__fmul_rn(__uint_as_float(x[i + 1]), s.y), sw), T());
    w[i / 2 + 1] = pack2(__fmul_rn(__fmul_rn(__uint_as_float(x[i + 2]), s.z), sw), __fmul_rn(__fmul_rn(__uint_as_float(x[i + 3]), s.w), sw), T());
  }
  const uint32_t pick = to.odd ? 0x3276u : 0x5410u;  // own word, then the neighbour's: even the low halves, odd the high ones
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = __byte_perm(w[i], __shfl_xor_sync(0xffffffffu, w[i], 1), pick);
  T* p = to.p;
  if (__all_sync(0xffffffffu, to.width == 2) && n >= 32) {
#pragma unroll
    for (int i = 0; i < 16; ++i, p += 2 * to.ld) *reinterpret_cast<uint32_t*>(p) = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i, p += 2 * to.ld)
      if (2 * i + to.odd < n) {
        if (to.width == 2)
          *reinterpret_cast<uint32_t*>(p) = w[i];
        else if (to.width == 1)
          *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(w[i]);
      }
  }
}

// (Loops stay rolled: an unrolled role is a kilobyte of instructions that each call fetches
// from HBM, 1200 cycles a line, for the weights before it have swept them out of L2.)
// Threads of a CTA.  Warps 12-15 widen every other step, or where sums over many columns are
// kept in registers share the epilogue.
constexpr int kThreadsI = 512;
constexpr int kChunkN = 32;  // columns of an accumulator that an epilogue warp takes at a time

template <class T, bool kDeep>
__global__ void __launch_bounds__(kThreadsI, 1)
logits_int8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h, const IArgs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ Bars sm;
  const uint32_t ring_a = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring_b = ring_a + a.slots_a * kTileA, block_b = static_cast<uint32_t>(a.N) * 128u, tile_b = 2 * block_b;
  volatile int* abort_flag = &sm.abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int n_units = a.n_tt * a.n_vt, steps = a.steps, N = a.N;
  const uint32_t slots_a = a.slots_a, slots_b = a.slots_b, slots_w = a.slots_w, slots_d = a.slots_d;
  constexpr int kEpilogue = kDeep ? 8 : 4;  // epilogue warps
  constexpr int kGroups = kDeep ? 1 : 2;  // of four widening warps, which take the steps in turn

  if (tid == 0) {
    for (int s = 0; s < a.slots_a; ++s) {
      mbar_init(smem_addr(&sm.full_a[s]), 1);
      mbar_init(smem_addr(&sm.empty_a[s]), 4);
    }
    for (int s = 0; s < a.slots_b; ++s) mbar_init(smem_addr(&sm.full_b[s]), 1);
    for (int s = 0; s < a.slots_w; ++s) mbar_init(smem_addr(&sm.wide_full[s]), 4);
    for (int s = 0; s < a.slots_d; ++s) mbar_init(smem_addr(&sm.done[s]), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&sm.acc_full[s]), 1);
      mbar_init(smem_addr(&sm.acc_empty[s]), kEpilogue);
    }
    mbar_init(smem_addr(&sm.drain), 1);
    sm.abort = 0;
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_h)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&sm.tmem_base), kTmemAll);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0), wide = tmem + 2 * a.N;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer: weight tiles (whole warp)
    Place pa;
    uint32_t issued = 0;
    bool stop = false;
#pragma unroll 1
    for (int u = blockIdx.x; u < n_units && !stop; u += gridDim.x) {
      int tt, vt;
      unit_tile(u, a.n_tt, a.n_vt, a.group, tt, vt);
#pragma unroll 1
      for (int k = 0; k < steps; ++k, ++issued) {
        // (a barrier that has completed no phase passes a wait for the one before its first)
        if (!warp_wait(smem_addr(&sm.empty_a[pa.i]), pa.parity ^ 1, abort_flag)) {
          stop = true;
          break;
        }
        if (lane == 0) {
          const uint32_t fa = smem_addr(&sm.full_a[pa.i]);
          mbar_arrive_expect_tx(fa, kTileA);
          tma_load_2d(ring_a + pa.i * kTileA, &map_w, k * kStepK, vt * kM, fa);
        }
        __syncwarp();
        pa.next(slots_a);
      }
    }
    // copies already issued land before the CTA can exit, whoever gave up (else they have)
    for (uint32_t k = issued > slots_a ? issued - slots_a : 0; k < issued; ++k)
      tc_wait<true>(smem_addr(&sm.full_a[k % slots_a]), (k / slots_a) & 1, abort_flag);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- TMA producer: token tiles (whole warp)
    Place pb, pd;
    uint32_t issued = 0;
    bool stop = false;
    grid_dependency_wait();  // the workspace is written by the launch before this one
#pragma unroll 1
    for (int u = blockIdx.x; u < n_units && !stop; u += gridDim.x) {
      int tt, vt;
      unit_tile(u, a.n_tt, a.n_vt, a.group, tt, vt);
#pragma unroll 1
      for (int k = 0; k < steps; ++k, ++issued) {
        if (issued >= slots_b) {  // the step that used the slot last
          if (!warp_wait(smem_addr(&sm.done[pd.i]), pd.parity, abort_flag)) {
            stop = true;
            break;
          }
          pd.next(slots_d);
        }
        if (lane == 0) {
          const uint32_t fb = smem_addr(&sm.full_b[pb.i]), to = ring_b + pb.i * tile_b;
          mbar_arrive_expect_tx(fb, tile_b);
          tma_load_2d(to, &map_h, k * kStepK, tt * N, fb);
          tma_load_2d(to + block_b, &map_h, k * kStepK + kBlockK, tt * N, fb);
        }
        __syncwarp();
        pb.next(slots_b);
      }
      if (a.resident) break;
    }
    for (uint32_t k = issued > slots_b ? issued - slots_b : 0; k < issued; ++k)
      tc_wait<true>(smem_addr(&sm.full_b[k % slots_b]), (k / slots_b) & 1, abort_flag);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (whole warp)
    Place pw, pb, pc, pd;
    const uint32_t idesc = a.idesc;
    bool stop = false, issued = false, loaded = false;
#pragma unroll 1
    for (int u = blockIdx.x; u < n_units && !stop; u += gridDim.x) {
      int in_sum = 0;  // steps in the accumulator
#pragma unroll 1
      for (int k = 0; k < steps; ++k) {
        if (in_sum == 0 && !warp_wait(smem_addr(&sm.acc_empty[pc.i]), pc.parity ^ 1, abort_flag)) {
          stop = true;
          break;
        }
        if (!(loaded ? warp_wait(smem_addr(&sm.wide_full[pw.i]), pw.parity, abort_flag)
                     : warp_wait(smem_addr(&sm.full_b[pb.i]), pb.parity, smem_addr(&sm.wide_full[pw.i]), pw.parity, abort_flag))) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + pc.i * N, a_tmem = wide + pw.i * kWideCols;
        const uint64_t desc = smem_desc_sw128(ring_b + pb.i * tile_b), desc1 = desc + (block_b >> 4);
#pragma unroll
        for (int q = 0; q < kBlockK / 16; ++q) umma_f16_ts(d_tmem, a_tmem + q * 8, desc + q * 2, idesc, q | in_sum);
#pragma unroll
        for (int q = 0; q < kBlockK / 16; ++q) umma_f16_ts(d_tmem, a_tmem + kBlockK / 2 + q * 8, desc1 + q * 2, idesc, 1);
        issued = true;
        umma_commit_elect(smem_addr(&sm.done[pd.i]));  // frees the widened tile and the token tile
        pw.next(slots_w);
        pb.next(slots_b);
        pd.next(slots_d);
        if (++in_sum == kChunkSteps || k == steps - 1) {
          umma_commit_elect(smem_addr(&sm.acc_full[pc.i]));
          pc.next(2);
          in_sum = 0;
        }
      }
      loaded = a.resident;
    }
    if (issued) {  // every MMA, and every arrival that stands for one, is done before the CTA can exit
      umma_commit_elect(smem_addr(&sm.drain));
      tc_wait<true>(smem_addr(&sm.drain), 0, abort_flag);
    }
  } else if ((warp >= 4 && warp < 8) || (!kDeep && warp >= 12)) {
    // ---------------------------------------------------------------- widening
    const int q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    Place pa, pw, pd;
    const int turn = warp >= 12 ? 1 : 0;
    uint32_t ahead = slots_w, step = 0;  // ahead: tiles that no step has to free
    bool stop = false;
#pragma unroll 1
    for (int u = blockIdx.x; u < n_units && !stop; u += gridDim.x) {
#pragma unroll 1
      for (int k = 0; k < steps; ++k, ++step) {
        if (kGroups == 2 && static_cast<int>(step & 1) != turn) {
          if (ahead > 0)
            --ahead;
          else
            pd.next(slots_d);
          pa.next(slots_a);
          pw.next(slots_w);
          continue;
        }
        // done before full_a: this group has not watched the other's steps, and tiles land in
        // any order.  A barrier whose phase before the awaited one is still open passes a wait
        // for the one to come; that step - slots_w is done says that this step's slot, last filled
        // at step - slots_a <= step - slots_w, has had that tile land.  (done itself is two
        // steps behind a done that this group waited for, and slots_d >= 2.)
        bool ok;
        if (ahead > 0) {
          --ahead;
          ok = warp_wait(smem_addr(&sm.full_a[pa.i]), pa.parity, abort_flag);
        } else {
          ok = warp_wait(smem_addr(&sm.done[pd.i]), pd.parity, smem_addr(&sm.full_a[pa.i]), pa.parity, abort_flag);
          pd.next(slots_d);
        }
        if (!ok) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t base = ring_a + pa.i * kTileA + row * 128, to = wide + pw.i * kWideCols + lane_addr;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t o[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 v = ld_shared_v4(base + (((half * 4 + c) ^ (row & 7)) << 4));
            widen4(v.x, o[8 * c], o[8 * c + 1]);
            widen4(v.y, o[8 * c + 2], o[8 * c + 3]);
            widen4(v.z, o[8 * c + 4], o[8 * c + 5]);
            widen4(v.w, o[8 * c + 6], o[8 * c + 7]);
          }
          tmem_st32(to + half * 32, o);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&sm.wide_full[pw.i]));
          mbar_arrive(smem_addr(&sm.empty_a[pa.i]));
        }
        pa.next(slots_a);
        pw.next(slots_w);
      }
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    Place pc;
    const int group = (warp - 8) >> 2, me = tid - 8 * 32;
    uint32_t parity = 0;
    bool stop = false;
    const int n_chunks = (a.steps + kChunkSteps - 1) / kChunkSteps;
    constexpr int kMine = (kMaxN + kEpilogue * 32 - 1) / (kEpilogue * 32);
    float mine[kMine];  // scales of the unit's tokens me, me + 32 kEpilogue
    const auto load_scales = [&](int u) {
      int tt, vt;
      unit_tile(u, a.n_tt, a.n_vt, a.group, tt, vt);
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int i = me + j * kEpilogue * 32;
        const long long r = static_cast<long long>(tt) * N + i;
        mine[j] = i < N && r < a.R ? __ldg(a.scale_h + r) : 0.f;
      }
    };
    if (static_cast<int>(blockIdx.x) < n_units) load_scales(blockIdx.x);
#pragma unroll 1
    for (int u = blockIdx.x; u < n_units; u += gridDim.x, parity ^= 1) {
      int tt, vt;
      unit_tile(u, a.n_tt, a.n_vt, a.group, tt, vt);
      const long long v = static_cast<long long>(vt) * kM + row, r0 = static_cast<long long>(tt) * N;
      const int n = static_cast<int>(min(static_cast<long long>(N), a.R - r0));
      const bool here = v < a.V;
      const float sw = here ? a.scale_w[v] : 0.f;
      T* out = static_cast<T*>(a.out) + r0 * a.ld + v;
      // the tokens' scales, in turn in two places: the barrier keeps the warps within a unit of
      // one another.  The next unit's are on their way while this one's are used.
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        if (me + j * kEpilogue * 32 < N) sm.scale[parity][me + j * kEpilogue * 32] = mine[j];
      named_barrier(1, kEpilogue * 32);
      if (u + static_cast<int>(gridDim.x) < n_units) load_scales(u + gridDim.x);
      Rows<T> to(static_cast<T*>(a.out) + (r0 + group * kChunkN) * a.ld, v, a.V, a.ld, lane);
      int sum[kDeep ? kMaxNDeep / 2 : 1];  // deep: chunks of 32 tokens go to the two groups of warps in turn
#pragma unroll 1
      for (int ch = 0; ch < n_chunks; ++ch) {
        stop = stop || !warp_wait(smem_addr(&sm.acc_full[pc.i]), pc.parity, abort_flag);
        if (stop) break;
        tc_fence_after();
        const uint32_t from = tmem + lane_addr + pc.i * N;
        if (kDeep) {
#pragma unroll
          for (int c = 0; c < kMaxNDeep / 64; ++c) {
            const int col = (2 * c + group) * kChunkN;
            if (col < N) {
              uint32_t x[32];
              tmem_ld32_issue(from + col, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                sum[c * 32 + i] = __float2int_rn(__uint_as_float(x[i])) + (ch > 0 ? sum[c * 32 + i] : 0);
            }
          }
        } else {
          const float* scale = sm.scale[parity];
          uint32_t x[2][32];  // (columns behind N: what lies there, and goes nowhere)
          tmem_ld32_issue(from, x[0]);
#pragma unroll 1
          for (int c = 0; c < N; c += 2 * kChunkN) {
            tmem_wait_ld();
            if (c + kChunkN < N) tmem_ld32_issue(from + c + kChunkN, x[1]);
            store32(x[0], scale + c, sw, n - c, to);
            to.next(kChunkN);
            if (c + kChunkN >= N) break;
            tmem_wait_ld();
            if (c + 2 * kChunkN < N) tmem_ld32_issue(from + c + 2 * kChunkN, x[0]);
            store32(x[1], scale + c + kChunkN, sw, n - c - kChunkN, to);
            to.next(kChunkN);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.acc_empty[pc.i]));
        pc.next(2);
      }
      if (stop) {  // not known to be right
        for (int t = 0; t < n; ++t)
          if (here) out[t * a.ld] = rounded<T>(__int_as_float(0x7fc00000));
      } else if (kDeep) {
#pragma unroll
        for (int c = 0; c < kMaxNDeep / 64; ++c) {
          const int col = (2 * c + group) * kChunkN;
          if (col < N) {
            uint32_t x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(static_cast<float>(sum[c * 32 + i]));
            store32(x, sm.scale[parity] + col, sw, n - col, to);
            to.next(2 * kChunkN);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0 && a.status) atomicOr(a.status, RL_DEVERR_TIMEOUT);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

// ------------------------------------------------------------------ host side
bool shape_ok(long long R, long long D) { return R >= 0 && R < (1LL << 31) && D >= 1 && D <= RL_INT8_MAX_D; }

// Row stride of the widened codes, in elements.
long long wide_ld(long long D) { return (D + kBlockK - 1) / kBlockK * kBlockK; }

// Whether [x, x + nx) and [y, y + ny) share a byte.
bool overlap(const void* x, long long nx, const void* y, long long ny) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + static_cast<uintptr_t>(ny) && b < a + static_cast<uintptr_t>(nx);
}

// Token tiles that the CTAs working at one time may touch: about 40 MB of L2.
constexpr long long kTokenL2Bytes = 40LL << 20;

struct IPlan {
  int n_tt, n_vt, group, N, steps, slots_a, slots_b, slots_w, slots_d, resident;
};

IPlan int8_plan(long long R, long long D, long long V) {
  IPlan p;
  const int most = D > kExactK ? kMaxNDeep : kMaxN;
  p.n_tt = static_cast<int>((R + most - 1) / most);
  const long long each = (R + p.n_tt - 1) / p.n_tt;
  p.N = static_cast<int>((each + 15) / 16 * 16);
  p.n_tt = static_cast<int>((R + p.N - 1) / p.N);
  p.n_vt = static_cast<int>((V + kM - 1) / kM);
  p.steps = static_cast<int>((D + kStepK - 1) / kStepK);
  const long long tile_b = static_cast<long long>(p.N) * 256, ring = kRingBytes;
  // weights in flight are what a small batch waits for: at least 80 KB of them beside resident tokens
  p.resident = p.n_tt == 1 && p.steps <= kMaxB && p.steps * tile_b + 5 * static_cast<long long>(kTileA) <= ring;
  if (p.resident) {
    p.slots_b = p.steps;
    const long long room = (ring - p.steps * tile_b) / kTileA;
    p.slots_a = static_cast<int>(room < kMaxA ? room : kMaxA);
  } else {
    p.slots_a = kMaxWide;
    const long long room = (ring - p.slots_a * static_cast<long long>(kTileA)) / tile_b;
    p.slots_b = static_cast<int>(room < kMaxDone ? room : kMaxDone);
  }
  const int wide = (static_cast<int>(kTmemAll) - 2 * p.N) / kWideCols;
  p.slots_w = wide < kMaxWide ? wide : kMaxWide;  // 2 to 4, and never more than slots_a: the widening warps' waits need both
  p.slots_d = p.resident || p.slots_w > p.slots_b ? p.slots_w : p.slots_b;
  const long long g = kTokenL2Bytes / (static_cast<long long>(p.N) * wide_ld(D) * 2);
  p.group = static_cast<int>(g < 1 ? 1 : (g > p.n_tt ? p.n_tt : g));
  return p;
}

// 2-D tensor map of bytes over [rows, cols], box 128 x 128, 128-byte swizzle, zeros outside.
bool byte_map(EncodeTiled enc, CUtensorMap* map, const void* base, long long rows, long long cols, long long ld) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kStepK, kM};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's dynamic shared memory allowed, once per device (a bit each).
template <class T, bool kDeep>
rl_status launch(const CUtensorMap& map_w, const CUtensorMap& map_h, const IArgs& a, int grid, int dev, cudaStream_t s) {
  constexpr int smem = kRingBytes + 1024;
  static std::atomic<unsigned long long> allowed{0};
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(logits_int8_kernel<T, kDeep>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return RL_ERR_CUDA;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreadsI);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the weight's first tiles load while the codes are widened
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logits_int8_kernel<T, kDeep>, map_w, map_h, a) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

template <class T>
rl_status launch_any(const CUtensorMap& map_w, const CUtensorMap& map_h, const IArgs& a, int grid, int dev, cudaStream_t s) {
  return a.steps > kChunkSteps ? launch<T, true>(map_w, map_h, a, grid, dev, s) : launch<T, false>(map_w, map_h, a, grid, dev, s);
}

}  // namespace
}  // namespace rl

extern "C" size_t rl_lmhead_int8_workspace_size(long long R, long long D) {
  using namespace rl;
  if (!shape_ok(R, D)) return 0;
  return (static_cast<size_t>(R) * static_cast<size_t>(wide_ld(D)) * 2 + 255) & ~size_t(255);
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
  const IPlan p = int8_plan(R, D, V);
  const long long units = static_cast<long long>(p.n_tt) * p.n_vt;
  if (units > (1LL << 30)) return RL_ERR_SHAPE;
  if (!hidden || !weight || !scale_h || !scale_w || !logits) return RL_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(hidden) & 15) || (reinterpret_cast<uintptr_t>(weight) & 15) ||
      (reinterpret_cast<uintptr_t>(logits) & 15) || (reinterpret_cast<uintptr_t>(workspace) & 15) || (ld_h & 15) ||
      (ld_w & 15) || ((ld * es) & 15) || (reinterpret_cast<uintptr_t>(scale_h) & 3) ||
      (reinterpret_cast<uintptr_t>(scale_w) & 3))
    return RL_ERR_ALIGN;
  if (R > (1LL << 60) / (ld * es) || R > (1LL << 60) / ld_h || V > (1LL << 60) / ld_w) return RL_ERR_SHAPE;  // more than 64 bits address
  const long long out_bytes = ((R - 1) * ld + V) * es;
  if (overlap(logits, out_bytes, hidden, (R - 1) * ld_h + D) || overlap(logits, out_bytes, weight, (V - 1) * ld_w + D))
    return RL_ERR_ALIAS;
  const size_t scratch = rl_lmhead_int8_workspace_size(R, D);
  if (!workspace || workspace_bytes < scratch) return RL_ERR_WORKSPACE;
  const long long taken = static_cast<long long>(scratch);
  if (overlap(workspace, taken, logits, out_bytes) || overlap(workspace, taken, hidden, (R - 1) * ld_h + D) ||
      overlap(workspace, taken, weight, (V - 1) * ld_w + D) || overlap(workspace, taken, scale_h, R * 4) || overlap(workspace, taken, scale_w, V * 4) ||
      overlap(logits, out_bytes, scale_h, R * 4) || overlap(logits, out_bytes, scale_w, V * 4))
    return RL_ERR_ALIAS;
  EncodeTiled enc = nullptr;
  int dev = 0, sms = 0;
  if (tc_encode_fn(&enc) != RL_OK || cudaGetDevice(&dev) != cudaSuccess || tc_device_sms(&sms) != RL_OK) return RL_ERR_CUDA;
  const long long ldw = wide_ld(D);
  CUtensorMap map_w, map_h;
  if (!byte_map(enc, &map_w, weight, V, D, ld_w) ||
      !tc_make_map(enc, &map_h, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, workspace, R, D, ldw, kBlockK, p.N))
    return RL_ERR_CUDA;
  IArgs a;
  a.R = R;
  a.V = V;
  a.ld = ld;
  a.n_tt = p.n_tt;
  a.n_vt = p.n_vt;
  a.group = p.group;
  a.N = p.N;
  a.steps = p.steps;
  a.slots_a = p.slots_a;
  a.slots_b = p.slots_b;
  a.slots_w = p.slots_w;
  a.slots_d = p.slots_d;
  a.resident = p.resident;
  a.idesc = make_idesc_f16(false, kM, p.N, false, false);
  a.scale_h = scale_h;
  a.scale_w = scale_w;
  a.out = logits;
  a.status = status_dev;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long pieces = R * ((D + 15) / 16);
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((pieces + kWidenThreads - 1) / kWidenThreads));
  cfg.blockDim = dim3(kWidenThreads);
  cfg.stream = s;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, widen_kernel, hidden, ld_h, R, D, static_cast<unsigned char*>(workspace), ldw) != cudaSuccess) return RL_ERR_CUDA;
  const int grid = static_cast<int>(units < sms ? units : sms);
  if (dtype == RL_F32) return launch_any<float>(map_w, map_h, a, grid, dev, s);
  if (dtype == RL_BF16) return launch_any<__nv_bfloat16>(map_w, map_h, a, grid, dev, s);
  return launch_any<__half>(map_w, map_h, a, grid, dev, s);
}
