// token_logprobs.cu — rl_token_logprobs and rl_token_logprobs_bwd: the
// log-probabilities of given tokens with entropy and top alternatives, and
// their gradient, over logits in memory (sm_103a).
#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxPieces = 8192;  // pieces of a row one CTA can search for alternatives
constexpr int kMaxK = RL_TOKEN_MAX_K;
constexpr int kList = 256;        // survivors a search ranks directly

// ------------------------------------------------------------------ top-k search
// The K largest of n unique keys by one group of kRowThreads threads, sorted.
// Each thread takes the maximum of its keys (i * kRowThreads + tid); the K-th
// largest of nb >= 2 K bucket maxima is a bound that at least K keys reach
// and few others do; those that reach it are listed and ranked by counting.
// If more than kList reach it (keys in an order that puts the large ones on
// one thread), the bound is raised by bisection until exactly K do.
template <class K>
struct SelSmem {
  alignas(16) K a[kList];
  alignas(16) K b[kList];
  K bound;
  int count;
  int sums[2];
};

template <class K>
__device__ __forceinline__ int rank_of(const K* list, int n, K key) {
  int r = 0;
  for (int j = 0; j < n; ++j) r += list[j] > key;
  return r;
}

// get(i): key i (0 = none), i < n.  out[0 .. K-1]: the keys, largest first, 0
// where there are fewer.  All kRowThreads threads; ends with a barrier.
template <class K, class Get>
__device__ __forceinline__ void block_select(Get get, int n, int k, K* out, SelSmem<K>& s, int tid) {
  K best = 0;
  for (int i = tid; i < n; i += kRowThreads) {
    const K v = get(i);
    best = v > best ? v : best;
  }
  const int nb = k <= 16 ? 32 : k <= 32 ? 64 : k <= 64 ? 128 : 256;
  const int per = kRowThreads / nb;  // neighbouring lanes that share a bucket
  for (int o = 1; o < per; o <<= 1) {
    const K v = __shfl_xor_sync(0xffffffffu, best, o);
    best = v > best ? v : best;
  }
  if (tid % per == 0) s.a[tid / per] = best;
  if (tid == 0) {
    s.bound = 1;
    s.count = 0;
    s.sums[0] = s.sums[1] = 0;
  }
  if (tid < k) out[tid] = 0;
  __syncthreads();
  if (tid < nb && s.a[tid] != 0 && rank_of(s.a, nb, s.a[tid]) == k - 1) s.bound = s.a[tid];
  __syncthreads();
  K bound = s.bound;
  for (int i = tid; i < n; i += kRowThreads) {
    const K v = get(i);
    if (v >= bound) {
      const int p = atomicAdd(&s.count, 1);
      if (p < kList) s.b[p] = v;
    }
  }
  __syncthreads();
  int cnt = s.count;
  if (cnt > kList) {
    // bisection over the key's bits: the largest bound that k keys still reach
    K lo = bound, hi = ~static_cast<K>(0);
    for (int round = 0; lo < hi; ++round) {
      const K mid = lo + (hi - lo) / 2 + 1;
      int c = 0;
      for (int i = tid; i < n; i += kRowThreads) c += get(i) >= mid;
      c = __reduce_add_sync(0xffffffffu, c);
      if ((tid & 31) == 0 && c) atomicAdd(&s.sums[round & 1], c);
      __syncthreads();
      const int total = s.sums[round & 1];
      if (tid == 0) s.sums[(round + 1) & 1] = 0;
      __syncthreads();
      if (total >= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    if (tid == 0) s.count = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kRowThreads) {
      const K v = get(i);
      if (v >= lo) s.b[atomicAdd(&s.count, 1)] = v;  // keys are unique: exactly k reach it
    }
    __syncthreads();
    cnt = s.count;
  }
  if (tid < cnt) {
    const K v = s.b[tid];
    const int r = rank_of(s.b, cnt, v);
    if (r < k) out[r] = v;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ forward
struct LpArgs {
  const unsigned char* logits;
  const long long* ids;
  const unsigned char* mask;
  float* logp;
  float* entropy;
  float* lse;
  long long* topk_ids;
  float* topk_logp;
  unsigned int* status;
  long long R, V, row_bytes;
  float inv_temp, c;  // 1 / temperature, log2(e) / temperature
  int n_ids, k;
};

// The search key of a piece or an element: value key above position, so that
// the lower position wins a tie.  32 bits for 16-bit formats, 64 for fp32.
template <class V>
struct Composite;
template <>
struct Composite<uint16_t> {
  using K = uint32_t;
  __device__ static K make(uint16_t v, int pos) { return v ? (static_cast<K>(v) << 16) | (0xffffu - pos) : 0u; }
  __device__ static int pos(K k) { return static_cast<int>(0xffffu - (k & 0xffffu)); }
  __device__ static uint16_t value(K k) { return static_cast<uint16_t>(k >> 16); }
};
template <>
struct Composite<uint32_t> {
  using K = unsigned long long;
  __device__ static K make(uint32_t v, int pos) {
    return v ? (static_cast<K>(v) << 32) | (0xffffffffu - static_cast<uint32_t>(pos)) : 0ull;
  }
  __device__ static int pos(K k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }
  __device__ static uint32_t value(K k) { return static_cast<uint32_t>(k >> 32); }
};

template <int DT>
struct LpSmem {
  using F = Fmt<DT>;
  using C = Composite<typename F::Key>;
  alignas(16) typename F::Key keys[kMaxPieces];  // piece maxima, then the chosen pieces' elements
  SelSmem<typename C::K> sel;
  typename C::K top[kMaxK];
  int slots[kMaxK];
  RowStats part[kRowWarps];
};

__device__ __forceinline__ RowStats merge_parts(const RowStats* part, float c) {
  RowStats s = part[0];
#pragma unroll
  for (int w = 1; w < kRowWarps; ++w) s = merge_row(s, part[w], c);
  return s;
}

// A row whose maximum is at most kExact: its statistics without the floor, -inf elements skipped.
// Rare, so it reads the row again.  m = -inf: no element is finite.
template <class F>
__device__ __noinline__ RowStats exact_row(const unsigned char* row, int V, float c, RowStats* part, int tid) {
  float m = -INFINITY;
  for (int i = tid; i < V; i += kRowThreads) m = max_nan(m, F::load(row, i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();
  if ((tid & 31) == 0) part[tid >> 5].m = m;
  __syncthreads();
  for (int w = 0; w < kRowWarps; ++w) m = max_nan(m, part[w].m);
  __syncthreads();
  float s = 0.f, t = 0.f;
  if (m > -INFINITY)
    for (int i = tid; i < V; i += kRowThreads) {
      const float x = (F::load(row, i) - m) * c;
      const float e = ex2_approx(x);
      s += e;
      if (e > 0.f) t = fmaf(e, x, t);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  if ((tid & 31) == 0) part[tid >> 5] = RowStats{m, s, t};
  __syncthreads();
  s = t = 0.f;
  for (int w = 0; w < kRowWarps; ++w) {
    s += part[w].r;
    t += part[w].t;
  }
  return RowStats{m, s - 1.f, t};
}

template <int DT, bool kEntropy>
__global__ void __launch_bounds__(kRowThreads) token_logprobs_kernel(const LpArgs a) {
  using F = Fmt<DT>;
  using Key = typename F::Key;
  using C = Composite<Key>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  LpSmem<DT>& sm = *reinterpret_cast<LpSmem<DT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = static_cast<int>(a.V);
  const int n_pieces = (V + F::kPiece - 1) / F::kPiece;
  const int k = a.k, n_ids = a.n_ids;
  unsigned int err = 0;

  for (long long row = blockIdx.x; row < a.R; row += gridDim.x) {
    if (a.mask && a.mask[row] == 0) {
      if (tid < n_ids) a.logp[row * n_ids + tid] = 0.f;
      if (tid < k) {
        a.topk_ids[row * k + tid] = -1;
        a.topk_logp[row * k + tid] = 0.f;
      }
      if (tid == 0 && a.entropy) a.entropy[row] = 0.f;
      if (tid == 0 && a.lse) a.lse[row] = 0.f;
      continue;
    }
    const unsigned char* src = a.logits + row * a.row_bytes;
    long long y = -1;
    float zy = 0.f;
    if (tid < n_ids) {
      y = a.ids[row * n_ids + tid];
      if (y >= 0 && y < V) zy = F::load(src, y);
    }
    WarpStats st;
    warp_stats_init(st, F::kFloor, lane);
    for (int p0 = 0; p0 < n_pieces; p0 += kRowThreads) {
      const int p = p0 + tid;
      uint32_t w[16];
      const long long row_bytes16 = (static_cast<long long>(V) * F::kBytes + 15) & ~15LL;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long off = static_cast<long long>(p) * kPieceBytes + j * 16;
        uint4 v = make_uint4(F::kNegInf2, F::kNegInf2, F::kNegInf2, F::kNegInf2);
        if (off < row_bytes16) v = __ldg(reinterpret_cast<const uint4*>(src + off));
        w[4 * j] = v.x;
        w[4 * j + 1] = v.y;
        w[4 * j + 2] = v.z;
        w[4 * j + 3] = v.w;
      }
      if ((p + 1) * F::kPiece > V) F::cut(w, max(0, V - p * F::kPiece));
      const uint32_t rm = F::raw_max(w);
      if (k && p < n_pieces) sm.keys[p] = F::raw_key(rm);
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = F::clamp(w[i]);
      add_piece<F, kEntropy>(st, w, max_nan(F::raw_value(rm), F::kFloor), a.c, lane);
    }
    const RowStats ws = warp_stats_sum(st);
    if (lane == 0) sm.part[warp] = ws;
    __syncthreads();
    RowStats rs = merge_parts(sm.part, a.c);
    if (!(rs.m > F::kExact)) rs = exact_row<F>(src, V, a.c, sm.part, tid);
    const float log_s = log1pf(rs.r);
    if (tid < n_ids) {
      const bool ok = y >= 0 && y < V;
      if (!ok) err |= RL_DEVERR_ID_RANGE;
      a.logp[row * n_ids + tid] = ok ? fmaf(zy - rs.m, a.inv_temp, -log_s) : __int_as_float(0x7fc00000);
    }
    if (tid == 0) {
      if (a.lse) a.lse[row] = fmaf(rs.m, a.inv_temp, log_s);
      if (kEntropy && a.entropy)
        a.entropy[row] = rs.m > -INFINITY ? fmaf(-kLn2, rs.t / (1.f + rs.r), log_s) : __int_as_float(0x7fc00000);
    }
    if (k) {
      // the k pieces with the largest maxima hold the k largest elements
      int n_slots = n_pieces;
      const bool direct = n_pieces <= kMaxPieces / F::kPiece;  // every element fits the key array
      __syncthreads();
      if (!direct) {
        block_select<typename C::K>([&](int i) { return C::make(sm.keys[i], i); }, n_pieces, k, sm.top, sm.sel, tid);
        n_slots = k;
        if (tid < k) {  // back into the row's order
          const int g = C::pos(sm.top[tid]);
          int r = 0;
          for (int j = 0; j < k; ++j) r += C::pos(sm.top[j]) < g;
          sm.slots[r] = g;
        }
        __syncthreads();
      }
      for (int i = tid; i < n_slots * F::kPiece; i += kRowThreads) {
        const int e = (direct ? i / F::kPiece : sm.slots[i / F::kPiece]) * F::kPiece + i % F::kPiece;
        sm.keys[i] = e < V ? F::load_key(src, e) : Key(0);
      }
      __syncthreads();
      block_select<typename C::K>([&](int i) { return C::make(sm.keys[i], i); }, n_slots * F::kPiece, k, sm.top,
                                  sm.sel, tid);
      if (tid < k) {
        const typename C::K key = sm.top[tid];
        const int i = C::pos(key);
        const int e = (direct ? i / F::kPiece : sm.slots[i / F::kPiece]) * F::kPiece + i % F::kPiece;
        a.topk_ids[row * k + tid] = e;
        a.topk_logp[row * k + tid] = fmaf(F::key_value(C::value(key)) - rs.m, a.inv_temp, -log_s);
      }
    }
    __syncthreads();
  }
  if (err && a.status) atomicOr(a.status, err);
}

// ------------------------------------------------------------------ backward
struct LpBwdArgs {
  const unsigned char* logits;
  const long long* ids;
  const unsigned char* mask;
  const float* lse;
  const float* entropy;
  const float* dlogp;
  const float* dentropy;
  unsigned char* dlogits;
  unsigned int* status;
  long long R, V, row_bytes;
  float inv_temp;
  int n_ids;
  int n_seg;  // segments of a row
  long long seg_vecs;
};

// One unit is a segment of a row.  dz_v = 2^x (a0 + a1 x) with
// x = (z_v / T - lse) log2(e); the given ids' elements are computed once
// more and written after the segment's own stores.
template <int DT, bool kEntropy>
__global__ void __launch_bounds__(kRowThreads) token_logprobs_bwd_kernel(const LpBwdArgs a) {
  using F = Fmt<DT>;
  constexpr int kVec = F::kVec;
  __shared__ long long s_id[kMaxK];
  __shared__ float s_g[kMaxK];
  const int tid = threadIdx.x;
  const int V = static_cast<int>(a.V), n_ids = a.n_ids;
  const int n_vecs = (V + kVec - 1) / kVec;
  unsigned int err = 0;
  for (long long u = blockIdx.x; u < a.R * a.n_seg; u += gridDim.x) {
    const long long row = u / a.n_seg;
    const int v0 = static_cast<int>((u - row * a.n_seg) * a.seg_vecs);
    const int v1 = static_cast<int>(min(static_cast<long long>(n_vecs), v0 + a.seg_vecs));
    const unsigned char* src = a.logits + row * a.row_bytes;
    unsigned char* dst = a.dlogits + row * a.row_bytes;
    const bool on = !a.mask || a.mask[row] != 0;
    float a0 = 0.f, a1 = 0.f, lse = 0.f, zj = 0.f;
    long long idj = -1;
    bool mine = false;
    if (on) {
      lse = a.lse[row];
      if (tid < n_ids) {
        idj = a.ids[row * n_ids + tid];
        s_id[tid] = idj;
        s_g[tid] = a.dlogp[row * n_ids + tid];
        if (idj < 0 || idj >= V) err |= RL_DEVERR_ID_RANGE;
        mine = idj >= static_cast<long long>(v0) * kVec && idj < min(static_cast<long long>(V), static_cast<long long>(v1) * kVec);
        if (mine) zj = F::load(src, idj);
      }
      __syncthreads();
      float g = 0.f;
      for (int j = 0; j < n_ids; ++j) {
        g += s_g[j];
        if (s_id[j] < 0 || s_id[j] >= V) g = __int_as_float(0x7fc00000);
      }
      a0 = -g * a.inv_temp;
      if (kEntropy) {
        const float h = a.dentropy[row] * a.inv_temp;
        a0 = fmaf(-h, a.entropy[row], a0);
        a1 = -h * kLn2;
      }
    }
    auto grad = [&](float z) {
      float x = fmaf(z, a.inv_temp, -lse) * kLog2e;
      const float p = ex2_approx(x);
      if (!kEntropy) return p * a0;
      x = fmaxf(x, -1024.f);  // p is 0 there; 0 * -inf would not be
      return p * fmaf(a1, x, a0);
    };
    for (int v = v0 + tid; v < v1; v += kRowThreads) {
      float d[kVec];
      if (on) {
        F::unpack(*reinterpret_cast<const uint4*>(src + static_cast<long long>(v) * 16), d);
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[i] = grad(d[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[i] = 0.f;
      }
      if ((v + 1) * kVec <= V) {
        st_global_cs_v4(dst + static_cast<long long>(v) * 16, F::pack(d));
      } else {
        for (int i = 0; i < kVec; ++i)
          if (v * kVec + i < V) F::store(dst, v * kVec + i, d[i]);
      }
    }
    if (on && n_ids) {
      __syncthreads();  // the segment's stores come first
      if (mine) {
        float g = 0.f;
        for (int j = 0; j < n_ids; ++j)
          if (s_id[j] == idj) g += s_g[j];
        F::store(dst, idj, fmaf(g, a.inv_temp, grad(zj)));
      }
      __syncthreads();
    }
  }
  if (err && a.status) atomicOr(a.status, err);
}

// ------------------------------------------------------------------ host side
int elem_bytes(rl_dtype dt) { return dt == RL_F32 ? 4 : dt == RL_BF16 || dt == RL_F16 ? 2 : 0; }

bool temperature_ok(float t) { return std::isfinite(t) && t >= kMinTemperature && t <= kMaxTemperature; }

rl_status device_sms(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess || *sms < 1)
    return RL_ERR_CUDA;
  return RL_OK;
}

// The kernel's dynamic shared memory allowed once per device.
rl_status allow_smem(const void* fn, int dev, int smem) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, bool> done;
  std::lock_guard<std::mutex> lock(mu);
  bool& d = done[std::make_pair(fn, dev)];
  if (!d) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return RL_ERR_CUDA;
    d = true;
  }
  return RL_OK;
}

template <int DT, bool kEntropy>
rl_status launch_fwd(const LpArgs& a, int dev, int sms, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(&token_logprobs_kernel<DT, kEntropy>);
  const int smem = static_cast<int>(sizeof(LpSmem<DT>));
  const rl_status st = allow_smem(fn, dev, smem);
  if (st != RL_OK) return st;
  const long long want = 4LL * sms;
  token_logprobs_kernel<DT, kEntropy><<<static_cast<unsigned>(a.R < want ? a.R : want), kRowThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

template <int DT, bool kEntropy>
rl_status launch_bwd(const LpBwdArgs& a, int sms, cudaStream_t stream) {
  const long long units = a.R * a.n_seg, want = 8LL * sms;
  token_logprobs_bwd_kernel<DT, kEntropy><<<static_cast<unsigned>(units < want ? units : want), kRowThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

bool shape_ok(long long R, long long V, long long ld) {
  return R >= 0 && R < (1LL << 31) && V >= 1 && V <= (1LL << 30) && ld >= V && ld <= (1LL << 31);
}

}  // namespace
}  // namespace rl

extern "C" rl_status rl_token_logprobs(const void* logits, rl_dtype dtype, long long R, long long V, long long ld,
                                       const long long* ids, int n_ids, const unsigned char* mask,
                                       float temperature, int k, float* logp_out, float* entropy_out,
                                       float* lse_out, long long* topk_ids, float* topk_logp,
                                       unsigned int* status_dev, void* stream) {
  using namespace rl;
  const int es = elem_bytes(dtype);
  if (es == 0) return RL_ERR_DTYPE;
  if (!shape_ok(R, V, ld)) return RL_ERR_SHAPE;
  if (n_ids < 0 || n_ids > RL_TOKEN_MAX_K || k < 0 || k > RL_TOKEN_MAX_K || !temperature_ok(temperature))
    return RL_ERR_ARG;
  if (k > V || (k > 0 && V * es > static_cast<long long>(kMaxPieces) * kPieceBytes)) return RL_ERR_SHAPE;
  if (R == 0) return RL_OK;
  if (!logits || (n_ids > 0 && (!ids || !logp_out)) || (k > 0 && (!topk_ids || !topk_logp))) return RL_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(logits) & 15) || ((ld * es) & 15)) return RL_ERR_ALIGN;
  int dev = 0, sms = 0;
  const rl_status st = device_sms(&dev, &sms);
  if (st != RL_OK) return st;
  LpArgs a;
  a.logits = static_cast<const unsigned char*>(logits);
  a.ids = ids;
  a.mask = mask;
  a.logp = logp_out;
  a.entropy = entropy_out;
  a.lse = lse_out;
  a.topk_ids = topk_ids;
  a.topk_logp = topk_logp;
  a.status = status_dev;
  a.R = R;
  a.V = V;
  a.row_bytes = ld * es;
  a.inv_temp = 1.f / temperature;
  a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
  a.n_ids = n_ids;
  a.k = k;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ent = entropy_out != nullptr;
  switch (dtype) {
    case RL_F32: return ent ? launch_fwd<RL_F32, true>(a, dev, sms, s) : launch_fwd<RL_F32, false>(a, dev, sms, s);
    case RL_BF16: return ent ? launch_fwd<RL_BF16, true>(a, dev, sms, s) : launch_fwd<RL_BF16, false>(a, dev, sms, s);
    case RL_F16: return ent ? launch_fwd<RL_F16, true>(a, dev, sms, s) : launch_fwd<RL_F16, false>(a, dev, sms, s);
  }
  return RL_ERR_DTYPE;
}

extern "C" rl_status rl_token_logprobs_bwd(const void* logits, rl_dtype dtype, long long R, long long V,
                                           long long ld, const long long* ids, int n_ids,
                                           const unsigned char* mask, float temperature, const float* lse,
                                           const float* entropy, const float* dlogp, const float* dentropy,
                                           void* dlogits, unsigned int* status_dev, void* stream) {
  using namespace rl;
  const int es = elem_bytes(dtype);
  if (es == 0) return RL_ERR_DTYPE;
  if (!shape_ok(R, V, ld)) return RL_ERR_SHAPE;
  if (n_ids < 0 || n_ids > RL_TOKEN_MAX_K || !temperature_ok(temperature)) return RL_ERR_ARG;
  if (R == 0) return RL_OK;
  if (!logits || !dlogits || !lse || (n_ids > 0 && (!ids || !dlogp)) || ((entropy != nullptr) != (dentropy != nullptr)) ||
      (n_ids == 0 && !dentropy))
    return RL_ERR_NULL;
  const long long row_bytes = ld * es;
  if ((reinterpret_cast<uintptr_t>(logits) & 15) || (reinterpret_cast<uintptr_t>(dlogits) & 15) || (row_bytes & 15))
    return RL_ERR_ALIGN;
  if (dlogits != logits) {
    const uintptr_t l0 = reinterpret_cast<uintptr_t>(logits), d0 = reinterpret_cast<uintptr_t>(dlogits);
    const uintptr_t n = static_cast<uintptr_t>(R) * static_cast<uintptr_t>(row_bytes);
    if (l0 < d0 + n && d0 < l0 + n) return RL_ERR_ALIAS;
  }
  int dev = 0, sms = 0;
  const rl_status st = device_sms(&dev, &sms);
  if (st != RL_OK) return st;
  LpBwdArgs a;
  a.logits = static_cast<const unsigned char*>(logits);
  a.ids = ids;
  a.mask = mask;
  a.lse = lse;
  a.entropy = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.dlogits = static_cast<unsigned char*>(dlogits);
  a.status = status_dev;
  a.R = R;
  a.V = V;
  a.row_bytes = row_bytes;
  a.inv_temp = 1.f / temperature;
  a.n_ids = n_ids;
  const long long n_vecs = (V * es + 15) / 16;
  long long seg = (16LL * sms + R - 1) / R;  // enough units for every CTA
  const long long most = (n_vecs + 2 * kRowThreads - 1) / (2 * kRowThreads);
  if (seg > most) seg = most;
  a.seg_vecs = (n_vecs + seg - 1) / seg;
  a.n_seg = static_cast<int>((n_vecs + a.seg_vecs - 1) / a.seg_vecs);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ent = dentropy != nullptr;
  switch (dtype) {
    case RL_F32: return ent ? launch_bwd<RL_F32, true>(a, sms, s) : launch_bwd<RL_F32, false>(a, sms, s);
    case RL_BF16: return ent ? launch_bwd<RL_BF16, true>(a, sms, s) : launch_bwd<RL_BF16, false>(a, sms, s);
    case RL_F16: return ent ? launch_bwd<RL_F16, true>(a, sms, s) : launch_bwd<RL_F16, false>(a, sms, s);
  }
  return RL_ERR_DTYPE;
}
