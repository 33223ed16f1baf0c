// verify_drafts.cu — rl_verify_drafts: which drafted tokens a sequence keeps,
// and the token drawn after them (include/rlrollout.h).
//
// A CTA takes a sequence.
//  1. Its target rows in order, until a draft does not stay: maximum and sum of
//     e^((z - m) / T) of the row in one pass, fp32, online.  The maxima, whose
//     terms are exactly 1, are counted beside the sum, so that log S keeps its
//     relative precision where one token holds nearly all the mass.
//  2. The weights of the row that the token is drawn from, in fine arithmetic (fine_exp.cuh),
//     summed for each warp's part of the row: the row's own softmax, and where a
//     draft with a distribution was refused, in a second pass max(p S - q S, 0).
//  3. The part in which the running sum passes the border is split again among
//     the warps, until one warp walks through what is left.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "fine_exp.cuh"
#include "rlrollout.h"
#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr double kLog2eD = 1.4426950408889634074;

struct Args {
  const unsigned char* target;
  const unsigned char* draft;
  const float* draft_lse;
  const long long* ids;
  const int* n_draft;
  const double* u;
  long long V, row_bytes, draft_bytes;
  int G;
  float c;       // log2(e) / temperature
  double c_d, inv_t;
  long long* tokens;
  long long* n_accepted;
  float* logp;
  float* lse;
  unsigned int* status;
};

// Which weights a token is drawn from.
enum Mode { kSoftmax, kWithout, kRest };  // p; p without the drafted token; max(p - q, 0)

// Maximum, how many hold it, and the sum of 2^((z - m) c) of the rest.
struct Stats {
  float m, n, s;
};

__device__ __forceinline__ Stats merged(Stats a, Stats b, float c) {
  if (!(a.m >= b.m)) {  // (a NaN becomes the result's maximum)
    const Stats x = a;
    a = b;
    b = x;
  }
  if (a.m == b.m) {
    a.n += b.n;
    a.s += b.s;
  } else {
    a.s = fmaf(b.n + b.s, ex2_approx((b.m - a.m) * c), a.s);
    a.m = max_nan(a.m, b.m);
  }
  return a;
}

struct Smem {
  float T[kPow], delta[kPow];
  Stats part[kWarps];
  double sums[kWarps];
  double log2_total;
  long long found;
  int verdict;  // of a row's draft
};

enum Verdict { kStays, kRefused, kNoDistribution };

// log p of logit z of a row.
__device__ __forceinline__ float log_prob(float z, const Stats& st, double inv_t) {
  return static_cast<float>((static_cast<double>(z) - static_cast<double>(st.m)) * inv_t - log1pf((st.n - 1.f) + st.s));
}

template <int DT>
__device__ __forceinline__ void load_elems(float (&z)[Fmt<DT>::kVec], const unsigned char* row, long long i, long long end) {
  using F = Fmt<DT>;
  // (16 bytes at a time: the stride is a multiple of that, what lies behind the row is dropped)
  F::unpack(__ldg(reinterpret_cast<const uint4*>(row + i * F::kBytes)), z);
  if (i + F::kVec > end) {
#pragma unroll
    for (int j = 0; j < F::kVec; ++j)
      if (i + j >= end) z[j] = -INFINITY;
  }
}

template <int DT>
__device__ __forceinline__ Stats row_stats(const unsigned char* row, long long V, float c, Smem& sm) {
  using F = Fmt<DT>;
  Stats a{-FLT_MAX, 0.f, 0.f};
  for (long long i = static_cast<long long>(threadIdx.x) * F::kVec; i < V; i += static_cast<long long>(kThreads) * F::kVec) {
    float z[F::kVec];
    load_elems<DT>(z, row, i, V);
    float vm = z[0];
#pragma unroll
    for (int j = 1; j < F::kVec; ++j) vm = max_nan(vm, z[j]);
    if (!(vm < a.m)) {
      if (!(vm == a.m)) {
        a.s = (a.n + a.s) * ex2_approx((a.m - vm) * c);
        a.n = 0.f;
        a.m = max_nan(a.m, vm);
      }
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) {
        if (z[j] == a.m) {
          a.n += 1.f;
          z[j] = -INFINITY;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < F::kVec; ++j) a.s += ex2_approx((z[j] - a.m) * c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merged(a, Stats{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.n, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, c);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.part[threadIdx.x >> 5] = a;
  __syncthreads();
  a = sm.part[0];
  for (int w = 1; w < kWarps; ++w) a = merged(a, sm.part[w], c);
  return a;
}

// The weights of one row.
template <int DT, int MODE>
struct Weights {
  const unsigned char* row;
  const unsigned char* draft_row;
  long long V, without;
  FineExp p, q;
  const float* T;
  const float* delta;
  bool bad;

  // weights of elements i .. i + kVec - 1
  __device__ __forceinline__ void at(long long i, long long end, Term (&w)[Fmt<DT>::kVec]) {
    using F = Fmt<DT>;
    constexpr bool wide = DT == RL_F32;
    float z[F::kVec];
    load_elems<DT>(z, row, i, end);
    if (MODE == kWithout && without >= i && without < i + F::kVec) {
#pragma unroll
      for (int j = 0; j < F::kVec; ++j)
        if (i + j == without) z[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < F::kVec; ++j) w[j] = p.template at<wide>(z[j], T, delta);
    if (MODE == kRest) {
      load_elems<DT>(z, draft_row, i, end);
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) {
        bad = bad || !(z[j] < INFINITY);
        w[j] = minus(w[j], q.template at<wide>(z[j], T, delta));
        if (!(w[j].a + w[j].b + w[j].c > 0.f)) w[j].a = w[j].b = w[j].c = 0.f;
      }
    }
  }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// [lo, hi) of part w of n parts of [begin, end): multiples of `step` long
__device__ __forceinline__ long long part_size(long long length, int n, int step) {
  return ((length + n - 1) / n + step - 1) / step * step;
}

// The warp's sum over [lo, hi), whole vectors from lo.
template <int DT, int MODE>
__device__ __forceinline__ double part_sum(Weights<DT, MODE>& f, long long lo, long long hi, int lane) {
  using F = Fmt<DT>;
  double total = 0.0;
  FineSum s;
  s.clear();
  int n = 0;
  for (long long i = lo + lane * F::kVec; i < hi; i += 32 * F::kVec) {
    Term w[F::kVec];
    f.at(i, hi, w);
#pragma unroll
    for (int j = 0; j < F::kVec; ++j) s.add(w[j]);
    if (++n == 128 / F::kVec) {
      total += s.value();
      s.clear();
      n = 0;
    }
  }
  return warp_sum(total + s.value());
}

// Sums of the CTA's warps over their parts of [begin, end); the total.
template <int DT, int MODE>
__device__ __forceinline__ double all_parts(Weights<DT, MODE>& f, long long begin, long long end, Smem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long size = part_size(end - begin, kWarps, 32 * Fmt<DT>::kVec);
  const long long lo = min(end, begin + warp * size), hi = min(end, lo + size);
  const double s = part_sum<DT, MODE>(f, lo, hi, lane);
  __syncthreads();
  if (lane == 0) sm.sums[warp] = s;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < kWarps; ++w) total += sm.sums[w];
  return total;
}

// The first token at which the running sum exceeds u times the total of sm.sums, whose parts are those of [0, V).
template <int DT, int MODE>
__device__ __forceinline__ long long search(Weights<DT, MODE>& f, double want, Smem& sm) {
  using F = Fmt<DT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long begin = 0, end = f.V;
  while (true) {
    // the part that holds the border; past the last weight (a rounding), the last part that has any
    const long long size = part_size(end - begin, kWarps, 32 * F::kVec);
    double before = 0.0, last_before = 0.0;
    int at = -1, last = 0;
    for (int w = 0; w < kWarps; ++w) {
      const double s = sm.sums[w];
      if (s > 0.0) {
        last = w;
        last_before = before;
        if (before + s > want) {
          at = w;
          break;
        }
      }
      before += s;
    }
    if (at < 0) {
      at = last;
      before = last_before;
    }
    want -= before;
    begin = min(end, begin + at * size);
    end = min(end, begin + size);
    if (end - begin <= 4 * 32 * F::kVec) break;
    all_parts<DT, MODE>(f, begin, end, sm);
  }
  __syncthreads();
  if (warp == 0) {
    long long found = -1, last = -1;
    for (long long base = begin; base < end && found < 0; base += 32 * F::kVec) {
      const long long i = base + lane * F::kVec;
      Term w[F::kVec];
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) w[j].a = w[j].b = w[j].c = 0.f;
      if (i < end) f.at(i, end, w);
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) sum += w[j].value();
      double upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      double run = __shfl_up_sync(0xffffffffu, upto, 1);
      if (lane == 0) run = 0.0;
      long long mine = -1, mine_last = -1;
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) {
        const double x = w[j].value();
        run += x;
        if (x > 0.0) {
          mine_last = i + j;
          if (mine < 0 && run > want) mine = i + j;
        }
      }
      const uint32_t who = __ballot_sync(0xffffffffu, mine >= 0);
      if (who) found = __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
      const uint32_t some = __ballot_sync(0xffffffffu, mine_last >= 0);
      if (some) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(some));
      want -= __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) sm.found = found >= 0 ? found : last;
  }
  __syncthreads();
  return sm.found;
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
verify_drafts_kernel(const Args a) {
  using F = Fmt<DT>;
  constexpr bool wide = DT == RL_F32;
  __shared__ Smem sm;
  const long long b = blockIdx.x;
  const int tid = threadIdx.x, G = a.G;
  const long long V = a.V, rows = static_cast<long long>(G) + 1;
  long long* tokens = a.tokens + b * rows;
  float* logp = a.logp ? a.logp + b * rows : nullptr;
  float* lse = a.lse ? a.lse + b * rows : nullptr;
  const float nan = __int_as_float(0x7fc00000);
  if (tid < kPow) {
    sm.T[tid] = kPowT[tid];
    sm.delta[tid] = kPowD[tid];
  }
  const int n = a.n_draft ? a.n_draft[b] : G;
  bool wrong = n < -1 || n > G;
  if (!wrong)
    for (int i = tid; i < n; i += kThreads) wrong = wrong || a.ids[b * G + i] < 0 || a.ids[b * G + i] >= V;
  wrong = __syncthreads_or(wrong);
  if (wrong || n < 0) {
    for (int i = tid; i <= G; i += kThreads) {
      tokens[i] = -1;
      if (logp) logp[i] = wrong ? nan : 0.f;
      if (lse) lse[i] = wrong ? nan : 0.f;
    }
    if (tid == 0) {
      if (a.n_accepted) a.n_accepted[b] = 0;
      if (wrong && a.status) atomicOr(a.status, RL_DEVERR_ID_RANGE);
    }
    return;
  }

  FineExp fp;
  int kept = 0;
  Stats st;
  bool lost = false, bad = false;
  const unsigned char* row = nullptr;
  for (int i = 0;; ++i) {
    row = a.target + (b * rows + i) * a.row_bytes;
    st = row_stats<DT>(row, V, a.c, sm);
    bad = !(fabsf(st.m) < INFINITY) || !(st.n > 0.f);
    fp.init(a.c_d, st.m, 0.0);
    if (tid == 0 && lse) lse[i] = bad ? nan : static_cast<float>(static_cast<double>(st.m) * a.inv_t + log1pf((st.n - 1.f) + st.s));
    if (bad || i == n) break;
    if (tid == 0) {
      const long long d = a.ids[b * G + i];
      const float zd = F::load(row, d);
      int v = kStays;
      double qd = 1.0;
      if (a.draft) {
        const float zq = F::load(a.draft + (b * G + i) * a.draft_bytes, d), lq = a.draft_lse[b * G + i];
        if (!(zq < INFINITY) || !(fabsf(lq) < INFINITY)) v = kNoDistribution;
        qd = exp(static_cast<double>(zq) * a.inv_t - static_cast<double>(lq));
      }
      const Term w = fp.template at<wide>(zd, sm.T, sm.delta);
      const double total = static_cast<double>(st.n) + static_cast<double>(st.s);
      if (v == kStays && !(a.u[b * rows + i] * qd * total < w.value())) v = kRefused;
      if (v == kStays) {
        tokens[i] = d;
        if (logp) logp[i] = log_prob(zd, st, a.inv_t);
      }
      sm.verdict = v;
    }
    __syncthreads();
    lost = sm.verdict == kRefused;
    bad = sm.verdict == kNoDistribution;
    if (lost || bad) break;
    kept = i + 1;
  }

  long long token = -1;
  if (!bad) {
    double u = a.u[b * rows + G];
    u = u > 0.0 ? fmin(u, 1.0 - 0x1p-53) : 0.0;
    bool own = !lost;
    if (lost && !a.draft) {
      Weights<DT, kWithout> f{row, nullptr, V, a.ids[b * G + kept], fp, fp, sm.T, sm.delta, false};
      const double total = all_parts(f, 0, V, sm);
      if (total > 0.0)
        token = search(f, u * total, sm);
      else
        own = true;
    }
    if (own || a.draft) {
      Weights<DT, kSoftmax> f{row, nullptr, V, -1, fp, fp, sm.T, sm.delta, false};
      double total = all_parts(f, 0, V, sm);
      if (lost && a.draft) {
        // S q_v = 2^(z c - k), k = lse_q log2(e) - log2 S, in the frame of a number with few digits
        if (tid == 0) sm.log2_total = log2(total);
        __syncthreads();
        const double k = static_cast<double>(a.draft_lse[b * G + kept]) * kLog2eD - sm.log2_total;
        const double near = rint(k / a.c_d * 4096.0) / 4096.0;
        const float mq = static_cast<float>(near);
        FineExp fq;
        fq.init(a.c_d, mq, k - static_cast<double>(mq) * a.c_d);
        Weights<DT, kRest> r{row, a.draft + (b * G + kept) * a.draft_bytes, V, -1, fp, fq, sm.T, sm.delta, false};
        const double rest = all_parts(r, 0, V, sm);
        bad = __syncthreads_or(r.bad);
        if (!bad && rest > 0.0)
          token = search(r, u * rest, sm);
        else
          own = !bad;
        if (own) total = all_parts(f, 0, V, sm);
      }
      if (own) token = search(f, u * total, sm);
    }
  }
  for (int i = tid; i <= G; i += kThreads) {
    if (i > kept) {
      tokens[i] = -1;
      if (logp) logp[i] = 0.f;
      if (lse) lse[i] = 0.f;
    }
  }
  if (tid == 0) {
    if (a.n_accepted) a.n_accepted[b] = kept;
    tokens[kept] = bad ? -1 : token;
    if (logp) logp[kept] = bad ? nan : log_prob(F::load(row, token), st, a.inv_t);
  }
}

}  // namespace
}  // namespace rl

extern "C" void rl_verify_drafts_desc_init(rl_verify_drafts_desc* desc) {
  if (!desc) return;
  *desc = rl_verify_drafts_desc{};
  desc->dtype = RL_BF16;
  desc->temperature = 1.0;
}

extern "C" rl_status rl_verify_drafts(const rl_verify_drafts_desc* desc, void* stream) {
  using namespace rl;
  if (!desc) return RL_ERR_NULL;
  const rl_verify_drafts_desc& d = *desc;
  if (d.dtype != RL_F32 && d.dtype != RL_BF16 && d.dtype != RL_F16) return RL_ERR_DTYPE;
  const long long es = d.dtype == RL_F32 ? 4 : 2, most = 1LL << 40;
  if (d.B < 0 || d.B >= (1LL << 31) || d.G < 0 || d.G > RL_VERIFY_MAX_DRAFT || d.B * (d.G + 1) >= (1LL << 31) || d.V < 1 ||
      d.V > kMaxVocab || d.ld < d.V || d.ld >= most || (d.draft_logits && (d.ld_draft < d.V || d.ld_draft >= most)))
    return RL_ERR_SHAPE;
  if (!(d.temperature >= 0.01 && d.temperature <= 100.0)) return RL_ERR_ARG;
  if (d.B == 0) return RL_OK;
  if (!d.target_logits || !d.uniforms || !d.tokens || (d.G > 0 && !d.draft_ids) || (d.G > 0 && d.draft_logits && !d.draft_lse))
    return RL_ERR_NULL;
  const auto off = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (off(d.target_logits, 16) || ((d.ld * es) & 15) || (d.draft_logits && (off(d.draft_logits, 16) || ((d.ld_draft * es) & 15))) ||
      off(d.uniforms, 8) || off(d.tokens, 8) || off(d.n_accepted, 8) || off(d.draft_ids, 8) || off(d.draft_lse, 4) ||
      off(d.n_draft, 4) || off(d.logp_out, 4) || off(d.lse_out, 4) || off(d.status_dev, 4))
    return RL_ERR_ALIGN;
  Args a;
  a.target = static_cast<const unsigned char*>(d.target_logits);
  a.draft = d.G > 0 ? static_cast<const unsigned char*>(d.draft_logits) : nullptr;
  a.draft_lse = d.draft_lse;
  a.ids = d.draft_ids;
  a.n_draft = d.n_draft;
  a.u = d.uniforms;
  a.V = d.V;
  a.row_bytes = d.ld * es;
  a.draft_bytes = d.ld_draft * es;
  a.G = static_cast<int>(d.G);
  a.inv_t = 1.0 / d.temperature;
  a.c_d = kLog2eD / d.temperature;
  a.c = static_cast<float>(a.c_d);
  a.tokens = d.tokens;
  a.n_accepted = d.n_accepted;
  a.logp = d.logp_out;
  a.lse = d.lse_out;
  a.status = d.status_dev;
  const unsigned grid = static_cast<unsigned>(d.B);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d.dtype == RL_F32)
    verify_drafts_kernel<RL_F32><<<grid, kThreads, 0, s>>>(a);
  else if (d.dtype == RL_BF16)
    verify_drafts_kernel<RL_BF16><<<grid, kThreads, 0, s>>>(a);
  else
    verify_drafts_kernel<RL_F16><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}
