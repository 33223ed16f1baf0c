// topk_distill.cu — rl_topk_distill_fwd_bwd: distillation from a teacher's
// top log-probabilities, the loss and its logits gradient in one launch
// (sm_103a).
//
// A row's loss needs the student's log-probability of the K given tokens and
// of all others together.  Pass 1 sums the others: each given token's logit
// is taken out of the row where it is met (a table by 64-byte piece says
// which pieces hold one), so the tail's mass is never a difference of nearly
// equal numbers.  The K logits and the tail then give the loss, one factor for
// every token of the tail and one value for each given token; pass 2 writes
// p_v times the factor, and the given tokens' values are stored over it.
#include <cmath>
#include <cstring>

#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxEntries = RL_TOKEN_MAX_K;
constexpr int kPerLane = kMaxEntries / 32;
constexpr int kTable = 4096;  // pieces that share a place of the table differ by a multiple of this
constexpr float kLnTiny = -87.33654475f;  // ln 2^-126
constexpr float kTiny = 0x1p-126f;

struct DistillArgs {
  const unsigned char* logits;
  unsigned char* dlogits;
  const long long* ids;
  const float* lq;
  const unsigned char* mask;
  const float* weight;
  float* row_loss;
  float* loss_out;
  rl_distill_stats* stats;
  WsHeader* ws;
  WsPartial* partials;
  long long R, V, row_bytes;
  float inv_temp, c;  // 1 / temperature, log2(e) / temperature
  float reverse, grad_scale;
  double norm;
  int K, renorm;
};

struct DistillSmem {
  int head[kTable];            // 1 + the last entry whose piece falls on this place, 0 none
  int next[kMaxEntries];       // the entry before it there
  int id[kMaxEntries];         // -1: empty
  float z[kMaxEntries];        // the entry's logit
  float d[kMaxEntries];        // the entry's gradient
  RowStats part[kRowWarps];
  long long wcount[kRowWarps];
  float m, factor;             // pass 2: dz = 2^((z - m) c) factor
  int bad, is_last;
};

// The entry at element e, or -1.
__device__ __forceinline__ int entry_at(const DistillSmem& sm, int e, int piece) {
  for (int j = sm.head[piece & (kTable - 1)]; j; j = sm.next[j - 1])
    if (sm.id[j - 1] == e) return j - 1;
  return -1;
}

// A row whose maximum is at most kExact (all -inf, or at the type's lowest):
// the tail's statistics without the floor.  Rare, so it reads the row again.
template <class F>
__device__ __noinline__ RowStats exact_tail(const unsigned char* row, int V, float c, DistillSmem& sm, int tid) {
  float m = -INFINITY;
  for (int i = tid; i < V; i += kRowThreads)
    if (entry_at(sm, i, i / F::kPiece) < 0) m = max_nan(m, F::load(row, i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();
  if ((tid & 31) == 0) sm.part[tid >> 5].m = m;
  __syncthreads();
  for (int w = 0; w < kRowWarps; ++w) m = max_nan(m, sm.part[w].m);
  __syncthreads();
  float s = 0.f;
  if (m > -INFINITY)
    for (int i = tid; i < V; i += kRowThreads)
      if (entry_at(sm, i, i / F::kPiece) < 0) s += ex2_approx((F::load(row, i) - m) * c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((tid & 31) == 0) sm.part[tid >> 5].r = s;
  __syncthreads();
  s = 0.f;
  for (int w = 0; w < kRowWarps; ++w) s += sm.part[w].r;
  return RowStats{m, s - 1.f, 0.f};
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

struct RowSums {
  double loss, fwd, rev, qt, pt;
};

// One warp: a row's loss terms and gradient values from the entries' logits
// (sm.z), the teacher's entries and the tail's statistics.
__device__ __forceinline__ RowSums row_values(const DistillArgs& a, DistillSmem& sm, RowStats tail, bool has_tail,
                                              const float (&lq_in)[kPerLane], float w, float s, int lane) {
  float lq[kPerLane], q[kPerLane], z[kPerLane];
  bool given[kPerLane];
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int j = lane + 32 * i;
    given[i] = j < a.K && sm.id[j] >= 0;
    z[i] = given[i] ? sm.z[j] : -INFINITY;
    lq[i] = given[i] ? lq_in[i] : -INFINITY;
    n += given[i];
  }
  n = __reduce_add_sync(0xffffffffu, n);
  // the teacher: 1 - sum q in fp64, where it is a difference of near numbers
  double sum = 0.0;
  float qt = 0.f, lqt = 0.f;
  if (a.renorm) {
    float mx = lq[0];
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) mx = fmaxf(mx, lq[i]);
    mx = warp_max(mx);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) sum += given[i] ? exp(static_cast<double>(lq[i]) - static_cast<double>(mx)) : 0.0;
    sum = warp_sum_d(sum);
    const float ls = static_cast<float>(static_cast<double>(mx) + log(sum));
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      lq[i] = given[i] ? lq[i] - ls : -INFINITY;
      q[i] = given[i] ? expf(lq[i]) : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const double e = given[i] ? exp(static_cast<double>(lq[i])) : 0.0;
      sum += e;
      q[i] = static_cast<float>(e);
    }
    sum = warp_sum_d(sum);
    if (has_tail) {
      const double t = 1.0 - sum;
      qt = static_cast<float>(t < 0x1p-24 ? 0x1p-24 : t);  // a NaN stays one
      lqt = logf(qt);
    }
  }
  const float Q = a.renorm ? 1.f : static_cast<float>(sum) + qt;
  // the student: the entries joined to the tail
  float zm = z[0];
#pragma unroll
  for (int i = 1; i < kPerLane; ++i) zm = max_nan(zm, z[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) zm = max_nan(zm, __shfl_xor_sync(0xffffffffu, zm, o));
  const bool tail_any = has_tail && tail.m > -INFINITY;
  const bool top_in = !tail_any || zm >= tail.m;  // the row's maximum is an entry
  const float M = top_in ? zm : tail.m;
  float e[kPerLane], in = 0.f;
  bool holder = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    e[i] = given[i] ? ex2_approx((z[i] - M) * a.c) : 0.f;
    holder = holder || (given[i] && z[i] == M);
  }
  // one maximum stays out of the sum of the others (r)
  const uint32_t holders = __ballot_sync(0xffffffffu, holder);
  bool out = top_in && lane == __ffs(holders) - 1;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    if (out && given[i] && z[i] == M)
      out = false;
    else
      in += e[i];
  }
  in = warp_sum(in);                          // entries without the left-out one
  const float s_in = top_in ? 1.f + in : in;  // all entries
  const float f_t = tail_any ? ex2_approx((tail.m - M) * a.c) : 0.f;
  const float s_t = tail_any ? f_t * (1.f + tail.r) : 0.f;
  const float r = top_in ? in + s_t : tail.r + in;
  const float log_s = log1pf(r), inv_s = 1.f / (1.f + r);
  float pt = 0.f, lpt = 0.f;
  if (has_tail) {
    pt = fmaxf(s_t * inv_s, kTiny);
    lpt = fmaxf(s_t > 0.f ? -log1pf(s_in / s_t) : -INFINITY, kLnTiny);
  }
  float F = 0.f, G = 0.f, lp[kPerLane], p[kPerLane], gap[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    lp[i] = fmaf(z[i] - M, a.inv_temp, -log_s);
    p[i] = e[i] * inv_s;
    gap[i] = lp[i] - fmaxf(lq[i], kLnTiny);
    if (q[i] > 0.f || q[i] != q[i]) F += q[i] * (lq[i] - lp[i]);
    if (p[i] > 0.f || p[i] != p[i]) G += p[i] * gap[i];
  }
  F = warp_sum(F);
  G = warp_sum(G);
  if (a.renorm) {
    G = 0.f;
  } else if (has_tail) {
    F += qt * (lqt - lpt);
    G += pt * (lpt - lqt);
  }
  const float v = a.reverse, u = 1.f - v;
  float L = u != 0.f ? u * F : 0.f;  // F may be infinite
  float ct = u * (Q - (has_tail && !a.renorm ? qt / pt : 0.f));
  if (v != 0.f) {
    L += v * G;
    ct += v * (lpt - lqt - G);
  }
  bool nothing = a.renorm && n == 0;
  if (sm.bad) L = __int_as_float(0x7fc00000);
  if (!(M > -INFINITY)) L = __int_as_float(0x7fc00000);  // no distribution
  if (L != L) ct = L;
  if (nothing && L == L) L = ct = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int j = lane + 32 * i;
    if (given[i]) {
      float d = u * (p[i] * Q - q[i]);
      if (v != 0.f && p[i] > 0.f) d += v * p[i] * (gap[i] - G);
      sm.d[j] = L != L ? L : s * d;
    }
  }
  if (lane == 0) {
    sm.m = M;
    sm.factor = nothing ? 0.f : fmaxf(fminf(s * ct, 3.0e38f), -3.0e38f) * inv_s;
    if (L != L) sm.factor = L;
  }
  if (nothing) F = 0.f;
  return RowSums{static_cast<double>(w) * L, F, G, qt, a.renorm ? 0.f : pt};
}

template <int DT>
__global__ void __launch_bounds__(kRowThreads) topk_distill_kernel(const DistillArgs a) {
  using F = Fmt<DT>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  DistillSmem& sm = *reinterpret_cast<DistillSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = static_cast<int>(a.V), K = a.K;
  const int n_pieces = (V + F::kPiece - 1) / F::kPiece;
  const int n_vecs = (V + F::kVec - 1) / F::kVec;
  unsigned int err = 0;
  double acc[5] = {0.0, 0.0, 0.0, 0.0, 0.0};

  for (int i = tid; i < kTable; i += kRowThreads) sm.head[i] = 0;
  // N: every CTA counts the mask
  long long N = a.R;
  if (a.mask) {
    int cnt = 0;
    for (long long i = tid; i < a.R; i += kRowThreads) cnt += a.mask[i] != 0;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) sm.wcount[warp] = cnt;
    __syncthreads();
    N = 0;
    for (int w = 0; w < kRowWarps; ++w) N += sm.wcount[w];
  }
  const double norm = a.norm > 0.0 ? a.norm : static_cast<double>(N);
  __syncthreads();

  for (long long row = blockIdx.x; row < a.R; row += gridDim.x) {
    const unsigned char* src = a.logits + row * a.row_bytes;
    unsigned char* dst = a.dlogits ? a.dlogits + row * a.row_bytes : nullptr;
    if (a.mask && a.mask[row] == 0) {
      if (dst)
        for (int v = tid; v < n_vecs; v += kRowThreads) {
          if ((v + 1) * F::kVec <= V)
            st_global_cs_v4(dst + static_cast<long long>(v) * 16, make_uint4(0u, 0u, 0u, 0u));
          else
            for (int i = v * F::kVec; i < V; ++i) F::store(dst, i, 0.f);
        }
      if (tid == 0 && a.row_loss) a.row_loss[row] = 0.f;
      continue;
    }
    // the row's entries into the table
    if (tid == 0) sm.bad = 0;
    __syncthreads();
    if (tid < K) {
      const long long id = a.ids[row * K + tid];
      sm.id[tid] = id >= 0 && id < V ? static_cast<int>(id) : -1;
      if (id < -1 || id >= V) {
        err |= RL_DEVERR_ID_RANGE;
        sm.bad = 1;
      }
      if (id >= 0 && id < V)
        sm.next[tid] = atomicExch(&sm.head[(static_cast<int>(id) / F::kPiece) & (kTable - 1)], tid + 1);
    }
    __syncthreads();
    int n_given = 0;
    if (tid < K && sm.id[tid] >= 0) {
      n_given = 1;
      const int id = sm.id[tid];
      int same = 0;
      for (int j = sm.head[(id / F::kPiece) & (kTable - 1)]; j; j = sm.next[j - 1]) same += sm.id[j - 1] == id;
      if (same > 1) {
        err |= RL_DEVERR_ID_REPEAT;
        sm.bad = 1;
      }
    }
    n_given = __syncthreads_count(n_given);
    const bool has_tail = n_given < V;
    // pass 1: the statistics of every token that is not given
    WarpStats st;
    st.low = false;
    warp_stats_init<F>(st, a.c);
    for (int p0 = 0; p0 < n_pieces; p0 += kRowThreads) {
      const int p = p0 + tid;
      uint32_t w[16];
      const long long row_bytes16 = (static_cast<long long>(V) * F::kBytes + 15) & ~15LL;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long off = static_cast<long long>(p) * kPieceBytes + j * 16;
        uint4 v = make_uint4(F::kNegInf2, F::kNegInf2, F::kNegInf2, F::kNegInf2);
        if (off < row_bytes16) v = *reinterpret_cast<const uint4*>(src + off);
        w[4 * j] = v.x;
        w[4 * j + 1] = v.y;
        w[4 * j + 2] = v.z;
        w[4 * j + 3] = v.w;
      }
      if ((p + 1) * F::kPiece > V) F::cut(w, 0, max(0, V - p * F::kPiece));
      if (p < n_pieces) {
        for (int j = sm.head[p & (kTable - 1)]; j; j = sm.next[j - 1]) {
          const int e = sm.id[j - 1] - p * F::kPiece;
          if (e >= 0 && e < F::kPiece) {
            sm.z[j - 1] = F::load(src, sm.id[j - 1]);
            F::drop(w, 0, e);
          }
        }
      }
      const uint32_t rm = F::raw_max(w, 0);
      add_piece<F, false>(st, w, max_nan(F::raw_value(rm), F::kFloor), a.c, lane, false);
    }
    const RowStats wst = warp_stats_sum<F>(st, a.c);
    if (lane == 0) sm.part[warp] = wst;
    __syncthreads();
    RowStats tail = sm.part[0];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) tail = merge_row(tail, sm.part[w], a.c);
    if (needs_exact<F>(tail.m, a.c)) tail = exact_tail<F>(src, V, a.c, sm, tid);
    if (warp == 0) {
      float lq[kPerLane];
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) lq[i] = lane + 32 * i < K ? a.lq[row * K + lane + 32 * i] : 0.f;
      const float w = a.weight ? a.weight[row] : 1.f;
      const float s = static_cast<float>(static_cast<double>(a.grad_scale) * w / norm) * a.inv_temp;
      const RowSums t = row_values(a, sm, tail, has_tail, lq, w, s, lane);
      if (lane == 0) {
        acc[0] += t.loss;
        acc[1] += t.fwd;
        acc[2] += t.rev;
        acc[3] += t.qt;
        acc[4] += t.pt;
        if (a.row_loss) a.row_loss[row] = static_cast<float>(t.loss);
      }
    }
    __syncthreads();
    // pass 2
    if (dst) {
      const float2 nm = make_float2(-sm.m, -sm.m), c2 = make_float2(a.c, a.c);
      const float2 f2 = make_float2(sm.factor, sm.factor);
      for (int v = tid; v < n_vecs; v += kRowThreads) {
        float z[F::kVec];
        F::unpack(*reinterpret_cast<const uint4*>(src + static_cast<long long>(v) * 16), z);
#pragma unroll
        for (int i = 0; i < F::kVec; i += 2) {
          const float2 x = __fmul2_rn(__fadd2_rn(make_float2(z[i], z[i + 1]), nm), c2);
          const float2 d = __fmul2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), f2);
          z[i] = d.x;
          z[i + 1] = d.y;
        }
        if ((v + 1) * F::kVec <= V) {
          st_global_cs_v4(dst + static_cast<long long>(v) * 16, F::pack(z));
        } else {
#pragma unroll
          for (int i = 0; i < F::kVec; ++i)
            if (v * F::kVec + i < V) F::store(dst, v * F::kVec + i, z[i]);
        }
      }
    }
    __syncthreads();
    if (tid < K && sm.id[tid] >= 0) {
      if (dst) F::store(dst, sm.id[tid], sm.d[tid]);
      sm.head[(sm.id[tid] / F::kPiece) & (kTable - 1)] = 0;
    }
    __syncthreads();
  }

  // this CTA's sums, then the last CTA adds all of them in CTA order
  if (err) atomicOr(&a.ws->status, err);
  __syncthreads();
  if (tid == 0) {
    WsPartial& P = a.partials[blockIdx.x];
    for (int i = 0; i < 5; ++i) P.v[i] = acc[i];
    __threadfence();
    sm.is_last = atomicInc(&a.ws->ticket, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (sm.is_last && warp == 0) {
    __threadfence();
    double v[5] = {0.0, 0.0, 0.0, 0.0, 0.0};
    for (int i = lane; i < static_cast<int>(gridDim.x); i += 32)
      for (int q = 0; q < 5; ++q) v[q] += __ldcg(&a.partials[i].v[q]);
    for (int q = 0; q < 5; ++q) v[q] = warp_sum_d(v[q]);
    if (lane == 0) {
      const unsigned int stw = atomicExch(&a.ws->status, 0u);
      a.ws->last_status = stw;
      const double inv = N > 0 ? 1.0 / static_cast<double>(N) : 0.0;
      rl_distill_stats o;
      o.loss = norm > 0.0 ? v[0] / norm : 0.0;
      o.forward_kl = v[1] * inv;
      o.reverse_kl = v[2] * inv;
      o.teacher_tail = v[3] * inv;
      o.student_tail = v[4] * inv;
      o.n_rows = N;
      o.device_error = static_cast<int>(stw);
      o.reserved = 0;
      *a.stats = o;
      if (a.loss_out) *a.loss_out = static_cast<float>(o.loss);
    }
  }
}

// ------------------------------------------------------------------ host side
template <int DT>
rl_status launch(const DistillArgs& a, int sms, cudaStream_t stream) {
  long long grid = 4LL * sms;
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (grid > a.R) grid = a.R > 0 ? a.R : 1;
  topk_distill_kernel<DT><<<static_cast<unsigned>(grid), kRowThreads, sizeof(DistillSmem), stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // namespace
}  // namespace rl

extern "C" size_t rl_topk_distill_workspace_size(void) { return rl::kWorkspaceBytes; }

extern "C" void rl_topk_distill_desc_init(rl_topk_distill_desc* d) {
  if (!d) return;
  std::memset(d, 0, sizeof(*d));
  d->dtype = RL_BF16;
  d->tail = RL_DISTILL_TAIL_BUCKET;
  d->temperature = 1.f;
  d->grad_scale = 1.f;
}

extern "C" rl_status rl_topk_distill_fwd_bwd(const rl_topk_distill_desc* d, void* stream) {
  using namespace rl;
  if (!d) return RL_ERR_NULL;
  const int es = d->dtype == RL_F32 ? 4 : d->dtype == RL_BF16 || d->dtype == RL_F16 ? 2 : 0;
  if (es == 0 || (d->tail != RL_DISTILL_TAIL_BUCKET && d->tail != RL_DISTILL_TAIL_RENORM)) return RL_ERR_DTYPE;
  const long long R = d->R, V = d->V, ld = d->ld;
  if (R < 0 || R >= (1LL << 31) || V < 1 || V > kMaxVocab || ld < V || ld > (1LL << 31)) return RL_ERR_SHAPE;
  if (d->K < 1 || d->K > RL_TOKEN_MAX_K || !(d->reverse >= 0.f && d->reverse <= 1.f) ||
      !(d->temperature >= kMinTemperature && d->temperature <= kMaxTemperature) || !std::isfinite(d->grad_scale) ||
      !(d->norm >= 0.0) || !std::isfinite(d->norm) || (d->reverse != 0.f && d->tail == RL_DISTILL_TAIL_RENORM))
    return RL_ERR_ARG;
  if (!d->stats_dev) return RL_ERR_NULL;
  if (!d->workspace || d->workspace_bytes < kWorkspaceBytes) return RL_ERR_WORKSPACE;
  if (R > 0 && (!d->logits || !d->teacher_ids || !d->teacher_logp)) return RL_ERR_NULL;
  const long long row_bytes = ld * es;
  if ((reinterpret_cast<uintptr_t>(d->logits) & 15) || (reinterpret_cast<uintptr_t>(d->dlogits) & 15) || (row_bytes & 15) ||
      (reinterpret_cast<uintptr_t>(d->workspace) & 15))
    return RL_ERR_ALIGN;
  if (d->dlogits && d->dlogits != d->logits && R > 0) {
    const uintptr_t l0 = reinterpret_cast<uintptr_t>(d->logits), d0 = reinterpret_cast<uintptr_t>(d->dlogits);
    const uintptr_t n = static_cast<uintptr_t>(R) * static_cast<uintptr_t>(row_bytes);
    if (l0 < d0 + n && d0 < l0 + n) return RL_ERR_ALIAS;
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return RL_ERR_CUDA;
  DistillArgs a;
  a.logits = static_cast<const unsigned char*>(d->logits);
  a.dlogits = static_cast<unsigned char*>(d->dlogits);
  a.ids = d->teacher_ids;
  a.lq = d->teacher_logp;
  a.mask = d->mask;
  a.weight = d->weight;
  a.row_loss = d->row_loss_out;
  a.loss_out = d->loss_out;
  a.stats = d->stats_dev;
  a.ws = static_cast<WsHeader*>(d->workspace);
  a.partials = reinterpret_cast<WsPartial*>(static_cast<unsigned char*>(d->workspace) + sizeof(WsHeader));
  a.R = R;
  a.V = V;
  a.row_bytes = row_bytes;
  a.inv_temp = 1.f / d->temperature;
  a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(d->temperature));
  a.reverse = d->reverse;
  a.grad_scale = d->grad_scale;
  a.norm = d->norm;
  a.K = d->K;
  a.renorm = d->tail == RL_DISTILL_TAIL_RENORM;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (d->dtype) {
    case RL_F32: return launch<RL_F32>(a, sms, s);
    case RL_BF16: return launch<RL_BF16>(a, sms, s);
    case RL_F16: return launch<RL_F16>(a, sms, s);
  }
  return RL_ERR_DTYPE;
}
