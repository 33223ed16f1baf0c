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
//
//   * A CTA takes a row at a time.  The producer warp streams its chunks
//     through a ring of shared-memory slots twice: the first load keeps its L2
//     lines (evict-last), the second takes them from L2 (evict-first), so the
//     logits cross the HBM bus once.
//   * The consumer warps run pass 1 (one 64-byte piece a thread and chunk) and
//     pass 2 (16-byte vectors, streaming stores) without a barrier of their
//     own.
//   * The row warp fills the table with the next row's entries, turns the
//     consumers' partial statistics into the row's loss and gradient values,
//     and stores the given tokens' gradients once the consumers have written
//     the row.  The teacher's side is formed a row ahead.
//   * A few long rows get a cluster each: its CTAs exchange their slices'
//     statistics and given logits, and every one of them forms the same values.
//
// What bounds it: a row read once and written once, 734 us at 8192 x 151,936
// bf16; measured 812 us (6.1 TB/s).  The two passes take about the same time,
// and the consumers wait for data in an eighth of it: the rest is their own
// instructions, two exponentials an element.  Chunks of the next row's first
// pass run before a row's second (kLead), so that the row warp's serial part
// hides: 441 -> 427 us at 4096 rows.
#include <cmath>
#include <cstring>

#include "lost_rows.h"
#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kMaxEntries = RL_TOKEN_MAX_K;
constexpr int kPerLane = kMaxEntries / 32;
constexpr int kTable = 2048;  // pieces that share a place of the table differ by a multiple of this
constexpr int kLead = 2;      // chunks of the next row's first pass before a row's second
constexpr int kMaxCluster = 8;
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
  float temperature, reverse, grad_scale;
  double norm;
  int K, renorm;
};

// A row's entries by the piece that holds them.
struct EntryTable {
  int head[kTable];            // 1 + the last entry whose piece falls on this place, 0 none
  int next[kMaxEntries];       // the entry before it there
  int id[kMaxEntries];         // -1: empty
  float z[kMaxEntries];        // the entry's logit (from the consumers)
  // the teacher's side, known before the student's row has streamed
  float lq[kMaxEntries], q[kMaxEntries];
  float qt, lqt, Q;            // the tail's probability and its logarithm; all probabilities
  float w, s;                  // the row's weight, its gradient's scale
  int n, bad;                  // entries; an id is out of range or named twice
};

// kThreads consumers; a chunk is one piece of each.
template <int kThreads>
struct DistillSmem {
  static constexpr int kWarps = kThreads / 32, kChunk = kThreads * kPieceBytes;
  static constexpr int kSlots = kThreads >= 512 ? 6 : kThreads >= 256 ? 5 : 4;
  Ring<kSlots, kChunk> ring;
  long long row_of[kSlots];    // the row a chunk belongs to
  EntryTable tab[2];           // of the even and the odd rows of this CTA
  RowStats part[kWarps];
  long long wcount[kWarps + 2];
  unsigned long long table[2];  // a row's entries are in tab[k & 1]
  unsigned long long sums, values, written;  // once a row: sums in, values out, row written
  // clusters (of one row): what every CTA found in its slice, in every CTA's memory
  float slice_z[kMaxEntries];
  float2 slice_tail[kMaxCluster];               // m, r
  unsigned long long slices, read_again;        // all are in; a row taken again has been read
  float m, factor;             // pass 2: dz = 2^((z - m) c) factor
  int plain;                   // pass 2 by differences to m
  int abort;
};

// The entry at element e, or -1.
__device__ __forceinline__ int entry_at(const EntryTable& tab, int e, int piece) {
  for (int j = tab.head[piece & (kTable - 1)]; j; j = tab.next[j - 1])
    if (tab.id[j - 1] == e) return j - 1;
  return -1;
}

// The tail's statistics by differences to its maximum (needs_exact).  Rare, so
// one warp reads the row again.
template <class F>
__device__ __noinline__ RowStats exact_tail(const unsigned char* row, int V, float c, const EntryTable& tab, int lane) {
  const int n_vecs = (V + F::kVec - 1) / F::kVec;
  auto each = [&](auto f) {
#pragma unroll 4
    for (int v = lane; v < n_vecs; v += 32) {
      float z[F::kVec];
      F::unpack(*reinterpret_cast<const uint4*>(row + static_cast<long long>(v) * 16), z);
#pragma unroll
      for (int i = 0; i < F::kVec; ++i) {
        const int e = v * F::kVec + i;
        if (e < V && entry_at(tab, e, e / F::kPiece) < 0) f(z[i]);
      }
    }
  };
  float m = -INFINITY;
  each([&](float z) { m = max_nan(m, z); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.f;
  if (m > -INFINITY) each([&](float z) { s += ex2_approx((z - m) * c); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
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

// e^y for y <= 88 as the sum of two floats (in fp64), relative error below
// 2^-34, and 2^-35.5 from y = -20 on: 1 - sum q keeps 2^-12 of a tail of 2^-24, and
// 20 bits from 2^-15 on.  Cody and Waite's reduction: y - n ln 2 is exact (the head
// of ln 2 has 16 bits).  Then Horner's scheme for the Taylor series, its last five
// steps on an unevaluated sum h + l (Dekker's product and sum: p + e = f h exactly,
// s + rounding = c + p exactly).  A fraction of the fp64 exponential's time on a
// GPU with few fp64 units.
__device__ __forceinline__ void horner_pair(float c, float c_low, float f, float& h, float& l) {
  const float p = __fmul_rn(f, h), e = fmaf(f, l, fmaf(f, h, -p));
  h = c + p;
  l = (p - (h - c)) + (e + c_low);
}
__device__ __forceinline__ double exp_sum(float y) {
  constexpr float kLn2Head = 45426.0f / 65536.0f;
  constexpr float kLn2Rest = static_cast<float>(0.69314718055994530942 - 45426.0 / 65536.0);
  if (!(y > -87.f)) return y != y ? static_cast<double>(y) : 0.0;  // (2^-126 and less)
  const float n = fminf(rintf(y * kLog2e), 128.f);
  const float f = fmaf(n, -kLn2Head, y);
  float h = 1.f / 362880.f, l = 0.f;
  h = fmaf(h, f, 1.f / 40320.f);
  h = fmaf(h, f, 1.f / 5040.f);
  h = fmaf(h, f, 1.f / 720.f);
  h = fmaf(h, f, 1.f / 120.f);
  constexpr float k24 = static_cast<float>(1.0 / 24.0), k6 = static_cast<float>(1.0 / 6.0);
  horner_pair(k24, static_cast<float>(1.0 / 24.0 - k24), f, h, l);
  horner_pair(k6, static_cast<float>(1.0 / 6.0 - k6), f, h, l);
  horner_pair(0.5f, 0.f, f, h, l);
  horner_pair(1.f, 0.f, f, h, l);
  horner_pair(1.f, 0.f, f, h, l);
  const float g = -n * kLn2Rest;  // e^(f + g) = e^f (1 + g + g^2 / 2 ...), |g| < 1e-3
  l = fmaf(h, g * fmaf(0.5f, g, 1.f), l);
  const float scale = __int_as_float((static_cast<int>(n) + 127) << 23);
  return static_cast<double>(h * scale) + static_cast<double>(l * scale);
}

// The teacher's side of a row into its table, by one warp, from the entries'
// ids (-1: none) and log-probabilities, four a lane.
__device__ __forceinline__ void teacher_values(const DistillArgs& a, EntryTable& tab, const int (&id)[kPerLane],
                                               float (&lq)[kPerLane], float w, int n, bool bad, double scale,
                                               int lane) {
  double sum = 0.0;  // 1 - sum q is a difference of near numbers
  float q[kPerLane], qt = 0.f, lqt = 0.f, Q = 1.f;
  if (a.renorm) {
    float mx = -INFINITY, e = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) mx = id[i] >= 0 ? fmaxf(mx, lq[i]) : mx;
    mx = warp_max(mx);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      q[i] = id[i] >= 0 ? expf(lq[i] - mx) : 0.f;
      e += q[i];
    }
    e = warp_sum(e);
    const float inv = 1.f / e, ls = logf(e);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      lq[i] = id[i] >= 0 ? (lq[i] - mx) - ls : -INFINITY;
      q[i] = id[i] >= 0 ? q[i] * inv : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      q[i] = 0.f;
      if (id[i] >= 0) {
        const double e = exp_sum(lq[i]);
        sum += e;
        q[i] = static_cast<float>(e);
      } else {
        lq[i] = -INFINITY;
      }
    }
    sum = warp_sum_d(sum);
    if (n < a.V) {
      const double u = 1.0 - sum;
      qt = static_cast<float>(u < 0x1p-24 ? 0x1p-24 : u);  // a NaN stays one
      lqt = logf(qt);
    }
    Q = static_cast<float>(sum) + qt;
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    tab.lq[lane + 32 * i] = lq[i];
    tab.q[lane + 32 * i] = q[i];
  }
  if (lane == 0) {
    tab.qt = qt;
    tab.lqt = lqt;
    tab.Q = Q;
    tab.w = w;
    tab.s = static_cast<float>(scale * w);
    tab.n = n;
    tab.bad = bad;
  }
}

struct RowSums {
  double loss, fwd, rev, qt, pt;
  float m, factor;  // of the tail's gradient
};

// One warp: a row's loss terms and gradient values from the teacher's side,
// the entries' logits z and the tail's statistics; d: the given tokens'
// gradients.
__device__ __forceinline__ RowSums row_values(const DistillArgs& a, const EntryTable& t, const int (&id)[kPerLane],
                                              const float (&z)[kPerLane], RowStats tail, float M, float (&d)[kPerLane], int lane) {
  const bool has_tail = t.n < a.V;
  // the student: the entries joined to the tail, in the frame of M, the larger
  // of the entries' maximum and the tail's reference
  const bool tail_any = has_tail && tail.m > -INFINITY;
  const bool top_in = !tail_any || M > tail.m || !(tail.m >= M);  // M is an entry's
  float e[kPerLane], in = 0.f;
  bool holder = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    e[i] = id[i] >= 0 ? ex2_approx((z[i] - M) * a.c) : 0.f;
    holder = holder || (id[i] >= 0 && z[i] == M);
  }
  // one maximum stays out of the sum of the others (r)
  const uint32_t holders = __ballot_sync(0xffffffffu, holder);
  bool out = top_in && lane == __ffs(holders) - 1;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    if (out && id[i] >= 0 && z[i] == M)
      out = false;
    else
      in += e[i];
  }
  in = warp_sum(in);                          // entries without the left-out one
  const float s_in = top_in ? 1.f + in : in;  // all entries
  // 2^((tail.m - M) c) in two halves: far below M it has no place in fp32, while
  // its product with the sum of many tokens, or with q_t / p_t, has
  const float half = tail_any ? ex2_approx(0.5f * ((tail.m - M) * a.c)) : 0.f;
  const float s_t = (half * (1.f + tail.r)) * half;
  const float r = top_in ? in + s_t : tail.r + in;
  const float log_s = log1pf(r), inv_s = __frcp_rn(1.f + r);
  float pt = 0.f, lpt = 0.f;
  if (has_tail) {
    pt = fmaxf(s_t * inv_s, kTiny);
    lpt = fmaxf(s_t > 0.f ? -log1pf(s_in / s_t) : -INFINITY, kLnTiny);
  }
  float F = 0.f, G = 0.f, p[kPerLane], q[kPerLane], gap[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const float lp = fmaf(z[i] - M, a.inv_temp, -log_s);
    p[i] = e[i] * inv_s;
    const float lq = t.lq[lane + 32 * i];
    q[i] = t.q[lane + 32 * i];
    gap[i] = lp - fmaxf(lq, kLnTiny);
    if (q[i] > 0.f || q[i] != q[i]) F += q[i] * (lq - lp);
    if (p[i] > 0.f || p[i] != p[i]) G += p[i] * gap[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    F += __shfl_xor_sync(0xffffffffu, F, o);
    G += __shfl_xor_sync(0xffffffffu, G, o);
  }
  if (a.renorm) {
    G = 0.f;
  } else if (has_tail) {
    F += t.qt * (t.lqt - lpt);
    G += pt * (lpt - t.lqt);
  }
  const float v = a.reverse, u = 1.f - v;
  float L = u != 0.f ? u * F : 0.f;  // F may be infinite
  float ct = u * (t.Q - (has_tail && !a.renorm ? t.qt / pt : 0.f));
  if (v != 0.f) {
    L += v * G;
    ct += v * (lpt - t.lqt - G);
  }
  const bool nothing = a.renorm && t.n == 0;
  if (t.bad || r != r) L = __int_as_float(0x7fc00000);
  // a maximum of -inf: no distribution; +inf (left out of r, or of teacher
  // probability 0, it is in no other term) and NaN: none either
  if (!(fabsf(M) < INFINITY)) L = __int_as_float(0x7fc00000);
  if (nothing && L == L) L = F = ct = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    float g = u * (p[i] * t.Q - q[i]);
    if (v != 0.f && p[i] > 0.f) g += v * p[i] * (gap[i] - G);
    d[i] = L != L ? L : t.s * g;
  }
  // The tail's gradient s ct p_v as 2^((z_v - m) c) factor, m the tail's own
  // reference: of a tail far below M, ct holds q_t / p_t of up to 2^126, and p_v as
  // little, and s ct would overflow.
  const bool in_tail = tail_any && tail.r > -1.f;
  const float m = in_tail ? tail.m : M;
  float factor = t.s * ((in_tail ? (ct * half) * half : ct) * inv_s);
  if (L != L) factor = L;
  return RowSums{static_cast<double>(t.w) * L, F, G, t.qt, a.renorm ? 0.f : pt, m, factor};
}

// The consumer warps' partial statistics joined, one a lane (kWarps <= 32):
// the maximum first, then the sums in its frame.  The first warp that holds the
// maximum leaves its term out, the others' maxima come back in.
template <int kWarps>
__device__ __forceinline__ RowStats join_parts(const RowStats* part, float floor, float c, int lane) {
  RowStats p = lane < kWarps ? part[lane] : RowStats{floor, -1.f, 0.f};
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(p.m));
  const uint32_t holders = __ballot_sync(0xffffffffu, p.m == m && lane < kWarps);
  const float f = ex2_approx((p.m - m) * c);
  const float r = lane == __ffs(holders) - 1 ? p.r : f * (1.f + p.r);
  return RowStats{m, warp_sum(r), 0.f};
}

// Takes a row's entries into the table (which holds no other row's) and looks
// for ids out of range (-1 in `id` then) and named twice.  Whole warp.
template <class F>
__device__ __forceinline__ void table_row(const DistillArgs& a, EntryTable& tab, const long long (&id_in)[kPerLane],
                                          int (&id)[kPerLane], int& n, bool& bad, int lane, unsigned int& err) {
  const int V = static_cast<int>(a.V);
  bad = false;
  n = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int j = lane + 32 * i;
    const bool out = id_in[i] < -1 || id_in[i] >= V;
    if (out) err |= RL_DEVERR_ID_RANGE;
    bad = bad || out;
    id[i] = id_in[i] >= 0 && !out ? static_cast<int>(id_in[i]) : -1;
    tab.id[j] = id[i];
    if (id[i] >= 0) {
      ++n;
      tab.next[j] = atomicExch(&tab.head[(id[i] / F::kPiece) & (kTable - 1)], j + 1);
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    if (id[i] < 0) continue;
    int same = 0;
    for (int j = tab.head[(id[i] / F::kPiece) & (kTable - 1)]; j; j = tab.next[j - 1]) same += tab.id[j - 1] == id[i];
    if (same > 1) {
      err |= RL_DEVERR_ID_REPEAT;
      bad = true;
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  n = __reduce_add_sync(0xffffffffu, n);
}

// N, the number of valid rows: every CTA counts the mask, its consumers and
// its row warp together while the producer starts.  `at`: the consumer's
// number; the row warp counts nothing, it takes the sum.
template <int kWarps>
__device__ __forceinline__ long long count_rows(const DistillArgs& a, long long (&wcount)[kWarps], int at) {
  constexpr int kCounting = (kWarps - 2) * 32;
  if (!a.mask) return a.R;
  if (at < kCounting) {
    int cnt = 0;
    const bool wide = (reinterpret_cast<uintptr_t>(a.mask) & 15) == 0;
    const long long n16 = wide ? a.R / 16 : 0;
    auto add = [&](uint32_t w) { cnt += __popc(__vcmpne4(w, 0u)) >> 3; };
#pragma unroll 2
    for (long long i = at; i < n16; i += kCounting) {
      const uint4 v = reinterpret_cast<const uint4*>(a.mask)[i];
      add(v.x);
      add(v.y);
      add(v.z);
      add(v.w);
    }
    for (long long i = n16 * 16 + at; i < a.R; i += kCounting) cnt += a.mask[i] != 0;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if ((at & 31) == 0) wcount[at / 32] = cnt;
  }
  named_barrier(2, kCounting + 32);
  long long N = 0;
  for (int w = 0; w < kWarps - 2; ++w) N += wcount[w];
  return N;
}

// One warp: NaN to every row's loss and gradient.
template <class F>
__device__ __noinline__ void lose_rows(float* row_loss, unsigned char* dlogits, long long R, long long row_bytes, int V, int lane) {
  for (long long row = 0; row < R; ++row) {
    if (lane == 0 && row_loss) row_loss[row] = __int_as_float(0x7fc00000);
    if (dlogits)
      for (int v = lane; v < V; v += 32) F::store(dlogits + row * row_bytes, v, __int_as_float(0x7fc00000));
  }
}

// kThreads consumers, the producer warp and the row warp.  kCluster: the CTAs
// of a cluster share its one row.
template <int DT, int kThreads, int kCtas, bool kCluster>
__global__ void __launch_bounds__(kThreads + 64, kCtas) topk_distill_kernel(const DistillArgs a) {
  using F = Fmt<DT>;
  using S = DistillSmem<kThreads>;
  constexpr int kWarps = S::kWarps, kChunk = S::kChunk;
  constexpr int kVecs = kChunk / 16, kVecsPerThread = kVecs / kThreads;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  volatile int* abort = &sm.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = static_cast<int>(a.V), K = a.K;
  // this CTA's pieces are g0 .. g0 + n_mine - 1: n_elems elements from byte b0 on
  const int csize = kCluster ? static_cast<int>(cluster_size()) : 1, rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
  const long long first = blockIdx.x / csize, stride = gridDim.x / csize;
  const int n_pieces = (V + F::kPiece - 1) / F::kPiece, per = (n_pieces + csize - 1) / csize;
  const int g0 = kCluster ? min(n_pieces, rank * per) : 0, n_mine = kCluster ? min(n_pieces, g0 + per) - g0 : n_pieces;
  const int e0 = g0 * F::kPiece, n_elems = kCluster ? min(V - e0, n_mine * F::kPiece) : V;
  const long long b0 = static_cast<long long>(g0) * kPieceBytes;
  const int n_vecs = (n_elems + F::kVec - 1) / F::kVec;
  const long long n_bytes = static_cast<long long>(n_vecs) * 16;
  const int n_chunks = static_cast<int>((n_bytes + kChunk - 1) / kChunk);
  const int lead = min(n_chunks, kLead);

  if (tid == 0) {
    sm.ring.init(kWarps);
    mbar_init(smem_addr(&sm.table[0]), 1);
    mbar_init(smem_addr(&sm.table[1]), 1);
    mbar_init(smem_addr(&sm.sums), kWarps);
    mbar_init(smem_addr(&sm.values), 1);
    mbar_init(smem_addr(&sm.written), kWarps);
    mbar_init(smem_addr(&sm.slices), csize);
    mbar_init(smem_addr(&sm.read_again), csize);
    sm.abort = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < 2 * kTable; i += kThreads + 64) sm.tab[i / kTable].head[i % kTable] = 0;
  __syncthreads();
  if (kCluster) cluster_sync_all();

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    // The row of a chunk goes with it; a chunk of no bytes and row -1 is the end.
    const uint64_t keep = policy_keep(), once = policy_evict_first();
    uint32_t it = 0;
    bool ok = true;
    RowsOf<true> rows(a.mask, a.R, first, lane);
    const int passes = a.dlogits ? 2 : 1;
    // chunks [q0, q1) of a row, lane 0; none of row -1
    auto issue = [&](long long row, int q0, int q1, uint64_t pol) {
      const unsigned char* src = a.logits + row * a.row_bytes + b0;
      for (int q = q0; q < q1 && ok; ++q) {
        ok = sm.ring.reserve(it, abort);
        if (!ok) break;
        sm.row_of[it % S::kSlots] = row;
        const long long off = static_cast<long long>(q) * kChunk;
        sm.ring.fill(it, src + off, static_cast<uint32_t>(min(static_cast<long long>(kChunk), n_bytes - off)), pol);
        ++it;
      }
    };
    long long prev = -1;  // the row whose second pass is still to be issued
    while (ok) {
      const long long row = rows.next(stride, lane);
      if (lane == 0) {
        const int first_q = prev >= 0 ? lead : n_chunks;
        if (row >= 0) {
          issue(row, 0, first_q, passes == 2 ? keep : once);
        } else if (ok && (ok = sm.ring.reserve(it, abort))) {
          sm.row_of[it % S::kSlots] = -1;
          mbar_arrive(smem_addr(&sm.ring.full[it % S::kSlots]));
          ++it;
        }
        if (prev >= 0 && passes == 2) issue(prev, 0, n_chunks, once);
        if (row >= 0) issue(row, first_q, n_chunks, passes == 2 ? keep : once);
        if (!ok) sm.ring.drain(it);
      }
      prev = row;
      ok = __shfl_sync(0xffffffffu, ok, 0) && row >= 0;
    }
  } else if (warp == kWarps + 1) {
    // ---------------------------------------------------------------- row warp
    const long long N = count_rows(a, sm.wcount, kThreads);
    const double norm = a.norm > 0.0 ? a.norm : static_cast<double>(N);
    unsigned int err = 0;
    double acc[5] = {0.0, 0.0, 0.0, 0.0, 0.0};
    RowsOf<true> rows(a.mask, a.R, first, lane);
    // the table and the teacher's side of this CTA's k-th row, from what was
    // fetched a row ahead
    const double scale = static_cast<double>(a.grad_scale) / (norm * static_cast<double>(a.temperature));
    long long id_in[kPerLane];
    float lq_in[kPerLane], w_in = 1.f;
    auto fetch = [&](long long row) {
      if (row < 0) return;
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        const int j = lane + 32 * i;
        id_in[i] = j < K ? a.ids[row * K + j] : -1;
        lq_in[i] = j < K ? a.lq[row * K + j] : 0.f;
      }
      if (a.weight) w_in = a.weight[row];
    };
    auto prepare = [&](uint32_t k) {
      int id[kPerLane], n;
      bool bad;
      table_row<F>(a, sm.tab[k & 1], id_in, id, n, bad, lane, err);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.table[k & 1]));
      teacher_values(a, sm.tab[k & 1], id, lq_in, w_in, n, bad, scale, lane);
      __syncwarp();
    };
    long long row = rows.next(stride, lane);
    fetch(row);
    long long row_1 = row >= 0 ? rows.next(stride, lane) : -1;
    if (row >= 0) prepare(0);
    fetch(row_1);
    long long row_2 = row_1 >= 0 ? rows.next(stride, lane) : -1;
    if (row_1 >= 0) prepare(1);
    fetch(row_2);
    for (uint32_t k = 0; row >= 0; ++k) {
      EntryTable& tab = sm.tab[k & 1];
      if (!__all_sync(0xffffffffu, wait_bounded<false>(smem_addr(&sm.sums), k & 1, abort))) break;
      RowStats tail = join_parts<kWarps>(sm.part, F::kFloor, a.c, lane);
      int id[kPerLane];
      float z[kPerLane];
      bool mine[kPerLane];  // in this CTA's slice
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        id[i] = tab.id[lane + 32 * i];
        mine[i] = kCluster ? id[i] >= e0 && id[i] < e0 + n_elems : id[i] >= 0;
        z[i] = mine[i] ? tab.z[lane + 32 * i] : -INFINITY;
      }
      if (kCluster) {
        // everything to everyone; the same values follow in every CTA
        for (int q = 0; q < csize; ++q) {
#pragma unroll
          for (int i = 0; i < kPerLane; ++i)
            if (mine[i]) st_cluster_f32(map_to_rank(smem_addr(&sm.slice_z[lane + 32 * i]), q), z[i]);
          if (lane == 0) {
            const uint32_t to = map_to_rank(smem_addr(&sm.slice_tail[rank]), q);
            st_cluster_f32(to, tail.m);
            st_cluster_f32(to + 4, tail.r);
          }
        }
        fence_cluster();
        __syncwarp();
        if (lane < csize) mbar_arrive_remote(map_to_rank(smem_addr(&sm.slices), lane));
        if (!__all_sync(0xffffffffu, wait_bounded<true>(smem_addr(&sm.slices), 0, abort))) break;
        tail = RowStats{sm.slice_tail[0].x, sm.slice_tail[0].y, 0.f};
        for (int q = 1; q < csize; ++q)
          tail = merge_row(tail, RowStats{sm.slice_tail[q].x, sm.slice_tail[q].y, 0.f}, a.c);
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) z[i] = id[i] >= 0 ? sm.slice_z[lane + 32 * i] : -INFINITY;
      }
      float M = tail.m;
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) M = max_nan(M, z[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
      const bool plain = needs_exact<F>(M, a.c);
      if (plain) {
        tail = exact_tail<F>(a.logits + row * a.row_bytes, V, a.c, tab, lane);
        if (kCluster) {  // no CTA may write its slice (of logits in place) before all have read the row
          __syncwarp();
          if (lane < csize) mbar_arrive_remote(map_to_rank(smem_addr(&sm.read_again), lane));
          if (!__all_sync(0xffffffffu, wait_bounded<true>(smem_addr(&sm.read_again), 0, abort))) break;
        }
        M = tail.m;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) M = max_nan(M, z[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
      }
      float d[kPerLane];
      const RowSums t = row_values(a, tab, id, z, tail, M, d, lane);
      if (lane == 0) {
        sm.m = t.m;
        sm.factor = t.factor;
        sm.plain = plain;
        mbar_arrive(smem_addr(&sm.values));
        if (rank == 0) {
          acc[0] += t.loss;
          acc[1] += t.fwd;
          acc[2] += t.rev;
          acc[3] += t.qt;
          acc[4] += t.pt;
          if (a.row_loss) a.row_loss[row] = static_cast<float>(t.loss);
        }
      }
      // this row's table for the row after next (every consumer is past its first pass)
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (id[i] >= 0) tab.head[(id[i] / F::kPiece) & (kTable - 1)] = 0;
      __syncwarp();
      const long long done_row = row;
      row = row_1;
      row_1 = row_2;
      row_2 = row_1 >= 0 ? rows.next(stride, lane) : -1;
      if (row_1 >= 0) prepare(k);
      fetch(row_2);
      // the given tokens' gradients over what the consumers have written there
      if (a.dlogits) {
        if (!__all_sync(0xffffffffu, wait_bounded<false>(smem_addr(&sm.written), k & 1, abort))) break;
        unsigned char* dst = a.dlogits + done_row * a.row_bytes;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (mine[i]) F::store(dst, id[i], d[i]);
      }
    }
    // this CTA's sums, then the last CTA adds all of them in CTA order
    err = __reduce_or_sync(0xffffffffu, err);
    bool last = false;
    if (lane == 0) {
      if (*abort) err |= RL_DEVERR_TIMEOUT;
      if (err) atomicOr(&a.ws->status, err);
      WsPartial& P = a.partials[blockIdx.x];
      for (int i = 0; i < 5; ++i) P.v[i] = acc[i];
      __threadfence();
      last = atomicInc(&a.ws->ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    if (__shfl_sync(0xffffffffu, last, 0)) {
      __threadfence();
      double v[5] = {0.0, 0.0, 0.0, 0.0, 0.0};
      const int n = static_cast<int>(gridDim.x);
      for (int i0 = lane; i0 < n; i0 += 128) {  // four CTAs' loads in flight
        double p[4][5];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < 5; ++q) p[j][q] = i0 + 32 * j < n ? __ldcg(&a.partials[i0 + 32 * j].v[q]) : 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < 5; ++q) v[q] += p[j][q];
      }
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
        if (stw & RL_DEVERR_TIMEOUT) lose_record(o);
        *a.stats = o;
        if (a.loss_out) *a.loss_out = static_cast<float>(o.loss);
      }
    }
  } else {
    // ---------------------------------------------------------------- consumers
    count_rows(a, sm.wcount, tid);
    // masked rows: an all-zero gradient, shared out evenly
    if (a.mask) {
      RowsOf<false> masked(a.mask, a.R, first, lane);
      for (long long row = masked.next(stride, lane); row >= 0; row = masked.next(stride, lane)) {
        if (tid == 0 && rank == 0 && a.row_loss) a.row_loss[row] = 0.f;
        if (!a.dlogits) continue;
        unsigned char* dst = a.dlogits + row * a.row_bytes + b0;
        for (int v = tid; v < n_vecs; v += kThreads) {
          if ((v + 1) * F::kVec <= n_elems)
            st_global_cs_v4(dst + static_cast<long long>(v) * 16, make_uint4(0u, 0u, 0u, 0u));
          else
            for (int i = v * F::kVec; i < n_elems; ++i) F::store(dst, i, 0.f);
        }
      }
    }
    const int n_full = n_elems / F::kPiece / kThreads;  // chunks whose every piece is a full one
    uint32_t it = 0;
    WarpSum st;  // of the row whose first pass is under way
    // pass 1 over chunks [i0, i1) of the k-th row: every token that is not given
    auto pass1 = [&](uint32_t k, int i0, int i1) {
      EntryTable& tab = sm.tab[k & 1];
      for (int i = i0; i < i1; ++i, ++it) {
        const uint32_t buf = sm.ring.wait(it, abort);
        const int p = i * kThreads + tid;
        const bool last = i >= n_full;
        uint32_t w[16];
        const int sh = last ? 0 : lane >> 1;
        load_piece(w, 0, buf + tid * kPieceBytes, sh);
        int j = p < n_mine ? tab.head[(g0 + p) & (kTable - 1)] : 0;
        while (j) {
          const int e = tab.id[j - 1] - (g0 + p) * F::kPiece;
          if (e >= 0 && e < F::kPiece) {
            tab.z[j - 1] = F::load_shared(sm.ring.data[it % S::kSlots] + tid * kPieceBytes, e);
            F::drop(w, 0, (((e / F::kVec) - sh) & 3) * F::kVec + e % F::kVec);
          }
          j = tab.next[j - 1];
        }
        sm.ring.release(it, lane);
        if (last) F::cut(w, 0, p < n_mine ? min(F::kPiece, n_elems - p * F::kPiece) : 0);
        __syncwarp();
        if (i == 0) sum_init<F>(st, w, a.c);
        sum_piece<F>(st, w, a.c);
      }
    };
    // pass 2: 2^((z - m) c) factor.  16-bit outputs take |factor| into the
    // exponent and the sign on the packed result: the offset b = log2|factor| -
    // m c is rounded by at most 2^-15 for |b| <= 1024, 2.1e-5 of the result, a
    // twelfth to a 23rd of fp16's own half step.  Beyond, and where a row is taken by
    // differences, they multiply, as fp32 outputs do.
    const int n_full2 = n_vecs / kVecs - (n_elems % F::kVec && n_vecs % kVecs == 0 ? 1 : 0);  // chunks of full vectors only
    auto pass2 = [&](long long row) {
      unsigned char* dst = a.dlogits + row * a.row_bytes + b0;
      const float m = sm.m, factor = sm.factor;
      constexpr bool kFold = F::kBytes == 2;
      const float nm = __fmul_rn(-m, a.c), rho = fmaf(-m, a.c, -nm);
      const float add = kFold ? log2f(fabsf(factor)) : 0.f;
      const float b = kFold ? nm + (rho + add) : nm;
      const bool plain = sm.plain != 0 || (kFold && factor != 0.f && !(fabsf(b) <= 1024.f));  // by differences to m
      const float mul = kFold ? 1.f : plain ? factor : factor * ex2_approx(rho);
      const uint32_t sign = kFold && factor < 0.f ? 0x80008000u : 0u;
      const float2 c2 = make_float2(a.c, a.c), m2 = make_float2(mul, mul);
      const float2 b2 = make_float2(b, b);
      auto vec = [&](const uint4& w) {
        float z[F::kVec];
        F::unpack(w, z);
#pragma unroll
        for (int j = 0; j < F::kVec; j += 2) {
          const float2 x = __ffma2_rn(make_float2(z[j], z[j + 1]), c2, b2);
          float2 d = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          if (!kFold) d = __fmul2_rn(d, m2);
          z[j] = d.x;
          z[j + 1] = d.y;
        }
        uint4 u = F::pack(z);
        if (kFold) u = make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
        return u;
      };
      auto vec_plain = [&](const uint4& w) {
        float z[F::kVec];
        F::unpack(w, z);
#pragma unroll
        for (int j = 0; j < F::kVec; ++j) z[j] = ex2_approx((z[j] - m) * a.c) * factor;
        return F::pack(z);
      };
      for (int i = 0; i < n_chunks; ++i, ++it) {
        const uint32_t buf = sm.ring.wait(it, abort);
        uint4 w[kVecsPerThread];
#pragma unroll
        for (int q = 0; q < kVecsPerThread; ++q) w[q] = ld_shared_v4(buf + (tid + q * kThreads) * 16);
        sm.ring.release(it, lane);
        const int v0 = i * kVecs + tid;
        unsigned char* out = dst + static_cast<long long>(v0) * 16;
        if (i < n_full2 && !plain) {
#pragma unroll
          for (int q = 0; q < kVecsPerThread; ++q) st_global_cs_v4(out + q * kThreads * 16, vec(w[q]));
        } else {
#pragma unroll 1
          for (int q = 0; q < kVecsPerThread; ++q) {
            const int v = v0 + q * kThreads;
            uint4 wq = w[0];
#pragma unroll
            for (int j = 1; j < kVecsPerThread; ++j) wq = j == q ? w[j] : wq;
            const uint4 u = plain ? vec_plain(wq) : vec(wq);
            if ((v + 1) * F::kVec <= n_elems) {
              st_global_cs_v4(out + q * kThreads * 16, u);
            } else if (v < n_vecs) {
              float z[F::kVec];
              F::unpack(u, z);
#pragma unroll
              for (int j = 0; j < F::kVec; ++j)
                if (v * F::kVec + j < n_elems) F::store(dst, v * F::kVec + j, z[j]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.written));
    };
    // Each step: the first `lead` chunks of the next row's first pass (the time
    // the row warp has for the row before), that row's second pass, then the
    // rest of the first pass.  The first step has no row before, the last no
    // next one.  After a timeout the whole warp stops; nothing meets another warp.
    long long prev = -1;
    for (uint32_t k = 0;; ++k) {
      sm.ring.wait(it, abort);
      const long long row = sm.row_of[it % S::kSlots];
      if (__any_sync(0xffffffffu, *abort)) break;
      const int lead_q = prev >= 0 ? lead : n_chunks;
      if (row >= 0) {
        wait_bounded<false>(smem_addr(&sm.table[k & 1]), (k >> 1) & 1, abort);
      } else {
        sm.ring.release(it++, lane);  // the end's empty chunk
      }
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        if (row >= 0) pass1(k, part ? lead_q : 0, part ? n_chunks : lead_q);
        if (part == 0 && prev >= 0) {
          wait_bounded<false>(smem_addr(&sm.values), (k - 1) & 1, abort);
          if (a.dlogits) pass2(prev);
        }
      }
      if (row < 0) break;
      const RowStats ws = warp_sum_stats<F>(st, a.c);
      if (lane == 0) sm.part[warp] = ws;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.sums));
      prev = row;
    }
  }
  if (kCluster) cluster_sync_all();  // no CTA leaves while another may still write its memory
  // A wait has given up: every row's outputs become NaN.  Each warp writes all of
  // them once it is done, for a warp that wrote wrong values finds `abort` set, and
  // what other warps and CTAs write later is right.  (A barrier before it cost the
  // 32-thread build 8%: registers.)
  if (*abort) lose_rows<F>(a.row_loss, a.dlogits, a.R, a.row_bytes, V, lane);
}

// ------------------------------------------------------------------ host side
template <int DT, int kThreads, int kCtas, bool kCluster>
rl_status launch(const DistillArgs& a, int cluster, int dev, int sms, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(&topk_distill_kernel<DT, kThreads, kCtas, kCluster>);
  const int smem = static_cast<int>(sizeof(DistillSmem<kThreads>));
  static std::atomic<unsigned long long> allowed{0};
  const rl_status st = allow_smem(fn, dev, smem, allowed);
  if (st != RL_OK) return st;
  long long grid = static_cast<long long>(kCtas) * sms;
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (kCluster || grid > a.R) grid = a.R > 0 ? a.R * cluster : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads + 64);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, topk_distill_kernel<DT, kThreads, kCtas, kCluster>, a) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

// CTAs of 128 threads that share a row: up to 8, each with a few chunks, where
// that leaves two a SM at most.  Rows x 151,936 bf16, 64 entries, us on 8 CTAs
// and on one of 512 threads: 1 row 16.4, 22.2; 38 rows 20.8, 22.4; 64 rows 22.6,
// 23.0; 76 rows 26.5, 23.0.  A row costs the entries' table, the exchange and the
// values once in any case.
int cluster_for(long long R, long long n_pieces, int sms) {
  int c = 1;
  if (R > 0 && R * kMaxCluster <= 2LL * sms && R * kMaxCluster <= kMaxGrid)
    while (c < kMaxCluster && n_pieces >= static_cast<long long>(c) * 4 * 128) c *= 2;
  return c;
}

// Rows of more than kLongRow bytes go one to a SM, on 512 consumer threads: the
// second pass finds them in L2 then.  Shorter rows go four to a SM, on 128
// each, so that one row's serial part overlaps the others' passes.  512 x 1
// against 128 x 4, us, bf16: 4096 x 151,936: 427, 585; 4096 x 60,000: 208, 208;
// 4096 x 50,000: 205, 177; 16,384 x 32,000: 561, 465; 16,384 x 8000: 522, 205.
// Many rows of at most kTinyRow bytes, which are bound by the row warp's serial
// steps, go seven to a SM, on 32 consumer threads each: 32,768 x 1000 bf16, 16
// entries: 271 against 176; x 2000: 268, 209; x 4000: 271, 285; 1100 x 1000: 24, 26.
constexpr long long kLongRow = 100 * 1024, kTinyRow = 4 * 1024;

template <int DT>
rl_status launch_any(const DistillArgs& a, int dev, int sms, cudaStream_t stream) {
  const int c = cluster_for(a.R, (a.V + Fmt<DT>::kPiece - 1) / Fmt<DT>::kPiece, sms);
  if (c > 1) return launch<DT, 128, 4, true>(a, c, dev, sms, stream);
  const long long bytes = a.V * Fmt<DT>::kBytes;
  if (bytes > kLongRow) return launch<DT, 512, 1, false>(a, 1, dev, sms, stream);
  if (bytes <= kTinyRow && a.R >= 14LL * sms) return launch<DT, 32, 7, false>(a, 1, dev, sms, stream);
  return launch<DT, 128, 4, false>(a, 1, dev, sms, stream);
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
  if (d->mask && R > kMaxMaskedRows) return RL_ERR_SHAPE;
  if (d->K < 1 || d->K > RL_TOKEN_MAX_K || !(d->reverse >= 0.f && d->reverse <= 1.f) ||
      !(d->temperature >= kMinTemperature && d->temperature <= kMaxTemperature) || !std::isfinite(d->grad_scale) ||
      !(d->norm >= 0.0) || !std::isfinite(d->norm) || (d->reverse != 0.f && d->tail == RL_DISTILL_TAIL_RENORM))
    return RL_ERR_ARG;
  if (!d->stats_dev) return RL_ERR_NULL;
  if (!d->workspace || d->workspace_bytes < kWorkspaceBytes) return RL_ERR_WORKSPACE;
  if (R > 0 && (!d->logits || !d->teacher_ids || !d->teacher_logp)) return RL_ERR_NULL;
  const long long row_bytes = ld * es;
  if ((reinterpret_cast<uintptr_t>(d->logits) & 15) || (reinterpret_cast<uintptr_t>(d->dlogits) & 15) || (row_bytes & 15) ||
      (reinterpret_cast<uintptr_t>(d->workspace) & 15) || (reinterpret_cast<uintptr_t>(d->stats_dev) & 7))
    return RL_ERR_ALIGN;
  if (d->dlogits && d->dlogits != d->logits && rows_overlap(d->logits, d->dlogits, R, row_bytes, V * es)) return RL_ERR_ALIAS;
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
  a.temperature = d->temperature;
  a.reverse = d->reverse;
  a.grad_scale = d->grad_scale;
  a.norm = d->norm;
  a.K = d->K;
  a.renorm = d->tail == RL_DISTILL_TAIL_RENORM;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (d->dtype) {
    case RL_F32: return launch_any<RL_F32>(a, dev, sms, s);
    case RL_BF16: return launch_any<RL_BF16>(a, dev, sms, s);
    case RL_F16: return launch_any<RL_F16>(a, dev, sms, s);
  }
  return RL_ERR_DTYPE;
}
