// verify_drafts.cu — rl_verify_drafts: which drafted tokens a sequence keeps,
// and the token drawn after them (include/rlrollout.h).
//
// A cluster of 1 to 16 CTAs takes a sequence; each warp has a part of every row.
//  1. The sequence's target rows in order, until a draft does not stay: maximum
//     and sum of e^((z - m) / T) of the row in one pass, fp32, online, with the warp's
//     maximum as the frame (one FMA an element: x = z c + nm; the rounding of nm = -m c, common
//     to a frame's terms, is put right when the frame ends).  A maximum that rises by less than 2^4 keeps
//     the frame: each change costs the sum some units of its last place, and a row may rise all along (2^26
//     fp32 numbers from 0 to 0.01: off by 669 units with a frame for each maximum, by 3 so).  The maxima, whose terms are exactly 1,
//     are counted beside the sum, so that log S keeps its relative precision
//     where one token holds nearly all the mass.  Rows behind a refused draft
//     are not read.
//  2. The token.  The sums of the warps' parts, then of parts of that part, lead to the
//     one in which the running sum passes the border u S.  These fp32 sums are good to
//     kCoarse of S (below): where the border is nearer than that to either side of the
//     token's own weight, everything is summed again in fine arithmetic (fine_exp.cuh).
//  3. Where a draft with a distribution was refused, the weights max(p - q, 0)
//     are sums of differences, and always taken in fine arithmetic, in one pass over
//     the target's and the draft's row: S is known to fp32 from step 1, and W - S Q of the sums over the set of tokens
//     with p > q takes the S of the same pass.  The set is right but for tokens with p / q within S's error of 1; what they
//     have of q is summed too, and where it counts (a draft's row that nearly equals the target's) the pass is made again with the
//     new S.
//
// What bounds it.  One row of 151,936 bf16 logits takes 9.6 us: launch, one pass (2 us) and a
// chain of short steps; 21 where it falls back to fine sums.  Few sequences are such chains of rows (64 with four drafts each: 73 us,
// 71 where all stay).  Many are bound by instructions and their latency where drafts are refused, 66 packed operations for two
// tokens of both rows (512 with four drafts: 328 us, all kept 265).  Draws are bound by waiting: one CTA of a cluster searches
// while the others stand at its barrier, the last round of clusters is nearly empty (512: 67 us, 2.3 TB/s), and where a row
// falls back its few CTAs sum it again while the rest of the chip has nothing to do (512: 116 us; 64: 42, 20 where none does).
//
// fp32 sums, in units of 2^-24: a term 2^x carries 4 of the hardware exponential and 2 ln 2 |x|
// of its argument (the FMA's rounding and c's), |x| weighted by p at most log2 V <= 26;
// 32 terms are added in chains of 10, the chains' sums with their errors kept; then
// 12 where a frame ends, 5 joins in the warp, 10 for the frames of lanes and warps, and up to 50 roundings in the running
// sums of the search.  What a comparison with the border takes of the terms' errors is at most half of the largest (they are in
// the total too), 45 units if all that depends on the values adds up, and the roundings of the search are of both signs.
// Over 6 10^5 batches of rows built to add them up (halves, blocks and cycles of few values, ramps, one value just below a
// top, sorted ones; 2,000 to 400,000 numbers of each type, temperatures of 0.011 to 90) a token drawn from the fp32 sums
// alone was never further than 12.3 units of S from its border.  Where the border is within 32 units the fine sums decide.
// (64 units, more than all but the search can add up to: a draw of 24 rows in turn 11.6 us against 10.6, 64 draws 42.0 against 41.0, 512
// 121 against 117.  192 units, the sum of all bounds: 22% of N(0, 9) rows fell back instead of 5%.)  fp64 is kept for what a
// single lane decides: the unit does two operations a cycle and SM, and a warp that adds in fp64 holds it for 16 cycles.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "fine_exp.cuh"
#include "rlrollout.h"
#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtasPerSm = 3;
constexpr int kMaxCluster = 16, kMaxParts = kMaxCluster * kWarps;
constexpr double kLog2eD = 1.4426950408889634074;
constexpr float kSlack = 4.f;         // a frame stays while the maximum's term is below 2^4
constexpr float kCoarse = 0x1p-19f;  // 2.6 times the largest error met (above)
constexpr float kWindow = 0x1p-17f;   // of p / q around 1, in which a row's fp32 sum may leave open which is larger
constexpr double kOpen = 0x1p-17;     // relative: a draft's test that is nearer asks for the row's fine sum
constexpr float kNothing = 0x1p-90f;  // sums of weights that are 0 (e^-86 each) stay below

struct Args {
  const unsigned char* target;
  const unsigned char* draft;
  const float* draft_lse;
  const long long* ids;
  const int* n_draft;
  const double* u;
  long long V, row_bytes, draft_bytes;
  int G;
  float c;             // log2(e) / temperature
  float T, r_hi, r_lo;  // temperature, and 1 / temperature as two floats
  double inv_t;        // 1 / temperature
  long long* tokens;
  long long* n_accepted;
  float* logp;
  float* lse;
  unsigned int* status;
};

// Which weights a token is drawn from: p; p without the drafted token; max(p - q, 0).
enum Mode { kSoftmax, kWithout, kRest };

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

enum Verdict { kStays, kRefused, kNoDistribution, kNear };

// What the CTAs of a cluster tell one another, in turn in two places: whoever writes the
// one has passed the barrier behind which everybody had read the other.
struct Exchange {
  Stats stats[kMaxParts];  // of a fine pass over two rows: (q beside p, -, q below p)
  Wide sum[kMaxParts], plus[kMaxParts];
  long long token;
  int unsure;
};
// Of a warp's ring: one chunk on its way while one is read.  What shared memory leaves is L1, which the
// passes behind the first read through (64 x 151,936, four drafts: with 4 slots 4% longer, with 3 3%).
constexpr int kSlots = 2, kChunkBytes = 2048;
struct Smem {
  unsigned long long full[kWarps][kSlots];
  uint2 powers[kPow];
  Exchange ex[2];
  Wide sums[kWarps];   // of the search
  float top[kWarps];   // of the row, the warps' maxima
  float coarse[kWarps];
  float gap;
  long long found;
  int verdict;
  Wide u;              // for the draw
  double left, right;  // of a draft's test that fp32 sums leave open: u q, and p's term
};

// ------------------------------------------------------------------ the cluster
struct Group {
  int size, rank;  // CTAs of the cluster
  uint32_t turn;
  __device__ __forceinline__ void sync() const {
    if (size > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
};

template <class T>
__device__ __forceinline__ void put(uint32_t addr, const T& v) {
  static_assert(sizeof(T) % 4 == 0, "words");
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 4); ++i)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr + 4 * i), "r"(w[i]) : "memory");
}
// v at `place` of this CTA, written in every CTA of the cluster by the lanes of a warp.
template <class T>
__device__ __forceinline__ void tell(const Group& g, T* place, const T& v, int lane) {
  if (lane < g.size) put(map_to_rank(smem_addr(place), lane), v);
}

// ------------------------------------------------------------------ rows
// elements behind `end` become -inf in a vector that begins at i
template <int DT>
__device__ __forceinline__ void cut_vec(uint4& v, long long i, long long end) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const int n = static_cast<int>(end - i);  // of those, valid
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (DT == RL_F32) {
      if (j >= n) w[j] = 0xff800000u;
    } else {
      if (2 * j >= n)
        w[j] = Fmt<DT>::kNegInf2;
      else if (2 * j + 1 >= n)
        w[j] = (w[j] & 0xffffu) | (Fmt<DT>::kNegInf2 & 0xffff0000u);
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}

// The next load of this lane, from element i on, comes to L1.
template <int DT>
__device__ __forceinline__ void fetch(const unsigned char* row, long long i, long long end) {
  i += 32 * Fmt<DT>::kVec;
  if (i < end) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + i * Fmt<DT>::kBytes));
}

// 16 bytes of a row from element i on (the stride is a multiple of that); -inf behind `end`.
template <int DT>
__device__ __forceinline__ uint4 load_vec(const unsigned char* row, long long i, long long end) {
  uint4 v = make_uint4(Fmt<DT>::kNegInf2, Fmt<DT>::kNegInf2, Fmt<DT>::kNegInf2, Fmt<DT>::kNegInf2);
  if (i < end) {
    v = __ldg(reinterpret_cast<const uint4*>(row + i * Fmt<DT>::kBytes));
    if (i + Fmt<DT>::kVec > end) cut_vec<DT>(v, i, end);
  }
  return v;
}

// Where part p of n of [begin, end) begins, parts being multiples of a warp's vectors.
__device__ __forceinline__ long long part_size(long long length, int n, int step) {
  return ((length + n - 1) / n + step - 1) / step * step;
}

// The chunks of a warp's part of the rows, in the order of the rows: bulk copies into a ring
// of its own in shared memory.  They run ahead of the warp, into the next row too
// before it is known whether that is needed, so that a row's end costs no waiting for memory.
template <int DT>
struct Stream {
  static constexpr int kElems = kChunkBytes / Fmt<DT>::kBytes;
  const unsigned char* next;  // row of the next copy, from the part's first element on
  long long row_bytes, length, at;  // bytes to the next row; elements of the part, and of them copied
  int rows;                   // rows left to copy
  uint32_t data, bars, issued, taken;
  uint64_t policy;

  __device__ __forceinline__ void init(const unsigned char* row, long long row_bytes_, int rows_, long long lo, long long hi,
                                       uint32_t data_, uint32_t bars_, int lane) {
    next = row + lo * Fmt<DT>::kBytes;
    row_bytes = row_bytes_;
    length = hi - lo;
    at = 0;
    rows = length > 0 ? rows_ : 0;
    data = data_;
    bars = bars_;
    issued = taken = 0;
    policy = policy_normal();
    for (int j = 0; j < kSlots - 1; ++j) copy(lane);
  }
  __device__ __forceinline__ void copy(int lane) {
    if (rows == 0) return;
    const uint32_t slot = issued % kSlots;
    if (lane == 0) {
      const long long left = (length - at) * Fmt<DT>::kBytes;  // (the stride is a multiple of 16)
      const uint32_t bytes = left >= kChunkBytes ? kChunkBytes : static_cast<uint32_t>((left + 15) & ~15LL);
      mbar_arrive_expect_tx(bars + 8 * slot, bytes);
      bulk_load(data + slot * kChunkBytes, next + at * Fmt<DT>::kBytes, bytes, bars + 8 * slot, policy);
    }
    ++issued;
    at += kElems;
    if (at >= length) {
      at = 0;
      next += row_bytes;
      --rows;
    }
  }
  // The next chunk's words of this lane; its vectors are j 32 kVec + lane kVec elements from the
  // chunk's begin, of which `left` belong to the part.  false: a wait gave up.
  __device__ __forceinline__ bool take(uint32_t (&w)[16], long long left, int lane, volatile int* abort) {
    __syncwarp();  // the slot before is read
    copy(lane);
    const uint32_t slot = taken % kSlots;
    const bool ok = __all_sync(0xffffffffu, wait_bounded<false>(bars + 8 * slot, (taken / kSlots) & 1, abort));
    ++taken;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 v = ld_shared_v4(data + slot * kChunkBytes + j * 512 + lane * 16);
      if (left < kElems) {
        const int i = (j * 32 + lane) * Fmt<DT>::kVec;
        if (i + Fmt<DT>::kVec > left) cut_vec<DT>(v, i, left);
      }
      w[4 * j] = v.x;
      w[4 * j + 1] = v.y;
      w[4 * j + 2] = v.z;
      w[4 * j + 3] = v.w;
    }
    return ok;
  }
  // copies still on their way land before the CTA can exit
  __device__ __forceinline__ void drain(volatile int* abort) {
    for (; taken < issued; ++taken) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(bars + 8 * (taken % kSlots), (taken / kSlots) & 1) && global_ns() - t0 <= kWaitLimitNs) {
      }
    }
  }
};

// A warp's statistics of its part of the stream's next row, in every lane.
template <int DT>
__device__ __forceinline__ Stats part_stats(Stream<DT>& in, float c, int lane, volatile int* abort) {
  using F = Fmt<DT>;
  float m = F::kFloor, nm = -F::kFloor * c;
  float n = 0.f, s = 0.f, err = 0.f;
  bool ok = true;
#pragma unroll 1
  for (long long left = in.length; left > 0; left -= Stream<DT>::kElems) {
    uint32_t w[16];
    ok = in.take(w, left, lane, abort) && ok;
    float wm;
    {
      const float pm = max_nan(F::raw_value(F::raw_max(w, 0)), F::kFloor);
      asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(wm) : "f"(pm));
    }
    if (!(wm < m)) {
      if (!(wm == m)) {  // the old maxima join the sum
        float lost;
        s = two_sum(s, n * ex2_approx(fmaf(m, c, nm)), lost);
        err += lost;
        n = 0.f;
        m = max_nan(m, wm);  // (a NaN stays)
        if (!(fmaf(m, c, nm) < kSlack)) {  // the frame ends, and its sum goes along
          s = (s + err) * ex2_approx(-fmaf(m, c, nm));
          err = 0.f;
          nm = -m * c;
          // what the new frame's terms are off by, s is now off by too
          s *= ex2_approx(-fmaf(-m, c, -nm));
        }
      }
      n += static_cast<float>(F::template drop_value<16>(w, m, true));
    }
    const float2 c2 = make_float2(c, c), nm2 = make_float2(nm, nm);
    float2 t0 = make_float2(0.f, 0.f), t1 = t0;
#pragma unroll
    for (int i = 0; i < F::kPiece / 2; ++i) {
      float2 z;
      F::template pair<16>(w, i, z.x, z.y);
      const float2 x = __ffma2_rn(z, c2, nm2);
      const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      if (i & 1)
        t1 = __fadd2_rn(t1, e);
      else
        t0 = __fadd2_rn(t0, e);
    }
    float lost;
    s = two_sum(s, (t0.x + t0.y) + (t1.x + t1.y), lost);
    err += lost;
  }
  s = (s + err) * ex2_approx(fmaf(-m, c, -nm));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  return Stats{ok ? m : __int_as_float(0x7fc00000), n, s};  // a wait that gave up: no distribution
}

// The same by differences to the maximum, without a floor: rows of very large
// or very small numbers.
template <int DT>
__device__ __noinline__ Stats part_stats_exact(const unsigned char* row, long long lo, long long hi, float c, int lane) {
  using F = Fmt<DT>;
  Stats a{-FLT_MAX, 0.f, 0.f};
  float frame = a.m, err = 0.f, lost;
  for (long long i = lo + lane * F::kVec; i < hi; i += 32 * F::kVec) {
    float z[F::kVec];
    F::unpack(load_vec<DT>(row, i, hi), z);
    float vm = z[0];
#pragma unroll
    for (int j = 1; j < F::kVec; ++j) vm = max_nan(vm, z[j]);
    if (!(vm < a.m)) {
      if (!(vm == a.m)) {
        a.s = two_sum(a.s, a.n * ex2_approx((a.m - frame) * c), lost);
        err += lost;
        a.n = 0.f;
        a.m = max_nan(a.m, vm);
        if (!((a.m - frame) * c < kSlack)) {
          a.s = (a.s + err) * ex2_approx((frame - a.m) * c);
          err = 0.f;
          frame = a.m;
        }
      }
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) {
        if (z[j] == a.m) {
          a.n += 1.f;
          z[j] = -INFINITY;
        }
      }
    }
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < F::kVec; ++j) t += ex2_approx((z[j] - frame) * c);
    a.s = two_sum(a.s, t, lost);
    err += lost;
  }
  a.s = (a.s + err) * ex2_approx((frame - a.m) * c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merged(a, Stats{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.n, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, c);
  return a;
}

// ------------------------------------------------------------------ weights
// log p of logit z of a row.
__device__ __forceinline__ float log_prob(float z, const Stats& st, double inv_t) {
  return static_cast<float>((static_cast<double>(z) - static_cast<double>(st.m)) * inv_t - log1pf((st.n - 1.f) + st.s));
}

// q = e^(z / temperature - lse) (fp64's own exponential is some hundred dependent steps of a
// unit with a 64th of fp32's rate, and everybody waits for this one number).
template <bool kUnit>
__device__ __forceinline__ double draft_prob(float z, float lse, const Args& a, const uint2* powers) {
  const double x = static_cast<double>(z) * a.inv_t - static_cast<double>(lse);
  if (!(x > -80.0 && x < 1.0 && fabsf(lse) < 256.f)) return exp(x);
  FineExp q;
  q.init_around(a.r_hi, a.r_lo, a.T, a.inv_t, lse, Wide(0.f), -86.f);
  const Wide v = q.template at<true, false, kUnit>(z, powers).value();
  return static_cast<double>(v.h) + static_cast<double>(v.l);
}

// u e^x S < e^y, for what fp32 or fp64 numbers do not hold: y below -86, or u = 0 beside a q that may be anything.
__device__ __noinline__ bool stays_by_logs(double u, double x, double S, double y) {
  if (!(y > -INFINITY)) return false;
  return u <= 0.0 || log(u) + x + log(S) < y;
}

template <int DT, int MODE, bool kFine, bool kUnit>
struct Weights {
  const unsigned char* row;
  const unsigned char* draft_row;
  long long without;
  float c, nm;      // coarse: 2^(z c + nm)
  FineExp p, q;
  const uint2* powers;
  float start;      // fine: a power of two, twice the weights or more

  __device__ __forceinline__ Term2 fine(float2 z) const { return p.template at<DT == RL_F32, false, kUnit>(z, powers); }
  __device__ __forceinline__ Term2 drafted(float2 z) const { return q.template at<DT == RL_F32, true, kUnit>(z, powers); }

  // a vector's logits, -inf behind `end` and at the token that is left out
  __device__ __forceinline__ void logits(long long i, long long end, float (&z)[Fmt<DT>::kVec]) const {
    Fmt<DT>::unpack(load_vec<DT>(row, i, end), z);
    if (MODE == kWithout && without >= i && without < i + Fmt<DT>::kVec) {
#pragma unroll
      for (int j = 0; j < Fmt<DT>::kVec; ++j)
        if (i + j == without) z[j] = -INFINITY;
    }
  }
  // weights of elements i .. i + kVec - 1, in pairs
  __device__ __forceinline__ void at(long long i, long long end, Term2 (&w)[Fmt<DT>::kVec / 2]) const {
    using F = Fmt<DT>;
    float z[F::kVec], y[F::kVec];
    logits(i, end, z);
    if (MODE == kRest) F::unpack(load_vec<DT>(draft_row, i, end), y);
#pragma unroll
    for (int j = 0; j < F::kVec / 2; ++j) {
      const float2 zz = make_float2(z[2 * j], z[2 * j + 1]);
      if (!kFine) {
        const float2 x = __ffma2_rn(zz, both(c), both(nm));
        w[j].a = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        w[j].b = w[j].c = both(0.f);
      } else {
        w[j] = fine(zz);
        if (MODE == kRest) {
          float2 more;
          w[j] = above(w[j], drafted(make_float2(y[2 * j], y[2 * j + 1])), more);
          w[j].a = mul2(w[j].a, more);
          w[j].b = mul2(w[j].b, more);
          w[j].c = mul2(w[j].c, more);
        }
      }
    }
  }
  // the same as numbers, 0 where a token cannot occur
  template <class N>
  __device__ __forceinline__ void exactly(long long i, long long end, N (&x)[Fmt<DT>::kVec]) {
    using F = Fmt<DT>;
    float z[F::kVec];
    Term2 w[F::kVec / 2];
    logits(i, end, z);
    at(i, end, w);
#pragma unroll
    for (int j = 0; j < F::kVec; ++j) {
      const Term x1 = j & 1 ? w[j / 2].y() : w[j / 2].x();
      if constexpr (kFine)
        x[j] = p.is_zero(z[j]) ? Wide(0.f) : x1.value();
      else
        x[j] = x1.a;
    }
  }
};

// Where sums of a part's terms start: four times e^((top - m) / T) at most, as a power of two.
__device__ __forceinline__ float fine_start(float top, const FineExp& p, float c) {
  const float x = ceilf(((top - p.off) - p.m) * c) + 1.f;
  return __int_as_float((127 + static_cast<int>(fminf(fmaxf(x, -60.f), 1.f))) << 23);
}

template <class N>
__device__ __forceinline__ N warp_sum(N v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += from_xor(v, o);
  return v;
}

// The warp's sum over [lo, hi) in fine arithmetic, whole vectors from lo.
template <int DT, int MODE, bool kUnit>
__device__ __forceinline__ Wide part_sum(Weights<DT, MODE, true, kUnit>& f, long long lo, long long hi, int lane) {
  using F = Fmt<DT>;
  Wide total(0.f);
  FineSum s;
  s.clear(f.start);
  int n = 0;
#pragma unroll 1
  for (long long i = lo + lane * F::kVec; i < hi; i += 32 * F::kVec) {
    Term2 w[F::kVec / 2];
    fetch<DT>(f.row, i, hi);
    f.at(i, hi, w);
#pragma unroll
    for (int j = 0; j < F::kVec / 2; ++j) s.add(w[j]);
    s.settle();
    if (++n == 64) {
      total += s.value(f.start);
      s.clear(f.start);
      n = 0;
    }
  }
  return warp_sum(total + s.value(f.start));
}
// The same in fp32.
template <int DT, int MODE, bool kUnit>
__device__ __forceinline__ float part_sum(Weights<DT, MODE, false, kUnit>& f, long long lo, long long hi, int lane) {
  using F = Fmt<DT>;
  float total = 0.f, err = 0.f;
#pragma unroll 2
  for (long long i = lo + lane * F::kVec; i < hi; i += 32 * F::kVec) {
    Term2 w[F::kVec / 2];
    f.at(i, hi, w);
#pragma unroll
    for (int j = 1; j < F::kVec / 2; ++j) w[0].a = __fadd2_rn(w[0].a, w[j].a);
    float lost;
    total = two_sum(total, w[0].a.x + w[0].a.y, lost);
    err += lost;
  }
  return warp_sum(total + err);
}

// Of the lanes' kPer sums each, in order: the one in which the running sum exceeds `want` and
// what is before it (past the last weight, a rounding: the last one that has any; -1: none has).
// `none`: what a sum of nothing stays below.  Whole warp.
template <class N, int kPer>
__device__ __forceinline__ int find_part(const N (&v)[kPer], N want, float none, N& before, int lane) {
  N own = v[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) own += v[j];
  N upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const N up = from_below(upto, o);
    if (lane >= o) upto += up;
  }
  N run = from_below(upto, 1);
  if (lane == 0) run = N(0.f);
  int at = -1, last = -1;
  N at_before = N(0.f), last_before = N(0.f);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (static_cast<float>(v[j]) > none) {
      last = lane * kPer + j;
      last_before = run;
      if (at < 0 && run + v[j] > want) {
        at = last;
        at_before = run;
      }
    }
    run += v[j];
  }
  const uint32_t hit = __ballot_sync(0xffffffffu, at >= 0), some = __ballot_sync(0xffffffffu, last >= 0);
  const int src = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : 0;
  before = from_lane(hit ? at_before : last_before, src);
  return __shfl_sync(0xffffffffu, hit ? at : last, src);
}

// The first token of [begin, end) at which the running sum exceeds `want`, by one CTA (sm.found; -1:
// no weight there); sm.gap: how far `want` is from the nearer end of its weight.
template <int DT, int MODE, bool kFine, class N, bool kUnit>
__device__ __forceinline__ void search(Weights<DT, MODE, kFine, kUnit>& f, long long begin, long long end, N want, Smem& sm) {
  using F = Fmt<DT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kStep = 32 * F::kVec;
  constexpr float none = kFine && MODE != kRest ? kNothing : 0.f;
  while (end - begin > 2 * kStep) {
    const long long size = part_size(end - begin, kWarps, kStep);
    const long long lo = min(end, begin + warp * size), hi = min(end, lo + size);
    const N s = part_sum(f, lo, hi, lane);
    N* sums;
    if constexpr (kFine)
      sums = sm.sums;
    else
      sums = sm.coarse;
    __syncthreads();
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    N v[1], before;
    v[0] = lane < kWarps ? sums[lane] : N(0.f);
    const int at = max(0, find_part(v, want, none, before, lane));
    want -= before;
    begin = min(end, begin + at * size);
    end = min(end, begin + size);
  }
  __syncthreads();
  if (warp == 0) {
    long long found = -1, last = -1;
    N near = N(0.f);
    for (long long base = begin; base < end && found < 0; base += kStep) {
      const long long i = base + lane * F::kVec;
      N x[F::kVec];
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) x[j] = N(0.f);
      if (i < end) f.exactly(i, end, x);
      N sum = N(0.f);
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) sum += x[j];
      N upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const N up = from_below(upto, o);
        if (lane >= o) upto += up;
      }
      N run = from_below(upto, 1);
      if (lane == 0) run = N(0.f);
      long long mine = -1, mine_last = -1;
      N mine_near = N(0.f);
#pragma unroll
      for (int j = 0; j < F::kVec; ++j) {
        if (static_cast<float>(x[j]) > 0.f) {
          mine_last = i + j;
          if (mine < 0 && run + x[j] > want) {
            mine = i + j;
            mine_near = smaller(want - run, run + x[j] - want);
          }
        }
        run += x[j];
      }
      const uint32_t who = __ballot_sync(0xffffffffu, mine >= 0);
      if (who) {
        found = __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
        near = from_lane(mine_near, __ffs(who) - 1);
      }
      const uint32_t some = __ballot_sync(0xffffffffu, mine_last >= 0);
      if (some) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(some));
      want -= from_lane(upto, 31);
    }
    if (lane == 0) {
      sm.found = found >= 0 ? found : last;
      sm.gap = found >= 0 ? static_cast<float>(near) : 0.f;
    }
  }
  __syncthreads();
}

// The CTA that has part `at` (of `size` elements) looks for the token there and tells the others.
// The answer is sure if the border is more than `unsure` away from the ends of the token's weight.
template <int DT, int MODE, bool kUnit>
__device__ __forceinline__ long long draw_coarse(Weights<DT, MODE, false, kUnit>& f, int at, float want, float unsure, long long V,
                                                 long long size, Group& g, Smem& sm, bool& sure) {
  Exchange& ex = sm.ex[g.turn ^ 1];
  if (at / kWarps == g.rank) {
    const long long lo = min(V, at * size), hi = min(V, lo + size);
    search<DT, MODE, false, float>(f, lo, hi, want, sm);
    if (threadIdx.x < 32) {
      tell(g, &ex.token, sm.found, threadIdx.x);
      tell(g, &ex.unsure, static_cast<int>(!(sm.gap > unsure)), threadIdx.x);
    }
  }
  g.turn ^= 1;
  g.sync();
  sure = !ex.unsure;
  return ex.token;
}

// The parts' fine sums, told to the whole cluster; then the token at u of their total.
template <int DT, int MODE, bool kUnit>
__device__ __forceinline__ void tell_sum(Weights<DT, MODE, true, kUnit>& f, long long lo, long long hi, Group& g, Smem& sm) {
  const int lane = threadIdx.x & 31, part = g.rank * kWarps + (threadIdx.x >> 5);
  const Wide s = part_sum(f, lo, hi, lane);
  g.turn ^= 1;
  tell(g, &sm.ex[g.turn].sum[part], s, lane);
  g.sync();
}
// The row's sum in fine arithmetic, in every thread of the cluster.  (Out of line, for one draft in 2^16 asks for it.  A draw
// that falls back, one in twenty, has the sum in line: 64 draws take 41 us, 44 with a call.)
template <int DT, bool kUnit>
__device__ __noinline__ double row_sum(const unsigned char* row, long long lo, long long hi, FineExp p, float c, Group& g, Smem& sm) {
  Weights<DT, kSoftmax, true, kUnit> f{row, nullptr, -1, c, 0.f, p, p, sm.powers, fine_start(sm.top[threadIdx.x >> 5], p, c)};
  tell_sum(f, lo, hi, g, sm);
  Wide total(0.f);
  for (int j = threadIdx.x & 31; j < g.size * kWarps; j += 32) total += sm.ex[g.turn].sum[j];
  total = warp_sum(total);
  return static_cast<double>(total.h) + static_cast<double>(total.l);
}

// The token, in the CTA that has it; kElsewhere in the others, which have nothing left to do;
// kNowhere in all where the parts' weights are `nothing`.
constexpr long long kElsewhere = -2, kNowhere = -3;
template <int DT, int MODE, bool kUnit>
__device__ __forceinline__ long long draw_fine(Weights<DT, MODE, true, kUnit>& f, const Wide* sums, long long V, long long size, const Group& g,
                                               Smem& sm, float nothing = kNothing) {
  const int lane = threadIdx.x & 31, parts = g.size * kWarps;
  constexpr float none = MODE != kRest ? kNothing : 0.f;
  Wide v[kMaxParts / 32], own(0.f), before;
#pragma unroll
  for (int j = 0; j < kMaxParts / 32; ++j) {
    const int i = lane * (kMaxParts / 32) + j;
    v[j] = i < parts ? sums[i] : Wide(0.f);
    own += v[j];
  }
  const Wide total = warp_sum(own), want = sm.u * total;
  const int at = total.h > nothing ? find_part(v, want, none, before, lane) : -1;  // the same in every CTA
  if (at < 0) return kNowhere;
  if (at / kWarps != g.rank) return kElsewhere;
  const long long lo = min(V, at * size), hi = min(V, lo + size);
  f.start = fine_start(sm.top[at % kWarps], f.p, f.c);
  search<DT, MODE, true, Wide>(f, lo, hi, want - before, sm);
  long long t = sm.found;
  if (MODE == kRest && t < 0) {  // p = q to the last digit kept in the whole part: its first token
    for (long long i = lo; i < hi && t < 0; i += 32) {
      const uint32_t some = __ballot_sync(0xffffffffu, i + lane < hi && !f.p.is_zero(Fmt<DT>::load(f.row, min(i + lane, hi - 1))));
      if (some) t = i + __ffs(some) - 1;
    }
  }
  return t;
}

template <int DT, bool kUnit>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
verify_drafts_kernel(const Args a, int cluster) {
  using F = Fmt<DT>;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Smem sm;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  Group g{cluster, cluster > 1 ? static_cast<int>(cluster_rank()) : 0, 0u};
  const long long b = blockIdx.x / cluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.G;
  const bool writes = g.rank == 0 && tid == 0;
  const long long V = a.V, rows = static_cast<long long>(G) + 1;
  long long* tokens = a.tokens + b * rows;
  float* logp = a.logp ? a.logp + b * rows : nullptr;
  float* lse = a.lse ? a.lse + b * rows : nullptr;
  const float nan = __int_as_float(0x7fc00000);
  static_assert(kPow == kThreads, "one power a thread");
  sm.powers[tid] = kPowers[tid];
  if (tid < kWarps * kSlots) mbar_init(smem_addr(&sm.full[0][0]) + 8 * tid, 1);
  if (tid == 0) abort_word = 0;
  grid_dependency_wait();  // the launch before this one may have ended only now
  if (tid == 0) {
    double u = a.u[b * rows + G];
    u = u > 0.0 ? fmin(u, 1.0 - 0x1p-53) : 0.0;
    const float h = static_cast<float>(u);
    sm.u = Wide(h, static_cast<float>(u - static_cast<double>(h)));
  }
  fence_mbar_init();
  long long id = 0;
  if (tid < G) id = a.ids[b * G + tid];
  const int n = a.n_draft ? a.n_draft[b] : G;
  const bool wrong = __syncthreads_or(n < -1 || n > G || (tid < n && (id < 0 || id >= V)));
  if (wrong || n < 0) {  // the same in every CTA of the cluster
    if (g.rank == 0) {
      for (int i = tid; i <= G; i += kThreads) {
        tokens[i] = -1;
        if (logp) logp[i] = wrong ? nan : 0.f;
        if (lse) lse[i] = wrong ? nan : 0.f;
      }
      if (tid == 0) {
        if (a.n_accepted) a.n_accepted[b] = 0;
        if (wrong && a.status) atomicOr(a.status, RL_DEVERR_ID_RANGE);
      }
    }
    return;
  }

  const int parts = cluster * kWarps, part = g.rank * kWarps + warp;
  const long long size = part_size(V, parts, 32 * F::kVec);
  const long long lo = min(V, part * size), hi = min(V, lo + size);

  Stream<DT> in;
  in.init(a.target + b * rows * a.row_bytes, a.row_bytes, n + 1, lo, hi, smem_addr(ring) + warp * kSlots * kChunkBytes,
          smem_addr(&sm.full[warp][0]), lane);
  if (cluster > 1) cluster_sync_all();  // every CTA runs before its shared memory is written
  FineExp fp;
  int kept = 0;
  // what thread 0 needs of a row's draft, on its way while the row is summed
  long long d = 0, d_next = id;
  Stats st, of_lane[kMaxParts / 32];  // of the row; of the parts that this lane looks after
  bool lost = false, bad = false, exact = false;
  const unsigned char* row = nullptr;
#pragma unroll 1
  for (int i = 0;; ++i) {
    row = a.target + (b * rows + i) * a.row_bytes;
    float zd = 0.f, zq = 0.f, lq = 0.f;
    double ui = 0.0;
    if (tid == 0 && i < n) {
      d = d_next;
      if (i + 1 < n) d_next = a.ids[b * G + i + 1];
      zd = F::load(row, d);
      ui = a.u[b * rows + i];
      if (a.draft) {
        zq = F::load(a.draft + (b * G + i) * a.draft_bytes, d);
        lq = a.draft_lse[b * G + i];
      }
    }
    Stats mine = part_stats<DT>(in, a.c, lane, abort_flag);
    exact = false;
#pragma unroll 1
    while (true) {
      g.turn ^= 1;
      tell(g, &sm.ex[g.turn].stats[part], mine, lane);
      if (lane == 0) sm.top[warp] = mine.m;
      g.sync();
      // maximum, then the parts' sums in its frame
      float m = -FLT_MAX;
#pragma unroll
      for (int j = 0; j < kMaxParts / 32; ++j) {
        const int k = lane * (kMaxParts / 32) + j;
        of_lane[j] = k < parts ? sm.ex[g.turn].stats[k] : Stats{-FLT_MAX, 0.f, 0.f};
        m = max_nan(m, of_lane[j].m);
      }
      asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(st.m) : "f"(m));
      st.n = st.s = 0.f;
#pragma unroll
      for (int j = 0; j < kMaxParts / 32; ++j) {
        const bool top = of_lane[j].m == st.m;
        st.n += top ? of_lane[j].n : 0.f;
        st.s += top ? of_lane[j].s : (of_lane[j].n + of_lane[j].s) * ex2_approx((of_lane[j].m - st.m) * a.c);
      }
      st.n = warp_sum(st.n);
      st.s = warp_sum(st.s);
      if (exact || !needs_exact<F>(st.m, a.c) || st.m != st.m) break;
      exact = true;
      mine = part_stats_exact<DT>(row, lo, hi, a.c, lane);
    }
    bad = !(fabsf(st.m) < INFINITY) || !(st.n > 0.f);
    fp.init(a.r_hi, a.r_lo, a.T, st.m, fabsf(st.m) * a.c > kFar);
    if (bad || i == n) {
      if (writes && lse) lse[i] = bad ? nan : static_cast<float>(static_cast<double>(st.m) * a.inv_t + log1pf((st.n - 1.f) + st.s));
      break;
    }
    if (tid == 0) {
      const Term w = fp.is_zero(zd) ? Term{0.f, 0.f, 0.f} : fp.template at<DT == RL_F32, false, kUnit>(zd, sm.powers);
      int v;
      if (a.draft && (!(zq < INFINITY) || !(fabsf(lq) < INFINITY))) {
        v = kNoDistribution;
      } else {
        // u q S < w, where fp32 decides it (an exponent of up to 128: 2^-17 of the value)
        const float x = a.draft ? fmaf(zq, a.c, -lq * kLog2e) : 0.f;
        const float left = static_cast<float>(ui) * ex2_approx(x) * (st.n + st.s);
        if (fabsf(x) < 128.f && fabsf(zq * a.c) < 1024.f && fabsf(left - w.a) > 0x1p-8f * w.a && w.a > 0x1p-100f) {
          v = left < w.a ? kStays : kRefused;
        } else if (w.a == 0.f || !(ui > 0.0)) {
          const double xq = a.draft ? static_cast<double>(zq) * a.inv_t - static_cast<double>(lq) : 0.0;
          v = stays_by_logs(ui, xq, static_cast<double>(st.n) + static_cast<double>(st.s),
                            (static_cast<double>(zd) - static_cast<double>(st.m)) * a.inv_t) ? kStays : kRefused;
        } else {
          const double qd = a.draft ? draft_prob<kUnit>(zq, lq, a, sm.powers) : 1.0;
          const Wide p = w.value();
          const double uq = ui * qd, right = static_cast<double>(p.h) + static_cast<double>(p.l);
          const double over = uq * (static_cast<double>(st.n) + static_cast<double>(st.s)) - right;
          v = over < 0.0 ? kStays : kRefused;
          if (fabs(over) <= kOpen * right) {
            v = kNear;
            sm.left = uq;
            sm.right = right;
          }
        }
      }
      sm.verdict = v;
    }
    __syncthreads();
    int v = sm.verdict;
    if (v == kNear) {  // the same in every CTA
      Group h = g;
      v = sm.left * row_sum<DT, kUnit>(row, lo, hi, fp, a.c, h, sm) < sm.right ? kStays : kRefused;
      g.turn = h.turn;
    }
    if (writes) {
      if (lse) lse[i] = static_cast<float>(static_cast<double>(st.m) * a.inv_t + log1pf((st.n - 1.f) + st.s));
      if (v == kStays) {
        tokens[i] = d;
        if (logp) logp[i] = log_prob(zd, st, a.inv_t);
      }
    }
    lost = v == kRefused;
    bad = v == kNoDistribution;
    if (lost || bad) break;
    kept = i + 1;
  }

  long long token = kNowhere;
  if (!bad) {
    const unsigned char* draft_row = a.draft ? a.draft + (b * G + kept) * a.draft_bytes : nullptr;
    if (lost && a.draft) {
      // S q_v = e^(z / T - lse_q + ln S)
      Weights<DT, kRest, true, kUnit> f{row, draft_row, -1, a.c, 0.f, fp, fp, sm.powers, fine_start(sm.top[warp], fp, a.c)};
      Wide total;
      total.h = two_sum(st.n, st.s, total.l);
      const float lq = a.draft_lse[b * G + kept];
      float close = 0.f;
      bool sure = false;
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        const Wide S = total;
        // (q's least term is above p's: a token that neither can give, -inf twice or behind the row, has no p - q)
        f.q.init_around(a.r_hi, a.r_lo, a.T, a.inv_t, lq, ln_wide(S, sm.powers), -84.f);
        if (sure) break;
        // sums of p over all tokens, of p - q and of q over those with p > q, and of q over those with p next to q
        Wide all(0.f), plus(0.f);
        FineSum fa, fb;
        fa.clear(f.start);
        fb.clear(f.start);
        float2 qs = both(0.f), ns = both(0.f);
        int count = 0;
#pragma unroll 1
        for (long long i = lo + lane * F::kVec; i < hi; i += 32 * F::kVec) {
          float z[F::kVec], y[F::kVec];
          fetch<DT>(row, i, hi);  // (512 sequences take 4% longer without)
          fetch<DT>(draft_row, i, hi);
          F::unpack(load_vec<DT>(row, i, hi), z);
          F::unpack(load_vec<DT>(draft_row, i, hi), y);
#pragma unroll
          for (int j = 0; j < F::kVec; j += 2) {
            bad = bad || !(y[j] < INFINITY) || !(y[j + 1] < INFINITY);
            const Term2 w = f.fine(make_float2(z[j], z[j + 1])), q = f.drafted(make_float2(y[j], y[j + 1]));
            float2 more, beside;
            fa.add(w);
            const Term2 r = above(w, q, more, kWindow, beside);
            fb.add(r, more);
            qs = __ffma2_rn(more, q.a, qs);
            ns = __ffma2_rn(beside, q.a, ns);
          }
          fa.settle();
          fb.settle();
          if (++count == 64) {
            all += fa.value(f.start);
            plus += fb.value(f.start);
            fa.clear(f.start);
            fb.clear(f.start);
            count = 0;
          }
        }
        all = warp_sum(all + fa.value(f.start));
        plus = warp_sum(plus + fb.value(f.start));
        const float drafted = warp_sum(qs.x + qs.y), next_to = warp_sum(ns.x + ns.y);
        bad = __any_sync(0xffffffffu, bad);
        g.turn ^= 1;
        Exchange& ex = sm.ex[g.turn];
        tell(g, &ex.sum[part], bad ? Wide(-1.f) : all, lane);
        tell(g, &ex.plus[part], plus, lane);
        tell(g, &ex.stats[part], Stats{next_to, 0.f, drafted}, lane);
        g.sync();
        total = Wide(0.f);
        close = 0.f;
        bad = false;
        for (int j = lane; j < parts; j += 32) {
          bad = bad || ex.sum[j].h < 0.f;
          total += ex.sum[j];
          close += ex.stats[j].m;
        }
        total = warp_sum(total);
        close = warp_sum(close);
        bad = __any_sync(0xffffffffu, bad);
        if (bad) break;
        // q's terms were taken with S, and belong to `total`.  Which tokens have p > q was asked with S too: those
        // that it decides otherwise have p / q within (total - S) / S of 1, and a weight below that much of q.  Where they may
        // have more than 2^-36 of the total together, all is done once more with the total for S.
        const float more = (total - S).h / S.h;
        sure = pass == 2 || (fabsf(more) < 0.5f * kWindow && fabsf(more) * close < 0x1p-36f * total.h);
        if (!sure) continue;
        __syncthreads();
        if (warp == 0) {
          for (int j = lane; j < parts; j += 32) {
            const Wide r = ex.plus[j] - Wide(more * ex.stats[j].s);
            ex.plus[j] = r.h > 0.f ? r : Wide(0.f);
          }
        }
        __syncthreads();
      }
      if (!bad) {  // (terms are good to 2^-39: of tokens with p next to q nothing below that is known to be left)
        token = draw_fine(f, sm.ex[g.turn].plus, V, size, g, sm, 0x1p-38f * close);
      }
    } else {
      // the parts' sums of step 1 in the frame of the row, without the draft that was looked up
      const bool without = lost;
      const long long d_out = without ? a.ids[b * G + kept] : -1;
      if (!exact) {
        const float nm = -st.m * a.c, back = ex2_approx(fmaf(st.m, a.c, nm));  // true terms to the search's
        float v[kMaxParts / 32], own = 0.f, before;
#pragma unroll
        for (int j = 0; j < kMaxParts / 32; ++j) {
          const long long k = lane * (kMaxParts / 32) + j;
          v[j] = (of_lane[j].n + of_lane[j].s) * ex2_approx((of_lane[j].m - st.m) * a.c) * back;
          if (without && d_out >= k * size && d_out < (k + 1) * size) v[j] = fmaxf(0.f, v[j] - ex2_approx(fmaf(F::load(row, d_out), a.c, nm)));
          own += v[j];
        }
        const float total = warp_sum(own), want = sm.u.h * total;
        const int at = max(0, find_part(v, want, 0.f, before, lane));
        bool sure;
        long long t;
        if (without) {
          Weights<DT, kWithout, false, kUnit> f{row, nullptr, d_out, a.c, nm, fp, fp, sm.powers, 1.f};
          t = draw_coarse(f, at, want - before, kCoarse * (st.n + st.s), V, size, g, sm, sure);
        } else {
          Weights<DT, kSoftmax, false, kUnit> f{row, nullptr, -1, a.c, nm, fp, fp, sm.powers, 1.f};
          t = draw_coarse(f, at, want - before, kCoarse * (st.n + st.s), V, size, g, sm, sure);
        }
        if (sure && t >= 0) token = g.rank == 0 ? t : kElsewhere;
      }
      if (token == kNowhere && without) {
        Weights<DT, kWithout, true, kUnit> f{row, nullptr, d_out, a.c, 0.f, fp, fp, sm.powers, fine_start(sm.top[warp], fp, a.c)};
        tell_sum(f, lo, hi, g, sm);
        token = draw_fine(f, sm.ex[g.turn].sum, V, size, g, sm);
      }
    }
    if (token == kNowhere && !bad) {
      Weights<DT, kSoftmax, true, kUnit> f{row, nullptr, -1, a.c, 0.f, fp, fp, sm.powers, fine_start(sm.top[warp], fp, a.c)};
      tell_sum(f, lo, hi, g, sm);
      token = draw_fine(f, sm.ex[g.turn].sum, V, size, g, sm);
    }
  }
  in.drain(abort_flag);
  if (*abort_flag && lane == 0 && a.status) atomicOr(a.status, RL_DEVERR_TIMEOUT);
  // One CTA writes: the one that found the token, or the first.  (Nobody writes another's shared
  // memory behind the last barrier, so all may leave as they are done.)
  if (token == kElsewhere || (token == kNowhere && g.rank != 0)) return;
  bad = bad || token < 0;
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

// CTAs of a cluster, no more than leave a warp 256 elements.  Few sequences take the largest
// clusters of which all are at work at once; 5 and 10 of them fill the chip's parts best (435 and 430 of 456
// places; 8: 408, 16: 336).  us, V = 151,936, four drafts / a draw (2% less than with settled fine sums):
//   B = 4    16: 30 / 16    10: 31 / 17    8: 37 / 19
//   B = 40   10: 53 / 28     8: 60 / 32    5: 64 / 36    4: 69 / 41
//   B = 64    8: 86 / 39     5: 77 / 39    4: 77 / 45    2: 102 / 64
//   B = 130   5: 123 / 52    4: 124 / 55   2: 133 / 70   1: 179 / 72
//   B = 300   5: 229 / 82    4: 221 / 81   2: 228 / 92   1: 236 / 87
//   B = 512   4: 346 / 117   2: 327 / 117  1: 365 / 124
// Of short rows a cluster's barriers are a larger share.  What counts is their number of elements, not of bytes:
//   V = 32,000 bf16            V = 50,257 bf16               V = 50,257 fp32               V = 66,000 bf16
//   4: 41 / 25   2: 46 / 31    4: 51 / 31    2: 64 / 40      4: 58 / 31    2: 70 / 40      4: 64 / 38    2: 76 / 45      B = 100
//   2: 56 / 34   1: 66 / 29    2: 75 / 44    1: 92 / 39      2: 84 / 48    1: 114 / 44     4: 106 / 47   2: 95 / 48      B = 200
//   2: 88 / 45   1: 83 / 33    2: 128 / 58   1: 119 / 43     2: 146 / 63   1: 141 / 51     2: 153 / 67   1: 150 / 56     B = 400
// (At 66,000 and 100,000 elements 200 sequences with four drafts would be 4 to 10% faster by 2 CTAs, and 400 draws by one.)
constexpr long long kShortRow = 1 << 16;
int cluster_for(long long B, long long V, int sms) {
  const long long slots = static_cast<long long>(sms) * kCtasPerSm, most = (V + 256 * kWarps - 1) / (256 * kWarps);
  const long long filled = slots - slots / 32;
  int c;
  if (B * kMaxCluster <= slots / 7)
    c = kMaxCluster;
  else if (B * 10 <= filled)
    c = 10;
  else if (B * 5 <= filled)
    c = 5;
  else if (B * 4 <= (V < kShortRow ? slots : 3 * slots))
    c = 4;
  else
    c = V < kShortRow && B >= 2 * sms ? 1 : 2;
  return static_cast<int>(c < most ? c : most);
}

template <int DT, bool kUnit>
rl_status launch_kernel(const Args& a, long long B, int cluster, int dev, cudaStream_t stream) {
  static std::atomic<unsigned long long> allowed{0};
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(verify_drafts_kernel<DT, kUnit>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(verify_drafts_kernel<DT, kUnit>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kSlots * kChunkBytes) !=
            cudaSuccess)
      return RL_ERR_CUDA;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWarps * kSlots * kChunkBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // starts while the launch before it ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<DT, kUnit>, a, cluster) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

template <int DT>
rl_status launch(const Args& a, long long B, int cluster, int dev, cudaStream_t stream) {
  return a.inv_t == 1.0 ? launch_kernel<DT, true>(a, B, cluster, dev, stream) : launch_kernel<DT, false>(a, B, cluster, dev, stream);
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
  const long long rows = d.B * (d.G + 1), drafts = d.B * d.G;
  if (rows > (1LL << 60) / (d.ld * es) || (d.draft_logits && drafts > 0 && drafts > (1LL << 60) / (d.ld_draft * es)))
    return RL_ERR_SHAPE;  // more than 64 bits address
  // what is written shares no byte with what is read, nor with what else is written
  struct Span {
    const void* p;
    long long bytes;
  };
  const Span out[4] = {{d.tokens, rows * 8}, {d.n_accepted, d.B * 8}, {d.logp_out, rows * 4}, {d.lse_out, rows * 4}};
  const Span in[6] = {{d.target_logits, ((rows - 1) * d.ld + d.V) * es},
                      {drafts > 0 ? d.draft_logits : nullptr, ((drafts - 1) * d.ld_draft + d.V) * es},
                      {drafts > 0 && d.draft_logits ? d.draft_lse : nullptr, drafts * 4},
                      {drafts > 0 ? d.draft_ids : nullptr, drafts * 8},
                      {d.n_draft, d.B * 4},
                      {d.uniforms, rows * 8}};
  const auto meet = [](const Span& x, const Span& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return a && b && a < b + static_cast<uintptr_t>(y.bytes) && b < a + static_cast<uintptr_t>(x.bytes);
  };
  for (int i = 0; i < 4; ++i) {
    for (const Span& s : in)
      if (meet(out[i], s)) return RL_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return RL_ERR_ALIAS;
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return RL_ERR_CUDA;
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
  a.c = static_cast<float>(kLog2eD / d.temperature);
  a.T = static_cast<float>(d.temperature);
  a.r_hi = static_cast<float>(a.inv_t);
  a.r_lo = static_cast<float>(a.inv_t - static_cast<double>(a.r_hi));
  a.tokens = d.tokens;
  a.n_accepted = d.n_accepted;
  a.logp = d.logp_out;
  a.lse = d.lse_out;
  a.status = d.status_dev;
  const int cluster = cluster_for(d.B, d.V, sms);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d.dtype == RL_F32) return launch<RL_F32>(a, d.B, cluster, dev, s);
  if (d.dtype == RL_BF16) return launch<RL_BF16>(a, d.B, cluster, dev, s);
  return launch<RL_F16>(a, d.B, cluster, dev, s);
}
