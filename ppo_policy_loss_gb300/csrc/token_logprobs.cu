// token_logprobs.cu — rl_token_logprobs and rl_token_logprobs_bwd: the
// log-probabilities of given tokens with entropy and top alternatives, and
// their gradient, over logits in memory (sm_103a).
#include <cmath>

#include "dealt_rows.h"
#include "lost_rows.h"
#include "token_rows.cuh"

namespace rl {
namespace {

constexpr int kMaxPieces = 8192;  // pieces of a row one CTA can search for alternatives
constexpr int kMaxK = RL_TOKEN_MAX_K;
constexpr int kList = 256;        // survivors a search ranks directly

// ------------------------------------------------------------------ top-k search
// The k largest of n unique keys (0 = none) by kT threads, sorted.
// Each thread takes the maxima of the even and the odd blocks of its keys; the
// k-th largest of nb >= 2 k bucket maxima is a bound that at least k keys
// reach and few others do; those that reach it are listed and ranked by
// counting.  If more than kList reach it (an order of the keys that puts the
// large ones on few threads), the bound is raised by bisection until exactly k
// do.
template <class K, int kT>
struct SelSmem {
  alignas(16) K a[2 * kT];
  alignas(16) K b[kList + 4];
  K bound;
  int count;
  int sums[2];
};

// kT: threads that work on a row.
template <int kT>
__device__ __forceinline__ void row_barrier() {
  named_barrier(1, kT);
}

// Keys of list[0 .. n-1] above `key`; n up to a multiple of 16 bytes is read,
// the places past n hold 0.
__device__ __forceinline__ int rank_of(const uint32_t* list, int n, uint32_t key) {
  int r = 0;
#pragma unroll 4
  for (int j = 0; j < n; j += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(list + j);
    r += (v.x > key) + (v.y > key) + (v.z > key) + (v.w > key);
  }
  return r;
}
__device__ __forceinline__ int rank_of(const unsigned long long* list, int n, unsigned long long key) {
  int r = 0;
#pragma unroll 4
  for (int j = 0; j < n; j += 2) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(list + j);
    r += (v.x > key) + (v.y > key);
  }
  return r;
}

// f(key) for this thread's keys get(tid), get(tid + kT), ... below n,
// eight loads at a time; f also gets the block's parity.
template <class K, int kT, class Get, class Fn>
__device__ __forceinline__ void each_key(Get get, int n, int tid, Fn f) {
  for (int base = tid; base < n; base += 8 * kT) {
    K v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = base + j * kT < n ? get(base + j * kT) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) f(v[j], j & 1);
  }
}

// get(i): key i, i < n.  out[0 .. k-1]: the largest first, 0 where there are
// fewer.  All kT threads, after a barrier; ends with a barrier.
template <class K, int kT, class Get>
__device__ __forceinline__ void block_select(Get get, int n, int k, K* out, SelSmem<K, kT>& s, int tid) {
  K best[2] = {0, 0};
  each_key<K, kT>(get, n, tid, [&](K v, int odd) { best[odd] = v > best[odd] ? v : best[odd]; });
  const int nb = k <= 16 ? 32 : k <= 32 ? 64 : k <= 64 ? 128 : 256;
  const K most = best[0] > best[1] ? best[0] : best[1];
  if (nb == 2 * kT) {
    s.a[2 * tid] = best[0];
    s.a[2 * tid + 1] = best[1];
  } else {
    const int per = kT / nb;  // neighbouring lanes that share a bucket
    K top = most;
    for (int o = 1; o < per; o <<= 1) {
      const K v = __shfl_xor_sync(0xffffffffu, top, o);
      top = v > top ? v : top;
    }
    if (tid % per == 0) s.a[tid / per] = top;
  }
  if (tid == 0) {
    s.bound = 1;
    s.count = 0;
    s.sums[0] = s.sums[1] = 0;
  }
  if (tid < k) out[tid] = 0;
  row_barrier<kT>();
  for (int q = tid; q < nb; q += kT) {
    const K v = s.a[q];
    if (v != 0 && rank_of(s.a, nb, v) == k - 1) s.bound = v;
  }
  row_barrier<kT>();
  const K bound = s.bound;
  if (most >= bound)
    each_key<K, kT>(get, n, tid, [&](K v, int) {
      if (v >= bound) {
        const int p = atomicAdd(&s.count, 1);
        if (p < kList) s.b[p] = v;
      }
    });
  row_barrier<kT>();
  int cnt = s.count;
  if (cnt > kList) {
    // bisection over the key's bits: the largest bound that k keys still reach
    K lo = bound, hi = ~static_cast<K>(0);
    for (int round = 0; lo < hi; ++round) {
      const K mid = lo + (hi - lo) / 2 + 1;
      int c = 0;
      if (most >= mid) each_key<K, kT>(get, n, tid, [&](K v, int) { c += v >= mid; });
      c = __reduce_add_sync(0xffffffffu, c);
      if ((tid & 31) == 0 && c) atomicAdd(&s.sums[round & 1], c);
      row_barrier<kT>();
      const int total = s.sums[round & 1];
      if (tid == 0) s.sums[(round + 1) & 1] = 0;
      row_barrier<kT>();
      if (total >= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    if (tid == 0) s.count = 0;
    row_barrier<kT>();
    each_key<K, kT>(get, n, tid, [&](K v, int) {
      if (v >= lo) s.b[atomicAdd(&s.count, 1)] = v;  // keys are unique: exactly k reach it
    });
    row_barrier<kT>();
    cnt = s.count;
  }
  if (tid < 4) s.b[cnt + tid] = 0;  // what rank_of reads past the list
  row_barrier<kT>();
  for (int q = tid; q < cnt; q += kT) {
    const K v = s.b[q];
    const int r = rank_of(s.b, cnt, v);
    if (r < k) out[r] = v;
  }
  row_barrier<kT>();
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
  int resident;  // CTAs the GPU holds at once
};

// The search key of a piece or an element: its value's order above its place,
// so that the lower place wins a tie.  32 bits for 16-bit formats, 64 for fp32.
template <class V>
struct PlaceKey;
template <>
struct PlaceKey<uint16_t> {
  using K = uint32_t;
  __device__ static K make(uint16_t v, int at) { return v ? (static_cast<K>(v) << 16) | (0xffffu - at) : 0u; }
  __device__ static int at(K k) { return static_cast<int>(0xffffu - (k & 0xffffu)); }
  __device__ static uint32_t value(K k) { return k >> 16; }
};
template <>
struct PlaceKey<uint32_t> {
  using K = unsigned long long;
  __device__ static K make(uint32_t v, int at) {
    return v ? (static_cast<K>(v) << 32) | (0xffffffffu - static_cast<uint32_t>(at)) : 0ull;
  }
  __device__ static int at(K k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }
  __device__ static uint32_t value(K k) { return static_cast<uint32_t>(k >> 32); }
};
// Across CTAs: the value's order above the element's place in the row.
using ElemKey = unsigned long long;

constexpr int kMaxCluster = 8;
constexpr int kSlots = 4;
// CTAs a SM holds, for kT threads: what their registers have to allow.  Shared
// memory lets in five of 128 threads without alternatives; with them four (151,936
// 16-bit or 50,257 fp32 logits) down to two (151,936 fp32).  Against a bound of
// six, which takes them to 64 registers and spills: 4096 x 151,936 bf16, us, k = 0
// and 64: 209.5, 217.7 and 256.7, 258.7; 8192 rows at k = 64: 479, 477.
template <int kT>
constexpr int kLpCtas = kT == 128 ? 5 : 8;
constexpr int kSmemPerSm = 228 * 1024;

template <int DT, int kT>
struct LpSmem {
  using F = Fmt<DT>;
  using C = PlaceKey<typename F::Key>;
  Ring<kSlots, kT * kPieceBytes> ring;  // a chunk has one piece per consumer thread
  long long row_of[kSlots];  // the row a chunk belongs to
  union {  // one search at a time
    SelSmem<typename C::K, kT> sel;
    SelSmem<ElemKey, kT> join_sel;
  };
  int pieces[kList];             // fast search: pieces that reach its bound
  int n_pieces, n_elems;
  alignas(16) typename C::K top[kMaxK];
  alignas(16) int slots[kMaxK];  // slow search: the k pieces with the largest maxima, in the row's order
  alignas(16) ElemKey found[kMaxK];  // the CTA's k largest elements, largest first, 0 where there are fewer
  RowStats part[kT / 32];
  RowStats join_part[kMaxCluster];  // clusters: every slice's statistics, in rank 0's memory
  alignas(16) uint4 dealt;            // the answer to the producer's request for another row
  unsigned long long deal;            // it has come
  unsigned long long arrived, freed;  // rank 0: every slice is in; the others: rank 0 has taken the row
  int abort;
};

// After it, as much as the launch needs: with clusters and alternatives, what
// every CTA of the row found (in rank 0's memory) and the row's choice of it;
// then the keys: piece maxima, then the chosen pieces' elements.
constexpr int kJoinKeys = (kMaxCluster + 1) * kMaxK;
constexpr int kAllElems = 4096;  // slices of at most this many elements search them without choosing pieces
template <class F>
__host__ __device__ constexpr bool takes_all(int per, int k) {
  return per <= k || per * F::kPiece <= kAllElems;
}
template <class F>
__host__ __device__ constexpr int key_places(int per, int k) {
  const int elems = (takes_all<F>(per, k) ? per : k) * F::kPiece;
  return k == 0 ? 0 : per > elems ? per : elems;
}

__device__ __forceinline__ ElemKey elem_key(uint32_t order, int e) {
  return (static_cast<ElemKey>(order) << 32) | (0xffffffffu - static_cast<uint32_t>(e));
}

// Asks the hardware for the number of a CTA that has not been started, which
// this CTA then does the work of; the answer arrives at `deal`.  One thread.
__device__ __forceinline__ void ask_for_cta(uint32_t answer, uint32_t deal) {
  fence_proxy_async_shared();
  mbar_arrive_expect_tx(deal, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
      "r"(deal)
      : "memory");
}
// The answer: a CTA's number, or -1 when all have been started (ask no more).
__device__ __forceinline__ long long cta_dealt(uint32_t answer) {
  uint32_t given, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\tmov.u32 %1, 0;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(given), "=r"(x)
      : "r"(answer)
      : "memory");
  return given ? static_cast<long long>(x) : -1;
}

// How many of the threads' two maxima reach `bound` (all consumer threads).
template <int kT>
__device__ __forceinline__ int count_reaching(const uint32_t (&best)[2], uint32_t bound, bool both) {
  int n;
  const uint32_t top = best[0] > best[1] ? best[0] : best[1];
  const uint32_t first = both ? best[0] : top;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ge.u32 p, %1, %2;\n\tbar.red.popc.u32 %0, 1, %3, p;\n\t}"
      : "=r"(n)
      : "r"(first), "r"(bound), "n"(kT)
      : "memory");
  if (both) {
    int n1;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ge.u32 p, %1, %2;\n\tbar.red.popc.u32 %0, 1, %3, p;\n\t}"
        : "=r"(n1)
        : "r"(best[1]), "r"(bound), "n"(kT)
        : "memory");
    n += n1;
  }
  return n;
}

// The k largest elements of the CTA's pieces into sm.found.  `best`: the
// largest piece orders this thread met in its even and odd steps.  A bound
// that at least k of these maxima reach, and not many more, is found from the
// row's maximum downwards in widening steps; at least k elements reach it
// then, nearly all of them in pieces of their own, so the pieces that reach
// it are listed, their elements read again (from L2), and those that reach it
// ranked by counting.  False if a list overflows, or would (many
// equal values, or a large k of few pieces): search_slow then.
template <int DT, int kT>
__device__ __noinline__ bool search_fast(LpSmem<DT, kT>& sm, const typename Fmt<DT>::Key* keys, const unsigned char* src,
                                            int g0, int n_mine, int V, int k, const uint32_t (&best)[2], uint32_t top,
                                            int tid) {
  using F = Fmt<DT>;
  const bool both = k > kT / 4;
  const int enough = k + k / 8 + 4;
  if (tid == 0) sm.n_pieces = sm.n_elems = 0;  // the counts below are the barrier before the lists' first entries
  if (tid < k) sm.found[tid] = 0;
  // no more pieces than alternatives: no bound between them, every element
  // would be listed (32,768 x 1000, k = 32: 400 us with the attempt, 298 without)
  if (n_mine <= k && n_mine * F::kPiece > kList) return false;
  uint32_t hi = top + 1, lo = 1;  // fewer than k reach hi, unless NaN does
  int n = 0;
  for (uint32_t step = F::kOrderStep;; step *= 4) {
    const uint32_t mid = hi > step && step < 0x40000000u ? hi - step : 1u;
    n = count_reaching<kT>(best, mid, both);
    if (n >= k || mid == 1u) {
      lo = mid;
      break;
    }
    hi = mid;
  }
  while (n > enough && hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int m = count_reaching<kT>(best, mid, both);
    if (m >= k) {
      lo = mid;
      n = m;
    } else {
      hi = mid;
    }
  }
  // a vector of keys, or of a piece's elements, a lane at a time; hits are few
  const float thr = F::order_value(lo);  // of lo = 1 a NaN: everything passes
  const uint4* kv = reinterpret_cast<const uint4*>(keys);
  for (int q = tid; q * F::kVec < n_mine; q += kT) {
    uint32_t hits = F::hits(kv[q], thr);
    while (hits) {
      const int p = q * F::kVec + F::hit_elem(__ffs(hits) - 1);
      hits &= hits - 1;
      if (p < n_mine) {
        const int at = atomicAdd(&sm.n_pieces, 1);
        if (at < kList) sm.pieces[at] = g0 + p;
      }
    }
  }
  row_barrier<kT>();
  const int n_pieces = sm.n_pieces;
  if (n_pieces > kList) return false;
  const long long row_vecs = (static_cast<long long>(V) * F::kBytes + 15) / 16;
  for (int q0 = tid; q0 < n_pieces * 4; q0 += 4 * kT) {
    uint4 v[4];
    int e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = q0 + j * kT;
      const int vec = sm.pieces[min(q >> 2, n_pieces - 1)] * 4 + (q & 3);
      e[j] = q < n_pieces * 4 ? vec * F::kVec : V;
      v[j] = *reinterpret_cast<const uint4*>(src + min(static_cast<long long>(vec), row_vecs - 1) * 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t hits = e[j] < V ? F::hits(v[j], thr) : 0u;
      while (hits) {
        const int i = F::hit_elem(__ffs(hits) - 1);
        hits &= hits - 1;
        if (e[j] + i < V) {
          const int at = atomicAdd(&sm.n_elems, 1);
          if (at < kList) sm.join_sel.b[at] = elem_key(F::raw_order(static_cast<typename F::Raw>(F::pick(v[j], i))), e[j] + i);
        }
      }
    }
  }
  row_barrier<kT>();
  const int n_elems = sm.n_elems;
  if (n_elems > kList) return false;
  if (tid < 2) sm.join_sel.b[n_elems + tid] = 0;  // what rank_of reads past the list
  row_barrier<kT>();
  for (int q = tid; q < n_elems; q += kT) {
    const ElemKey key = sm.join_sel.b[q];
    const int r = rank_of(sm.join_sel.b, n_elems, key);
    if (r < k) sm.found[r] = key;
  }
  row_barrier<kT>();
  return true;
}

// The same by two exact searches: the k pieces with the largest maxima (the
// lower piece first among equals) hold the k largest elements.
template <int DT, int kT>
__device__ __noinline__ void search_slow(LpSmem<DT, kT>& sm, typename Fmt<DT>::Key* keys, const unsigned char* src, int g0,
                                         int n_mine, int V, int per, int k, int tid) {
  using F = Fmt<DT>;
  using C = PlaceKey<typename F::Key>;
  int n_slots = n_mine;
  const bool all = takes_all<F>(per, k);
  auto element = [&](int i) {  // the row's element at place i of the key array
    return (g0 + (all ? i / F::kPiece : sm.slots[i / F::kPiece])) * F::kPiece + i % F::kPiece;
  };
  auto key_at = [&](int i) { return C::make(keys[i], i); };
  row_barrier<kT>();
  for (int i = tid; i < n_mine; i += kT) keys[i] = static_cast<typename F::Key>(F::raw_order(keys[i]));
  row_barrier<kT>();
  if (!all) {
    block_select<typename C::K, kT>(key_at, n_mine, k, sm.top, sm.sel, tid);
    n_slots = min(k, n_mine);
    if (tid < n_slots) {  // back into the row's order
      const int g = C::at(sm.top[tid]);
      int r = 0;
      for (int j = 0; j < n_slots; ++j) r += C::at(sm.top[j]) < g;
      sm.slots[r] = g;
    }
    row_barrier<kT>();
  }
  const int n_elems = n_slots * F::kPiece;
  for (int i = tid; i < n_elems; i += kT) {
    const int e = element(i);
    keys[i] = e < V ? static_cast<typename F::Key>(F::load_order(src, e)) : typename F::Key(0);
  }
  row_barrier<kT>();
  block_select<typename C::K, kT>(key_at, n_elems, k, sm.top, sm.sel, tid);
  if (tid < k) {
    const typename C::K key = sm.top[tid];
    sm.found[tid] = key ? elem_key(C::value(key), element(C::at(key))) : 0;
  }
  row_barrier<kT>();
}

// The row's statistics where an -inf has made t NaN: the warps that met one take
// their pieces once more, from memory and with every word clamped.  The pieces,
// lanes, order and steps are the stream's, so a warp gets the bits that it would
// have got by clamping while the row streamed, and a row's results are the same
// whether an earlier row had made the CTA clamp or not.  All consumer threads.
template <int DT, int kT>
__device__ __noinline__ RowStats clamped_row(RowStats* part, const unsigned char* src, int V, int g0, int n_mine, int n_full,
                                             float c, int tid) {
  using F = Fmt<DT>;
  const int lane = tid & 31, row_vecs = (V + F::kVec - 1) / F::kVec;
  row_barrier<kT>();
  if (part[tid >> 5].t != part[tid >> 5].t) {
    WarpStats st;
    warp_stats_init<F>(st, c);
    st.low = true;
#pragma unroll 1
    for (int i = 0; i * kT < n_mine; ++i) {
      const int at = i * kT + tid;
      const bool last = i >= n_full;
      const int sh = last ? 0 : lane >> 1;
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int vec = (g0 + at) * 4 + ((j + sh) & 3);
        const uint4 v = at < n_mine && vec < row_vecs ? *reinterpret_cast<const uint4*>(src + static_cast<long long>(vec) * 16)
                                                      : make_uint4(0u, 0u, 0u, 0u);
        w[4 * j] = v.x;
        w[4 * j + 1] = v.y;
        w[4 * j + 2] = v.z;
        w[4 * j + 3] = v.w;
      }
      if (last) F::cut(w, 0, at < n_mine ? min(F::kPiece, V - (g0 + at) * F::kPiece) : 0);
      const float pm = max_nan(F::raw_value(F::raw_max(w, 0)), F::kFloor);
      if (last) {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = F::clamp(w[j]);
      }
      add_piece<F, true>(st, w, pm, c, lane, false);
    }
    const RowStats ws = warp_stats_sum<F>(st, c);
    if (lane == 0) part[tid >> 5] = ws;
  }
  row_barrier<kT>();
  RowStats rs = part[0];
#pragma unroll
  for (int w = 1; w < kT / 32; ++w) rs = merge_row(rs, part[w], c);
  return rs;
}

// The statistics of a row that needs_exact names, by differences to its
// maximum, -inf elements skipped.  Rare, so it reads the row again.  The maxima
// are counted, not summed, and one of them stays out, so that r is a sum of
// small terms here too.  m = -inf: no element is finite.  All consumer threads.
template <class F, int kT>
__device__ __noinline__ RowStats exact_row(const unsigned char* row, int V, float c, RowStats* part, int tid) {
  const int n_vecs = (V + F::kVec - 1) / F::kVec;
  auto each = [&](auto f) {
#pragma unroll 4
    for (int v = tid; v < n_vecs; v += kT) {
      float z[F::kVec];
      F::unpack(*reinterpret_cast<const uint4*>(row + static_cast<long long>(v) * 16), z);
#pragma unroll
      for (int i = 0; i < F::kVec; ++i)
        if (v * F::kVec + i < V) f(z[i]);
    }
  };
  float m = -INFINITY;
  each([&](float z) { m = max_nan(m, z); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  row_barrier<kT>();
  if ((tid & 31) == 0) part[tid >> 5].m = m;
  row_barrier<kT>();
  for (int w = 0; w < kT / 32; ++w) m = max_nan(m, part[w].m);
  row_barrier<kT>();
  float s = 0.f, t = 0.f;
  int top = 0;
  if (m > -INFINITY)
    each([&](float z) {
      const float x = (z - m) * c;
      const float e = ex2_approx(x);
      top += z == m;
      s += z == m ? 0.f : e;
      if (e > 0.f) t = fmaf(e, x, t);
    });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  top = __reduce_add_sync(0xffffffffu, top);
  if ((tid & 31) == 0) part[tid >> 5] = RowStats{static_cast<float>(top), s, t};  // exact: at most 2^24 in a warp's share
  row_barrier<kT>();
  s = t = 0.f;
  float others = -1.f;
  for (int w = 0; w < kT / 32; ++w) {
    others += part[w].m;
    s += part[w].r;
    t += part[w].t;
  }
  s += others;
  if (!(m < INFINITY)) s = t = __int_as_float(0x7fc00000);  // NaN, +inf
  return RowStats{m, s, t};
}

// A CTA (or, for few rows, a cluster of up to 8, each with a slice of the
// row's pieces) takes a row at a time.  The producer warp streams the valid
// rows' chunks through the ring; the consumers keep one key per piece (its
// maximum) and the running statistics, then search the keys for the
// alternatives while the producer fills the ring with the next row.  One pass
// over the logits; nothing else of their size is read or written.
//
// What bounds it: with the entropy, the instructions around the exponentials
// (an element's unpacking, two packed FMAs and a packed add a pair): the issue
// slots are 65-70% busy and the rest is their latency.  4096 x 151,936 bf16:
// 205 us (6.1 TB/s), without the entropy 184 us (6.8 TB/s).  The search waits on
// barriers and on L2: 16 alternatives add 35 us there, 64 add 50 us, and 16 add
// 50 us to 210 us at 16,384 x 32,000; many small CTAs cover that for one
// another.  One warp that searched a row behind the consumers took 234 us there,
// but 440 us against 331 at 16,384 x 32,000 and k = 64, and 27 us against 19 for
// a single row.
template <int DT, bool kEntropy, int kT>
__global__ void __launch_bounds__(kT + 32, kLpCtas<kT>) token_logprobs_kernel(const LpArgs a) {
  using F = Fmt<DT>;
  using C = PlaceKey<typename F::Key>;
  constexpr int kWarps = kT / 32, kChunk = kT * kPieceBytes;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  LpSmem<DT, kT>& sm = *reinterpret_cast<LpSmem<DT, kT>*>(smem_raw);
  volatile int* abort = &sm.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  static_assert(sizeof(LpSmem<DT, kT>) % 16 == 0, "the key arrays follow");
  const int csize = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const long long first = blockIdx.x / csize, stride = gridDim.x / csize;
  const bool dealt = kT == 128 && csize == 1 && gridDim.x > static_cast<unsigned>(a.resident);
  const int V = static_cast<int>(a.V);
  const int n_pieces = (V + F::kPiece - 1) / F::kPiece;
  const int per = (n_pieces + csize - 1) / csize;
  const int g0 = min(n_pieces, rank * per), g1 = min(n_pieces, g0 + per);  // this CTA's pieces
  const long long row_bytes16 = (static_cast<long long>(V) * F::kBytes + 15) & ~15LL;
  const long long b0 = static_cast<long long>(g0) * kPieceBytes;
  const long long n_bytes = min(row_bytes16, static_cast<long long>(g1) * kPieceBytes) - b0;
  const int n_chunks = static_cast<int>((n_bytes + kChunk - 1) / kChunk);
  ElemKey* const join_keys = reinterpret_cast<ElemKey*>(smem_raw + sizeof(LpSmem<DT, kT>));
  ElemKey* const join_top = join_keys + kMaxCluster * kMaxK;
  typename F::Key* const keys = reinterpret_cast<typename F::Key*>(csize > 1 && a.k ? join_keys + kJoinKeys : join_keys);

  if (tid == 0) {
    sm.ring.init(kWarps);
    mbar_init(smem_addr(&sm.deal), 1);
    mbar_init(smem_addr(&sm.arrived), csize);
    mbar_init(smem_addr(&sm.freed), 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (csize > 1) cluster_sync_all();

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    // The row of a chunk goes with it; a chunk of no bytes and row -1 is the end.
    const uint64_t pol = policy_normal();
    uint32_t it = 0;
    bool ok = true;
    RowsOf<true> rows(a.mask, a.R, first, lane);
    // a row a CTA of the grid: the next one is asked for while a row streams
    uint32_t asked = 0;
    auto ask = [&]() {
      if (lane == 0) ask_for_cta(smem_addr(&sm.dealt), smem_addr(&sm.deal));
      ++asked;
    };
    auto answer = [&]() {  // -1: no more; then nothing is asked again
      long long n = -1;
      if (lane == 0) {
        ok = wait_bounded<false>(smem_addr(&sm.deal), (asked - 1) & 1, abort) && ok;
        if (ok) n = cta_dealt(smem_addr(&sm.dealt));
      }
      return __shfl_sync(0xffffffffu, n, 0);
    };
    auto masked_row = [&](long long row) {
      if (!a.mask || row >= a.R || a.mask[row]) return;
      for (int q = lane; q < a.n_ids; q += 32) a.logp[row * a.n_ids + q] = 0.f;
      for (int q = lane; q < a.k; q += 32) {
        a.topk_ids[row * a.k + q] = -1;
        a.topk_logp[row * a.k + q] = 0.f;
      }
      if (lane == 0 && a.entropy) a.entropy[row] = 0.f;
      if (lane == 0 && a.lse) a.lse[row] = 0.f;
    };
    auto stream = [&](long long row) {  // its chunks; of row -1 the end's
      if (lane == 0) {
        const unsigned char* src = a.logits + row * a.row_bytes + b0;
        const int n = row < 0 ? 1 : n_chunks;
        for (int q = 0; q < n && ok; ++q) {
          const long long off = static_cast<long long>(q) * kChunk;
          const uint32_t slot = it % kSlots;
          ok = sm.ring.reserve(it, abort);
          if (!ok) break;
          sm.row_of[slot] = row;
          if (row < 0)
            mbar_arrive(smem_addr(&sm.ring.full[slot]));
          else
            sm.ring.fill(it, src + off, static_cast<uint32_t>(min(static_cast<long long>(kChunk), n_bytes - off)), pol);
          ++it;
        }
        if (!ok) sm.ring.drain(it);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      return ok;
    };
    take_rows(first, stride, dealt, ask, answer, [&](long long n) { return rows.at(n, lane); }, stream, masked_row);
    if (!ok && asked && lane == 0) {  // an answer on its way lands before the CTA may exit
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(smem_addr(&sm.deal), (asked - 1) & 1) && global_ns() - t0 <= kWaitLimitNs) {
      }
    }
  } else {
    // ---------------------------------------------------------------- consumers
    const int k = a.k, n_ids = a.n_ids, n_mine = g1 - g0;
    const int n_full = min(n_mine, V / F::kPiece - g0) / kT;  // steps whose every piece is a full one
    if (a.mask && rank == 0 && !dealt) {  // masked rows
      for (long long row = first + tid * stride; row < a.R; row += kT * stride) {
        if (a.mask[row]) continue;
        for (int q = 0; q < n_ids; ++q) a.logp[row * n_ids + q] = 0.f;
        for (int q = 0; q < k; ++q) {
          a.topk_ids[row * k + q] = -1;
          a.topk_logp[row * k + q] = 0.f;
        }
        if (a.entropy) a.entropy[row] = 0.f;
        if (a.lse) a.lse[row] = 0.f;
      }
    }
    unsigned int err = 0;
    uint32_t it = 0;  // chunks taken
    WarpStats st;
    st.low = false;
    for (uint32_t done = 0;; ++done) {  // rows done
      // the row's first chunk brings its number; the barrier also frees the
      // shared arrays of the row before.  After a timeout every thread stops here.
      sm.ring.wait(it, abort);
      const long long row = sm.row_of[it % kSlots];
      if (named_barrier_or(1, kT, row < 0 || *abort)) break;
      const unsigned char* src = a.logits + row * a.row_bytes;
      const long long y = rank == 0 && tid < n_ids ? a.ids[row * n_ids + tid] : -1;
      const bool y_ok = y >= 0 && y < V;
      float zy = 0.f;
      float best[2] = {-INFINITY, -INFINITY};
      warp_stats_init<F>(st, a.c);
      for (int i = 0; i < n_chunks; ++i, ++it) {
        const uint32_t buf = sm.ring.wait(it, abort);
        const int at = i * kT + tid;  // this lane's piece in the slice
        const bool last = i >= n_full;         // a step that reaches the slice's or the row's end
        uint32_t w[16];
        load_piece(w, 0, buf + tid * kPieceBytes, last ? 0 : lane >> 1);
        sm.ring.release(it, lane);
        if (last) F::cut(w, 0, at < n_mine ? min(F::kPiece, V - (g0 + at) * F::kPiece) : 0);
        const uint32_t rm = F::raw_max(w, 0);
        if (k && at < n_mine) {
          keys[at] = static_cast<typename F::Key>(rm);
          const float v = max_nan(i & 1 ? best[1] : best[0], F::raw_value(rm));
          best[0] = i & 1 ? best[0] : v;
          best[1] = i & 1 ? v : best[1];
        }
        if (i == 1 && y_ok) zy = F::load(src, y);  // its id has arrived by now
        if (last) {
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = F::clamp(w[j]);
        }
        add_piece<F, kEntropy>(st, w, max_nan(F::raw_value(rm), F::kFloor), a.c, lane, done == 0);
      }
      if (n_chunks < 2 && y_ok) zy = F::load(src, y);
      const RowStats ws = warp_stats_sum<F>(st, a.c);
      if (lane == 0) sm.part[warp] = ws;
      row_barrier<kT>();
      RowStats rs = sm.part[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) rs = merge_row(rs, sm.part[w], a.c);
      if (k) {
        const uint32_t order[2] = {tid < n_mine ? F::order_of(best[0]) : 0u,
                                   tid + kT < n_mine ? F::order_of(best[1]) : 0u};
        if (!search_fast<DT, kT>(sm, keys, src, g0, n_mine, V, k, order, F::order_of(rs.m), tid))
          search_slow<DT, kT>(sm, keys, src, g0, n_mine, V, per, k, tid);
      }
      if (kEntropy && rs.t != rs.t) {  // a first -inf, or NaN: clamp from now on, and this row again
        st.low = true;
        rs = clamped_row<DT, kT>(sm.part, src, V, g0, n_mine, n_full, a.c, tid);
      }
      if (csize > 1) {
        // every CTA's findings into rank 0's memory
        if (done > 0 && rank != 0) wait_bounded<true>(smem_addr(&sm.freed), (done - 1) & 1, abort);
        if (tid < k) st_cluster_u64(map_to_rank(smem_addr(&join_keys[rank * k + tid]), 0), sm.found[tid]);
        if (tid == 0) {
          const uint32_t to = map_to_rank(smem_addr(&sm.join_part[rank]), 0);
          st_cluster_f32(to, rs.m);
          st_cluster_f32(to + 4, rs.r);
          st_cluster_f32(to + 8, rs.t);
        }
        fence_cluster();
        row_barrier<kT>();
        if (tid == 0) mbar_arrive_remote(map_to_rank(smem_addr(&sm.arrived), 0));
        if (rank == 0) {
          wait_bounded<true>(smem_addr(&sm.arrived), done & 1, abort);
          rs = sm.join_part[0];
          for (int q = 1; q < csize; ++q) rs = merge_row(rs, sm.join_part[q], a.c);
          const int n = csize * k;
          if (n > kList) {
            block_select<ElemKey, kT>([&](int i) { return join_keys[i]; }, n, k, join_top, sm.join_sel, tid);
          } else {
            for (int q = tid; q < n; q += kT) {
              const ElemKey key = join_keys[q];
              const int r = rank_of(join_keys, n, key);
              if (key && r < k) join_top[r] = key;
            }
          }
          row_barrier<kT>();  // everything has been read: the others may send the next row
          if (tid > 0 && tid < csize) mbar_arrive_remote(map_to_rank(smem_addr(&sm.freed), tid));
        }
        if (rank != 0) continue;
      }
      if (needs_exact<F>(rs.m, a.c)) rs = exact_row<F, kT>(src, V, a.c, sm.part, tid);
      const float log_s = log1pf(rs.r);
      if (tid < n_ids) {
        if (!y_ok) err |= RL_DEVERR_ID_RANGE;
        a.logp[row * n_ids + tid] = y_ok ? fmaf(zy - rs.m, a.inv_temp, -log_s) : __int_as_float(0x7fc00000);
      }
      if (tid == 0) {
        if (a.lse) a.lse[row] = fmaf(rs.m, a.inv_temp, log_s);
        if (kEntropy && a.entropy)
          a.entropy[row] = rs.m > -INFINITY ? fmaf(-kLn2, rs.t / (1.f + rs.r), log_s) : __int_as_float(0x7fc00000);
      }
      if (tid < k) {
        const ElemKey key = csize > 1 ? join_top[tid] : sm.found[tid];
        a.topk_ids[row * k + tid] = 0xffffffffu - static_cast<uint32_t>(key);
        a.topk_logp[row * k + tid] = fmaf(F::order_value(static_cast<uint32_t>(key >> 32)) - rs.m, a.inv_temp, -log_s);
      }
    }
    if (err && a.status) atomicOr(a.status, err);
  }
  if (csize > 1) cluster_sync_all();  // no CTA leaves while another may still write its memory
  __syncthreads();
  // a wait has given up: which rows this CTA would still have been given is not
  // known, so every row's outputs become NaN (other CTAs may write theirs after)
  if (*abort) {
    if (tid == 0 && a.status) atomicOr(a.status, RL_DEVERR_TIMEOUT);
    for (long long row = warp; row < a.R; row += kWarps + 1) lose_logprobs(a, row, lane, 32);
  }
}

// ------------------------------------------------------------------ backward
constexpr int kBwdThreads = 256;  // at most; fewer where a row is short
constexpr int kBwdVecs = 4;       // vectors a thread has in flight
constexpr int kIdsPerThread = kMaxK / 32;

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
  long long n_seg;  // units of a row
};

// dz_v = 2^x (a0 + a1 x) with x = (z_v / T - lse) log2(e), a0 = -(sum_j g_j + h H) / T
// and a1 = -h ln(2) / T: one read and one write of the row, which is all that
// bounds it.  One CTA takes a unit of up to 16 KB of a row and the hardware deals
// the units out, so that none waits for the slowest of a static share.  All of a
// thread's loads, the row's scalars and ids among them, are in flight at once,
// and six CTAs a SM cover that one latency.  The given ids' elements are
// computed once more and written after the unit's own stores.  Measured at
// 4096 x 151,936 bf16: 360 us with the entropy's term, 6.9 TB/s (five CTAs 394;
// two vectors a thread 376, eight 419; 512 threads 437); a persistent grid of
// whole rows took 409.  Rows shorter than a unit get a CTA of just their length:
// 23 us against 105 at 30,000 x 1000.
// kList: several ids a row, in shared memory; else one id, or none, that every
// thread reads itself, and a barrier only in the id's own unit.
template <int DT, bool kEntropy, bool kList>
__global__ void __launch_bounds__(kBwdThreads, 6) token_logprobs_bwd_kernel(const LpBwdArgs a) {
  using F = Fmt<DT>;
  constexpr int kVec = F::kVec;
  __shared__ long long s_id[kList ? kMaxK : 1];
  __shared__ float s_g[kList ? kMaxK : 1];
  const int tid = threadIdx.x, n_threads = blockDim.x, unit = n_threads * kBwdVecs;
  const int V = static_cast<int>(a.V), n_ids = a.n_ids;
  const int n_vecs = (V + kVec - 1) / kVec;
  unsigned int err = 0;
  for (long long u = blockIdx.x; u < a.R * a.n_seg; u += gridDim.x) {
    const long long row = u / a.n_seg;
    const int v0 = static_cast<int>(u - row * a.n_seg) * unit;
    const int v1 = min(n_vecs, v0 + unit);
    const unsigned char* src = a.logits + row * a.row_bytes;
    unsigned char* dst = a.dlogits + row * a.row_bytes;
    const bool full = (v0 + unit) * static_cast<long long>(kVec) <= V;
    if (a.mask && a.mask[row] == 0) {
      for (int v = v0 + tid; v < v1; v += n_threads) {
        if ((v + 1) * kVec <= V)
          st_global_cs_v4(dst + static_cast<long long>(v) * 16, make_uint4(0u, 0u, 0u, 0u));
        else
          for (int i = v * kVec; i < V; ++i) F::store(dst, i, 0.f);
      }
      continue;
    }
    auto in_unit = [&](long long id) {
      return id >= static_cast<long long>(v0) * kVec && id < min(static_cast<long long>(V), static_cast<long long>(v1) * kVec);
    };
    uint4 w[kBwdVecs];
#pragma unroll
    for (int q = 0; q < kBwdVecs; ++q) {
      const int v = v0 + tid + q * n_threads;
      w[q] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(min(v, n_vecs - 1)) * 16);
    }
    const float lse = a.lse[row];
    float a0 = 0.f, a1 = 0.f, h = 0.f, H = 0.f;
    if (kEntropy) {
      h = a.dentropy[row];
      H = a.entropy[row];
    }
    float zj[kList ? kIdsPerThread : 1], g0 = 0.f;
    long long id0 = -1;
    bool mine = false;
    if (!kList && n_ids) {
      id0 = a.ids[row];
      g0 = a.dlogp[row];
      if (id0 < 0 || id0 >= V) {
        err |= RL_DEVERR_ID_RANGE;
        g0 = __int_as_float(0x7fc00000);
      }
      mine = in_unit(id0);
      if (mine) zj[0] = F::load(src, id0);  // before the unit is overwritten in place
      a0 = -g0 * a.inv_temp;
    }
    if constexpr (kList) {
      long long id[kIdsPerThread];
#pragma unroll
      for (int i = 0; i < kIdsPerThread; ++i) {
        const int j = tid + i * n_threads;
        id[i] = -1;
        if (j < n_ids) {
          id[i] = a.ids[row * n_ids + j];
          s_id[j] = id[i];
          s_g[j] = a.dlogp[row * n_ids + j];
          if (id[i] < 0 || id[i] >= V) err |= RL_DEVERR_ID_RANGE;
        }
      }
#pragma unroll
      for (int i = 0; i < kIdsPerThread; ++i) {
        const bool here = in_unit(id[i]);
        mine = mine || here;
        zj[i] = here ? F::load(src, id[i]) : 0.f;  // before the unit is overwritten in place
      }
      __syncthreads();
      float g = 0.f;
      for (int j = tid & 31; j < n_ids; j += 32)
        g += s_id[j] < 0 || s_id[j] >= V ? __int_as_float(0x7fc00000) : s_g[j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
      a0 = -g * a.inv_temp;
    }
    if (kEntropy) {
      h *= a.inv_temp;
      a0 = fmaf(-h, H, a0);
      a1 = -h * kLn2;
    }
    const float2 T2 = make_float2(a.inv_temp, a.inv_temp), nl2 = make_float2(-lse, -lse);
    const float2 L2 = make_float2(kLog2e, kLog2e), A0 = make_float2(a0, a0), A1 = make_float2(a1, a1);
    auto grad = [&](float2 z) {
      float2 x = __fmul2_rn(__ffma2_rn(z, T2, nl2), L2);
      const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      if (!kEntropy) return __fmul2_rn(p, A0);
      x = make_float2(fmaxf(x.x, -1024.f), fmaxf(x.y, -1024.f));  // p is 0 there; 0 * -inf would not be
      return __fmul2_rn(p, __ffma2_rn(A1, x, A0));
    };
#pragma unroll
    for (int q = 0; q < kBwdVecs; ++q) {
      float d[kVec];
      F::unpack(w[q], d);
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float2 g = grad(make_float2(d[i], d[i + 1]));
        d[i] = g.x;
        d[i + 1] = g.y;
      }
      w[q] = F::pack(d);
    }
    // the CTA stores at once: 7% faster than each warp when it is done (fewer
    // turns between reads and writes in DRAM)
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kBwdVecs; ++q) {
      const int v = v0 + tid + q * n_threads;
      if (full || (v + 1) * kVec <= V) {
        st_global_cs_v4(dst + static_cast<long long>(v) * 16, w[q]);
      } else if (v < n_vecs) {
        float d[kVec];
        F::unpack(w[q], d);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (v * kVec + i < V) F::store(dst, v * kVec + i, d[i]);
      }
    }
    if constexpr (!kList) {
      if (mine) {
        __syncthreads();  // the unit's stores come first
        if (tid == 0) F::store(dst, id0, fmaf(g0, a.inv_temp, grad(make_float2(zj[0], zj[0])).x));
      }
    } else {
      if (__syncthreads_or(mine) && mine) {
#pragma unroll
        for (int i = 0; i < kIdsPerThread; ++i) {
          const int j = tid + i * n_threads;
          const long long id = j < n_ids ? s_id[j] : -1;
          if (!in_unit(id)) continue;
          float g = 0.f;
#pragma unroll 8
          for (int q = 0; q < n_ids; ++q) g += s_id[q] == id ? s_g[q] : 0.f;
          F::store(dst, id, fmaf(g, a.inv_temp, grad(make_float2(zj[i], zj[i])).x));
        }
      }
      if (u + gridDim.x < a.R * a.n_seg) __syncthreads();  // the lists are free for the next unit
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

// CTAs that share a row.  One while there are rows for every CTA the GPU
// holds; for fewer rows the row's slices spread over up to 8 CTAs, as long as
// each gets a few chunks, or as many as its pieces need.  Rows x 151,936 bf16,
// 20 alternatives, us on 1, 2, 4, 8 CTAs: 1 row 27.0 18.4 14.2 13.2; 38 rows
// 28.0 19.3 15.3 15.5 (none: 24.8 15.7 12.0 10.0); 64 rows 27.9 19.2 15.5 17.5;
// 110 rows on 2 and 4: 20.7 17.6; 150 rows 20.9 30.9 (clusters of 4 wait for a
// second round); 300 rows on 1 and 2: 32.0 29.3.  Hence at most 4, 3 and 2 CTAs
// a SM in clusters of 2, 4 and 8.
int cluster_for(long long R, long long n_pieces, int sms) {
  int c = 1;
  for (int most = 4; c < kMaxCluster; c *= 2, --most)
    if (R * 2 * c > static_cast<long long>(most) * sms || n_pieces < static_cast<long long>(c) * 4 * 128) break;
  return c;
}

// Long rows in at least this many rounds are dealt out one by one (the grid has
// a CTA a row, and running CTAs take over those not started): CTAs of one SM do
// not run at the same speed, and a fixed share leaves the slowest behind.  Fixed
// against dealt, us: 4096 x 151,936 bf16, k = 0 and 64: 213, 204 and 264, 254;
// 70% of its rows valid: 164, 154; 8192 x 64,000: 200, 186.  Fewer rounds have
// nothing to even out: 777 x 50,257 fp32: 42, 47; 1300: 59, 60; 2000: 81, 80.
// Nor are short rows: the request's answer and the masked rows that it stands
// for come on top (16,384 x 32,000 fp16, k = 16, 57% valid: 167, 186).
constexpr int kDealtRounds = 3;
template <int DT, bool kEntropy, int kT>
rl_status launch_fwd(LpArgs a, int dev, int sms, cudaStream_t stream) {
  using F = Fmt<DT>;
  const void* fn = reinterpret_cast<const void*>(&token_logprobs_kernel<DT, kEntropy, kT>);
  const long long n_pieces = (a.V + F::kPiece - 1) / F::kPiece;
  int c = kT < 128 ? 1 : cluster_for(a.R, n_pieces, sms);
  while (a.k > 0 && c < kMaxCluster && (n_pieces + c - 1) / c > kMaxPieces) c *= 2;
  const int places = key_places<F>(static_cast<int>((n_pieces + c - 1) / c), a.k);
  constexpr int join_bytes = kJoinKeys * static_cast<int>(sizeof(ElemKey));
  // (keys are read a vector at a time: 16 bytes past the last)
  const int smem = static_cast<int>(sizeof(LpSmem<DT, kT>) + places * sizeof(typename F::Key)) + 16 + (c > 1 && a.k ? join_bytes : 0);
  constexpr int most_smem = static_cast<int>(sizeof(LpSmem<DT, kT>) + kMaxPieces * sizeof(typename F::Key)) + 16 + join_bytes;
  static std::atomic<unsigned long long> allowed{0};
  const rl_status st = allow_smem(fn, dev, most_smem, allowed);
  if (st != RL_OK) return st;
  int held = kSmemPerSm / (smem + 1024);  // CTAs a SM holds at once (1 KB each is the system's)
  if (held > kLpCtas<kT>) held = kLpCtas<kT>;
  const long long most = static_cast<long long>(held) * sms / c;
  a.resident = static_cast<int>(most);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(c);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  const bool dealt = kT == 128 && c == 1 && a.R >= kDealtRounds * most;
  cfg.gridDim = dim3(static_cast<unsigned>(dealt ? a.R : c * (a.R < most ? a.R : most)));
  cfg.blockDim = dim3(kT + 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = c > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<DT, kEntropy, kT>, a) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

// Rows of at most kShortRow bytes, where there are enough of them, go to CTAs of
// half the size: what a row costs at its end (joining the warps, the search's
// chain of barriers) then stalls a smaller part of the SM.  128 against 64
// threads, us: 30,000 x 1000 bf16, k = 16: 233, 156; 16,384 x 32,000: 285, 259;
// 8192 x 50,000: 201, 186; 8192 x 64,000, k = 0: 193, 194, k = 64: 254, 260;
// 4096 x 151,936: 243, 284.
constexpr long long kShortRow = 100 * 1024;
template <int DT, bool kEntropy>
rl_status launch_fwd(const LpArgs& a, int dev, int sms, cudaStream_t stream) {
  if (a.V * Fmt<DT>::kBytes <= kShortRow && a.R >= 8LL * sms && a.k <= 64 && a.n_ids <= 64)
    return launch_fwd<DT, kEntropy, 64>(a, dev, sms, stream);
  return launch_fwd<DT, kEntropy, 128>(a, dev, sms, stream);
}

template <int DT, bool kEntropy>
rl_status launch_bwd(const LpBwdArgs& a, int threads, cudaStream_t stream) {
  const long long units = a.R * a.n_seg, most = 1LL << 30;
  const unsigned grid = static_cast<unsigned>(units < most ? units : most);
  if (a.n_ids > 1)
    token_logprobs_bwd_kernel<DT, kEntropy, true><<<grid, threads, 0, stream>>>(a);
  else
    token_logprobs_bwd_kernel<DT, kEntropy, false><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

bool shape_ok(long long R, long long V, long long ld) {
  return R >= 0 && R < (1LL << 31) && V >= 1 && V <= kMaxVocab && ld >= V && ld <= (1LL << 31);
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
  if (mask && R > kMaxMaskedRows) return RL_ERR_SHAPE;
  if (k > V || (k > 0 && V * es > static_cast<long long>(kMaxPieces) * kPieceBytes * kMaxCluster)) return RL_ERR_SHAPE;
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
  if (dlogits != logits && rows_overlap(logits, dlogits, R, row_bytes, V * es)) return RL_ERR_ALIAS;
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
  const int threads = static_cast<int>(n_vecs >= kBwdThreads * kBwdVecs ? kBwdThreads
                                                                        : ((n_vecs + 32 * kBwdVecs - 1) / (32 * kBwdVecs)) * 32);
  a.n_seg = (n_vecs + threads * kBwdVecs - 1) / (threads * kBwdVecs);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ent = dentropy != nullptr;
  switch (dtype) {
    case RL_F32: return ent ? launch_bwd<RL_F32, true>(a, threads, s) : launch_bwd<RL_F32, false>(a, threads, s);
    case RL_BF16: return ent ? launch_bwd<RL_BF16, true>(a, threads, s) : launch_bwd<RL_BF16, false>(a, threads, s);
    case RL_F16: return ent ? launch_bwd<RL_F16, true>(a, threads, s) : launch_bwd<RL_F16, false>(a, threads, s);
  }
  return RL_ERR_DTYPE;
}
