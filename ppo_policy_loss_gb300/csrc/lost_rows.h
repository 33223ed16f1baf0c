// lost_rows.h — what the token operators leave behind when a wait has given up
// (RL_DEVERR_TIMEOUT): NaN.  Plain C++, so that a host can run it.
#pragma once

#include <cmath>

#include "rltoken.h"

#ifdef __CUDACC__
#define RL_LOST_FN __host__ __device__ __forceinline__
#else
#define RL_LOST_FN inline
#endif

namespace rl {

// A row's outputs of rl_token_logprobs, share `part` of `parts` of them.
template <class Out>
RL_LOST_FN void lose_logprobs(const Out& o, long long row, int part, int parts) {
  for (int q = part; q < o.n_ids; q += parts) o.logp[row * o.n_ids + q] = NAN;
  for (int q = part; q < o.k; q += parts) {
    o.topk_ids[row * o.k + q] = -1;
    o.topk_logp[row * o.k + q] = NAN;
  }
  if (part == 0 && o.entropy) o.entropy[row] = NAN;
  if (part == 0 && o.lse) o.lse[row] = NAN;
}

// The record of rl_topk_distill_fwd_bwd.
RL_LOST_FN void lose_record(rl_distill_stats& o) {
  o.loss = o.forward_kl = o.reverse_kl = o.teacher_tail = o.student_tail = static_cast<double>(NAN);
}

}  // namespace rl
