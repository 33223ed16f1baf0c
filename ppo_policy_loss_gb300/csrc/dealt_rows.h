// dealt_rows.h — the order in which a CTA takes its rows: every stride-th of
// them, or one number after another as the hardware deals them out.  Plain C++,
// so that a host can run it on any order of numbers.
#pragma once

#ifdef __CUDACC__
#define RL_ROWS_FN __host__ __device__ __forceinline__
#else
#define RL_ROWS_FN inline
#endif

namespace rl {

// Number n stands for the n-th valid row, if there are so many, and for row n
// itself, if that is masked.  A CTA that is dealt its numbers asks for the next
// one while a row streams; they may come in any order, so only the answer that
// none is left (-1) ends its work, and nothing is asked after it.
//   ask()        asks for a number
//   answer()     waits for it
//   row_of(n)    the n-th valid row, -1 past the last
//   stream(row)  false once a wait has given up; row -1: the end
//   masked(n)    writes row n, if it is masked
template <class Ask, class Answer, class RowOf, class Stream, class Masked>
RL_ROWS_FN void take_rows(long long first, long long stride, bool dealt, Ask ask, Answer answer, RowOf row_of,
                          Stream stream, Masked masked) {
  for (long long n = first;;) {
    const bool end = n < 0;
    if (dealt && !end) ask();
    const long long row = end ? -1 : row_of(n);
    if ((end || row >= 0) && !stream(row)) return;
    if (end) return;
    if (dealt) masked(n);
    n = dealt ? answer() : row >= 0 ? n + stride : -1;
  }
}

}  // namespace rl
