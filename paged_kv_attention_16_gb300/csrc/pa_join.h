// pa_join.h -- the reference exponent of two partials' join, in pa_span.cu's merge and
// sums over rows (plain C++ too, so that it is tested without a GPU; not part of the
// public C ABI).
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define PA_JOIN_FN __host__ __device__ inline
#else
#define PA_JOIN_FN inline
#endif

namespace pa {

// Of two log-sum-exps or references the larger one; a NaN stays (a score that is none
// makes its row NaN), and +inf stays above all, NaN too: it is the mark of a piece that
// met a bad page, whose rows are zero and whose request's weights are left alone.
PA_JOIN_FN float join_top(float a, float b) {
  if (a == INFINITY || b == INFINITY) return INFINITY;
  return b > a || b != b ? b : a;
}

}  // namespace pa
