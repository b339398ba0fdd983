// Instantiations of the 8-bit product kernels for one output type.
#pragma once

#include "eql_q8_launch.h"

namespace eql {

template <typename Elt, int T>
static hipError_t q8_fwd_one(bool large, const Q8FwdArgs& a, unsigned grid, hipStream_t s) {
  if (large) return launch_kernel((const void*)&eql_q8_large_kernel<T, Elt, q8_mb(T), q8_nb(T), 1>, grid, a, s);
  return launch_kernel((const void*)&eql_q8_small_kernel<T, Elt, q8_waves(T)>, grid, a, s, 64u * q8_waves(T));
}

template <typename Elt>
static hipError_t q8_fwd_launch(int T, bool large, const Q8FwdArgs& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return q8_fwd_one<Elt, t>(large, a, grid, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
