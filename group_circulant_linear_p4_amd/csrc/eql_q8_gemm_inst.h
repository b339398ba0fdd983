// Instantiations of the 8-bit product kernels for one output type.
#pragma once

#include "eql_q8_launch.h"

namespace eql {

template <typename Elt, int T>
static hipError_t q8_fwd_one(Q8Kind kind, const Q8FwdArgs& a, unsigned grid, hipStream_t s) {
  constexpr Q8Tile M = q8_tile(T, false), B = q8_tile(T, true);
  if (kind == Q8Kind::kToken) return launch_kernel((const void*)&eql_q8_token_kernel<T, Elt>, grid, a, s);
  if (kind == Q8Kind::kSmall) return launch_kernel((const void*)&eql_q8_small_kernel<T, Elt>, grid, a, s, 64u * (unsigned)a.waves);
  if constexpr (T <= kQ8LargeT) {
    if (kind == Q8Kind::kBig) return launch_kernel((const void*)&eql_q8_large_kernel<T, Elt, B.mb, B.nb>, grid, a, s);
    return launch_kernel((const void*)&eql_q8_large_kernel<T, Elt, M.mb, M.nb>, grid, a, s);
  }
  return hipErrorInvalidValue;
}

template <typename Elt>
static hipError_t q8_fwd_launch(int T, Q8Kind kind, const Q8FwdArgs& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return q8_fwd_one<Elt, t>(kind, a, grid, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
