// Instantiations of the 8-bit row kernels for one element type.
#pragma once

#include "eql_q8_launch.h"

namespace eql {

// The lanes and chunks that q8_shape gives.
template <typename Elt, int T>
static const void* q8_rows_fn(NormShape sh) {
  constexpr int SOME = q8_some(T, sizeof(Elt)), KEEP = q8_keep(T, sizeof(Elt));
  if (sh.k == 0) return (const void*)&eql_q8_rows_wide_kernel<Elt, T>;
  if (sh.k == 1) {
    if (sh.lpr == 16) return (const void*)&eql_q8_rows_kernel<Elt, T, 16, 1>;
    return sh.lpr == 64 ? (const void*)&eql_q8_rows_kernel<Elt, T, 64, 1> : (const void*)&eql_q8_rows_kernel<Elt, T, 256, 1>;
  }
  if (sh.lpr == 256) {
    if (sh.k == 2) return (const void*)&eql_q8_rows_kernel<Elt, T, 256, 2>;
    if (sh.k == 4) return (const void*)&eql_q8_rows_kernel<Elt, T, 256, 4>;
    if constexpr (KEEP == 8) return (const void*)&eql_q8_rows_kernel<Elt, T, 256, 8>;
    return nullptr;
  }
  if constexpr (SOME >= 2) {
    if (sh.k == 2) return sh.lpr == 16 ? (const void*)&eql_q8_rows_kernel<Elt, T, 16, 2> : (const void*)&eql_q8_rows_kernel<Elt, T, 64, 2>;
  }
  if constexpr (SOME >= 4) {
    if (sh.k == 4) return sh.lpr == 16 ? (const void*)&eql_q8_rows_kernel<Elt, T, 16, 4> : (const void*)&eql_q8_rows_kernel<Elt, T, 64, 4>;
  }
  return nullptr;
}

template <typename Elt>
static hipError_t q8_rows_launch(int T, NormShape sh, const Q8RowsArgs& a, unsigned grid, hipStream_t s) {
  const void* fn = nullptr;
  switch (T) {
#define EQL_CASE(t) case t: fn = q8_rows_fn<Elt, t>(sh); break;
    EQL_CASE(1) EQL_CASE(2) EQL_CASE(3) EQL_CASE(4) EQL_CASE(5) EQL_CASE(6) EQL_CASE(7) EQL_CASE(8)
    EQL_CASE(9) EQL_CASE(10) EQL_CASE(11) EQL_CASE(12) EQL_CASE(13) EQL_CASE(14) EQL_CASE(15) EQL_CASE(16)
#undef EQL_CASE
  }
  return fn ? launch_kernel(fn, grid, a, s) : hipErrorInvalidValue;
}

}  // namespace eql
