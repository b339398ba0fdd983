// Weight-gradient transform instantiations for the f16 element type, T = 1..16.  A source of its own
// because it is compiled without the straight-line vectoriser (build.py), which the reduce's bits
// were taken with.
#include "eql_launch.h"

namespace eql {

template <int T>
static hipError_t spec_one(const SpecArgs& a, unsigned grid, hipStream_t s) {
  return launch_kernel((const void*)&eql_spec_kernel<T, _Float16>, grid, a, s);
}

hipError_t launch_spec_f16(int T, const SpecArgs& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return spec_one<t>(a, grid, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
