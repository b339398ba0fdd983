// Instantiations of the half spectrum from an 8-bit checkpoint: every T, both element types.
#include "eql_block.h"

namespace eql {

hipError_t launch_spec8_f16(int T, const Spec8Args& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return launch_kernel((const void*)&eql_spec8_kernel<t, _Float16>, grid, a, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

hipError_t launch_spec8_f32(int T, const Spec8Args& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return launch_kernel((const void*)&eql_spec8_kernel<t, float>, grid, a, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
