// Instantiations of the half spectrum from an 8-bit checkpoint (fp16): every T and view.
#include "eql_spec8_inst.h"

namespace eql {

hipError_t launch_spec8_f16(int T, int view, const Spec8Args& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return spec8_view<t, _Float16>(view, a, grid, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
