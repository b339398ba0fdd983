// Instantiations of the kernel that packs a weight in 8 bits.
#include "eql_q8_launch.h"

namespace eql {

hipError_t launch_q8_pack(bool f16, int T, const Q8PackArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.Dpad / 4;
#define EQL_CASE(t) \
  return launch_kernel(f16 ? (const void*)&eql_q8_pack_kernel<_Float16, t> : (const void*)&eql_q8_pack_kernel<float, t>, grid, a, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
