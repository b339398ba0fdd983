// Instantiations of the 8-bit product kernels: f32 outputs.
#include "eql_q8_gemm_inst.h"

namespace eql {

hipError_t launch_q8_fwd_f32(int T, Q8Kind kind, const Q8FwdArgs& a, unsigned grid, hipStream_t s) {
  return q8_fwd_launch<float>(T, kind, a, grid, s);
}

}  // namespace eql
