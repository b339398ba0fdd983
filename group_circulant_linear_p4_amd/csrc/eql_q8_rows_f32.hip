// Instantiations of the 8-bit row kernels: f32.
#include "eql_q8_rows_inst.h"

namespace eql {

hipError_t launch_q8_rows_f32(int T, NormShape sh, const Q8RowsArgs& a, unsigned grid, hipStream_t s) {
  return q8_rows_launch<float>(T, sh, a, grid, s);
}

}  // namespace eql
