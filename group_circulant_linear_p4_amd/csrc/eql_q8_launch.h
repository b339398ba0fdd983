// Internal launch interface of the 8-bit rows, weights and products: between eql_q8_api.hip and the
// kernel instantiations.
#pragma once

#include "eql_block.h"
#include "eql_q8_gemm.h"

namespace eql {

// Lanes per row of the row kernels and chunks per lane, for rows of `chunks` chunks; k = 0: the row
// does not fit a workgroup's registers.
constexpr NormShape q8_shape(int64_t chunks, int T) {
  const int keep = q8_keep(T);
  if (chunks <= 32 && keep >= 2) return {16, chunks <= 16 ? 1 : 2};
  const int lpr = chunks <= 64 * keep ? 64 : 256;
  const int64_t k = (chunks + lpr - 1) / lpr;
  return {lpr, k > keep ? 0 : (k > 2 ? 4 : (int)k)};
}

// Tile of the large product kernel: 32 MB rows x 128 NB output channels.
constexpr int q8_mb(int T) { return T <= 4 ? 4 : (T <= 8 ? 2 : 1); }
constexpr int q8_nb(int T) { return T <= 2 ? 2 : 1; }
// Waves of the small one: eight where their accumulators leave room.
constexpr int q8_waves(int T) { return T <= 8 ? 8 : 4; }

hipError_t launch_q8_rows_f16(int T, NormShape sh, const Q8RowsArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_q8_rows_f32(int T, NormShape sh, const Q8RowsArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_q8_pack(bool f16, int T, const Q8PackArgs& a, hipStream_t s);
hipError_t launch_q8_fwd_f16(int T, bool large, const Q8FwdArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_q8_fwd_f32(int T, bool large, const Q8FwdArgs& a, unsigned grid, hipStream_t s);

}  // namespace eql
