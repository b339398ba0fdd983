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
  const int lpr = chunks <= 64 * (keep < 2 ? keep : 2) ? 64 : 256;
  const int64_t k = (chunks + lpr - 1) / lpr;
  return {lpr, k > keep ? 0 : (k > 2 ? 4 : (int)k)};
}

// How a product runs (eql_q8_gemm.h).
enum class Q8Kind { kToken, kSmall, kMedium, kBig };
// Tiles of the large kernel: 32 MB rows x 128 NB output channels.  Accumulators of two workgroups a compute unit
// (128 registers each) for the big tile up to T = 4, where the medium one has half the rows.
struct Q8Tile {
  int mb, nb;
};
constexpr Q8Tile q8_tile(int T, bool big) {
  if (T == 1) return {big ? 4 : 2, 2};
  if (T == 2) return {big ? 2 : 1, 2};
  return {big && T <= 4 ? 2 : 1, 1};
}
// Group orders whose accumulators leave the large kernel enough registers.
constexpr int kQ8LargeT = 12;
// Waves of the small kernel at most: eight where their accumulators leave room.
constexpr int q8_waves(int T) { return T <= 8 ? 8 : 4; }

hipError_t launch_q8_rows_f16(int T, NormShape sh, const Q8RowsArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_q8_rows_f32(int T, NormShape sh, const Q8RowsArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_q8_pack(bool f16, int T, const Q8PackArgs& a, hipStream_t s);
hipError_t launch_q8_fwd_f16(int T, Q8Kind kind, const Q8FwdArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_q8_fwd_f32(int T, Q8Kind kind, const Q8FwdArgs& a, unsigned grid, hipStream_t s);

}  // namespace eql
