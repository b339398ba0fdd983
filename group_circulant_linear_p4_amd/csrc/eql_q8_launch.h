// Internal launch interface of the 8-bit rows, weights and products: between eql_q8_api.hip and the
// kernel instantiations.
#pragma once

#include "eql_block.h"
#include "eql_q8_gemm.h"

namespace eql {

// Lanes per row of the row kernels and chunks per lane, for N rows of C channels; k = 0: the row does not fit a
// workgroup's registers.  Few rows take more lanes a row, one chunk each: their time is one wave's (197 rows of 96
// channels, T = 4 fp16, the norm: 4.9 us on 16 lanes a row, 3.8 on 64).  Otherwise 32 values a lane: with 64, too few
// waves hide the memory's latency (65536 rows of 1024 channels, T = 4 fp16: 165 us on 64 lanes a row, 139 on 256).
constexpr NormShape q8_shape(int64_t C, int T, int elt, int64_t N) {
  const int64_t chunks = (C + q8_chunk(T, elt) - 1) / q8_chunk(T, elt);
  const int some = N <= 1024 ? 1 : q8_some(T, elt), keep = q8_keep(T, elt);
  const int lpr = N > 4096 && chunks <= 16 * some ? 16 : (chunks <= 64 * some ? 64 : 256);
  const int64_t k = (chunks + lpr - 1) / lpr;
  return {lpr, k > keep ? 0 : (k > 4 ? 8 : (k > 2 ? 4 : (int)k))};
}

// How a product runs (eql_q8_gemm.h).
enum class Q8Kind { kToken, kSmall, kMedium, kBig };
// Tiles of the large kernel: 32 MB rows x 128 NB output channels.  The big tile's accumulators (128 registers up to T = 4)
// leave two workgroups a compute unit; the medium one has half to a quarter of the outputs, and more workgroups (T = 1,
// 1000 rows of 1024 -> 1024: 5.9 us, with 256 channels 7.2; T = 2, 2000 rows of 768 -> 768: 7.7, with 32 rows x 256 8.7).
struct Q8Tile {
  int mb, nb;
};
constexpr Q8Tile q8_tile(int T, bool big) {
  if (T <= 2) return {big && T == 1 ? 4 : 2, big ? 2 : 1};
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
