// Instantiations of the RMS norm's kernels.
#include "eql_block.h"

namespace eql {

// The chunks a lane that norm_shape gives for LPR lanes (as eql_norm_fwd.hip and eql_norm_bwd.hip).
template <typename Elt, int LPR, bool WHOLE, bool STREAM>
static const void* fwd_k(int k) {
  if constexpr (LPR <= 64) {
    if (k == 1) return (const void*)&eql_rms_fwd_kernel<Elt, LPR, 1, WHOLE, STREAM>;
  } else {
    if (k == 6) return (const void*)&eql_rms_fwd_kernel<Elt, LPR, 6, WHOLE, STREAM>;
    if (k == 8) return (const void*)&eql_rms_fwd_kernel<Elt, LPR, 8, WHOLE, STREAM>;
  }
  if (k == 2) return (const void*)&eql_rms_fwd_kernel<Elt, LPR, 2, WHOLE, STREAM>;
  if constexpr (LPR >= 64) {
    if (k == 3) return (const void*)&eql_rms_fwd_kernel<Elt, LPR, 3, WHOLE, STREAM>;
    if (k == 4) return (const void*)&eql_rms_fwd_kernel<Elt, LPR, 4, WHOLE, STREAM>;
  }
  return nullptr;
}

template <typename Elt, int LPR, bool WHOLE, bool STREAM>
static const void* bwd_k(int k) {
  if constexpr (LPR <= 64) {
    if (k == 1) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 1, WHOLE, STREAM, false, true>;
  }
  if (k == 2) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 2, WHOLE, STREAM, false, true>;
  if constexpr (LPR >= 64) {
    if (k == 3) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 3, WHOLE, STREAM, false, true>;
    if (k == 4) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 4, WHOLE, STREAM, false, true>;
  }
  return nullptr;
}

template <typename Elt, bool WHOLE, bool STREAM>
static const void* shape_fn(bool bwd, NormShape sh) {
  if (bwd)
    return sh.lpr == 16 ? bwd_k<Elt, 16, WHOLE, STREAM>(sh.k)
                        : (sh.lpr == 64 ? bwd_k<Elt, 64, WHOLE, STREAM>(sh.k) : bwd_k<Elt, 256, WHOLE, STREAM>(sh.k));
  return sh.lpr == 16 ? fwd_k<Elt, 16, WHOLE, STREAM>(sh.k)
                      : (sh.lpr == 64 ? fwd_k<Elt, 64, WHOLE, STREAM>(sh.k) : fwd_k<Elt, 256, WHOLE, STREAM>(sh.k));
}

// Rows that start inside a line are never streamed (load_chunk8).
static const void* rms_fn(bool bwd, bool f16, bool whole, bool stream, NormShape sh) {
  if (!whole) return f16 ? shape_fn<_Float16, false, false>(bwd, sh) : shape_fn<float, false, false>(bwd, sh);
  if (stream) return f16 ? shape_fn<_Float16, true, true>(bwd, sh) : shape_fn<float, true, true>(bwd, sh);
  return f16 ? shape_fn<_Float16, true, false>(bwd, sh) : shape_fn<float, true, false>(bwd, sh);
}

hipError_t launch_rms_fwd(bool f16, bool stream, NormShape sh, const NormArgs& a, unsigned grid, hipStream_t s) {
  const void* fn = rms_fn(false, f16, a.R % 8 == 0, stream, sh);
  if (!fn) return hipErrorInvalidValue;
  void* kargs[] = {const_cast<NormArgs*>(&a)};
  const size_t lds = a.table ? (size_t)norm_table_row(a.R) * (f16 ? 2 : 4) : 0;
  return hipLaunchKernel(fn, dim3(grid), dim3(256), kargs, lds, s);
}

hipError_t launch_rms_fwd_wide(bool f16, const NormArgs& a, hipStream_t s) {
  return launch_kernel(f16 ? (const void*)&eql_rms_fwd_wide_kernel<_Float16> : (const void*)&eql_rms_fwd_wide_kernel<float>,
                       (unsigned)a.N, a, s, 1024);
}

hipError_t launch_rms_bwd(bool f16, bool stream, NormShape sh, const NormArgs& a, unsigned grid, hipStream_t s) {
  const void* fn = rms_fn(true, f16, a.R % 8 == 0, stream, sh);
  if (!fn) return hipErrorInvalidValue;
  void* kargs[] = {const_cast<NormArgs*>(&a)};
  const size_t sums = a.part || a.dgamma ? (size_t)norm_bwd_copies(sh.lpr) * (size_t)a.R * sizeof(float) : 0;
  const size_t table = a.table ? (size_t)norm_table_row(a.R) * (f16 ? 2 : 4) : 0;
  return hipLaunchKernel(fn, dim3(grid), dim3(256), kargs, sums > table ? sums : table, s);
}

template <typename Elt>
static hipError_t bwd_wide(const NormArgs& a, unsigned colGrid, hipStream_t s) {
  const hipError_t e = launch_kernel((const void*)&eql_norm_bwd_rows_kernel<Elt, false, true>, (unsigned)a.N, a, s, 1024);
  if (e != hipSuccess) return e;
  return launch_kernel((const void*)&eql_norm_bwd_cols_kernel<Elt, false, true>, colGrid, a, s);
}

hipError_t launch_rms_bwd_wide(bool f16, const NormArgs& a, unsigned colGrid, hipStream_t s) {
  return f16 ? bwd_wide<_Float16>(a, colGrid, s) : bwd_wide<float>(a, colGrid, s);
}

}  // namespace eql
