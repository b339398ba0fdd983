// Instantiations of the layer norm's backward kernels and of the parameter gradients' sum.
#include "eql_block.h"

namespace eql {

// The chunks a lane that norm_shape gives for LPR lanes (rows of up to kNormBwdMaxRow features).
template <typename Elt, int LPR, bool WHOLE, bool STREAM, bool CKPT>
static const void* bwd_k(int k) {
  if constexpr (LPR <= 64) {
    if (k == 1) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 1, WHOLE, STREAM, CKPT>;
  }
  if (k == 2) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 2, WHOLE, STREAM, CKPT>;
  if constexpr (LPR >= 64) {
    if (k == 3) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 3, WHOLE, STREAM, CKPT>;
    if (k == 4) return (const void*)&eql_norm_bwd_kernel<Elt, LPR, 4, WHOLE, STREAM, CKPT>;
  }
  return nullptr;
}

template <typename Elt, bool WHOLE, bool STREAM, bool CKPT>
static const void* bwd_shape(NormShape sh) {
  return sh.lpr == 16 ? bwd_k<Elt, 16, WHOLE, STREAM, CKPT>(sh.k)
                      : (sh.lpr == 64 ? bwd_k<Elt, 64, WHOLE, STREAM, CKPT>(sh.k) : bwd_k<Elt, 256, WHOLE, STREAM, CKPT>(sh.k));
}

// Of rows that start inside a line only the codes are streamed (load_chunk8).
template <typename Elt, bool CKPT>
static const void* bwd_fn(NormShape sh, bool whole, bool stream) {
  if (whole) return stream ? bwd_shape<Elt, true, true, CKPT>(sh) : bwd_shape<Elt, true, false, CKPT>(sh);
  if constexpr (CKPT) {
    if (stream) return bwd_shape<Elt, false, true, CKPT>(sh);
  }
  return bwd_shape<Elt, false, false, CKPT>(sh);
}

hipError_t launch_norm_bwd(bool f16, bool stream, NormShape sh, bool ckpt, const NormArgs& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  const void* fn = f16 ? (ckpt ? bwd_fn<_Float16, true>(sh, whole, stream) : bwd_fn<_Float16, false>(sh, whole, stream))
                       : (ckpt ? bwd_fn<float, true>(sh, whole, stream) : bwd_fn<float, false>(sh, whole, stream));
  if (!fn) return hipErrorInvalidValue;
  void* kargs[] = {const_cast<NormArgs*>(&a)};
  const size_t sums = a.part || a.dgamma || a.dbeta ? (size_t)norm_bwd_copies(sh.lpr) * (size_t)a.R * sizeof(float) : 0;
  const size_t table = a.table ? (size_t)norm_table_row(a.R) * (f16 ? 2 : 4) : 0;
  const size_t lds = sums > table ? sums : table;
  return hipLaunchKernel(fn, dim3(grid), dim3(256), kargs, lds, s);
}

template <typename Elt, bool CKPT>
static hipError_t bwd_wide(const NormArgs& a, unsigned colGrid, hipStream_t s) {
  const hipError_t e = launch_kernel((const void*)&eql_norm_bwd_rows_kernel<Elt, CKPT>, (unsigned)a.N, a, s, 1024);
  if (e != hipSuccess) return e;
  return launch_kernel((const void*)&eql_norm_bwd_cols_kernel<Elt, CKPT>, colGrid, a, s);
}

hipError_t launch_norm_bwd_wide(bool f16, bool ckpt, const NormArgs& a, unsigned colGrid, hipStream_t s) {
  return f16 ? (ckpt ? bwd_wide<_Float16, true>(a, colGrid, s) : bwd_wide<_Float16, false>(a, colGrid, s))
             : (ckpt ? bwd_wide<float, true>(a, colGrid, s) : bwd_wide<float, false>(a, colGrid, s));
}

hipError_t launch_norm_param(bool f16, const NormParamArgs& a, hipStream_t s) {
  return launch_kernel(f16 ? (const void*)&eql_norm_param_kernel<_Float16> : (const void*)&eql_norm_param_kernel<float>,
                       (a.dbeta ? 2u : 1u) * (unsigned)a.groups, a, s, 1024);
}

}  // namespace eql
