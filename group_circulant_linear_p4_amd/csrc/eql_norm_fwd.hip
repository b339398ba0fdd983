// Instantiations of the layer norm's forward kernels.
#include "eql_block.h"

namespace eql {

// The chunks a lane that norm_shape gives for LPR lanes (rows of up to kNormFwdMaxRow features).
template <typename Elt, int LPR, bool WHOLE, bool STREAM>
static const void* fwd_k(int k) {
  if constexpr (LPR == 16) {
    if (k == 1) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 1, WHOLE, STREAM>;
    if (k == 2) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 2, WHOLE, STREAM>;
  } else {
    if constexpr (LPR == 64) {
      if (k == 1) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 1, WHOLE, STREAM>;
    } else {
      if (k == 6) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 6, WHOLE, STREAM>;
      if (k == 8) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 8, WHOLE, STREAM>;
    }
    if (k == 2) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 2, WHOLE, STREAM>;
    if (k == 3) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 3, WHOLE, STREAM>;
    if (k == 4) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 4, WHOLE, STREAM>;
  }
  return nullptr;
}

template <typename Elt, bool WHOLE, bool STREAM>
static const void* fwd_shape(NormShape sh) {
  return sh.lpr == 16 ? fwd_k<Elt, 16, WHOLE, STREAM>(sh.k) : (sh.lpr == 64 ? fwd_k<Elt, 64, WHOLE, STREAM>(sh.k) : fwd_k<Elt, 256, WHOLE, STREAM>(sh.k));
}

// Rows that start inside a line are never streamed (load_chunk8).
template <typename Elt>
static const void* fwd_fn(NormShape sh, bool whole, bool stream) {
  return !whole ? fwd_shape<Elt, false, false>(sh) : (stream ? fwd_shape<Elt, true, true>(sh) : fwd_shape<Elt, true, false>(sh));
}

hipError_t launch_norm_fwd(bool f16, bool stream, NormShape sh, const NormArgs& a, unsigned grid, hipStream_t s) {
  const void* fn = f16 ? fwd_fn<_Float16>(sh, a.R % 8 == 0, stream) : fwd_fn<float>(sh, a.R % 8 == 0, stream);
  if (!fn) return hipErrorInvalidValue;
  void* kargs[] = {const_cast<NormArgs*>(&a)};
  const size_t lds = a.table ? (size_t)norm_table_row(a.R) * (f16 ? 2 : 4) * 2 : 0;
  return hipLaunchKernel(fn, dim3(grid), dim3(256), kargs, lds, s);
}

hipError_t launch_norm_fwd_wide(bool f16, const NormArgs& a, hipStream_t s) {
  return launch_kernel(f16 ? (const void*)&eql_norm_fwd_wide_kernel<_Float16> : (const void*)&eql_norm_fwd_wide_kernel<float>,
                       (unsigned)a.N, a, s, 1024);
}

}  // namespace eql
