// Instantiations of the layer norm's forward kernels.
#include "eql_block.h"

namespace eql {

template <typename Elt, int LPR, bool WHOLE>
static const void* fwd_k(int k) {
  if constexpr (LPR == 256) {
    if (k == 6) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 6, WHOLE>;
    if (k == 8) return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 8, WHOLE>;
  }
  switch (k) {
    case 1: return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 1, WHOLE>;
    case 2: return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 2, WHOLE>;
    case 3: return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 3, WHOLE>;
    case 4: return (const void*)&eql_norm_fwd_kernel<Elt, LPR, 4, WHOLE>;
    default: return nullptr;
  }
}

template <typename Elt, bool WHOLE>
static const void* fwd_shape(NormShape sh) {
  return sh.lpr == 16 ? fwd_k<Elt, 16, WHOLE>(sh.k) : (sh.lpr == 64 ? fwd_k<Elt, 64, WHOLE>(sh.k) : fwd_k<Elt, 256, WHOLE>(sh.k));
}

hipError_t launch_norm_fwd(bool f16, NormShape sh, const NormArgs& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  const void* fn = f16 ? (whole ? fwd_shape<_Float16, true>(sh) : fwd_shape<_Float16, false>(sh))
                       : (whole ? fwd_shape<float, true>(sh) : fwd_shape<float, false>(sh));
  return fn ? launch_kernel(fn, grid, a, s) : hipErrorInvalidValue;
}

hipError_t launch_norm_fwd_wide(bool f16, const NormArgs& a, hipStream_t s) {
  return launch_kernel(f16 ? (const void*)&eql_norm_fwd_wide_kernel<_Float16> : (const void*)&eql_norm_fwd_wide_kernel<float>,
                       (unsigned)a.N, a, s, 1024);
}

}  // namespace eql
