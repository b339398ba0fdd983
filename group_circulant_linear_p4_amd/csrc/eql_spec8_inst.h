// Shared by the translation units that instantiate eql_spec8_kernel.
#pragma once

#include "eql_block.h"

namespace eql {

template <int T, typename Elt>
static hipError_t spec8_view(int view, const Spec8Args& a, unsigned grid, hipStream_t s) {
  switch (view) {
    case kViewPlain: return launch_kernel((const void*)&eql_spec8_kernel<T, Elt, kViewPlain>, grid, a, s);
    case kViewAffine: return launch_kernel((const void*)&eql_spec8_kernel<T, Elt, kViewAffine>, grid, a, s);
    case kViewGelu: return launch_kernel((const void*)&eql_spec8_kernel<T, Elt, kViewGelu>, grid, a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace eql
