// Instantiations of the 8-bit checkpoint kernels: pack, unpack and the GELU epilogue's backward.
#include "eql_block.h"

namespace eql {

hipError_t launch_ckpt_pack(bool f16, const CkptArgs& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  const void* fn = f16 ? (whole ? (const void*)&eql_ckpt_pack_kernel<_Float16, true> : (const void*)&eql_ckpt_pack_kernel<_Float16, false>)
                       : (whole ? (const void*)&eql_ckpt_pack_kernel<float, true> : (const void*)&eql_ckpt_pack_kernel<float, false>);
  return launch_kernel(fn, grid, a, s);
}

hipError_t launch_ckpt_unpack(bool f16, const CkptArgs& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  const void* fn = f16 ? (whole ? (const void*)&eql_ckpt_unpack_kernel<_Float16, true> : (const void*)&eql_ckpt_unpack_kernel<_Float16, false>)
                       : (whole ? (const void*)&eql_ckpt_unpack_kernel<float, true> : (const void*)&eql_ckpt_unpack_kernel<float, false>);
  return launch_kernel(fn, grid, a, s);
}

hipError_t launch_epi8(bool f16, const Epi8Args& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  const void* fn = f16 ? (whole ? (const void*)&eql_epi8_kernel<_Float16, true> : (const void*)&eql_epi8_kernel<_Float16, false>)
                       : (whole ? (const void*)&eql_epi8_kernel<float, true> : (const void*)&eql_epi8_kernel<float, false>);
  return launch_kernel(fn, grid, a, s);
}

}  // namespace eql
