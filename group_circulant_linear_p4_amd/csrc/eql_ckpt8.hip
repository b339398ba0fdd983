// Instantiations of the 8-bit checkpoint kernels: pack, unpack and the GELU epilogue's backward.
#include "eql_block.h"

namespace eql {

#define EQL_PICK(kernel)                                                                                 \
  (f16 ? (whole ? (stream ? (const void*)&kernel<_Float16, true, true> : (const void*)&kernel<_Float16, true, false>)   \
                : (stream ? (const void*)&kernel<_Float16, false, true> : (const void*)&kernel<_Float16, false, false>)) \
       : (whole ? (stream ? (const void*)&kernel<float, true, true> : (const void*)&kernel<float, true, false>)         \
                : (stream ? (const void*)&kernel<float, false, true> : (const void*)&kernel<float, false, false>)))

hipError_t launch_ckpt_pack(bool f16, bool stream, const CkptArgs& a, unsigned grid, hipStream_t s) {
  // Rows that start inside a line are never streamed (load_chunk8).
  const bool whole = a.R % 8 == 0;
  const void* fn;
  if (!whole) fn = f16 ? (const void*)&eql_ckpt_pack_kernel<_Float16, false, false> : (const void*)&eql_ckpt_pack_kernel<float, false, false>;
  else if (stream) fn = f16 ? (const void*)&eql_ckpt_pack_kernel<_Float16, true, true> : (const void*)&eql_ckpt_pack_kernel<float, true, true>;
  else fn = f16 ? (const void*)&eql_ckpt_pack_kernel<_Float16, true, false> : (const void*)&eql_ckpt_pack_kernel<float, true, false>;
  return launch_kernel(fn, grid, a, s);
}

hipError_t launch_ckpt_unpack(bool f16, bool stream, const CkptArgs& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  return launch_kernel(EQL_PICK(eql_ckpt_unpack_kernel), grid, a, s);
}

hipError_t launch_epi8(bool f16, bool stream, const Epi8Args& a, unsigned grid, hipStream_t s) {
  const bool whole = a.R % 8 == 0;
  return launch_kernel(EQL_PICK(eql_epi8_kernel), grid, a, s, kEpi8Threads);
}

}  // namespace eql
