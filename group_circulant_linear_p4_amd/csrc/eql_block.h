// Internal launch interface of the block operators (layer norm, 8-bit checkpoints): between
// eql_block_api.hip and the kernel instantiations, and what it shares with eql_api.hip.
#pragma once

#include "eql_launch.h"
#include "eql_norm.h"

namespace eql {

// Rows that the register-resident norm kernels hold (features), forward and backward.
constexpr int kNormFwdMaxRow = 16384;
constexpr int kNormBwdMaxRow = 8192;

// Lanes per row of the register-resident norm kernels and chunks per lane, for rows of `chunks`
// 8-feature chunks.  A whole wave for a row from 33 chunks on: at N = 16384, R = 512 fp32 one
// chunk on each of 64 lanes takes 25 us backward where four on each of 16 take 29, and at N =
// 197, R = 384 fp16 3.3 us forward where three on each of 16 take 4.4.
struct NormShape {
  int lpr, k;
};
constexpr NormShape norm_shape(int64_t chunks) {
  const int lpr = chunks <= 32 ? 16 : (chunks <= 64 * 4 ? 64 : 256);
  const int k = (int)((chunks + lpr - 1) / lpr);
  return {lpr, k > 6 ? 8 : (k > 4 ? 6 : k)};
}

hipError_t launch_ckpt_pack(bool f16, bool stream, const CkptArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_ckpt_unpack(bool f16, bool stream, const CkptArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_epi8(bool f16, bool stream, const Epi8Args& a, unsigned grid, hipStream_t s);
hipError_t launch_spec8_f16(int T, int view, const Spec8Args& a, unsigned grid, hipStream_t s);
hipError_t launch_spec8_f32(int T, int view, const Spec8Args& a, unsigned grid, hipStream_t s);
hipError_t launch_norm_fwd(bool f16, bool stream, NormShape sh, const NormArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_norm_fwd_wide(bool f16, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(bool f16, bool stream, NormShape sh, bool ckpt, const NormArgs& a, unsigned grid, hipStream_t s);
hipError_t launch_norm_bwd_wide(bool f16, bool ckpt, const NormArgs& a, unsigned colGrid, hipStream_t s);
hipError_t launch_norm_param(bool f16, const NormParamArgs& a, hipStream_t s);

// Shared host code of eql_api.hip.
namespace host {

// EQL_OK, or the status that the sizes deserve.
int check_sizes(int64_t N, int64_t Cp, int64_t Dp, int T, int dtype);

// Launch shape of the epilogue backward (rows per partial sum and their bytes).
void epilogue_rows(int64_t N, int64_t Dp, int T, int dtype, int64_t* rowsPerBlock, int64_t* rowBlocks, size_t* partBytes);

// The layer's input as a checkpoint and how to read it: act(gamma[c] value + beta[c]).
struct CkptView {
  const void* ckpt;
  const void* gamma;
  const void* beta;
  int act;
};

// The weight gradient from dy and the checkpointed input (eqlinear_bwd_w's plan and checks).
int bwd_w_from_ckpt(const CkptView& view, const void* dy, void* dw, void* workspace, size_t ws_bytes, int64_t N,
                    int64_t Cp, int64_t Dp, int T, int dtype, void* stream);
// Only the checkpointed input's spectrum, into its section of the weight-gradient workspace.
int spectrum_from_ckpt(const CkptView& view, void* workspace, size_t ws_bytes, int64_t N, int64_t Cp, int64_t Dp, int T,
                       int dtype, void* stream);

}  // namespace host

}  // namespace eql
