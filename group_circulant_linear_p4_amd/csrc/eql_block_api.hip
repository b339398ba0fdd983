// C ABI of the block operators (include/eqlinear_block.h, include/eqlinear_rmsnorm.h): argument checks, launch
// shapes and launches on the caller's stream.  Nothing here allocates device memory or
// synchronises the host.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <numeric>

#include "eql_block.h"
#include "eqlinear_block.h"
#include "eqlinear_rmsnorm.h"

using namespace eql;

namespace {

constexpr int64_t kMaxGrid = (1LL << 24) - 1;  // workgroups of 256 threads per launch

int elt_bytes(int dtype) { return dtype == EQL_F16 ? 2 : 4; }
bool off(const void* p, uintptr_t to) { return p && reinterpret_cast<uintptr_t>(p) % to != 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int status_of(hipError_t e) { return e == hipSuccess ? EQL_OK : EQL_EHIP; }

// Passes that move more than the last-level cache holds (256 MB) read their operands past the
// caches; smaller ones often find them there.
bool streams(int64_t bytes) { return bytes > (256LL << 20); }

// Workgroups of 1024 threads that the GELU backward aims at: one per compute unit.  More do not
// read faster (N = 12608, R = 1536 fp16: 20.4 us with 256, 20.3 with 512; N = 65536, R = 4096: 242 and
// 252) and leave more partial sums to add.
constexpr int64_t kEpi8Workgroups = 256;

// Workgroups for `turns` turns of a grid-stride loop: at most `most`, all with the same number
// of turns or one less.
int64_t even_grid(int64_t turns, int64_t most) { return ceil_div(turns, ceil_div(turns, most)); }

// Forward: two turns or more once every compute unit has four workgroups (the first turn's loads
// then hide the parameters', the second's its own), and otherwise many workgroups, which visit
// memory nearly in order: N = 65536, R = 4096 fp16 takes 175-186 us in 8192 to 16384 workgroups and 195
// in 1024; N = 12608, R = 384 takes 8.0 us in two turns and 9.5 in one.
int64_t norm_fwd_grid(int64_t turns) { return even_grid(turns, std::clamp<int64_t>(turns / 2, 1024, 8192)); }
// Backward: as few as keep the memory busy, since each leaves two sums a channel to add: N =
// 65536, R = 4096 fp16 takes 318 us in 512 workgroups, 359 in 256 and 373 in 768; N = 16384, R =
// 512 fp32 25 us in 256 to 768.
// One for up to three turns: it writes the parameters' gradients itself, which saves a launch
// (14 rows of R = 56 fp16: 12.6 -> 10.7 us for both passes).
int64_t norm_bwd_grid(int64_t turns) { return turns <= 3 ? 1 : even_grid(turns, 512); }

// Launch shape of the norm's backward.  wide: rows longer than the registers hold.
struct BwdPlan {
  bool wide = false;
  NormShape shape{};
  int64_t grid = 0;                                   // register path; also the blocks of column sums
  int64_t colBlocks = 0, rowsPerBlock = 0, rowBlocks = 0;  // wide path
  size_t rowBytes = 0, partBytes = 0;
  size_t total() const { return rowBytes + partBytes; }
};

// kinds: column sums a feature (the layer norm's weight and bias, the RMS norm's weight).
BwdPlan plan_norm_bwd(int64_t N, int64_t Cp, int T, int kinds) {
  BwdPlan p;
  if (N == 0) return p;
  const int64_t R = Cp * T;
  if (R <= kNormBwdMaxRow) {
    p.shape = norm_shape(ceil_div(R, 8));
    p.grid = norm_bwd_grid(ceil_div(N, 256 / p.shape.lpr));
    p.partBytes = (size_t)p.grid * kinds * (size_t)Cp * sizeof(float);
    return p;
  }
  p.wide = true;
  p.colBlocks = ceil_div(R, 2048);
  p.rowsPerBlock = 256;
  while (p.rowsPerBlock > 1 && ceil_div(N, p.rowsPerBlock) * p.colBlocks < 1024) p.rowsPerBlock /= 2;
  p.rowBlocks = ceil_div(N, p.rowsPerBlock);
  p.rowBytes = ((size_t)N * 2 * sizeof(float) + 255) / 256 * 256;
  p.partBytes = (size_t)p.rowBlocks * kinds * (size_t)R * sizeof(float);
  return p;
}

void set_ckpt(NormArgs& a, const void* ckpt) {
  a.codes = static_cast<unsigned char*>(const_cast<void*>(ckpt));
  a.scales = a.codes ? a.codes + a.N * a.pitch : nullptr;
}

NormArgs norm_args(int64_t N, int64_t Cp, int T) {
  NormArgs a{};
  a.N = N;
  a.C = (int)Cp;
  a.T = T;
  a.R = (int)(Cp * T);
  a.pitch = (int)ckpt_pitch(a.R);
  a.perT = T > 1 ? (uint32_t)(((1ULL << 32) + T - 1) / T) : 0;
  a.invR = (float)(1.0 / (double)a.R);
  return a;
}

// What a norm's backward pass reads beside dy: x and the layer norm's mean, its checkpoint, or x alone.
enum class From { kMean, kCkpt, kRms };

// The backward entry points of both norms.
int norm_bwd(From from, const void* dy, const void* x, const void* ckpt, const float* mean, const float* rstd,
             const void* gamma, const void* dres, void* dx, void* dgamma, void* dbeta, void* workspace, size_t ws_bytes,
             int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  const int st = host::check_sizes(N, Cp, 1, T, dtype);
  if (st != EQL_OK) return st;
  const bool fromCkpt = from == From::kCkpt, rms = from == From::kRms;
  const BwdPlan p = plan_norm_bwd(N, Cp, T, rms ? 1 : 2);
  const bool params = dgamma || dbeta;
  if (N > 0) {
    if (!dy || !dx || !rstd || (fromCkpt ? !ckpt : (!x || (!rms && !mean)))) return EQL_EINVAL;
    // The wide path keeps its row means in the workspace, the others only parameter sums.
    const size_t need = params ? p.total() : p.rowBytes;
    if (need && (!workspace || ws_bytes < need)) return EQL_EINVAL;
    if (p.wide && (N > kMaxGrid / 4 || p.rowBlocks * p.colBlocks > kMaxGrid)) return EQL_EINVAL;
  }
  const uintptr_t elt = (uintptr_t)elt_bytes(dtype);
  if (off(dy, 16) || off(x, 16) || off(ckpt, 16) || off(dres, 16) || off(dx, 16) || off(workspace, 16) || off(mean, 4) ||
      off(rstd, 4) || off(gamma, elt) || off(dgamma, elt) || off(dbeta, elt))
    return EQL_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == EQL_F16;
  NormArgs a = norm_args(N, Cp, T);
  a.dy = dy;
  a.x = x;
  set_ckpt(a, ckpt);
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.gamma = gamma;
  a.dres = dres;
  a.dx = dx;
  if (N > 0) {
    char* ws = static_cast<char*>(workspace);
    const bool direct = params && !p.wide && p.grid == 1;
    a.part = params && !direct ? reinterpret_cast<float*>(ws + p.rowBytes) : nullptr;
    a.dgamma = direct ? dgamma : nullptr;
    a.dbeta = direct ? dbeta : nullptr;
    a.table = !p.wide && norm_table(p.shape.lpr, a.R, T, elt_bytes(dtype), 1);
    hipError_t e;
    if (p.wide) {
      a.rowSums = reinterpret_cast<float*>(ws);
      a.colBlocks = (int)p.colBlocks;
      a.rowsPerBlock = (int)p.rowsPerBlock;
      const unsigned grid = (unsigned)(p.rowBlocks * p.colBlocks);
      e = rms ? launch_rms_bwd_wide(f16, a, grid, s) : launch_norm_bwd_wide(f16, fromCkpt, a, grid, s);
    } else {
      const int64_t moved = elt_bytes(dtype) * (2 + (dres ? 1 : 0)) + (fromCkpt ? 1 : elt_bytes(dtype));
      const bool stream_in = streams(N * (int64_t)a.R * moved);
      e = rms ? launch_rms_bwd(f16, stream_in, p.shape, a, (unsigned)p.grid, s)
              : launch_norm_bwd(f16, stream_in, p.shape, fromCkpt, a, (unsigned)p.grid, s);
    }
    if (e != hipSuccess) return EQL_EHIP;
    if (direct) return EQL_OK;
  }
  if (!params) return EQL_OK;
  NormParamArgs q{};
  q.part = a.part;
  q.dgamma = dgamma;
  q.dbeta = dbeta;
  q.blocks = (int)(p.wide ? p.rowBlocks : p.grid);  // 0 without rows: zero gradients
  q.C = (int)Cp;
  q.F = p.wide ? T : 1;
  q.groups = (int)ceil_div(Cp, 16);
  q.blockStride = (rms ? 1 : 2) * Cp * q.F;
  return status_of(launch_norm_param(f16, q, s));
}

// Pack and unpack.
int ckpt_copy(bool pack, const void* x, const void* ckpt, int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  const int st = host::check_sizes(N, Cp, 1, T, dtype);
  if (st != EQL_OK) return st;
  if (N == 0) return EQL_OK;
  if (!x || !ckpt) return EQL_EINVAL;
  if (off(x, 16) || off(ckpt, 16)) return EQL_EALIGN;
  CkptArgs a{};
  a.R = (int)(Cp * T);
  const int64_t pitch = ckpt_pitch(a.R);
  a.rowChunks = (int)(pitch / 8);
  a.chunks = N * a.rowChunks;
  a.x = x;
  a.codes = static_cast<unsigned char*>(const_cast<void*>(ckpt));
  a.scales = a.codes + N * pitch;
  const int64_t grid = ceil_div(a.chunks, 256);
  if (grid > kMaxGrid) return EQL_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool stream_in = streams(N * (int64_t)a.R * (elt_bytes(dtype) + 1));
  return status_of(pack ? launch_ckpt_pack(dtype == EQL_F16, stream_in, a, (unsigned)grid, s)
                        : launch_ckpt_unpack(dtype == EQL_F16, stream_in, a, (unsigned)grid, s));
}

}  // namespace

extern "C" {

int eqlinear_block_abi_version(void) { return 100; }

int eqlinear_rmsnorm_abi_version(void) { return 100; }

size_t eqlinear_ckpt8_bytes(int64_t N, int64_t Cp, int T) {
  if (host::check_sizes(N, Cp, 1, T, EQL_F16) != EQL_OK) return 0;
  const size_t pitch = (size_t)ckpt_pitch(Cp * T);
  return (size_t)N * (pitch + pitch / kCkptBlock);
}

int eqlinear_ckpt8_pack(const void* x, void* ckpt, int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  return ckpt_copy(true, x, ckpt, N, Cp, T, dtype, stream);
}

int eqlinear_ckpt8_unpack(const void* ckpt, void* x, int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  return ckpt_copy(false, x, ckpt, N, Cp, T, dtype, stream);
}

int eqlinear_layernorm_fwd(const void* x, const void* gamma, const void* beta, void* y, void* ckpt, float* mean,
                           float* rstd, int64_t N, int64_t Cp, int T, float eps, int dtype, void* stream) {
  const int st = host::check_sizes(N, Cp, 1, T, dtype);
  if (st != EQL_OK) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return EQL_EINVAL;
  if (N == 0) return EQL_OK;
  if (!x || !y) return EQL_EINVAL;
  const uintptr_t elt = (uintptr_t)elt_bytes(dtype);
  if (off(x, 16) || off(y, 16) || off(ckpt, 16) || off(mean, 4) || off(rstd, 4) || off(gamma, elt) || off(beta, elt))
    return EQL_EALIGN;
  NormArgs a = norm_args(N, Cp, T);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  set_ckpt(a, ckpt);
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == EQL_F16;
  if (a.R > kNormFwdMaxRow) {
    if (N > kMaxGrid / 4) return EQL_EINVAL;
    return status_of(launch_norm_fwd_wide(f16, a, s));
  }
  const NormShape sh = norm_shape(a.pitch / 8);
  a.table = norm_table(sh.lpr, a.R, T, elt_bytes(dtype), 2);
  const int64_t grid = norm_fwd_grid(ceil_div(N, 256 / sh.lpr));
  return status_of(launch_norm_fwd(f16, streams(N * (int64_t)a.R * (2 * elt_bytes(dtype) + (ckpt ? 1 : 0))), sh, a, (unsigned)grid, s));
}

size_t eqlinear_layernorm_bwd_workspace_bytes(int64_t N, int64_t Cp, int T, int dtype) {
  if (host::check_sizes(N, Cp, 1, T, dtype) != EQL_OK) return 0;
  return plan_norm_bwd(N, Cp, T, 2).total();
}

int eqlinear_layernorm_bwd(const void* dy, const void* x, const float* mean, const float* rstd, const void* gamma,
                           const void* dres, void* dx, void* dgamma, void* dbeta, void* workspace, size_t ws_bytes,
                           int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  return norm_bwd(From::kMean, dy, x, nullptr, mean, rstd, gamma, dres, dx, dgamma, dbeta, workspace, ws_bytes, N, Cp, T,
                  dtype, stream);
}

int eqlinear_layernorm_bwd_ckpt8(const void* dy, const void* ckpt, const float* rstd, const void* gamma,
                                 const void* dres, void* dx, void* dgamma, void* dbeta, void* workspace,
                                 size_t ws_bytes, int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  return norm_bwd(From::kCkpt, dy, nullptr, ckpt, nullptr, rstd, gamma, dres, dx, dgamma, dbeta, workspace, ws_bytes, N, Cp, T,
                  dtype, stream);
}

int eqlinear_rmsnorm_fwd(const void* x, const void* residual, const void* gamma, void* sum, void* y, float* rstd, int64_t N,
                         int64_t Cp, int T, float eps, int dtype, void* stream) {
  const int st = host::check_sizes(N, Cp, 1, T, dtype);
  if (st != EQL_OK) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return EQL_EINVAL;
  if (N == 0) return EQL_OK;
  if (!x || !y || sum == y) return EQL_EINVAL;
  if (off(x, 16) || off(residual, 16) || off(sum, 16) || off(y, 16) || off(rstd, 4) || off(gamma, (uintptr_t)elt_bytes(dtype)))
    return EQL_EALIGN;
  NormArgs a = norm_args(N, Cp, T);
  a.x = x;
  a.res = residual;
  a.gamma = gamma;
  a.sum = sum;
  a.y = y;
  a.rstd = rstd;
  a.eps = eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == EQL_F16;
  if (a.R > kNormFwdMaxRow) {
    if (N > kMaxGrid / 4) return EQL_EINVAL;
    return status_of(launch_rms_fwd_wide(f16, a, s));
  }
  const NormShape sh = norm_shape(ceil_div(a.R, 8));
  a.table = norm_table(sh.lpr, a.R, T, elt_bytes(dtype), 1);
  const int64_t grid = norm_fwd_grid(ceil_div(N, 256 / sh.lpr));
  const int64_t moved = elt_bytes(dtype) * (2 + (residual ? 1 : 0) + (sum ? 1 : 0));
  return status_of(launch_rms_fwd(f16, streams(N * (int64_t)a.R * moved), sh, a, (unsigned)grid, s));
}

size_t eqlinear_rmsnorm_bwd_workspace_bytes(int64_t N, int64_t Cp, int T, int dtype) {
  if (host::check_sizes(N, Cp, 1, T, dtype) != EQL_OK) return 0;
  return plan_norm_bwd(N, Cp, T, 1).total();
}

int eqlinear_rmsnorm_bwd(const void* dy, const void* sum, const float* rstd, const void* gamma, const void* dres, void* dx,
                         void* dgamma, void* workspace, size_t ws_bytes, int64_t N, int64_t Cp, int T, int dtype,
                         void* stream) {
  return norm_bwd(From::kRms, dy, sum, nullptr, nullptr, rstd, gamma, dres, dx, dgamma, nullptr, workspace, ws_bytes, N, Cp,
                  T, dtype, stream);
}

int eqlinear_fused_epilogue_bwd_ckpt8(const void* dy, const void* pre_ckpt, void* dpre, void* dbias, void* workspace,
                                      size_t ws_bytes, int64_t N, int64_t Dp, int T, int dtype, void* stream) {
  const int st = host::check_sizes(N, 1, Dp, T, dtype);
  if (st != EQL_OK) return st;
  int64_t rowsPerBlock = 0, rowBlocks = 0;
  size_t partBytes = 0;
  host::epilogue_rows(N, Dp, T, dtype, &rowsPerBlock, &rowBlocks, &partBytes);
  const bool parts = dbias && N > 0;
  if (N > 0 && (!dy || !pre_ckpt || !dpre)) return EQL_EINVAL;
  if (parts && (!workspace || ws_bytes < partBytes)) return EQL_EINVAL;
  if (off(dy, 16) || off(pre_ckpt, 16) || off(dpre, 16) || off(workspace, 16) || off(dbias, (uintptr_t)elt_bytes(dtype)))
    return EQL_EALIGN;
  Epi8Args a{};
  a.R = (int)(Dp * T);
  a.pitch = (int)ckpt_pitch(a.R);
  a.N = N;
  a.dy = dy;
  a.dpre = dpre;
  a.codes = static_cast<const unsigned char*>(pre_ckpt);
  a.scales = a.codes ? a.codes + N * a.pitch : nullptr;
  a.T = T;
  // Up to 32 rows are one row block, whose workgroups write the bias gradient themselves: one
  // launch instead of two (9 rows of 240 fp32: 8.4 -> 5.6 us; 64 rows of 3600 would take 9.4 in one
  // and 7.8 in two).
  if (N <= 32) rowsPerBlock = 32;
  rowBlocks = ceil_div(N, rowsPerBlock);
  // Chunks across a workgroup: the row's chunks spread evenly over column blocks, which leaves room
  // for 1024 / lanes rows at a time.  As few column blocks as hold the row, or more (down to 32
  // lanes) until there is a workgroup per compute unit; then row blocks as tall as keep it so,
  // each leaving one sum a channel to add (and no more of them than the workspace is sized for).
  const int64_t chunks = ceil_div(a.R, 8);
  int64_t colBlocks = ceil_div(chunks, kEpi8Threads);
  while (rowBlocks * colBlocks < kEpi8Workgroups && ceil_div(chunks, 2 * colBlocks) >= 32) colBlocks *= 2;
  // Whole channels in each: they add a channel's T features themselves, T times fewer partial sums
  // for the second launch (5003 rows of 513, T = 3 fp16: 12.5 -> 10.3 us).
  const int64_t whole = colBlocks == 1 ? 1 : T / std::gcd(T, 8);
  a.lanes = (int)std::min(ceil_div(ceil_div(chunks, colBlocks), whole), kEpi8Threads / whole) * (int)whole;
  a.colBlocks = (int)ceil_div(chunks, a.lanes);
  rowsPerBlock = std::max(rowsPerBlock, ceil_div(N, std::max<int64_t>(1, kEpi8Workgroups / a.colBlocks)));
  rowBlocks = ceil_div(N, rowsPerBlock);
  const bool direct = parts && rowBlocks == 1;
  a.part = parts && !direct ? static_cast<float*>(workspace) : nullptr;
  a.dbias = direct ? dbias : nullptr;
  a.groups = (int)std::min<int64_t>(kEpi8Threads / a.lanes, rowsPerBlock);
  a.rowsPerBlock = (int)rowsPerBlock;
  if (rowBlocks * a.colBlocks > kMaxGrid / 4) return EQL_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == EQL_F16;
  if (N > 0 && launch_epi8(f16, streams(N * (int64_t)a.R * (2 * elt_bytes(dtype) + 1)), a, (unsigned)(rowBlocks * a.colBlocks), s) != hipSuccess) return EQL_EHIP;
  if (!dbias || direct) return EQL_OK;
  NormParamArgs q{};
  q.part = a.part;
  q.dgamma = dbias;
  q.blocks = N > 0 ? (int)rowBlocks : 0;  // 0 without rows: a zero gradient
  q.C = (int)Dp;
  q.F = 1;
  q.groups = (int)ceil_div(Dp, 16);
  q.blockStride = Dp;
  return status_of(launch_norm_param(f16, q, s));
}

int eqlinear_ckpt8_spectrum(const void* ckpt, const void* gamma, const void* beta, int act, void* workspace,
                            size_t ws_bytes, int64_t N, int64_t Cp, int64_t Dp, int T, int dtype, void* stream) {
  return host::spectrum_from_ckpt({ckpt, gamma, beta, act}, workspace, ws_bytes, N, Cp, Dp, T, dtype, stream);
}

int eqlinear_bwd_w_ckpt8(const void* ckpt, const void* gamma, const void* beta, int act, const void* dy, void* dw,
                         void* workspace, size_t ws_bytes, int64_t N, int64_t Cp, int64_t Dp, int T, int dtype,
                         void* stream) {
  return host::bwd_w_from_ckpt({ckpt, gamma, beta, act}, dy, dw, workspace, ws_bytes, N, Cp, Dp, T, dtype, stream);
}

}  // extern "C"
