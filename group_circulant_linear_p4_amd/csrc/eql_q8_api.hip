// C ABI of the layer in 8-bit integers (declared in include/eqlinear_q8.h): argument checks, launch
// shapes and launches on the caller's stream.  Nothing here allocates device memory or synchronises
// the host.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "eql_q8_launch.h"
#include "eqlinear_q8.h"

using namespace eql;

namespace {

constexpr int64_t kMaxGrid = (1LL << 24) - 1;  // workgroups of 256 threads per launch
constexpr int64_t kMaxC = 65536;               // channels whose products' sums fit 32 bits

int elt_bytes(int dtype) { return dtype == EQL_F16 ? 2 : 4; }
bool off(const void* p, uintptr_t to) { return p && reinterpret_cast<uintptr_t>(p) % to != 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int status_of(hipError_t e) { return e == hipSuccess ? EQL_OK : EQL_EHIP; }

int check(int64_t N, int64_t Cp, int64_t Dp, int T, int dtype) {
  const int st = host::check_sizes(N, Cp, Dp, T, dtype);
  if (st != EQL_OK) return st;
  return Cp > kMaxC ? EQL_EUNSUPPORTED : EQL_OK;
}

size_t row_codes(int64_t N, int64_t Cp, int T) { return (size_t)N * (size_t)T * (size_t)q8_pitch(Cp); }
size_t weight_codes(int64_t Dp, int64_t Cp, int T) { return (size_t)(q8_out(Dp) / 32 * q8_blocks(Cp)) * (size_t)T * 2048; }

// Which kernel a product takes (fp16, rows of input -> output channels).  Up to four rows the token kernel, but for long
// sums of T = 1, where the small one reads the weight faster (4 rows of 4096 -> 4096: 9.2 us and 5.1, of 4096 -> 1024: 6.1
// and 5.0; one row the same).  For T > 1 it is the shorter one at every T of 2, 3, 4, 5, 8, 12 and 16 with 256 to 4096 -> 1024
// channels (one row of 4096: 3.6 us and 6.2 at T = 2, 4.5 and 10.3 at T = 4, 16.0 and 120 at T = 16; four rows 5.7 and 6.9, 8.8 and
// 11.5, 35.7 and 122) and level or shorter with 1024 -> 4096 but for T = 12 (two rows 16.7 and 15.0, four 22.8 and 15.3).
// The small one splits the input channels of each of its 32 x 32 tiles over eight waves and is the shorter while every
// tile has a compute unit and the sums are long: T = 4, 256 rows of 1024 -> 1024, 256 tiles: 8.5 us and the medium tile's 10.7, of
// 4096 -> 1024: 24.7 and 33.5; 500 rows, 512 tiles: 14.0 and 11.1.  T = 1, 500 rows of 4096 -> 1024, 512 tiles: 12.1 and 17.7;
// 1000 rows, 1024 tiles: 21.9 and 18.8.  (Where it is not, the rule does not follow: T = 4, 64 to 500 rows of 96 -> 384: 5.2 and 4.3;
// T = 8, 64 to 1000 rows of 256 -> 256: 8.7 to 11.1 and 7.8 to 8.1.)
// The big tile reads the operands least, once it has a tile for most compute units: T = 4, 12608 rows of 384 -> 96, 197
// tiles: 10.8 us and the medium one's 11.9; 1000 rows of 1024 -> 1024, 128 tiles: 15.0 and 12.2.  For T <= 2 it is 256
// channels wide instead of 128 and four workgroups of the medium one share a compute unit, so it needs long sums or many
// tiles (T = 1, 256 tiles of 1024 -> 1024: 11.6 us and 13.6, of 256 -> 1024: 8.5 and 7.4, 2048 of these: 38.1 and 43.9)
// and few channels past the last one (T = 2, 65536 rows of 384 -> 384: 53.5 and 44.5).  Where these rules are
// furthest off: T = 4, 256 rows of 1024 -> 4096 take 22.9 us on the medium tile and 15.5 on the big one; T = 1, 4096 rows of
// 1024 -> 1024 fp32 take 8.8 with the narrower medium tile, 8.5 with the wider one.
Q8Kind product_kind(int64_t N, int64_t Cp, int64_t Dp, int T) {
  if (N <= kQ8Tokens) return T > 1 || N * Cp <= 4096 ? Q8Kind::kToken : Q8Kind::kSmall;
  if (T > kQ8LargeT || ceil_div(N, 32) * ceil_div(Dp, 32) <= (T == 1 ? 512 : 256)) return Q8Kind::kSmall;
  const Q8Tile b = q8_tile(T, true);
  const int64_t tiles = ceil_div(N, 32 * b.mb) * ceil_div(Dp, 128 * b.nb);
  if (T > 2) return tiles >= 192 ? Q8Kind::kBig : Q8Kind::kMedium;
  const bool filled = ceil_div(Dp, 128) % 2 == 0 || Dp > 1024;
  return filled && tiles >= (q8_blocks(Cp) >= 8 ? 256 : 1024) ? Q8Kind::kBig : Q8Kind::kMedium;
}

// Both entry points that write rows.
int write_rows(bool norm, const void* x, const void* res, const void* gamma, void* sum, void* rows8, int64_t N, int64_t Cp,
               int T, float eps, int dtype, void* stream) {
  const int st = check(N, Cp, 1, T, dtype);
  if (st != EQL_OK) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return EQL_EINVAL;
  if (N == 0) return EQL_OK;
  if (!x || !rows8) return EQL_EINVAL;
  if (off(x, 16) || off(res, 16) || off(sum, 16) || off(rows8, 16) || off(gamma, (uintptr_t)elt_bytes(dtype))) return EQL_EALIGN;
  Q8RowsArgs a{};
  a.x = x;
  a.res = res;
  a.gamma = gamma;
  a.sum = sum;
  a.codes = static_cast<unsigned char*>(rows8);
  a.scales = reinterpret_cast<float*>(a.codes + row_codes(N, Cp, T));
  a.N = N;
  a.C = (int)Cp;
  a.pitch = (int)q8_pitch(Cp);
  a.norm = norm;
  a.eps = eps;
  a.invR = (float)(1.0 / (double)(Cp * T));
  a.tw = host::twiddles(T);
  const NormShape sh = q8_shape(Cp, T, elt_bytes(dtype), N);
  int64_t grid = N;
  if (sh.k) grid = std::min(ceil_div(N, 256 / sh.lpr), kMaxGrid);
  else if (N > kMaxGrid) return EQL_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(dtype == EQL_F16 ? launch_q8_rows_f16(T, sh, a, (unsigned)grid, s) : launch_q8_rows_f32(T, sh, a, (unsigned)grid, s));
}

}  // namespace

extern "C" {

int eqlinear_q8_abi_version(void) { return 100; }

size_t eqlinear_q8_rows_bytes(int64_t N, int64_t Cp, int T) {
  if (check(N, Cp, 1, T, EQL_F16) != EQL_OK) return 0;
  return row_codes(N, Cp, T) + (size_t)N * n_freqs(T) * sizeof(float);
}

size_t eqlinear_q8_weight_bytes(int64_t Dp, int64_t Cp, int T) {
  if (check(0, Cp, Dp, T, EQL_F16) != EQL_OK) return 0;
  return weight_codes(Dp, Cp, T) + (size_t)q8_out(Dp) * n_freqs(T) * sizeof(float);
}

int eqlinear_q8_pack_weight(const void* w, void* w8, int64_t Dp, int64_t Cp, int T, int dtype, void* stream) {
  const int st = check(0, Cp, Dp, T, dtype);
  if (st != EQL_OK) return st;
  if (!w || !w8) return EQL_EINVAL;
  if (off(w, 16) || off(w8, 16)) return EQL_EALIGN;
  Q8PackArgs a{};
  a.w = w;
  a.codes = static_cast<unsigned char*>(w8);
  a.scales = reinterpret_cast<float*>(a.codes + weight_codes(Dp, Cp, T));
  a.D = (int)Dp;
  a.C = (int)Cp;
  a.Dpad = (int)q8_out(Dp);
  a.kblocks = (int)q8_blocks(Cp);
  a.tw = host::twiddles(T);
  return status_of(launch_q8_pack(dtype == EQL_F16, T, a, static_cast<hipStream_t>(stream)));
}

int eqlinear_q8_quantize(const void* x, void* rows8, int64_t N, int64_t Cp, int T, int dtype, void* stream) {
  return write_rows(false, x, nullptr, nullptr, nullptr, rows8, N, Cp, T, 0.0f, dtype, stream);
}

int eqlinear_q8_rmsnorm(const void* x, const void* residual, const void* gamma, void* sum, void* rows8, int64_t N,
                        int64_t Cp, int T, float eps, int dtype, void* stream) {
  return write_rows(true, x, residual, gamma, sum, rows8, N, Cp, T, eps, dtype, stream);
}

int eqlinear_q8_fwd(const void* rows8, const void* w8, const void* bias, const void* residual, void* y, int64_t N,
                    int64_t Cp, int64_t Dp, int T, int dtype, int act, void* stream) {
  const int st = check(N, Cp, Dp, T, dtype);
  if (st != EQL_OK) return st;
  if (act != EQL_ACT_NONE && act != EQL_ACT_GELU) return EQL_EINVAL;
  if (N == 0) return EQL_OK;
  if (!rows8 || !w8 || !y) return EQL_EINVAL;
  if (off(rows8, 16) || off(w8, 16) || off(y, 16) || off(residual, 16) || off(bias, (uintptr_t)elt_bytes(dtype))) return EQL_EALIGN;
  Q8FwdArgs a{};
  a.f.y = y;
  a.f.N = (int)N;
  a.f.Dout = (int)Dp;
  a.f.tw = host::twiddles(T);
  a.f.bias = bias;
  a.f.res = residual;
  a.f.act = act;
  a.codes = static_cast<const unsigned char*>(rows8);
  a.rowScales = reinterpret_cast<const float*>(a.codes + row_codes(N, Cp, T));
  a.w = static_cast<const unsigned char*>(w8);
  a.wScales = reinterpret_cast<const float*>(a.w + weight_codes(Dp, Cp, T));
  a.pitch = (int)q8_pitch(Cp);
  a.kblocks = (int)q8_blocks(Cp);
  a.Dpad = (int)q8_out(Dp);
  const Q8Kind kind = product_kind(N, Cp, Dp, T);
  const Q8Tile tile = q8_tile(T, kind == Q8Kind::kBig);
  const bool small = kind == Q8Kind::kSmall, token = kind == Q8Kind::kToken;
  const int64_t rowTiles = token ? 1 : ceil_div(N, small ? 32 : 32 * tile.mb);
  const int64_t colTiles = ceil_div(Dp, token ? 8 : (small ? 32 : 128 * tile.nb));
  const int64_t grid = rowTiles * colTiles;
  if (grid > kMaxGrid) return EQL_EINVAL;  // 512 threads only in grids of up to 256
  a.colTiles = (int)colTiles;
  // Eight waves a tile while there is a compute unit for each (32 rows of 1024 -> 1024 channels: 5.9 us, with four 6.2),
  // else four (300 rows: 15.8 and 13.7).
  a.waves = (int)std::min<int64_t>(grid <= 256 ? q8_waves(T) : 4, ceil_div(a.pitch, 32));
  hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(dtype == EQL_F16 ? launch_q8_fwd_f16(T, kind, a, (unsigned)grid, s) : launch_q8_fwd_f32(T, kind, a, (unsigned)grid, s));
}

}  // extern "C"
