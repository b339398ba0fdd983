// Host-code check of include/eqlinear_rmsnorm.h and include/eqlinear_q8.h, built with the sanitizers by
// test_q8_abi_sanitized.py: every entry point with invalid arguments, with N = 0 and with the largest sizes
// the ABI accepts.  Nothing is launched and no pointer is dereferenced: each call fails a check or has
// nothing to do.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "eqlinear_q8.h"
#include "eqlinear_rmsnorm.h"

static int checks = 0, failed = 0;
#define CHECK(cond)                                           \
  do {                                                        \
    ++checks;                                                 \
    if (!(cond)) {                                            \
      ++failed;                                               \
      std::printf("line %d: %s\n", __LINE__, #cond);          \
    }                                                         \
  } while (0)

static void* at(uintptr_t a) { return reinterpret_cast<void*>(a); }

int main() {
  const int64_t big[] = {INT64_MIN, -1, INT64_MAX, INT64_MAX / 2, (int64_t)1 << 40, (int64_t)1 << 31};
  void *a = at(0x10000), *b = at(0x20000), *c = at(0x30000), *d = at(0x40000), *e = at(0x50000), *mis = at(0x10008);
  float* r = static_cast<float*>(at(0x70000));
  void* ws = at(0x80000);
  CHECK(eqlinear_rmsnorm_abi_version() == 100 && eqlinear_q8_abi_version() == 100);
  for (int dt : {EQL_F16, EQL_F32})
    for (int64_t v : big)
      for (int which = 0; which < 3; ++which) {
        const int64_t N = which == 1 ? 8 : v, C = which == 0 ? 4 : v, D = which == 0 ? 4 : v;
        CHECK(eqlinear_q8_rows_bytes(N, C, 4) == 0);
        CHECK(eqlinear_q8_weight_bytes(v, 4, 4) == 0 && eqlinear_q8_weight_bytes(4, v, 4) == 0);
        CHECK(eqlinear_rmsnorm_bwd_workspace_bytes(N, C, 4, dt) == 0);
        CHECK(eqlinear_rmsnorm_fwd(a, b, c, d, e, r, N, C, 4, 1e-5f, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_rmsnorm_bwd(a, b, r, c, d, e, a, ws, SIZE_MAX, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_q8_quantize(a, b, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_q8_rmsnorm(a, b, c, d, e, N, C, 4, 1e-5f, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_q8_pack_weight(a, b, v, 4, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_q8_pack_weight(a, b, 4, v, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_q8_fwd(a, b, c, d, e, N, C, D, 4, dt, EQL_ACT_NONE, nullptr) == EQL_EINVAL);
      }
  // The largest rows and row counts: sizes come out, a misaligned pointer is what is refused.
  const int64_t rows = ((int64_t)1 << 31) - ((int64_t)1 << 20), wide = ((int64_t)1 << 23) / 2;
  for (int T : {1, 2, 3, 4, 5, 7, 8, 12, 16}) {
    const int64_t C = wide / T < 65536 ? wide / T : 65536;
    CHECK(eqlinear_q8_rows_bytes(rows, C, T) >= (size_t)rows * (size_t)(C * T));
    CHECK(eqlinear_q8_weight_bytes(wide / T, C, T) >= (size_t)(wide / T) * (size_t)(C * T));
    CHECK(eqlinear_q8_weight_bytes(C, wide / T + 1, T) == 0);
    CHECK(eqlinear_rmsnorm_fwd(mis, b, c, d, e, r, rows, 64 / T, T, 0.0f, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_rmsnorm_fwd(a, b, c, d, e, r, rows, wide / T, T, 0.0f, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_q8_quantize(mis, b, rows, 64 / T, T, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_q8_quantize(a, b, rows, C, T, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_q8_rmsnorm(mis, b, c, d, e, 1000, C, T, 0.0f, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_q8_pack_weight(mis, b, wide / T, C, T, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_q8_fwd(mis, b, c, d, e, 1000, C, 64, T, EQL_F16, EQL_ACT_GELU, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_q8_fwd(a, b, c, d, e, rows, C, wide / T, T, EQL_F16, EQL_ACT_GELU, nullptr) == EQL_EINVAL);
    const size_t need = eqlinear_rmsnorm_bwd_workspace_bytes(1000, C, T, EQL_F16);
    CHECK(eqlinear_rmsnorm_bwd(a, b, r, c, d, e, a, ws, need - 1, 1000, C, T, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_rmsnorm_bwd(mis, b, r, c, d, e, a, ws, need, 1000, C, T, EQL_F16, nullptr) == EQL_EALIGN);
  }
  CHECK(eqlinear_q8_rows_bytes(4, 65537, 1) == 0 && eqlinear_q8_weight_bytes(4, 65537, 1) == 0);
  CHECK(eqlinear_q8_quantize(a, b, 4, 65537, 1, EQL_F16, nullptr) == EQL_EUNSUPPORTED);
  for (float eps : {-1.0f, -0x1p-149f, (float)NAN, INFINITY, -INFINITY}) {
    CHECK(eqlinear_rmsnorm_fwd(a, b, c, d, e, r, 8, 4, 4, eps, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_q8_rmsnorm(a, b, c, d, e, 8, 4, 4, eps, EQL_F16, nullptr) == EQL_EINVAL);
  }
  for (int act : {-1, 2, INT32_MAX, INT32_MIN}) CHECK(eqlinear_q8_fwd(a, b, c, d, e, 8, 4, 4, 4, EQL_F16, act, nullptr) == EQL_EINVAL);
  // Nothing to do.
  CHECK(eqlinear_rmsnorm_fwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 4, 4, 0.0f, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_rmsnorm_bwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, 4, 4, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_q8_quantize(nullptr, nullptr, 0, 4, 4, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_q8_rmsnorm(nullptr, nullptr, nullptr, nullptr, nullptr, 0, 4, 4, 0.0f, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_q8_fwd(nullptr, nullptr, nullptr, nullptr, nullptr, 0, 4, 4, 4, EQL_F16, EQL_ACT_NONE, nullptr) == EQL_OK);
  std::printf("%d checks, %d failed\n", checks, failed);
  return failed ? 1 : 0;
}
