// Host-code check of include/eqlinear_block.h, built with the sanitizers by
// test_block_abi_sanitized.py: every entry point with invalid arguments, with N = 0 and with the
// largest sizes the ABI accepts.  Nothing is launched and no pointer is dereferenced: each call
// fails a check or has nothing to do.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "eqlinear_block.h"

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
  float *m = static_cast<float*>(at(0x60000)), *r = static_cast<float*>(at(0x70000));
  void* ws = at(0x80000);
  CHECK(eqlinear_block_abi_version() == 100);
  for (int dt : {EQL_F16, EQL_F32})
    for (int64_t v : big) {
      // Row counts and channel counts far outside the range, alone and together.
      for (int which = 0; which < 3; ++which) {
        const int64_t N = which == 1 ? 8 : v, C = which == 0 ? 4 : v, D = which == 0 ? 4 : v;
        CHECK(eqlinear_ckpt8_bytes(N, C, 4) == 0);
        CHECK(eqlinear_layernorm_bwd_workspace_bytes(N, C, 4, dt) == 0);
        CHECK(eqlinear_ckpt8_pack(a, b, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_ckpt8_unpack(a, b, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_layernorm_fwd(a, b, c, d, e, m, r, N, C, 4, 1e-5f, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_layernorm_bwd(a, b, m, r, c, d, e, a, b, ws, SIZE_MAX, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_layernorm_bwd_ckpt8(a, b, r, c, d, e, a, b, ws, SIZE_MAX, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_fused_epilogue_bwd_ckpt8(a, b, c, d, ws, SIZE_MAX, N, C, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_ckpt8_spectrum(a, b, c, EQL_ACT_NONE, ws, SIZE_MAX, N, C, D, 4, dt, nullptr) == EQL_EINVAL);
        CHECK(eqlinear_bwd_w_ckpt8(a, b, c, EQL_ACT_NONE, d, e, ws, SIZE_MAX, N, C, D, 4, dt, nullptr) == EQL_EINVAL);
      }
    }
  // The largest rows and row counts: sizes come out, a misaligned pointer is what is refused.
  const int64_t rows = ((int64_t)1 << 31) - ((int64_t)1 << 20), wide = ((int64_t)1 << 23) / 2;
  for (int T : {1, 2, 3, 4, 5, 7, 8, 12, 16}) {
    const int64_t C = wide / T;
    CHECK(eqlinear_ckpt8_bytes(rows, C, T) >= (size_t)rows * (size_t)(C * T));
    CHECK(eqlinear_layernorm_bwd_workspace_bytes(rows, C, T, EQL_F16) > 0);
    CHECK(eqlinear_layernorm_fwd(mis, b, c, d, e, m, r, rows, 64 / T, T, 0.0f, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_layernorm_fwd(a, b, c, d, e, m, r, rows, C, T, 0.0f, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_ckpt8_pack(a, b, rows, C, T, EQL_F16, nullptr) == EQL_EINVAL);
    const size_t need = eqlinear_layernorm_bwd_workspace_bytes(1000, C, T, EQL_F16);
    CHECK(eqlinear_layernorm_bwd_ckpt8(a, b, r, c, d, e, a, b, ws, need - 1, 1000, C, T, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_layernorm_bwd_ckpt8(mis, b, r, c, d, e, a, b, ws, need, 1000, C, T, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_layernorm_bwd_ckpt8(a, b, r, c, d, e, a, b, ws, SIZE_MAX, rows, C, T, EQL_F16, nullptr) == EQL_EINVAL);
    CHECK(eqlinear_fused_epilogue_bwd_ckpt8(mis, b, c, d, ws, SIZE_MAX, 1000, C, T, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_bwd_w_ckpt8(mis, b, c, EQL_ACT_GELU, d, e, ws, SIZE_MAX, 1000, 64, 64, T, EQL_F16, nullptr) == EQL_EALIGN);
    CHECK(eqlinear_ckpt8_spectrum(mis, b, c, EQL_ACT_GELU, ws, SIZE_MAX, 1000, 64, 64, T, EQL_F32, nullptr) == EQL_EALIGN);
  }
  for (float eps : {-1.0f, -0x1p-149f, (float)NAN, INFINITY, -INFINITY})
    CHECK(eqlinear_layernorm_fwd(a, b, c, d, e, m, r, 8, 4, 4, eps, EQL_F16, nullptr) == EQL_EINVAL);
  // Nothing to do.
  CHECK(eqlinear_ckpt8_pack(nullptr, nullptr, 0, 4, 4, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_ckpt8_unpack(nullptr, nullptr, 0, 4, 4, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_layernorm_fwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 4, 4, 0.0f, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_layernorm_bwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, 4, 4,
                               EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_fused_epilogue_bwd_ckpt8(nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, 4, 4, EQL_F16, nullptr) == EQL_OK);
  CHECK(eqlinear_ckpt8_spectrum(nullptr, nullptr, nullptr, EQL_ACT_NONE, nullptr, 0, 0, 4, 4, 4, EQL_F16, nullptr) == EQL_OK);
  std::printf("%d checks, %d failed\n", checks, failed);
  return failed ? 1 : 0;
}
