// Weight-gradient GEMM instantiations (complex pairs), f32 element type, T = 1..16.
#include "eql_launch.h"

namespace eql {

template <int T>
static hipError_t gemm_one(int DB, int CB, int WCN, const BwdwArgs& a, unsigned grid, hipStream_t s) {
  if constexpr (n_pairs(T) == 0) {
    return hipErrorInvalidValue;
  } else {
    if (DB == 4 && CB == 2 && WCN == 2) return launch_kernel((const void*)&eql_bwdw_gemm<T, float, true, 4, 2, 2>, grid, a, s);
    if (DB == 4 && CB == 1 && WCN == 4) return launch_kernel((const void*)&eql_bwdw_gemm<T, float, true, 4, 1, 4>, grid, a, s, 512);
    if (DB == 4 && CB == 1 && WCN == 2) return launch_kernel((const void*)&eql_bwdw_gemm<T, float, true, 4, 1, 2>, grid, a, s);
    if (DB == 1 && CB == 2 && WCN == 2) return launch_kernel((const void*)&eql_bwdw_gemm<T, float, true, 1, 2, 2>, grid, a, s);
    if (DB == 1 && CB == 1 && WCN == 2) return launch_kernel((const void*)&eql_bwdw_gemm<T, float, true, 1, 1, 2>, grid, a, s);
    return hipErrorInvalidValue;
  }
}

hipError_t launch_bwdw_pair_f32(int T, int DB, int CB, int WCN, const BwdwArgs& a, unsigned grid, hipStream_t s) {
#define EQL_CASE(t) return gemm_one<t>(DB, CB, WCN, a, grid, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

template <int T>
static hipError_t both_one(const BwdwArgs& pair, const BwdwArgs& real, hipStream_t s) {
  if constexpr (n_pairs(T) == 0) {
    return hipErrorInvalidValue;
  } else {
    void* kargs[] = {const_cast<BwdwArgs*>(&pair), const_cast<BwdwArgs*>(&real)};
    return hipLaunchKernel((const void*)&eql_bwdw_gemm_both<T, float>, dim3((unsigned)(pair.numItems + real.numItems)),
                           dim3(256), kargs, 0, s);
  }
}

hipError_t launch_bwdw_both_f32(int T, const BwdwArgs& pair, const BwdwArgs& real, hipStream_t s) {
#define EQL_CASE(t) return both_one<t>(pair, real, s);
  EQL_FOR_EACH_T(T, EQL_CASE)
#undef EQL_CASE
}

}  // namespace eql
