// RMS norm of an equivariant block with the residual's addition, forward; its backward pass is the
// layer norm's without the means (eql_norm.h, RMS).
//     s = x + r, rounded to the element type;  rstd = 1 / sqrt(mean(s^2) + eps),  y = gamma[c] s rstd
// over rows of R = C'*T features, gamma one value per channel: the mean square is the whole row's, so
// the norm commutes with the group action.  The norm is of the rounded sum, which is what the
// residual stream keeps and the backward pass reads.
// Bound by memory, two reads and two writes; laid out as the layer norm (LPR lanes a row, K chunks of
// 8 features a lane, in registers between the sum of squares and the result): 65536 rows of 4096 fp16 in 384 us,
// 5.6 TB/s, and their backward pass in 357 us, 6.0 TB/s.
#pragma once

#include "eql_norm.h"

namespace eql {

template <typename Elt, int LPR, int K, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(256) eql_rms_fwd_kernel(const NormArgs a) {
  using V = typename Chunk<Elt>::V;
  constexpr int G = 256 / LPR;
  extern __shared__ __align__(16) float lds[];  // the weight's table, if there is one
  __shared__ float red[2][8];
  const int lane = (int)threadIdx.x % LPR, grp = (int)threadIdx.x / LPR;
  const int64_t step = (int64_t)gridDim.x * G;
  // The row after the one at work is loaded before it is needed.
  V next[K], nextR[K];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8, n = row < a.N ? a.R - f0 : 0;
      next[i] = load_chunk8<Elt, WHOLE, STREAM>(static_cast<const Elt*>(a.x) + row * a.R + f0, n);
      if (a.res) nextR[i] = load_chunk8<Elt, WHOLE, STREAM>(static_cast<const Elt*>(a.res) + row * a.R + f0, n);
    }
  };
  load((int64_t)blockIdx.x * G + grp);
  V gam[K];
  if (a.table) {
    Elt* table = reinterpret_cast<Elt*>(lds);
    fill_table(a, table, a.gamma, 1.0f);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i)
      gam[i] = *reinterpret_cast<const V*>(table + min((lane + i * LPR) * 8, norm_table_row(a.R) - 8));
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i) gam[i] = spread<Elt>(a, a.gamma, (lane + i * LPR) * 8, 1.0f);
  }
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * G; base < a.N; base += step) {
    const int64_t row = base + grp;
    const bool live = row < a.N;
    float v[K][8];
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
      if (a.res) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = (float)(Elt)((float)next[i][e] + (float)nextR[i][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = (float)next[i][e];
      }
      if (a.sum) store_chunk8<Elt, WHOLE>(static_cast<Elt*>(a.sum) + row * a.R + f0, live ? a.R - f0 : 0, v[i]);
      // Missing features are zero.
      float t = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) t = __builtin_fmaf(v[i][e], v[i][e], t);
      q[0] += t;
    }
    if (base + step < a.N) load(row + step);
    row_sums<LPR>(q, red[turn]);
    turn ^= 1;
    const float rstd = inv_sqrt(__builtin_fmaf(q[0], a.invR, a.eps));
    if (live && lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = v[i][e] * rstd * (float)gam[i][e];
      store_chunk8<Elt, WHOLE>(static_cast<Elt*>(a.y) + row * a.R + f0, live ? a.R - f0 : 0, o);
    }
  }
}

// Rows longer than the registers hold: a workgroup a row, which reads it twice (the second time, the
// stored sum or both operands, from cache).
template <typename Elt>
__global__ void __launch_bounds__(1024) eql_rms_fwd_wide_kernel(const NormArgs a) {
  __shared__ float red[16];
  const int64_t at = (int64_t)blockIdx.x * a.R;
  float q[1] = {0.0f};
  auto value = [&](int f0, bool again, float (&v)[8]) __attribute__((always_inline)) {
    const int n = a.R - f0;
    const bool kept = again && a.sum;
    const auto u = load_chunk8<Elt, false, false>(static_cast<const Elt*>(kept ? a.sum : a.x) + at + f0, n);
    if (!kept && a.res) {
      const auto r = load_chunk8<Elt, false, false>(static_cast<const Elt*>(a.res) + at + f0, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)(Elt)((float)u[e] + (float)r[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)u[e];
    }
    if (!again && a.sum) store_chunk8<Elt, false>(static_cast<Elt*>(a.sum) + at + f0, n, v);
  };
  for (int f0 = (int)threadIdx.x * 8; f0 < a.R; f0 += 8192) {
    float v[8];
    value(f0, false, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[0] = __builtin_fmaf(v[e], v[e], q[0]);
  }
  block_sums(q, red);
  const float rstd = inv_sqrt(__builtin_fmaf(q[0], a.invR, a.eps));
  if (threadIdx.x == 0 && a.rstd) a.rstd[blockIdx.x] = rstd;
  for (int f0 = (int)threadIdx.x * 8; f0 < a.R; f0 += 8192) {
    float v[8], o[8];
    value(f0, true, v);
    const auto gam = spread<Elt>(a, a.gamma, f0, 1.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[e] * rstd * (float)gam[e];
    store_chunk8<Elt, false>(static_cast<Elt*>(a.y) + at + f0, a.R - f0, o);
  }
}

}  // namespace eql
