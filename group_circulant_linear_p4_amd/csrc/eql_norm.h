// Layer norm of an equivariant block, forward and backward.
//
// A row holds R = C'*T features.  Mean and variance are taken over the whole row, so a cyclic
// shift of every channel's group axis leaves them alone, and weight and bias are one value per
// channel, shared by its T group elements: the norm commutes with the group action.
//     h = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  y = gamma[c] h + beta[c]
// Backward, with g = dy gamma[c]:
//     dx        = rstd (g - mean(g) - h mean(g h)) [+ dres]
//     dgamma[c] = sum over rows and t of dy h,   dbeta[c] = sum over rows and t of dy
// h comes from x and the row's statistics, or from the 8-bit checkpoint of h that the forward
// pass wrote (eql_ckpt8.h).
//
// All of it is bound by memory: one read of each operand, one write of each result.  Rows of up
// to kNormFwdMaxRow (backward kNormBwdMaxRow) features are held in registers between the two uses
// (statistics, result): LPR lanes take a row, K chunks of 8 features a lane, chunk j of the row on
// lane j % LPR.  The variance is the mean square of the centred row, a second pass over registers.  Sums are fp32.
// A workgroup takes rows 256 / LPR at a time in a grid-stride loop, with gamma and beta, and in
// the backward pass the column sums of dy h and dy, in registers for the whole loop.
// Longer rows go through the kernels at the end of this file.
#pragma once

#include "eql_ckpt8.h"

namespace eql {

struct NormArgs {
  const void* x;      // [N][R] (backward: unless the checkpoint is read)
  const void* gamma;  // [C] or null (1)
  const void* beta;   // [C] or null (0)
  void* y;            // forward: [N][R]
  unsigned char* codes;   // checkpoint of h, or null
  unsigned char* scales;
  float* mean;        // [N] or null
  float* rstd;        // [N] or null
  const void* dy;     // backward: [N][R]
  const void* dres;   // [N][R] or null
  void* dx;           // [N][R] (may be dy or dres)
  void* dgamma;       // backward by one workgroup: [C], written by it (then part is null)
  void* dbeta;
  float* part;        // [gridDim][2][C] column sums (wide: [rowBlocks][2][R]), or null
  float* rowSums;     // wide backward: [N][2], mean(g) and mean(g h)
  int64_t N;
  int R, C, T, pitch;
  uint32_t perT;      // ceil(2^32 / T) for T > 1: f / T is the product's high word (f < 2^28)
  int table;          // 1: parameters spread through LDS (norm_table)
  float eps, invR;
  int rowsPerBlock, colBlocks;  // wide backward
  const void* res;    // RMS norm forward: added to x, or null
  void* sum;          // RMS norm forward: receives x + res, or null (may be x or res)
};

// Sum over the LPR lanes of a row (LPR <= 64), on every lane.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v = dpp_add<kDppXor1>(v);
  v = dpp_add<kDppXor2>(v);
  if constexpr (LPR >= 8) v = dpp_add<kDppMirror8>(v);
  if constexpr (LPR >= 16) v = dpp_add<kDppMirror16>(v);
  if constexpr (LPR >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  }
  if constexpr (LPR >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  }
  return v;
}

// Sums of M values over the lanes of a row; LPR > 64: over the workgroup's waves through LDS
// (`red`: M x waves floats, one barrier before the reads; the caller alternates two areas).
template <int LPR, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], float* red) {
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = row_sum<(LPR < 64 ? LPR : 64)>(v[m]);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = (int)threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) red[m * W + wave] = v[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float t = red[m * W];
#pragma unroll
      for (int w = 1; w < W; ++w) t += red[m * W + w];
      v[m] = t;
    }
  }
}

// A row's mean from its sum: times the rounded 1 / R, and the exact remainder of that once more,
// which gives the rounded quotient.  The product alone misses the mean of R equal features by an ulp
// for one row length in seven (41, 47, 55, 82, 164, 656, ...), and rstd amplifies that: R = 656
// features of 16384 gave h = 0.3 at eps = 1e-5 where the definition has 0.  (65536 rows of R = 32 both
// ways: 18.4 us with the product alone, 19.0 so and 19.6 with a division.)
__device__ __forceinline__ float row_mean(const NormArgs& a, float sum) {
  const float q = sum * a.invR, m = __builtin_fmaf(__builtin_fmaf(-q, (float)a.R, sum), a.invR, q);
  return __builtin_isfinite(q) ? m : q;
}

__device__ __forceinline__ int channel_of(const NormArgs& a, int f) {
  return a.T == 1 ? f : (int)__umulhi((uint32_t)f, a.perT);
}

// One per-channel parameter spread over the 8 features of a chunk (as elements; features past the
// row's end take any channel's).  The chunk's channels are fetched once each: 8 / T in one load
// where T is 1, 2 or 4, one where 8 divides T, else the four that it can touch at most.
template <typename Elt>
__device__ __forceinline__ typename Chunk<Elt>::V spread(const NormArgs& a, const void* p, int f0, float missing) {
  typedef Elt E2 __attribute__((ext_vector_type(2), aligned(sizeof(Elt))));
  typedef Elt E4 __attribute__((ext_vector_type(4), aligned(sizeof(Elt))));
  const int R = a.R, T = a.T;
  typename Chunk<Elt>::V v = (typename Chunk<Elt>::V)(Elt)missing;
  if (!p || f0 >= R) return v;
  const Elt* q = static_cast<const Elt*>(p);
  const bool whole = f0 + 8 <= R;
  if (T == 4) {
    E2 u = (E2)q[f0 / 4];  // a partial chunk is one channel
    if (whole) u = *reinterpret_cast<const E2*>(q + f0 / 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u[e / 4];
  } else if (T == 2 && whole) {
    const E4 u = *reinterpret_cast<const E4*>(q + f0 / 2);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u[e / 2];
  } else if (T == 1 && whole) {
    v = *reinterpret_cast<const typename Chunk<Elt>::VU*>(q + f0);
  } else if ((T & 7) == 0) {
    v = (typename Chunk<Elt>::V)q[channel_of(a, f0)];
  } else if (T == 1) {  // the row's last, partial chunk
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (f0 + e < R) v[e] = q[f0 + e];
  } else {
    const int last = a.C - 1, c = channel_of(a, f0), t = f0 - c * T;
    const Elt u0 = q[c], u1 = q[min(c + 1, last)], u2 = q[min(c + 2, last)], u3 = q[min(c + 3, last)];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = t + e;  // at most T + 6, below 4 T
      v[e] = x >= 2 * T ? (x >= 3 * T ? u3 : u2) : (x >= T ? u1 : u0);
    }
  }
  return v;
}

// The other group orders' parameters go through a table of the row's features in LDS, filled by
// the whole workgroup: selecting among four channels for every chunk is some 100 operations, and
// in a small launch, one wave to a SIMD, they took longer than the rows (37 rows of R = 1752,
// T = 12 fp16: 8.0 us forward and 5.1 with the table).  Not where a row takes the whole workgroup:
// each entry would serve one lane once (199 rows of R = 4542, T = 6: 8.2 us and 10.4 with it).
// Features to the end of the last chunk are defined.
constexpr int64_t kNormTableBytes = 32768;
__host__ __device__ constexpr int norm_table_row(int R) { return (R + 7) / 8 * 8; }
__host__ constexpr bool norm_table(int lpr, int R, int T, int elt, int params) {
  return lpr < 256 && T != 1 && T != 2 && T != 4 && T != 8 && T != 16 && (int64_t)norm_table_row(R) * elt * params <= kNormTableBytes;
}
template <typename Elt>
__device__ __forceinline__ void fill_table(const NormArgs& a, Elt* table, const void* p, float missing) {
  const Elt* q = static_cast<const Elt*>(p);
#pragma unroll 4
  for (int f = (int)threadIdx.x; f < norm_table_row(a.R); f += 256) {
    const int c = min(channel_of(a, f), a.C - 1);
    table[f] = q ? q[c] : (Elt)missing;
  }
}

// 1 / sqrt(a) from the hardware's approximation and one Newton step, within an ulp or so.  NaN for
// a = 0 and a = infinity: a constant row without eps, and one whose squares overflow.
__device__ __forceinline__ float inv_sqrt(float a) {
  const float r = __builtin_amdgcn_rsqf(a);
  return __builtin_fmaf(0.5f * r, __builtin_fmaf(-a * r, r, 1.0f), r);
}

// A checkpoint block of normalised rows: h is NaN throughout exactly when rstd is.
__device__ __forceinline__ void store_block(const NormArgs& a, int64_t row, int f0, const float (&h)[8], float back,
                                            uint32_t scale, float rstd, bool scaleLane) {
  *reinterpret_cast<u32x2*>(a.codes + row * a.pitch + f0) = encode8(h, back);
  if (scaleLane)
    a.scales[row * (a.pitch / kCkptBlock) + f0 / kCkptBlock] = (unsigned char)(__builtin_isnan(rstd) ? 255u : scale);
}

template <typename Elt, int LPR, int K, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(256) eql_norm_fwd_kernel(const NormArgs a) {
  using V = typename Chunk<Elt>::V;
  constexpr int G = 256 / LPR;
  extern __shared__ __align__(16) float lds[];  // the parameters' table, if there is one
  __shared__ float red[2][8];
  const int lane = (int)threadIdx.x % LPR, grp = (int)threadIdx.x / LPR;
  const int64_t step = (int64_t)gridDim.x * G;
  // The row after the one at work is loaded before it is needed.
  V next[K];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    const Elt* xr = static_cast<const Elt*>(a.x) + row * a.R;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
      next[i] = load_chunk8<Elt, WHOLE, STREAM>(xr + f0, row < a.N ? a.R - f0 : 0);
    }
  };
  load((int64_t)blockIdx.x * G + grp);
  V gam[K], bet[K];
  if (a.table) {
    Elt* table = reinterpret_cast<Elt*>(lds);
    const int size = norm_table_row(a.R);
    fill_table(a, table, a.gamma, 1.0f);
    fill_table(a, table + size, a.beta, 0.0f);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = min((lane + i * LPR) * 8, size - 8);
      gam[i] = *reinterpret_cast<const V*>(table + f0);
      bet[i] = *reinterpret_cast<const V*>(table + size + f0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      gam[i] = spread<Elt>(a, a.gamma, (lane + i * LPR) * 8, 1.0f);
      bet[i] = spread<Elt>(a, a.beta, (lane + i * LPR) * 8, 0.0f);
    }
  }
  for (int64_t base = (int64_t)blockIdx.x * G; base < a.N; base += step) {
    const int64_t row = base + grp;
    const bool live = row < a.N;
    float v[K][8];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = (float)next[i][e];
        s[0] += v[i][e];
      }
    if (base + step < a.N) load(row + step);
    row_sums<LPR>(s, red[0]);
    const float mean = row_mean(a, s[0]);
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float t = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] -= mean;
      int n = a.R - (lane + i * LPR) * 8;
      if (!WHOLE && a.R < (i + 1) * LPR * 8) {
        // The row ends among these chunks: its missing features count as zero.  (Compared afresh
        // in every turn: kept over the loop, the lane masks would spill the scalar registers.)
        asm volatile("" : "+v"(n));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = e < n ? v[i][e] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) t = __builtin_fmaf(v[i][e], v[i][e], t);
      q[0] += WHOLE && n < 8 ? 0.0f : t;
    }
    row_sums<LPR>(q, red[1]);
    const float rstd = inv_sqrt(__builtin_fmaf(q[0], a.invR, a.eps));
    if (live && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] *= rstd;
        o[e] = __builtin_fmaf(v[i][e], (float)gam[i][e], (float)bet[i][e]);
      }
      if (live) store_chunk8<Elt, WHOLE>(static_cast<Elt*>(a.y) + row * a.R + f0, a.R - f0, o);
      if (a.codes) {
        // A missing chunk of the row's last block has codes zero (h is rstd times minus the mean).
        const bool here = !WHOLE || f0 < a.R;
        const uint32_t top = __builtin_bit_cast(uint32_t, chunk_top(v[i]));
        const BlockStep st = block_step(quad_max(here ? top : 0u));
        if (live && f0 < a.pitch) store_block(a, row, f0, v[i], here ? st.back : 0.0f, st.scale, rstd, (lane & 3) == 0);
      }
    }
  }
}

// Sum over the lanes of a wave that hold the same chunks (LPR < 64), on all of them.
template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
  static_assert(LPR >= 16, "row groups of 16 lanes or more");
  if constexpr (LPR <= 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  }
  if constexpr (LPR <= 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  }
  return v;
}

// Copies of a feature's column sum that the end of the backward kernel adds through LDS: one a
// wave, or one in all where a row takes the whole workgroup.
__host__ __device__ constexpr int norm_bwd_copies(int lpr) { return lpr > 64 ? 1 : 4; }

// CKPT: h from the checkpoint (codes, scales, rstd), else from x, mean and rstd.  RMS: the RMS norm's
// backward, which is this without the mean of x, the mean of g and the bias; its blocks of column
// sums are [C].
// Dynamic LDS: norm_bwd_copies(LPR) * R floats, for the column sums at the end, or the table.
template <typename Elt, int LPR, int K, bool WHOLE, bool STREAM, bool CKPT, bool RMS = false>
__global__ void __launch_bounds__(256) eql_norm_bwd_kernel(const NormArgs a) {
  using V = typename Chunk<Elt>::V;
  constexpr int G = 256 / LPR;
  extern __shared__ __align__(16) float lds[];  // the weight's table, then the column sums
  __shared__ float red[2][8];
  const int lane = (int)threadIdx.x % LPR, grp = (int)threadIdx.x / LPR;
  const int64_t step = (int64_t)gridDim.x * G;
  // All operands of the row after the one at work are loaded before it is needed: the loop
  // otherwise waits out the memory's latency once before the row's sums and, for dres, again.
  V dyN[K], xN[K], rN[K];
  u32x2 wN[K];
  uint32_t scN[K];
  float rstdN = 0.0f, meanN = 0.0f;
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    const bool live = row < a.N;
    rstdN = live ? a.rstd[row] : 0.0f;
    if constexpr (!CKPT && !RMS) meanN = live ? a.mean[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
      const int m = live ? a.R - f0 : 0;
      dyN[i] = load_chunk8<Elt, WHOLE, STREAM>(static_cast<const Elt*>(a.dy) + row * a.R + f0, m);
      if constexpr (CKPT) {
        wN[i] = (u32x2){0, 0};
        scN[i] = 0;
        if (m > 0) {
          wN[i] = load_codes8<STREAM>(a.codes + row * a.pitch + f0);
          scN[i] = a.scales[row * (a.pitch / kCkptBlock) + f0 / kCkptBlock];
        }
      } else {
        xN[i] = load_chunk8<Elt, WHOLE, STREAM>(static_cast<const Elt*>(a.x) + row * a.R + f0, m);
      }
      rN[i] = zero_chunk<Elt>();
      if (a.dres) rN[i] = load_chunk8<Elt, WHOLE, STREAM>(static_cast<const Elt*>(a.dres) + row * a.R + f0, m);
    }
  };
  load((int64_t)blockIdx.x * G + grp);
  V gam[K];
  float sg[K][8], sb[K][8];
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
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sg[i][e] = sb[i][e] = 0.0f;
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * G; base < a.N; base += step) {
    const int64_t row = base + grp;
    const bool live = row < a.N;
    const float rstd = rstdN;
    float h[K][8];
    V dy[K], r[K];
    constexpr int SUMS = RMS ? 1 : 2;
    float s[SUMS] = {};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      dy[i] = dyN[i];
      r[i] = rN[i];
      if constexpr (CKPT) {
        decode8(wN[i], scale_step(scN[i]), h[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = (RMS ? (float)xN[i][e] : (float)xN[i][e] - meanN) * rstd;
        int n = a.R - (lane + i * LPR) * 8;
        if (!RMS && a.R < (i + 1) * LPR * 8) {
          // Missing features count as zero: mean rstd may overflow where no h does.
          asm volatile("" : "+v"(n));
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] = (WHOLE ? n > 0 : e < n) ? h[i][e] : 0.0f;
        }
      }
    }
    if (base + step < a.N) load(row + step);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // Past the row's end dy and h are zero.
        const float d = (float)dy[i][e];
        const float g = d * (float)gam[i][e];
        if constexpr (!RMS) {
          s[0] += g;
          sb[i][e] += d;
        }
        s[SUMS - 1] = __builtin_fmaf(g, h[i][e], s[SUMS - 1]);
        sg[i][e] = __builtin_fmaf(d, h[i][e], sg[i][e]);
      }
    row_sums<LPR>(s, red[turn]);
    turn ^= 1;
    const float m1 = RMS ? 0.0f : row_mean(a, s[0]), m2 = row_mean(a, s[SUMS - 1]);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = (float)dy[i][e] * (float)gam[i][e];
        o[e] = __builtin_fmaf(rstd, __builtin_fmaf(-h[i][e], m2, RMS ? g : g - m1), (float)r[i][e]);
      }
      store_chunk8<Elt, WHOLE>(static_cast<Elt*>(a.dx) + row * a.R + f0, live ? a.R - f0 : 0, o);
    }
  }
  if (!a.part && !a.dgamma && !a.dbeta) return;
  // Column sums: the row groups of a wave across its lanes, the waves through LDS, then per
  // channel its T features, in a fixed order.
  constexpr int COPIES = norm_bwd_copies(LPR);
  const int copy = LPR > 64 ? 0 : (int)threadIdx.x >> 6;
  const bool writes = LPR >= 64 || (threadIdx.x & 63) < LPR;
  constexpr int KINDS = RMS ? 1 : 2;
  float* out = a.part + (int64_t)blockIdx.x * KINDS * a.C;
#pragma unroll
  for (int which = 0; which < KINDS; ++which) {
    void* direct = which ? a.dbeta : a.dgamma;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int f0 = (lane + i * LPR) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t = which ? sb[i][e] : sg[i][e];
        if constexpr (LPR < 64) t = group_sum<LPR>(t);
        if (writes && f0 + e < a.R) lds[copy * a.R + f0 + e] = t;
      }
    }
    __syncthreads();
    for (int c = (int)threadIdx.x; c < a.C; c += 256) {
      float t = 0.0f;
      for (int j = 0; j < a.T; ++j)
#pragma unroll
        for (int q = 0; q < COPIES; ++q) t += lds[q * a.R + c * a.T + j];
      if (a.part) out[which * a.C + c] = t;
      else if (direct) static_cast<Elt*>(direct)[c] = (Elt)t;
    }
  }
}

// dgamma and dbeta from the blocks' column sums part[b][2][C * F] (F features a channel left to
// add), or one gradient from part[b][C]: a workgroup takes 16 channels x 64 slices of the blocks,
// slice l blocks l, l + 64, ...; the slices are added in a fixed order and the result rounded once.
// The launch is latency: at 451 blocks of 96 channels 3.1 us, and 3.8 with 16 slices.
struct NormParamArgs {
  const float* part;
  void* dgamma;  // [C] or null
  void* dbeta;   // [C] or null
  int blocks, C, F, groups;  // groups = ceil(C / 16); workgroups groups .. 2 groups - 1: dbeta
  int64_t blockStride;       // floats from a block's sums to the next one's
};

template <typename Elt>
__global__ void __launch_bounds__(1024) eql_norm_param_kernel(const NormParamArgs a) {
  __shared__ float red[16][17];
  const bool beta = (int)blockIdx.x >= a.groups;
  const int c = ((int)blockIdx.x - (beta ? a.groups : 0)) * 16 + ((int)threadIdx.x & 15), sl = (int)threadIdx.x >> 4;
  void* dst = beta ? a.dbeta : a.dgamma;
  if (!dst) return;
  const int64_t stride = (int64_t)a.C * a.F;
  float s = 0.0f;
  if (c < a.C) {
    const float* p = a.part + (beta ? stride : 0) + (int64_t)c * a.F;
    // Eight blocks' loads in flight.
    for (int b = sl; b < a.blocks; b += 512)
      for (int f = 0; f < a.F; ++f) {
        float t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = b + 64 * u < a.blocks ? p[(b + 64 * u) * a.blockStride + f] : 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) s += t[u];
      }
  }
  // The wave's four slices, then the waves.
  s = group_sum<16>(s);
  if ((threadIdx.x & 63) < 16) red[threadIdx.x >> 6][threadIdx.x & 15] = s;
  __syncthreads();
  if (sl == 0 && c < a.C) {
    float t = red[0][threadIdx.x];
#pragma unroll
    for (int l = 1; l < 16; ++l) t += red[l][threadIdx.x];
    static_cast<Elt*>(dst)[c] = (Elt)t;
  }
}

// ---------------------------------------------------------------------------
// Rows longer than the registers hold.  Forward: a workgroup per row reads it three times
// (sum, centred squares, result), the second and third time from cache.  Backward: a
// workgroup per row for the two row means, then a kernel over column blocks and row blocks
// that writes dx and the column sums.
// ---------------------------------------------------------------------------
template <int M>
__device__ __forceinline__ void block_sums(float (&v)[M], float* red) {
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = row_sum<64>(v[m]);
  const int wave = (int)threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) red[m * 16 + wave] = v[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) {
    float t = red[m * 16];
#pragma unroll
    for (int w = 1; w < 16; ++w) t += red[m * 16 + w];
    v[m] = t;
  }
}

template <typename Elt>
__global__ void __launch_bounds__(1024) eql_norm_fwd_wide_kernel(const NormArgs a) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const Elt* xr = static_cast<const Elt*>(a.x) + row * a.R;
  float s[1] = {0.0f};
  for (int f0 = (int)threadIdx.x * 8; f0 < a.R; f0 += 8192) {
    const auto u = load_chunk8<Elt, false, false>(xr + f0, a.R - f0);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += (float)u[e];
  }
  block_sums(s, red);
  const float mean = row_mean(a, s[0]);
  float q[1] = {0.0f};
  for (int f0 = (int)threadIdx.x * 8; f0 < a.R; f0 += 8192) {
    const auto u = load_chunk8<Elt, false, false>(xr + f0, a.R - f0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = f0 + e < a.R ? (float)u[e] - mean : 0.0f;
      q[0] = __builtin_fmaf(d, d, q[0]);
    }
  }
  block_sums(q, red);
  const float rstd = inv_sqrt(__builtin_fmaf(q[0], a.invR, a.eps));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  // To the end of the row's last block of 32: whole quads stay together for its scale.
  for (int f0 = (int)threadIdx.x * 8; f0 < a.pitch; f0 += 8192) {
    const int n = a.R - f0;
    const auto u = load_chunk8<Elt, false, false>(xr + f0, n);
    const auto gam = spread<Elt>(a, a.gamma, f0, 1.0f), bet = spread<Elt>(a, a.beta, f0, 0.0f);
    float h[8], o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[e] = e < n ? ((float)u[e] - mean) * rstd : 0.0f;
      o[e] = __builtin_fmaf(h[e], (float)gam[e], (float)bet[e]);
    }
    store_chunk8<Elt, false>(static_cast<Elt*>(a.y) + row * a.R + f0, n, o);
    if (a.codes) {
      const BlockStep st = block_step(quad_max(__builtin_bit_cast(uint32_t, chunk_top(h))));
      store_block(a, row, f0, h, st.back, st.scale, rstd, (threadIdx.x & 3) == 0);
    }
  }
}

// h of one chunk, from x or the checkpoint (zero past the row's end).
template <typename Elt, bool CKPT, bool RMS>
__device__ __forceinline__ void wide_h(const NormArgs& a, int64_t row, int f0, int n, float mean, float rstd, float (&h)[8]) {
  if constexpr (CKPT) {
    const float step = scale_step(a.scales[row * (a.pitch / kCkptBlock) + f0 / kCkptBlock]);
    decode8(load_codes8<false>(a.codes + row * a.pitch + f0), step, h);
  } else {
    const auto u = load_chunk8<Elt, false, false>(static_cast<const Elt*>(a.x) + row * a.R + f0, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = RMS ? (float)u[e] * rstd : (e < n ? ((float)u[e] - mean) * rstd : 0.0f);
  }
}

template <typename Elt, bool CKPT, bool RMS = false>
__global__ void __launch_bounds__(1024) eql_norm_bwd_rows_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const float rstd = a.rstd[row], mean = CKPT || RMS ? 0.0f : a.mean[row];
  float s[2] = {0.0f, 0.0f};
  for (int f0 = (int)threadIdx.x * 8; f0 < a.R; f0 += 8192) {
    const int n = a.R - f0;
    const auto d = load_chunk8<Elt, false, false>(static_cast<const Elt*>(a.dy) + row * a.R + f0, n);
    const auto gam = spread<Elt>(a, a.gamma, f0, 1.0f);
    float h[8];
    wide_h<Elt, CKPT, RMS>(a, row, f0, n, mean, rstd, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = (float)d[e] * (float)gam[e];
      s[0] += g;
      s[1] = __builtin_fmaf(g, h[e], s[1]);
    }
  }
  block_sums(s, red);
  if (threadIdx.x < 2) a.rowSums[row * 2 + threadIdx.x] = row_mean(a, s[threadIdx.x]);
}

// Workgroup: 256 chunks across (one a lane), rowsPerBlock rows down.
template <typename Elt, bool CKPT, bool RMS = false>
__global__ void __launch_bounds__(256) eql_norm_bwd_cols_kernel(const NormArgs a) {
  const int cb = (int)blockIdx.x % a.colBlocks, rb = (int)blockIdx.x / a.colBlocks;
  const int f0 = (cb * 256 + (int)threadIdx.x) * 8;
  const int n = a.R - f0;
  if (n <= 0) return;
  const auto gam = spread<Elt>(a, a.gamma, f0, 1.0f);
  float sg[8], sb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sg[e] = sb[e] = 0.0f;
  const int64_t r0 = (int64_t)rb * a.rowsPerBlock, r1 = min(a.N, r0 + a.rowsPerBlock);
  for (int64_t row = r0; row < r1; ++row) {
    const float rstd = a.rstd[row], mean = CKPT || RMS ? 0.0f : a.mean[row];
    const float m1 = RMS ? 0.0f : a.rowSums[row * 2], m2 = a.rowSums[row * 2 + 1];
    const auto d = load_chunk8<Elt, false, false>(static_cast<const Elt*>(a.dy) + row * a.R + f0, n);
    auto r = zero_chunk<Elt>();
    if (a.dres) r = load_chunk8<Elt, false, false>(static_cast<const Elt*>(a.dres) + row * a.R + f0, n);
    float h[8], o[8];
    wide_h<Elt, CKPT, RMS>(a, row, f0, n, mean, rstd, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float dv = (float)d[e], g = dv * (float)gam[e];
      sb[e] += dv;
      sg[e] = __builtin_fmaf(dv, h[e], sg[e]);
      o[e] = __builtin_fmaf(rstd, __builtin_fmaf(-h[e], m2, RMS ? g : g - m1), (float)r[e]);
    }
    store_chunk8<Elt, false>(static_cast<Elt*>(a.dx) + row * a.R + f0, n, o);
  }
  if (a.part) {
    float* out = a.part + (int64_t)rb * (RMS ? 1 : 2) * a.R + f0;
    store_chunk8<float, false>(out, n, sg);
    if constexpr (!RMS) store_chunk8<float, false>(out + a.R, n, sb);
  }
}

}  // namespace eql
