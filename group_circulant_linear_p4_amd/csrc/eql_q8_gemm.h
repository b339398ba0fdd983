// The EQ-Linear layer on 8-bit integer rows and weights (eql_q8.h): for each plane of the half
// spectrum integer products with 32-bit sums, which are exact (|sum| <= 2 C 127^2 < 2^31), then
//     plane = sum * (scale of the output channel * scale of the row),
// the inverse transform, and the fused layer's epilogue (bias, GELU, residual).  A row's outputs
// depend on nothing but the row and the weight: sums are exact in any order, so every kernel and
// every split gives the same bits.
//   real planes    S_p  = X_p W_p
//   complex pairs  S_re = Xr Wr + Xi (-Wi),  S_im = Xr Wi + Xi Wr   (codes are in [-127, 127], so
//                  negating Wi stays in 8 bits)
// Matrix step: 32 x 32 x 32 int8.  Lane l holds row (or output channel) l % 32 and 16 input channels
// from 16 (l / 32) on; result slot r of lane l is row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
#pragma once

#include "eql_fwd.h"
#include "eql_q8.h"

namespace eql {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

struct Q8FwdArgs {
  FwdArgs f;                    // y, N, Dout, tw, bias, res, act (x, wp, Cin unused)
  const unsigned char* codes;   // rows
  const float* rowScales;       // [N][F]
  const unsigned char* w;       // weight
  const float* wScales;         // [F][Dpad]
  int pitch, kblocks, Dpad;
  int colTiles;
  int waves;                    // small kernel
};

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ void q8_mfma(i32x16& acc, const u32x4& a, const u32x4& b) {
  acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), acc, 0, 0, 0);
}

// Each byte negated: ~v + 1 without carries between bytes.
__device__ __forceinline__ u32x4 q8_neg(const u32x4& v) {
  const u32x4 n = ~v;
  return ((n & 0x7F7F7F7Fu) + 0x01010101u) ^ (n & 0x80808080u);
}

#endif

// GELU, v Phi(v) = max(v, 0) - |v| Q(|v|) with Q = 1 - Phi = 2^p(|v|): p is a polynomial of degree 8 with p(0) = -1,
// fitted to log2 Q up to 5.6, where |v| Q is off by at most 4.6e-5 of it and 7.9e-8 (in fp32 4.8e-5 and 1.1e-7, and GELU, which
// is rounded to its own fp32, by 2.4e-7; gelu_erf: 3.8e-7, and 1.7e-3 of the value at -4.2).  Beyond, where it is below 6e-8, p falls
// without end and faster than log2 Q.  One transcendental operation and eleven others where gelu_erf has two and 13: a
// product's epilogue is bound by them.  The bound on |v| keeps infinity times zero out; a NaN stays one.
__device__ __forceinline__ float gelu_power(float v) {
  const float a = __builtin_fabsf(v);
  float q = __builtin_fmaf(-6.174803389e-7f, a, 1.057548525e-5f);
  q = __builtin_fmaf(q, a, -3.799108526e-5f);
  q = __builtin_fmaf(q, a, -5.224814522e-4f);
  q = __builtin_fmaf(q, a, 7.600945886e-3f);
  q = __builtin_fmaf(q, a, -5.288746953e-2f);
  q = __builtin_fmaf(q, a, -0.4590758979f);
  q = __builtin_fmaf(q, a, -1.151120067f);
  q = __builtin_fmaf(q, a, -1.0f);
  return __builtin_fmaf(-__builtin_fminf(a, 1e30f), __builtin_amdgcn_exp2f(q), __builtin_fmaxf(v, 0.0f));
}

#if defined(__HIP_DEVICE_COMPILE__)
// The T outputs of one (row, output channel) before the activation: scaled planes, inverse transform,
// bias.  sum * (scale of the channel * scale of the row) in one fused operation each where the transform's
// coefficients are 0 and +-1, which also makes a cyclic shift exact (each output is the same expression).
template <int T>
__device__ __forceinline__ void q8_outputs(const int32_t (&sum)[T], const float (&scale)[n_freqs(T)], float bias, float (&y)[T],
                                           const Twiddles& tw) {
  if constexpr (T == 1) {
    y[0] = __builtin_fmaf((float)sum[0], scale[0], bias);
  } else if constexpr (T == 2 || T == 4) {
    const float e = __builtin_fmaf((float)sum[0], scale[0], bias), a1 = (float)sum[1];
    const float ep = __builtin_fmaf(a1, scale[1], e), em = __builtin_fmaf(-a1, scale[1], e);
    if constexpr (T == 2) {
      y[0] = ep;
      y[1] = em;
    } else {
      const float re = (float)sum[2], im = (float)sum[3];
      y[0] = __builtin_fmaf(re, scale[2], ep);
      y[1] = __builtin_fmaf(-im, scale[2], em);
      y[2] = __builtin_fmaf(-re, scale[2], ep);
      y[3] = __builtin_fmaf(im, scale[2], em);
    }
  } else {
    float P[T];
#pragma unroll
    for (int p = 0; p < T; ++p) P[p] = (float)sum[p] * scale[freq_of(T, p)];
    Idft<T, false>::run(P, y, tw);
#pragma unroll
    for (int g = 0; g < T; ++g) y[g] += bias;
  }
}
#endif

// The fused layer's end for one (row, output channel).
template <int T, typename Elt>
__device__ __forceinline__ void q8_finish(const Q8FwdArgs& a, const int32_t (&sum)[T], const float (&scale)[n_freqs(T)], float bias,
                                          const float (&res)[T], int64_t at) {
#if defined(__HIP_DEVICE_COMPILE__)
  float y[T];
  q8_outputs<T>(sum, scale, bias, y, a.f.tw);
#pragma unroll
  for (int g = 0; g < T; ++g) y[g] = (a.f.act == 1 ? gelu_power(y[g]) : y[g]) + res[g];
  store_group<T, Elt>(static_cast<Elt*>(a.f.y) + at, y);
#endif
}

// One to kQ8Tokens rows: nothing but the weight's bytes matters.  A workgroup takes eight output channels (128
// bytes of every 512 in the weight's operand order), so that the weight spreads over the chip (1024 channels: 128
// workgroups); lane l takes channel l % 8 and the 16 input channels number l / 8 of each pair of K blocks, its wave
// every fourth pair.  Dot products of four codes, eight lanes' and four waves' sums added at the end.  Bound by one
// memory latency after the other (one row, 1024 -> 1024 channels, T = 4 fp16: 3.8 us, 4.2 MB of weight; with the weight in
// cache 2.8, on the small kernel's tiles then 5.1).
constexpr int kQ8Tokens = 4;
template <int T, typename Elt>
__global__ void __launch_bounds__(256) eql_q8_token_kernel(const Q8FwdArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NR = n_real_planes(T), NP = n_pairs(T), F = n_freqs(T);
  __shared__ int32_t sums[kQ8Tokens][T][4][8];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int ol = lane & 7, piece = lane >> 3;  // piece: K block of the pair, its half, quarter
  const int col0 = (int)blockIdx.x * 8;
  // Eight threads a row end with its outputs (the first 32 at most); their operands are on their way before the sums.
  const int n = (int)threadIdx.x >> 3, col = col0 + ((int)threadIdx.x & 7);
  const bool ends = n < a.f.N && n < kQ8Tokens && col < a.f.Dout;
  float scale[F], res[T], bias = 0.0f;
  const int64_t at = ((int64_t)n * a.f.Dout + col) * T;
#pragma unroll
  for (int g = 0; g < T; ++g) res[g] = 0.0f;
  if (ends) {
#pragma unroll
    for (int f = 0; f < F; ++f) scale[f] = a.wScales[(int64_t)f * a.Dpad + col] * a.rowScales[(int64_t)n * F + f];
    if (a.f.bias) bias = (float)static_cast<const Elt*>(a.f.bias)[col];
    if (a.f.res) load_group<T, Elt>(static_cast<const Elt*>(a.f.res) + at, res);
  }
  int32_t acc[kQ8Tokens][T + NP];
#pragma unroll
  for (int r = 0; r < kQ8Tokens; ++r)
#pragma unroll
    for (int p = 0; p < T + NP; ++p) acc[r][p] = 0;
  const unsigned char* w = a.w + (size_t)(col0 / 32) * a.kblocks * T * 2048 + (size_t)((col0 & 31) + ol) * 16;
  const int64_t rowBytes = (int64_t)a.pitch * T;
  auto dot = [](int32_t& s, const u32x4& x, const u32x4& y) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_sdot4((int)x[i], (int)y[i], s, false);
  };
#pragma unroll 2
  for (int kb = wave * 2 + (piece >> 2); kb < a.kblocks; kb += 8) {
    const int k = kb * kQ8Block + (piece & 3) * 16;  // this lane's first input channel
    if (k >= a.pitch) continue;                       // whole pieces: a row's planes are multiples of 16
    u32x4 wv[T];
#pragma unroll
    for (int p = 0; p < T; ++p)
      wv[p] = *reinterpret_cast<const u32x4*>(w + ((size_t)kb * T + p) * 2048 + (piece & 3) * 512);
#pragma unroll
    for (int r = 0; r < kQ8Tokens; ++r) {
      if (r >= a.f.N) break;
      u32x4 xv[T];
#pragma unroll
      for (int p = 0; p < T; ++p) xv[p] = *reinterpret_cast<const u32x4*>(a.codes + r * rowBytes + p * a.pitch + k);
#pragma unroll
      for (int p = 0; p < NR; ++p) dot(acc[r][p], xv[p], wv[p]);
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const int re = NR + 2 * q, im = re + 1;
        dot(acc[r][re], xv[re], wv[re]);
        dot(acc[r][T + q], xv[im], wv[im]);  // subtracted at the end
        dot(acc[r][im], xv[re], wv[im]);
        dot(acc[r][im], xv[im], wv[re]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kQ8Tokens; ++r) {
    if (r >= a.f.N) break;
#pragma unroll
    for (int q = 0; q < NP; ++q) acc[r][NR + 2 * q] -= acc[r][T + q];
#pragma unroll
    for (int p = 0; p < T; ++p) {
      // Lanes 8, 16 and 32 apart: within a row of 16 by a rotation, then the swaps of half rows and halves.
      int32_t v = acc[r][p] + (int32_t)dpp_move<0x128>((uint32_t)acc[r][p]);
      const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
      v = (int32_t)h[0] + (int32_t)h[1];
      const auto g = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
      v = (int32_t)g[0] + (int32_t)g[1];
      if (lane < 8) sums[r][p][wave][lane] = v;
    }
  }
  __syncthreads();
  if (!ends) return;
  int32_t sum[T];
#pragma unroll
  for (int p = 0; p < T; ++p) {
    sum[p] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[p] += sums[n][p][i][threadIdx.x & 7];
  }
  q8_finish<T, Elt>(a, sum, scale, bias, res, at);
#endif
}

// Few rows or few output channels: a workgroup takes a 32 x 32 tile of outputs, its waves every so-manieth step
// of 32 input channels each (operands straight from memory), and adds its integer sums in LDS.  Epilogue: a thread a
// (row, channel), a row's channels on neighbouring lanes; its operands are on their way before the sums.  Bound by
// latency (197 rows, 96 -> 384 channels, T = 4 fp16, GELU: 6.8 us; the bytes would take 0.2).
template <int T, typename Elt>
__global__ void __launch_bounds__(T <= 8 ? 512 : 256) eql_q8_small_kernel(const Q8FwdArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NR = n_real_planes(T), NP = n_pairs(T), F = n_freqs(T);
  __shared__ int32_t sums[T][32 * 32];
  __shared__ float rowScale[32 * F];
  const int threads = (int)blockDim.x, W = threads >> 6;
  const int colTile = (int)blockIdx.x % a.colTiles, rowTile = (int)blockIdx.x / a.colTiles;
  const int row0 = rowTile * 32;
  const int lane = lane_index(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int rows = min(32, a.f.N - row0);
  const uint32_t rowBytes = (uint32_t)a.pitch * T;
  const uint32_t blockBytes = (uint32_t)T * 2048u;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.codes + (size_t)row0 * rowBytes, (uint32_t)rows * rowBytes);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (size_t)colTile * a.kblocks * blockBytes, (uint32_t)a.kblocks * blockBytes);
  i32x16 acc[T];
#pragma unroll
  for (int p = 0; p < T; ++p) acc[p] = (i32x16){};
  // Offsets past the last row's end (also of the last plane's last block) read as zero; bytes past
  // another plane's end belong to the next one and meet zeros in the weight.
  const uint32_t xOff = (uint32_t)(lane & 31) * rowBytes + (uint32_t)(lane >> 5) * 16u;
  const int steps = (a.pitch + 31) / 32;
  // Long sums of T = 1 go in turns of four steps next to each other, the next turn's under way: a row's 128 bytes are read
  // at once (8 rows of 11000 -> 4096 channels, fp16: 9.8 us, with one step a turn 17.1; T = 2 gains nothing, and T = 4 has
  // no registers for it).
  constexpr int DEPTH = T == 1 ? 4 : 1;
  u32x4 xa[DEPTH][T], wb[DEPTH][T];
  auto load = [&](int st, int d) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < T; ++p) {
      xa[d][p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, xOff + (uint32_t)(st * 32 + p * a.pitch), 0, 0));
      wb[d][p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16 + p * 2048, (st >> 1) * (int)blockBytes + (st & 1) * 1024, 0));
    }
  };
  const bool turns = DEPTH > 1 && steps >= DEPTH * W;
  if (turns) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(min(wave * DEPTH + d, steps - 1), d);
  } else if (wave < steps) {
    load(wave, 0);
  }
  // What the epilogue reads, and zeros, while the first operands come.
  const int col = colTile * 32 + ((int)threadIdx.x & 31), at = min(col, a.f.Dout - 1);
  float ws[F];
#pragma unroll
  for (int f = 0; f < F; ++f) ws[f] = a.wScales[(int64_t)f * a.Dpad + at];
  const float bias = a.f.bias ? (float)static_cast<const Elt*>(a.f.bias)[at] : 0.0f;
  for (int i = (int)threadIdx.x; i < rows * F; i += threads) rowScale[i] = a.rowScales[(int64_t)row0 * F + i];
  for (int i = (int)threadIdx.x; i < T * 256; i += threads) reinterpret_cast<i32x4*>(&sums[0][0])[i] = (i32x4){0, 0, 0, 0};
  auto products = [&](const u32x4 (&x)[T], const u32x4 (&w)[T]) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < NR; ++p) q8_mfma(acc[p], x[p], w[p]);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int re = NR + 2 * q, im = re + 1;
      const u32x4 neg = q8_neg(w[im]);
      q8_mfma(acc[re], x[re], w[re]);
      q8_mfma(acc[im], x[re], w[im]);
      q8_mfma(acc[re], x[im], neg);
      q8_mfma(acc[im], x[im], w[re]);
    }
  };
  if (turns) {
    for (int st = wave * DEPTH;; st += DEPTH * W) {
      const int next = st + DEPTH * W;
      if (next >= steps) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
          if (st + d < steps) products(xa[d], wb[d]);
        break;
      }
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        products(xa[d], wb[d]);
        load(min(next + d, steps - 1), d);
      }
    }
  } else {
    for (int st = wave; st < steps; st += W) {
      u32x4 x[T], w[T];
#pragma unroll
      for (int p = 0; p < T; ++p) {
        x[p] = xa[0][p];
        w[p] = wb[0][p];
      }
      if (st + W < steps) load(st + W, 0);
      products(x, w);
    }
  }
  __syncthreads();
  if (wave < steps) {
#pragma unroll
    for (int p = 0; p < T; ++p)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (row < rows) __hip_atomic_fetch_add(&sums[p][row * 32 + (lane & 31)], acc[p][r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      }
  }
  __syncthreads();
  if (col >= a.f.Dout) return;
  for (int row = (int)threadIdx.x >> 5; row < rows; row += threads >> 5) {
    const int64_t out = ((int64_t)(row0 + row) * a.f.Dout + col) * T;
    float scale[F], res[T];
    int32_t sum[T];
#pragma unroll
    for (int g = 0; g < T; ++g) res[g] = 0.0f;
    if (a.f.res) load_group<T, Elt>(static_cast<const Elt*>(a.f.res) + out, res);
#pragma unroll
    for (int p = 0; p < T; ++p) sum[p] = sums[p][row * 32 + (col & 31)];
#pragma unroll
    for (int f = 0; f < F; ++f) scale[f] = ws[f] * rowScale[row * F + f];
    q8_finish<T, Elt>(a, sum, scale, bias, res, out);
  }
#endif
}

// Many rows: a workgroup takes a tile of 32 MB rows x 128 NB output channels of all planes, its four waves side by
// side, MB x NB blocks of 32 x 32 each (two waves down and two across read the rows' LDS half as often and the weight
// twice: no faster).
//   * Rows' codes go through an LDS ring of four slots, a K block (64 input channels of every plane) each, by
//     loads that write LDS directly (1 KB: 16 rows x 64 bytes of a plane), three blocks ahead.  Piece q (16
//     bytes) of row r lies at place q ^ (r / 4) % 4 of its 64 bytes, so the 16 rows that a fragment read takes
//     at a time touch every bank once.  The slots are separate arrays and every slot's code is its own, so
//     the compiler knows which loads a read of LDS has to wait for.
//   * The weight's operands lie in memory as the matrix instruction wants them, and no two waves across read
//     the same: each wave loads its own straight into registers, a block ahead (more than six planes' blocks:
//     each plane's next step as soon as this one's products have been issued).
//   * A block is 2 MB groups (a step of 32 input channels, 32 rows) of products.  Each plane of the next
//     group's rows is read from LDS as soon as this group's products of the plane have been issued; at the last
//     group from the next slot, so the wait for its loads and the barrier come before that group's products.
//   * The last block is code of its own, which loads nothing ahead but the first residuals, into the registers that the
//     next operands would have taken (50176 rows of 192 -> 192, T = 4 fp16, with a residual: 42.1 -> 40.6 us).
// At 65536 rows of 1024 -> 1024, T = 4 fp16, call after call: 578 us with a residual, 495 without (825 G integer operations,
// 1.34 and 0.81 GB), 605 with rows and residual out of the caches.  The matrix unit is busy 36% of that (counted); these instructions
// alone, on such codes, reach 3.6 P operations/s, held by the card's power: on zeros the kernel takes 517 and 399 us.  The
// residual's reads, 83 and 118 us of these, hardly overlap the main loops: both workgroups of a compute unit share the way from
// L2 that the weight's operands take.
template <int T, typename Elt, int MB, int NB>
__global__ void __launch_bounds__(256, (T * MB * NB <= 8 ? 2 : 1)) eql_q8_large_kernel(const Q8FwdArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NR = n_real_planes(T), NP = n_pairs(T), F = n_freqs(T);
  constexpr int BM = 32 * MB, NS = 4;
  constexpr int CHUNKS = T * BM / 16;              // 1 KB loads of a slot
  constexpr int PER = (CHUNKS + 3) / 4;            // of a wave (where four do not divide them, some twice)
  constexpr int SLOT = CHUNKS * 64;                // 16-byte pieces
  constexpr int SCALES = (BM * F * 4 + 1023) / 1024;  // 1 KB loads of the rows' scales
  constexpr bool WHOLE = T * NB <= 6;
  constexpr int WSETS = WHOLE ? 2 : 1, WSTEPS = WHOLE ? 2 : 1;
  constexpr int WLOADS = WSTEPS * NB * T;          // operand loads of a set
  static_assert(BM <= kFwdRows && (NS * SLOT + SCALES * 64) * 16 <= 160 * 1024, "LDS");
  typedef __attribute__((address_space(3))) void* Lds;

  __shared__ u32x4 ring0[SLOT], ring1[SLOT], ring2[SLOT], ring3[SLOT];
  __shared__ u32x4 scaleRing[SCALES * 64];
  const float* rowScale = reinterpret_cast<const float*>(scaleRing);
  auto slot_of = [&](auto tag) __attribute__((always_inline)) -> u32x4* {
    constexpr int S = decltype(tag)::value % NS;
    if constexpr (S == 0) return ring0;
    else if constexpr (S == 1) return ring1;
    else if constexpr (S == 2) return ring2;
    else return ring3;
  };

  const int tile = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int colTile = tile % a.colTiles, rowTile = tile / a.colTiles;
  const int row0 = rowTile * BM;
  const int rows = min(BM, a.f.N - row0);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lane = (int)threadIdx.x & 63, lrow = lane & 31;
  const int block0 = (colTile * 4 + wave) * NB;     // this wave's first block of 32 output channels
  const int nblk = a.Dpad / 32;
  const uint32_t rowBytes = (uint32_t)a.pitch * T;
  const uint32_t blockBytes = (uint32_t)T * 2048u;
  const uint32_t colBytes = (uint32_t)a.kblocks * blockBytes;

  {
    // Rows past N have the scale zero.
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a.rowScales + (int64_t)row0 * F, (uint32_t)rows * F * 4u);
#pragma unroll
    for (int i = 0; i < (SCALES + 3) / 4; ++i) {
      const int j = min(wave + 4 * i, SCALES - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (Lds)(scaleRing + j * 64), 16, j * 1024 + lane * 16, 0, 0, 0);
    }
  }
  // Rows past N and, at the last row's end, bytes past the codes read as zero; bytes past a plane's end belong
  // to the next one and meet zeros in the weight.  Blocks past the last one are outside of the range.
  const char* xBase = reinterpret_cast<const char*>(a.codes) + (size_t)row0 * rowBytes;
  const uint32_t xBytes = (uint32_t)rows * rowBytes;
  uint32_t xOff[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = min(wave * PER + i, CHUNKS - 1), p = j / (BM / 16), rg = j % (BM / 16);
    const int r = rg * 16 + (lane >> 2), q = (lane & 3) ^ ((r >> 2) & 3);
    xOff[i] = (uint32_t)r * rowBytes + (uint32_t)p * (uint32_t)a.pitch + (uint32_t)q * 16u;
  }
  auto issue_rows = [&](int kb, u32x4* slot, int i0, int i1) __attribute__((always_inline)) {
    const uint32_t skip = (uint32_t)kb * 64u;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(xBase + skip, kb < a.kblocks ? xBytes - skip : 0u);
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      const int j = min(wave * PER + i, CHUNKS - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (Lds)(slot + j * 64), 16, (int)xOff[i], 0, 0, 0);
    }
  };

  // One block alone is followed by one of zeros, past the rows' descriptor: a loop that may not run costs registers.
  const int last = max(a.kblocks - 1, 1);
  // A wave past the last block of output channels does nothing but its share of the rows' loads, with the others'
  // waits and barriers (12608 rows of 384 -> 96 channels, T = 4 fp16: 10.0 us with its products, 9.3 without).
  if (block0 >= nblk) {
    auto slot_at = [&](int kb) __attribute__((always_inline)) {
      return kb & 2 ? (kb & 1 ? ring3 : ring2) : (kb & 1 ? ring1 : ring0);
    };
    issue_rows(0, ring0, 0, PER);
    issue_rows(1, ring1, 0, PER);
    issue_rows(2, ring2, 0, PER);
    for (int kb = 0; kb < last; ++kb) {
      wait_vmcnt<(2 * PER < 63 ? 2 * PER : 63)>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue_rows(kb + NS - 1, slot_at(kb + NS - 1), 0, PER);
    }
    wait_vmcnt<(2 * PER < 63 ? 2 * PER : 63)>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    wait_vmcnt<0>();
    return;
  }

  // Blocks of output channels past the last one read the last one's operands, and store nothing.
  const int first = min(block0, nblk - 1), more = nblk - 1 - first;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (size_t)first * colBytes, (uint32_t)(min(NB - 1, more) + 1) * colBytes);
  u32x4 wb[WSETS][WSTEPS][NB][T];
  auto load_w1 = [&](int kb, int s, int nb, int p) __attribute__((always_inline)) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
        wr, lane * 16, min(kb, a.kblocks - 1) * (int)blockBytes + min(nb, more) * (int)colBytes + (p * 2 + s) * 1024, 0));
  };
  auto load_w = [&](int kb, u32x4 (&to)[WSTEPS][NB][T], int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
    for (int i = i0; i < i1; ++i) to[i / (NB * T)][i / T % NB][i % T] = load_w1(kb, i / (NB * T), i / T % NB, i % T);
  };

  i32x16 acc[MB][NB][T];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int p = 0; p < T; ++p) acc[mb][nb][p] = (i32x16){};

  u32x4 xa[T];
  auto read_row = [&](const u32x4* slot, int s, int mb, int p) __attribute__((always_inline)) {
    const int r = mb * 32 + lrow;
    const int q = (s * 2 + (lane >> 5)) ^ ((r >> 2) & 3);
    xa[p] = slot[p * (BM * 4) + r * 4 + q];
  };

  // Epilogue in chunks of CH rows: outputs past the rows or channels get an offset beyond the descriptor's
  // range.  A chunk's residual is loaded while the one before is finished (and before the chunk's own stores:
  // it may be y), the first one's in the last block, or before the first where registers are left.
  constexpr int ELT = (int)sizeof(Elt);
  constexpr int RW = group_words<T, Elt>(), CH = T > 8 ? 1 : (RW <= 2 ? 16 : (RW <= 4 ? 8 : 4)), PARTS = 16 / CH;
  const uint32_t outRow = (uint32_t)a.f.Dout * T * ELT;
  const __amdgpu_buffer_rsrc_t yr = make_rsrc(static_cast<char*>(a.f.y) + (size_t)row0 * outRow, (uint32_t)rows * outRow);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(static_cast<const char*>(a.f.res) + (size_t)row0 * outRow, (uint32_t)rows * outRow);
  constexpr bool EARLY = T * MB * NB <= 4 && CH * RW <= 32;
  uint32_t res[2][CH][RW];
  auto offset_of = [&](int nb, int mb, int r) __attribute__((always_inline)) {
    const int col = (block0 + nb) * 32 + lrow, row = mb * 32 + 4 * (lane >> 5);
    const uint32_t off = col < a.f.Dout ? (uint32_t)row * outRow + (uint32_t)(col * T * ELT) : kOob;
    return off + (uint32_t)(8 * (r >> 2) + (r & 3)) * outRow;
  };
  auto load_res = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      load_group_raw<T, Elt>(rr, offset_of(i / PARTS / MB, i / PARTS % MB, i % PARTS * CH + j), res[i & 1][j]);
  };

  constexpr int GROUPS = 2 * MB, ISSUE = GROUPS > 2 ? GROUPS / 2 : 1;  // groups that issue the loads ahead
  // Loads of this wave that may be under way when the next block's rows have to be there: at least so many have
  // been issued after them (two blocks' rows, and the operands of two blocks, or of two steps; before the first
  // block the order is rows 0, rows 1, operands, rows 2).
  constexpr int AHEAD = 2 * PER + 2 * WLOADS;
  auto stage = [&](int kb, auto tag, auto lastTag) __attribute__((always_inline)) {
    constexpr bool LAST = decltype(lastTag)::value;
    constexpr int S = decltype(tag)::value, wcur = WHOLE && !LAST ? S & 1 : 0;
    const u32x4* cur = slot_of(tag);
    const u32x4* nxt = slot_of(std::integral_constant<int, S + 1>{});
    u32x4* ahead = slot_of(std::integral_constant<int, S + NS - 1>{});
    if constexpr (LAST) {
      // Its slot is known at run time only: every load into LDS has come first (so none outlives the workgroup).
      const int at = kb & (NS - 1);
      cur = at & 2 ? (at & 1 ? ring3 : ring2) : (at & 1 ? ring1 : ring0);
      wait_vmcnt<0>();
      if constexpr (!EARLY && WHOLE)
        if (a.f.res) load_res(0);
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int s = g / MB, mb = g % MB, ws = WHOLE ? s : 0;
      if (!LAST && g < ISSUE) {
        issue_rows(kb + NS - 1, ahead, g * PER / ISSUE, (g + 1) * PER / ISSUE);
        if constexpr (WHOLE) load_w(kb + 1, wb[wcur ^ 1], g * WLOADS / ISSUE, (g + 1) * WLOADS / ISSUE);
      }
      if (!LAST && g + 1 == GROUPS) {
        // The next block's rows are in LDS, and every wave has read this one's.
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(AHEAD < 63 ? AHEAD : 63)>();
        wait_lgkm0();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      auto next = [&](int p) __attribute__((always_inline)) {
        if (g + 1 < GROUPS) read_row(cur, (g + 1) / MB, (g + 1) % MB, p);
        else if (!LAST) read_row(nxt, 0, 0, p);
        if constexpr (!WHOLE) {
          if (mb + 1 == MB && !(LAST && s == 1)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) wb[0][0][nb][p] = load_w1(kb + s, s ^ 1, nb, p);
          }
        }
      };
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 0; p < NR; ++p) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) q8_mfma(acc[mb][nb][p], xa[p], wb[wcur][ws][nb][p]);
        next(p);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const int re = NR + 2 * q, im = re + 1;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const u32x4(&w)[T] = wb[wcur][ws][nb];
          const u32x4 neg = q8_neg(w[im]);
          q8_mfma(acc[mb][nb][re], xa[re], w[re]);
          q8_mfma(acc[mb][nb][im], xa[re], w[im]);
          q8_mfma(acc[mb][nb][re], xa[im], neg);
          q8_mfma(acc[mb][nb][im], xa[im], w[re]);
        }
        next(re);
        next(im);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  // What the epilogue reads of the output channels, and where registers are left its first residuals.
  float ws[NB][F], bias[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int col = (block0 + nb) * 32 + lrow;
#pragma unroll
    for (int f = 0; f < F; ++f) ws[nb][f] = a.wScales[(int64_t)f * a.Dpad + min(col, a.Dpad - 1)];
    bias[nb] = a.f.bias ? (float)static_cast<const Elt*>(a.f.bias)[min(col, a.f.Dout - 1)] : 0.0f;
  }
  if constexpr (EARLY)
    if (a.f.res) load_res(0);
  __builtin_amdgcn_sched_barrier(0);
  issue_rows(0, ring0, 0, PER);
  __builtin_amdgcn_sched_barrier(0);
  issue_rows(1, ring1, 0, PER);
  __builtin_amdgcn_sched_barrier(0);
  load_w(0, wb[0], 0, WLOADS);
  issue_rows(2, ring2, 0, PER);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<(2 * PER + WLOADS < 63 ? 2 * PER + WLOADS : 63)>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int p = 0; p < T; ++p) read_row(ring0, 0, 0, p);
  using Yes = std::true_type;
  using No = std::false_type;
  for (int kb = 0;;) {
    stage(kb, I0{}, No{});
    if (++kb == last) break;
    stage(kb, I1{}, No{});
    if (++kb == last) break;
    stage(kb, I2{}, No{});
    if (++kb == last) break;
    stage(kb, I3{}, No{});
    if (++kb == last) break;
  }
  if constexpr (WHOLE) {
    if (last & 1) {
#pragma unroll
      for (int i = 0; i < WLOADS; ++i) wb[0][i / (NB * T)][i / T % NB][i % T] = wb[1][i / (NB * T)][i / T % NB][i % T];
    }
  }
  stage(last, I0{}, Yes{});

  auto finish = [&](auto geluTag, auto resTag) __attribute__((always_inline)) {
    constexpr bool GELU = decltype(geluTag)::value, RES = decltype(resTag)::value;
#pragma unroll
    for (int i = 0; i < NB * MB * PARTS; ++i) {
      const int nb = i / PARTS / MB, mb = i / PARTS % MB, c = i % PARTS * CH;
      if (RES && i + 1 < NB * MB * PARTS) load_res(i + 1);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int r = c + j, row = mb * 32 + 4 * (lane >> 5) + 8 * (r >> 2) + (r & 3);
        int32_t sum[T];
        float scale[F], y[T], v[T] = {};
#pragma unroll
        for (int p = 0; p < T; ++p) sum[p] = acc[mb][nb][p][r];
#pragma unroll
        for (int f = 0; f < F; ++f) scale[f] = ws[nb][f] * rowScale[row * F + f];
        q8_outputs<T>(sum, scale, bias[nb], y, a.f.tw);
        if constexpr (RES) group_from_raw<T, Elt>(res[i & 1][j], v);
#pragma unroll
        for (int g = 0; g < T; ++g) y[g] = (GELU ? gelu_power(y[g]) : y[g]) + (RES ? v[g] : 0.0f);
        store_group_buf<T, Elt>(yr, offset_of(nb, mb, r), y);
        // A few rows at a time: all interleaved, their sums leave the accumulators together and spill.
        if (T > 8 || (j & 3) == 3) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  if (a.f.res) {
    if constexpr (!EARLY && !WHOLE) load_res(0);
    if (a.f.act == 1) finish(Yes{}, Yes{});
    else finish(No{}, Yes{});
  } else {
    if (a.f.act == 1) finish(Yes{}, No{});
    else finish(No{}, No{});
  }
#endif
}

}  // namespace eql
