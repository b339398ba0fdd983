// 8-bit integer rows and weights of the EQ-Linear layer: their layout, and the kernels that
// write them.
//
// The layer is one channel product per frequency of the group axis ("Abordagem Algoritmica" in
// "Resumo Tecnico: Flash EQ-Linear"), so what goes into 8 bits is the half spectrum: the products
// keep their 2 T / T^2 share of the dense layer's operations and each runs on integers.  (On 8-bit
// group values the transform would leave 8 bits: four codes add up to ten.)  With the planes of
// eql_device.h, every row n has for each frequency f (f < NR: plane f; then one for each Re / Im pair)
//     m = max over channels of |plane| (both planes of a pair), at least 2^-100,
//     code = plane * (127 (1 / m)) rounded to nearest even,  scale[n][f] = m / 127,
// and the weight the same for each output channel, with the inverse transform's 1 / T (pairs: 2 / T)
// in its scales.  A row with an infinity or a NaN among a frequency's planes has the scale NaN there.
//
// Rows: N rows of T planes of P = 16 ceil(C / 16) bytes (zero past C), then N rows of F floats.
// Weight: see q8_weight_unit; then F rows of floats, one for each output channel of the padded 32s.
#pragma once

#include "eql_ckpt8.h"
#include "eql_norm.h"

namespace eql {

constexpr float kQ8Floor = 0x1p-100f;  // least m: a row of zeros has finite scales

__host__ __device__ constexpr int n_freqs(int T) { return n_real_planes(T) + n_pairs(T); }
// Frequency of a plane.
__host__ __device__ constexpr int freq_of(int T, int p) { return p < n_real_planes(T) ? p : n_real_planes(T) + (p - n_real_planes(T)) / 2; }

// Bytes of one plane of a row.
__host__ __device__ constexpr int64_t q8_pitch(int64_t C) { return (C + 15) / 16 * 16; }
// Input channels of a K block of the weight: two steps of a 32 x 32 x 32 product.
constexpr int kQ8Block = 64;
__host__ __device__ constexpr int64_t q8_blocks(int64_t C) { return (C + kQ8Block - 1) / kQ8Block; }
__host__ __device__ constexpr int64_t q8_out(int64_t D) { return (D + 31) / 32 * 32; }

// Byte of the weight's code for output channel o, input channel i, plane p: for each 32 output
// channels and 64 input channels T planes of two 1 KB matrix operands (input channels 0..31 and
// 32..63), in which lane l holds output channel l % 32 and 16 input channels from 16 (l / 32) on: a
// wave's operand load is 1 KB in one piece.
__host__ __device__ inline size_t q8_weight_unit(int o, int i, int p, int T, int kblocks) {
  const int ob = o / 32, ol = o % 32, kb = i / kQ8Block, il = i % kQ8Block;
  return ((((size_t)ob * kblocks + kb) * T + p) * 2 + il / 32) * 1024 + (size_t)((il % 32 / 16) * 32 + ol) * 16 + il % 16;
}

// m's bits (a float's without its sign) to m held at the floor; NaN for an infinity or a NaN.
__device__ __forceinline__ float q8_top(uint32_t bits) {
  return bits >= 0x7F800000u ? __builtin_nanf("") : __builtin_fmaxf(__builtin_bit_cast(float, bits), kQ8Floor);
}

// 127 / m as the codes are defined: the reciprocal and the product each rounded.
__device__ __forceinline__ float q8_inv(float m) { return 127.0f * (1.0f / m); }

// Four codes as a word, of values times their 127 / m.  The product is rounded to fp32, then adding 1.5 2^23 rounds it
// to an integer (ties to even), which is in the sum's low bits.  With inv a NaN the codes are not
// specified (their scale is NaN).
__device__ __forceinline__ uint32_t q8_encode4(float a, float b, float c, float d) {
  const uint32_t w0 = __builtin_bit_cast(uint32_t, a + 12582912.0f), w1 = __builtin_bit_cast(uint32_t, b + 12582912.0f);
  const uint32_t w2 = __builtin_bit_cast(uint32_t, c + 12582912.0f), w3 = __builtin_bit_cast(uint32_t, d + 12582912.0f);
  const uint32_t lo = __builtin_amdgcn_perm(w1, w0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(w3, w2, 0x04000c0cu);
  return lo | hi;
}

// Transposes the 4 x 4 bytes of a quad of lanes: lane i gets byte i of each lane's word, lane 0's lowest.
__device__ __forceinline__ uint32_t quad_transpose(uint32_t w) {
  const int i = (int)threadIdx.x & 3;
  // Lanes 1 apart: even lanes keep their bytes 0 and 2 and take the other's, odd ones 1 and 3.
  const uint32_t o = dpp_move<kDppXor1>(w);
  w = __builtin_amdgcn_perm(o, w, i & 1 ? 0x03070105u : 0x06020400u);
  // Lanes 2 apart: lanes 0 and 1 keep the low halves, lanes 2 and 3 the high ones.
  const uint32_t q = dpp_move<kDppXor2>(w);
  return __builtin_amdgcn_perm(q, w, i & 2 ? 0x03020706u : 0x05040100u);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

// Largest of the LPR lanes of a row (LPR <= 64), on every lane.
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp_move<kDppXor1>(v));
  v = max(v, dpp_move<kDppXor2>(v));
  if constexpr (LPR >= 8) v = max(v, dpp_move<kDppMirror8>(v));
  if constexpr (LPR >= 16) v = max(v, dpp_move<kDppMirror16>(v));
  if constexpr (LPR >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)p[0], (uint32_t)p[1]);
  }
  if constexpr (LPR >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)p[0], (uint32_t)p[1]);
  }
  return v;
}

struct Q8RowsArgs {
  const void* x;      // [N][C*T]
  const void* res;    // [N][C*T] or null: added to x, the sum rounded to the element type
  const void* gamma;  // [C] or null (1): the norm's weight
  void* sum;          // [N][C*T] or null: receives that sum (may be x or res)
  unsigned char* codes;  // [N][T][pitch]
  float* scales;         // [N][F]
  int64_t N;
  int C, pitch;
  int norm;           // 1: rows are divided by their root mean square (in the scales)
  float eps, invR;
  Twiddles tw;
};

// Channels that a lane takes at a time.  Where 4 to 16 of them are at most 32 bytes, as many (whole words of codes);
// else one, and a quad of lanes exchanges bytes to make words: with more bytes between neighbouring lanes a load
// touches a line a lane (16384 rows of 64 channels, T = 8 fp32, the norm: 69 us with four channels a lane).
__host__ __device__ constexpr int q8_chunk(int T, int elt) {
  return elt == 2 ? (T == 1 ? 16 : (T == 2 ? 8 : (T <= 4 ? 4 : 1))) : (T == 1 ? 8 : (T == 2 ? 4 : 1));
}
// Chunks that a lane holds at most (64 values), and where a row is not spread over more lanes (32).
__host__ __device__ constexpr int q8_keep(int T, int elt) {
  const int n = 64 / (q8_chunk(T, elt) * T);
  return n >= 8 ? 8 : 4;
}
__host__ __device__ constexpr int q8_some(int T, int elt) {
  const int n = 32 / (q8_chunk(T, elt) * T);
  return n >= 4 ? 4 : (n >= 2 ? 2 : 1);
}

// The E elements at p (at element alignment) to floats, and back: pieces of 16 bytes, then 4, 2 and 1.
template <typename Elt, int E, int FROM = 0>
__device__ __forceinline__ void load_elts(const Elt* p, float (&v)[E]) {
  constexpr int N = E - FROM >= 8 && sizeof(Elt) == 2 ? 8 : (E - FROM >= 4 ? 4 : (E - FROM >= 2 ? 2 : 1));
  if constexpr (E - FROM > 0) {
    if constexpr (N == 1) {
      v[FROM] = (float)p[FROM];
    } else {
      typedef Elt EN __attribute__((ext_vector_type(N), aligned(sizeof(Elt))));
      const EN u = *reinterpret_cast<const EN*>(p + FROM);
#pragma unroll
      for (int e = 0; e < N; ++e) v[FROM + e] = (float)u[e];
    }
    load_elts<Elt, E, FROM + N>(p, v);
  }
}
template <typename Elt, int E, int FROM = 0>
__device__ __forceinline__ void store_elts(Elt* p, const float (&v)[E]) {
  constexpr int N = E - FROM >= 8 && sizeof(Elt) == 2 ? 8 : (E - FROM >= 4 ? 4 : (E - FROM >= 2 ? 2 : 1));
  if constexpr (E - FROM > 0) {
    if constexpr (N == 1) {
      p[FROM] = (Elt)v[FROM];
    } else {
      typedef Elt EN __attribute__((ext_vector_type(N), aligned(sizeof(Elt))));
      EN u;
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] = (Elt)v[FROM + e];
      __builtin_nontemporal_store(u, reinterpret_cast<EN*>(p + FROM));
    }
    store_elts<Elt, E, FROM + N>(p, v);
  }
}

// Chunk at channel c0 of a row: its values (zero past C) after the residual's addition, which it
// stores.  `again`: the second reading of a row that is not held in registers.
template <typename Elt, int T>
__device__ __forceinline__ void q8_load(const Q8RowsArgs& a, int64_t row, int c0, bool again, float (&v)[q8_chunk(T, sizeof(Elt)) * T]) {
  constexpr int CH = q8_chunk(T, sizeof(Elt)), E = CH * T;
  const int64_t at = row * ((int64_t)a.C * T) + (int64_t)c0 * T;
  const bool kept = again && a.sum;
  const Elt* x = static_cast<const Elt*>(kept ? a.sum : a.x) + at;
  const Elt* r = kept || !a.res ? nullptr : static_cast<const Elt*>(a.res) + at;
  Elt* out = again || !a.sum ? nullptr : static_cast<Elt*>(a.sum) + at;
  if (c0 + CH <= a.C) {
    load_elts<Elt, E>(x, v);
    if (r) {
      float u[E];
      load_elts<Elt, E>(r, u);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = (float)(Elt)(v[e] + u[e]);
    }
    if (out) store_elts<Elt, E>(out, v);
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int e = c * T + t;
        float q = 0.0f;
        if (c0 + c < a.C) {
          q = (float)x[e];
          if (r) q = (float)(Elt)(q + (float)r[e]);
          if (out) out[e] = (Elt)q;
        }
        v[e] = q;
      }
  }
}

// That chunk's planes, times the norm's weight; `top` collects each frequency's largest magnitude,
// `sq` the sum of squares of the values.
template <typename Elt, int T>
__device__ __forceinline__ void q8_planes(const Q8RowsArgs& a, int c0, const float (&v)[q8_chunk(T, sizeof(Elt)) * T],
                                          float (&pl)[T][q8_chunk(T, sizeof(Elt))], uint32_t (&top)[n_freqs(T)], float& sq) {
  constexpr int CH = q8_chunk(T, sizeof(Elt));
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float g[T], o[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      g[t] = v[c * T + t];
      sq = __builtin_fmaf(g[t], g[t], sq);
    }
    Dft<T>::run(g, o, a.tw);
    if (a.gamma) {
      const float w = (float)static_cast<const Elt*>(a.gamma)[min(c0 + c, a.C - 1)];
#pragma unroll
      for (int p = 0; p < T; ++p) o[p] *= w;
    }
#pragma unroll
    for (int p = 0; p < T; ++p) {
      pl[p][c] = o[p];
      top[freq_of(T, p)] = max(top[freq_of(T, p)], abs_bits(o[p]));
    }
  }
}

template <typename Elt, int T>
__device__ __forceinline__ void q8_store(const Q8RowsArgs& a, int64_t row, int c0, const float (&pl)[T][q8_chunk(T, sizeof(Elt))],
                                         const float (&inv)[n_freqs(T)]) {
  constexpr int CH = q8_chunk(T, sizeof(Elt)), W = CH / 4;
  if (c0 >= a.pitch) return;  // whole quads: rows of codes are multiples of 16
  unsigned char* out = a.codes + row * ((int64_t)a.pitch * T);
  if constexpr (CH == 1) {
    const int lane = (int)threadIdx.x & 3;
#pragma unroll
    for (int p0 = 0; p0 < T; p0 += 4) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p0 + i < T ? pl[p0 + i < T ? p0 + i : 0][0] * inv[freq_of(T, p0 + i < T ? p0 + i : 0)] : 0.0f;
      const uint32_t w = quad_transpose(q8_encode4(v[0], v[1], v[2], v[3]));
      if (p0 + lane < T) *reinterpret_cast<uint32_t*>(out + (p0 + lane) * a.pitch + (c0 & ~3)) = w;
    }
  } else {
#pragma unroll
    for (int p = 0; p < T; ++p) {
      const float f = inv[freq_of(T, p)];
      uint32_t w[W];
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = q8_encode4(pl[p][4 * i] * f, pl[p][4 * i + 1] * f, pl[p][4 * i + 2] * f, pl[p][4 * i + 3] * f);
      unsigned char* q = out + p * a.pitch + c0;
      if constexpr (W == 4) *reinterpret_cast<u32x4*>(q) = (u32x4){w[0], w[1], w[2], w[3]};
      else if constexpr (W == 2) *reinterpret_cast<u32x2*>(q) = (u32x2){w[0], w[1]};
      else *reinterpret_cast<uint32_t*>(q) = w[0];
    }
  }
}

// Rows to 8 bits: LPR lanes a row, K chunks a lane.  One read of each operand; the planes stay in
// registers between the maxima and the codes.  Bound by memory: 65536 rows of 1024 channels, T = 4 fp16, 139 us (5.8 TB/s);
// the norm with a residual, 50176 rows of 192, 57 us (4.8 TB/s).
template <typename Elt, int T, int LPR, int K>
__global__ void __launch_bounds__(256) eql_q8_rows_kernel(const Q8RowsArgs a) {
  constexpr int G = 256 / LPR, CH = q8_chunk(T, sizeof(Elt)), F = n_freqs(T), W = LPR / 64;
  __shared__ uint32_t redTop[2][W > 1 ? F * W : 1];
  __shared__ float redSq[2][W > 1 ? W : 1];
  const int lane = (int)threadIdx.x % LPR, grp = (int)threadIdx.x / LPR;
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * G; base < a.N; base += (int64_t)gridDim.x * G, turn ^= 1) {
    const int64_t row = base + grp;
    const bool live = row < a.N;
    float pl[K][T][CH];
    uint32_t top[F];
    float sq = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f) top[f] = 0;
    {
      float v[K][CH * T];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int c0 = (lane + i * LPR) * CH;
        if (live && c0 < a.C) {
          q8_load<Elt, T>(a, row, c0, false, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < CH * T; ++e) v[i][e] = 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < K; ++i) q8_planes<Elt, T>(a, (lane + i * LPR) * CH, v[i], pl[i], top, sq);
    }
#pragma unroll
    for (int f = 0; f < F; ++f) top[f] = row_max<(LPR < 64 ? LPR : 64)>(top[f]);
    sq = row_sum<(LPR < 64 ? LPR : 64)>(sq);
    if constexpr (W > 1) {
      const int wave = (int)threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int f = 0; f < F; ++f) redTop[turn][f * W + wave] = top[f];
        redSq[turn][wave] = sq;
      }
      __syncthreads();
      sq = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) sq += redSq[turn][w];
#pragma unroll
      for (int f = 0; f < F; ++f) {
        top[f] = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) top[f] = max(top[f], redTop[turn][f * W + w]);
      }
    }
    const float rstd = a.norm ? inv_sqrt(__builtin_fmaf(sq, a.invR, a.eps)) : 1.0f;
    float inv[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const float m = q8_top(top[f]);
      inv[f] = q8_inv(m);
      if (live && lane == 0) a.scales[row * F + f] = m / 127.0f * rstd;
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < K; ++i) q8_store<Elt, T>(a, row, (lane + i * LPR) * CH, pl[i], inv);
    }
  }
}

// Rows longer than the registers hold: a workgroup a row, which reads it twice (the second time from
// cache).
template <typename Elt, int T>
__global__ void __launch_bounds__(256) eql_q8_rows_wide_kernel(const Q8RowsArgs a) {
  constexpr int CH = q8_chunk(T, sizeof(Elt)), F = n_freqs(T);
  __shared__ uint32_t redTop[F * 4];
  __shared__ float redSq[4];
  const int64_t row = blockIdx.x;
  uint32_t top[F];
  float sq = 0.0f;
#pragma unroll
  for (int f = 0; f < F; ++f) top[f] = 0;
  for (int c0 = (int)threadIdx.x * CH; c0 < a.C; c0 += 256 * CH) {
    float v[CH * T], pl[T][CH];
    q8_load<Elt, T>(a, row, c0, false, v);
    q8_planes<Elt, T>(a, c0, v, pl, top, sq);
  }
  const int wave = (int)threadIdx.x >> 6;
  sq = row_sum<64>(sq);
#pragma unroll
  for (int f = 0; f < F; ++f) top[f] = row_max<64>(top[f]);
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int f = 0; f < F; ++f) redTop[f * 4 + wave] = top[f];
    redSq[wave] = sq;
  }
  __syncthreads();
  sq = redSq[0] + redSq[1] + redSq[2] + redSq[3];
  const float rstd = a.norm ? inv_sqrt(__builtin_fmaf(sq, a.invR, a.eps)) : 1.0f;
  float inv[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const float m = q8_top(max(max(redTop[f * 4], redTop[f * 4 + 1]), max(redTop[f * 4 + 2], redTop[f * 4 + 3])));
    inv[f] = q8_inv(m);
    if (threadIdx.x == 0) a.scales[row * F + f] = m / 127.0f * rstd;
  }
  for (int c0 = (int)threadIdx.x * CH; c0 < a.pitch; c0 += 256 * CH) {
    float v[CH * T], pl[T][CH], none = 0.0f;
    uint32_t unused[F];
#pragma unroll
    for (int f = 0; f < F; ++f) unused[f] = 0;
    if (c0 < a.C) {
      q8_load<Elt, T>(a, row, c0, true, v);
    } else {
#pragma unroll
      for (int e = 0; e < CH * T; ++e) v[e] = 0.0f;
    }
    q8_planes<Elt, T>(a, c0, v, pl, unused, none);
    q8_store<Elt, T>(a, row, c0, pl, inv);
  }
}

// The weight to 8 bits: a wave an output channel, in two readings (maxima, codes); the padding of
// both axes has code and scale zero.  Done once for a weight (1024 -> 1024 channels, T = 4 fp16: 15 us).
struct Q8PackArgs {
  const void* w;         // [D][C][T]
  unsigned char* codes;  // q8_weight_unit
  float* scales;         // [F][Dpad]
  int D, C, Dpad, kblocks;
  Twiddles tw;
};

template <typename Elt, int T>
__global__ void __launch_bounds__(256) eql_q8_pack_kernel(const Q8PackArgs a) {
  constexpr int F = n_freqs(T), NR = n_real_planes(T);
  const int o = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
  if (o >= a.Dpad) return;
  const Elt* w = static_cast<const Elt*>(a.w) + (int64_t)o * a.C * T;
  const int live = o < a.D ? a.C : 0;
  uint32_t top[F];
#pragma unroll
  for (int f = 0; f < F; ++f) top[f] = 0;
  for (int i = lane; i < live; i += 64) {
    float v[T], pl[T];
    load_group<T, Elt>(w + (int64_t)i * T, v);
    Dft<T>::run(v, pl, a.tw);
#pragma unroll
    for (int p = 0; p < T; ++p) top[freq_of(T, p)] = max(top[freq_of(T, p)], abs_bits(pl[p]));
  }
  float inv[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const float m = q8_top(row_max<64>(top[f]));
    inv[f] = q8_inv(m);
    if (lane == 0) a.scales[(int64_t)f * a.Dpad + o] = o < a.D ? m / 127.0f * (f < NR ? 1.0f : 2.0f) / (float)T : 0.0f;
  }
  // Four input channels a lane, a word of each plane's codes.
  for (int i = lane * 4; i < a.kblocks * kQ8Block; i += 256) {
    float pl[4][T];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float v[T];
#pragma unroll
      for (int t = 0; t < T; ++t) v[t] = 0.0f;
      if (i + c < live) load_group<T, Elt>(w + (int64_t)(i + c) * T, v);
      Dft<T>::run(v, pl[c], a.tw);
    }
#pragma unroll
    for (int p = 0; p < T; ++p) {
      const float f = inv[freq_of(T, p)];
      *reinterpret_cast<uint32_t*>(a.codes + q8_weight_unit(o, i, p, T, a.kblocks)) =
          q8_encode4(pl[0][p] * f, pl[1][p] * f, pl[2][p] * f, pl[3][p] * f);
    }
  }
}

}  // namespace eql
