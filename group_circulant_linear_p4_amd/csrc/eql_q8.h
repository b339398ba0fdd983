// 8-bit integer rows and weights of the EQ-Linear layer: their layout, and the kernels that
// write them.
//
// The layer is one channel product per frequency of the group axis ("Abordagem Algoritmica" in
// "Resumo Tecnico: Flash EQ-Linear"), so what goes into 8 bits is the half spectrum: the products
// keep their 2 T / T^2 share of the dense layer's operations and each runs on integers.  (On 8-bit
// group values the transform would leave 8 bits: four codes add up to ten.)  With the planes of
// eql_device.h, every row n has for each frequency f (f < NR: plane f; then one for each Re / Im pair)
//     m = max over channels of |plane| (both planes of a pair), at least 2^-100,
//     code = plane * (127 * (1 / m)) rounded to nearest even,  scale[n][f] = m / 127
// with the reciprocal and each product rounded to fp32,
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

// m / 127 rounded to nearest: the quotient by the rounded 1 / 127, and one correction (all 2^23 mantissas agree with the
// division, which takes 11 operations).
__device__ __forceinline__ float q8_scale(float m) {
  constexpr float inv = 1.0f / 127.0f;
  const float q = m * inv;
  return __builtin_fmaf(__builtin_fmaf(-127.0f, q, m), inv, q);
}

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

// Each frequency's largest magnitude: the largest of the positive values' bits and of the negative ones' (a NaN's
// is above infinity's).  As signed and unsigned integers the instruction that takes three operands does both without
// the mask: an operation a value instead of two.
template <int F>
struct Q8Top {
  int32_t pos[F];
  uint32_t neg[F];
  __device__ __forceinline__ Q8Top() {
#pragma unroll
    for (int f = 0; f < F; ++f) pos[f] = 0, neg[f] = 0;
  }
  __device__ __forceinline__ void take(int f, float v) {
    pos[f] = max(pos[f], __builtin_bit_cast(int32_t, v));
    neg[f] = max(neg[f], __builtin_bit_cast(uint32_t, v));
  }
  __device__ __forceinline__ uint32_t bits(int f) const { return max((uint32_t)pos[f], neg[f] & 0x7FFFFFFFu); }
};

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

// Sum of squares of a row from those of its chunks, in one order for every arrangement: chunk j lies on lane j % LPR as
// its piece j / LPR, and the sums are joined bit by bit of j from the highest down (a missing chunk adds a zero, which
// changes nothing).  How many lanes take a row depends on N (q8_shape), and with it would the last bit of a sum that each
// arrangement takes in its own order: 1 / rms, which goes into every scale, differed for one row in six between
// batches of 4096 and 4097 rows.
template <int K>
__device__ __forceinline__ float chunk_sum(float (&q)[K]) {
#pragma unroll
  for (int s = K / 2; s > 0; s /= 2)
#pragma unroll
    for (int i = 0; i < s; ++i) q[i] += q[i + s];
  return q[0];
}
// The lanes' part, on every lane (LPR 16 or 64).  Where the higher bits are joined already, a rotation within a row of 16
// lanes is an exchange.
template <int LPR>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (LPR == 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
    const auto q = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)q[0]) + __builtin_bit_cast(float, (uint32_t)q[1]);
  }
  v = dpp_add<0x128>(v);  // 8 lanes on
  v = dpp_add<0x124>(v);
  v = dpp_add<0x122>(v);
  return dpp_add<0x121>(v);
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

// E elements as they lie in memory.
template <typename Elt, int E>
constexpr int q8_words() {
  return (E * (int)sizeof(Elt) + 3) / 4;
}
// The E elements at p (at element alignment), or its first n where a chunk may have a TAIL: pieces of 16 bytes, then 8, 4 and 2.
template <typename Elt, int E, int FROM = 0>
__device__ __forceinline__ void load_words(const Elt* p, uint32_t (&w)[q8_words<Elt, E>()]) {
  constexpr int LEFT = E * (int)sizeof(Elt) - FROM * 4, N = LEFT >= 16 ? 4 : (LEFT >= 8 ? 2 : 1);
  if constexpr (LEFT >= 4) {
    typedef uint32_t UN __attribute__((ext_vector_type(N), aligned(sizeof(Elt))));
    const UN u = *reinterpret_cast<const UN*>(reinterpret_cast<const char*>(p) + FROM * 4);
#pragma unroll
    for (int e = 0; e < N; ++e) w[FROM + e] = u[e];
    load_words<Elt, E, FROM + N>(p, w);
  } else if constexpr (LEFT == 2) {
    w[FROM] = __builtin_bit_cast(uint16_t, p[E - 1]);
  }
}
template <typename Elt, int E, bool TAIL>
__device__ __forceinline__ void load_some(const Elt* p, int n, uint32_t (&w)[q8_words<Elt, E>()]) {
#pragma unroll
  for (int i = 0; i < q8_words<Elt, E>(); ++i) w[i] = 0;
  if (n >= E) {
    load_words<Elt, E>(p, w);
  } else if (TAIL && n > 0) {
#pragma unroll
    for (int e = 0; e < E - 1; ++e)
      if (e < n) {
        if constexpr (sizeof(Elt) == 2) w[e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[e]) << (e % 2 * 16);
        else w[e] = __builtin_bit_cast(uint32_t, p[e]);
      }
  }
}
template <typename Elt>
__device__ __forceinline__ float word_elt(const uint32_t* w, int e) {
  if constexpr (sizeof(Elt) == 2) return (float)__builtin_bit_cast(Elt, (uint16_t)(w[e / 2] >> (e % 2 * 16)));
  else return __builtin_bit_cast(float, w[e]);
}
// Floats to the E elements at p.
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

// A lane's K chunks of a row (LANES lanes apart), as they lie in memory, and the norm's weight for them.  All loads
// first: the sum that is stored may be x or the residual, so no later load passes it, and the weight in whole words
// (16384 rows of 2000 channels, T = 1 fp16, the norm: 42 us; chunk by chunk, the weight channel by channel, 96).
template <typename Elt, int T, int K>
struct Q8Chunks {
  static constexpr int CH = q8_chunk(T, sizeof(Elt)), E = CH * T;
  uint32_t x[K][q8_words<Elt, E>()], r[K][q8_words<Elt, E>()], g[K][q8_words<Elt, CH>()];
};
template <typename Elt, int T, int K>
__device__ __forceinline__ void q8_weight(const Q8RowsArgs& a, int c, int lanes, Q8Chunks<Elt, T, K>& u) {
  constexpr int CH = q8_chunk(T, sizeof(Elt));
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int c0 = (c + i * lanes) * CH;
    if (a.gamma) load_some<Elt, CH, (CH > 1)>(static_cast<const Elt*>(a.gamma) + c0, a.C - c0, u.g[i]);
  }
}
// `again`: the second reading of a row that is not held in registers.
template <typename Elt, int T, int K>
__device__ __forceinline__ void q8_load(const Q8RowsArgs& a, int64_t row, bool live, int c, int lanes, bool again, Q8Chunks<Elt, T, K>& u) {
  constexpr int CH = q8_chunk(T, sizeof(Elt)), E = CH * T;
  const int64_t at = row * ((int64_t)a.C * T);
  const bool kept = again && a.sum;
  const Elt* x = static_cast<const Elt*>(kept ? a.sum : a.x) + at;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int c0 = (c + i * lanes) * CH;
    load_some<Elt, E, (CH > 1)>(x + (int64_t)c0 * T, live ? (a.C - c0) * T : 0, u.x[i]);
  }
  if (kept || !a.res) return;
  const Elt* r = static_cast<const Elt*>(a.res) + at;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int c0 = (c + i * lanes) * CH;
    load_some<Elt, E, (CH > 1)>(r + (int64_t)c0 * T, live ? (a.C - c0) * T : 0, u.r[i]);
  }
}
// Chunk i's values (zero past C) after the residual's addition, which it stores; `sq` collects the sum of their squares.
template <typename Elt, int T, int K>
__device__ __forceinline__ void q8_values(const Q8RowsArgs& a, int64_t row, bool live, int c0, bool again, const Q8Chunks<Elt, T, K>& u,
                                          int i, float (&v)[q8_chunk(T, sizeof(Elt)) * T], float& sq) {
  constexpr int E = q8_chunk(T, sizeof(Elt)) * T;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = word_elt<Elt>(u.x[i], e);
  if (a.res && !(again && a.sum)) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (float)(Elt)(v[e] + word_elt<Elt>(u.r[i], e));
  }
  if (again) return;
  if (a.norm) {
#pragma unroll
    for (int e = 0; e < E; ++e) sq = __builtin_fmaf(v[e], v[e], sq);
  }
  if (!a.sum || !live) return;
  Elt* out = static_cast<Elt*>(a.sum) + row * ((int64_t)a.C * T) + (int64_t)c0 * T;
  const int n = (a.C - c0) * T;
  if (n >= E) {
    store_elts<Elt, E>(out, v);
  } else if (q8_chunk(T, sizeof(Elt)) > 1 && n > 0) {
#pragma unroll
    for (int e = 0; e < E - 1; ++e)
      if (e < n) out[e] = (Elt)v[e];
  }
}

// That chunk's planes, times the norm's weight.
template <typename Elt, int T>
__device__ __forceinline__ void q8_planes(const Q8RowsArgs& a, const uint32_t* gam, const float (&v)[q8_chunk(T, sizeof(Elt)) * T],
                                          float (&pl)[T][q8_chunk(T, sizeof(Elt))], Q8Top<n_freqs(T)>& top) {
  constexpr int CH = q8_chunk(T, sizeof(Elt));
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float g[T], o[T];
#pragma unroll
    for (int t = 0; t < T; ++t) g[t] = v[c * T + t];
    Dft<T>::run(g, o, a.tw);
#pragma unroll
    for (int p = 0; p < T; ++p) pl[p][c] = o[p];
  }
  if (a.gamma) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const float w = word_elt<Elt>(gam, c);
#pragma unroll
      for (int p = 0; p < T; ++p) pl[p][c] *= w;
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int p = 0; p < T; ++p) top.take(freq_of(T, p), pl[p][c]);
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
// registers between the maxima and the codes.  Bound by memory, with the vector unit close behind (some 300 operations a
// wave and 1024 values): 65536 rows of 1024 channels, T = 4 fp16, 144 us (5.6 TB/s), 12608 rows of 384 13.1 (4.4 TB/s;
// 11.9 where the rows are in the last-level cache); the norm with a residual, 50176 rows of 192, 50 us (5.4 TB/s).
template <typename Elt, int T, int LPR, int K>
__global__ void __launch_bounds__(256) eql_q8_rows_kernel(const Q8RowsArgs a) {
  constexpr int G = 256 / LPR, CH = q8_chunk(T, sizeof(Elt)), F = n_freqs(T), W = LPR / 64;
  static_assert(LPR == 16 || LPR == 64 || LPR == 256, "lane_sum");
  __shared__ uint32_t redTop[2][W > 1 ? F * W : 1];
  __shared__ float redSq[2][W > 1 ? 256 : 1];
  const int lane = (int)threadIdx.x % LPR, grp = (int)threadIdx.x / LPR;
  int turn = 0;
  Q8Chunks<Elt, T, K> u;
  q8_weight(a, lane, LPR, u);
  for (int64_t base = (int64_t)blockIdx.x * G; base < a.N; base += (int64_t)gridDim.x * G, turn ^= 1) {
    const int64_t row = base + grp;
    const bool live = row < a.N;
    q8_load(a, row, live, lane, LPR, false, u);
    float pl[K][T][CH];
    Q8Top<F> tops;
    float sqs[K] = {};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float v[CH * T];
      q8_values(a, row, live, (lane + i * LPR) * CH, false, u, i, v, sqs[i]);
      q8_planes<Elt, T>(a, u.g[i], v, pl[i], tops);
    }
    uint32_t top[F];
#pragma unroll
    for (int f = 0; f < F; ++f) top[f] = row_max<(LPR < 64 ? LPR : 64)>(tops.bits(f));
    float sq = chunk_sum(sqs);
    if constexpr (W > 1) {
      const int wave = (int)threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int f = 0; f < F; ++f) redTop[turn][f * W + wave] = top[f];
      }
      redSq[turn][threadIdx.x] = sq;
      __syncthreads();
      const float* q = &redSq[turn][threadIdx.x & 63];
      sq = (q[0] + q[128]) + (q[64] + q[192]);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        top[f] = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) top[f] = max(top[f], redTop[turn][f * W + w]);
      }
    }
    const float rstd = a.norm ? inv_sqrt(__builtin_fmaf(lane_sum<(LPR < 64 ? LPR : 64)>(sq), a.invR, a.eps)) : 1.0f;
    float inv[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const float m = q8_top(top[f]);
      inv[f] = q8_inv(m);
      if (live && lane == 0) a.scales[row * F + f] = q8_scale(m) * rstd;
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
  Q8Top<F> tops;
  float sq = 0.0f;
  for (int c0 = (int)threadIdx.x * CH; c0 < a.C; c0 += 256 * CH) {
    float v[CH * T], pl[T][CH];
    Q8Chunks<Elt, T, 1> u;
    q8_weight(a, c0 / CH, 0, u);
    q8_load(a, row, true, c0 / CH, 0, false, u);
    q8_values(a, row, true, c0, false, u, 0, v, sq);
    q8_planes<Elt, T>(a, u.g[0], v, pl, tops);
  }
  const int wave = (int)threadIdx.x >> 6;
  sq = row_sum<64>(sq);
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const uint32_t top = row_max<64>(tops.bits(f));
    if ((threadIdx.x & 63) == 0) redTop[f * 4 + wave] = top;
  }
  if ((threadIdx.x & 63) == 0) {
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
    if (threadIdx.x == 0) a.scales[row * F + f] = q8_scale(m) * rstd;
  }
  for (int c0 = (int)threadIdx.x * CH; c0 < a.pitch; c0 += 256 * CH) {
    float v[CH * T], pl[T][CH], none = 0.0f;
    Q8Top<F> unused;
    Q8Chunks<Elt, T, 1> u;
    q8_weight(a, c0 / CH, 0, u);
    q8_load(a, row, true, c0 / CH, 0, true, u);
    q8_values(a, row, true, c0, true, u, 0, v, none);
    q8_planes<Elt, T>(a, u.g[0], v, pl, unused);
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
  Q8Top<F> top;
  for (int i = lane; i < live; i += 64) {
    float v[T], pl[T];
    load_group<T, Elt>(w + (int64_t)i * T, v);
    Dft<T>::run(v, pl, a.tw);
#pragma unroll
    for (int p = 0; p < T; ++p) top.take(freq_of(T, p), pl[p]);
  }
  float inv[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const float m = q8_top(row_max<64>(top.bits(f)));
    inv[f] = q8_inv(m);
    if (lane == 0) a.scales[(int64_t)f * a.Dpad + o] = o < a.D ? q8_scale(m) * (f < NR ? 1.0f : 2.0f) / (float)T : 0.0f;
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
