// 8-bit activation checkpoints and the passes that read them.
//
// A training step keeps activations from the forward to the backward pass.  A checkpoint
// holds an [N][R] matrix (R = C'*T features a row) in about a quarter of fp32's bytes: blocks
// of 32 consecutive features of a row (the last one may be short) share one power-of-two step,
//     a = max |v| over the block,  e = the smallest integer >= -126 with a 2^-e < 127.5,
//     code = v 2^-e rounded to nearest even, in [-127, 127],   value = code 2^e,
// so the error is at most half a step, 2^(e-1) <= a / 127.  e stops at 121 (fp16 matrices: 9), the
// largest step of which the type holds 127: a block that would take the next one (a of 127.5 2^121
// or more; 65280 or more) keeps this one, its largest values become +-127 steps, still within
// a / 127, and everything that reads it sees finite values.  A power-of-two step makes both
// directions exact but for that one rounding: codes are the same whatever computed them, and a
// code's value is exact in fp32 and, for values of ordinary size, in fp16.  A block that holds
// an infinity or a NaN reads back as NaN throughout (a training step must not lose an
// overflow).  Layout: N rows of P = 32 ceil(R / 32) signed bytes (codes past R are zero), then
// N rows of P / 32 scale bytes e + 127 (255 marks the NaN block).
//
// Every kernel here streams its operands once.  A lane takes 8 consecutive features ("chunk":
// 16 bytes of fp16, 32 of fp32, 8 of codes), so a block is four neighbouring lanes and its
// maximum two cross-lane moves; rows of any length are read at the alignment of one element,
// which the hardware's global loads allow, so an odd row costs no narrower loads.
#pragma once

#include "eql_device.h"
#include "eql_fwd.h"

namespace eql {

constexpr int kCkptBlock = 32;
// Bytes of one row of codes.
__host__ __device__ constexpr int64_t ckpt_pitch(int64_t row) { return (row + kCkptBlock - 1) / kCkptBlock * kCkptBlock; }

// Eight elements at element alignment.
template <typename Elt>
struct Chunk;
template <>
struct Chunk<_Float16> {
  typedef _Float16 V __attribute__((ext_vector_type(8)));
  typedef _Float16 VU __attribute__((ext_vector_type(8), aligned(2)));
};
template <>
struct Chunk<float> {
  typedef float V __attribute__((ext_vector_type(8)));
  typedef float VU __attribute__((ext_vector_type(8), aligned(4)));
};

template <typename Elt>
__device__ __forceinline__ typename Chunk<Elt>::V zero_chunk() {
  return (typename Chunk<Elt>::V)(Elt)0;
}

// The chunk at p, of which `n` elements exist (the others are zero).  WHOLE: every chunk is
// whole or missing (R a multiple of 8), so no tail is compiled and rows are 16-byte aligned.
// STREAM: a non-temporal load, for operands that the caches cannot hold anyway; never of rows
// that start inside a line, whose lines two loads share.
template <typename Elt, bool WHOLE, bool STREAM>
__device__ __forceinline__ typename Chunk<Elt>::V load_chunk8(const Elt* p, int n) {
  typename Chunk<Elt>::V v = zero_chunk<Elt>();
  if (n >= 8) {
    const auto* q = reinterpret_cast<const typename Chunk<Elt>::VU*>(p);
    if constexpr (WHOLE && STREAM) v = __builtin_nontemporal_load(q);
    else v = *q;
  } else if (!WHOLE && n > 0) {
    // The row's last 1 to 7 elements as 4 + 2 + 1.
    typedef Elt E4 __attribute__((ext_vector_type(4), aligned(sizeof(Elt))));
    typedef Elt E2 __attribute__((ext_vector_type(2), aligned(sizeof(Elt))));
    E4 a = (E4)(Elt)0;
    E2 b = (E2)(Elt)0;
    Elt c = (Elt)0;
    if (n & 4) a = *reinterpret_cast<const E4*>(p);
    if (n & 2) b = *reinterpret_cast<const E2*>(p + (n & 4));
    if (n & 1) c = p[n & 6];
    const bool four = n & 4, two = n & 2;
    const Elt z = (Elt)0, r0 = two ? b[0] : c, r1 = two ? b[1] : z, r2 = two ? c : z;
    v[0] = four ? a[0] : r0;
    v[1] = four ? a[1] : r1;
    v[2] = four ? a[2] : r2;
    v[3] = four ? a[3] : z;
    v[4] = four ? r0 : z;
    v[5] = four ? r1 : z;
    v[6] = four ? r2 : z;
  }
  return v;
}

// Results are written past the caches, 16 bytes a lane: nothing in the same kernel reads them
// again (also where rows start inside a line: N = 19019, R = 1452 fp16, the norm's forward pass
// 30 us and 40 through the caches).  Codes, 8 bytes a lane, are not: as non-temporal stores they
// took that pass with its checkpoint at N = 65536, R = 4096 from 228 to 273 us.
template <typename Elt, bool WHOLE>
__device__ __forceinline__ void store_chunk8(Elt* p, int n, const float (&f)[8]) {
  typename Chunk<Elt>::VU v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (Elt)f[e];
  if (n >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<typename Chunk<Elt>::VU*>(p));
  } else if (!WHOLE && n > 0) {
    // As 4 + 2 + 1.
    typedef Elt E4 __attribute__((ext_vector_type(4), aligned(sizeof(Elt))));
    typedef Elt E2 __attribute__((ext_vector_type(2), aligned(sizeof(Elt))));
    const bool four = n & 4;
    const Elt g0 = four ? v[4] : v[0], g1 = four ? v[5] : v[1], g2 = four ? v[6] : v[2];
    if (four) *reinterpret_cast<E4*>(p) = (E4){v[0], v[1], v[2], v[3]};
    if (n & 2) *reinterpret_cast<E2*>(p + (n & 4)) = (E2){g0, g1};
    if (n & 1) p[n & 6] = n & 2 ? g2 : g0;
  }
}

// Eight codes at p (8-byte aligned: rows of codes are a multiple of 32 bytes).
template <bool STREAM>
__device__ __forceinline__ u32x2 load_codes8(const unsigned char* p) {
  const auto* q = reinterpret_cast<const u32x2*>(p);
  if constexpr (STREAM) return __builtin_nontemporal_load(q);
  else return *q;
}

// Cross-lane moves inside a row of 16 lanes (DPP): neighbours 1 and 2 apart in a quad, the
// mirror of 8 and of 16 lanes.
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, dpp_move<CTRL>(__builtin_bit_cast(uint32_t, v)));
}

// Largest |v| of a chunk, and over the quad of lanes that holds a block.  NaN loses against a
// number here; whether a block is finite is asked separately.
__device__ __forceinline__ float chunk_top(const float (&v)[8]) {
  float t = __builtin_fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1]));
#pragma unroll
  for (int e = 2; e < 8; ++e) t = __builtin_fmaxf(t, __builtin_fabsf(v[e]));
  return t;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, dpp_move<kDppXor1>(v));
  return max(v, dpp_move<kDppXor2>(v));
}

// A block's step from its largest magnitude (a finite float's bits): e + 127 as the exponent field
// of `top` less 6.  127.5 2^e has exponent e + 6 and mantissa field 0x7F0000, so adding 0x10000
// carries into the exponent exactly from there on; e is at least -126.
struct BlockStep {
  float back;      // 2^-e
  uint32_t scale;  // e + 127
};
__device__ __forceinline__ BlockStep block_step(uint32_t top) {
  const uint32_t t = max((top + 0x10000u) & 0x7F800000u, 7u << 23);
  return {__builtin_bit_cast(float, 0x82000000u - t), (t >> 23) - 6u};
}

// Codes of eight values, as two words.  v 2^-e + 1.5 2^23 in one fused operation: the product is
// exact, the sum rounds to the integer (ties to even), and the integer is in the low bits.
__device__ __forceinline__ u32x2 encode8(const float (&v)[8], float back) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = __builtin_bit_cast(uint32_t, __builtin_fmaf(v[e], back, 12582912.0f));
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(w[4 * h + 1], w[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(w[4 * h + 3], w[4 * h + 2], 0x04000c0cu);
    r[h] = lo | hi;
  }
  return r;
}

// The step 2^e of a scale byte (NaN for 255).
__device__ __forceinline__ float scale_step(uint32_t s) {
  return __builtin_bit_cast(float, s == 255u ? 0x7FC00000u : s << 23);
}

// Four codes of a word to values (exact: seven bits times a power of two).
__device__ __forceinline__ void decode4(uint32_t w, float step, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)(int)(int8_t)(w >> (8 * e)) * step;
}
__device__ __forceinline__ void decode8(u32x2 w, float step, float (&v)[8]) {
  decode4(w[0], step, v);
  decode4(w[1], step, v + 4);
}

struct CkptArgs {
  const void* x;          // pack: read; unpack: written (as void*)
  unsigned char* codes;   // [N][pitch]
  unsigned char* scales;  // [N][pitch / 32]
  int64_t chunks;         // N * pitch / 8
  int R, rowChunks;       // rowChunks = pitch / 8
};

// Flat order over the chunks of all rows (pitch / 8 a row, a multiple of four, so a block's
// four chunks are four neighbouring lanes).  A workgroup's first chunk is split into row and
// offset once, in 64 bits; a lane adds its own offset and divides in 32 bits.
__device__ __forceinline__ void chunk_place(const CkptArgs& a, int64_t first, int o, int64_t& row, int& f0, int& n) {
  const int64_t row0 = first / a.rowChunks;
  const uint32_t rest = (uint32_t)(first - row0 * a.rowChunks) + (uint32_t)o;
  const uint32_t dr = rest / (uint32_t)a.rowChunks;
  row = row0 + dr;
  f0 = (int)(rest - dr * (uint32_t)a.rowChunks) * 8;
  n = a.R - f0;
}

template <typename Elt, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(256) eql_ckpt_pack_kernel(const CkptArgs a) {
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t idx = first + threadIdx.x;
  if (idx >= a.chunks) return;  // a multiple of four: a quad is live or not as a whole
  int64_t row;
  int f0, n;
  chunk_place(a, first, (int)threadIdx.x, row, f0, n);
  const auto v = load_chunk8<Elt, WHOLE, STREAM>(static_cast<const Elt*>(a.x) + row * a.R + f0, n);
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
  // As bits, an infinity or a NaN compares above every finite magnitude.
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu);
  top = quad_max(top);
  BlockStep st = block_step(top);
  constexpr int last = sizeof(Elt) == 2 ? 9 : 121;  // the largest e
  if (st.scale > last + 127u) {
    constexpr float step = sizeof(Elt) == 2 ? 0x1p9f : 0x1p121f;
    st = {1.0f / step, last + 127u};
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_fminf(__builtin_fmaxf(f[e], -127.0f * step), 127.0f * step);
  }
  *reinterpret_cast<u32x2*>(a.codes + idx * 8) = encode8(f, st.back);
  if ((threadIdx.x & 3) == 0) a.scales[idx >> 2] = (unsigned char)(top >= 0x7F800000u ? 255u : st.scale);
}

template <typename Elt, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(256) eql_ckpt_unpack_kernel(const CkptArgs a) {
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t idx = first + threadIdx.x;
  if (idx >= a.chunks) return;
  int64_t row;
  int f0, n;
  chunk_place(a, first, (int)threadIdx.x, row, f0, n);
  const float step = scale_step(a.scales[idx >> 2]);
  float f[8];
  decode8(load_codes8<STREAM>(a.codes + idx * 8), step, f);
  store_chunk8<Elt, WHOLE>(static_cast<Elt*>(const_cast<void*>(a.x)) + row * a.R + f0, n, f);
}

// Backward of the bias + GELU epilogue with GELU's input read from a checkpoint:
//     dpre = dy GELU'(value),   part[row block][channel] = sum over the block's rows and t of dpre.
// A workgroup of 1024 threads takes `lanes` chunks across and `groups` = 1024 / lanes rows at a
// time down its block of rows, the next rows' operands in flight; the column sums of its row
// groups are added pairwise through LDS, then the T of each channel.
struct Epi8Args {
  const void* dy;
  const unsigned char* codes;
  const unsigned char* scales;
  void* dpre;  // may be dy
  float* part; // [rowBlocks][R / T], or null
  void* dbias; // [R / T]: written by the kernel itself (one row block), or null
  int64_t N;
  int R, T, pitch, lanes, groups, colBlocks, rowsPerBlock;
};
constexpr int kEpi8Threads = 1024;

template <typename Elt, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(kEpi8Threads) eql_epi8_kernel(const Epi8Args a) {
  __shared__ float red[8][kEpi8Threads];
  const int grp = (int)threadIdx.x / a.lanes, l = (int)threadIdx.x - grp * a.lanes;
  const int cb = (int)blockIdx.x % a.colBlocks, rb = (int)blockIdx.x / a.colBlocks;
  const int f0 = (cb * a.lanes + l) * 8;
  const int n = a.R - f0;
  const int64_t r0 = (int64_t)rb * a.rowsPerBlock;
  const int64_t r1 = grp < a.groups && n > 0 ? min(a.N, r0 + a.rowsPerBlock) : r0;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  const Elt* dy = static_cast<const Elt*>(a.dy) + f0;
  Elt* dpre = static_cast<Elt*>(a.dpre) + f0;
  auto row_step = [&](const typename Chunk<Elt>::V& g, const u32x2& w, uint32_t sc, int64_t r) __attribute__((always_inline)) {
    float v[8], d[8];
    decode8(w, scale_step(sc), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      d[e] = (float)g[e] * gelu_grad(v[e]);
      s[e] += d[e];
    }
    store_chunk8<Elt, WHOLE>(dpre + r * a.R, n, d);
  };
  int64_t r = r0 + grp;
  typename Chunk<Elt>::V g;
  u32x2 w;
  uint32_t sc = 0;
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    g = load_chunk8<Elt, WHOLE, STREAM>(dy + row * a.R, n);
    w = load_codes8<STREAM>(a.codes + row * a.pitch + f0);
    sc = a.scales[row * (a.pitch / kCkptBlock) + f0 / kCkptBlock];
  };
  if (r < r1) load(r);
  while (r < r1) {
    const auto g0 = g;
    const u32x2 w0 = w;
    const uint32_t sc0 = sc;
    const int64_t at = r;
    r += a.groups;
    if (r < r1) load(r);
    row_step(g0, w0, sc0, at);
  }
  if (!a.part && !a.dbias) return;
  int half = 1;
  while (half < a.groups) half *= 2;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[e][threadIdx.x] = s[e];
  for (half /= 2; half > 0; half /= 2) {
    __syncthreads();
    if (grp < half && grp + half < a.groups) {
#pragma unroll
      for (int e = 0; e < 8; ++e) red[e][threadIdx.x] += red[e][threadIdx.x + half * a.lanes];
    }
  }
  // Column blocks hold whole channels (lanes * 8 is a multiple of T, or there is one block).
  __syncthreads();
  const int first = cb * a.lanes * 8, channels = min(a.lanes * 8, a.R - first) / a.T, c0 = first / a.T;
  for (int c = (int)threadIdx.x; c < channels; c += kEpi8Threads) {
    float t = 0.0f;
    for (int j = c * a.T; j < (c + 1) * a.T; ++j) t += red[j & 7][j >> 3];
    if (a.part) a.part[(int64_t)rb * (a.R / a.T) + c0 + c] = t;
    else static_cast<Elt*>(a.dbias)[c0 + c] = (Elt)t;
  }
}

// x's half spectrum for the weight gradient, as eql_spec_kernel writes it, with the layer's
// input rebuilt from a checkpoint: v = act(gamma[c] value + beta[c]).  The same launch can
// transform dy, in blocks1 of its workgroups.  Padding channels are left alone (spec_thread), so
// narrow layers neither compute nor write them.
// The transform is fp32; the spectrum is rounded to the element type once, since that is what the
// GEMM's matrix instructions take: with dy's it leaves an fp16 gradient 3.7 to 4.0e-4 of its norm
// off, where its own last rounding alone is 2.1e-4.  Carrying a remainder beside one operand would
// double the products (N = 65536, 1024 x 1024 channels: 710 us of GEMM more).
struct Spec8Args {
  const unsigned char* codes;
  const unsigned char* scales;
  const void* gamma;  // [K] or null
  const void* beta;   // [K] or null
  void* out;          // units [kgCount][T][2][Kpad]
  int N, K, Kpad, kgCount, pitch;
  Twiddles tw;
  const void* m2;     // dy [N][K2*T]
  void* out2;         // units [kgCount][T][2][Kpad2]
  int K2, Kpad2, blocks1;
};

// What a checkpoint's values become on the way into the layer.  A GELU costs the transform 21
// operations a feature of about 30; a kernel of its own keeps the other views free of it.
constexpr int kSpec8Turn = 64;  // both matrices' workgroups are rounded up to this
enum Ckpt8View { kViewPlain = 0, kViewAffine = 1, kViewGelu = 2 };

template <int T, typename Elt, int VIEW>
__global__ void __launch_bounds__(256) eql_spec8_kernel(const Spec8Args a) {
  using E = EltT<Elt>;
  constexpr int G = E::kPerUnit;
  // dy's workgroups are spread evenly among x's, kSpec8Turn at a time (every XCD gets both
  // kinds): those move memory, these compute.
  const uint32_t turn = blockIdx.x / kSpec8Turn, turns = gridDim.x / kSpec8Turn, dyTurns = a.blocks1 / kSpec8Turn;
  const uint32_t before = (uint32_t)((uint64_t)turn * dyTurns / turns);
  if ((uint32_t)((uint64_t)(turn + 1) * dyTurns / turns) > before) {
    spec_thread<T, Elt>(static_cast<const Elt*>(a.m2), a.out2, a.N, a.K2, a.Kpad2, a.K2, a.kgCount,
                        (size_t)(before * kSpec8Turn + blockIdx.x % kSpec8Turn) * 256 + threadIdx.x, a.tw);
    return;
  }
  const size_t idx = (size_t)(blockIdx.x - before * kSpec8Turn) * 256 + threadIdx.x;
  if (idx >= (size_t)a.kgCount * 2 * a.K) return;
  const int k = (int)(idx % a.K);
  const size_t rest = idx / a.K;
  const int half = (int)(rest & 1);
  const int kg = (int)(rest >> 1);
  const int row0 = kg * 2 * G + half * G;
  const int rows = min(G, a.N - row0);  // rows of this thread that exist
  constexpr int WORDS = (T + 3) / 4;
  // A channel's T features lie in one block of 32 where T divides 32, else in at most two.
  constexpr bool ONE = kCkptBlock % T == 0;
  const int b0 = k * T / kCkptBlock, b1 = (k * T + T - 1) / kCkptBlock;
  const int cut = b1 > b0 ? b1 * kCkptBlock - k * T : T;  // features from `cut` on take the second block's step
  uint32_t w[G][WORDS], s0[G], s1[G];
#pragma unroll
  for (int e = 0; e < G; ++e) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[e][i] = 0;
    s0[e] = s1[e] = 0;
  }
  float gam = 1.0f, bet = 0.0f;
  if (rows > 0) {
    const unsigned char* c = a.codes + (size_t)row0 * a.pitch + (size_t)k * T;
    const unsigned char* sc = a.scales + (size_t)row0 * (a.pitch / kCkptBlock);
    auto fetch = [&](int e) __attribute__((always_inline)) {
      __builtin_memcpy(w[e], c + (size_t)e * a.pitch, T);
      s0[e] = sc[(size_t)e * (a.pitch / kCkptBlock) + b0];
      if (!ONE) s1[e] = sc[(size_t)e * (a.pitch / kCkptBlock) + b1];
    };
    if (rows >= G) {
#pragma unroll
      for (int e = 0; e < G; ++e) fetch(e);
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (e < rows) fetch(e);
    }
    if constexpr (VIEW != kViewPlain) {
      if (a.gamma) gam = (float)static_cast<const Elt*>(a.gamma)[k];
      if (a.beta) bet = (float)static_cast<const Elt*>(a.beta)[k];
    }
  }
  float pl[T][G];
#pragma unroll
  for (int e = 0; e < G; ++e) {
    float v[T], o[T];
    const float st0 = scale_step(s0[e]), st1 = ONE ? st0 : scale_step(s1[e]);
#pragma unroll
    for (int h = 0; h < T; ++h) {
      const float q = (float)(int)(int8_t)(w[e][h / 4] >> (8 * (h % 4))) * (ONE || h < cut ? st0 : st1);
      if constexpr (VIEW == kViewPlain) {
        v[h] = q;
      } else {
        // Missing rows are zero before GELU, which keeps them so.
        const float u = e < rows ? __builtin_fmaf(q, gam, bet) : 0.0f;
        v[h] = VIEW == kViewGelu ? gelu_erf(u) : u;
      }
    }
    Dft<T>::run(v, o, a.tw);
#pragma unroll
    for (int p = 0; p < T; ++p) pl[p][e] = o[p];
  }
  u32x4* out = static_cast<u32x4*>(a.out) + ((size_t)kg * T * 2 + half) * a.Kpad + k;
#pragma unroll
  for (int p = 0; p < T; ++p) __builtin_nontemporal_store(E::pack(pl[p]), &out[(size_t)p * 2 * a.Kpad]);
}

}  // namespace eql
