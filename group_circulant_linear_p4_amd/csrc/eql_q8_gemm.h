// The EQ-Linear layer on 8-bit integer rows and weights (eql_q8.h): for each plane of the half
// spectrum integer products with 32-bit sums, which are exact (|sum| <= 2 C 127^2 < 2^31), then
//     plane = sum * scale of the output channel * scale of the row
// (in this order: rows near fp32's end stay finite),
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
  int rowTiles, colTiles;
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

// One K step of all planes: A and B operands of the T planes into the accumulators.
template <int T>
__device__ __forceinline__ void q8_step(i32x16 (&acc)[T], const u32x4 (&a)[T], const u32x4 (&b)[T], const u32x4 (&neg)[n_pairs(T) + 1]) {
  constexpr int NR = n_real_planes(T);
#pragma unroll
  for (int p = 0; p < NR; ++p) q8_mfma(acc[p], a[p], b[p]);
#pragma unroll
  for (int q = 0; q < n_pairs(T); ++q) {
    const int re = NR + 2 * q, im = re + 1;
    q8_mfma(acc[re], a[re], b[re]);
    q8_mfma(acc[im], a[re], b[im]);
    q8_mfma(acc[re], a[im], neg[q]);
    q8_mfma(acc[im], a[im], b[re]);
  }
}
#endif

// Few rows or few output channels: a workgroup takes a 32 x 32 tile of outputs, its waves every
// W-th K block each (operands straight from memory, a block ahead), and adds its integer sums in
// LDS.  Epilogue: a thread a (row, channel).
template <int T, typename Elt, int W>
__global__ void __launch_bounds__(64 * W) eql_q8_small_kernel(const Q8FwdArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NR = n_real_planes(T), NP = n_pairs(T), F = n_freqs(T);
  __shared__ int32_t sums[T][32 * 32];
  const int colTile = (int)blockIdx.x % a.colTiles, rowTile = (int)blockIdx.x / a.colTiles;
  const int row0 = rowTile * 32;
  const int lane = lane_index(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int rows = min(32, a.f.N - row0);
  const uint32_t rowBytes = (uint32_t)a.pitch * T;
  const uint32_t blockBytes = (uint32_t)T * 2048u;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.codes + (size_t)row0 * rowBytes, (uint32_t)rows * rowBytes);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (size_t)colTile * a.kblocks * blockBytes, (uint32_t)a.kblocks * blockBytes);
  for (int i = (int)threadIdx.x; i < T * 1024; i += 64 * W) (&sums[0][0])[i] = 0;
  i32x16 acc[T];
#pragma unroll
  for (int p = 0; p < T; ++p) acc[p] = (i32x16){};
  // Offsets past the last row's end (also of the last plane's last block) read as zero; bytes past
  // another plane's end belong to the next one and meet zeros in the weight.
  const uint32_t xOff = (uint32_t)(lane & 31) * rowBytes + (uint32_t)(lane >> 5) * 16u;
  for (int kb = wave; kb < a.kblocks; kb += W) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 xa[T], wb[T], neg[NP + 1];
#pragma unroll
      for (int p = 0; p < T; ++p) {
        xa[p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, xOff + (uint32_t)(kb * 64 + s * 32 + p * a.pitch), 0, 0));
        wb[p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16 + (p * 2 + s) * 1024, kb * (int)blockBytes, 0));
      }
#pragma unroll
      for (int q = 0; q < NP; ++q) neg[q] = q8_neg(wb[NR + 2 * q + 1]);
      q8_step<T>(acc, xa, wb, neg);
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < T; ++p)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (row < rows) __hip_atomic_fetch_add(&sums[p][row * 32 + (lane & 31)], acc[p][r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < rows * 32; i += 64 * W) {
    const int row = row0 + (i >> 5), col = colTile * 32 + (i & 31);
    if (col >= a.f.Dout) continue;
    float P[T], y[T];
#pragma unroll
    for (int p = 0; p < T; ++p)
      P[p] = (float)sums[p][i] * a.wScales[(int64_t)freq_of(T, p) * a.Dpad + col] * a.rowScales[(int64_t)row * F + freq_of(T, p)];
    Idft<T, false>::run(P, y, a.f.tw);
    const float bias = a.f.bias ? (float)static_cast<const Elt*>(a.f.bias)[col] : 0.0f;
    const int64_t at = ((int64_t)row * a.f.Dout + col) * T;
    float r[T];
#pragma unroll
    for (int g = 0; g < T; ++g) r[g] = 0.0f;
    if (a.f.res) load_group<T, Elt>(static_cast<const Elt*>(a.f.res) + at, r);
#pragma unroll
    for (int g = 0; g < T; ++g) {
      const float v = y[g] + bias;
      y[g] = (a.f.act == 1 ? gelu_erf(v) : v) + r[g];
    }
    store_group<T, Elt>(static_cast<Elt*>(a.f.y) + at, y);
  }
#endif
}

// Rows of a workgroup of the large kernel: WM waves down, MB blocks of 32 each.  Waves across: 4 / WM,
// NB blocks of 32 output channels each.
//   * Rows' codes go through LDS, two slots of one K block (64 input channels of every plane): loads
//     that write LDS directly, 1 KB (16 rows x 64 bytes of a plane) each.  Piece q (16 bytes) of row r
//     lies at place q ^ (r / 4) % 4 of its 64 bytes, so the 16 rows that a fragment read takes at a
//     time touch every bank once.
//   * The weight's operands are read by no other wave of the row block, and lie in memory as the
//     matrix instruction wants them: each wave loads its own straight into registers.
//   * While a K block is multiplied, the next one's rows and operands are on their way.
template <int T, typename Elt, int MB, int NB, int WM>
__global__ void __launch_bounds__(256) eql_q8_large_kernel(const Q8FwdArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NR = n_real_planes(T), NP = n_pairs(T), F = n_freqs(T);
  constexpr int BM = 32 * MB * WM, WN = 4 / WM;
  constexpr int CHUNKS = T * BM / 16;              // 1 KB loads of a slot
  constexpr int PER = (CHUNKS + 3) / 4;            // of a wave
  constexpr int SLOT = CHUNKS * 1024;
  static_assert(BM <= kFwdRows, "the epilogue's rows");
  static_assert(2 * SLOT + F * BM * 4 <= 160 * 1024, "LDS");
  __shared__ u32x4 ring[2][SLOT / 16];
  __shared__ float rowScale[F][BM];

  const int tile = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int colTile = tile % a.colTiles, rowTile = tile / a.colTiles;
  const int row0 = rowTile * BM;
  const int rows = min(BM, a.f.N - row0);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int lane = lane_index();
  const int block0 = (colTile * WN + wn) * NB;     // this wave's first block of 32 output channels
  const int nblk = a.Dpad / 32;
  const uint32_t rowBytes = (uint32_t)a.pitch * T;
  const uint32_t blockBytes = (uint32_t)T * 2048u;
  const uint32_t colBytes = (uint32_t)a.kblocks * blockBytes;

  for (int i = (int)threadIdx.x; i < F * BM; i += 256) {
    const int f = i / BM, r = i - f * BM;
    rowScale[f][r] = r < rows ? a.rowScales[((int64_t)row0 + r) * F + f] : 0.0f;
  }

  // Rows past N and (at the last row's end) bytes past the codes read as zero; bytes past a plane's
  // end belong to the next one and meet zeros in the weight.
  const uint64_t xBase = reinterpret_cast<uint64_t>(a.codes) + (uint64_t)row0 * rowBytes;
  const uint32_t xBytes = (uint32_t)rows * rowBytes;
  uint32_t xOff[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = wave * PER + i, p = j / (BM / 16), rg = j % (BM / 16);
    const int r = rg * 16 + (lane >> 2), q = (lane & 3) ^ ((r >> 2) & 3);
    xOff[i] = j < CHUNKS ? (uint32_t)r * rowBytes + (uint32_t)p * (uint32_t)a.pitch + (uint32_t)q * 16u : kOob;
  }
  const uint32_t ringAt = lds_addr(&ring[0][0]) + (uint32_t)wave * PER * 1024u;
  auto issue_rows = [&](int kb, int slot) __attribute__((always_inline)) {
    const uint32_t skip = (uint32_t)kb * 64u;
    const BufDesc d = desc_at(xBase + skip, xBytes - skip);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (CHUNKS % 4 == 0 || wave * PER + i < CHUNKS) dma16(d, xOff[i], ringAt + (uint32_t)slot * SLOT + (uint32_t)i * 1024u);
  };

  // Blocks past the last one read the last one's operands, and store nothing.
  const int first = min(block0, nblk - 1), more = nblk - 1 - first;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (size_t)first * colBytes, (uint32_t)(min(NB - 1, more) + 1) * colBytes);
  u32x4 wb[2][2][NB][T];
  auto load_w = [&](int kb, u32x4 (&to)[2][NB][T]) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int p = 0; p < T; ++p)
          to[s][nb][p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              wr, lane * 16 + (p * 2 + s) * 1024, kb * (int)blockBytes + min(nb, more) * (int)colBytes, 0));
  };

  i32x16 acc[MB][NB][T];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int p = 0; p < T; ++p) acc[mb][nb][p] = (i32x16){};

  const int lrow = lane & 31;
  auto read_rows = [&](int slot, int s, int mb, u32x4 (&xa)[T]) __attribute__((always_inline)) {
    const int r = (wm * MB + mb) * 32 + lrow;
    const int q = (s * 2 + (lane >> 5)) ^ ((r >> 2) & 3);
#pragma unroll
    for (int p = 0; p < T; ++p) xa[p] = ring[slot][p * (BM * 4) + r * 4 + q];
  };

  auto stage = [&](int kb, auto curTag) __attribute__((always_inline)) {
    constexpr int cur = decltype(curTag)::value;
    if (kb + 1 < a.kblocks) {
      issue_rows(kb + 1, cur ^ 1);
      load_w(kb + 1, wb[cur ^ 1]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 neg[NB][NP + 1];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int q = 0; q < NP; ++q) neg[nb][q] = q8_neg(wb[cur][s][nb][NR + 2 * q + 1]);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        u32x4 xa[T];
        read_rows(cur, s, mb, xa);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) q8_step<T>(acc[mb][nb], xa, wb[cur][s][nb], neg[nb]);
      }
    }
    // The next block's rows are in LDS, and every wave is done with this one's.
    wait_vmcnt<0>();
    wait_lgkm0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  issue_rows(0, 0);
  load_w(0, wb[0]);
  wait_vmcnt<0>();
  __syncthreads();
  int kb = 0;
  for (; kb + 2 <= a.kblocks; kb += 2) {
    stage(kb, std::integral_constant<int, 0>{});
    stage(kb + 1, std::integral_constant<int, 1>{});
  }
  if (kb < a.kblocks) stage(kb, std::integral_constant<int, 0>{});

  // Scales, and the fused layer's epilogue for each block of 32 rows.
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    f32x16 out[T][NB];
    const int rowOff = (wm * MB + mb) * 32;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int col = min((block0 + nb) * 32 + lrow, a.Dpad - 1);
#pragma unroll
      for (int p = 0; p < T; ++p) {
        const float ws = a.wScales[(int64_t)freq_of(T, p) * a.Dpad + col];
#pragma unroll
        for (int r = 0; r < 16; ++r)
          out[p][nb][r] = (float)acc[mb][nb][p][r] * ws * rowScale[freq_of(T, p)][rowOff + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)];
      }
    }
    fwd_epilogue<T, Elt, NB, 1>(a.f, out, row0, rowOff, block0 * 32);
  }
#endif
}

}  // namespace eql
