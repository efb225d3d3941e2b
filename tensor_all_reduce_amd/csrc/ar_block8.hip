// bf16 matrices to E4M3 codes with a scale for each 1 x 128 or 128 x 128
// block, as they stand or transposed: the operands of the fp8 matrix product.
//
// One 256-lane workgroup takes a 128 x 128 tile of x, which holds whole
// blocks of every form, so each element is read once and its scale is known
// before it is written.  Bound by memory: three bytes an element, [8192 x
// 8192] in 128 x 128 blocks 36 us from memory (5.5 TB/s) and 33 from the
// last-level cache, [4097 x 8192] transposed 23.8 us (4.2 TB/s; 2112 tiles
// are a little more than the device holds at once).
#include "ar_device.hpp"
#include "ar_e4m3.hpp"
#include "ar_internal.hpp"

namespace ar {
namespace {

typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kTile = AR_BLOCK;

template <bool E8M0>
__device__ __forceinline__ void put_scale(const QuantArgs& a, size_t r, size_t c, uint32_t kept) {
  const size_t k = r * a.scale_rs + c * a.scale_cs;
  if constexpr (E8M0) static_cast<uint8_t*>(a.scales)[k] = (uint8_t)kept;
  else static_cast<uint32_t*>(a.scales)[k] = kept;
}

// Lane t holds columns 8 (t % 16) .. + 7 of rows 8 (t / 16) .. + 7, as bf16:
// widened for the maximum and again for the codes, since half the registers
// let twice the workgroups wait for memory at once.
template <bool SQUARE, bool TURN, bool E8M0, bool NT>
__global__ __launch_bounds__(256) void k_quant_block(QuantArgs a, unsigned tiles_c) {
  __shared__ uint32_t top[4][kTile];
  __shared__ __align__(16) uint8_t turned[TURN ? kTile * kTile : 16];
  const size_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;
  const int lc = (threadIdx.x % 16) * 8, lr = (threadIdx.x / 16) * 8, wave = threadIdx.x / kWave;
  const size_t r0 = tr * kTile + lr, c0 = tc * kTile + lc;
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (r0 + i < a.rows && c0 < a.cols) {
      const uint16_t* p = a.x + (r0 + i) * a.ldx + c0;
      if (c0 + 8 <= a.cols) {
        if constexpr (NT) v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4u*>(p));
        else v[i] = *reinterpret_cast<const u32x4u*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t e = c0 + j < a.cols ? (uint32_t)p[j] : 0u;
          v[i][j >> 1] |= (j & 1) ? (e << 16) : e;
        }
      }
    }
  }
  auto at = [&](int i, int j) { return (j & 1) ? hi_f32(v[i][j >> 1]) : lo_f32(v[i][j >> 1]); };

  // inv[i]: of row i (straight) or of column i (transposed)
  float inv[8];
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, finite_mag(at(i, j)));
    m = row16_max(m);
    if (threadIdx.x % 16 == 0) top[0][threadIdx.x / 16] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, top[0][i]);
    const BlockScale s = block_scale<E8M0>(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = s.inv;
    if (threadIdx.x == 0) put_scale<E8M0>(a, TURN ? tc : tr, TURN ? tr : tc, s.kept);
  } else if constexpr (!TURN) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, finite_mag(at(i, j)));
      const BlockScale s = block_scale<E8M0>(row16_max(m));
      inv[i] = s.inv;
      if (threadIdx.x % 16 == 0 && r0 + i < a.rows) put_scale<E8M0>(a, r0 + i, tc, s.kept);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, finite_mag(at(i, j)));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lane_id() < 16) top[wave][lc + j] = m;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = max(max(top[0][lc + j], top[1][lc + j]), max(top[2][lc + j], top[3][lc + j]));
      const BlockScale s = block_scale<E8M0>(m);
      inv[j] = s.inv;
      if (threadIdx.x < 16 && c0 + j < a.cols) put_scale<E8M0>(a, c0 + j, tr, s.kept);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(v[i]));

  if constexpr (!TURN) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i >= a.rows || c0 >= a.cols) continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at(i, j);
      const uint32_t lo = codes4_scaled(f, inv[i]), hi = codes4_scaled(f + 4, inv[i]);
      uint8_t* c = a.codes + (r0 + i) * a.codes_ld + c0;
      if (c0 + 8 <= a.cols) {
        *reinterpret_cast<uint64_t*>(c) = (uint64_t)lo | ((uint64_t)hi << 32);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < a.cols) c[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
      }
    }
  } else {
    // 16 pieces of 8 codes a row of the turned tile, piece q of row c at
    // q ^ (c / 8): the 16 lanes that write one piece of 16 rows spread over
    // the banks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float col[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) col[i] = at(i, j);
      const uint32_t lo = codes4_scaled(col, inv[j]), hi = codes4_scaled(col + 4, inv[j]);
      *reinterpret_cast<uint64_t*>(&turned[(lc + j) * kTile + ((lr ^ lc) & (kTile - 1))]) = (uint64_t)lo | ((uint64_t)hi << 32);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int q = k * 256 + threadIdx.x, c = q / 8, r = (q % 8) * 16;  // 16 codes of output row c
      const size_t gc = tc * kTile + c, gr = tr * kTile + r;
      if (gc >= a.cols || gr >= a.rows) continue;
      const int turn = c & ~7;
      union { uint64_t h[2]; u32x4 w; } x;
      x.h[0] = *reinterpret_cast<const uint64_t*>(&turned[c * kTile + (r ^ turn)]);
      x.h[1] = *reinterpret_cast<const uint64_t*>(&turned[c * kTile + ((r + 8) ^ turn)]);
      uint8_t* p = a.codes + gc * a.codes_ld + gr;
      if (gr + 16 <= a.rows) {
        *reinterpret_cast<u32x4*>(p) = x.w;
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (gr + j < a.rows) p[j] = (uint8_t)(x.w[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

// Non-temporal loads of an x that the L2s of the 8 XCDs (32 MiB together)
// cannot hold: of three [4097 x 8192] in turn, transposed, 23.7 us, plain
// 26.2; of three [8192 x 8192] 36.0 and 41.7; the same [8192 x 8192] again and
// again, which the last-level cache keeps, 36.0 and 33.4.  Plain stores: the
// codes are short lines that meet in the L2 (non-temporal ones 35.9 and 37.2).
constexpr size_t kColdBytes = (size_t)32 << 20;

template <bool SQUARE, bool TURN, bool E8M0>
hipError_t quant_f(const Launch& L, const QuantArgs& a) {
  const size_t tc = cdiv(a.cols, kTile), tr = cdiv(a.rows, kTile);
  const dim3 grid((unsigned)(tr * tc));
  auto k = a.rows * a.cols * 2 > kColdBytes ? k_quant_block<SQUARE, TURN, E8M0, true> : k_quant_block<SQUARE, TURN, E8M0, false>;
  return launch_k(k, grid, dim3(256), 0, L.stream, a, (unsigned)tc);
}

template <bool SQUARE, bool TURN>
hipError_t quant_st(const Launch& L, const QuantArgs& a, bool e8m0) {
  return e8m0 ? quant_f<SQUARE, TURN, true>(L, a) : quant_f<SQUARE, TURN, false>(L, a);
}

}  // namespace

// 256 lanes a tile: HIP takes fewer than 2^32 lanes along one axis.
bool quant_block_fits(size_t rows, size_t cols) {
  const size_t tc = (cols - 1) / kTile + 1, tr = (rows - 1) / kTile + 1;
  return tc <= 0xFFFFFFu && tr <= 0xFFFFFFu / tc;
}

hipError_t launch_quant_block(const Launch& L, const QuantArgs& a, int block_rows, bool turn, bool e8m0) {
  if (block_rows == AR_BLOCK) return turn ? quant_st<true, true>(L, a, e8m0) : quant_st<true, false>(L, a, e8m0);
  return turn ? quant_st<false, true>(L, a, e8m0) : quant_st<false, false>(L, a, e8m0);
}

}  // namespace ar
