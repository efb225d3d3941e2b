// Product of two E4M3 matrices with a scale for each block of 128 along K:
//   C[m,n] = sum over blocks j of  sa[m,j] * sb[n,j] * sum over k in j of a[m,k] b[n,k]
// (sb of a row of b, or of 128 rows), accumulated in binary32, one rounding
// to bf16 or none.
#include "ar_device.hpp"
#include "ar_internal.hpp"

namespace ar {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBK = AR_BLOCK;  // one scale block: 128 codes = 8 chunks of 16 bytes

// 16 codes k .. k+15 of a row; codes at K and after read as zero, so that
// neither operand's padding (which may hold NaN codes) reaches a product.
__device__ __forceinline__ u32x4 load_chunk(const uint8_t* row, unsigned k, unsigned K) {
  if (k + 16 <= K) return *reinterpret_cast<const u32x4*>(row + k);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (unsigned j = 0; j < 16; ++j)
    if (k + j < K) v[j >> 2] |= (uint32_t)row[k + j] << (8 * (j & 3));
  return v;
}

// Chunk c of row r sits at position c ^ (r % 8): the 16 rows that a wave
// reads at one chunk then spread over all banks.
__device__ __forceinline__ int lds_at(int r, int c) { return r * 8 + (c ^ (r & 7)); }

__device__ __forceinline__ float e8m0_f32(uint8_t b) {
  return b == 255 ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(1.0f, (int)b - 127);
}

// 128 x 128 tile of C in a 256-lane workgroup, 64 x 64 a wave as 4 x 4
// products of 16 x 16 x 128.  b is the first operand, so a lane ends with
// four consecutive n of one m.
template <bool E8M0, bool BROWS, bool OUT32>
__global__ __launch_bounds__(256) void k_gemm_tile(GemmArgs g) {
  constexpr int BM = 128, BN = 128;
  __shared__ u32x4 la[BM * 8], lb[BN * 8];
  const int z = blockIdx.z, t = threadIdx.x, lane = lane_id(), wave = t / kWave;
  const unsigned m0 = blockIdx.x * BM, n0 = blockIdx.y * BN;
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
  const int lr = lane & 15, lq = lane >> 4;
  const uint8_t *A = g.a[z], *B = g.b[z];
  f32x4 acc[4][4];  // [n tile][m tile]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const unsigned nkb = (g.K + kBK - 1) / kBK;
  for (unsigned kb = 0; kb < nkb; ++kb) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = i * 256 + t, r = q / 8, c = q % 8;
      const size_t ra = min(m0 + r, g.M - 1), rb = min(n0 + r, g.N - 1);
      la[lds_at(r, c)] = load_chunk(A + ra * g.lda, kb * kBK + c * 16, g.K);
      lb[lds_at(r, c)] = load_chunk(B + rb * g.ldb, kb * kBK + c * 16, g.K);
    }
    __syncthreads();
    i32x8 fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ra = wm + i * 16 + lr, rb = wn + i * 16 + lr;
      union { u32x4 h[2]; i32x8 v; } u;
      u.h[0] = la[lds_at(ra, 2 * lq)];
      u.h[1] = la[lds_at(ra, 2 * lq + 1)];
      fa[i] = u.v;
      u.h[0] = lb[lds_at(rb, 2 * lq)];
      u.h[1] = lb[lds_at(rb, 2 * lq + 1)];
      fb[i] = u.v;
    }
    if constexpr (E8M0) {
      int sa[4], sb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t m = min(m0 + wm + i * 16 + lr, g.M - 1);
        const size_t n = min(n0 + wn + i * 16 + lr, g.N - 1);
        sa[i] = static_cast<const uint8_t*>(g.sa[z])[m * g.sa_rs + kb * g.sa_cs];
        sb[i] = static_cast<const uint8_t*>(g.sb[z])[(BROWS ? n : n / AR_BLOCK) * g.sb_rs + kb * g.sb_cs];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i], fa[j], acc[i][j], 0, 0, 0, sb[i], 0, sa[j]);
    } else {
      float sa[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const size_t m = min(m0 + wm + j * 16 + lr, g.M - 1);
        sa[j] = static_cast<const float*>(g.sa[z])[m * g.sa_rs + kb * g.sa_cs];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float sb[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const size_t n = min(n0 + wn + i * 16 + lq * 4 + r, g.N - 1);
          sb[r] = static_cast<const float*>(g.sb[z])[(BROWS ? n : n / AR_BLOCK) * g.sb_rs + kb * g.sb_cs];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i], fa[j], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                                        0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], sa[j] * sb[r], acc[i][j][r]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned m = m0 + wm + j * 16 + lr, n = n0 + wn + i * 16 + lq * 4;
      if (m >= g.M) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < g.N) {
          if constexpr (OUT32) static_cast<float*>(g.c[z])[m * g.ldc + n + r] = acc[i][j][r];
          else static_cast<uint16_t*>(g.c[z])[m * g.ldc + n + r] = to_bf16(acc[i][j][r]);
        }
    }
}

template <bool E8M0, bool BROWS>
hipError_t gemm_o(const Launch& L, const GemmArgs& g, int G, bool out_f32) {
  const dim3 grid((unsigned)cdiv(g.M, 128), (unsigned)cdiv(g.N, 128), (unsigned)G);
  if (out_f32) return launch_k(k_gemm_tile<E8M0, BROWS, true>, grid, dim3(256), 0, L.stream, g);
  return launch_k(k_gemm_tile<E8M0, BROWS, false>, grid, dim3(256), 0, L.stream, g);
}

}  // namespace

size_t gemm_fp8_workspace(size_t, size_t, size_t, int) { return 0; }

hipError_t launch_gemm_fp8(const Launch& L, const GemmArgs& g, int G, bool e8m0, bool b_rows, bool out_f32, void*) {
  if (e8m0) return b_rows ? gemm_o<true, true>(L, g, G, out_f32) : gemm_o<true, false>(L, g, G, out_f32);
  return b_rows ? gemm_o<false, true>(L, g, G, out_f32) : gemm_o<false, false>(L, g, G, out_f32);
}

}  // namespace ar
