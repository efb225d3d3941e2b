// Rank contributions summed, residual added, root-mean-square norm, and its
// gradient: the step that follows a tensor-parallel all-reduce in every
// transformer block, in one pass over the data.
//
//   h = ((x_0 + x_1) + ... + x_{P-1}) (+ residual)         binary32
//   y = h * (1 / sqrt(mean(h^2) + eps)) * weight           binary32
//
// res_out is h rounded to bf16 once, y comes as bf16 (one rounding) and / or
// as E4M3 codes with a scale for each 128 elements of the row, taken from
// the binary32 y.  The norm reads the unrounded h.
#include "ar_device.hpp"
#include "ar_e4m3.hpp"
#include "ar_internal.hpp"

namespace ar {
namespace {

// 16-byte groups that may start on any 2-byte boundary (rows of an odd
// length): global loads and stores take such addresses.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));

// Group g (8 elements) of a bf16 row of `cols` elements; a group that runs
// past the row is read element by element, zeros after its end.
template <bool NT, bool WHOLE>
__device__ __forceinline__ u32x4 load_group(const uint16_t* row, unsigned g, unsigned cols) {
  if constexpr (WHOLE) return ld4<NT>(reinterpret_cast<const u32x4*>(row) + g);
  if (8 * g + 8 <= cols) return *reinterpret_cast<const u32x4u*>(row + 8 * (size_t)g);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (unsigned j = 0; j < 8; ++j) {
    const uint32_t e = 8 * g + j < cols ? (uint32_t)row[8 * g + j] : 0u;
    v[j >> 1] |= (j & 1) ? (e << 16) : e;
  }
  return v;
}

template <bool NT, bool WHOLE>
__device__ __forceinline__ void store_group(uint16_t* row, unsigned g, unsigned cols, u32x4 v) {
  if constexpr (WHOLE) {
    st4<NT>(reinterpret_cast<u32x4*>(row) + g, v);
    return;
  }
  if (8 * g + 8 <= cols) {
    *reinterpret_cast<u32x4u*>(row + 8 * (size_t)g) = v;
    return;
  }
#pragma unroll
  for (unsigned j = 0; j < 8; ++j)
    if (8 * g + j < cols) row[8 * g + j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
}

__device__ __forceinline__ void widen(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = lo_f32(v[k]);
    f[2 * k + 1] = hi_f32(v[k]);
  }
}

__device__ __forceinline__ u32x4 narrow(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// 8 gains from `w` (bf16 or binary32; nullptr: ones).
template <bool WHOLE>
__device__ __forceinline__ void load_gain(const void* w, int w_f32, unsigned g, unsigned cols, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.0f;
  } else if (w_f32) {
    const float* p = static_cast<const float*>(w) + 8 * (size_t)g;
#pragma unroll
    for (unsigned j = 0; j < 8; ++j) f[j] = WHOLE || 8 * g + j < cols ? p[j] : 0.0f;
  } else {
    widen(load_group<false, WHOLE>(static_cast<const uint16_t*>(w), g, cols), f);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Sum over the workgroup, the same in every lane; `part` holds one value per
// wave.  The order is fixed by the workgroup's size.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = wave_sum(v);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  if (lane_id() == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = part[0];
  for (int i = 1; i < waves; ++i) s += part[i];
  return s;
}

constexpr int kMaxWaves = 16;

// One workgroup per row; lane t holds groups t, t + T, ... (V of them).
template <int P, int V, bool WHOLE, bool E8M0>
__global__ __launch_bounds__(1024) void k_reduce_norm(InPtrs in, NormArgs a) {
  __shared__ float part[kMaxWaves];
  const size_t row = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const unsigned cols = a.cols, groups = (cols + 7) / 8;
  const size_t at = row * cols;
  float h[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[u][j] = 0.0f;
    if (g >= groups) continue;
    u32x4 x[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
      x[p] = load_group<false, WHOLE>(static_cast<const uint16_t*>(in.p[p]) + at, g, cols);
    u32x4 r = {0u, 0u, 0u, 0u};
    if (a.residual) r = load_group<false, WHOLE>(a.residual + at, g, cols);
    widen(x[0], h[u]);
#pragma unroll
    for (int p = 1; p < P; ++p) {
      float f[8];
      widen(x[p], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] += f[j];
    }
    if (a.residual) {
      float f[8];
      widen(r, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] += f[j];
    }
    if (a.res_out) store_group<false, WHOLE>(a.res_out + at, g, cols, narrow(h[u]));
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[u][j], h[u][j], ss);
  }
  if (!a.y && !a.codes) return;
  // a lane's sum is divided before lanes are added, so that only a mean
  // square beyond binary32 overflows, not the sum of a whole row's squares
  const float r = 1.0f / sqrtf(block_sum(ss / (float)cols, part) + a.eps);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = 0.0f;
    if (g < groups) {
      float w[8];
      load_gain<WHOLE>(a.weight, a.weight_f32, g, cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[u][j] * r * w[j];
      if (a.y) store_group<false, WHOLE>(a.y + at, g, cols, narrow(y));
    }
    if (a.codes) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (WHOLE || 8 * g + j < cols) m = max(m, finite_mag(y[j]));
      m = row16_max(m);
      const BlockScale s = block_scale<E8M0>(m);
      const uint32_t lo = codes4_scaled(y, s.inv), hi = codes4_scaled(y + 4, s.inv);
      if (g < groups) {
        uint8_t* c = a.codes + row * a.codes_ld + 8 * (size_t)g;
        if (WHOLE || 8 * g + 8 <= cols) {
          *reinterpret_cast<uint64_t*>(c) = (uint64_t)lo | ((uint64_t)hi << 32);
        } else {
#pragma unroll
          for (unsigned j = 0; j < 8; ++j)
            if (8 * g + j < cols) c[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
        }
        if ((threadIdx.x & 15u) == 0) {
          const size_t k = row * a.scale_rs + (g >> 4) * a.scale_cs;
          if constexpr (E8M0) static_cast<uint8_t*>(a.scales)[k] = (uint8_t)s.kept;
          else static_cast<uint32_t*>(a.scales)[k] = s.kept;
        }
      }
    }
  }
}

// Gradient.  With r = 1 / sqrt(mean(h^2) + eps), x = h r and g = dy w:
//   dx = dres + r (g - x mean(g x)),   dweight = sum over rows of dy x.
// Workgroup b takes rows b, b + grid, ...; a lane keeps the sums of dy x of
// its own columns in registers and writes them once, to row b of `partial`.
template <int V, bool WHOLE>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormBwdArgs a) {
  __shared__ float part[2][2][kMaxWaves];
  const unsigned cols = a.cols, groups = (cols + 7) / 8;
  const int waves = blockDim.x / kWave;
  float dw[V][8];
#pragma unroll
  for (int u = 0; u < V; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[u][j] = 0.0f;
  int flip = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const size_t at = row * cols;
    float h[V][8], dy[V][8], w[V][8];
    float ss = 0.0f, gh = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const unsigned g = u * blockDim.x + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = dy[u][j] = w[u][j] = 0.0f;
      if (g >= groups) continue;
      widen(load_group<false, WHOLE>(a.h + at, g, cols), h[u]);
      widen(load_group<false, WHOLE>(a.dy + at, g, cols), dy[u]);
      load_gain<WHOLE>(a.weight, a.weight_f32, g, cols, w[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = __builtin_fmaf(h[u][j], h[u][j], ss);
        gh = __builtin_fmaf(dy[u][j] * w[u][j], h[u][j], gh);
      }
    }
    ss = wave_sum(ss / (float)cols);
    gh = wave_sum(gh / (float)cols);
    // two sets of slots in turn: a wave may write the next row's sums while
    // another still reads this row's, and is held at the next barrier before
    // it could write these slots again
    if (lane_id() == 0) {
      part[flip][0][threadIdx.x / kWave] = ss;
      part[flip][1][threadIdx.x / kWave] = gh;
    }
    __syncthreads();
    ss = part[flip][0][0];
    gh = part[flip][1][0];
    for (int i = 1; i < waves; ++i) {
      ss += part[flip][0][i];
      gh += part[flip][1][i];
    }
    const float r = 1.0f / sqrtf(ss + a.eps);
    const float m = r * gh;   // mean(g x)
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const unsigned g = u * blockDim.x + threadIdx.x;
      if (g >= groups) continue;
      float dx[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = h[u][j] * r;
        dx[j] = r * (dy[u][j] * w[u][j] - x * m);
        dw[u][j] = __builtin_fmaf(dy[u][j], x, dw[u][j]);
      }
      if (a.dres) {
        float f[8];
        widen(load_group<false, WHOLE>(a.dres + at, g, cols), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] += f[j];
      }
      if (a.dx) store_group<false, WHOLE>(a.dx + at, g, cols, narrow(dx));
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
#pragma unroll
    for (unsigned j = 0; j < 8; ++j)
      if (8 * g + j < cols) a.partial[(size_t)blockIdx.x * cols + 8 * g + j] = dw[u][j];
  }
}

// dweight[c] = sum of `n` rows of partial sums: 64 columns a workgroup, four
// waves take a quarter of the rows each.
__global__ __launch_bounds__(256) void k_sum_rows(const float* partial, float* out, unsigned n, unsigned cols) {
  __shared__ float part[4][kWave];
  const unsigned c = blockIdx.x * kWave + lane_id(), q = threadIdx.x / kWave;
  float s = 0.0f;
  if (c < cols)
    for (unsigned i = q; i < n; i += 4) s += partial[(size_t)i * cols + c];
  part[q][lane_id()] = s;
  __syncthreads();
  if (q == 0 && c < cols) out[c] = (part[0][lane_id()] + part[1][lane_id()]) + (part[2][lane_id()] + part[3][lane_id()]);
}

// Lanes and groups per lane for a row of `cols` elements.
struct RowShape {
  int block, v;
};
RowShape row_shape(size_t cols) {
  const size_t groups = cdiv(cols, 8);
  int v = 1;
  while (v < 8 && cdiv(groups, v) > 1024) v *= 2;
  return RowShape{(int)(cdiv(cdiv(groups, v), kWave) * kWave), v};
}

// One workgroup per row; HIP takes fewer than 2^32 lanes along one axis.
dim3 row_grid(size_t rows) {
  const size_t x = rows < (1u << 20) ? rows : (1u << 20);
  return dim3((unsigned)x, (unsigned)cdiv(rows, x));
}

template <int P, int V>
hipError_t norm_pv(const Launch& L, const InPtrs& in, const NormArgs& a, int block) {
  const bool whole = a.cols % 8 == 0;
  const dim3 grid = row_grid(a.rows), blk(block);
  if (a.scale_e8m0) {
    if (whole) return launch_k(k_reduce_norm<P, V, true, true>, grid, blk, 0, L.stream, in, a);
    return launch_k(k_reduce_norm<P, V, false, true>, grid, blk, 0, L.stream, in, a);
  }
  if (whole) return launch_k(k_reduce_norm<P, V, true, false>, grid, blk, 0, L.stream, in, a);
  return launch_k(k_reduce_norm<P, V, false, false>, grid, blk, 0, L.stream, in, a);
}

template <int P>
hipError_t norm_p(const Launch& L, const InPtrs& in, const NormArgs& a) {
  const RowShape s = row_shape(a.cols);
  switch (s.v) {
    case 1: return norm_pv<P, 1>(L, in, a, s.block);
    case 2: return norm_pv<P, 2>(L, in, a, s.block);
    case 4: return norm_pv<P, 4>(L, in, a, s.block);
    default: return norm_pv<P, 8>(L, in, a, s.block);
  }
}

template <int V>
hipError_t bwd_v(const Launch& L, const NormBwdArgs& a, unsigned grid, int block) {
  if (a.cols % 8 == 0) return launch_k(k_norm_bwd<V, true>, dim3(grid), dim3(block), 0, L.stream, a);
  return launch_k(k_norm_bwd<V, false>, dim3(grid), dim3(block), 0, L.stream, a);
}

}  // namespace

hipError_t launch_reduce_norm(const Launch& L, const InPtrs& in, int P, const NormArgs& a) {
  switch (P) {
    case 1: return norm_p<1>(L, in, a);
    case 2: return norm_p<2>(L, in, a);
    case 3: return norm_p<3>(L, in, a);
    case 4: return norm_p<4>(L, in, a);
    case 5: return norm_p<5>(L, in, a);
    case 6: return norm_p<6>(L, in, a);
    case 7: return norm_p<7>(L, in, a);
    case 8: return norm_p<8>(L, in, a);
    default: return hipErrorInvalidValue;
  }
}

unsigned norm_bwd_grid(size_t rows) { return (unsigned)(rows < 512 ? rows : 512); }

hipError_t launch_norm_bwd(const Launch& L, const NormBwdArgs& a, float* dweight) {
  const RowShape s = row_shape(a.cols);
  const unsigned grid = norm_bwd_grid(a.rows);
  hipError_t e = hipSuccess;
  if (grid) {
    switch (s.v) {
      case 1: e = bwd_v<1>(L, a, grid, s.block); break;
      case 2: e = bwd_v<2>(L, a, grid, s.block); break;
      case 4: e = bwd_v<4>(L, a, grid, s.block); break;
      default: e = bwd_v<8>(L, a, grid, s.block); break;
    }
  }
  if (e != hipSuccess || !dweight) return e;
  return launch_k(k_sum_rows, dim3((unsigned)cdiv(a.cols, kWave)), dim3(256), 0, L.stream,
                  static_cast<const float*>(a.partial), dweight, grid, a.cols);
}

}  // namespace ar
