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
//
// Both kernels are bound by memory.  A row stays in registers between the sum
// of its squares and its result, so every input is read once and every output
// written once; the two passes over a row that the formulas ask for cost no
// traffic.  Measured: 8 ranks, [16384 x 8192], fp8 result, 464-476 us, 6.0
// TB/s; a single row 4.7-4.8 us, where an empty call takes 3.4; gradient of
// [16384 x 16384] 358-370 us, 5.9 TB/s.
#include "ar_device.hpp"
#include "ar_e4m3.hpp"
#include "ar_internal.hpp"

#include <algorithm>

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

// Sum over the wave, the same in every lane: DPP swaps within rows of 16
// lanes (a trip through LDS for each step takes several times as long), then
// the four rows.
__device__ __forceinline__ float wave_sum(float v) {
  auto swapped = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += swapped(v, SPc<0xB1>{});              // lane ^ 1
  v += swapped(v, SPc<0x4E>{});              // lane ^ 2
  v += swapped(v, SPc<0x141>{});             // the other quad of 8
  v += swapped(v, SPc<0x140>{});             // the other half of 16
  auto row = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Means over a row are sums of terms times 2^-k, 2^k the power of two from the
// row's length up, and a factor from 1 to 2: the power multiplies one of a
// term's factors (exactly) before the fused multiply-add, so that no square and
// no sum overflows unless the mean does.
struct RowMean {
  float part, rest;   // 2^-k, 2^k / cols
};
__device__ __forceinline__ RowMean row_mean(unsigned cols) {
  const int k = cols > 1 ? 32 - __builtin_clz(cols - 1) : 0;
  return RowMean{__builtin_ldexpf(1.0f, -k), __builtin_ldexpf(1.0f, k) / (float)cols};
}

constexpr int kMaxWaves = 16;

// Sums of one value a wave, of up to 16 waves, kept in `part`: 16 slots, those
// of waves that the workgroup lacks zero.  put_part, a barrier, sum_parts.
__device__ __forceinline__ void put_part(float v, float* part) {
  const unsigned waves = blockDim.x / kWave;
  if (lane_id() == 0) part[threadIdx.x / kWave] = v;
  if (threadIdx.x >= waves && threadIdx.x < kMaxWaves) part[threadIdx.x] = 0.0f;
}
__device__ __forceinline__ float sum_parts(const float* part) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  const f32x4* p = reinterpret_cast<const f32x4*>(part);
  const f32x4 a = (p[0] + p[1]) + (p[2] + p[3]);
  return (a[0] + a[1]) + (a[2] + a[3]);
}

// Elements from row to row of the gradient's partial sums.
__host__ __device__ constexpr size_t sum_stride(size_t cols) { return (cols + 3) & ~(size_t)3; }

// The row kernel's three forms: rows of whole aligned groups, with plain or
// non-temporal accesses, and ragged rows.
enum RowForm { kRagged = 0, kWhole, kStream };

// Longest ragged row whose aligned groups 8 x 1024 lanes hold; groups of a
// longer one start with the row, wherever that is.
constexpr unsigned kMaxShifted = AR_NORM_MAX_COLS - 14;

// One workgroup per row; lane t holds groups t, t + T, ... (V of them).
//
// kRagged (cols no multiple of 8): rows start anywhere, but all of them at
// the same place in every [rows x cols] buffer.  Groups are those of the
// buffer, aligned, so the row's first and last are shared with its
// neighbours; elements of other rows are read (where the buffer holds the
// whole group), zeroed and not written.  A group then spans up to two scale
// blocks, whose maxima meet in LDS.
template <int P, int V, int FORM>
__global__ __launch_bounds__(1024) void k_reduce_norm(InPtrs in, NormArgs a) {
  __shared__ __align__(16) float part[kMaxWaves];
  __shared__ uint32_t top[FORM == kRagged ? AR_NORM_MAX_COLS / AR_BLOCK : 1];
  constexpr bool NT = FORM == kStream;
  const size_t row = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const unsigned cols = a.cols;
  const int off = FORM == kRagged && cols <= kMaxShifted ? (int)((row * cols) & 7) : 0;
  const unsigned groups = (cols + off + 7) / 8;
  const size_t at = row * cols - off;        // of group 0
  auto load = [&](const void* base, unsigned g) -> u32x4 {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at + 8 * (size_t)g;
    if constexpr (FORM != kRagged) return ld4<NT>(reinterpret_cast<const u32x4*>(p));
    if (at + 8 * (size_t)g + 8 <= a.rows * cols) return *reinterpret_cast<const u32x4u*>(p);
    u32x4 v = {0u, 0u, 0u, 0u};              // the buffer's last group
#pragma unroll
    for (unsigned j = 0; j < 8; ++j)
      if (at + 8 * (size_t)g + j < a.rows * cols) v[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    return v;
  };
  auto mine = [&](unsigned g, int j) {       // element j of group g belongs to this row
    const int e = (int)(8 * g) - off + j;
    return FORM != kRagged || (e >= 0 && e < (int)cols);
  };
  auto store = [&](uint16_t* base, unsigned g, u32x4 v) {
    uint16_t* p = base + at + 8 * (size_t)g;
    if constexpr (FORM != kRagged) {
      st4<NT>(reinterpret_cast<u32x4*>(p), v);
      return;
    }
    if (mine(g, 0) && mine(g, 7)) {
      *reinterpret_cast<u32x4u*>(p) = v;
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (mine(g, j)) p[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
  };
  auto gain = [&](unsigned g, float (&w)[8]) {
    if (FORM != kRagged) {
      load_gain<true>(a.weight, a.weight_f32, g, cols, w);
      return;
    }
    const int e = (int)(8 * g) - off;
    if (a.weight && !a.weight_f32 && mine(g, 0) && mine(g, 7)) {
      widen(*reinterpret_cast<const u32x4u*>(static_cast<const uint16_t*>(a.weight) + e), w);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = 1.0f;
      if (a.weight && mine(g, j))
        w[j] = a.weight_f32 ? static_cast<const float*>(a.weight)[e + j]
                            : bf16_f32(static_cast<const uint16_t*>(a.weight)[e + j]);
    }
  };

  // gains are fetched with the row where registers allow: after the row's sum
  // they would be one more trip to memory
  constexpr bool EARLY = V <= 2;
  const RowMean mean = row_mean(cols);
  float h[V][8], w[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[u][j] = w[u][j] = 0.0f;
    if (g >= groups) continue;
    u32x4 x[P];
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = load(in.p[p], g);
    u32x4 r = {0u, 0u, 0u, 0u};
    if (a.residual) r = load(a.residual, g);
    if (EARLY && (a.y || a.codes)) gain(g, w[u]);
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
    if (a.res_out) store(a.res_out, g, narrow(h[u]));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!mine(g, j)) h[u][j] = 0.0f;
      ss = __builtin_fmaf(h[u][j], h[u][j] * mean.part, ss);
    }
  }
  if (!a.y && !a.codes) return;
  if (FORM == kRagged && a.codes)
    for (unsigned i = threadIdx.x; i < (cols + AR_BLOCK - 1) / AR_BLOCK; i += blockDim.x) top[i] = 0;
  put_part(wave_sum(ss), part);
  __syncthreads();
  const float r = 1.0f / sqrtf(sum_parts(part) * mean.rest + a.eps);

  auto keep_scale = [&](size_t block, uint32_t kept) {
    const size_t k = row * a.scale_rs + block * a.scale_cs;
    if (a.scale_e8m0) static_cast<uint8_t*>(a.scales)[k] = (uint8_t)kept;
    else static_cast<uint32_t*>(a.scales)[k] = kept;
  };
  auto scale_of = [&](uint32_t m) { return a.scale_e8m0 ? block_scale<true>(m) : block_scale<false>(m); };
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
    uint32_t m = 0;
    if (g < groups) {
      if (!EARLY) gain(g, w[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = h[u][j] * r * w[u][j];   // y from here on
      if (a.y) store(a.y, g, narrow(h[u]));
    }
    if (!a.codes) continue;
    if constexpr (FORM != kRagged) {
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, finite_mag(h[u][j]));
      const BlockScale s = scale_of(row16_max(m));
      const uint64_t c = codes4_scaled(h[u], s.inv) | (uint64_t)codes4_scaled(h[u] + 4, s.inv) << 32;
      if (g < groups) {
        st8<NT>(reinterpret_cast<uint64_t*>(a.codes + row * a.codes_ld) + g, c);
        if ((threadIdx.x & 15u) == 0) keep_scale(g >> 4, s.kept);
      }
    } else if (g < groups) {
      const int e = (int)(8 * g) - off, split = AR_BLOCK - (e & (AR_BLOCK - 1));   // elements before the next block
      uint32_t m2 = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!mine(g, j)) continue;
        const uint32_t f = finite_mag(h[u][j]);
        if (e >= 0 && j < split) m = max(m, f);
        else m2 = max(m2, f);
      }
      if (e >= 0) atomicMax(&top[e / AR_BLOCK], m);
      if (e < 0) atomicMax(&top[0], m2);
      else if (split < 8 && e + split < (int)cols) atomicMax(&top[e / AR_BLOCK + 1], m2);
    }
  }
  if (FORM != kRagged || !a.codes) return;
  __syncthreads();
  for (unsigned i = threadIdx.x; i < (cols + AR_BLOCK - 1) / AR_BLOCK; i += blockDim.x) keep_scale(i, scale_of(top[i]).kept);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
    if (g >= groups) continue;
    const int e = (int)(8 * g) - off, b0 = max(e, 0) / AR_BLOCK, b1 = min(e + 7, (int)cols - 1) / AR_BLOCK;
    const float i0 = scale_of(top[b0]).inv, i1 = b1 == b0 ? i0 : scale_of(top[b1]).inv;
    const uint64_t c0 = codes4_scaled(h[u], i0) | (uint64_t)codes4_scaled(h[u] + 4, i0) << 32;
    const uint64_t c1 = codes4_scaled(h[u], i1) | (uint64_t)codes4_scaled(h[u] + 4, i1) << 32;
    uint8_t* to = a.codes + row * a.codes_ld + e;
    if (b0 == b1 && mine(g, 0) && mine(g, 7)) {
      typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
      *reinterpret_cast<u32x2u*>(to) = u32x2u{(uint32_t)c0, (uint32_t)(c0 >> 32)};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (mine(g, j)) to[j] = (uint8_t)(((e + j) / AR_BLOCK == b0 ? c0 : c1) >> (8 * j));
    }
  }
}

// Gradient.  With r = 1 / sqrt(mean(h^2) + eps), x = h r and g = dy w:
//   dx = dres + r (g - x mean(g x)),   dweight = sum over rows of dy x.
// Workgroup b takes rows b, b + grid, ...; a lane keeps the sums of dy x of
// its own columns in registers and writes them once, to row b of `partial`.
// A row costs two sums over the workgroup, so the next row's data are on
// their way while this one's are summed (V = 8 has no registers for that).
template <int V, int FORM>
__global__ __launch_bounds__(V == 8 ? 1024 : 512) void k_norm_bwd(NormBwdArgs a) {
  __shared__ __align__(16) float part[2][2][kMaxWaves];
  const unsigned cols = a.cols, groups = (cols + 7) / 8;
  constexpr bool AHEAD = V < 8, WHOLE = FORM != kRagged, NT = FORM == kStream;
  const RowMean mean = row_mean(cols);
  struct Row {
    u32x4 h[V], dy[V], dres[V];
  };
  auto fetch = [&](size_t row, Row& x) {
    const size_t at = row * cols;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const unsigned g = u * blockDim.x + threadIdx.x;
      x.h[u] = x.dy[u] = x.dres[u] = u32x4{0u, 0u, 0u, 0u};
      if (g >= groups) continue;
      x.h[u] = load_group<NT, WHOLE>(a.h + at, g, cols);
      x.dy[u] = load_group<NT, WHOLE>(a.dy + at, g, cols);
      if (a.dres) x.dres[u] = load_group<NT, WHOLE>(a.dres + at, g, cols);
    }
  };
  float dw[V][8], w[V][8];
  Row now;
  fetch(blockIdx.x, now);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[u][j] = w[u][j] = 0.0f;
    if (g < groups) load_gain<WHOLE>(a.weight, a.weight_f32, g, cols, w[u]);
  }
  int flip = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    Row next = now;
    if (AHEAD && row + gridDim.x < a.rows) fetch(row + gridDim.x, next);
    float ss = 0.0f, gh = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float h[8], dy[8];
      widen(now.h[u], h);
      widen(now.dy[u], dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hp = h[j] * mean.part;
        ss = __builtin_fmaf(h[j], hp, ss);
        gh = __builtin_fmaf(dy[j] * w[u][j], hp, gh);
      }
    }
    // two sets of slots in turn: a wave may write the next row's sums while
    // another still reads this row's, and is held at the next barrier before
    // it could write these slots again
    put_part(wave_sum(ss), part[flip][0]);
    put_part(wave_sum(gh), part[flip][1]);
    __syncthreads();
    const float r = 1.0f / sqrtf(sum_parts(part[flip][0]) * mean.rest + a.eps);
    const float m = r * (sum_parts(part[flip][1]) * mean.rest);   // mean(g x)
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const unsigned g = u * blockDim.x + threadIdx.x;
      float h[8], dy[8], dx[8];
      // widened again, not kept in twice the registers over the barrier
      asm volatile("" : "+v"(now.h[u]), "+v"(now.dy[u]));
      widen(now.h[u], h);
      widen(now.dy[u], dy);
      widen(now.dres[u], dx);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = h[j] * r;
        const float d = r * (dy[j] * w[u][j] - x * m);
        dx[j] = a.dres ? d + dx[j] : d;
        dw[u][j] = __builtin_fmaf(dy[j], x, dw[u][j]);
      }
      if (a.dx && g < groups) store_group<NT, WHOLE>(a.dx + row * cols, g, cols, narrow(dx));
    }
    if (AHEAD) now = next;
    else if (row + gridDim.x < a.rows) fetch(row + gridDim.x, now);
  }
  if (!a.partial) return;
  float* out = a.partial + (size_t)blockIdx.x * sum_stride(cols);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const unsigned g = u * blockDim.x + threadIdx.x;
#pragma unroll
    for (unsigned j = 0; j < 8; ++j)
      if (WHOLE ? g < groups : 8 * g + j < cols) out[8 * g + j] = dw[u][j];
  }
}

// dweight[c] = sum of `n` rows of partial sums: a workgroup takes 64 columns,
// four a lane, and each 16 lanes every 64th row.
__global__ __launch_bounds__(1024) void k_sum_rows(const float* partial, float* out, unsigned n, unsigned cols) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ __align__(16) float part[64][64 + 4];
  const unsigned c = (threadIdx.x % 16) * 4, q = threadIdx.x / 16, c0 = blockIdx.x * 64;
  const size_t ld = sum_stride(cols);
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c0 + c < cols) {
    const float* p = partial + c0 + c;
#pragma unroll 8
    for (unsigned i = q; i < n; i += 64) s += *reinterpret_cast<const f32x4*>(p + i * ld);
  }
  *reinterpret_cast<f32x4*>(&part[q][c]) = s;
  __syncthreads();
  if (threadIdx.x >= 64 || c0 + threadIdx.x >= cols) return;
  float t = 0.0f;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) t += part[i][threadIdx.x];
  out[c0 + threadIdx.x] = t;
}

// Lanes and groups per lane for a row of at most `groups` groups: one group a
// lane, or `v` where one gives a lane too few loads to wait for, doubled until
// 1024 lanes hold the row.
struct RowShape {
  int block, v;
};
RowShape row_shape(size_t groups, int v) {
  while (v < 8 && cdiv(groups, v) > 1024) v *= 2;
  return RowShape{(int)(cdiv(cdiv(groups, v), kWave) * kWave), v};
}

// One workgroup per row; HIP takes fewer than 2^32 lanes along one axis.
dim3 row_grid(size_t rows) {
  const size_t x = rows < (1u << 20) ? rows : (1u << 20);
  return dim3((unsigned)x, (unsigned)cdiv(rows, x));
}

// Non-temporal accesses where a call moves more than the last-level cache
// holds (256 MiB): 8 ranks, [16384 x 8192], fp8 result: 464 us, plain 526;
// [1024 x 8192] 31.6, plain 28.9; [128 x 8192] 7.4, plain 5.9.
constexpr size_t kStreamBytes = (size_t)256 << 20;

template <int P, int V>
hipError_t norm_pv(const Launch& L, const InPtrs& in, const NormArgs& a, int block) {
  const dim3 grid = row_grid(a.rows), blk(block);
  if (a.cols % 8) return launch_k(k_reduce_norm<P, V, kRagged>, grid, blk, 0, L.stream, in, a);
  const size_t bytes = a.rows * a.cols * (2 * (P + (a.residual ? 1 : 0) + (a.res_out ? 1 : 0) + (a.y ? 1 : 0)) + (a.codes ? 1 : 0));
  if (bytes > kStreamBytes) return launch_k(k_reduce_norm<P, V, kStream>, grid, blk, 0, L.stream, in, a);
  return launch_k(k_reduce_norm<P, V, kWhole>, grid, blk, 0, L.stream, in, a);
}

// Two groups a lane for up to 3 contributions (1 rank, [16384 x 8192]: 168
// us, with one 208; 3 ranks, [1001 x 5003]: 14.1 and 16.9), one for more (8
// ranks, [16384 x 8192]: 464 us, with two 483; a single row 5.0 and 5.2).
template <int P>
hipError_t norm_p(const Launch& L, const InPtrs& in, const NormArgs& a) {
  const RowShape s = row_shape((a.cols + (a.cols % 8 && a.cols <= kMaxShifted ? 14 : 7)) / 8, P < 4 ? 2 : 1);
  switch (s.v) {
    case 1: return norm_pv<P, 1>(L, in, a, s.block);
    case 2: return norm_pv<P, 2>(L, in, a, s.block);
    case 4: return norm_pv<P, 4>(L, in, a, s.block);
    default: return norm_pv<P, 8>(L, in, a, s.block);
  }
}

template <int V>
hipError_t bwd_v(const Launch& L, const NormBwdArgs& a, unsigned grid, int block) {
  const dim3 g(grid), blk(block);
  if (a.cols % 8) return launch_k(k_norm_bwd<V, kRagged>, g, blk, 0, L.stream, a);
  const size_t bytes = a.rows * a.cols * 2 * (2 + (a.dres ? 1 : 0) + (a.dx ? 1 : 0));
  if (bytes > kStreamBytes) return launch_k(k_norm_bwd<V, kStream>, g, blk, 0, L.stream, a);
  return launch_k(k_norm_bwd<V, kWhole>, g, blk, 0, L.stream, a);
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

namespace {

// Two groups a lane up to 256 lanes a row (one in a single wave), four beyond,
// to have loads on their way; 8 waves a CU, which the registers allow
// ([1000 x 4096]: two groups 14.0 us, four 17.3; [16384 x 4096] 95 and 103;
// [4096 x 5003] in 320 lanes of two 72, in 192 of four 56).
RowShape bwd_shape(size_t cols) {
  const size_t groups = cdiv(cols, 8);
  int v = groups <= kWave ? 1 : cdiv(groups, 2) <= 256 ? 2 : 4;
  if (cdiv(groups, v) > 512) v = 8;
  return RowShape{(int)(cdiv(cdiv(groups, v), kWave) * kWave), v};
}

// Four rows a workgroup at least, once there is one for each CU: each costs a
// row of partial sums, written and read ([1000 x 4096]: 1000 workgroups 20.3
// us, 256 18.1).  (Counted for 256 CUs, so that the order of the sums, and
// the workspace, do not depend on the device.)
size_t bwd_grid(size_t rows, size_t cols) {
  const size_t most = 256 * std::max(1, 8 * kWave / bwd_shape(cols).block);
  return std::min({rows, most, std::max<size_t>(256, rows / 4)});
}

}  // namespace

size_t norm_bwd_sums(size_t rows, size_t cols) { return cols ? bwd_grid(rows, cols) * sum_stride(cols) : 0; }

hipError_t launch_norm_bwd(const Launch& L, const NormBwdArgs& a, float* dweight) {
  const RowShape s = bwd_shape(a.cols);
  const unsigned grid = (unsigned)bwd_grid(a.rows, a.cols);
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
  return launch_k(k_sum_rows, dim3((unsigned)cdiv(a.cols, 64)), dim3(1024), 0, L.stream,
                  static_cast<const float*>(a.partial), dweight, grid, a.cols);
}

}  // namespace ar
