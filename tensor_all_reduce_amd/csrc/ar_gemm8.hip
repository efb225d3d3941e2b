// Product of two E4M3 matrices with a scale for each block of 128 along K:
//   C[m,n] = sum over blocks j of  sa[m,j] * sb[n,j] * sum over k in j of a[m,k] b[n,k]
// (sb of a row of b, or of 128 rows), accumulated in binary32, one rounding
// to bf16 or none.
//
// A block of 128 is one matrix instruction deep (16 x 16 x 128), so scales
// meet the products at its boundary:
// - E8M0 scales are operands of the instruction and cost nothing;
// - binary32 scales: the product of a block starts from zero and is scaled
//   and added to the sum by four fused multiply-adds a lane, which run beside
//   the next instructions of the matrix cores (alone, random operands: 4.2
//   PFLOP/s, with the four 3.6);
// - a binary32 result takes its products as bf16.  The fp8 instructions drop
//   the low bits of terms far below the largest of their sum: 1.2e-5 to
//   2.6e-5 of the result's size, far below bf16's rounding of 1.7e-3 but not
//   below binary32's.  bf16 holds every code exactly, its products reach 1e-7
//   at half the rate.
#include "ar_device.hpp"
#include "ar_internal.hpp"

#include <algorithm>
#include <utility>

namespace ar {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBK = AR_BLOCK;  // one scale block: 128 codes = 8 chunks of 16 bytes

// Keeps codes k .. k+15 of a row that lie before K, zeros after: neither
// operand's padding (which may hold NaN codes) reaches a product.
__device__ __forceinline__ u32x4 mask_chunk(u32x4 v, unsigned k, unsigned K) {
#pragma unroll
  for (unsigned w = 0; w < 4; ++w) {
    const unsigned at = k + 4 * w, n = K > at ? K - at : 0;
    v[w] &= n >= 4 ? ~0u : (1u << (8 * n)) - 1u;
  }
  return v;
}

// Start of the 16 codes read for codes k .. k+15: k itself, or, past the
// row's end, its last 16 (masked away by the caller).
__device__ __forceinline__ unsigned chunk_at(unsigned k, unsigned K) { return min(k, (K - 1) & ~15u); }

__device__ __forceinline__ u32x4 load_chunk(const uint8_t* row, unsigned k, unsigned K) {
  return mask_chunk(*reinterpret_cast<const u32x4*>(row + chunk_at(k, K)), k, K);
}

// Chunk c of row r sits at position c ^ (r % 8): the 16 rows that a wave
// reads at one chunk then spread over all banks.
__device__ __forceinline__ int lds_at(int r, int c) { return r * 8 + (c ^ (r & 7)); }

__device__ __forceinline__ float e8m0_f32(uint8_t b) {
  return b == 255 ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(1.0f, (int)b - 127);
}

// Two results as bf16, nearest even by the conversion instruction; NaN as the
// canonical 0x7FC0.
__device__ __forceinline__ uint32_t results_bf16x2(float lo, float hi) {
  typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
  union { b16x2 b; uint32_t u; } r;
  const float nan = __uint_as_float(0x7FC00000u);
  r.b = b16x2{(__bf16)(__builtin_isnan(lo) ? nan : lo), (__bf16)(__builtin_isnan(hi) ? nan : hi)};
  return r.u;
}

// Four consecutive results of a row from element `at` (column n).
template <bool OUT32>
__device__ __forceinline__ void store4(void* c, size_t at, unsigned n, unsigned N, bool aligned, f32x4 v) {
  if (n + 4 <= N && aligned) {
    if constexpr (OUT32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(c) + at) = v;
    } else {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(c) + at) = u32x2{results_bf16x2(v[0], v[1]), results_bf16x2(v[2], v[3])};
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < N) {
      if constexpr (OUT32) static_cast<float*>(c)[at + r] = v[r];
      else static_cast<uint16_t*>(c)[at + r] = to_bf16(v[r]);
    }
}

typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));

// 32 codes of one row: what a lane gives to one 16 x 16 x 128 product.
union Frag {
  u32x4 h[2];
  i32x8 v;
  uint32_t w[8];
};

// The same 32 codes as bf16 (exact), for four 16 x 16 x 32 products; times
// `scale`, a power of two.
struct Wide {
  b16x8 p[4];
};
__device__ __forceinline__ Wide widen(const Frag& f, float scale = 1.0f) {
  typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
  Wide r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const b16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f.w[i], scale, false);
    const b16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f.w[i], scale, true);
    b16x8& d = r.p[i / 2];
    const int o = 4 * (i & 1);
    d[o] = lo[0];
    d[o + 1] = lo[1];
    d[o + 2] = hi[0];
    d[o + 3] = hi[1];
  }
  return r;
}

// f(0) ... f(N - 1), each index a compile-time constant.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F& f, std::integer_sequence<int, I...>) {
  (f(SPc<I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// Copies 16 bytes a lane from byte `lane` + `at` of a buffer to LDS, the lanes
// of a wave side by side from byte address `lds`: no register holds them on the
// way.  A lane beyond the buffer's end reads nothing, which tiles past the last
// row and blocks past the last of K rely on; the two parts are added in the
// lane's register, whose check against the buffer's size is certain, and not in
// the instruction, whose check of a scalar offset beyond that size is not.
// (Added at each copy: sums kept over the loop would take registers.)  The
// caller waits for the copy (vmcnt) before a barrier.  Five wait states come
// before it: the compiler may have written one of its scalar registers by a
// vector instruction (v_readfirstlane, or v_readlane of a spilled one) right
// before, and adds waits only to instructions that it emits itself.  M0 it keeps
// for its own short uses and sets before each.
typedef uint32_t Resource __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void copy_to_lds(Resource r, uint32_t lane, uint32_t at, uint32_t lds) {
  asm("" : "+s"(at));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(lane + at), "s"(r) : "memory");
}

// `rows` rows of a code matrix from `p` on, as a bounded buffer.  (Word 3:
// the 32-bit data format; untyped access takes any.)
__device__ __forceinline__ Resource rows_buffer(const uint8_t* p, unsigned rows, unsigned most, size_t ld, unsigned K) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t bytes = (min(rows, most) - 1) * (uint32_t)ld + ((K + 15) & ~15u);
  return Resource{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                  (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                  (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Joins the parts of a result that waves of different workgroups have summed
// over slices of K: a wave's part holds its lanes' accumulators, `Q` vectors,
// as the lanes have them, and parts of one result are joined wave by wave, so
// that no wave waits for its workgroup and the last ones to arrive, which do
// the work, are spread over the device.  The last wave adds all parts in slice
// order, so the result does not depend on which was last.  Parts are written
// through the L2 of the writer's XCD; the counter is zero again afterwards.
// Returns whether this wave has the result (in v).
template <int Q>
__device__ __forceinline__ bool join_parts(f32x4 (&v)[Q], uint32_t* counter, char* parts, int slice, int slices) {
  constexpr unsigned bytes = Q * kWave * 16;
  char* mine = parts + (size_t)slice * bytes;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    union { f32x4 f; u32x4 u; } x;
    x.f = v[q];
    st16<2>(mine, bytes, (q * kWave + lane_id()) * 16, x.u);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the part is out
  uint32_t before = 0;
  if (lane_id() == 0) before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  before = __builtin_amdgcn_readfirstlane((int)before);
  if (before != (uint32_t)slices - 1) return false;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  if (lane_id() == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  // 16 vectors at a time are on their way at once: read one after the other,
  // each would cost a trip to memory
  constexpr int QB = Q < 4 ? Q : 4, SB = 16 / QB;
#pragma unroll
  for (int q0 = 0; q0 < Q; q0 += QB) {
    f32x4 sum[QB];
#pragma unroll
    for (int q = 0; q < QB; ++q) sum[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < slices; s += SB) {
      f32x4 x[SB][QB];
#pragma unroll
      for (int b = 0; b < SB; ++b)
#pragma unroll
        for (int q = 0; q < QB; ++q) {
          x[b][q] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (s + b < slices)
            x[b][q] = *reinterpret_cast<const f32x4*>(parts + (size_t)(s + b) * bytes + ((q0 + q) * kWave + lane_id()) * 16);
        }
#pragma unroll
      for (int b = 0; b < SB; ++b)
#pragma unroll
        for (int q = 0; q < QB; ++q) sum[q] += x[b][q];
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) v[q0 + q] = sum[q];
  }
  return true;
}

// BM x 256 tiles of C in 512 lanes, K >= 1.  8 waves, 2 along M by 4 along N,
// each with JT x 4 products of 16 x 16 x 128 a block.
//
// A wave holds the four b fragments of its block and a ring of four fragments
// of a; each register is refilled as soon as its last product is issued, from
// the same block or from the next one, which by then is in the other LDS
// buffer.  One barrier a block, after which the copies of block k + 2 start
// into the buffer of block k.  A workgroup takes tile after tile, and the
// blocks of the next follow those of one without a gap.  SPLIT: it has one
// tile and a slice of K, `per` blocks of it, and the parts are joined.
//
// Why this shape: 256 x 256 is the largest tile whose sums leave registers
// for the fragments, two waves a SIMD, and whose two blocks fit LDS; each
// byte copied serves 256 products.  b through registers straight from memory
// was slower (a fragment's lanes are 16 rows apart in memory, and the vector
// cache serves 16 bytes an access: 1446 us where this took 959).  Measured,
// 16384 x 8192 x 8192: E8M0 820-890 us (2.5-2.7 PFLOP/s), binary32 scales
// 890-940 (2.3-2.5); the same without its copies 700 and 782, with copies
// that always hit the L2 785 and 882: what is left is the trip of each
// block's first reader beyond the L2, for which there is no third buffer.
template <int BM, bool E8M0, bool BROWS, bool OUT32, bool SPLIT>
__global__ __launch_bounds__(512) void k_gemm_big(GemmArgs g, unsigned tiles_m, unsigned tiles_n, int problems, int slices,
                                                  unsigned per, uint32_t* counters, char* parts) {
  constexpr int BN = 256, IT = 4, JT = BM / 32, R = 4;
  constexpr bool HW = E8M0 && !OUT32;        // scales applied by the matrix cores
  constexpr bool FOLD = E8M0 && OUT32;       // or as codes become bf16
  constexpr uint32_t kBuf = (BM + BN) * kBK;
  constexpr int kOut = OUT32 ? 4 : 2;        // bytes of a result
  __shared__ __align__(16) char lab[2][kBuf];  // rows of a, then of b
  // scales of a block, the four rows r, r + 16, r + 32, r + 48 of each 64
  // side by side: bytes (HW) or binary32 words
  __shared__ __align__(16) uint32_t ls[3][HW ? 128 : 512];
  __shared__ __align__(16) char lout[8][16 * 64 * kOut];  // 16 rows of a wave's results
  const int slice = SPLIT ? blockIdx.z % slices : 0;
  const int t = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int lr = lane & 15, lq = lane >> 4;
  const int wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * 64;
  const unsigned kb0 = SPLIT ? slice * per : 0;  // first block
  const unsigned K = SPLIT ? min(g.K - kb0 * kBK, per * kBK) : g.K;
  const unsigned real = (K + kBK - 1) / kBK;
  // 128-row tiles take any K: copies and scales run three blocks ahead, and
  // blocks past K are masked (256-row tiles have no register for that: K > 256)
  constexpr bool SHORT = BM == 128 && !SPLIT;
  const unsigned nk = SHORT ? max(real, 3u) : real;
  const unsigned whole = K / kBK;            // K blocks without a tail
  const unsigned each_tiles = tiles_m * tiles_n, tiles = SPLIT ? each_tiles : each_tiles * (unsigned)problems;

  // XCD x (workgroups reach the 8 XCDs in turn) takes a contiguous run of
  // tiles, ordered in columns of 8 tiles along M, so that the tiles an XCD
  // works on at once share rows of a and of b in its L2
  struct Tile {
    unsigned m0, n0;
    int z;                                   // problem
  };
  auto tile_at = [&](unsigned id) {
    if (id < (tiles & ~7u)) id = (id & 7u) * (tiles >> 3) + (id >> 3);
    const unsigned z = SPLIT ? blockIdx.z / slices : id / each_tiles, one = SPLIT ? id : id % each_tiles;
    const unsigned per = 8 * tiles_n, band = one / per, in = one % per;
    const unsigned bm = min(8u, tiles_m - band * 8);
    return Tile{(unsigned)__builtin_amdgcn_readfirstlane((int)((band * 8 + in % bm) * BM)),
                (unsigned)__builtin_amdgcn_readfirstlane((int)(in / bm * BN)), __builtin_amdgcn_readfirstlane((int)z)};
  };
  auto a_rows = [&](Tile q) { return rows_buffer(g.a[q.z] + (size_t)q.m0 * g.lda + kb0 * kBK, g.M - q.m0, BM, g.lda, K); };
  auto b_rows = [&](Tile q) { return rows_buffer(g.b[q.z] + (size_t)q.n0 * g.ldb + kb0 * kBK, g.N - q.n0, BN, g.ldb, K); };

  // a wave copies 8 rows at a time; chunk c of a row goes to position c ^ (row % 8)
  const unsigned crow = wave * 8 + (lane >> 3), ccol = ((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t va = crow * (uint32_t)g.lda + ccol, vb = crow * (uint32_t)g.ldb + ccol;
  auto piece = [&](auto qq, Resource ra, Resource rb, uint32_t at, unsigned buf) {
    constexpr int q = decltype(qq)::value;
    const uint32_t to = lds_address(lab[buf]) + (wave + q * 8) * 8 * kBK;
    if constexpr (q < BM / 64) copy_to_lds(ra, va, q * 64 * (uint32_t)g.lda + at, to);
    else copy_to_lds(rb, vb, (q - BM / 64) * 64 * (uint32_t)g.ldb + at, to);
  };
  constexpr int kPieces = (BM + BN) / 64;

  // this lane's scale: of row t of a, or of row t - BM of b
  const bool is_a = wave * kWave < BM;       // the same in a wave
  const uint32_t srs = (uint32_t)(is_a ? g.sa_rs : g.sb_rs), scs = (uint32_t)(is_a ? g.sa_cs : g.sb_cs);
  const unsigned slast = (is_a ? g.M : g.N) - 1, slane = is_a ? t : t - BM;
  const int sput = ((t >> 6) * 16 + (t & 15)) * 4 + ((t >> 4) & 3);
  auto load_scale = [&](Tile q, unsigned k) -> uint32_t {
    unsigned row = min((is_a ? q.m0 : q.n0) + slane, slast);
    if (!BROWS && !is_a) row /= AR_BLOCK;
    const void* sbase = is_a ? g.sa[q.z] : g.sb[q.z];
    const size_t i = (uint64_t)row * srs + (uint64_t)(kb0 + min(k, real - 1)) * scs;
    if constexpr (E8M0) {
      const uint8_t b = static_cast<const uint8_t*>(sbase)[i];
      if constexpr (HW) return b;
      else return __float_as_uint(e8m0_f32(b));
    } else {
      return static_cast<const uint32_t*>(sbase)[i];
    }
  };
  auto put_scale = [&](int r, uint32_t v) {
    if constexpr (HW) reinterpret_cast<uint8_t*>(ls[r])[sput] = (uint8_t)v;
    else ls[r][sput] = v;
  };
  // codes 16 lq .. + 15 and 64 + 16 lq .. + 15 of row lr of a fragment: both
  // operands take K in this order
  const uint32_t r0 = lds_at(lr, lq) * 16, r1 = lds_at(lr, lq + 4) * 16;
  auto read_a = [&](unsigned buf, int j, Frag& f) {
    const char* p = lab[buf] + wm * kBK;
    f.h[0] = *reinterpret_cast<const u32x4*>(p + r0 + j * 16 * kBK);
    f.h[1] = *reinterpret_cast<const u32x4*>(p + r1 + j * 16 * kBK);
  };
  auto read_b = [&](unsigned buf, int i, Frag& f) {
    const char* p = lab[buf] + (BM + wn) * kBK;
    f.h[0] = *reinterpret_cast<const u32x4*>(p + r0 + i * 16 * kBK);
    f.h[1] = *reinterpret_cast<const u32x4*>(p + r1 + i * 16 * kBK);
  };
  auto mask = [&](unsigned k, Frag& f) {
    f.h[0] = mask_chunk(f.h[0], k * kBK + lq * 16, K);
    f.h[1] = mask_chunk(f.h[1], k * kBK + lq * 16 + 64, K);
  };

  f32x4 acc[IT][JT];
  Frag fa[R], fb[IT];
  // binary32 scales: a block's product waits D products for its turn to be
  // scaled and added, while the matrix cores run on
  constexpr int D = OUT32 ? IT : 3, NP = 2 * IT;
  f32x4 p[HW || FOLD ? 1 : NP];
  using ScaleA = std::conditional_t<HW, uint32_t, f32x4>;  // of a: four rows of this lane
  struct ScaleB {
    uint32_t bytes;                          // HW: of row lr of each fragment
    f32x4 row[!HW && !FOLD && BROWS ? IT : 1];  // FOLD: the same; else of this lane's four rows of each, or [0][0] of all
  };
  ScaleA sa[JT / 4];
  ScaleB sb;
  uint32_t sc;
  int cur = 0, nxt = 1, aft = 2;             // scale buffers of blocks k, k + 1, k + 2

  auto read_sa = [&](int buf, int h, ScaleA& v) {
    if constexpr (HW) v = ls[buf][wm / 4 + h * 16 + lr];
    else v = *reinterpret_cast<const f32x4*>(&ls[buf][wm + h * 64 + lr * 4]);
  };
  auto read_sb = [&](int buf, ScaleB& v) {
    if constexpr (HW) {
      v.bytes = ls[buf][(BM + wn) / 4 + lr];
    } else if constexpr (FOLD) {
      v.row[0] = *reinterpret_cast<const f32x4*>(&ls[buf][BM + wn + lr * 4]);
    } else if constexpr (BROWS) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(&ls[buf][BM + wn + (lq * 4 + r) * 4]);
#pragma unroll
        for (int i = 0; i < IT; ++i) v.row[i][r] = q[i];
      }
    } else {
      v.row[0][0] = __uint_as_float(ls[buf][BM + wn]);
    }
  };

  // Order of a block's products: column by column of a's fragments but for
  // the last four columns, which go row by row.  So the first part frees
  // fragments of a one by one, for the block's last four, and the second
  // fragments of b, for the next block.
  constexpr int F = (JT - 4) * IT;           // products of the first part
  constexpr int BAR = F + 3;                 // the barrier comes after this product
  auto add = [&](auto nn) {
    constexpr int n = decltype(nn)::value, i = n < F ? n % IT : (n - F) / 4, j = n < F ? n / IT : JT - 4 + (n - F) % 4;
    if constexpr (!HW && !FOLD) {
      const float s = sa[j / 4][j % 4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = __builtin_fmaf(p[n % NP][r], s * sb.row[BROWS ? i : 0][BROWS ? r : 0], acc[i][j][r]);
    }
  };

  unsigned buf = 0;                          // LDS buffer of block k
  Tile now, then;                            // this tile and the next
  Resource now_a, now_b, then_a, then_b;
  // block k + d: of this tile, or from the next one's start
  auto ahead = [&](unsigned k, unsigned d) { return k + d < nk ? k + d : k + d - nk; };

  auto step = [&](unsigned k, auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
    if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < IT; ++i) mask(k, fb[i]);
    }
    const bool over1 = k + 1 >= nk, over2 = k + 2 >= nk, over3 = k + 3 >= nk;
    const Resource ra1 = over1 ? then_a : now_a, rb1 = over1 ? then_b : now_b;
    const Resource ra2 = over2 ? then_a : now_a, rb2 = over2 ? then_b : now_b;
    const uint32_t at1 = ahead(k, 1) * kBK, at2 = ahead(k, 2) * kBK;
    ScaleA nsa;
    ScaleB nsb;
    if constexpr (JT == 8) read_sa(cur, 1, sa[JT / 4 - 1]);
    Wide wa[OUT32 ? 4 : 1];
    auto cell = [&](auto nn) {
      constexpr int n = decltype(nn)::value, i = n < F ? n % IT : (n - F) / 4, j = n < F ? n / IT : JT - 4 + (n - F) % 4;
      Frag& a = fa[j % R];
      if constexpr (TAIL && i == 0) mask(k, a);
      if constexpr (HW) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i].v, a.v, acc[i][j], 0, 0, i, (int)sb.bytes, j % 4,
                                                                  (int)sa[j / 4]);
      } else if constexpr (!OUT32) {
        p[n % NP] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i].v, a.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
      } else {
        // JT is 4: a row of four products, each the sum of four of 32 codes
        if constexpr (n < 4) wa[n] = widen(a, FOLD ? sa[0][n] : 1.0f);
        if constexpr (FOLD && n % 4 == 3) {
          const Wide wb = widen(fb[i], sb.row[0][i]);
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb.p[h], wa[c].p[h], acc[i][c], 0, 0, 0);
        }
        if constexpr (!FOLD && n % 4 == 3) {
          const Wide wb = widen(fb[i]);
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              p[(n - 3 + c) % NP] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  wb.p[h], wa[c].p[h], h ? p[(n - 3 + c) % NP] : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        }
      }
      if constexpr (!HW && !OUT32 && n >= D) add(SPc<n - D>{});
      if constexpr (OUT32 && !FOLD && n >= 7 && n % 4 == 3) {
        each<4>([&](auto c) { add(SPc<n - 7 + decltype(c)::value>{}); });
      }
      if constexpr (n == BAR) {
        // every wave's copies of block k + 1 are in LDS, and none still
        // reads block k, whose buffer block k + 2 takes
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      }
      if constexpr (n == BAR + 1) {
        // scales go through a register: those of block k + 2 came during the
        // last block (nothing is in flight here, so nothing is waited for)
        put_scale(aft, sc);
        sc = load_scale(over3 ? then : now, ahead(k, 3));
      }
      if constexpr (n == BAR + 3) {
        read_sb(nxt, nsb);
        read_sa(nxt, 0, nsa);
      }
      // a wave's copies, spread over the products so that they never queue
      // up before one: the first of block k + 2, then, before the barrier,
      // the rest of block k + 1
      constexpr int after = n - BAR - 1, EARLY = (JT * IT - BAR) / 2;
      if constexpr (after >= 1 && after % 2 == 1 && after / 2 < EARLY && after / 2 < kPieces) {
        piece(SPc<after / 2>{}, ra2, rb2, at2, buf);
      } else if constexpr (n < BAR && n % 3 == 0 && EARLY + n / 3 < kPieces) {
        piece(SPc<EARLY + n / 3>{}, ra1, rb1, at1, buf ^ 1);
      }
      if constexpr (n < F) {
        if constexpr (i == IT - 1) read_a(buf, j + 4, fa[j % R]);
      } else {
        if constexpr (j == JT - 1) read_b(buf ^ 1, i, fb[i]);
        if constexpr (i == IT - 1) read_a(buf ^ 1, j - (JT - 4), fa[j % R]);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    each<JT * IT>(cell);
    if constexpr (!HW) each<D>([&](auto n) { add(SPc<JT * IT - D + decltype(n)::value>{}); });
    sb = nsb;
    sa[0] = nsa;
    const int r = cur;
    cur = nxt;
    nxt = aft;
    aft = r;
    buf ^= 1;
  };

  // Results go out 16 rows of a wave at a time through its own LDS, so that
  // neighbouring lanes store neighbouring bytes of a row.
  auto store = [&](Tile q) {
    char* const out = lout[wave];
    constexpr int kRow = 64 * kOut, kLanes = kRow / 16;  // bytes of a row, lanes that store it
    const unsigned n = q.n0 + wn + (lane % kLanes) * (16 / kOut);
    const bool vec = (g.ldc * kOut) % 16 == 0 && n + 16 / kOut <= g.N;
#pragma unroll
    for (int j = 0; j < JT; ++j) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const f32x4 v = acc[i][j];
        if constexpr (OUT32) {
          *reinterpret_cast<f32x4*>(out + lr * kRow + ((i * 4 + lq) ^ (lr & 7)) * 16) = v;
        } else {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          *reinterpret_cast<u32x2*>(out + lr * kRow + ((i * 2 + (lq >> 1)) ^ (lr & 7)) * 16 + (lq & 1) * 8) =
              u32x2{results_bf16x2(v[0], v[1]), results_bf16x2(v[2], v[3])};
        }
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < 16 * kLanes / kWave; ++h) {
        const int row = h * (kWave / kLanes) + lane / kLanes;
        const u32x4 v = *reinterpret_cast<const u32x4*>(out + row * kRow + ((lane % kLanes) ^ (row & 7)) * 16);
        const unsigned m = q.m0 + wm + j * 16 + row;
        if (m >= g.M) continue;
        char* to = static_cast<char*>(g.c[q.z]) + (m * g.ldc + n) * kOut;
        if (vec) {
          st4<true>(reinterpret_cast<u32x4*>(to), v);   // streamed: the L2 keeps a and b
        } else {
#pragma unroll
          for (unsigned e = 0; e < 16 / kOut; ++e)
            if (n + e < g.N) {
              if constexpr (OUT32) reinterpret_cast<uint32_t*>(to)[e] = v[e];
              else reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
            }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  unsigned id = blockIdx.x;
  now = tile_at(id);
  now_a = a_rows(now);
  now_b = b_rows(now);
  // the next tile (without one, this tile again: its blocks are copied and not used)
  auto look_ahead = [&] {
    if (!SPLIT && id + gridDim.x < tiles) then = tile_at(id + gridDim.x);
    else then = now;
    then_a = a_rows(then);
    then_b = b_rows(then);
  };
  look_ahead();
  {
    const bool one = nk == 1;
    const Resource ra1 = one ? then_a : now_a, rb1 = one ? then_b : now_b;
    each<kPieces>([&](auto q) { piece(q, now_a, now_b, 0, 0); });
    each<kPieces>([&](auto q) { piece(q, ra1, rb1, ahead(0, 1) * kBK, 1); });
    put_scale(0, load_scale(now, 0));
    put_scale(1, load_scale(one ? then : now, ahead(0, 1)));
    sc = load_scale(nk <= 2 ? then : now, ahead(0, 2));
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  read_sb(0, sb);
  read_sa(0, 0, sa[0]);
#pragma unroll
  for (int i = 0; i < IT; ++i) read_b(0, i, fb[i]);
#pragma unroll
  for (int j = 0; j < R; ++j) read_a(0, j, fa[j]);
  for (;;) {
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (unsigned k = 0; k < whole; ++k) step(k, std::false_type{});
    if constexpr (SHORT) {
      for (unsigned k = whole; k < nk; ++k) step(k, std::true_type{});
    } else {
      if (whole < nk) step(whole, std::true_type{});
    }
    if constexpr (SPLIT) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy outlives the workgroup's LDS
      const size_t w = ((size_t)now.z * tiles + id) * 8 + wave;
      if (join_parts(reinterpret_cast<f32x4(&)[IT * JT]>(acc), counters + w, parts + w * slices * (IT * JT * kWave * 16), slice,
                     slices))
        store(now);
      return;
    }
    store(now);
    id += gridDim.x;
    if (id >= tiles) break;
    now = then;
    now_a = then_a;
    now_b = then_b;
    look_ahead();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy outlives the workgroup's LDS
}

// Few rows of a: 16 MT x 64 of C in four waves of 16 columns, K >= 1.  The
// codes of b are read once and there is little to compute on them, so the
// kernel is a copy engine: a ring of groups of BG blocks in LDS, all but one of
// them on their way, and two to four workgroups a CU.  A group costs a barrier
// and a chain of latencies, so a group has two blocks, unless rings of one,
// which are smaller, save a second round of workgroups (gemm_few).
// blockIdx: columns, rows, problem and slice of K (`per` blocks each).
constexpr int kFewCols = 64, kFewBlocks = 16;  // columns; blocks whose scales are held at a time
constexpr int few_ring(int mt, int bg) { return bg * (bg == 1 ? 3 : 2) * (16 * mt + kFewCols) * kBK; }  // bytes
constexpr int few_scales(int mt, bool brows) { return kFewBlocks * 4 * (16 * mt + (brows ? kFewCols : 1)); }
template <int MT, int BG, bool E8M0, bool BROWS, bool OUT32>
__global__ __launch_bounds__(256) void k_gemm_few(GemmArgs g, int slices, unsigned per, uint32_t* counters, char* parts) {
  constexpr int BM = 16 * MT, NP = BG == 1 ? 3 : 2, ST = BG * NP;  // groups and blocks in the ring
  constexpr bool HW = E8M0 && !OUT32;
  constexpr int kCopies = 2 + MT / 2;        // of a wave and block
  __shared__ __align__(16) char ring[ST][(BM + kFewCols) * kBK];  // rows of a, then of b
  __shared__ uint32_t lsa[kFewBlocks][BM], lsb[kFewBlocks][BROWS ? kFewCols : 1];
  static_assert(sizeof(ring) == few_ring(MT, BG) && sizeof(lsa) + sizeof(lsb) == few_scales(MT, BROWS));
  const int z = blockIdx.z / slices, slice = blockIdx.z % slices, t = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int lr = lane & 15, lq = lane >> 4;
  const unsigned n0 = blockIdx.x * kFewCols, m0 = blockIdx.y * BM;
  const unsigned nk = (g.K + kBK - 1) / kBK, kb0 = slice * per, kb1 = min(kb0 + per, nk);
  const Resource ra = rows_buffer(g.a[z] + (size_t)m0 * g.lda, g.M - m0, BM, g.lda, g.K);
  const Resource rb = rows_buffer(g.b[z] + (size_t)n0 * g.ldb, g.N - n0, kFewCols, g.ldb, g.K);
  const unsigned crow = lane >> 3, ccol = ((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t va = crow * (uint32_t)g.lda + ccol, vb = crow * (uint32_t)g.ldb + ccol;
  auto copy = [&](unsigned kb, unsigned buf) {
    Resource a = ra, b = rb;
    if (kb >= kb1) a[2] = b[2] = 0;          // past the slice: nothing is read
    const uint32_t to = lds_address(ring[buf]), at = kb * kBK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const unsigned r = wave * 16 + i * 8;
      copy_to_lds(b, vb, r * (uint32_t)g.ldb + at, to + (BM + r) * kBK);
    }
#pragma unroll
    for (int i = 0; i < MT / 2; ++i) {
      const unsigned r = (wave * (MT / 2) + i) * 8;
      copy_to_lds(a, va, r * (uint32_t)g.lda + at, to + r * kBK);
    }
  };
  auto scale_at = [&](const void* p, size_t i) -> uint32_t {
    if constexpr (HW) return static_cast<const uint8_t*>(p)[i];
    else if constexpr (E8M0) return __float_as_uint(e8m0_f32(static_cast<const uint8_t*>(p)[i]));
    else return static_cast<const uint32_t*>(p)[i];
  };

  f32x4 acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t r0 = lds_at(lr, lq) * 16, r1 = lds_at(lr, lq + 4) * 16;
  for (unsigned base = kb0; base < kb1; base += kFewBlocks) {
    const unsigned n = min((unsigned)kFewBlocks, kb1 - base);
    // no wave still uses the last round's blocks and scales
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (unsigned c = 0; c < ST - BG; ++c) copy(c < n ? base + c : kb1, c);
    for (unsigned i = t; i < n * BM; i += 256)
      lsa[i / BM][i % BM] = scale_at(g.sa[z], (size_t)min(m0 + i % BM, g.M - 1) * g.sa_rs + (size_t)(base + i / BM) * g.sa_cs);
    constexpr int BS = BROWS ? kFewCols : 1;
    for (unsigned i = t; i < n * BS; i += 256) {
      const unsigned row = min(n0 + i % BS, g.N - 1);
      lsb[i / BS][i % BS] = scale_at(g.sb[z], (size_t)(BROWS ? row : row / AR_BLOCK) * g.sb_rs + (size_t)(base + i / BS) * g.sb_cs);
    }
    unsigned buf = 0;
    for (unsigned c0 = 0; c0 < n; c0 += BG) {
      // this wave's copies of the group have landed (those of the NP - 2
      // groups after it may be on their way), then every wave's
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NP - 2) * BG * kCopies) : "memory");
      const unsigned free = buf == 0 ? ST - BG : buf - BG;   // the group before: no wave reads it any more
#pragma unroll
      for (unsigned h = 0; h < BG; ++h) {
        const unsigned c = c0 + ST - BG + h;
        copy(c < n ? base + c : kb1, free + h);
      }
      Frag fa[BG][MT], fb[BG];
#pragma unroll
      for (unsigned h = 0; h < BG; ++h) {
        const unsigned kb = base + c0 + h;
        auto read = [&](int row, Frag& f) {
          f.h[0] = *reinterpret_cast<const u32x4*>(ring[buf + h] + row * kBK + r0);
          f.h[1] = *reinterpret_cast<const u32x4*>(ring[buf + h] + row * kBK + r1);
        };
        read(BM + wave * 16, fb[h]);
#pragma unroll
        for (int j = 0; j < MT; ++j) read(j * 16, fa[h][j]);
        if ((kb + 1) * kBK > g.K) {
          auto mask = [&](Frag& f) {
            f.h[0] = mask_chunk(f.h[0], kb * kBK + lq * 16, g.K);
            f.h[1] = mask_chunk(f.h[1], kb * kBK + lq * 16 + 64, g.K);
          };
          mask(fb[h]);
#pragma unroll
          for (int j = 0; j < MT; ++j) mask(fa[h][j]);
        }
      }
#pragma unroll
      for (unsigned h = 0; h < BG; ++h) {
        const unsigned c = c0 + h;
        if (c >= n) break;
        if constexpr (HW) {
          const uint32_t sb = lsb[c][BROWS ? wave * 16 + lr : 0];
#pragma unroll
          for (int j = 0; j < MT; ++j)
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[h].v, fa[h][j].v, acc[j], 0, 0, 0, (int)sb, 0,
                                                                   (int)lsa[c][j * 16 + lr]);
        } else {
          float sb[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) sb[r] = __uint_as_float(lsb[c][BROWS ? wave * 16 + lq * 4 + r : 0]);
          Wide wb;
          if constexpr (OUT32) wb = widen(fb[h]);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
            if constexpr (OUT32) {
              const Wide wa = widen(fa[h][j]);
#pragma unroll
              for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb.p[q], wa.p[q], p, 0, 0, 0);
            } else {
              p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[h].v, fa[h][j].v, p, 0, 0, 0, 0, 0, 0);
            }
            const float sa = __uint_as_float(lsa[c][j * 16 + lr]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][r] = __builtin_fmaf(p[r], sa * sb[r], acc[j][r]);
          }
        }
      }
      buf = buf + BG == ST ? 0 : buf + BG;
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy outlives the workgroup's LDS
  if (slices > 1) {
    const size_t w = (((size_t)z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * 4 + wave;
    if (!join_parts(acc, counters + w, parts + w * slices * (MT * kWave * 16), slice, slices)) return;
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const unsigned m = m0 + j * 16 + lr, n = n0 + wave * 16 + lq * 4;
    if (m < g.M) store4<OUT32>(g.c[z], m * g.ldc + n, n, g.N, (g.ldc & 3) == 0, acc[j]);
  }
}

// 128 x 128 tile of C in a 256-lane workgroup, 64 x 64 a wave as 4 x 4
// products of 16 x 16 x 128: any strides, any K (the other kernels address a
// tile's rows in 32 bits, and are faster: 4096 x 4096 x 4096 278 us here, 65
// in large tiles).  b is the first operand, so a lane ends with four
// consecutive n of one m.  blockIdx: rows, columns, and problem with the rows
// beyond the first axis (HIP takes fewer than 2^32 lanes along one).
template <bool E8M0, bool BROWS, bool OUT32>
__global__ __launch_bounds__(256) void k_gemm_tile(GemmArgs g, int problems) {
  constexpr int BM = 128, BN = 128;
  __shared__ u32x4 la[BM * 8], lb[BN * 8];
  const int z = blockIdx.z % problems, t = threadIdx.x, lane = lane_id(), wave = t / kWave;
  const size_t first = ((size_t)(blockIdx.z / problems) * gridDim.x + blockIdx.x) * BM;
  if (first >= g.M) return;
  const unsigned m0 = (unsigned)first, n0 = blockIdx.y * BN;
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
    Frag fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ra = wm + i * 16 + lr, rb = wn + i * 16 + lr;
      fa[i].h[0] = la[lds_at(ra, 2 * lq)];
      fa[i].h[1] = la[lds_at(ra, 2 * lq + 1)];
      fb[i].h[0] = lb[lds_at(rb, 2 * lq)];
      fb[i].h[1] = lb[lds_at(rb, 2 * lq + 1)];
    }
    auto byte_of = [&](const void* p, size_t i) { return static_cast<const uint8_t*>(p)[i]; };
    auto scale_of = [&](const void* p, size_t i) {
      if constexpr (E8M0) return e8m0_f32(byte_of(p, i));
      else return static_cast<const float*>(p)[i];
    };
    auto at_a = [&](unsigned m) { return (size_t)min(m, g.M - 1) * g.sa_rs + kb * g.sa_cs; };
    auto at_b = [&](unsigned n) {
      const size_t r = min(n, g.N - 1);
      return (BROWS ? r : r / AR_BLOCK) * g.sb_rs + kb * g.sb_cs;
    };
    if constexpr (E8M0 && !OUT32) {
      int sa[4], sb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sa[i] = byte_of(g.sa[z], at_a(m0 + wm + i * 16 + lr));
        sb[i] = byte_of(g.sb[z], at_b(n0 + wn + i * 16 + lr));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i].v, fa[j].v, acc[i][j], 0, 0, 0, sb[i], 0, sa[j]);
    } else {
      float sa[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) sa[j] = scale_of(g.sa[z], at_a(m0 + wm + j * 16 + lr));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float sb[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) sb[r] = scale_of(g.sb[z], at_b(n0 + wn + i * 16 + lq * 4 + r));
        Wide wb;
        if constexpr (OUT32) wb = widen(fb[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
          if constexpr (OUT32) {
            const Wide wa = widen(fa[j]);
#pragma unroll
            for (int h = 0; h < 4; ++h) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb.p[h], wa.p[h], p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i].v, fa[j].v, p, 0, 0, 0, 0, 0, 0);
          }
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

// How a product is cut: the tile, and the slices of K that different
// workgroups take.  Planned for the 256 CUs of the device, so that a
// workspace's size does not depend on where it is asked for.
constexpr unsigned kPlanCus = 256;
constexpr unsigned kLdsBytes = 160 * 1024;  // of a CU
struct Plan {
  int mt;           // few rows: fragments of 16 rows of a; 0: large tiles
  unsigned slices, per;
  size_t tiles;     // of all problems
};

unsigned blocks_of(unsigned K) { return (K + kBK - 1) / kBK; }

// 32 or 64 rows of a and 64 columns a workgroup; slices of at least 8 blocks
// until there are two workgroups a CU.  A join costs 3 to 5 us (parts out to
// memory, a counter, parts back), so more slices lose what they gain: 48 x
// 4096 x 8192 takes 15.1 us in 4 slices, 15.4 in 8 and 20.1 in 16; 1 x 1024 x
// 8192 10.0, 9.2 and 11.3.
Plan plan_few(unsigned M, unsigned N, unsigned K, int G) {
  Plan p{};
  p.mt = M <= 32 ? 2 : 4;
  p.tiles = cdiv(M, 16 * p.mt) * cdiv(N, kFewCols) * G;
  const unsigned nk = blocks_of(K);
  p.slices = (unsigned)std::max<size_t>(1, std::min<size_t>(2 * kPlanCus / p.tiles, nk / 8));
  p.per = (unsigned)cdiv(nk, p.slices);
  p.slices = (unsigned)cdiv(nk, p.per);
  return p;
}

// Which kernel.  Few rows where
// - its workgroups are all resident at once and read the codes of b once: up
//   to 768 of 32 rows, 512 of 64;
// - or there are up to 192 of its 64 x 64 tiles;
// - or up to 1024, and tiles times blocks stay within 16384, where large tiles,
//   cut into slices, lose to their join.
// Either side, us, few rows first.  8192 columns of each of several problems,
// K 8192: 1 row, 512 tiles 58 and 78, 768 81 and 95, 896 112 and 100; 64 rows,
// 384 tiles 60 and 67, 512 69 and 80, 640 107 and 96.  One problem, N 8192, K
// 8192: M 64 21 and 32, M 128 30 and 33, M 192 40 and 35; N 8192, K 1024: M 256
// 8 and 17, M 512 14 and 17, M 768 20 and 17; N 1024, K 8192: M 512 18 and 25,
// M 1024 30 and 30; N 4096, K 4096: M 512 22 and 27, M 768 35 and 32.
bool few_rows(unsigned M, unsigned N, unsigned K, int G) {
  const size_t tiles = cdiv(M, 64) * cdiv(N, kFewCols) * G;
  if (cdiv(M, 32) > 65535) return false;     // a launch's second axis
  return tiles <= (M <= 32 ? 768 : M <= 64 ? 512 : 192) || (tiles <= 1024 && tiles * blocks_of(K) <= 16384);
}

// The counters' part of a workspace, the same for every shape, so that one
// workspace serves products of all shapes in turn: 1024 counters, a wave each.
// Cut into slices are at most 256 tiles of four waves or 128 of eight.
constexpr size_t kCounterBytes = 1024 * 4;
static_assert(kPlanCus <= 256, "counters for every wave of a product in slices");

size_t few_bytes(const Plan& p) {
  return p.slices > 1 ? kCounterBytes + p.tiles * p.slices * (p.mt * 256 * 16) : 0;
}

template <bool E8M0, bool BROWS, bool OUT32>
hipError_t gemm_few(const Launch& L, const GemmArgs& g, int G, void* ws) {
  Plan p = plan_few(g.M, g.N, g.K, G);
  if (!ws) {
    p.slices = 1;
    p.per = blocks_of(g.K);
  }
  uint32_t* counters = static_cast<uint32_t*>(ws);
  char* parts = ws ? static_cast<char*>(ws) + kCounterBytes : nullptr;
  const dim3 grid((unsigned)cdiv(g.N, kFewCols), (unsigned)cdiv(g.M, 16 * p.mt), (unsigned)G * p.slices);
  // Rings of one block where the workgroups of rings of two are more than the
  // device's LDS holds at once and those of one are not: 769 to 1024, with
  // scales for each row of b 513 to 768.  Us, one and two blocks, rows of
  // 1024: 768 workgroups 10.4 and 10.4, 800 11.6 and 13.6, 896 11.8 and 13.8,
  // 1024 12.3 and 14.4; with row scales 512 9.3 and 9.2, 516 9.4 and 12.1, 768
  // 10.7 and 12.8, 896 14.8 and 13.6.
  constexpr size_t held1 = kPlanCus * (kLdsBytes / (few_ring(2, 1) + few_scales(2, BROWS)));
  constexpr size_t held2 = kPlanCus * (kLdsBytes / (few_ring(2, 2) + few_scales(2, BROWS)));
  const size_t groups = p.tiles * p.slices;
  const bool one = groups > held2 && groups <= held1;
  auto k = p.mt == 4 ? k_gemm_few<4, 2, E8M0, BROWS, OUT32>
                     : one ? k_gemm_few<2, 1, E8M0, BROWS, OUT32> : k_gemm_few<2, 2, E8M0, BROWS, OUT32>;
  return launch_k(k, grid, dim3(256), 0, L.stream, g, (int)p.slices, p.per, counters, parts);
}

// Large tiles, one workgroup a CU.  Where 128 x 256 tiles fill half the CUs at
// most, they are cut into slices of about 8 blocks or more.
Plan plan_big(unsigned M, unsigned N, unsigned K, int G) {
  Plan p{};
  p.tiles = cdiv(M, 128) * cdiv(N, 256) * G;
  const unsigned nk = blocks_of(K);
  p.slices = (unsigned)std::max<size_t>(1, std::min<size_t>(kPlanCus / p.tiles, nk / 8));
  p.per = (unsigned)cdiv(nk, p.slices);
  p.slices = (unsigned)cdiv(nk, p.per);
  return p;
}
size_t big_bytes(const Plan& p) { return p.slices > 1 ? kCounterBytes + p.tiles * p.slices * (128 * 256 * 4) : 0; }

template <int BM, bool E8M0, bool BROWS, bool OUT32, bool SPLIT>
hipError_t gemm_tiles(const Launch& L, const GemmArgs& g, int G, const Plan& p, void* ws) {
  uint32_t* counters = static_cast<uint32_t*>(ws);
  char* parts = ws ? static_cast<char*>(ws) + kCounterBytes : nullptr;
  const unsigned tm = (unsigned)cdiv(g.M, BM), tn = (unsigned)cdiv(g.N, 256);
  const dim3 grid(SPLIT ? tm * tn : std::min(tm * tn * G, (unsigned)L.cus), 1, SPLIT ? (unsigned)G * p.slices : 1);
  return launch_k(k_gemm_big<BM, E8M0, BROWS, OUT32, SPLIT>, grid, dim3(512), 0, L.stream, g, tm, tn, G, (int)p.slices,
                  p.per, counters, parts);
}

template <bool E8M0, bool BROWS, bool OUT32>
hipError_t gemm_big(const Launch& L, const GemmArgs& g, int G, void* ws) {
  Plan p = plan_big(g.M, g.N, g.K, G);
  if (ws && p.slices > 1) return gemm_tiles<128, E8M0, BROWS, OUT32, true>(L, g, G, p, ws);
  p.slices = 1;
  p.per = blocks_of(g.K);
  // 256 rows a tile unless registers do not hold it (products as bf16, a
  // binary32 scale for each row of b), it leaves CUs without one, K is short,
  // or 128 rows hold all (8 problems of 8192 columns, K 4096: 16 rows 57 us, in
  // tiles of 256 rows 69; 128 rows 67 and 76)
  if constexpr (!OUT32 && (E8M0 || !BROWS))
    if (g.K > 256 && g.M > 128 && (cdiv(g.M, 256) * cdiv(g.N, 256) * G >= (size_t)L.cus / 2 || g.M % 256 == 0 || g.M % 256 > 128))
      return gemm_tiles<256, E8M0, BROWS, OUT32, false>(L, g, G, p, ws);
  return gemm_tiles<128, E8M0, BROWS, OUT32, false>(L, g, G, p, ws);
}

template <bool E8M0, bool BROWS>
hipError_t gemm_o(const Launch& L, const GemmArgs& g, int G, bool out_f32, void* ws) {
  const size_t wide = (g.lda | g.ldb) >> 23 | (g.sa_rs | g.sa_cs | g.sb_rs | g.sb_cs) >> 32;
  if (!wide && g.K > 0 && few_rows(g.M, g.N, g.K, G))
    return out_f32 ? gemm_few<E8M0, BROWS, true>(L, g, G, ws) : gemm_few<E8M0, BROWS, false>(L, g, G, ws);
  if (!wide && g.K > 0)
    return out_f32 ? gemm_big<E8M0, BROWS, true>(L, g, G, ws) : gemm_big<E8M0, BROWS, false>(L, g, G, ws);
  const size_t tm = cdiv(g.M, 128), x = std::min<size_t>(tm, 1u << 20);
  const dim3 grid((unsigned)x, (unsigned)cdiv(g.N, 128), (unsigned)(G * cdiv(tm, x)));
  if (out_f32) return launch_k(k_gemm_tile<E8M0, BROWS, true>, grid, dim3(256), 0, L.stream, g, G);
  return launch_k(k_gemm_tile<E8M0, BROWS, false>, grid, dim3(256), 0, L.stream, g, G);
}

}  // namespace

size_t gemm_fp8_workspace(size_t M, size_t N, size_t K, int G) {
  const unsigned m = (unsigned)M, n = (unsigned)N, k = (unsigned)K;
  if (few_rows(m, n, k, G)) return few_bytes(plan_few(m, n, k, G));
  return big_bytes(plan_big(m, n, k, G));
}

hipError_t launch_gemm_fp8(const Launch& L, const GemmArgs& g, int G, bool e8m0, bool b_rows, bool out_f32,
                           void* ws) {
  if (e8m0) return b_rows ? gemm_o<true, true>(L, g, G, out_f32, ws) : gemm_o<true, false>(L, g, G, out_f32, ws);
  return b_rows ? gemm_o<false, true>(L, g, G, out_f32, ws) : gemm_o<false, false>(L, g, G, out_f32, ws);
}

}  // namespace ar
