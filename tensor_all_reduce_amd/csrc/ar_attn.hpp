// Building blocks shared by the attention kernels.
//
// Scores are formed transposed, S^T = K Q^T, on the 32 x 32 x 16 (or
// 16 x 16 x 32) matrix instructions: a lane then holds one query's scores of
// several keys, so that a softmax needs one exchange between lanes, and the
// registers that hold P^T are, as they stand, the second operand of
// O^T = V^T P^T.  The order in which that product takes its keys is the order
// of those registers; V^T follows it through transposing reads of LDS.
#pragma once

#include "ar_device.hpp"
#include "ar_internal.hpp"

namespace ar {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Eight bf16 values: what a lane gives to one matrix instruction.
union Frag8 {
  b16x8 b;
  u32x4 u;
  uint32_t w[4];
  s16x4 s[2];
};

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
#define AR_NEG_INF (-__builtin_huge_valf())

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Two values as bf16, nearest even, by the conversion instruction.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  union { b16x2 b; uint32_t u; } r;
  r.b = b16x2{(__bf16)lo, (__bf16)hi};
  return r.u;
}
// The same with any NaN as the canonical 0x7FC0: for results.
__device__ __forceinline__ uint32_t result_bf16x2(float lo, float hi) {
  const float nan = __uint_as_float(0x7FC00000u);
  return cvt_bf16x2(__builtin_isnan(lo) ? nan : lo, __builtin_isnan(hi) ? nan : hi);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Four b16 values of one column out of four rows of LDS: lanes 4 i .. 4 i + 3
// of a group of 16 point to row i's 16 columns, 8 bytes each, and lane c of
// the group gets column c.
__device__ __forceinline__ s16x4 read_tr16(uint32_t addr) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(uintptr_t)addr);
}
// Eight bytes of one column out of eight rows: lanes 2 i, 2 i + 1 point to
// row i's 16 columns.
__device__ __forceinline__ i32x2 read_tr8(uint32_t addr) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(uintptr_t)addr);
}

// Copies 16 bytes a lane from `from` to LDS, the lanes of a wave side by side
// from byte address `lds`, past the registers; a lane that is switched off
// copies nothing and leaves its place as it is.  The caller waits (vmcnt) and
// meets a barrier before the data are read.  The wait states cover the write
// of M0 before the copy reads it.
__device__ __forceinline__ void copy16_to_lds(const void* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(from) : "memory");
}

__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// x / size of a page, x < 2^31.
__device__ __forceinline__ unsigned page_of(unsigned x, const Pages& c) {
  return c.shift == 32 ? x : __umulhi(x, c.magic) >> c.shift;
}

// A wave's inclusive sums over its lanes.
__device__ __forceinline__ unsigned wave_scan(unsigned v) {
  const int lane = lane_id();
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const unsigned u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Rows first .. first + count - 1 of sequence s out of the offsets cu.  Any
// contents of cu give rows below `rows`.
struct Rows {
  unsigned first, count;
};
__device__ __forceinline__ Rows rows_of(const int32_t* cu, unsigned s, unsigned rows) {
  const unsigned a = (unsigned)min(max(cu[s], 0), (int)rows), b = (unsigned)min(max(cu[s + 1], 0), (int)rows);
  return Rows{a, b > a ? b - a : 0u};
}

// Tile `rank` of all sequences' tiles of `bm` rows, the last first (of a
// causal sequence's queries those with the most keys).  False if there are
// fewer.  SKIP: without each sequence's first tile.  Every lane of the wave
// takes part and gets the same answer.
struct Tile {
  unsigned seq, row;            // sequence, its row at which the tile begins
  unsigned at;                  // number among all, the first tile 0
};
template <bool SKIP = false>
__device__ __forceinline__ bool find_tile(const int32_t* cu, unsigned seqs, unsigned rows, unsigned bm, unsigned rank,
                                          Tile* t) {
  const unsigned lane = lane_id();
  auto tiles_of = [&](unsigned s) {
    const unsigned n = s < seqs ? rows_of(cu, s, rows).count : 0;
    return SKIP ? (n ? (n - 1) / bm : 0) : (n + bm - 1) / bm;
  };
  unsigned total = 0;
  for (unsigned s0 = 0; s0 < seqs; s0 += kWave) total += __shfl(wave_scan(tiles_of(s0 + lane)), kWave - 1);
  if (rank >= total) return false;
  unsigned at = total - 1 - rank;
  t->at = at;
  for (unsigned s0 = 0; s0 < seqs; s0 += kWave) {
    const unsigned tiles = tiles_of(s0 + lane), upto = wave_scan(tiles), here = __shfl(upto, kWave - 1);
    if (at < here) {
      const uint64_t past = __ballot(upto > at);
      const int who = __builtin_ctzll(past);
      t->seq = s0 + who;
      t->row = (at - (__shfl(upto, who) - __shfl(tiles, who)) + (SKIP ? 1 : 0)) * bm;
      t->seq = __builtin_amdgcn_readfirstlane((int)t->seq);
      t->row = __builtin_amdgcn_readfirstlane((int)t->row);
      return true;
    }
    at -= here;
  }
  return false;
}

// First key in the window of the query at position p.
__device__ __forceinline__ int window_start(int p, unsigned window) {
  return p >= 0 && (unsigned)p >= window ? p - (int)window + 1 : 0;
}

// Where row r of a tile keeps its chunk of 16 bytes c: rows of DP bf16
// values, XORed so that neither the 16 rows read at one chunk (scores) nor
// the 8 rows read at four neighbouring chunks (transposing reads) meet in a
// bank.
template <int DP>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (DP == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
  else return ((r & 2) << 1) | ((r >> 2) & 3);
}
template <int DP>
__device__ __forceinline__ uint32_t chunk_addr(int r, int c) {
  return (uint32_t)(r * DP * 2 + ((c ^ swizzle<DP>(r)) * 16));
}

// The larger of a value and its counterpart 32 lanes away; the sum of both.
__device__ __forceinline__ float max_halves(float x) { return fmaxf(x, __shfl_xor(x, 32)); }
__device__ __forceinline__ float add_halves(float x) { return x + __shfl_xor(x, 32); }

}  // namespace ar
