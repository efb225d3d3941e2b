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

#include <utility>

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
#define AR_RARE(x) (__builtin_expect((x), 0))

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

// Neither infinite nor NaN; two bf16 values with 0 in the place of such.
__device__ __forceinline__ bool is_number(float x) { return __builtin_fabsf(x) < __builtin_huge_valf(); }
__device__ __forceinline__ uint32_t numbers_only(uint32_t w) {
  return w & ((w & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : ~0u) & ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFFu : ~0u);
}

// x, of which the compiler knows nothing: what rare code makes of it is not
// formed ahead of the branch to that code.
__device__ __forceinline__ int late(int x) {
  asm volatile("" : "+v"(x));
  return x;
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
// meets a barrier before the data are read.  The wait state covers the write
// of M0 before the copy reads it.
__device__ __forceinline__ void copy16_to_lds(const void* from, uint32_t lds) {
  lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(from) : "memory");
}

// The same from a base that the wave shares and an offset of the lane's own.
// (Five wait states lie before the copy: a vector instruction may have
// written the base's scalar registers right before.)
__device__ __forceinline__ void copy16_to_lds(const void* base, uint32_t off, uint32_t lds) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t at = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b) |
                      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)) << 32;
  lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" :: "s"(lds), "v"(off), "s"(at) : "memory");
}

// Until all copies are done.  (The builtin, which the compiler counts: it then
// waits no more for loads from before, and not for copies under way.)
__device__ __forceinline__ void wait_copies() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
  asm volatile("" ::: "memory");
}

// x / size of a page, x < 2^31.
__device__ __forceinline__ unsigned page_of(unsigned x, const Pages& c) {
  return c.shift == 32 ? x : __umulhi(x, c.magic) >> c.shift;
}

// A wave's inclusive sums over its lanes, which are all switched on: within
// rows of 16 by DPP shifts, then a row's last lane to the rows after it.
__device__ __forceinline__ unsigned wave_scan(unsigned v) {
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
  return v;
}
__device__ __forceinline__ unsigned last_lane(unsigned v) { return (unsigned)__builtin_amdgcn_readlane((int)v, kWave - 1); }

// Rows first .. first + count - 1 of sequence s out of the offsets cu.  Any
// contents of cu give rows below `rows`.
struct Rows {
  unsigned first, count;
};
__device__ __forceinline__ Rows rows_of(const int32_t* cu, unsigned s, unsigned rows) {
  const unsigned a = (unsigned)min(max(cu[s], 0), (int)rows), b = (unsigned)min(max(cu[s + 1], 0), (int)rows);
  return Rows{a, b > a ? b - a : 0u};
}

// The same for one sequence of the whole wave, in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ Rows rows_at(const int32_t* cu, unsigned s, unsigned rows) {
  const Rows r = rows_of(cu, s, rows);
  return Rows{(unsigned)uniform((int)r.first), (unsigned)uniform((int)r.count)};
}

// Tile `rank` of all sequences' tiles of `bm` rows, those with the most work of
// a causal sequence first: of queries the last (DOWN), of keys the first.
// False if there are fewer.  (Counts go through lane exchanges: with scalar
// ones, and so a scalar exit, the compiler spills 25 registers of k_attn.)  SKIP: without each sequence's first tile.  Every
// lane of the wave takes part and gets the same answer.
struct Tile {
  unsigned seq, row;            // sequence, its row at which the tile begins
  unsigned at;                  // number among all, the first tile 0
};
template <bool DOWN, bool SKIP = false>
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
  unsigned at = DOWN ? total - 1 - rank : rank;
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

// The keys that a tile of queries at positions p0 .. p1 looks at: sinks
// 0 .. sinks - 1, all visible up to a query's own position, then lo .. end - 1,
// of which it sees those from its window's start on.  In steps of `step`.
struct KeyRange {
  int sinks, lo, end, sink_steps, steps;
};
__device__ __forceinline__ KeyRange key_range(int p0, int p1, unsigned window, unsigned sinks, int step) {
  KeyRange r;
  r.end = p1 + 1;
  r.sinks = window_start(p1, window) > 0 ? min((int)sinks, r.end) : 0;
  r.lo = max(window_start(p0, window), r.sinks);
  r.sink_steps = (r.sinks + step - 1) / step;
  r.steps = r.end <= 0 ? 0 : r.sink_steps + (max(r.end - r.lo, 0) + step - 1) / step;
  return r;
}
// Step n: its first key, the end of its part.
struct KeyStep {
  int j0, end;
  bool sinks;
};
__device__ __forceinline__ KeyStep key_step(const KeyRange& r, int n, int step) {
  const bool s = n < r.sink_steps;
  return KeyStep{s ? n * step : r.lo + (n - r.sink_steps) * step, s ? r.sinks : r.end, s};
}

// Whole numbers lo .. hi, asked for by one comparison.
struct Interval {
  int lo;
  unsigned width;
  __device__ __forceinline__ Interval(int lo_, int hi) : lo(lo_), width(hi >= lo_ ? (unsigned)hi - (unsigned)lo_ + 1u : 0u) {}
  __device__ __forceinline__ bool has(int x) const { return (unsigned)(x - lo) < width; }
};

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

// Where a lane reads its operands in a tile of DP-wide rows (byte addresses in
// LDS): 16 bytes of row `lane % 32` for one operand of 32 rows, and for a
// transposed one 8 bytes of two rows eight apart.  Chunk 2 x of the row, or
// columns 32 d, are one XOR away, and 32 rows further an offset.  An address
// is kept from being one of many that the compiler would form before the loop
// and hold in registers.
template <int DP>
struct LaneAddr {
  uint32_t row, tr0, tr1;
  __device__ __forceinline__ LaneAddr(uint32_t tile, int lane) {
    const int hh = lane >> 5, va = 4 * hh + (lane & 15) / 4, vch = 2 * ((lane >> 4) & 1) + (lane & 3) / 2;
    row = tile + chunk_addr<DP>(lane & 31, hh);
    tr0 = tile + chunk_addr<DP>(va, vch) + (lane & 1) * 8;
    tr1 = tile + chunk_addr<DP>(va + 8, vch) + (lane & 1) * 8;
    asm volatile("" : "+v"(row), "+v"(tr0), "+v"(tr1));
  }
  __device__ __forceinline__ LaneAddr(const LaneAddr& o, uint32_t by) : row(o.row + by), tr0(o.tr0 + by), tr1(o.tr1 + by) {
    asm volatile("" : "+v"(row), "+v"(tr0), "+v"(tr1));
  }
  // 16 bytes of row r0 + lane % 32, chunk 2 x + lane / 32
  __device__ __forceinline__ u32x4 rows(int r0, int x) const {
    const uint32_t a = (row ^ (uint32_t)(x * 32)) + (uint32_t)(r0 * DP * 2);
    return *(__attribute__((address_space(3))) const u32x4*)(uintptr_t)a;
  }
  // 8 values of column 32 d + lane % 32, of the 16 rows from r0 on
  __device__ __forceinline__ Frag8 columns(int r0, int d) const {
    Frag8 v;
    v.s[0] = read_tr16((tr0 ^ (uint32_t)(d * 64)) + (uint32_t)(r0 * DP * 2));
    v.s[1] = read_tr16((tr1 ^ (uint32_t)(d * 64)) + (uint32_t)(r0 * DP * 2));
    return v;
  }
};

// f(0) ... f(N - 1), each index a compile-time constant.
template <typename F, int... I>
__device__ __forceinline__ void steps_of(F& f, std::integer_sequence<int, I...>) {
  (f(SPc<I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void steps(F&& f) {
  steps_of(f, std::make_integer_sequence<int, N>{});
}
// Instructions stay on their side of it: operands are read as far ahead as
// written, no further.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// Copies tiles of 64 rows of two matrices (x, then y behind it) to LDS; NW
// waves share the work, 1 KiB of each a wave at a time.
template <int DP, int NW>
struct TileCopy {
  static constexpr int kRows = 64, RPC = 1024 / (DP * 2), CPR = DP / 8, COPIES = kRows / RPC / NW;
  static constexpr uint32_t kTile = kRows * DP * 2;
  static_assert(NW % (DP == 128 ? 4 : 2) == 0, "a lane's chunk is the same in every copy");
  int row, wave;                // of the lane's first copy
  uint32_t x_off, y_off, chunk; // bytes
  bool on, near;                // the chunk exists; offsets within a tile fit 32 bits
  __device__ __forceinline__ TileCopy(size_t xs, size_t ys, unsigned dim, int wave_, int lane) : wave(wave_) {
    row = wave * RPC + lane / CPR;
    chunk = (uint32_t)((lane % CPR) ^ swizzle<DP>(row)) * 16;
    on = chunk < dim * 2;
    near = ((xs | ys) >> 24) == 0;
    x_off = (uint32_t)(row * xs * 2) + chunk;
    y_off = (uint32_t)(row * ys * 2) + chunk;
  }
  // Rows first .. first + 63 of x and y; rows past `last` are copies of it.
  __device__ __forceinline__ void operator()(const uint16_t* x, size_t xs, const uint16_t* y, size_t ys, int first, int last,
                                             uint32_t lds) const {
    if (!on) return;
    const uint32_t to = lds + (uint32_t)wave * 1024;
    if (first + kRows - 1 <= last && near) {
      const char* xb = reinterpret_cast<const char*>(x + (size_t)first * xs);
      const char* yb = reinterpret_cast<const char*>(y + (size_t)first * ys);
#pragma unroll
      for (int i = 0; i < COPIES; ++i) {
        copy16_to_lds(xb + (size_t)i * NW * RPC * xs * 2, x_off, to + i * NW * 1024);
        copy16_to_lds(yb + (size_t)i * NW * RPC * ys * 2, y_off, to + i * NW * 1024 + kTile);
      }
      return;
    }
#pragma unroll 1
    for (int i = 0; i < COPIES; ++i) {
      const int j = min(first + i * NW * RPC + row, last);
      copy16_to_lds(reinterpret_cast<const char*>(x + (size_t)j * xs) + chunk, to + i * NW * 1024);
      copy16_to_lds(reinterpret_cast<const char*>(y + (size_t)j * ys) + chunk, to + i * NW * 1024 + kTile);
    }
  }
};

// The larger of a value and its counterpart 32 (16) lanes away, and the sum of
// both, by the instructions that swap halves (rows of 16) of two registers.
__device__ __forceinline__ u32x2 swap32(float x) {
  return __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
}
__device__ __forceinline__ u32x2 swap16(float x) {
  return __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
}
__device__ __forceinline__ float max_of(u32x2 p) { return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])); }
__device__ __forceinline__ float sum_of(u32x2 p) { return __uint_as_float(p[0]) + __uint_as_float(p[1]); }

}  // namespace ar
