// Attention of one new token a sequence over a paged cache.
//
// Bound by memory: a key and its value are read once for all query heads that
// share them.  A workgroup takes a tile of keys of one key head at a time, each
// of its eight waves a step of 16 or 32 keys; scores S^T = K Q^T and results
// O^T = V^T P^T are 16 x 16 products whose columns are the (up to 16) query
// heads of the key head.
//
// The keys of all sequences and key heads are one long row of tiles, which
// is cut into equal runs, one a workgroup, whatever the lengths are.  A
// sequence that is cut is joined by the last workgroup that arrives with a
// part, which adds all parts in their order, so that the result does not
// depend on which one was last.
//
// Keys and values are copied to LDS past the registers, two steps of a wave
// ahead: for heads of 128, 128 KiB a CU are on their way, which is what its share
// of the memory's rate takes over the memory's latency.  The page numbers of a
// step come the same way, two steps before its keys.
//
// 48 sequences of 111 to 16384 keys, 8 key heads of 128 in bf16: 122 us, 5.3
// TB/s; 8 of 120k to 131k in E4M3 382 us, 5.5.  Kept for what they gave there:
// eight waves instead of four (171 -> 156 and 750 -> 497 us), one loop a
// sequence (142 -> 134, 475 -> 458), copies past the caches (134 -> 122, 458
// -> 402), ends of sequences counted in the spread (156 -> 142).
//
// Narrower heads: a step holds rows of 64 or 128 whatever the head, so that of 80,
// 96 and 112 only 63 to 88% of those bytes are on their way (64 KiB in E4M3 of
// 64).  The same 48 sequences: of 64 in bf16 78 us, 4.2 TB/s (8 of 120k to 131k
// keys: 5.3), 80 95 us, 4.3, 96 105 us, 4.7, 112 134 us, 4.25; in E4M3 72, 94, 95,
// 98 us, 2.3 to 3.0 TB/s, and of 128 85 us, 4.0.  With a window of 4096 and 4
// sinks, which are a tile of their own, 79 us of 128 in bf16, 4.8 TB/s, 61 in
// E4M3, 3.2; with a window of 512 30, 2.9.
#include "ar_attn.hpp"

namespace ar {
namespace {

constexpr int kWaves = 8;
constexpr unsigned kWorkers = 256;             // one a CU of a whole device: the LDS of a workgroup fills it
constexpr unsigned kHeads = 16;                // query heads of a tile

// What a wave has in LDS: two steps' keys and values, four steps' page numbers.
template <int DP, bool E4M3>
struct Ring {
  static constexpr int kRow = E4M3 ? DP : DP * 2;              // bytes
  static constexpr int kStep = kRow == 256 ? 16 : 32;          // keys of a wave's step: two steps of eight waves fit LDS
  static constexpr int kTileKeys = kWaves * kStep;
  static constexpr int kKeys = kStep * kRow;                   // bytes of a step's keys, or values
  static constexpr int kScales = E4M3 ? 2 * kStep * 4 : 0;     // of the keys, then of the values
  static constexpr int kStage = 2 * kKeys + kScales;
  static constexpr int kIds = 4 * kWave * 4;                   // page numbers of four steps
  static constexpr int kBytes = 2 * kStage + kIds;
  static constexpr int kCopies = kKeys / 1024 * 2 + (E4M3 ? 1 : 0) + 1;  // instructions of a step
};

template <int RB>
__device__ __forceinline__ int swizzle_bytes(int r) {
  if constexpr (RB == 256) return swizzle<128>(r);
  else if constexpr (RB == 128) return swizzle<64>(r);
  else return (r >> 2) & 3;
}
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * RB + ((c ^ swizzle_bytes<RB>(r)) * 16)); }

// As copy16_to_lds, with the hint that the data are not read again.
__device__ __forceinline__ void stream16_to_lds(const void* from, uint32_t lds) {
  lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" :: "s"(lds), "v"(from) : "memory");
}

__device__ __forceinline__ void copy4_to_lds(const void* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" :: "s"(lds), "v"(from) : "memory");
}

// What a sequence costs beside its tiles, in tiles: the join of its waves and
// the start of the next.  (48 sequences of 100 to 16384 keys: 142 us, without
// it 156.)
constexpr unsigned kEnd = 2;

// What a sequence's keys are cut into.
struct Cut {
  int len, lo, sunk;            // keys; the window's first; sinks before it
  int ts, n;                    // tiles of sinks, of all (at least 1)
};
template <int kTileKeys>
__device__ __forceinline__ Cut cut_of(const AttnArgs& a, int len) {
  Cut c;
  c.len = (int)min((unsigned)max(len, 0), a.capacity);
  c.lo = window_start(c.len - 1, a.window);
  c.sunk = min((int)a.sinks, c.lo);
  c.ts = (c.sunk + kTileKeys - 1) / kTileKeys;
  c.n = max(c.ts + (c.len - c.lo + kTileKeys - 1) / kTileKeys, 1);
  return c;
}

// A sequence's tiles in a workgroup's run.
struct Part {
  int seq, hx;                  // sequence; key head and its tile of query heads
  unsigned seq_u, into, count;  // where the sequence begins in the row of all; first tile, number of tiles
  Cut cut;
};

template <int DP, bool E4M3>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attn_decode(AttnArgs a, unsigned head_tiles, uint32_t* counters, float* parts,
                                                                bool split) {
  using R = Ring<DP, E4M3>;
  constexpr int RB = R::kRow, KS = DP / 32, DT = DP / 16, STEP = R::kStep, TILE = R::kTileKeys, NB = STEP / 16;
  __shared__ __align__(1024) char ring[kWaves * R::kBytes];
  __shared__ __align__(16) float lo_[kWaves][kHeads][36];      // 32 columns of each wave's result
  __shared__ float lm[kWaves][kHeads], ll[kWaves][kHeads];
  __shared__ unsigned lcount;
  const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int hd = lane & 15, g = lane >> 4;
  const unsigned group = a.hq / a.hkv;

  // This workgroup's run of the row of all tiles, each sequence's followed by
  // kEnd empty ones; or (split false) one sequence's.
  auto tiles_of = [&](unsigned s, int& len) {
    if (s >= a.seqs) return 0u;
    len = a.lens[s];
    return (unsigned)cut_of<TILE>(a, len).n + kEnd;
  };
  int len = 0;
  unsigned u = 0, u_end, per = 0;              // tiles of a run
  int hx, seq;
  unsigned into = 0;                           // tile of the sequence
  if (split) {
    unsigned N = 0;
    for (unsigned s0 = 0; s0 < a.seqs; s0 += kWave) N += last_lane(wave_scan(tiles_of(s0 + lane, len)));
    // Runs of whole key heads where that leaves few workgroups idle: the heads
    // of a token, which lie side by side in memory, are then read at one time.
    const unsigned heads = a.hkv * head_tiles, each = kWorkers / heads;
    const bool aligned = each * heads * 10 >= kWorkers * 9;
    per = aligned ? (N + each - 1) / each : (N * heads + kWorkers - 1) / kWorkers;
    const unsigned wide = aligned ? per * each : N;   // a head's share of the row
    u = blockIdx.x * per;
    hx = (int)(u / wide);
    unsigned at = u % wide;
    if (hx >= (int)heads || at >= N) return;
    u_end = min(u + per, aligned ? hx * wide + N : N * heads);
    seq = 0;
    for (unsigned s0 = 0; s0 < a.seqs; s0 += kWave) {
      const unsigned n = tiles_of(s0 + lane, len), upto = wave_scan(n), here = last_lane(upto);
      if (at < here) {
        const int who = __builtin_ctzll(__ballot(upto > at));
        seq = (int)s0 + who;
        into = at - (unsigned)(__builtin_amdgcn_readlane((int)upto, who) - __builtin_amdgcn_readlane((int)n, who));
        len = __builtin_amdgcn_readlane(len, who);
        break;
      }
      at -= here;
    }
    seq = uniform(seq);
    into = (unsigned)uniform((int)into);
    len = uniform(len);
  } else {
    seq = (int)(blockIdx.x % a.seqs);
    hx = (int)(blockIdx.x / a.seqs);
    u_end = (unsigned)uniform((int)tiles_of((unsigned)seq, len)) - kEnd;
    len = uniform(len);
  }

  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  const Scalar lens = (Scalar)(uintptr_t)a.lens;
  Part now{seq, hx, u - into, into, 0, cut_of<TILE>(a, len)};
  // The run's next sequence; false at the run's end.
  auto follow = [&](Part& p) {
    const unsigned at = p.seq_u + (unsigned)p.cut.n + kEnd;
    if (at >= u_end) return false;
    if (++p.seq >= (int)a.seqs) {
      p.seq = 0;
      ++p.hx;
    }
    p.cut = cut_of<TILE>(a, lens[p.seq]);
    p.seq_u = at;
    p.into = 0;
    p.count = min((unsigned)p.cut.n, u_end - at);
    return true;
  };
  if ((int)into < now.cut.n) now.count = min((unsigned)now.cut.n - into, u_end - u);
  else if (!follow(now)) return;

  char* mine = ring + wave * R::kBytes;
  const uint32_t lmine = (uint32_t)uniform((int)lds_addr(mine));
  const uint32_t lids = lmine + 2 * R::kStage;
  const uint32_t* ids = reinterpret_cast<const uint32_t*>(mine + 2 * R::kStage);
  if (a.dim < DP) {                            // places that no copy fills
    for (int o = lane * 16; o < 2 * R::kStage; o += kWave * 16) *reinterpret_cast<u32x4*>(mine + o) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }

  // first key of a part's tile i, end of its keys
  struct Keys {
    int j0, end;
  };
  auto keys_of = [&](const Part& p, unsigned i) {
    const int n = (int)(p.into + i), ts = p.cut.ts;
    return n < ts ? Keys{n * TILE, p.cut.sunk} : Keys{p.cut.lo + (n - ts) * TILE, p.cut.len};
  };
  // key of the wave's row r, held within the tile's keys
  auto key_of = [&](Keys k, int r) { return (unsigned)max(min(k.j0 + wave * STEP + r, k.end - 1), 0); };
  auto fetch_ids = [&](const Part& p, unsigned i, int slot) {
    const unsigned pg = page_of(key_of(keys_of(p, i), lane & (STEP - 1)), a.cache);
    copy4_to_lds(a.table + (size_t)p.seq * a.table_ld + pg, lids + slot * kWave * 4);
  };
  constexpr int RPC = 1024 / RB, CPR = RB / 16, ES = E4M3 ? 1 : 2, COPIES = STEP / RPC;
  const int crow = lane / CPR;
  const uint32_t chunk = (uint32_t)((lane % CPR) ^ swizzle_bytes<RB>(crow)) * 16;
  // (a page number out of range is found again when the step is computed)
  const unsigned top_page = a.cache.pages - 1;
  // Where the step that is fetched next lies: its rows' chunks, and (E4M3) the
  // lane's scale.
  size_t from[COPIES], from_scale = 0;
  auto locate = [&](const Part& p, unsigned i, int slot) {
    uint32_t id[COPIES], id_scale = 0;
#pragma unroll
    for (int x = 0; x < COPIES; ++x) id[x] = ids[slot * kWave + x * RPC + crow];
    if constexpr (E4M3) id_scale = ids[slot * kWave + (lane & 31)];
    const Keys keys = keys_of(p, i);
    const unsigned kvh = (unsigned)p.hx / head_tiles;
#pragma unroll
    for (int x = 0; x < COPIES; ++x) {
      // the chunk of row crow is that of row x RPC + crow but for the rows' swizzle
      const uint32_t ch = chunk ^ (uint32_t)((swizzle_bytes<RB>(x * RPC + crow) ^ swizzle_bytes<RB>(crow)) * 16);
      const unsigned j = key_of(keys, x * RPC + crow), in = j - page_of(j, a.cache) * a.cache.size;
      from[x] = ((size_t)min(id[x], top_page) * a.cache.page + (size_t)in * a.cache.ts + kvh * a.cache.hs) * ES + ch;
    }
    if constexpr (E4M3) {
      const unsigned j = key_of(keys, lane & 31), in = j - page_of(j, a.cache) * a.cache.size;
      from_scale = (size_t)min(id_scale, top_page) * a.cache.spage + (size_t)in * a.cache.sts + kvh * a.cache.shs;
    }
  };
  // Starts tile i's copies, and those of the page numbers of tile i + 2.
  auto fetch = [&](const Part& p, unsigned i, int stage, int slot) {
    const uint32_t to = lmine + stage * R::kStage;
    const char *kb = static_cast<const char*>(a.cache.k), *vb = static_cast<const char*>(a.cache.v);
#pragma unroll
    for (int x = 0; x < COPIES; ++x) {
      const uint32_t ch = chunk ^ (uint32_t)((swizzle_bytes<RB>(x * RPC + crow) ^ swizzle_bytes<RB>(crow)) * 16);
      if (ch < a.dim * ES) {
        stream16_to_lds(kb + from[x], to + x * 1024);
        stream16_to_lds(vb + from[x], to + R::kKeys + x * 1024);
      }
    }
    if constexpr (E4M3)
      copy4_to_lds((lane < 32 ? a.cache.k_scales : a.cache.v_scales) + from_scale, to + 2 * R::kKeys);
    fetch_ids(p, min(i + 2, p.count - 1), (slot + 2) & 3);
  };
  // Starts a part's first two tiles: slots 0 and 1, stages 0 and 1.
  auto start = [&](const Part& p) {
    fetch_ids(p, 0, 0);
    fetch_ids(p, min(1u, p.count - 1), 1);
    wait_copies();
#pragma unroll 1
    for (unsigned x = 0; x < min(2u, p.count); ++x) {
      locate(p, x, (int)x);
      fetch(p, x, (int)x, (int)x);
    }
  };

  Frag8 q[KS];
  f32x4 o[DT];
  float m = AR_NEG_INF, l = 0.f;
  const float c = a.scale * kLog2e;
  // (columns past the last head are those of the last; their results are not kept)
  auto load_queries = [&](const Part& p) {
    const unsigned kvh = (unsigned)p.hx / head_tiles, ht = (unsigned)p.hx % head_tiles;
    const unsigned here = min(group - ht * kHeads, kHeads), h = kvh * group + ht * kHeads + min((unsigned)hd, here - 1);
    const uint16_t* qp = a.q.p + (size_t)p.seq * a.q.ts + h * a.q.hs;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const unsigned d = E4M3 ? 64 * (x / 2) + 16 * g + 8 * (x & 1) : 32 * x + 8 * g;
      q[x].u = d < a.dim ? *reinterpret_cast<const u32x4*>(qp + d) : u32x4{0, 0, 0, 0};
    }
  };
  // A part's copies are under way while the one before it is joined.
  Part s0 = now;                               // the part that is computed, or joined
  bool more = true, done = false;
  // Infinite values: 0 times one is NaN, and half of the numerators' rests
  // have the other sign.  So where a result is no number, the wave computes
  // its part again with care: values that are no numbers are 0 in the product
  // and summed apart, a column a lane, for all heads.  (The wave alone: no
  // barrier lies between a part's start and its join.)  So too where a sum is
  // 2^115 or more, of which the 2^11 that are joined could pass binary32's
  // end though their mean does not: with care the maximum is followed 2^lift
  // above, and numerators are at most 2^-2 of one over the keys.  (Code of its
  // own: as branches of one loop it cost heads of 64 in bf16 a tenth.)
  bool care = false;
  float odd[DP / 64];                          // columns lane, lane + 64
  for (;;) {
    if (more) {
      load_queries(now);
      start(now);
    }
    if (done) {
      const unsigned kvh = (unsigned)s0.hx / head_tiles, ht = (unsigned)s0.hx % head_tiles;
      const unsigned here = min(group - ht * kHeads, kHeads), head0 = kvh * group + ht * kHeads;
      // the waves' results are one
      l = sum_of(swap32(sum_of(swap16(l))));
      if (lane < 16) {
        lm[wave][hd] = m;
        ll[wave][hd] = l;
      }
      __syncthreads();
      float M = AR_NEG_INF, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lm[w][hd]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        sum += lm[w][hd] == AR_NEG_INF ? ll[w][hd] : ll[w][hd] * exp2_fast(lm[w][hd] - M);
      float f = m == AR_NEG_INF ? 0.f : exp2_fast(m - M);
      if (AR_RARE(care)) {                       // (no weight makes such values 0 any more)
        const int g = late(lane) >> 4;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[d][r] = o[d][r] * f + __shfl(odd[d / 4], (16 * d + 4 * g + r) & 63);
        f = 1.0f;
        care = false;
      }
      const unsigned begin = split ? s0.seq_u / per : 0, finish = split ? (s0.seq_u + (unsigned)s0.cut.n - 1) / per : 0;
      const unsigned count = finish - begin + 1;   // runs that hold parts of the sequence
      const float inv = sum > 0.f ? 1.0f / sum : sum;   // no key: zeros; NaN stays
      // results of a part: 16 maxima, 16 sums, then rows of a head's columns
      constexpr unsigned kPart = 2 * kHeads + kHeads * DP;
      float* part = count > 1 ? parts + (size_t)(blockIdx.x * 2 + (blockIdx.x == begin ? 1 : 0)) * kPart : nullptr;
      const unsigned oh = t / 32, od = t % 32;     // this lane's head and column of 32
      const float oinv = __shfl(inv, (int)oh);
#pragma unroll
      for (int d2 = 0; d2 < DT / 2; ++d2) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          f32x4 v = o[2 * d2 + x];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] *= f;
          *reinterpret_cast<f32x4*>(&lo_[wave][hd][16 * x + 4 * g]) = v;
        }
        __syncthreads();
        float sum2 = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum2 += lo_[w][oh][od];
        const unsigned at = 32 * d2 + od;
        if (oh < here && at < a.dim) {
          if (part) __hip_atomic_store(part + 2 * kHeads + oh * DP + at, sum2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          else a.out.p[(size_t)s0.seq * a.out.ts + (head0 + oh) * a.out.hs + at] = to_bf16(sum2 * oinv);
        }
        __syncthreads();
      }
      if (part) {
        if (t < (int)kHeads) {
          __hip_atomic_store(part + t, M, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(part + kHeads + t, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        wait_copies();                         // the part is out
        __syncthreads();
        uint32_t* counter = counters + (size_t)s0.hx * a.seqs + s0.seq;
        if (t == 0) lcount = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (lcount == count - 1) {
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
          if (t == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          // 32 lanes a head; 4 columns each
          auto part_of = [&](unsigned i) { return parts + (size_t)((begin + i) * 2 + (i == 0 ? 1 : 0)) * kPart; };
          const unsigned h = oh, lane32 = t % 32, d = lane32 * 4;
          if (h < here) {
            const unsigned col = h * DP + min(d, (unsigned)DP - 4);
            f32x4 v[8];
            // eight parts at a time are on their way at once
            auto load_parts = [&](unsigned i0) {
#pragma unroll
              for (unsigned i = 0; i < 8; ++i)
                v[i] = *reinterpret_cast<const f32x4*>(part_of(min(i0 + i, count - 1)) + 2 * kHeads + col);
            };
            // lane i's part: its maximum, its sum
            float pm = AR_NEG_INF, pl = 0.f;
            auto load_sums = [&](unsigned i) {
              pm = i < count ? part_of(i)[h] : AR_NEG_INF;
              pl = i < count ? part_of(i)[kHeads + h] : 0.f;
            };
            load_sums(lane32);
            load_parts(0);
            float M2 = pm, L2 = 0.f;
            for (unsigned i = 32 + lane32; i < count; i += 32) M2 = fmaxf(M2, part_of(i)[h]);
#pragma unroll
            for (int x = 1; x < 32; x *= 2) M2 = fmaxf(M2, __shfl_xor(M2, x));
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            for (unsigned i0 = 0; i0 < count; i0 += 32) {
              if (i0) load_sums(i0 + lane32);
              const float w = pm == AR_NEG_INF ? 0.f : exp2_fast(pm - M2), s = pm == AR_NEG_INF ? pl : pl * w;
              for (unsigned i1 = 0; i1 < min(32u, count - i0); i1 += 8) {
                if (i0 + i1) load_parts(i0 + i1);
#pragma unroll
                for (unsigned i = 0; i < 8; ++i) {
                  const int from = (int)((lane & 32) + i1 + i);
                  const float wi = __shfl(w, from);
                  L2 += __shfl(s, from);
                  if (i0 + i1 + i < count) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(v[i][r], wi, acc[r]);
                  }
                }
              }
            }
            if (AR_RARE(!is_number((acc[0] + acc[1]) + (acc[2] + acc[3])))) {
              // (a part's infinity has met a weight of 0)
              acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
              for (unsigned i = 0; i < count; ++i) {
                const float* from = part_of(i);
                const f32x4 x = *reinterpret_cast<const f32x4*>(from + 2 * kHeads + col);
                const float w = from[h] == AR_NEG_INF ? 0.f : exp2_fast(from[h] - M2);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] += is_number(x[r]) ? x[r] * w : x[r];
              }
            }
            const float i2 = L2 > 0.f ? 1.0f / L2 : L2;
            if (d < a.dim)
              *reinterpret_cast<u32x2*>(a.out.p + (size_t)s0.seq * a.out.ts + (head0 + h) * a.out.hs + d) =
                  u32x2{result_bf16x2(acc[0] * i2, acc[1] * i2), result_bf16x2(acc[2] * i2, acc[3] * i2)};
            if (a.lse && lane32 == 0)
              a.lse[(size_t)s0.seq * a.lse_ts + (head0 + h) * a.lse_hs] =
                  L2 > 0.f ? (M2 + __builtin_amdgcn_logf(L2)) * kLn2 : L2 == 0.f ? AR_NEG_INF : L2;
          }
        }
        __syncthreads();
      } else if (a.lse && t < (int)here) {
        a.lse[(size_t)s0.seq * a.lse_ts + (head0 + t) * a.lse_hs] =
            sum > 0.f ? (M + __builtin_amdgcn_logf(sum)) * kLn2 : sum == 0.f ? AR_NEG_INF : sum;
      }
    }
    if (!more) break;
    auto compute = [&](auto careful) __attribute__((always_inline)) {
      constexpr bool CARE = decltype(careful)::value;
      m = AR_NEG_INF;
      l = 0.f;
      const float lift = CARE ? (float)(10 + 31 - __builtin_clz(now.cut.len | 1)) : 0.f;   // 2^lift > 2^10 times the keys / 2
#pragma unroll
      for (int x = 0; x < DP / 64; ++x) odd[x] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (unsigned i = 0; i < now.count; ++i) {
        const int stage = i & 1, slot = i & 3;
        // the tile's copies are done when only the next one's are left
        if (i + 1 < now.count) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(R::kCopies) : "memory");
        else wait_copies();
        if (i + 2 < now.count) locate(now, i + 2, (slot + 2) & 3);
        const Keys tile = keys_of(now, i);
        const int keys = min(tile.end - tile.j0 - wave * STEP, STEP);   // of this wave's step
        if (keys > 0) {
          if (__any((lane & (STEP - 1)) < keys && ids[slot * kWave + (lane & (STEP - 1))] >= a.cache.pages))
            l = __uint_as_float(0x7FC00000u);
          const char* lk = mine + stage * R::kStage;
          const uint32_t lv = lmine + stage * R::kStage + R::kKeys;
          if constexpr (CARE) {
            const int lane = late(lane_id());
            char* tv = mine + stage * R::kStage + R::kKeys;
#pragma unroll 1
            for (int r = 0; r < keys; ++r) {
#pragma unroll
              for (int x = 0; x < DP / 64; ++x) {
                const char* p = tv + chunk_at<RB>(r, lane * ES / 16 + x * 4 * ES) + lane * ES % 16;
                const float v = E4M3 ? ((*p & 0x7F) == 0x7F ? __uint_as_float(0x7FC00000u) : 0.f)
                                     : bf16_f32(*reinterpret_cast<const uint16_t*>(p));
                if (!is_number(v)) odd[x] += v;
              }
            }
#pragma unroll 1
            for (int at = lane * 4; at < R::kKeys; at += kWave * 4) {
              uint32_t& w = *reinterpret_cast<uint32_t*>(tv + at);
              if constexpr (E4M3) w &= ~((((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xFFu);
              else w = numbers_only(w);
            }
          }
          // values are read first: they arrive while the scores are formed
          Frag8 v[DT];
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            if constexpr (E4M3) {
              const int e = (lane & 15) / 2, r = 4 * g + (e & 3) + (e >= 4 ? 16 : 0);
              const i32x2 w = read_tr8(lv + chunk_at<RB>(r, d) + (lane & 1) * 8);
              v[d].w[0] = (uint32_t)w[0];
              v[d].w[1] = (uint32_t)w[1];
            } else {
              const int r = 4 * g + (lane & 15) / 4, ch = 2 * d + (lane & 3) / 2;
#pragma unroll
              for (int b = 0; b < NB; ++b) v[d].s[b] = read_tr16(lv + chunk_at<RB>(r + 16 * b, ch) + (lane & 1) * 8);
            }
          }
          f32x4 scale_k[NB], scale_v[NB];
          if constexpr (E4M3) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              scale_k[b] = *reinterpret_cast<const f32x4*>(lk + 2 * R::kKeys + (16 * b + 4 * g) * 4);
              scale_v[b] = *reinterpret_cast<const f32x4*>(lk + 2 * R::kKeys + (STEP + 16 * b + 4 * g) * 4);
            }
          }
          f32x4 s[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            s[b] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (E4M3) {
#pragma unroll
              for (int x = 0; x < KS / 2; ++x) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(lk + chunk_at<RB>(16 * b + hd, 4 * x + g));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  Frag8 k;
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    union { b16x2 b; uint32_t u; } lo, hi;
                    lo.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * y + e], 1.0f, false);
                    hi.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * y + e], 1.0f, true);
                    k.w[2 * e] = lo.u;
                    k.w[2 * e + 1] = hi.u;
                  }
                  s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k.b, q[2 * x + y].b, s[b], 0, 0, 0);
                }
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) s[b][r] *= scale_k[b][r];
            } else {
#pragma unroll
              for (int x = 0; x < KS; ++x) {
                Frag8 k;
                k.u = *reinterpret_cast<const u32x4*>(lk + chunk_at<RB>(16 * b + hd, 4 * x + g));
                s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k.b, q[x].b, s[b], 0, 0, 0);
              }
            }
          }
          // register r of block b is key 16 b + 4 g + r of the step
          if (keys < STEP) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int r = 0; r < 4; ++r) s[b][r] = 16 * b + 4 * g + r < keys ? s[b][r] : AR_NEG_INF;
          }
          float top = AR_NEG_INF;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, s[b][r]);
          top = max_of(swap32(max_of(swap16(top)))) * c;
          if constexpr (CARE) top += lift;
          if (__any(top > m + 8.0f)) {
            const float up = fmaxf(m, top), f = m == AR_NEG_INF ? 1.0f : exp2_fast(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f;
          }
          const float base = m == AR_NEG_INF ? 0.f : m;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              s[b][r] = exp2_fast(__builtin_fmaf(s[b][r], c, -base));
              l += s[b][r];
            }
          if constexpr (E4M3) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
              for (int r = 0; r < 4; ++r) s[b][r] *= scale_v[b][r];
              if (keys < STEP) {                   // (a masked place's scale may be no number)
#pragma unroll
                for (int r = 0; r < 4; ++r) s[b][r] = 16 * b + 4 * g + r < keys ? s[b][r] : 0.f;
              }
            }
          }
          // as two bf16 numbers each, 2^-17 off: the matrix cores have the time
          Frag8 p, rest;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
              const uint32_t w = cvt_bf16x2(s[b][r], s[b][r + 1]);
              p.w[2 * b + r / 2] = w;
              rest.w[2 * b + r / 2] = cvt_bf16x2(s[b][r] - lo_f32(w), s[b][r + 1] - hi_f32(w));
            }
          // whether element e of the lane's values is of a key of the step: 0
          // times what a masked place holds must be 0
          const int beyond = keys - 4 * g;         // of keys 4 g + ...; 16 less for the second four
          if constexpr (E4M3) {
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const i32x2 w = {(int)v[d].w[0], (int)v[d].w[1]};
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                union { b16x2 b; uint32_t u; } lo, hi;
                lo.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[x], 1.0f, false);
                hi.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[x], 1.0f, true);
                v[d].w[2 * x] = lo.u;
                v[d].w[2 * x + 1] = hi.u;
              }
            }
          }
          if (keys < STEP) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int e = 0; e < 4 * NB; ++e)
                if ((e & 3) + (e >= 4 ? 16 : 0) >= beyond) v[d].w[e / 2] &= e & 1 ? 0xFFFFu : 0xFFFF0000u;
          }
          if constexpr (E4M3 && CARE) {            // (an infinite scale's numerator has no rest)
#pragma unroll
            for (int w = 0; w < 2 * NB; ++w) rest.w[w] = numbers_only(rest.w[w]);
          }
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            if constexpr (NB == 2) {
              o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[d].b, p.b, o[d], 0, 0, 0);
              o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[d].b, rest.b, o[d], 0, 0, 0);
            } else {
              // both in one: the second four of a lane's keys are the first again
              Frag8 twice;
              twice.s[0] = twice.s[1] = v[d].s[0];
              Frag8 both;
              both.s[0] = p.s[0];
              both.s[1] = rest.s[0];
              o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(twice.b, both.b, o[d], 0, 0, 0);
            }
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage has been read
        if (i + 2 < now.count) fetch(now, i + 2, stage, (slot + 2) & 3);
      }

    };
    compute(std::false_type{});
    f32x4 all = {0.f, 0.f, 0.f, 0.f};          // numbers only if every result is, and below 2^115
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) all[r] = __builtin_fmaf(o[d][r], 0x1p13f, all[r]);
    if (AR_RARE(__any(!is_number((all[0] + all[1]) + (all[2] + all[3]))))) {
      care = true;
      start(now);
      compute(std::true_type{});
    }
    s0 = now;
    done = true;
    more = follow(now);
  }
}

unsigned head_tiles_of(size_t hq, size_t hkv) { return (unsigned)cdiv(hq / hkv, kHeads); }
// The parts come first, with room for the widest heads, so that the counters
// lie in one place for every shape.
constexpr size_t kPartsBytes = (size_t)kWorkers * 2 * (2 * kHeads + kHeads * AR_ATTN_MAX_DIM) * 4;
size_t counters_bytes(size_t seqs, size_t hq, size_t hkv) { return cdiv(seqs * hkv * head_tiles_of(hq, hkv) * 4, 256) * 256; }

template <int DP, bool E4M3>
hipError_t launch(const Launch& L, const AttnArgs& a, void* ws) {
  const unsigned ht = head_tiles_of(a.hq, a.hkv);
  float* parts = static_cast<float*>(ws);
  uint32_t* counters = ws ? reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kPartsBytes) : nullptr;
  const unsigned grid = ws ? kWorkers : a.seqs * a.hkv * ht;
  return launch_k(k_attn_decode<DP, E4M3>, dim3(grid), dim3(kWaves * 64), 0, L.stream, a, ht, counters, parts, ws != nullptr);
}

}  // namespace

size_t attn_decode_workspace(size_t seqs, size_t hq, size_t hkv) { return kPartsBytes + counters_bytes(seqs, hq, hkv); }

bool attn_decode_fits(size_t seqs, size_t hq, size_t hkv) { return fits_launch(seqs, hkv * head_tiles_of(hq, hkv), kWaves * 64); }

hipError_t launch_attn_decode(const Launch& L, const AttnArgs& a, bool e4m3, void* ws) {
  if (a.dim > 64) return e4m3 ? launch<128, true>(L, a, ws) : launch<128, false>(L, a, ws);
  return e4m3 ? launch<64, true>(L, a, ws) : launch<64, false>(L, a, ws);
}

}  // namespace ar
