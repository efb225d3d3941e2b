// Gradient of attention: with P = exp(scale q k - lse) on visible keys and
// delta = rowsum(d_out * out),
//   dV = P^T dO,  dS = P (dO V^T - delta),  dQ = scale dS K,  dK = scale dS^T Q.
//
// Two passes over the pairs of queries and keys, each with the sums of its own
// rows in registers, so that no sum is shared and the order of every sum is
// fixed: one for queries (three products: S, dP, dQ), one for keys (four: S,
// dP, dV, dK).  A single pass would need five products, but sums of dQ that
// many workgroups add to, in no order.
//
// For keys, a workgroup takes some of a key head's query heads, and where that
// is not all of them their sums are joined afterwards.  The first keys of a
// sequence that all queries see (sinks) have their far queries cut into runs,
// joined there too.
//
// Bound by the matrix cores.  2 x 4096 tokens, 64 heads of 128 on 8, causal:
// 2010 us for both passes, 0.96 PFLOP/s of their seven products (the
// queries' alone 800, the keys' 1190); delta 74, of which the read of out and
// d_out is 42.
#include "ar_attn.hpp"

namespace ar {
namespace {

constexpr int kWavesQ = 8, kQueries = kWavesQ * 32;  // queries of a workgroup
constexpr int kWavesK = 8, kKeysB = kWavesK / 2 * 32;  // keys of a workgroup, each wave half of a tile's queries
constexpr int kBT = 64;                            // rows of the other side at a time
constexpr unsigned kFar = 2048;                    // queries of a run

__device__ __forceinline__ void zero_lds(char* lds, int bytes) {
  for (int o = threadIdx.x * 16; o < bytes; o += blockDim.x * 16) *reinterpret_cast<u32x4*>(lds + o) = u32x4{0, 0, 0, 0};
  __syncthreads();
}

// Row `col` of 32 as a second operand: 8 values at 16 s + 8 hh.
template <int KS>
__device__ __forceinline__ void load_row(Frag8 (&f)[KS], const uint16_t* p, int hh, unsigned dim) {
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const unsigned d = 16 * s + 8 * hh;
    f[s].u = d < dim ? *reinterpret_cast<const u32x4*>(p + d) : u32x4{0, 0, 0, 0};
  }
}

template <int DT>
__device__ __forceinline__ void clear(f32x16 (&o)[DT]) {
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[d][r] = 0.f;
}

// A lane's row of a result: 4 columns at 32 d + 8 g + 4 hh.
template <int DT>
__device__ __forceinline__ void store_row(uint16_t* p, const f32x16 (&o)[DT], float f, int hh, unsigned dim) {
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const unsigned at = 32 * d + 8 * g + 4 * hh;
      if (at < dim)
        *reinterpret_cast<u32x2*>(p + at) = u32x2{result_bf16x2(o[d][4 * g] * f, o[d][4 * g + 1] * f),
                                                  result_bf16x2(o[d][4 * g + 2] * f, o[d][4 * g + 3] * f)};
    }
}
template <int DT>
__device__ __forceinline__ void store_row(float* p, const f32x16 (&o)[DT], int hh, unsigned dim) {
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const unsigned at = 32 * d + 8 * g + 4 * hh;
      if (at < dim)
        *reinterpret_cast<f32x4*>(p + at) = f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
    }
}

// lse, of a query without keys 0.
__device__ __forceinline__ float finite_lse(float lse) { return lse == AR_NEG_INF ? 0.f : lse; }

// dQ: 256 queries of one head, 64 keys at a time.  DELTA: delta instead.
//
// delta is rowsum(d_out * out) from the out that was rounded to bf16, and its
// error reaches all of a row's dS alike.  Among many keys that is little beside
// dS' own rounding, among few it is most of the error (8 keys: dQ and dK 0.0034
// off, where their rounding alone leaves 0.0017).  So for queries that see up
// to kFew keys, and the others of their tile, delta is formed from its
// definition, the sum of P dP, which costs the first two products once more.
// (A window up to kFew: all queries.  16384 tokens, 64 heads of 128 on 8, all
// gradients: 1190 us with a window of 256, 970 with one of 257; 8 heads on 1:
// 188 and 165.)
constexpr int kFew = 256;
template <int DP, bool DELTA>
__device__ __forceinline__ void queries_pass(const AttnBwdArgs& b, float* delta, unsigned block, char* lds) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr uint32_t kTile = kBT * DP * 2;
  const AttnArgs& a = b.f;
  const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int col = lane & 31, hh = lane >> 5;
  const unsigned rank = block / a.hq, hi = block % a.hq;
  const unsigned kvh = hi % a.hkv, head = kvh * (a.hq / a.hkv) + hi / a.hkv;
  Tile tile;
  if (!find_tile<true>(a.cu_q, a.seqs, a.rows_q, kQueries, rank, &tile)) return;
  const Rows rq = rows_at(a.cu_q, tile.seq, a.rows_q), rk = rows_at(a.cu_k, tile.seq, a.rows_k);
  const int shift = (int)rk.count - (int)rq.count, last = (int)rq.count - 1;
  const int p0 = shift + (int)tile.row, p1 = shift + min((int)tile.row + kQueries - 1, last);
  const KeyRange keys = key_range(p0, p1, a.window, a.sinks, kBT);
  if constexpr (DELTA) {
    if (p0 + 1 > kFew && (long long)a.window + a.sinks > kFew) {
      // 16 lanes a row, eight rows of a lane on their way at once
      const unsigned i = t % 16, end = min(tile.row + kQueries, rq.count);
      constexpr int N = kQueries / (kWavesQ * 4);
      u32x4 x[N], y[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const size_t at = rq.first + min(tile.row + t / 16 + n * kWavesQ * 4, end - 1);
        const unsigned d = min(i * 8, a.dim - 8);
        x[n] = *reinterpret_cast<const u32x4*>(b.out.p + at * b.out.ts + head * b.out.hs + d);
        y[n] = *reinterpret_cast<const u32x4*>(b.d_out.p + at * b.d_out.ts + head * b.d_out.hs + d);
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const unsigned r = tile.row + t / 16 + n * kWavesQ * 4;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum = __builtin_fmaf(lo_f32(x[n][e]), lo_f32(y[n][e]), sum);
          sum = __builtin_fmaf(hi_f32(x[n][e]), hi_f32(y[n][e]), sum);
        }
        sum = i * 8 < a.dim ? sum : 0.f;
#pragma unroll
        for (int d = 1; d < 16; d *= 2) sum += __shfl_xor(sum, d);
        if (i == 0 && r < end) delta[(size_t)head * a.rows_q + rq.first + r] = sum;
      }
      return;
    }
  }
  const int row = (int)tile.row + wave * 32 + col, p = shift + min(row, last), start = window_start(p, a.window);
  const int wp0 = shift + min((int)tile.row + wave * 32, last), wp1 = shift + min((int)tile.row + wave * 32 + 31, last);
  const int wstart0 = window_start(wp0, a.window), wstart1 = window_start(wp1, a.window);

  if (a.dim < DP) zero_lds(lds, 4 * kTile);
  const size_t at = rq.first + min(row, last);
  Frag8 q[KS], g[KS];
  load_row(q, a.q.p + at * a.q.ts + head * a.q.hs, hh, a.dim);
  load_row(g, b.d_out.p + at * b.d_out.ts + head * b.d_out.hs, hh, a.dim);
  const float lse2 = finite_lse(a.lse[at * a.lse_ts + head * a.lse_hs]) * kLog2e, dl = DELTA ? 0.f : delta[(size_t)head * a.rows_q + at];
  const float c = a.scale * kLog2e;
  const uint16_t* kb = a.k.p + (size_t)rk.first * a.k.ts + kvh * a.k.hs;
  const uint16_t* vb = a.v.p + (size_t)rk.first * a.v.ts + kvh * a.v.hs;
  const uint32_t lbase = lds_addr(lds);
  const TileCopy<DP, kWavesQ> copy_rows(a.k.ts, a.v.ts, a.dim, wave, lane);
  auto copy = [&](int n, int buf) {
    const KeyStep k = key_step(keys, n, kBT);
    copy_rows(kb, a.k.ts, vb, a.v.ts, k.j0, k.end - 1, lbase + buf * 2 * kTile);
  };
  f32x16 o[DT];
  clear(o);
  float sum = 0.f;                             // DELTA: of P dP
  if (keys.steps > 0) copy(0, 0);
  for (int n = 0; n < keys.steps; ++n) {
    const int buf = n & 1;
    wait_copies();
    __syncthreads();
    if (n + 1 < keys.steps) copy(n + 1, buf ^ 1);
    const KeyStep k = key_step(keys, n, kBT);
    const int j0 = k.j0;
    if ((int)tile.row + wave * 32 > last || j0 > wp1 || (!k.sinks && j0 + kBT <= wstart0)) continue;
    const bool whole = j0 + kBT - 1 <= min(wp0, k.end - 1) && (k.sinks || j0 >= wstart1);
    const Interval view((k.sinks ? 0 : start) - j0 - 4 * hh, min(p, k.end - 1) - j0 - 4 * hh);
    const LaneAddr<DP> at_k(lbase + buf * 2 * kTile, lane);
    auto tile_step = [&](auto masked) {
      constexpr bool MASK = decltype(masked)::value;
#pragma unroll 1
      for (int r0 = 0; r0 < kBT; r0 += 32) {
        const LaneAddr<DP> from = {at_k, (uint32_t)(r0 * DP * 2)};
        // products 0 .. KS - 1: scores; then dP; then dQ
        constexpr int ALL = 2 * KS + (DELTA ? 0 : 2 * DT), AHEAD = 4;
        Frag8 f[AHEAD], pd[2];
        f32x16 s, d;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = 0.f;
          d[r] = -dl;                          // dP - delta
        }
        auto load = [&](auto ii) {
          constexpr int i = decltype(ii)::value;
          Frag8& x = f[i % AHEAD];
          if constexpr (i < KS) x.u = from.rows(0, i);
          else if constexpr (i < 2 * KS) x.u = from.rows(kBT, i - KS);
          else x = from.columns((i - 2 * KS) / DT * 16, (i - 2 * KS) % DT);
        };
        steps<AHEAD>(load);
        steps<ALL>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          const Frag8& x = f[i % AHEAD];
          if constexpr (i < KS) s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, q[i].b, s, 0, 0, 0);
          else if constexpr (i < 2 * KS) d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, g[i - KS].b, d, 0, 0, 0);
          else o[i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, pd[(i - 2 * KS) / DT].b, o[i % DT], 0, 0, 0);
          if constexpr (i + AHEAD < ALL) load(SPc<i + AHEAD>{});
          if constexpr (i >= KS && i < 2 * KS) {   // beside the products of dP
            constexpr int per = 16 / KS, a0 = (i - KS) * per;
#pragma unroll
            for (int r = a0; r < a0 + per; ++r) s[r] = exp2_fast(__builtin_fmaf(s[r], c, -lse2));
          }
          if constexpr (i == 2 * KS - 1) {
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                y[e] = s[r + e] * d[r + e];
                if (MASK) y[e] = view.has(r0 + 8 * (r / 4) + r % 4 + e) ? y[e] : 0.f;
              }
              if constexpr (DELTA) sum += y[0] + y[1];
              else pd[r / 8].w[r % 8 / 2] = cvt_bf16x2(y[0], y[1]);
            }
          }
          keep_order();
        });
      }
    };
    if (whole) tile_step(std::false_type{});
    else tile_step(std::true_type{});
  }
  if constexpr (DELTA) {
    sum += __shfl_xor(sum, 32);
    if (row <= last && hh == 0) delta[(size_t)head * a.rows_q + at] = sum;
  } else if (row <= last) {
    store_row(b.dq.p + at * b.dq.ts + head * b.dq.hs, o, a.scale, hh, a.dim);
  }
}

template <int DP>
__global__ __launch_bounds__(kWavesQ * 64, 2) void k_attn_delta(AttnBwdArgs b, float* delta) {
  __shared__ __align__(1024) char lds[4 * kBT * DP * 2];
  queries_pass<DP, true>(b, delta, blockIdx.x, lds);
}

// The queries that a tile of keys meets in its own pass, and of a tile with
// sinks those beyond, which are cut into runs.  A tile with sinks takes at
// least kFar queries itself, so only sequences with more have runs.
struct Band {
  int lo, hi;                  // first query, first beyond
};
__device__ __forceinline__ Band band_of(const AttnArgs& a, int j0, int shift, int nq) {
  const long long wide = (long long)j0 + kKeysB - 1 + a.window - shift;
  Band r;
  r.lo = min(max(j0 - shift, 0), nq);
  r.hi = (int)min((long long)nq, max(wide, (long long)r.lo));
  if (j0 < (int)a.sinks) r.hi = min(nq, max(r.hi, r.lo + (int)kFar));
  return r;
}

// Where sums of (dK, dV) go that are to be joined.  `near`: [sets][rows_k][dim]
// of dK, then of dV; `far`: [run][tile with sinks][set][dK, dV][kKeysB][dim].
struct KeySums {
  float *near, *far;           // nullptr: results are written; there are no runs
  unsigned per, sets;          // query heads of a workgroup; hq / per
  unsigned sink_tiles;         // tiles of a sequence that may have runs
  unsigned runs;               // at most, of all sequences
};

// dK, dV of 128 keys for some query heads of their key head, 64 queries at a
// time; the first workgroups take the runs of queries beyond tiles with sinks.
//
// A wave has 32 of the keys and half of a tile's queries, and its partner's
// sums are added at the end.  Two waves a SIMD hold their sums (128 registers)
// and two 32 x 32 tiles in registers only because the keys and values stay in
// LDS, too: with them in registers there is room for one wave a SIMD, which
// measured slower though it reads a third less from LDS (2 x 4096 tokens, 64
// heads of 128: 1437 us, this 1190).  The arithmetic of P and dS is spread
// over the products that do not need it.
template <int DP>
__device__ __forceinline__ void keys_pass(const AttnBwdArgs& b, const float* delta, const KeySums& sums, unsigned block,
                                          char* lds, float (*lrow)[2][kBT]) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr uint32_t kTile = kBT * DP * 2;
  // lds: two tiles of queries; the keys and values, 64 at a time.  lrow: lse, delta of the queries
  const AttnArgs& a = b.f;
  const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int col = lane & 31, hh = lane >> 5;
  unsigned rank = block / sums.sets;
  const unsigned hi = block % sums.sets;   // sets of one key head on one XCD, if there are eight heads
  const unsigned kvh = hi % a.hkv, set = kvh * (sums.sets / a.hkv) + hi / a.hkv, head0 = set * sums.per;
  const unsigned far_tiles = sums.runs * sums.sink_tiles;
  const bool far = rank < far_tiles;
  Tile tile;
  int j0, q_lo, q_hi;
  Rows rq, rk;
  if (far) {
    const unsigned st = rank % sums.sink_tiles;
    // (offsets that do not ascend can ask for more runs than there is room for)
    if (!find_tile<true, true>(a.cu_q, a.seqs, a.rows_q, kFar, rank / sums.sink_tiles, &tile) || tile.at >= sums.runs) return;
    rq = rows_at(a.cu_q, tile.seq, a.rows_q);
    rk = rows_at(a.cu_k, tile.seq, a.rows_k);
    j0 = (int)(st * kKeysB);
    if (j0 >= (int)rk.count) return;
    q_lo = max((int)tile.row, band_of(a, j0, (int)rk.count - (int)rq.count, (int)rq.count).hi);
    q_hi = min((int)(tile.row + kFar), (int)rq.count);
    if (q_lo >= q_hi) return;
  } else {
    if (!find_tile<false>(a.cu_k, a.seqs, a.rows_k, kKeysB, rank - far_tiles, &tile)) return;
    rq = rows_at(a.cu_q, tile.seq, a.rows_q);
    rk = rows_at(a.cu_k, tile.seq, a.rows_k);
    j0 = (int)tile.row;
    const Band band = band_of(a, j0, (int)rk.count - (int)rq.count, (int)rq.count);
    q_lo = band.lo;
    q_hi = band.hi;
  }
  const int shift = (int)rk.count - (int)rq.count, klast = (int)rk.count - 1;
  const int w0 = j0 + (wave & 3) * 32, key = w0 + col, r0 = (wave >> 2) * 32;   // the wave's keys, its rows of a tile
  const bool sinks = key < (int)a.sinks;
  const int nt = max((q_hi - q_lo + kBT - 1) / kBT, 0), all = nt * (int)sums.per;   // tiles of a head, of all

  if (a.dim < DP) zero_lds(lds, 8 * kTile);
  const size_t at = rk.first + min(key, klast);
  const float c = a.scale * kLog2e;
  const uint16_t* qb = a.q.p + (size_t)rq.first * a.q.ts + head0 * a.q.hs;
  const uint16_t* gb = b.d_out.p + (size_t)rq.first * b.d_out.ts + head0 * b.d_out.hs;
  const uint32_t lbase = lds_addr(lds);
  const float inv_scale = 1.0f / a.scale;
  float stat = 0.f;                            // of the tile's query t: lse, or delta
  const TileCopy<DP, kWavesK> copy_rows(a.q.ts, b.d_out.ts, a.dim, wave, lane);
  // from the last tile on: there the workgroups of a sequence's keys begin together, and share
  // what they read in the L2
  int next = 0, next_head = 0;                 // tile that is copied next
  auto copy = [&](int buf) {
    const int first = q_lo + (nt - 1 - next) * kBT;
    if (t < 2 * kBT) {
      const size_t i = rq.first + min(first + t % kBT, q_hi - 1), head = head0 + next_head;
      // what the sums start from: S - lse / scale, dP - delta
      stat = t < kBT ? -finite_lse(a.lse[i * a.lse_ts + head * a.lse_hs]) * inv_scale : -delta[head * a.rows_q + i];
    }
    copy_rows(qb + next_head * a.q.hs, a.q.ts, gb + next_head * b.d_out.hs, b.d_out.ts, first, q_hi - 1, lbase + buf * 2 * kTile);
    if (++next == nt) {
      next = 0;
      ++next_head;
    }
  };
  f32x16 dk[DT], dv[DT];
  clear(dk);
  clear(dv);
  int now = 0;
  if (all > 0) {
    const TileCopy<DP, kWavesK> copy_keys(a.k.ts, a.v.ts, a.dim, wave, lane);
    const uint16_t *kb = a.k.p + (size_t)rk.first * a.k.ts + kvh * a.k.hs, *vb = a.v.p + (size_t)rk.first * a.v.ts + kvh * a.v.hs;
    for (int x = 0; x < 2; ++x) copy_keys(kb, a.k.ts, vb, a.v.ts, j0 + 64 * x, klast, lbase + (4 + 2 * x) * kTile);
    copy(0);
  }
  const uint32_t lkeys = lbase + (4 + (wave >> 1 & 1) * 2) * kTile + (wave & 1) * 32 * DP * 2;
  for (int n = 0; n < all; ++n) {
    const int buf = n & 1;
    wait_copies();
    if (t < 2 * kBT) lrow[buf][t / kBT][t % kBT] = stat;
    __syncthreads();
    if (n + 1 < all) copy(buf ^ 1);
    const int i0 = q_lo + (nt - 1 - now) * kBT + r0, p0 = shift + i0, pn = shift + min(i0 + 32, q_hi) - 1;   // the wave's queries
    now = now + 1 == nt ? 0 : now + 1;
    const int wfar = window_start(p0, a.window);   // first key that one of them has in its window
    if (i0 >= q_hi || w0 > klast || w0 > pn || (w0 + 31 < wfar && w0 >= (int)a.sinks)) continue;
    const bool whole = i0 + 32 <= q_hi && w0 + 31 <= p0 && w0 + 31 <= klast &&
                       (w0 >= window_start(pn, a.window) || w0 + 31 < (int)a.sinks);
    // of the wave's queries, less 4 hh, those that see the lane's key
    const int far_end = sinks ? q_hi - 1 : (int)min((long long)q_hi - 1, (long long)key + a.window - 1 - shift);
    const Interval view(key - shift - i0 - 4 * hh, (key <= klast ? far_end : -0x40000000) - i0 - 4 * hh);
    const LaneAddr<DP> from(lbase + buf * 2 * kTile + r0 * DP * 2, lane), keys(lkeys, lane);
    auto tile_step = [&](auto masked) {
      constexpr bool MASK = decltype(masked)::value;
        f32x16 s, d;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 l = *reinterpret_cast<const f32x4*>(&lrow[buf][0][r0 + 8 * g + 4 * hh]);
          const f32x4 e = *reinterpret_cast<const f32x4*>(&lrow[buf][1][r0 + 8 * g + 4 * hh]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            s[4 * g + x] = l[x];
            d[4 * g + x] = e[x];
          }
        }
        // products 0 .. KS - 1: scores; then dP; dV; dK, 2 DT each
        constexpr int ALL = 2 * KS + 4 * DT, AHEAD = 3;
        Frag8 f[AHEAD], fk[AHEAD];
        auto load = [&](auto ii) {
          constexpr int i = decltype(ii)::value;
          Frag8& o = f[i % AHEAD];
          if constexpr (i < 2 * KS) {
            o.u = from.rows(i / KS * kBT, i % KS);
            fk[i % AHEAD].u = keys.rows(i / KS * kBT, i % KS);
          }
          else if constexpr (i < 2 * KS + 2 * DT) o = from.columns(kBT + (i - 2 * KS) / DT * 16, (i - 2 * KS) % DT);
          else o = from.columns((i - 2 * KS - 2 * DT) / DT * 16, (i - 2 * KS - 2 * DT) % DT);
        };
        Frag8 pp[2], pd[2];
        auto seen = [&](int r) { return view.has(8 * (r / 4) + r % 4); };
        steps<AHEAD>(load);
        steps<ALL>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          const Frag8& o = f[i % AHEAD];
          if constexpr (i < KS) {
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.b, fk[i % AHEAD].b, s, 0, 0, 0);
          } else if constexpr (i < 2 * KS) {
            d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.b, fk[i % AHEAD].b, d, 0, 0, 0);
          } else if constexpr (i < 2 * KS + 2 * DT) {
            constexpr int n = i - 2 * KS;
            dv[n % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.b, pp[n / DT].b, dv[n % DT], 0, 0, 0);
          } else {
            constexpr int n = i - 2 * KS - 2 * DT;
            dk[n % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.b, pd[n / DT].b, dk[n % DT], 0, 0, 0);
          }
          if constexpr (i + AHEAD < ALL) load(SPc<i + AHEAD>{});
          // beside the products of dP, P; beside those of dV, dS
          if constexpr (i >= KS && i < 2 * KS) {
            constexpr int per = 16 / KS, r0_ = (i - KS) * per;
#pragma unroll
            for (int r = r0_; r < r0_ + per; r += 2) {
#pragma unroll
              for (int x = r; x < r + 2; ++x) {
                s[x] = exp2_fast(s[x] * c);
                if (MASK) s[x] = seen(x) ? s[x] : 0.f;
              }
              pp[r / 8].w[r % 8 / 2] = cvt_bf16x2(s[r], s[r + 1]);
            }
          }
          if constexpr (i >= 2 * KS && i < 2 * KS + 2 * DT) {
            constexpr int per = 16 / (2 * DT), r0_ = (i - 2 * KS) * per;
#pragma unroll
            for (int r = r0_; r < r0_ + per; r += 2) {
              const float x = s[r] * d[r], y = s[r + 1] * d[r + 1];
              pd[r / 8].w[r % 8 / 2] = MASK ? cvt_bf16x2(s[r] == 0.f ? 0.f : x, s[r + 1] == 0.f ? 0.f : y) : cvt_bf16x2(x, y);
            }
          }
          keep_order();
        });
    };
    if (whole) tile_step(std::false_type{});
    else tile_step(std::true_type{});
  }
  // The sums of both halves: a wave gives its partner dK or dV, and takes the other.
  __syncthreads();
  const bool upper = wave >= 4;
  f32x4* lsum = reinterpret_cast<f32x4*>(lds) + lane;
  auto give = [&](const f32x16 (&sum)[DT]) {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        lsum[((wave * DT + d) * 4 + g) * kWave] = f32x4{sum[d][4 * g], sum[d][4 * g + 1], sum[d][4 * g + 2], sum[d][4 * g + 3]};
  };
  auto take = [&](f32x16 (&sum)[DT]) {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 x = lsum[(((wave ^ 4) * DT + d) * 4 + g) * kWave];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[d][4 * g + e] += x[e];
        keep_order();
      }
  };
  auto store = [&](f32x16 (&sum)[DT], const HeadOut& out, float f) {
    if (key > klast) return;
    if (far) {
      const size_t slot = ((size_t)tile.at * sums.sink_tiles + j0 / kKeysB) * sums.sets + set;
      store_row(sums.far + ((slot * 2 + upper) * kKeysB + key - j0) * a.dim, sum, hh, a.dim);
    } else if (sums.near) {
      store_row(sums.near + (((size_t)upper * sums.sets + set) * a.rows_k + at) * a.dim, sum, hh, a.dim);
    } else {
      store_row(out.p + at * out.ts + kvh * out.hs, sum, f, hh, a.dim);
    }
  };
  if (upper) give(dk);
  else give(dv);
  __syncthreads();
  if (upper) {
    take(dv);
    store(dv, b.dv, 1.0f);
  } else {
    take(dk);
    store(dk, b.dk, a.scale);
  }
}

// Both passes in one launch, the keys' first, whose workgroups have more to do:
// short batches wait for one of them only, and long ones end together.
template <int DP>
__global__ __launch_bounds__(kWavesQ * 64, 2) void k_attn_bwd(AttnBwdArgs b, float* delta, KeySums sums, unsigned key_blocks) {
  static_assert(kWavesQ == kWavesK, "both passes have one workgroup size");
  __shared__ __align__(1024) char lds[8 * kBT * DP * 2];
  __shared__ __align__(16) float lrow[2][2][kBT];
  if (blockIdx.x < key_blocks) keys_pass<DP>(b, delta, sums, blockIdx.x, lds, lrow);
  else queries_pass<DP, false>(b, delta, blockIdx.x - key_blocks, lds);
}

// Joins the sums of a key's query heads and runs: a workgroup takes 8 rows of
// one key head of dK, or of dV.
constexpr int kJoinRows = 8;
__global__ __launch_bounds__(256) void k_attn_join(AttnBwdArgs b, KeySums sums) {
  const AttnArgs& a = b.f;
  const unsigned which = blockIdx.x & 1, kvh = (blockIdx.x >> 1) % a.hkv, rank = (blockIdx.x >> 1) / a.hkv;
  const unsigned group = sums.sets / a.hkv;    // sets of a key head
  Tile tile;
  if (!find_tile<true>(a.cu_k, a.seqs, a.rows_k, kJoinRows, rank, &tile)) return;
  const Rows rq = rows_at(a.cu_q, tile.seq, a.rows_q), rk = rows_at(a.cu_k, tile.seq, a.rows_k);
  const int j0 = (int)(tile.row / kKeysB * kKeysB);   // of the rows' tile of keys
  // runs of the sequence: numbers first .. first + runs - 1, queries from (1 + i) kFar on
  unsigned first = 0, runs = 0, skip = 0;
  if (sums.sink_tiles && j0 < (int)a.sinks && (unsigned)(j0 / kKeysB) < sums.sink_tiles && rq.count > kFar) {
    runs = (rq.count - 1) / kFar;
    for (unsigned s0 = 0; s0 < tile.seq; s0 += kWave) {
      const unsigned s = s0 + lane_id(), n = s < tile.seq ? rows_of(a.cu_q, s, a.rows_q).count : 0;
      first += last_lane(wave_scan(n ? (n - 1) / kFar : 0));
    }
    runs = first < sums.runs ? min(runs, sums.runs - first) : 0;
    // the first runs' queries may all have been near
    const Band band = band_of(a, j0, (int)rk.count - (int)rq.count, (int)rq.count);
    while (skip < runs && (int)min((skip + 2) * kFar, rq.count) <= band.hi) ++skip;
  }
  const unsigned per = a.dim / 4, i = threadIdx.x;   // groups of 4 columns
  const unsigned r = i / per, d = i % per * 4;
  if (i >= kJoinRows * per || tile.row + r >= rk.count) return;
  const size_t at = rk.first + tile.row + r;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  const float* near = sums.near + (((size_t)which * sums.sets + kvh * group) * a.rows_k + at) * a.dim + d;
#pragma unroll 4
  for (unsigned h = 0; h < group; ++h) sum += *reinterpret_cast<const f32x4*>(near + (size_t)h * a.rows_k * a.dim);
  for (unsigned n = skip; n < runs; ++n) {
    const size_t slot = ((size_t)(first + n) * sums.sink_tiles + j0 / kKeysB) * sums.sets + kvh * group;
    const float* far = sums.far + ((slot * 2 + which) * kKeysB + tile.row - j0 + r) * a.dim + d;
#pragma unroll 4
    for (unsigned h = 0; h < group; ++h) sum += *reinterpret_cast<const f32x4*>(far + (size_t)h * 2 * kKeysB * a.dim);
  }
  const float f = which ? 1.0f : a.scale;
  const HeadOut& o = which ? b.dv : b.dk;
  *reinterpret_cast<u32x2*>(o.p + at * o.ts + kvh * o.hs + d) =
      u32x2{result_bf16x2(sum[0] * f, sum[1] * f), result_bf16x2(sum[2] * f, sum[3] * f)};
}

struct Room {
  size_t delta, near, far;     // binary32 values
  unsigned per, sets, sink_tiles, runs;
};
Room room_of(size_t rows_q, size_t rows_k, size_t hq, size_t hkv, size_t dim, size_t window, size_t sinks) {
  Room r{};
  r.delta = cdiv(rows_q * hq, 64) * 64;
  // Query heads of a key head that one workgroup takes one after the other, each
  // of which spares a write and a read of its sums and a start: as many as
  // leave 512 workgroups, two rounds of one a CU (whose LDS one fills).
  const size_t group = hq / hkv, tiles = cdiv(rows_k ? rows_k : 1, kKeysB) * hkv;
  size_t per = group;
  while (per > 1 && (group % per || tiles * (group / per) < 512)) --per;
  r.per = (unsigned)per;
  r.sets = (unsigned)(hq / per);
  if (window < rows_k && sinks) {
    r.sink_tiles = (unsigned)cdiv(sinks < rows_k ? sinks : rows_k, kKeysB);
    r.runs = (unsigned)(rows_q / kFar);
    if (r.runs == 0) r.sink_tiles = 0;
  }
  if (r.sets > hkv || r.sink_tiles) r.near = 2 * r.sets * rows_k * dim;
  r.far = (size_t)r.runs * r.sink_tiles * r.sets * 2 * kKeysB * dim;
  if (r.far == 0) r.runs = r.sink_tiles = 0;
  return r;
}

template <int DP>
hipError_t launch(const Launch& L, const AttnBwdArgs& b) {
  const AttnArgs& a = b.f;
  const Room room = room_of(a.rows_q, a.rows_k, a.hq, a.hkv, a.dim, a.window, a.sinks);
  float* delta = static_cast<float*>(b.workspace);
  hipError_t e;
  if (a.rows_q) {
    e = launch_k(k_attn_delta<DP>, dim3((a.rows_q / kQueries + a.seqs) * a.hq), dim3(kWavesQ * 64), 0, L.stream, b, delta);
    if (e != hipSuccess) return e;
  }
  const KeySums sums{room.near ? delta + room.delta : nullptr, room.far ? delta + room.delta + room.near : nullptr,
                     room.per, room.sets, room.sink_tiles, room.runs};
  const bool keys = b.dk.p && a.rows_k;
  const unsigned tiles = room.runs * room.sink_tiles + a.rows_k / kKeysB + a.seqs;
  const unsigned key_blocks = keys ? tiles * room.sets : 0;
  const unsigned query_blocks = b.dq.p && a.rows_q ? (a.rows_q / kQueries + a.seqs) * a.hq : 0;
  if (key_blocks + query_blocks == 0) return hipSuccess;
  e = launch_k(k_attn_bwd<DP>, dim3(key_blocks + query_blocks), dim3(kWavesQ * 64), 0, L.stream, b, delta, sums, key_blocks);
  if (e != hipSuccess || !keys || !sums.near) return e;
  return launch_k(k_attn_join, dim3((a.rows_k / kJoinRows + a.seqs) * a.hkv * 2), dim3(256), 0, L.stream, b, sums);
}

}  // namespace

size_t attn_bwd_workspace(size_t rows_q, size_t rows_k, size_t seqs, size_t hq, size_t hkv, size_t dim, size_t window,
                          size_t sinks) {
  const Room r = room_of(rows_q, rows_k, hq, hkv, dim, window, sinks);
  return (r.delta + r.near + r.far) * sizeof(float);
}

bool attn_bwd_fits(size_t rows_q, size_t rows_k, size_t seqs, size_t hq, size_t hkv, size_t dim, size_t window, size_t sinks) {
  const Room r = room_of(rows_q, rows_k, hq, hkv, dim, window, sinks);
  const size_t blocks = ((size_t)r.runs * r.sink_tiles + rows_k / kKeysB + seqs) * r.sets + (rows_q / kQueries + seqs) * hq;
  const size_t join = (rows_k / kJoinRows + seqs) * hkv * 2;
  return fits_launch(blocks, 1, kWavesQ * 64) && fits_launch(join, 1, 256);
}

hipError_t launch_attn_bwd(const Launch& L, const AttnBwdArgs& b) {
  return b.f.dim > 64 ? launch<128>(L, b) : launch<64>(L, b);
}

}  // namespace ar
