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
// For keys, each query head is a workgroup's work, and its sums are joined
// over the heads of a key head afterwards.  The first keys of a sequence that
// all queries see (sinks) have their far queries cut into runs, joined there
// too.
#include "ar_attn.hpp"

namespace ar {
namespace {

constexpr int kWavesB = 8, kRowsB = kWavesB * 32;  // rows of a workgroup: of queries, or of keys
constexpr int kBT = 64;                            // rows of the other side at a time
constexpr unsigned kFar = 2048;                    // queries of a run

// delta of every query and head, 16 lanes each: [hq][rows_q]
__global__ __launch_bounds__(256) void k_attn_delta(HeadRows out, HeadRows d_out, float* delta, unsigned rows, unsigned hq,
                                                    unsigned dim) {
  const size_t at = (size_t)blockIdx.x * 16 + threadIdx.x / 16;
  const unsigned row = (unsigned)(at / hq), head = (unsigned)(at % hq), i = threadIdx.x % 16;
  float sum = 0.f;
  if (row < rows && i * 8 < dim) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(out.p + (size_t)row * out.ts + head * out.hs + i * 8);
    const u32x4 y = *reinterpret_cast<const u32x4*>(d_out.p + (size_t)row * d_out.ts + head * d_out.hs + i * 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = __builtin_fmaf(lo_f32(x[e]), lo_f32(y[e]), sum);
      sum = __builtin_fmaf(hi_f32(x[e]), hi_f32(y[e]), sum);
    }
  }
#pragma unroll
  for (int d = 1; d < 16; d *= 2) sum += __shfl_xor(sum, d);
  if (row < rows && i == 0) delta[(size_t)head * rows + row] = sum;
}

// Copies rows first .. of two matrices to LDS, kBT rows each; rows past `last`
// are copies of it.
template <int DP>
__device__ __forceinline__ void copy_tiles(const uint16_t* x, size_t xs, const uint16_t* y, size_t ys, int first, int last,
                                           unsigned dim, uint32_t lds, int wave, int lane) {
  constexpr int RPC = 1024 / (DP * 2), CPR = DP / 8, COPIES = kBT / RPC / kWavesB;
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int r = (i * kWavesB + wave) * RPC + lane / CPR, j = min(first + r, last);
    const int ch = (lane % CPR) ^ swizzle<DP>(r);
    const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds + (i * kWavesB + wave) * 1024));
    if (ch * 8 < (int)dim) {
      copy16_to_lds(x + (size_t)j * xs + ch * 8, to);
      copy16_to_lds(y + (size_t)j * ys + ch * 8, to + kBT * DP * 2);
    }
  }
}

template <int DP>
__device__ __forceinline__ void zero_lds(char* lds, int bytes) {
  for (int o = threadIdx.x * 16; o < bytes; o += kWavesB * 64 * 16) *reinterpret_cast<u32x4*>(lds + o) = u32x4{0, 0, 0, 0};
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

// 32 rows of LDS (from row r0) times the rows held in f.
template <int DP>
__device__ __forceinline__ f32x16 times_rows(const char* tile, int r0, int col, int hh, const Frag8 (&f)[DP / 16]) {
  f32x16 s;
#pragma unroll
  for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
  for (int x = 0; x < DP / 16; ++x) {
    Frag8 k;
    k.u = *reinterpret_cast<const u32x4*>(tile + chunk_addr<DP>(r0 + col, 2 * x + hh));
    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, f[x].b, s, 0, 0, 0);
  }
  return s;
}

// acc += (32 rows of LDS from r0, transposed) times the 32 x 32 values s.
template <int DP>
__device__ __forceinline__ void add_columns(f32x16 (&acc)[DP / 32], uint32_t tile, int r0, int lane, const f32x16& s) {
  const int va = 4 * (lane >> 5) + (lane & 15) / 4, vch = 2 * ((lane >> 4) & 1) + (lane & 3) / 2;
  const uint32_t vhalf = (lane & 1) * 8;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    Frag8 p;
#pragma unroll
    for (int e = 0; e < 4; ++e) p.w[e] = cvt_bf16x2(s[8 * x + 2 * e], s[8 * x + 2 * e + 1]);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) {
      Frag8 v;
      const int r = r0 + 16 * x + va;
      v.s[0] = read_tr16(tile + chunk_addr<DP>(r, 4 * d + vch) + vhalf);
      v.s[1] = read_tr16(tile + chunk_addr<DP>(r + 8, 4 * d + vch) + vhalf);
      acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, p.b, acc[d], 0, 0, 0);
    }
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

// What an exponent subtracts: lse in powers of two; of a query without keys 0.
__device__ __forceinline__ float lse2_of(float lse) { return lse == AR_NEG_INF ? 0.f : lse * kLog2e; }

// dQ: 256 queries of one head, 64 keys at a time.
template <int DP>
__global__ __launch_bounds__(kWavesB * 64, 2) void k_attn_dq(AttnBwdArgs b, const float* delta) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr uint32_t kTile = kBT * DP * 2;
  __shared__ __align__(1024) char lds[4 * kTile];
  const AttnArgs& a = b.f;
  const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int col = lane & 31, hh = lane >> 5;
  const unsigned rank = blockIdx.x / a.hq, hi = blockIdx.x % a.hq;
  const unsigned kvh = hi % a.hkv, head = kvh * (a.hq / a.hkv) + hi / a.hkv;
  Tile tile;
  if (!find_tile(a.cu_q, a.seqs, a.rows_q, kRowsB, rank, &tile)) return;
  const Rows rq = rows_of(a.cu_q, tile.seq, a.rows_q), rk = rows_of(a.cu_k, tile.seq, a.rows_k);
  const int shift = (int)rk.count - (int)rq.count, last = (int)rq.count - 1;
  const int p0 = shift + (int)tile.row, p1 = shift + min((int)tile.row + kRowsB - 1, last);
  const int lo = window_start(p0, a.window), sunk = min((int)a.sinks, lo), end = p1 + 1;
  const int ts = (sunk + kBT - 1) / kBT, nt = end > lo ? ts + (end - lo + kBT - 1) / kBT : 0;
  const int row = (int)tile.row + wave * 32 + col, p = shift + min(row, last), start = window_start(p, a.window);
  const int wp0 = shift + min((int)tile.row + wave * 32, last), wp1 = shift + min((int)tile.row + wave * 32 + 31, last);
  const int wstart0 = window_start(wp0, a.window), wstart1 = window_start(wp1, a.window);

  if (a.dim < DP) zero_lds<DP>(lds, 4 * kTile);
  const size_t at = rq.first + min(row, last);
  Frag8 q[KS], g[KS];
  load_row(q, a.q.p + at * a.q.ts + head * a.q.hs, hh, a.dim);
  load_row(g, b.d_out.p + at * b.d_out.ts + head * b.d_out.hs, hh, a.dim);
  const float lse2 = lse2_of(a.lse[at * a.lse_ts + head * a.lse_hs]), dl = delta[(size_t)head * a.rows_q + at];
  const float c = a.scale * kLog2e;
  const uint16_t* kb = a.k.p + (size_t)rk.first * a.k.ts + kvh * a.k.hs;
  const uint16_t* vb = a.v.p + (size_t)rk.first * a.v.ts + kvh * a.v.hs;
  const uint32_t lbase = lds_addr(lds);
  auto copy = [&](int n, int buf) {
    copy_tiles<DP>(kb, a.k.ts, vb, a.v.ts, n < ts ? n * kBT : lo + (n - ts) * kBT, (n < ts ? sunk : end) - 1, a.dim,
                   lbase + buf * 2 * kTile, wave, lane);
  };
  f32x16 o[DT];
  clear(o);
  if (nt > 0) copy(0, 0);
  for (int n = 0; n < nt; ++n) {
    const int buf = n & 1;
    wait_copies();
    __syncthreads();
    if (n + 1 < nt) copy(n + 1, buf ^ 1);
    const int j0 = n < ts ? n * kBT : lo + (n - ts) * kBT, jend = n < ts ? sunk : end;
    if ((int)tile.row + wave * 32 > last || j0 > wp1 || (j0 + kBT <= wstart0 && j0 >= (int)a.sinks)) continue;
    const bool whole = j0 + kBT <= jend && j0 + kBT - 1 <= wp0 && j0 >= wstart1;
    const char* tk = lds + buf * 2 * kTile;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f32x16 s = times_rows<DP>(tk, 32 * x, col, hh, q);
      const f32x16 d = times_rows<DP>(tk + kTile, 32 * x, col, hh, g);
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = exp2_fast(__builtin_fmaf(s[r], c, -lse2)) * (d[r] - dl);
      if (!whole) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = j0 + 32 * x + 8 * (r / 4) + 4 * hh + r % 4;
          s[r] = j <= p && j < jend && (j >= start || j < (int)a.sinks) ? s[r] : 0.f;
        }
      }
      add_columns<DP>(o, lbase + buf * 2 * kTile, 32 * x, lane, s);
    }
  }
  if (row <= last) store_row(b.dq.p + at * b.dq.ts + head * b.dq.hs, o, a.scale, hh, a.dim);
}

// The queries that a tile of keys meets in its own pass, and of a tile with
// sinks those beyond, which are cut into runs.  A tile with sinks takes at
// least kFar queries itself, so only sequences with more have runs.
struct Band {
  int lo, hi;                  // first query, first beyond
};
__device__ __forceinline__ Band band_of(const AttnArgs& a, int j0, int shift, int nq) {
  const long long wide = (long long)j0 + kRowsB - 1 + a.window - shift;
  Band r;
  r.lo = min(max(j0 - shift, 0), nq);
  r.hi = (int)min((long long)nq, max(wide, (long long)r.lo));
  if (j0 < (int)a.sinks) r.hi = min(nq, max(r.hi, r.lo + (int)kFar));
  return r;
}

struct KeySums {
  float *near, *far;           // sums of (dK, dV) before they are joined; nullptr: results are written
  unsigned sink_tiles;         // tiles of a sequence that may have runs
  unsigned runs;               // at most, of all sequences
};

// dK, dV of 256 keys for one query head, 64 queries at a time; FAR: one run
// of queries for a tile with sinks.
template <int DP, bool FAR>
__global__ __launch_bounds__(kWavesB * 64, 2) void k_attn_dkv(AttnBwdArgs b, const float* delta, KeySums sums) {
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr uint32_t kTile = kBT * DP * 2;
  __shared__ __align__(1024) char lds[4 * kTile];
  __shared__ __align__(16) float lrow[2][2][kBT];  // lse, delta
  const AttnArgs& a = b.f;
  const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int col = lane & 31, hh = lane >> 5;
  unsigned rank = blockIdx.x / a.hq;
  const unsigned hi = blockIdx.x % a.hq;
  const unsigned kvh = hi % a.hkv, head = kvh * (a.hq / a.hkv) + hi / a.hkv;
  Tile tile;
  int j0, q_lo, q_hi;
  Rows rq, rk;
  if constexpr (FAR) {
    const unsigned st = rank % sums.sink_tiles;
    rank /= sums.sink_tiles;
    // (offsets that do not ascend can ask for more runs than there is room for)
    if (!find_tile<true>(a.cu_q, a.seqs, a.rows_q, kFar, rank, &tile) || tile.at >= sums.runs) return;
    rq = rows_of(a.cu_q, tile.seq, a.rows_q);
    rk = rows_of(a.cu_k, tile.seq, a.rows_k);
    j0 = (int)(st * kRowsB);
    if (j0 >= (int)rk.count) return;
    q_lo = max((int)tile.row, band_of(a, j0, (int)rk.count - (int)rq.count, (int)rq.count).hi);
    q_hi = min((int)(tile.row + kFar), (int)rq.count);
    if (q_lo >= q_hi) return;
  } else {
    if (!find_tile(a.cu_k, a.seqs, a.rows_k, kRowsB, rank, &tile)) return;
    rq = rows_of(a.cu_q, tile.seq, a.rows_q);
    rk = rows_of(a.cu_k, tile.seq, a.rows_k);
    j0 = (int)tile.row;
    const Band band = band_of(a, j0, (int)rk.count - (int)rq.count, (int)rq.count);
    q_lo = band.lo;
    q_hi = band.hi;
  }
  const int shift = (int)rk.count - (int)rq.count, klast = (int)rk.count - 1;
  const int key = j0 + wave * 32 + col, w0 = j0 + wave * 32;
  const bool sinks = key < (int)a.sinks;
  const int nt = (q_hi - q_lo + kBT - 1) / kBT;

  if (a.dim < DP) zero_lds<DP>(lds, 4 * kTile);
  const size_t at = rk.first + min(key, klast);
  Frag8 k[KS], v[KS];
  load_row(k, a.k.p + at * a.k.ts + kvh * a.k.hs, hh, a.dim);
  load_row(v, a.v.p + at * a.v.ts + kvh * a.v.hs, hh, a.dim);
  const float c = a.scale * kLog2e;
  const uint16_t* qb = a.q.p + (size_t)rq.first * a.q.ts + head * a.q.hs;
  const uint16_t* gb = b.d_out.p + (size_t)rq.first * b.d_out.ts + head * b.d_out.hs;
  const uint32_t lbase = lds_addr(lds);
  float stat = 0.f;                            // of the tile's query t: lse, or delta
  auto copy = [&](int n, int buf) {
    copy_tiles<DP>(qb, a.q.ts, gb, b.d_out.ts, q_lo + n * kBT, q_hi - 1, a.dim, lbase + buf * 2 * kTile, wave, lane);
    if (t < 2 * kBT) {
      const size_t i = rq.first + min(q_lo + n * kBT + t % kBT, q_hi - 1);
      stat = t < kBT ? lse2_of(a.lse[i * a.lse_ts + head * a.lse_hs]) : delta[(size_t)head * a.rows_q + i];
    }
  };
  f32x16 dk[DT], dv[DT];
  clear(dk);
  clear(dv);
  if (nt > 0) copy(0, 0);
  for (int n = 0; n < nt; ++n) {
    const int buf = n & 1;
    wait_copies();
    if (t < 2 * kBT) lrow[buf][t / kBT][t % kBT] = stat;
    __syncthreads();
    if (n + 1 < nt) copy(n + 1, buf ^ 1);
    const int i0 = q_lo + n * kBT, p0 = shift + i0, pn = shift + min(i0 + kBT, q_hi) - 1;
    const int wfar = window_start(p0, a.window);   // first key that a query of the tile has in its window
    if (w0 > klast || w0 > pn || (w0 + 31 < wfar && w0 >= (int)a.sinks)) continue;
    const bool whole = i0 + kBT <= q_hi && w0 + 31 <= p0 && w0 + 31 <= klast &&
                       (w0 >= window_start(pn, a.window) || w0 + 31 < (int)a.sinks);
    const char* tq = lds + buf * 2 * kTile;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f32x16 s = times_rows<DP>(tq, 32 * x, col, hh, k);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 l = *reinterpret_cast<const f32x4*>(&lrow[buf][0][32 * x + 8 * g + 4 * hh]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * g + e] = exp2_fast(__builtin_fmaf(s[4 * g + e], c, -l[e]));
      }
      uint32_t seen = 0xFFFFu;
      if (!whole) {
        seen = 0;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int i = i0 + 32 * x + 8 * (r / 4) + 4 * hh + r % 4, p = shift + i;
          if (i < q_hi && key <= p && key <= klast && (key >= window_start(p, a.window) || sinks)) seen |= 1u << r;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = seen >> r & 1 ? s[r] : 0.f;
      }
      add_columns<DP>(dv, lbase + buf * 2 * kTile + kTile, 32 * x, lane, s);
      const f32x16 d = times_rows<DP>(tq + kTile, 32 * x, col, hh, v);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 l = *reinterpret_cast<const f32x4*>(&lrow[buf][1][32 * x + 8 * g + 4 * hh]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * g + e] *= d[4 * g + e] - l[e];
      }
      if (!whole) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = seen >> r & 1 ? s[r] : 0.f;
      }
      add_columns<DP>(dk, lbase + buf * 2 * kTile, 32 * x, lane, s);
    }
  }
  if (key > klast) return;
  if constexpr (FAR) {
    const size_t slot = ((size_t)tile.at * sums.sink_tiles + j0 / kRowsB) * a.hq + head;
    float* o = sums.far + (slot * 2 * kRowsB + wave * 32 + col) * a.dim;
    store_row(o, dk, hh, a.dim);
    store_row(o + (size_t)kRowsB * a.dim, dv, hh, a.dim);
  } else if (sums.near) {
    float* o = sums.near + ((size_t)head * a.rows_k + at) * a.dim;
    store_row(o, dk, hh, a.dim);
    store_row(o + (size_t)a.hq * a.rows_k * a.dim, dv, hh, a.dim);
  } else {
    store_row(b.dk.p + at * b.dk.ts + kvh * b.dk.hs, dk, a.scale, hh, a.dim);
    store_row(b.dv.p + at * b.dv.ts + kvh * b.dv.hs, dv, 1.0f, hh, a.dim);
  }
}

// Joins the sums of a key's query heads and runs: a workgroup takes 64 rows of
// one key head, dK then dV.
__global__ __launch_bounds__(256) void k_attn_join(AttnBwdArgs b, KeySums sums) {
  const AttnArgs& a = b.f;
  const unsigned kvh = blockIdx.x % a.hkv, rank = blockIdx.x / a.hkv, group = a.hq / a.hkv;
  Tile tile;
  if (!find_tile(a.cu_k, a.seqs, a.rows_k, 64, rank, &tile)) return;
  const Rows rq = rows_of(a.cu_q, tile.seq, a.rows_q), rk = rows_of(a.cu_k, tile.seq, a.rows_k);
  const int j0 = (int)(tile.row / kRowsB * kRowsB);   // of the rows' tile of keys
  // runs of the sequence: numbers first .. first + runs - 1, queries from (1 + i) kFar on
  unsigned first = 0, runs = 0;
  Band band{0, 0};
  if (sums.sink_tiles && j0 < (int)a.sinks && (unsigned)(j0 / kRowsB) < sums.sink_tiles && rq.count > kFar) {
    runs = (rq.count - 1) / kFar;
    for (unsigned s0 = 0; s0 < tile.seq; s0 += kWave) {
      const unsigned s = s0 + lane_id(), n = s < tile.seq ? rows_of(a.cu_q, s, a.rows_q).count : 0;
      first += __shfl(wave_scan(n ? (n - 1) / kFar : 0), kWave - 1);
    }
    band = band_of(a, j0, (int)rk.count - (int)rq.count, (int)rq.count);
  }
  const unsigned per = a.dim / 4;              // groups of 4 columns
  const unsigned rows = min(64u, rk.count - tile.row);
  for (unsigned i = threadIdx.x; i < rows * per; i += 256) {
    const unsigned r = i / per, d = i % per * 4;
    const size_t at = rk.first + tile.row + r;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      const float* near = sums.near + (size_t)which * a.hq * a.rows_k * a.dim + at * a.dim + d;
#pragma unroll 4
      for (unsigned h = 0; h < group; ++h)
        sum += *reinterpret_cast<const f32x4*>(near + (size_t)(kvh * group + h) * a.rows_k * a.dim);
      for (unsigned n = 0; n < runs && first + n < sums.runs; ++n) {
        if ((int)min((n + 2) * kFar, rq.count) <= band.hi) continue;   // all of the run's queries were near
        const size_t slot = ((size_t)(first + n) * sums.sink_tiles + j0 / kRowsB) * a.hq + kvh * group;
        const float* far = sums.far + ((slot * 2 + which) * kRowsB + tile.row - j0 + r) * a.dim + d;
        for (unsigned h = 0; h < group; ++h) sum += *reinterpret_cast<const f32x4*>(far + (size_t)h * 2 * kRowsB * a.dim);
      }
      const float f = which ? 1.0f : a.scale;
      const HeadOut& o = which ? b.dv : b.dk;
      *reinterpret_cast<u32x2*>(o.p + at * o.ts + kvh * o.hs + d) =
          u32x2{result_bf16x2(sum[0] * f, sum[1] * f), result_bf16x2(sum[2] * f, sum[3] * f)};
    }
  }
}

struct Room {
  size_t delta, near, far;     // binary32 values
  unsigned sink_tiles, runs;
};
Room room_of(size_t rows_q, size_t rows_k, size_t hq, size_t hkv, size_t dim, size_t window, size_t sinks) {
  Room r{};
  r.delta = cdiv(rows_q * hq, 64) * 64;
  if (window < rows_k && sinks) {
    r.sink_tiles = (unsigned)cdiv(sinks < rows_k ? sinks : rows_k, kRowsB);
    r.runs = (unsigned)(rows_q / kFar);
    if (r.runs == 0) r.sink_tiles = 0;
  }
  if (hq > hkv || r.sink_tiles) r.near = 2 * hq * rows_k * dim;
  r.far = (size_t)r.runs * r.sink_tiles * hq * 2 * kRowsB * dim;
  return r;
}

template <int DP>
hipError_t launch(const Launch& L, const AttnBwdArgs& b) {
  const AttnArgs& a = b.f;
  const Room room = room_of(a.rows_q, a.rows_k, a.hq, a.hkv, a.dim, a.window, a.sinks);
  float* delta = static_cast<float*>(b.workspace);
  hipError_t e;
  if (a.rows_q) {
    e = launch_k(k_attn_delta, dim3((unsigned)cdiv((size_t)a.rows_q * a.hq, 16)), dim3(256), 0, L.stream, b.out, b.d_out, delta,
                 a.rows_q, a.hq, a.dim);
    if (e != hipSuccess) return e;
    if (b.dq.p) {
      const unsigned tiles = a.rows_q / kRowsB + a.seqs;
      e = launch_k(k_attn_dq<DP>, dim3(tiles * a.hq), dim3(kWavesB * 64), 0, L.stream, b, delta);
      if (e != hipSuccess) return e;
    }
  }
  if (!b.dk.p || a.rows_k == 0) return hipSuccess;
  const KeySums sums{room.near ? delta + room.delta : nullptr, room.far ? delta + room.delta + room.near : nullptr,
                     room.sink_tiles, room.runs};
  if (room.far) {
    e = launch_k(k_attn_dkv<DP, true>, dim3(room.runs * room.sink_tiles * a.hq), dim3(kWavesB * 64), 0, L.stream, b, delta, sums);
    if (e != hipSuccess) return e;
  }
  e = launch_k(k_attn_dkv<DP, false>, dim3((a.rows_k / kRowsB + a.seqs) * a.hq), dim3(kWavesB * 64), 0, L.stream, b, delta, sums);
  if (e != hipSuccess || !sums.near) return e;
  return launch_k(k_attn_join, dim3((a.rows_k / 64 + a.seqs) * a.hkv), dim3(256), 0, L.stream, b, sums);
}

}  // namespace

size_t attn_bwd_workspace(size_t rows_q, size_t rows_k, size_t seqs, size_t hq, size_t hkv, size_t dim, size_t window,
                          size_t sinks) {
  const Room r = room_of(rows_q, rows_k, hq, hkv, dim, window, sinks);
  return (r.delta + r.near + r.far) * sizeof(float);
}

hipError_t launch_attn_bwd(const Launch& L, const AttnBwdArgs& b) {
  return b.f.dim > 64 ? launch<128>(L, b) : launch<64>(L, b);
}

}  // namespace ar
