// Attention of ragged prompts: for the query at position p of its sequence
//   out = sum over visible keys j of softmax_j(scale q . k_j) v_j
// with key j visible if j <= p and (j > p - window or j < sinks).
//
// One pass over the keys with the running maximum and sum of the softmax.  A
// wave has 32 queries, whose scores of 64 keys at a time (S^T = K Q^T) are
// two 32 x 32 products; the workgroup's waves share the keys' and values'
// tiles in LDS, copied there past the registers one tile ahead.  Scores,
// maxima, sums and results are binary32; the softmax's numerators become bf16
// for their product with the values, 2^-9 of each, which is what the rounding
// of the values' own sum to bf16 costs once more.
#include "ar_attn.hpp"

#include <utility>

namespace ar {
namespace {

constexpr int kBN = 64;  // keys of a tile

template <int DP, int NW, KeySource SRC>
__global__ __launch_bounds__(NW * 64, 2) void k_attn(AttnArgs a) {
  constexpr int BM = NW * 32, KS = DP / 16, DT = DP / 32;
  constexpr uint32_t kTile = kBN * DP * 2;     // bytes of a tile of keys, or of values
  __shared__ __align__(1024) char lds[4 * kTile];            // keys, values; keys, values
  __shared__ __align__(16) float lscale[SRC == kKeyPagesE4M3 ? 4 * kBN : 4];  // their scales
  __shared__ int lflag[2];
  const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int col = lane & 31, hh = lane >> 5;

  // queries of one tile and, if there are eight heads of keys, those that
  // share keys on one XCD
  const unsigned rank = blockIdx.x / a.hq, hi = blockIdx.x % a.hq;
  const unsigned kvh = hi % a.hkv, head = kvh * (a.hq / a.hkv) + hi / a.hkv;
  Tile tile;
  if (!find_tile(a.cu_q, a.seqs, a.rows_q, BM, rank, &tile)) return;
  const Rows rq = rows_of(a.cu_q, tile.seq, a.rows_q);
  unsigned nk, k_first = 0;
  if constexpr (SRC == kKeyRows) {
    const Rows rk = rows_of(a.cu_k, tile.seq, a.rows_k);
    nk = rk.count;
    k_first = rk.first;
  } else {
    nk = min((unsigned)max(a.lens[tile.seq], 0), a.capacity);
  }
  const int shift = (int)nk - (int)rq.count;   // position of the sequence's first query
  const int last = (int)rq.count - 1;
  const int p0 = shift + (int)tile.row, p1 = shift + min((int)tile.row + BM - 1, last);
  // keys of the tile: the sinks before its window, then from its window's start
  const int lo = window_start(p0, a.window), sunk = min((int)min(a.sinks, 0x7FFFFFFFu), lo), end = p1 + 1;
  const int ts = (sunk + kBN - 1) / kBN, nt = end > lo ? ts + (end - lo + kBN - 1) / kBN : 0;
  // this lane's query, and the wave's
  const int row = (int)tile.row + wave * 32 + col, p = shift + min(row, last), start = window_start(p, a.window);
  const int wp0 = shift + min((int)tile.row + wave * 32, last), wp1 = shift + min((int)tile.row + wave * 32 + 31, last);
  const int wstart0 = window_start(wp0, a.window), wstart1 = window_start(wp1, a.window);

  Frag8 q[KS];
  {
    const uint16_t* qp = a.q.p + (size_t)(rq.first + min(row, last)) * a.q.ts + head * a.q.hs;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const unsigned d = 16 * s + 8 * hh;
      q[s].u = d < a.dim ? *reinterpret_cast<const u32x4*>(qp + d) : u32x4{0, 0, 0, 0};
    }
  }
  const float c = a.scale * kLog2e;
  const uint32_t lbase = lds_addr(lds);

  if (a.dim < DP) {   // places that no copy fills
    for (uint32_t o = t * 16; o < 4 * kTile; o += NW * 64 * 16) *reinterpret_cast<u32x4*>(lds + o) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }

  // the tile's rows that this lane copies: a wave copies 1 KiB at a time
  constexpr int RPC = 1024 / (DP * 2), COPIES = kBN / RPC / NW, CPR = DP / 8;
  const int crow = lane / CPR;
  unsigned bad = 0;                            // a page number out of range was met
  auto key_at = [&](int n) {                   // first key and number of keys of tile n
    return n < ts ? std::pair<int, int>{n * kBN, sunk} : std::pair<int, int>{lo + (n - ts) * kBN, end};
  };
  auto page_base = [&](int j, unsigned& in) {  // page of key j, its place in the page
    const unsigned pg = page_of((unsigned)j, a.cache);
    in = (unsigned)j - pg * a.cache.size;
    unsigned id = (unsigned)a.table[tile.seq * a.table_ld + pg];
    if (id >= a.cache.pages) {
      bad = 1;
      id = 0;
    }
    return id;
  };
  auto copy = [&](int n, int buf) {
    const std::pair<int, int> k = key_at(n);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int r = (i * NW + wave) * RPC + crow;
      const int j = min(k.first + r, k.second - 1);
      const int ch = (lane % CPR) ^ swizzle<DP>(r);
      const uint16_t *kp, *vp;
      if constexpr (SRC == kKeyRows) {
        kp = a.k.p + (size_t)(k_first + j) * a.k.ts + kvh * a.k.hs;
        vp = a.v.p + (size_t)(k_first + j) * a.v.ts + kvh * a.v.hs;
      } else {
        unsigned in;
        const size_t at = (size_t)page_base(j, in) * a.cache.page + (size_t)in * a.cache.ts + kvh * a.cache.hs;
        kp = static_cast<const uint16_t*>(a.cache.k) + at;
        vp = static_cast<const uint16_t*>(a.cache.v) + at;
      }
      const uint32_t to = lbase + buf * 2 * kTile + (i * NW + wave) * 1024;
      if (ch * 8 < (int)a.dim) {
        copy16_to_lds(kp + ch * 8, __builtin_amdgcn_readfirstlane((int)to));
        copy16_to_lds(vp + ch * 8, __builtin_amdgcn_readfirstlane((int)(to + kTile)));
      }
    }
  };
  // E4M3: codes through registers, which are the same values in bf16
  constexpr int ALL = kBN * DP / 16, CHUNKS = SRC == kKeyPagesE4M3 ? (ALL + NW * 64 - 1) / (NW * 64) : 1;  // of 16 codes
  u32x4 ck[CHUNKS], cv[CHUNKS];
  float cs = 0.f;
  auto fetch = [&](int n) {
    const std::pair<int, int> k = key_at(n);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int at = i * NW * 64 + t, r = at / (DP / 16), ch = at % (DP / 16);
      unsigned in;
      const size_t pg = page_base(min(k.first + r, k.second - 1), in);
      const size_t o = pg * a.cache.page + (size_t)in * a.cache.ts + kvh * a.cache.hs + ch * 16;
      ck[i] = cv[i] = u32x4{0, 0, 0, 0};
      if (at < ALL && ch * 16 < (int)a.dim) {
        ck[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.cache.k) + o);
        cv[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.cache.v) + o);
      }
    }
    if (t < 2 * kBN) {
      unsigned in;
      const size_t pg = page_base(min(k.first + t % kBN, k.second - 1), in);
      cs = (t < kBN ? a.cache.k_scales : a.cache.v_scales)[pg * a.cache.spage + (size_t)in * a.cache.sts + kvh * a.cache.shs];
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int at = i * NW * 64 + t, r = at / (DP / 16), ch = at % (DP / 16);
      if (at >= ALL) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const u32x4 w = x ? cv[i] : ck[i];
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          union { b16x2 b; uint32_t u; } l, h;
          l.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[e], 1.0f, false);
          h.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[e], 1.0f, true);
          o[2 * e] = l.u;
          o[2 * e + 1] = h.u;
        }
        char* to = lds + (buf * 2 + x) * kTile;
        *reinterpret_cast<u32x4*>(to + chunk_addr<DP>(r, 2 * ch)) = u32x4{o[0], o[1], o[2], o[3]};
        *reinterpret_cast<u32x4*>(to + chunk_addr<DP>(r, 2 * ch + 1)) = u32x4{o[4], o[5], o[6], o[7]};
      }
    }
    if (t < 2 * kBN) lscale[buf * 2 * kBN + t] = cs;
  };

  // addresses in a tile: of this lane's chunks of keys, and of the 8-byte
  // pieces that the transposing reads of values take
  const uint32_t va = (uint32_t)(4 * hh + (lane & 15) / 4);       // row, of 16 s + ...
  const int vch = 2 * ((lane >> 4) & 1) + (lane & 3) / 2;         // chunk, of 4 dt + ...
  const uint32_t vhalf = (lane & 1) * 8;

  f32x16 o[DT];
  float m, l;
  // Values that are no numbers under masked scores: such a score counts 0,
  // but 0 times them is NaN.  So where a result is no number the pass is made
  // again with care: tiles with masked scores put 0 for such values and add
  // them where they are visible.
  bool care = false;
  for (;;) {
    m = AR_NEG_INF;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = 0.f;
    if (nt > 0) {
      if constexpr (SRC == kKeyPagesE4M3) fetch(0);
      else copy(0, 0);
    }
    for (int n = 0; n < nt; ++n) {
      const int buf = n & 1;
      if constexpr (SRC == kKeyPagesE4M3) put(buf);
      else wait_copies();
      __syncthreads();
      if (n + 1 < nt) {
        if constexpr (SRC == kKeyPagesE4M3) fetch(n + 1);
        else copy(n + 1, buf ^ 1);
      }
      const std::pair<int, int> kr = key_at(n);
      const int j0 = kr.first, jend = kr.second;
      // no key of the tile is visible to the wave's queries
      if ((int)tile.row + wave * 32 > last || j0 > wp1 || (j0 + kBN <= wstart0 && j0 >= (int)a.sinks)) continue;
      const bool whole = j0 + kBN <= jend && j0 + kBN - 1 <= wp0 && j0 >= wstart1;
      const char* tk = lds + buf * 2 * kTile;
      const uint32_t tv = lbase + buf * 2 * kTile + kTile;

      f32x16 s[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          Frag8 k;
          k.u = *reinterpret_cast<const u32x4*>(tk + chunk_addr<DP>(32 * b + col, 2 * x + hh));
          s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, q[x].b, s[b], 0, 0, 0);
        }
      }
      // register r of block b is key 32 b + 8 (r / 4) + 4 hh + r % 4 of the tile
      if constexpr (SRC == kKeyPagesE4M3) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&lscale[buf * 2 * kBN + 32 * b + 8 * g + 4 * hh]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][4 * g + e] *= f[e];
          }
      }
      auto seen = [&](int b, int r) {
        const int j = j0 + 32 * b + 8 * (r / 4) + 4 * hh + r % 4;
        return j <= p && j < jend && (j >= start || j < (int)a.sinks);
      };
      if (!whole) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[b][r] = seen(b, r) ? s[b][r] : AR_NEG_INF;
      }
      float top = AR_NEG_INF;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
      top = max_halves(top) * c;
      // the running maximum follows only where it falls behind by 2^8: sums
      // stay far below binary32's range, and most tiles change nothing
      if (__any(top > m + 8.0f)) {
        const float up = fmaxf(m, top), f = up == AR_NEG_INF ? 1.0f : exp2_fast(m - up);
        m = up;
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] *= f;
      }
      const float base = m == AR_NEG_INF ? 0.f : m;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[b][r] = exp2_fast(__builtin_fmaf(s[b][r], c, -base));
          l += s[b][r];
        }
      if constexpr (SRC == kKeyPagesE4M3) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&lscale[buf * 2 * kBN + kBN + 32 * b + 8 * g + 4 * hh]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][4 * g + e] = whole || seen(b, 4 * g + e) ? s[b][4 * g + e] * f[e] : 0.f;
          }
      }
      auto values = [&](int b, int x, int d) {   // of 16 keys, 32 columns
        Frag8 v;
        const int r0 = 32 * b + 16 * x + (int)va;
        v.s[0] = read_tr16(tv + chunk_addr<DP>(r0, 4 * d + vch) + vhalf);
        v.s[1] = read_tr16(tv + chunk_addr<DP>(r0 + 8, 4 * d + vch) + vhalf);
        return v;
      };
      const bool sift = care && !whole;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag8 pf;
#pragma unroll
          for (int e = 0; e < 4; ++e) pf.w[e] = cvt_bf16x2(s[b][8 * x + 2 * e], s[b][8 * x + 2 * e + 1]);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            Frag8 v = values(b, x, d);
            if (sift) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((v.w[e] & 0x7F80u) == 0x7F80u) v.w[e] &= 0xFFFF0000u;
                if ((v.w[e] & 0x7F800000u) == 0x7F800000u) v.w[e] &= 0xFFFFu;
              }
            }
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, pf.b, o[d], 0, 0, 0);
          }
        }
      if (sift) {
        // infinities and NaN of the tile: how many of a kind each query sees
        for (int kind = 0; kind < 3; ++kind) {
          const uint32_t like = kind == 0 ? 0x7F80u : kind == 1 ? 0xFF80u : 0u;
          const float add = kind == 0 ? __builtin_huge_valf() : kind == 1 ? AR_NEG_INF : __uint_as_float(0x7FC00000u);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            f32x16 count;
#pragma unroll
            for (int r = 0; r < 16; ++r) count[r] = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                Frag8 v = values(b, x, d), pf;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t is = 0;
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    const uint32_t w = (v.w[e] >> (16 * z)) & 0xFFFFu;
                    const bool hit = kind < 2 ? w == like : (w & 0x7FFFu) > 0x7F80u;
                    is |= hit ? 0x3F80u << (16 * z) : 0u;
                  }
                  v.w[e] = is;
                  pf.w[e] = (seen(b, 8 * x + 2 * e) ? 0x3F80u : 0u) | (seen(b, 8 * x + 2 * e + 1) ? 0x3F800000u : 0u);
                }
                count = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, pf.b, count, 0, 0, 0);
              }
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (count[r] > 0.f) o[d][r] += add;
          }
        }
      }
    }
    float odd = 0.f;   // NaN if any result is no number
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) odd = __builtin_fmaf(o[d][r], 0.f, odd);
    if (t == 0) lflag[0] = lflag[1] = 0;
    __syncthreads();
    if (odd != 0.f) lflag[0] = 1;              // true of NaN
    if (bad) lflag[1] = 1;
    __syncthreads();
    if (care || lflag[0] == 0) break;
    care = true;
  }

  l = add_halves(l);
  if (row > last) return;
  float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;   // no visible key: zeros; NaN stays
  if (SRC != kKeyRows && lflag[1]) inv = __uint_as_float(0x7FC00000u);
  uint16_t* op = a.out.p + (size_t)(rq.first + row) * a.out.ts + head * a.out.hs;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const unsigned at = 32 * d + 8 * g + 4 * hh;
      if (at < a.dim)
        *reinterpret_cast<u32x2*>(op + at) =
            u32x2{result_bf16x2(o[d][4 * g] * inv, o[d][4 * g + 1] * inv), result_bf16x2(o[d][4 * g + 2] * inv, o[d][4 * g + 3] * inv)};
    }
  if (a.lse && hh == 0)
    a.lse[(size_t)(rq.first + row) * a.lse_ts + head * a.lse_hs] =
        inv != inv ? inv : l > 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : AR_NEG_INF;
}

constexpr unsigned tiles_at_most(size_t rows, size_t seqs, unsigned bm) { return (unsigned)(rows / bm + seqs); }

template <int DP, int NW, KeySource SRC>
hipError_t launch(const Launch& L, const AttnArgs& a) {
  const unsigned tiles = tiles_at_most(a.rows_q, a.seqs, NW * 32);
  return launch_k(k_attn<DP, NW, SRC>, dim3(tiles * a.hq), dim3(NW * 64), 0, L.stream, a);
}

template <KeySource SRC>
hipError_t launch_src(const Launch& L, const AttnArgs& a) {
  return a.dim > 64 ? launch<128, 8, SRC>(L, a) : launch<64, 8, SRC>(L, a);
}

}  // namespace

bool attn_fits(size_t rows_q, size_t seqs, size_t hq) { return (rows_q / 128 + seqs) <= 0x7FFFFFFFu / hq; }

hipError_t launch_attn(const Launch& L, const AttnArgs& a, KeySource src) {
  switch (src) {
    case kKeyRows: return launch_src<kKeyRows>(L, a);
    case kKeyPages: return launch_src<kKeyPages>(L, a);
    default: return launch_src<kKeyPagesE4M3>(L, a);
  }
}

}  // namespace ar
