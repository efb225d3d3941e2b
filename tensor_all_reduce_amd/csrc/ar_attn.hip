// Attention of ragged prompts: for the query at position p of its sequence
//   out = sum over visible keys j of softmax_j(scale q . k_j) v_j
// with key j visible if j <= p and (j > p - window or j < sinks).
//
// One pass over the keys with the running maximum and sum of the softmax.  A
// wave has 32 queries, whose scores of 64 keys at a time (S^T = K Q^T) are
// two 32 x 32 products; the workgroup's waves share the keys' and values'
// tiles in LDS, copied there past the registers one tile ahead.  Scores,
// maxima, sums and results are binary32; the softmax's numerators become bf16
// for their product with the values, up to 2^-8 of each, which is what the
// rounding of the values' own sum to bf16 costs once more.
//
// Bound by the matrix cores and, beside them, the softmax's arithmetic: of a
// tile of 64 keys a wave has 32 products of 32 cycles and about 240 vector
// instructions of 4, of which two waves a SIMD overlap a part.  Operands are
// read from LDS four products ahead, in a fixed order, so that nothing is
// spilled: a reload would wait for the copies under way, which share its
// counter.  16384 tokens, 64 heads of 128 on 8, causal: 4060 to 4350 us, 1.01 to
// 1.08 PFLOP/s (order left to the compiler 4932, one spilled register in the loop
// 4700; a third tile of LDS, wave priorities and 128 queries a workgroup within
// 4%); over E4M3 pages 5040, 0.87 PFLOP/s.
#include "ar_attn.hpp"

namespace ar {
namespace {

constexpr int kBN = 64;  // keys of a tile

// NW waves; KG 2: two halves of them have the same queries and every other tile
// of keys each, in LDS of their own, and are joined at the end.
template <int DP, int NW, int KG, KeySource SRC>
__global__ __launch_bounds__(NW * 64, 2) void k_attn(AttnArgs a) {
  constexpr int NQ = NW / KG, BM = NQ * 32, KS = DP / 16, DT = DP / 32;
  constexpr uint32_t kTile = kBN * DP * 2;     // bytes of a tile of keys, or of values
  __shared__ __align__(1024) char all_lds[KG * 4 * kTile];   // keys, values; keys, values
  __shared__ __align__(16) float all_scales[SRC == kKeyPagesE4M3 ? KG * 4 * kBN : 4];  // their scales
  __shared__ int lflag;
  const int lane = lane_id(), part = KG == 1 ? 0 : uniform(threadIdx.x / (NQ * kWave));   // the wave's half
  const int t = threadIdx.x - part * NQ * kWave, wave = uniform(t / kWave);               // in its half
  const int col = lane & 31, hh = lane >> 5;
  char* const lds = all_lds + part * 4 * kTile;
  float* const lscale = all_scales + (SRC == kKeyPagesE4M3 ? part * 4 * kBN : 0);

  // queries of one tile and, if there are eight heads of keys, those that
  // share keys on one XCD
  const unsigned rank = blockIdx.x / a.hq, hi = blockIdx.x % a.hq;
  const unsigned kvh = hi % a.hkv, head = kvh * (a.hq / a.hkv) + hi / a.hkv;
  Tile tile;
  if (!find_tile<true>(a.cu_q, a.seqs, a.rows_q, BM, rank, &tile)) return;
  const Rows rq = rows_at(a.cu_q, tile.seq, a.rows_q);
  unsigned nk, k_first = 0;
  if constexpr (SRC == kKeyRows) {
    const Rows rk = rows_at(a.cu_k, tile.seq, a.rows_k);
    nk = rk.count;
    k_first = rk.first;
  } else {
    nk = (unsigned)uniform((int)min((unsigned)max(a.lens[tile.seq], 0), a.capacity));
  }
  const int shift = (int)nk - (int)rq.count;   // position of the sequence's first query
  const int last = (int)rq.count - 1;
  const int p0 = shift + (int)tile.row, p1 = shift + min((int)tile.row + BM - 1, last);
  const KeyRange keys = key_range(p0, p1, a.window, a.sinks, kBN);
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
    for (uint32_t o = t * 16; o < 4 * kTile; o += NQ * 64 * 16) *reinterpret_cast<u32x4*>(lds + o) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }

  unsigned bad = 0;                            // a page number out of range was met
  const TileCopy<DP, NQ> copy_rows(a.k.ts, a.v.ts, a.dim, wave, lane);
  const uint16_t *kb = a.k.p + (size_t)k_first * a.k.ts + kvh * a.k.hs, *vb = a.v.p + (size_t)k_first * a.v.ts + kvh * a.v.hs;
  // Pages: the numbers of a tile's pages are read one tile before its keys.
  constexpr int ALL = kBN * DP / 16, CHUNKS = SRC == kKeyPagesE4M3 ? (ALL + NQ * 64 - 1) / (NQ * 64) : 1;  // of 16 codes
  constexpr int IDS = SRC == kKeyPagesE4M3 ? CHUNKS + 1 : copy_rows.COPIES;
  unsigned ids[IDS];
  auto id_row = [&](int i) {                   // the tile's row that number i is for
    if constexpr (SRC == kKeyPagesE4M3) return i < CHUNKS ? (i * NQ * 64 + t) / (DP / 16) : t % kBN;
    else return i * NQ * copy_rows.RPC + copy_rows.row;
  };
  auto look_up = [&](int n) {
    if constexpr (SRC != kKeyRows) {
      const KeyStep k = key_step(keys, n, kBN);
#pragma unroll
      for (int i = 0; i < IDS; ++i)
        ids[i] = (unsigned)a.table[tile.seq * a.table_ld + page_of((unsigned)min(k.j0 + id_row(i), k.end - 1), a.cache)];
    }
  };
  // Element of row r's token: in page `id` for strides ps of pages, ts of tokens.
  auto token = [&](const KeyStep& k, int r, unsigned id, size_t ps, size_t ts) {
    const unsigned j = (unsigned)min(k.j0 + r, k.end - 1), in = j - page_of(j, a.cache) * a.cache.size;
    if (id >= a.cache.pages) {
      bad = 1;
      id = 0;
    }
    return (size_t)id * ps + (size_t)in * ts;
  };
  auto copy = [&](int n, int buf) {
    const KeyStep k = key_step(keys, n, kBN);
    const uint32_t to = lbase + buf * 2 * kTile;
    if constexpr (SRC == kKeyRows) {
      copy_rows(kb, a.k.ts, vb, a.v.ts, k.j0, k.end - 1, to);
    } else {
#pragma unroll
      for (int i = 0; i < copy_rows.COPIES; ++i) {
        const int r = i * NQ * copy_rows.RPC + copy_rows.row;
        const size_t at = token(k, r, ids[SRC == kKeyPages ? i : 0], a.cache.page, a.cache.ts) + kvh * a.cache.hs;
        if (copy_rows.on) {
          const uint32_t here = to + (i * NQ + wave) * 1024;
          copy16_to_lds(reinterpret_cast<const char*>(static_cast<const uint16_t*>(a.cache.k) + at) + copy_rows.chunk, here);
          copy16_to_lds(reinterpret_cast<const char*>(static_cast<const uint16_t*>(a.cache.v) + at) + copy_rows.chunk, here + kTile);
        }
      }
    }
  };
  // E4M3: codes through registers, which are the same values in bf16
  u32x4 ck[CHUNKS], cv[CHUNKS];
  float cs = 0.f;
  auto fetch = [&](int n) {
    const KeyStep k = key_step(keys, n, kBN);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int at = i * NQ * 64 + t, r = at / (DP / 16), ch = at % (DP / 16);
      const size_t o = token(k, r, ids[SRC == kKeyPagesE4M3 ? i : 0], a.cache.page, a.cache.ts) + kvh * a.cache.hs + ch * 16;
      ck[i] = cv[i] = u32x4{0, 0, 0, 0};
      if (at < ALL && ch * 16 < (int)a.dim) {
        ck[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.cache.k) + o);
        cv[i] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.cache.v) + o);
      }
    }
    if (t < 2 * kBN)
      cs = (t < kBN ? a.cache.k_scales : a.cache.v_scales)[token(k, t % kBN, ids[IDS - 1], a.cache.spage, a.cache.sts) + kvh * a.cache.shs];
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int at = i * NQ * 64 + t, r = at / (DP / 16), ch = at % (DP / 16);
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

  f32x16 o[DT];
  float m, l;
  // Values that are no numbers under masked scores: such a score counts 0,
  // but 0 times them is NaN.  So where a result is no number the pass is made
  // again with such values as 0 (CARE 1), and then once more, without products,
  // to add them where they are visible (CARE 2): no weight makes them 0 any
  // more.  So too where a page number out of range was met: the queries that
  // see a key of that page have a sum that is no number.  And where a sum is
  // beyond binary32: numerators are up to 2^8, and as many as there are keys,
  // so that large values' sums can be though their mean is not.  With care
  // numerators are so much smaller that nothing is.  (These passes are code of
  // their own: as branches of one loop they cost the ordinary pass 10 to 20
  // registers and 1 to 3%.)
  const int headroom = 10 + 31 - __builtin_clz(nk | 1);   // 2^headroom > 2^8 times the keys, and twice that
  const float down = __uint_as_float((127u - headroom) << 23), up = __uint_as_float((127u + headroom) << 23);
  auto pass = [&](auto mode) __attribute__((always_inline)) {
    constexpr int CARE = decltype(mode)::value;
    if constexpr (CARE < 2) {
      m = AR_NEG_INF;
      l = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] = 0.f;
    }
    if (part < keys.steps) {
      look_up(part);
      if constexpr (SRC == kKeyPagesE4M3) fetch(part);
      else copy(part, 0);
      if (part + KG < keys.steps) look_up(part + KG);
    }
    // (the queries have come: a wait for them in the loop would be one for the
    // tile under way, too)
    if constexpr (SRC == kKeyPagesE4M3) wait_copies();
    for (int i = 0; i * KG < keys.steps; ++i) {
      const int buf = i & 1, n = i * KG + part;
      const bool mine = KG == 1 || n < keys.steps;   // the second half may have one tile less
      if constexpr (SRC == kKeyPagesE4M3) {
        if (mine) put(buf);
      } else {
        wait_copies();
      }
      __syncthreads();
      if (n + KG < keys.steps) {
        if constexpr (SRC == kKeyPagesE4M3) fetch(n + KG);
        else copy(n + KG, buf ^ 1);
        if (n + 2 * KG < keys.steps) look_up(n + 2 * KG);
      }
      const KeyStep k = key_step(keys, n, kBN);
      const int j0 = k.j0;
      // of the tile's keys, less 4 hh, those that the lane's query sees
      const Interval view((k.sinks ? 0 : start) - j0 - 4 * hh, min(p, k.end - 1) - j0 - 4 * hh);
      if constexpr (CARE > 0) {
        char* tv = lds + (buf * 2 + 1) * kTile;
        if constexpr (CARE == 2) {
#pragma unroll 1
          for (int r = 0; r < (mine ? kBN : 0); ++r) {
            const bool sees = view.has(r - 4 * hh);
#pragma unroll
            for (int x = 0; x < DT * 4; ++x) {
              const u32x2 w = *reinterpret_cast<const u32x2*>(tv + chunk_addr<DP>(r, x) + 8 * hh);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float v = e & 1 ? hi_f32(w[e / 2]) : lo_f32(w[e / 2]);
                if (sees && !is_number(v)) o[x / 4][x % 4 * 4 + e] += v;
              }
            }
          }
          continue;
        }
        if constexpr (SRC != kKeyRows) {
          if (mine) {
            const unsigned j = (unsigned)min(j0 + lane, k.end - 1);   // a lane's key
            const uint64_t lost = __ballot((unsigned)a.table[tile.seq * a.table_ld + page_of(j, a.cache)] >= a.cache.pages);
            const int from = max((k.sinks ? 0 : start) - j0, 0), to = min(min(p, k.end - 1) - j0, kBN - 1);
            if (to >= from && (lost >> from) << from << (kBN - 1 - to)) l = __uint_as_float(0x7FC00000u);
          }
        }
        for (uint32_t at = t * 4; at < (mine ? kTile : 0); at += NQ * 64 * 4) {
          uint32_t& w = *reinterpret_cast<uint32_t*>(tv + at);
          w = numbers_only(w);
        }
        __syncthreads();
      }
      // no key of the tile is visible to the wave's queries
      if (!mine || (int)tile.row + wave * 32 > last || j0 > wp1 || (!k.sinks && j0 + kBN <= wstart0)) continue;
      const bool whole = j0 + kBN - 1 <= min(wp0, k.end - 1) && (k.sinks || j0 >= wstart1);
      const LaneAddr<DP> from(lbase + buf * 2 * kTile, lane);
      // register r of block b: key 32 b + 8 (r / 4) + 4 hh + r % 4
      auto seen = [&](int b, int r) { return view.has(32 * b + 8 * (r / 4) + r % 4); };
      auto scales = [&](int x, int b, f32x16& f) {   // E4M3: of keys (x 0), of values (x 1)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(&lscale[(buf * 2 + x) * kBN + 32 * b + 8 * g + 4 * hh]);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[4 * g + e] = v[e];
        }
      };
      auto tile_step = [&](auto masked) {
        constexpr bool MASK = decltype(masked)::value;
        constexpr int AHEAD = 4, ALL = 2 * KS + 4 * DT;
        // products 0 .. 2 KS - 1: scores of 32 keys, then of 32 more; then
        // values of 16 keys each, DT at a time
        Frag8 f[AHEAD], pf[4];
        f32x16 s[2];
        auto load = [&](auto ii) {
          constexpr int i = decltype(ii)::value;
          if constexpr (i < 2 * KS) f[i % AHEAD].u = from.rows(i / KS * 32, i % KS);
          else f[i % AHEAD] = from.columns(kBN + (i - 2 * KS) / DT * 16, (i - 2 * KS) % DT);
        };
        auto fit = [&](int b) {                // scales and mask of a block of scores
          if constexpr (SRC == kKeyPagesE4M3) {
            f32x16 f;
            scales(0, b, f);
            s[b] *= f;
          }
          if constexpr (MASK) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[b][r] = seen(b, r) ? s[b][r] : AR_NEG_INF;
          }
        };
        auto largest = [&](int b, float top) {
#pragma unroll
          for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
          return top;
        };
        steps<AHEAD>(load);
        float top = AR_NEG_INF;
        steps<2 * KS>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          s[i / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % AHEAD].b, q[i % KS].b, i % KS ? s[i / KS] : f32x16{}, 0, 0, 0);
          load(SPc<i + AHEAD>{});
          if constexpr (i == KS + KS / 2) {
            fit(0);
            top = largest(0, top);
          }
          keep_order();
        });
        fit(1);
        top = largest(1, top);
        top = fmaxf(top, __shfl_xor(top, 32)) * c;
        // the running maximum follows only where it falls behind by 2^8: sums
        // stay far below binary32's range, and most tiles change nothing
        if (__any(top > m + 8.0f)) {
          const float up = fmaxf(m, top), f = m == AR_NEG_INF ? 1.0f : exp2_fast(m - up);   // (all is 0 before a first score)
          m = up;
          l *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] *= f;
        }
        const float base = m == AR_NEG_INF ? 0.f : m;
        float more = 0.f;
        auto weigh = [&](int b, int r, int n) {   // numerators of n scores, as bf16
          f32x16 f;
          if constexpr (SRC == kKeyPagesE4M3) scales(1, b, f);
#pragma unroll
          for (int x = r; x < r + n; x += 2) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              w[e] = exp2_fast(__builtin_fmaf(s[b][x + e], c, -base));
              if (e) more += w[e];
              else l += w[e];
              if constexpr (CARE > 0) w[e] *= down;
              if constexpr (SRC == kKeyPagesE4M3) w[e] = !MASK || seen(b, x + e) ? w[e] * f[x + e] : 0.f;
            }
            pf[2 * b + x / 8].w[x % 8 / 2] = cvt_bf16x2(w[0], w[1]);
          }
        };
        weigh(0, 0, 16);
        if constexpr (MASK) weigh(1, 0, 16);
        steps<4 * DT>([&](auto ii) {
          constexpr int n = decltype(ii)::value, i = n + 2 * KS;
          o[n % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % AHEAD].b, pf[n / DT].b, o[n % DT], 0, 0, 0);
          if constexpr (i + AHEAD < ALL) load(SPc<i + AHEAD>{});
          if constexpr (!MASK && n < 2 * DT) weigh(1, n * 8 / DT, 8 / DT);
          keep_order();
        });
        l += more;
      };
      if (CARE == 0 && whole) tile_step(std::false_type{});
      else tile_step(std::true_type{});
    }
  };
  pass(SPc<0>{});
  float odd = 0.f;                             // a number only if every result is, and below 2^126: halves are added
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd = __builtin_fmaf(o[d][r], 8.0f, odd);
  if (threadIdx.x == 0) lflag = 0;
  __syncthreads();
  if (!is_number(odd) || bad) lflag = 1;
  __syncthreads();
  const bool care = uniform(lflag) != 0;
  if (AR_RARE(care)) {
    pass(SPc<1>{});
    __syncthreads();                           // (no wave reads a tile any more)
  }

  l += __shfl_xor(l, 32);
  // (the tiles are no longer read) the second half's results, a wave's lane by lane
  float* give = reinterpret_cast<float*>(all_lds) + wave * (DT * 16 + 2) * kWave + lane;
  auto hand_over = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) give[(d * 16 + r) * kWave] = o[d][r];
  };
  if constexpr (KG == 2) {
    if (part == 1) {
      hand_over();
      give[DT * 16 * kWave] = m;
      give[(DT * 16 + 1) * kWave] = l;
    }
    __syncthreads();
    if (part == 1 && !care) return;
    const float m2 = give[DT * 16 * kWave], l2 = give[(DT * 16 + 1) * kWave], top = fmaxf(m, m2);
    const float f1 = m == AR_NEG_INF ? 1.0f : exp2_fast(m - top), f2 = m2 == AR_NEG_INF ? 1.0f : exp2_fast(m2 - top);
    m = top;                                   // (all is 0 of a half without scores)
    l = l * f1 + l2 * f2;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = o[d][r] * f1 + give[(d * 16 + r) * kWave] * f2;
  }
  if (AR_RARE(care)) {
    if constexpr (KG == 2) {
      __syncthreads();
      if (part == 1) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = f32x16{};
      }
    }
    pass(SPc<2>{});
    if constexpr (KG == 2) {
      __syncthreads();
      if (part == 1) hand_over();
      __syncthreads();
      if (part == 1) return;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] += give[(d * 16 + r) * kWave];
    }
  }
  if (row > last) return;
  const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;   // no visible key: zeros; NaN stays
  const float f = AR_RARE(care) ? inv * up : inv;
  uint16_t* op = a.out.p + (size_t)(rq.first + row) * a.out.ts + head * a.out.hs;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const unsigned at = 32 * d + 8 * g + 4 * hh;
      if (at < a.dim)
        *reinterpret_cast<u32x2*>(op + at) =
            u32x2{result_bf16x2(o[d][4 * g] * f, o[d][4 * g + 1] * f), result_bf16x2(o[d][4 * g + 2] * f, o[d][4 * g + 3] * f)};
    }
  if (a.lse && hh == 0)
    a.lse[(size_t)(rq.first + row) * a.lse_ts + head * a.lse_hs] =
        inv != inv ? inv : l > 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : AR_NEG_INF;
}

constexpr unsigned tiles_at_most(size_t rows, size_t seqs, unsigned bm) { return (unsigned)(rows / bm + seqs); }

template <int DP, int NW, int KG, KeySource SRC>
hipError_t launch(const Launch& L, const AttnArgs& a) {
  const unsigned tiles = tiles_at_most(a.rows_q, a.seqs, NW / KG * 32);
  return launch_k(k_attn<DP, NW, KG, SRC>, dim3(tiles * a.hq), dim3(NW * 64), 0, L.stream, a);
}

// 256 queries a workgroup where that gives every CU two, else 128, of which
// two share a CU (16384 tokens, 64 heads of 128: 4187 us and 4391; 647 tokens,
// 6 heads of 64: 15.4 and 11.9).  Where most CUs have no second workgroup, one
// of 128 queries has eight waves, half of them on every other tile of keys
// (4096 tokens, 8 heads of 128: 71 us, with four waves 95; 2048 of them behind
// 8192: 172 and 243; 7 sequences of 1 to 700 of them, 16 heads of 64, E4M3: 19
// and 24; but 16 prompts of 256 to 768 of them, 8 heads: 33 and 29; 32 of 128:
// 13.4 and 11.8).  So too where two would share a CU, if prompts are long and
// have no window, since the launch then waits for the last queries' keys (8192
// tokens, 8 heads of 128: 155 and 194; two prompts of 4096: 92 and 130; 10240
// tokens: 253 and 260; but 8 prompts of 1024: 45 and 40; 8192 tokens with a
// window of 4096: 144 and 135).
template <int DP, KeySource SRC>
hipError_t launch_dim(const Launch& L, const AttnArgs& a) {
  const size_t rows = a.rows_q, cus = L.cus;
  const size_t groups = (rows / 128 + a.seqs / 2) * a.hq;   // about: a sequence's last one is half full
  if (rows * a.hq >= 2 * cus * 256) return launch<DP, 8, 1, SRC>(L, a);
  const bool deep = rows >= (size_t)a.seqs * 2048 && (size_t)a.window * a.seqs >= rows;
  return groups * 20 <= cus * (deep ? 45 : 28) ? launch<DP, 8, 2, SRC>(L, a) : launch<DP, 4, 1, SRC>(L, a);
}
template <KeySource SRC>
hipError_t launch_src(const Launch& L, const AttnArgs& a) {
  return a.dim > 64 ? launch_dim<128, SRC>(L, a) : launch_dim<64, SRC>(L, a);
}

}  // namespace

// (512 work items for up to 256 queries, or 256 for up to 128; with 512 for 128
// only where there are few)
bool attn_fits(size_t rows_q, size_t seqs, size_t hq) { return fits_launch(rows_q / 256 + seqs, hq, 512); }

hipError_t launch_attn(const Launch& L, const AttnArgs& a, KeySource src) {
  switch (src) {
    case kKeyRows: return launch_src<kKeyRows>(L, a);
    case kKeyPages: return launch_src<kKeyPages>(L, a);
    default: return launch_src<kKeyPagesE4M3>(L, a);
  }
}

}  // namespace ar
