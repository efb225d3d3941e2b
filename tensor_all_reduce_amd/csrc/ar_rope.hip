// Rotation of queries and keys by their positions, and the append of keys and
// values to a paged cache.
//   u = a c - b s,  w = b c + a s
// for the pairs (a, b) of a head's first `rot` values, a and b `rot` / 2
// apart or neighbours, with the cosine and sine of the token's position; the
// gradient is the rotation back (s negated).
//
// Bound by memory.  A lane takes 16 values of a head: 8 pairs as two groups
// of 8, so that every access is 16 bytes wide and both values of a pair are
// in one lane; the lanes of a head lie side by side, and a head's largest
// magnitude (E4M3) is found by exchanges between them.
#include "ar_attn.hpp"
#include "ar_e4m3.hpp"

namespace ar {
namespace {

__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_f32(v[i]);
    f[2 * i + 1] = hi_f32(v[i]);
  }
}
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = result_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}

// 2^lg lanes a head, 256 >> lg heads a workgroup: of a token's queries, keys,
// then values, token after token.  NT: past the caches, of what is too much
// for them.
template <bool E4M3, bool PAIRS, bool NT>
__global__ __launch_bounds__(256) void k_rope_kv(RopeArgs a, int lg, unsigned heads) {
  const unsigned lanes = 1u << lg, i = threadIdx.x & (lanes - 1);
  const unsigned work = blockIdx.x * (256 >> lg) + (threadIdx.x >> lg);   // (token, head)
  const unsigned token = work / heads, head = work - token * heads;
  const bool on = token < a.tokens && i < a.dim / 16;
  const bool is_q = head < a.hq, is_v = head >= a.hq + a.hkv;
  const unsigned h = is_q ? head : is_v ? head - a.hq - a.hkv : head - a.hq;
  const HeadRows src = is_q ? a.q : is_v ? a.v : a.k;
  const bool turn = on && !is_v && i < a.rot / 16;
  // the lane's two groups of 8
  const bool apart = turn && !PAIRS;
  const unsigned g0 = apart ? 8 * i : 16 * i, g1 = apart ? a.rot / 2 + 8 * i : 16 * i + 8;
  u32x4 r0 = {0, 0, 0, 0}, r1 = r0;
  float c[8], s[8];
  int64_t slot = -1;
  if (on) {
    const uint16_t* p = src.p + token * src.ts + h * src.hs;
    r0 = ld4<NT>(reinterpret_cast<const u32x4*>(p + g0));
    r1 = ld4<NT>(reinterpret_cast<const u32x4*>(p + g1));
    if (a.cache.k && !is_q) slot = a.slots[token];
  }
  if (turn) {
    const unsigned pos = min((unsigned)max(a.positions[token], 0), a.table_rows - 1);
    const f32x4* row = reinterpret_cast<const f32x4*>(a.cos_sin + (size_t)pos * a.rot + 8 * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = row[e / 4][e % 4];
      s[e] = row[a.rot / 8 + e / 4][e % 4];
    }
  }
  float x[16];
  unpack8(r0, x);
  unpack8(r1, x + 8);
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      constexpr int step = PAIRS ? 2 : 1;
      const int at = step * e, bt = PAIRS ? at + 1 : at + 8;
      const float u = x[at], w = x[bt], sn = a.inverse ? -s[e] : s[e];
      x[at] = __builtin_fmaf(u, c[e], -(w * sn));
      x[bt] = __builtin_fmaf(w, c[e], u * sn);
    }
  }
  const HeadOut dst = is_q ? a.q_out : is_v ? HeadOut{nullptr, 0, 0} : a.k_out;
  if (on && dst.p) {
    uint16_t* p = dst.p + token * dst.ts + h * dst.hs;
    st4<NT>(reinterpret_cast<u32x4*>(p + g0), pack8(x));
    st4<NT>(reinterpret_cast<u32x4*>(p + g1), pack8(x + 8));
  }
  if (!a.cache.k) return;
  uint32_t amax = 0;
  if constexpr (E4M3) {
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = max(amax, finite_mag(x[e]));
    for (unsigned d = 1; d < lanes; d *= 2) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
  }
  if (!on || is_q) return;
  if (slot < 0 || slot >= (int64_t)a.cache.pages * a.cache.size) return;
  const unsigned page = page_of((unsigned)slot, a.cache), in = (unsigned)slot - page * a.cache.size;
  const size_t at = page * a.cache.page + in * a.cache.ts + h * a.cache.hs;
  void* base = is_v ? a.cache.v : a.cache.k;
  if constexpr (E4M3) {
    const BlockScale s = block_scale<false>(amax);
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    *reinterpret_cast<u32x2*>(p + g0) = u32x2{codes4_scaled(x, s.inv), codes4_scaled(x + 4, s.inv)};
    *reinterpret_cast<u32x2*>(p + g1) = u32x2{codes4_scaled(x + 8, s.inv), codes4_scaled(x + 12, s.inv)};
    if (i == 0)
      (is_v ? a.cache.v_scales : a.cache.k_scales)[page * a.cache.spage + in * a.cache.sts + h * a.cache.shs] =
          __uint_as_float(s.kept);
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    *reinterpret_cast<u32x4*>(p + g0) = pack8(x);
    *reinterpret_cast<u32x4*>(p + g1) = pack8(x + 8);
  }
}

// 2^lg lanes of 16 values each a head
int lanes_log(unsigned dim) {
  int lg = 0;
  while ((16u << lg) < dim) ++lg;
  return lg;
}

}  // namespace

bool rope_fits(size_t tokens, size_t heads, size_t dim) {
  return tokens * heads <= 0x7FFFFFFF && fits_launch(cdiv(tokens * heads, 256u >> lanes_log(dim)), 1, 256);
}

hipError_t launch_rope_kv(const Launch& L, const RopeArgs& a) {
  // heads of a token that have work: values only with a cache
  const unsigned heads = a.hq + a.hkv + (a.cache.k ? a.hkv : 0);
  const int lg = lanes_log(a.dim);
  const size_t work = a.tokens * heads, per = 256u >> lg;
  // (16384 tokens of 80 heads of 128: 126 us through the caches, 111 past them)
  const bool nt = a.tokens * (2 * a.hq + 2 * a.hkv) * a.dim * 2 > (size_t)256 << 20;
  auto pick = [&](auto e4m3, auto pairs) {
    constexpr bool E = decltype(e4m3)::value, P = decltype(pairs)::value;
    return nt ? k_rope_kv<E, P, true> : k_rope_kv<E, P, false>;
  };
  const std::true_type yes;
  const std::false_type no;
  auto* k = a.e4m3 ? (a.pairs ? pick(yes, yes) : pick(yes, no)) : (a.pairs ? pick(no, yes) : pick(no, no));
  return launch_k(k, dim3((unsigned)cdiv(work, per)), dim3(256), 0, L.stream, a, lg, heads);
}

}  // namespace ar
