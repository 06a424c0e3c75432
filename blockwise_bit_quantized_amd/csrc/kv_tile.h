// kv_tile.h -- the mathematics of attention over the paged FP4 cache: a wave's tile of rows, the loads of a step, and a
// workgroup's place in the work.
#pragma once

#include <type_traits>

#include "decode.h"

namespace mnb {

constexpr int kStep = 32;      // tokens of a wave's step
constexpr int kWaves = 4;      // of a workgroup

typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef _Float16 hh_t __attribute__((ext_vector_type(2)));
typedef __bf16 bb_t __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ f4_t mfma16(u4_t a, u4_t b, f4_t c) {
  if constexpr (DT == DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a), __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, a), __builtin_bit_cast(b8_t, b), c, 0, 0, 0);
}
// two numbers rounded to nearest even, in one instruction
template <int DT>
__device__ __forceinline__ uint32_t round2(float a, float b) {
  const f2_t v = {a, b};
  if constexpr (DT == DT_F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, hh_t));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bb_t));
}
// byte B of w as two 16-bit numbers, times the power of two in the exponent field of `s`
template <int DT, int B>
__device__ __forceinline__ uint32_t expand2(uint32_t w, uint32_t s) {
  const float f = __builtin_bit_cast(float, s);
  if constexpr (DT == DT_F16) return __builtin_bit_cast(uint32_t, (hh_t)__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, B));
  else return __builtin_bit_cast(uint32_t, (bb_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, B));
}
template <int DT>
__device__ __forceinline__ u4_t expand8(uint32_t w, uint32_t s) {
  return u4_t{expand2<DT, 0>(w, s), expand2<DT, 1>(w, s), expand2<DT, 2>(w, s), expand2<DT, 3>(w, s)};
}
// scale byte I of w in the exponent field (the conversion reads nothing else of it)
template <int I>
__device__ __forceinline__ uint32_t scale_of(uint32_t w) {
  if constexpr (I < 3) return w << (23 - 8 * I);
  else return w >> 1;
}

// Where 16 tokens of a step lie: their key codes and key scales in a page of a head, from the cache's first byte (values' lie a
// constant further).  Each lane works out the places of other steps; a step reads its two from theirs into
// scalar registers.
struct HalfStep {
  int64_t codes, scales;
};
__device__ __forceinline__ HalfStep half_step(const KvCache &c, int h, int page, int token) {
  const int S = 1 << c.shift, in = token & (S - 1);
  const int64_t head = (int64_t)page * c.page_stride + (int64_t)h * kv_head_bytes(S, c.D);
  return HalfStep{head + (int64_t)in * (c.D / 2), head + ((int64_t)S * c.D + in * (c.D / 32))};
}
__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
                   (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}
// An offset whose widening stays in the loop: widened before it, it costs a 64-bit addition at each load.
__device__ __forceinline__ uint32_t in_loop(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The value operand's parts: 16 lanes share 128, 64 or 32 elements, 8, 4 or 2 each; lane r of part k has the
// elements d0 + 8 word + (first nibble) + j of unit `word`.
template <int D> struct Parts {
  static constexpr int n8 = D / 128, n4 = D % 128 / 64, n2 = D % 64 / 32, count = n8 + n4 + n2, tiles = D / 16;
  static constexpr int nib(int k) { return k < n8 ? 8 : k < n8 + n4 ? 4 : 2; }
  static constexpr int d0(int k) { return k < n8 ? 128 * k : k < n8 + n4 ? 128 * n8 : 128 * n8 + 64 * n4; }
  static constexpr int tile0(int k) { return d0(k) / 16; }
  __device__ static __forceinline__ int word(int k, int r) { return d0(k) / 8 + (nib(k) == 8 ? r : nib(k) == 4 ? r & 7 : r & 3); }
  __device__ static __forceinline__ int shift(int k, int r) { return nib(k) == 8 ? 0 : nib(k) == 4 ? 16 * (r >> 3) : 8 * (r >> 2); }
  // first of the elements that row r of the tiles of part k holds (r = 4 g + i in a result)
  __device__ static __forceinline__ int first(int k, int r) { return 8 * word(k, r) + shift(k, r) / 4; }
};

// largest of the four lanes of a row
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
template <int DT, int D, int R>
struct Tile {
  typedef Parts<D> P;
  static constexpr int KS = D / 32;                       // matrix instructions along the head
  static constexpr float kOff = DT == DT_F16 ? 6.f : 0.f; // fp16 keeps small probabilities by 2^6
  static constexpr uint32_t kFar = DT == DT_F16 ? 141 : 253;   // first scale whose values may pass q's type
  static constexpr bool kOneBlock = D == 64 || D == 128;       // a lane's fourth of the head lies in one block
  u4_t q[R][KS];
  f4_t o[R][P::tiles];
  float base[R];           // what scores are taken against
  f4_t sum[R];             // the sum of the row's probabilities, in every place, as a product with ones
  int pos[R], lo[R];       // the row sees tokens lo .. pos
  uint32_t top;            // fp16: the largest scale of a key


  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int x = 0; x < R; ++x) {
#pragma unroll
      for (int j = 0; j < P::tiles; ++j) o[x][j] = f4_t{0.f, 0.f, 0.f, 0.f};
      base[x] = -__builtin_inff();
      sum[x] = f4_t{0.f, 0.f, 0.f, 0.f};
    }
    top = 0;
  }

  // O^T += V^T P^T for 32 tokens; with `only`, rows that do not see the token keep theirs
  template <bool ONLY>
  __device__ __forceinline__ void values(const u4_t *va, const u4_t *vb, const uint32_t *sa, const uint32_t *sb, const u4_t *prob, int r,
                                         const bool *sees) {
#pragma unroll
    for (int k = 0; k < P::count; ++k) {
      const int sh = P::shift(k, r);
      uint32_t a[4], b[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        a[t] = P::nib(k) == 8 ? va[k][t] : va[k][t] >> sh;
        b[t] = P::nib(k) == 8 ? vb[k][t] : vb[k][t] >> sh;
      }
      auto pair = [&](auto byte) {
        constexpr int B = decltype(byte)::value;
        const uint32_t a0 = expand2<DT, B>(a[0], scale_of<0>(sa[k])), a1 = expand2<DT, B>(a[1], scale_of<1>(sa[k]));
        const uint32_t a2 = expand2<DT, B>(a[2], scale_of<2>(sa[k])), a3 = expand2<DT, B>(a[3], scale_of<3>(sa[k]));
        const uint32_t b0 = expand2<DT, B>(b[0], scale_of<0>(sb[k])), b1 = expand2<DT, B>(b[1], scale_of<1>(sb[k]));
        const uint32_t b2 = expand2<DT, B>(b[2], scale_of<2>(sb[k])), b3 = expand2<DT, B>(b[3], scale_of<3>(sb[k]));
        constexpr uint32_t L = 0x05040100u, H = 0x07060302u;
        const u4_t lo4 = {__builtin_amdgcn_perm(a1, a0, L), __builtin_amdgcn_perm(a3, a2, L), __builtin_amdgcn_perm(b1, b0, L),
                          __builtin_amdgcn_perm(b3, b2, L)};
        const u4_t hi4 = {__builtin_amdgcn_perm(a1, a0, H), __builtin_amdgcn_perm(a3, a2, H), __builtin_amdgcn_perm(b1, b0, H),
                          __builtin_amdgcn_perm(b3, b2, H)};
#pragma unroll
        for (int w = 0; w < R; ++w) {
          f4_t &x = o[w][P::tile0(k) + 2 * B], &y = o[w][P::tile0(k) + 2 * B + 1];
          if constexpr (ONLY) {
            const f4_t zero = {0.f, 0.f, 0.f, 0.f};
            const f4_t dx = mfma16<DT>(lo4, prob[w], zero), dy = mfma16<DT>(hi4, prob[w], zero);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] += sees[w] ? dx[i] : 0.f;
              y[i] += sees[w] ? dy[i] : 0.f;
            }
          } else {
            x = mfma16<DT>(lo4, prob[w], x);
            y = mfma16<DT>(hi4, prob[w], y);
          }
        }
      };
      pair(std::integral_constant<int, 0>());
      if (P::nib(k) >= 4) pair(std::integral_constant<int, 1>());
      if (P::nib(k) == 8) {
        pair(std::integral_constant<int, 2>());
        pair(std::integral_constant<int, 3>());
      }
    }
  }

  // What a step reads: 16 tokens each of two places, K and V with their scales.
  struct Raw {
    uint32_t kw[2][KS], ke[2][2];
    u4_t v[2][P::count];
    uint32_t vs[2][P::count];
  };
  // A lane's offsets from the two addresses of a step's half (HalfStep): into codes and into scales, keys then values.
  struct Offsets {
    uint32_t k, ke[2], v[P::count], vs[P::count];
    __device__ __forceinline__ Offsets(int g, int r, uint32_t S) {
      k = r * (D / 2) + g * (D / 8);
      ke[0] = r * (D / 32) + g * (D / 4) / 32;
      ke[1] = r * (D / 32) + (g * (D / 4) + D / 4 - 1) / 32;
#pragma unroll
      for (int p = 0; p < P::count; ++p) {
        v[p] = S * (D / 2) + (g * (D / 8) + P::word(p, r)) * 16;
        vs[p] = S * (D / 32) + (g * (D / 32) + P::word(p, r) / 4) * 4;
      }
    }
  };
  __device__ static __forceinline__ void load(Raw &x, int half, const uint8_t *data, HalfStep at, const Offsets &o) {
    const uint8_t *codes = data + at.codes, *scales = data + at.scales;
    const uint32_t *k = reinterpret_cast<const uint32_t *>(codes + in_loop(o.k));
#pragma unroll
    for (int i = 0; i < KS; ++i) x.kw[half][i] = k[i];
    x.ke[half][0] = scales[in_loop(o.ke[0])];
    x.ke[half][1] = kOneBlock ? 0 : scales[in_loop(o.ke[1])];
#pragma unroll
    for (int p = 0; p < P::count; ++p) {
      x.v[half][p] = *reinterpret_cast<const u4_t *>(codes + in_loop(o.v[p]));
      x.vs[half][p] = *reinterpret_cast<const uint32_t *>(scales + in_loop(o.vs[p]));
    }
  }

  // Probabilities are rounded to q's type, half a step each: what the second product's instruction takes (32 bits would be two
  // products, of a high and a low part).  Their sum is taken of the rounded ones, so the weights add up to one.  Outputs are off from
  // 64 bits by 0.0017 to 0.0020 of their size (bf16) and 0.00023 to 0.00032 (fp16) where 32-bit probabilities give 0.0016 and
  // 0.0002, the output's own rounding.
  // The probabilities of scores s against the base, which is raised, and what was summed lowered, where a score passes it far.
  // (The maxima are taken of what the multiplication gives: of the matrix instruction's own results each would cost
  // another instruction, to quiet a NaN.)
  __device__ __forceinline__ void soften(const f4_t (*s)[2], float scale, u4_t *prob) {
    float t[R][8], most[R];
    bool raise = false;
#pragma unroll
    for (int w = 0; w < R; ++w) {
      const float from = base[w] == -__builtin_inff() ? 0.f : base[w];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[w][i] = fmaf(s[w][i >> 2][i & 3], scale, -from);
      most[w] = fmaxf(fmaxf(fmaxf(t[w][0], t[w][1]), fmaxf(t[w][2], t[w][3])), fmaxf(fmaxf(t[w][4], t[w][5]), fmaxf(t[w][6], t[w][7])));
      raise |= most[w] > (base[w] == -__builtin_inff() ? -__builtin_inff() : kOff + 8.f);
    }
    if (__builtin_expect(__any(raise), 0)) {
#pragma unroll
      for (int w = 0; w < R; ++w) {
        const float from = base[w] == -__builtin_inff() ? 0.f : base[w];
        const float now = fmaxf(base[w], row_max(most[w] + from) - kOff);
        const float f = now == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(base[w] - now);
        const float by = from - (now == -__builtin_inff() ? 0.f : now);
        base[w] = now;
        sum[w] *= f;
#pragma unroll
        for (int j = 0; j < P::tiles; ++j) o[w][j] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[w][i] += by;
      }
    }
#pragma unroll
    for (int w = 0; w < R; ++w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[w][i] = __builtin_amdgcn_exp2f(t[w][i]);
      prob[w] = u4_t{round2<DT>(t[w][0], t[w][1]), round2<DT>(t[w][2], t[w][3]), round2<DT>(t[w][4], t[w][5]), round2<DT>(t[w][6], t[w][7])};
      constexpr uint32_t one = DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
      sum[w] = mfma16<DT>(u4_t{one, one, one, one}, prob[w], sum[w]);
    }
  }

  // 32 tokens from t0; EDGE: some row does not see some of them.
  // FAR: a rotation or a weight can take fp16 keys past fp16, where a product has infinities for them.  `top` tells of such
  // scales after the steps (to ask in each took 29.9 us for 28.5 of 4 x 333 rows over 3001; this takes 29.0), and a wave that met
  // one takes its steps again so: those blocks by 2^-16 first, then all others.
  template <bool EDGE, bool FAR = false>
  __device__ __forceinline__ void step(const Raw &raw, float scale, int t0, int g, int r, int tile_lo, int tile_hi) {
    f4_t s[R][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int w = 0; w < R; ++w) s[w][h] = f4_t{0.f, 0.f, 0.f, 0.f};
      auto product = [&](auto scale_of_key) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const bool later = !kOneBlock && (g * (D / 4) + 8 * i) / 32 != g * (D / 4) / 32;
          const u4_t k = expand8<DT>(raw.kw[h][i], scale_of_key(later ? raw.ke[h][1] : raw.ke[h][0]) << 23);
#pragma unroll
          for (int w = 0; w < R; ++w) s[w][h] = mfma16<DT>(k, q[w][i], s[w][h]);
        }
      };
      if constexpr (FAR) {
        auto far = [](uint32_t e) { return e >= kFar && e < 255; };
        product([&](uint32_t e) { return far(e) ? e - 16 : 0; });
#pragma unroll
        for (int w = 0; w < R; ++w) s[w][h] *= 65536.f;
        product([&](uint32_t e) { return far(e) ? 0 : e; });
      } else {
        product([](uint32_t e) { return e; });
        if constexpr (DT == DT_F16) {
          const int t = t0 + 16 * h + r;                 // a token that no row sees may have any scale
          const uint32_t e = max(raw.ke[h][0], raw.ke[h][1]);
          top = max(top, !EDGE || (t >= tile_lo && t <= tile_hi) ? e : 0);
        }
      }
    }
    if constexpr (EDGE) {
#pragma unroll
      for (int w = 0; w < R; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
          s[w][i >> 2][i & 3] = tok < lo[w] || tok > pos[w] ? -__builtin_inff() : s[w][i >> 2][i & 3];
        }
    }
    u4_t prob[R];
    soften(s, scale, prob);
    if constexpr (!EDGE) {
      values<false>(raw.v[0], raw.v[1], raw.vs[0], raw.vs[1], prob, r, nullptr);
      return;
    }
    // Tokens that no row sees may hold anything: their scales become 0.  Of the others, one whose values
    // are no numbers of q's type must not reach a row that does not see it (0 times infinity): such tokens go
    // one at a time, into the rows that do.
    uint32_t far = 0, keep_a = 0, keep_b = 0, sa[P::count], sb[P::count], na[P::count], nb[P::count];   // n: without the far ones
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = t0 + 4 * g + i, b = a + 16;
      if (a >= tile_lo && a <= tile_hi) keep_a |= 0xffu << (8 * i);
      if (b >= tile_lo && b <= tile_hi) keep_b |= 0xffu << (8 * i);
    }
#pragma unroll
    for (int k = 0; k < P::count; ++k) {
      sa[k] = raw.vs[0][k] & keep_a;
      sb[k] = raw.vs[1][k] & keep_b;
      uint32_t fa = 0, fb = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((sa[k] >> (8 * i) & 255) >= kFar) fa |= 0xffu << (8 * i);
        if ((sb[k] >> (8 * i) & 255) >= kFar) fb |= 0xffu << (8 * i);
      }
      na[k] = sa[k] & ~fa;
      nb[k] = sb[k] & ~fb;
      far |= fa | fb;
    }
    values<false>(raw.v[0], raw.v[1], na, nb, prob, r, nullptr);
    if (!__any(far != 0)) return;
    for (int x = 0; x < 32; ++x) {                       // token t0 + x: lanes of group (x & 15) / 4, place x & 3
      const bool mine = (x & 15) >> 2 == g;
      const uint32_t byte = mine ? 0xffu << (8 * (x & 3)) : 0;
      uint32_t oa[P::count], ob[P::count], any = 0;
#pragma unroll
      for (int k = 0; k < P::count; ++k) {
        oa[k] = x < 16 ? sa[k] & ~na[k] & byte : 0;
        ob[k] = x < 16 ? 0 : sb[k] & ~nb[k] & byte;
        any |= oa[k] | ob[k];
      }
      if (!__any(any != 0)) continue;
      // probabilities of this token alone
      const uint32_t half = 0xffffu << (16 * (x & 1));
      u4_t one[R];
      bool sees[R];
#pragma unroll
      for (int w = 0; w < R; ++w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) one[w][i] = mine && i == (x >> 4) * 2 + ((x & 3) >> 1) ? prob[w][i] & half : 0;
        sees[w] = t0 + x >= lo[w] && t0 + x <= pos[w];
      }
      values<true>(raw.v[0], raw.v[1], oa, ob, one, r, sees);
    }
  }
};

// How a sequence's work is cut: its tiles of 16 or 32 rows, and the tokens that any of its rows sees.
struct Cut {
  KvSeq seq;
  int tiles, from, steps;      // from: a multiple of kStep
  bool beyond;                 // more tokens than the pages hold: its rows become NaN
};
__device__ __forceinline__ Cut cut_of(const KvAttnParams &p, int b) {
  Cut c;
  c.seq = kv_seq(p.rows, b);
  c.tiles = (int)(((int64_t)c.seq.n * p.G + p.tile_rows - 1) >> (p.tile_rows == 32 ? 5 : 4));
  const int lo = p.window ? max(0, c.seq.first() - p.window + 1) : 0;
  c.from = lo / kStep * kStep;
  c.beyond = c.seq.len > p.rows.width << p.cache.shift;
  // a row that sees nothing is written too
  c.steps = c.beyond ? 1 : max(1, (c.seq.len - c.from + kStep - 1) / kStep);
  return c;
}
// A sequence's items (tiles of each head), and the steps of one.
struct Cost {
  int64_t items;
  int steps;
};
__device__ __forceinline__ Cost cost_of(const KvAttnParams &p, int b) {
  const Cut c = cut_of(p, min(b, p.rows.batch - 1));
  const int tiles = b < p.rows.batch ? c.tiles : 0;
  return Cost{(int64_t)tiles * p.cache.heads, tiles ? c.steps : 0};
}

// Sums over the wave's lanes up to this one.  (Every wave finds the workgroup's place in the work by itself.)
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up((long long)v, d);
    if (lane >= d) v += o;
  }
  return v;
}
// The workgroup's share [at, end) of the work, in items (`whole`) or in steps of them (none left: end 0), and the sequence
// that holds `at` with the place where it begins.
struct Work {
  int64_t at, end, begin, share;
  int b;
  bool whole;
};
// What a sequence adds to the work: items, or steps of those items that may be cut.
__device__ __forceinline__ int64_t part_of(const KvAttnParams &p, bool whole, const Cost &c) {
  return whole ? c.items : c.steps > p.least ? c.items * c.steps : 0;
}
// The sequence that holds w.at: w.b and w.begin, or w.end = 0 if none does.  (`first`: costs of the first 64.)
__device__ __forceinline__ void find_holder(const KvAttnParams &p, Work &w, const Cost &first) {
  const int lane = threadIdx.x & 63;
  const int64_t end = w.end;
  int64_t before = 0;
  w.end = 0;                                             // (set behind the loop alone, it would not stay in scalar registers)
  for (int b0 = 0; b0 < p.rows.batch; b0 += 64) {
    const int64_t mine = part_of(p, w.whole, b0 ? cost_of(p, b0 + lane) : first), run = wave_scan(mine) + before;
    const uint64_t hit = __ballot(run > w.at);
    before = lane_of(run, 63);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      w.b = b0 + l;
      w.begin = lane_of(run - mine, l);
      w.end = end;
      return;
    }
  }
}
// The next sequence behind b that has work (the batch's size: none).  64 are looked at together: those without work in between cost no load
// behind a load.
__device__ __forceinline__ int next_holder(const KvAttnParams &p, bool whole, int b) {
  const int lane = (int)in_loop(threadIdx.x & 63);       // (addresses of lanes kept through the steps cost the tile's registers)
  for (int b0 = ++b & ~63; b0 < p.rows.batch; b0 += 64) {
    const int mine = b0 + lane;
    const uint64_t hit = __ballot(mine >= b && part_of(p, whole, cost_of(p, mine)) > 0);
    if (hit) return b0 + __builtin_ctzll(hit);
  }
  return p.rows.batch;
}
// Shares of steps balance what sequences of different lengths take, but cost parts of two items a workgroup and their
// join.  So where there is a workgroup for each item they are taken, by the lengths that the call finds, only if the
// longest item is longer than five shares and kPatience steps.  One row each of heads of 128 (32 query and 8 key/value),
// cut against whole: 32 sequences of 4096 35.0 and 30.2 us, 64 of 4096 57.0 and 51.3, 32 of 1024 22.4 and 10.9, 24 of 4096 28.0
// and 27.6, 32 of different lengths up to 4096 41.5 and 27.8; but one of 2048 11.4 and 16.6, four of 2048 12.2 and 16.9, 16 of 8192
// 35.3 and 36.4.  With other heads (14/2 of 64, 20/4 of 96, 8/1 of 256, 16/16 of 128; 1 to 64 sequences of 1024 to 32768) it took the
// faster of the two, or one within 2%, in all of 40 cases: 8/1 of 256, 32 of 4096 cut 22.0, whole 36.5; 16/16 of 128, 16 of 2048 26.4 and 19.4.
// Where a place on the card takes two rounds of items or more, only long ones (of more than p.least steps) are ever cut, if the
// longest is longer than an even share, by workgroups that wait for nothing else: those of other items need not know.  Cut
// against whole: 256 sequences of 500 with one of 8192 42 and 67 us, with one of 131072 67 and 594; 2048 rows of a prompt beside 32
// sequences of up to 32768 234 and 291; 4096 rows over 32768 (none longer than a share) 2274 and 2016.  Knowing it costs 2.7 us, of
// which the second kernel has most: 256 of 1024 49.4 us, 46.9 where the tables are too short for long ones.
constexpr int kPatience = 16;
__device__ __forceinline__ Work find_work(const KvAttnParams &p) {
  Work w{};
  const bool alone = p.whole || (int)blockIdx.x < p.lone;
  w.share = 1;
  w.whole = true;
  w.at = blockIdx.x;
  w.end = w.at + 1;
  if (alone && !p.rows.starts) {                         // as many items for each sequence
    const int each = (p.G + p.tile_rows - 1) / p.tile_rows * p.cache.heads;
    w.b = blockIdx.x / each;
    w.begin = (int64_t)w.b * each;
    if (p.whole || cut_of(p, w.b).steps <= p.least) return w;
  }
  const Cost first = cost_of(p, threadIdx.x & 63);
  if (alone && p.rows.starts) {
    find_holder(p, w, first);
    if (p.whole || w.end == 0 || cut_of(p, w.b).steps <= p.least) return w;
  }
  int64_t items = 0, steps = 0, part = 0;                // of the lane's sequences
  int most = 0;
#pragma unroll 4
  for (int b0 = 0; b0 < p.rows.batch; b0 += 64) {
    const Cost c = b0 ? cost_of(p, b0 + (int)(threadIdx.x & 63)) : first;
    items += c.items;
    steps += c.items * c.steps;
    part += c.steps > p.least ? c.items * c.steps : 0;
    most = max(most, c.steps);
  }
  auto whole_sum = [](int64_t v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor((long long)v, d);
    return lane_of(v, 0);
  };
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
  most = __builtin_amdgcn_readlane(most, 0);
  const int64_t all = whole_sum(steps);
  const int64_t cut = p.lone ? whole_sum(part) : all, count = p.lone ? 0 : whole_sum(items);
  const int64_t even = lane_of((all + p.sharers - 1) / p.sharers, 0);   // (a division's result is in vector registers)
  w.whole = p.lone ? most <= even : count <= p.workgroups && most <= 5 * even + kPatience;
  if (alone || (p.lone && w.whole)) {
    if (alone != w.whole) w.end = 0;                     // the others' work
    return w;
  }
  if (!w.whole) {
    w.share = p.lone ? lane_of((cut + p.sharers - 1) / p.sharers, 0) : even;
    if (w.share < 2 * kWaves) w.share = 2 * kWaves;      // no smaller parts than two steps a wave
  }
  const int64_t total = w.whole ? count : cut;
  w.at = ((int)blockIdx.x - p.lone) * w.share;
  w.end = min(w.at + w.share, total);
  if (w.at < total) find_holder(p, w, first);
  else w.end = 0;
  return w;
}

}  // namespace mnb
