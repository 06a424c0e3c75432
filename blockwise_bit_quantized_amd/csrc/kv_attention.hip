// kv_attention.hip -- attention over the paged FP4 cache, for rows that are few for each sequence.
//
// y = softmax(scale q K^T) V over the tokens a row sees.  A tile is 16 rows: the query heads that
// share a key/value head, of one token or of several.  A wave takes 32 tokens a step:
//   S^T [32 tokens x 16 rows] = K Q^T, two matrix instructions of 16 x 16 x 32 for each 32 elements.  The
//     sum over the head may run in any order that K and Q share, so lane (g, r) takes a fourth of
//     token r's row in one load.
//   p = 2^(S' - base), base the largest score seen, raised only when a score passes it by 2^8: scores
//     within that cost no exchange between lanes and no rescaling.  The sums are FP32.
//   O^T [D x 16 rows] += V^T P^T: the lane that holds the scores of 8 tokens holds the same 8 tokens'
//     probabilities as the instruction's operand, and the cache's value layout gives the lane the
//     same elements of these 8 tokens, so neither passes through LDS.
// FP4 codes become 16-bit numbers by the conversion instruction that applies the block's scale.
//
// Items (sequence, tile of rows, head) are cut in steps of 32 tokens, laid end to end and shared out evenly, so
// a long sequence among short ones does not keep one workgroup; a workgroup's first and last item
// may be parts, which a second kernel joins in their order.
#include <type_traits>

#include "decode.h"

namespace mnb {
namespace {

constexpr int kStep = 32;      // tokens of a wave's step
constexpr int kWaves = 4;
constexpr int kLeast = 2 * kWaves;   // steps of a workgroup's share at least

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
  u4_t q[R][KS];
  f4_t o[R][P::tiles];
  float base[R];           // what scores are taken against
  f4_t sum[R];             // the sum of the row's probabilities, in every place, as a product with ones
  int pos[R], lo[R];       // the row sees tokens lo .. pos

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int x = 0; x < R; ++x) {
#pragma unroll
      for (int j = 0; j < P::tiles; ++j) o[x][j] = f4_t{0.f, 0.f, 0.f, 0.f};
      base[x] = -__builtin_inff();
      sum[x] = f4_t{0.f, 0.f, 0.f, 0.f};
    }
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
  // head: uniform; in: the first token's place in the page
  __device__ static __forceinline__ void load(Raw &x, int half, const uint8_t *head, uint32_t in, uint32_t S, int g, int r) {
    const uint32_t tok = in + r, unit = (in >> 2) + g;
    const uint32_t *k = reinterpret_cast<const uint32_t *>(head + (tok * (D / 2) + g * (D / 8)));
#pragma unroll
    for (int i = 0; i < KS; ++i) x.kw[half][i] = k[i];
    const uint32_t block = g * (D / 4) / 32, last = (g * (D / 4) + D / 4 - 1) / 32;
    x.ke[half][0] = head[S * D + tok * (D / 32) + block];
    // a lane's fourth of the head lies in one block where D is 64 or 128
    x.ke[half][1] = D == 64 || D == 128 ? 0 : head[S * D + tok * (D / 32) + last];
#pragma unroll
    for (int p = 0; p < P::count; ++p) {
      const uint32_t word = P::word(p, r);
      x.v[half][p] = *reinterpret_cast<const u4_t *>(head + (S * (D / 2) + (unit * (D / 8) + word) * 16));
      x.vs[half][p] = *reinterpret_cast<const uint32_t *>(head + (S * D + S * (D / 32) + (unit * (D / 32) + word / 4) * 4));
    }
  }

  // 32 tokens from t0; EDGE: some row does not see some of them
  template <bool EDGE>
  __device__ __forceinline__ void step(const Raw &raw, float scale, int t0, int g, int r, int tile_lo, int tile_hi) {
    f4_t s[R][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int w = 0; w < R; ++w) s[w][h] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const bool later = D != 64 && D != 128 && (g * (D / 4) + 8 * i) / 32 != g * (D / 4) / 32;
        const u4_t k = expand8<DT>(raw.kw[h][i], (later ? raw.ke[h][1] : raw.ke[h][0]) << 23);
#pragma unroll
        for (int w = 0; w < R; ++w) s[w][h] = mfma16<DT>(k, q[w][i], s[w][h]);
      }
    }
    u4_t prob[R];
    float most[R];
    bool raise = false;
#pragma unroll
    for (int w = 0; w < R; ++w) {
      f4_t *t = s[w];
      if constexpr (EDGE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
          t[i >> 2][i & 3] = tok < lo[w] || tok > pos[w] ? -__builtin_inff() : t[i >> 2][i & 3];
        }
      }
      most[w] = fmaxf(fmaxf(fmaxf(t[0][0], t[0][1]), fmaxf(t[0][2], t[0][3])), fmaxf(fmaxf(t[1][0], t[1][1]), fmaxf(t[1][2], t[1][3]))) * scale;
      raise |= most[w] > base[w] + (kOff + 8.f);
    }
    if (__any(raise)) {
#pragma unroll
      for (int w = 0; w < R; ++w) {
        const float now = fmaxf(base[w], row_max(most[w]) - kOff);
        const float f = now == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(base[w] - now);
        base[w] = now;
        sum[w] *= f;
#pragma unroll
        for (int j = 0; j < P::tiles; ++j) o[w][j] *= f;
      }
    }
#pragma unroll
    for (int w = 0; w < R; ++w) {
      const float from = base[w] == -__builtin_inff() ? 0.f : base[w];
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = __builtin_amdgcn_exp2f(fmaf(s[w][i >> 2][i & 3], scale, -from));
      prob[w] = u4_t{round2<DT>(t[0], t[1]), round2<DT>(t[2], t[3]), round2<DT>(t[4], t[5]), round2<DT>(t[6], t[7])};
      constexpr uint32_t one = DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
      sum[w] = mfma16<DT>(u4_t{one, one, one, one}, prob[w], sum[w]);
    }
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
  c.tiles = (int)(((int64_t)c.seq.n * p.G + p.tile_rows - 1) / p.tile_rows);
  const int lo = p.window ? max(0, c.seq.first() - p.window + 1) : 0;
  c.from = lo / kStep * kStep;
  c.beyond = c.seq.len > p.rows.width << p.cache.shift;
  // a row that sees nothing is written too
  c.steps = c.beyond ? 1 : max(1, (c.seq.len - c.from + kStep - 1) / kStep);
  return c;
}
__device__ __forceinline__ int64_t cost_of(const KvAttnParams &p, int b) {
  if (b >= p.rows.batch) return 0;
  const Cut c = cut_of(p, b);
  return (int64_t)c.tiles * p.cache.heads * (p.whole ? 1 : c.steps);
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
__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
                   (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}
// The workgroup's steps [at, end) of the work (none left: end 0), and the sequence that holds `at` with the place where
// it begins.
struct Work {
  int64_t at, end, begin, share;
  int b;
};
__device__ __forceinline__ Work find_work(const KvAttnParams &p) {
  Work w{};
  const int lane = threadIdx.x & 63;
  w.share = 1;
  if (p.whole && !p.rows.starts) {                       // as many items for each sequence
    const int each = (p.G + p.tile_rows - 1) / p.tile_rows * p.cache.heads;
    w.at = blockIdx.x;
    w.end = w.at + 1;
    w.b = blockIdx.x / each;
    w.begin = (int64_t)w.b * each;
    return w;
  }
  const int64_t first = cost_of(p, lane), first_run = wave_scan(first);
  if (!p.whole) {
    int64_t total = lane_of(first_run, 63);
    for (int b0 = 64; b0 < p.rows.batch; b0 += 64) total += lane_of(wave_scan(cost_of(p, b0 + lane)), 63);
    w.share = (total + p.workgroups - 1) / p.workgroups;
    if (w.share < kLeast) w.share = kLeast;
  }
  w.at = (int64_t)blockIdx.x * w.share;
  int64_t before = 0;
  for (int b0 = 0; b0 < p.rows.batch; b0 += 64) {
    const int64_t mine = b0 ? cost_of(p, b0 + lane) : first, run = (b0 ? wave_scan(mine) : first_run) + before;
    const uint64_t hit = __ballot(run > w.at);
    before = lane_of(run, 63);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      w.b = b0 + l;
      w.begin = lane_of(run - mine, l);
      w.end = w.at + w.share;
      break;
    }
  }
  return w;
}

// What the second kernel is told of a workgroup: the item that ends in its first part, if it began in another's.
struct Joint {
  int rows;                    // 0: none
  int first, second;           // the workgroup where it began, and whether as its second part
  int row0, row, head;         // first row of the sequence, row of it where the tile begins, key/value head
  int pad[2];
};

// Workgroups of this kernel that share a CU, by the registers of its tile.
constexpr int resident(int D, int R) { return R == 1 ? (D <= 128 ? 3 : 2) : R == 2 && D <= 128 ? 2 : 1; }

template <int DT, int D, int R>
__global__ __launch_bounds__(kWaves * 64, resident(D, R)) void rows_kernel(KvAttnParams p) {
  typedef Parts<D> P;
  typedef Tile<DT, D, R> T;
  constexpr int kRows = 16 * R;
  constexpr int kRow = D + 4;                            // FP32 of a row in LDS, off the bank period
  __shared__ float acc[kWaves][16][kRow];
  __shared__ float stat[kWaves][16][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r = lane & 15;
  const uint32_t S = 1u << p.cache.shift;
  Joint *joint = reinterpret_cast<Joint *>(p.part) + blockIdx.x;
  float *parts = p.part + (int64_t)p.workgroups * (sizeof(Joint) / 4);
  const Work work = find_work(p);
  if (!p.whole && threadIdx.x == 0) joint->rows = 0;
  if (work.end == 0) return;
  int64_t at = work.at, begin = work.begin;
  int b = work.b;
  bool first_item = true;
  while (at < work.end && b < p.rows.batch) {
    const Cut c = cut_of(p, b);
    const int64_t span = p.whole ? 1 : c.steps, mine = span * c.tiles * p.cache.heads;
    if (at >= begin + mine) {                            // on to the next sequence
      begin += mine;
      ++b;
      continue;
    }
    const int item = (int)((at - begin) / span);
    const int64_t item0 = begin + item * span, stop = item0 + span < work.end ? item0 + span : work.end;
    const bool part = !(at == item0 && stop == item0 + span);
    const int s0 = p.whole ? 0 : (int)(at - item0), s1 = p.whole ? c.steps : (int)(stop - item0);
    // the last rows, which see most, first
    const int h = item % p.cache.heads, tile = c.tiles - 1 - item / p.cache.heads;

    T x;
    x.clear();
    const int tokens = c.seq.n, row0 = tile * kRows;     // row of the sequence: token row / G, head row % G
#pragma unroll
    for (int w = 0; w < R; ++w) {
      const int row = row0 + 16 * w + r, i = row / p.G, gh = row - i * p.G;
      const bool real = i < tokens;
      const uint16_t *q = p.q + (int64_t)(c.seq.row0 + i) * p.ldq + (int64_t)(h * p.G + gh) * D + g * (D / 4);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) x.q[w][k] = real ? reinterpret_cast<const u4_t *>(q)[k] ^ p.flip : u4_t{0, 0, 0, 0};
      x.pos[w] = real ? c.seq.first() + i : -1;
      x.lo[w] = p.window ? x.pos[w] - p.window + 1 : 0;
    }
    // what all rows of the tile see, and what any sees
    const int i0 = row0 / p.G, i1 = min(tokens - 1, (row0 + kRows - 1) / p.G);
    const int pos0 = c.seq.first() + i0, pos1 = c.seq.first() + i1;
    const int any_lo = p.window ? max(0, pos0 - p.window + 1) : 0, all_lo = p.window ? max(0, pos1 - p.window + 1) : 0;
    // the steps with tokens that any row sees
    const int e0 = max(s0, (any_lo - c.from) / kStep), e1 = c.beyond || pos1 < 0 ? e0 : min(s1, (pos1 - c.from) / kStep + 1);
    // ... and those whose tokens all see
    const int f0 = min(e1, max(e0, (all_lo - c.from + kStep - 1) / kStep)), f1 = max(f0, min(e1, (pos0 + 1 - c.from) / kStep));
    bool bad = c.beyond;
    const int32_t *pages = p.rows.pages + (int64_t)b * p.rows.ldp;
    const uint8_t *const data = p.cache.data + (int64_t)h * kv_head_bytes(S, D);
    auto page_of = [&](int t, bool needed) {
      const int col = t >> p.cache.shift;
      int page = needed && col < p.rows.width ? pages[col] : -1;
      if ((uint32_t)page >= (uint32_t)p.cache.pages) {
        bad |= needed;
        page = 0;
      }
      return page;
    };
    auto load = [&](typename T::Raw &raw, int half, int page, int t) {
      T::load(raw, half, data + (int64_t)page * p.cache.page_stride, t & (S - 1), S, g, r);
    };
    // Page numbers of 32 steps of the wave, two a step, a lane each; a step's data is loaded while the one before is used.
    for (int s = f0 + wave; s < f1;) {
      const int ahead = s + (lane >> 1) * kWaves;
      const int page = page_of(c.from + ahead * kStep + 16 * (lane & 1), ahead < f1);
      auto fetch = [&](typename T::Raw &raw, int n) {
        const int t = c.from + (s + n * kWaves) * kStep;
        load(raw, 0, __builtin_amdgcn_readlane(page, 2 * n), t);
        load(raw, 1, __builtin_amdgcn_readlane(page, 2 * n + 1), t + 16);
      };
      const int count = min(32, (f1 - s + kWaves - 1) / kWaves);
      typename T::Raw one, two;
      fetch(one, 0);
      // (the last step is loaded again behind itself: a load under a condition would make every step wait for all)
      for (int n = 0;;) {
        fetch(two, min(n + 1, count - 1));
        x.template step<false>(one, p.scale, 0, g, r, 0, 0);
        if (++n == count) break;
        fetch(one, min(n + 1, count - 1));
        x.template step<false>(two, p.scale, 0, g, r, 0, 0);
        if (++n == count) break;
      }
      s += count * kWaves;
    }
    for (int s = e0 + wave; s < e1; s += kWaves) {
      if (s >= f0 && s < f1) continue;
      const int t0 = c.from + s * kStep;
      typename T::Raw raw;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = t0 + 16 * k;
        load(raw, k, page_of(t, t <= pos1 && t + 15 >= any_lo), t);
      }
      x.template step<true>(raw, p.scale, t0, g, r, any_lo, pos1);
    }
    const int rows = (int)min((int64_t)kRows, (int64_t)tokens * p.G - row0);
    if (part && threadIdx.x == 0 && stop == item0 + span) {
      const int64_t w0 = item0 / work.share;
      *joint = Joint{rows, (int)w0, item0 > w0 * work.share, c.seq.row0, row0, h, {0, 0}};
    }
    // the waves' parts, 16 rows at a time, in the waves' order
    const bool nan = __any(bad);
#pragma unroll
    for (int w = 0; w < R; ++w) {
      const float base = x.base[w], sum = nan ? __builtin_nanf("") : x.sum[w][0];
      if (g == 0) {
        stat[wave][r][0] = base;
        stat[wave][r][1] = sum;
      }
      __syncthreads();
      float most = stat[0][r][0];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) most = fmaxf(most, stat[v][r][0]);
      // a part that saw nothing adds nothing, whatever it holds
      const bool saw = base != -__builtin_inff();
      const float f = saw ? __builtin_amdgcn_exp2f(base - most) : 0.f;
#pragma unroll
      for (int k = 0; k < P::count; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float *to = &acc[wave][r][P::first(k, 4 * g + j)];
#pragma unroll
          for (int n = 0; n < P::nib(k); ++n) to[n] = saw ? x.o[w][P::tile0(k) + n][j] * f : 0.f;
        }
      __syncthreads();
      for (int e = threadIdx.x; e < min(16, rows - 16 * w) * (D / 8); e += kWaves * 64) {
        const int rr = e / (D / 8), d = (e - rr * (D / 8)) * 8;
        float m = stat[0][rr][0], l = 0.f, v[8] = {};
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, stat[i][rr][0]);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
          const float bw = stat[i][rr][0], sw = stat[i][rr][1];
          l += bw == -__builtin_inff() ? sw : sw * __builtin_amdgcn_exp2f(bw - m);
#pragma unroll
          for (int n = 0; n < 8; ++n) v[n] += acc[i][rr][d + n];
        }
        const int row = row0 + 16 * w + rr;
        if (part) {
          float *to = parts + (((int64_t)blockIdx.x * 2 + (first_item ? 0 : 1)) * p.slot_rows + 16 * w + rr) * (D + 4);
          if (d == 0) {
            to[D] = m;
            to[D + 1] = l;
          }
          *reinterpret_cast<f4_t *>(to + d) = f4_t{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f4_t *>(to + d + 4) = f4_t{v[4], v[5], v[6], v[7]};
        } else {
          const int ri = row / p.G, rh = row - ri * p.G;
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int n = 0; n < 8; ++n) v[n] = l == 0.f ? 0.f : v[n] * inv;
          store8<DT>(p.y + (int64_t)(c.seq.row0 + ri) * p.ldy + (int64_t)(h * p.G + rh) * D + d, v);
        }
      }
      __syncthreads();
    }
    at = stop;
    first_item = false;
  }
}

// The parts of items that lie in more than one workgroup's share, joined by a workgroup for each that holds the end of
// one, 16 rows each.  Groups of threads take the parts in turn, and the groups' results meet in their order.
constexpr int kJoinThreads = 1024;
template <int DT, int D>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(KvAttnParams p) {
  const Joint j = reinterpret_cast<const Joint *>(p.part)[blockIdx.x];
  const int from_row = 16 * blockIdx.y, rows = min(16, j.rows - from_row);
  if (rows <= 0) return;
  const float *parts = p.part + (int64_t)p.workgroups * (sizeof(Joint) / 4);
  const int n = (int)blockIdx.x - j.first + 1, slots = rows * (D / 4);   // at most 1024, of 16 rows of 256
  const int groups = kJoinThreads / slots, t = threadIdx.x, group = t / slots, s = t - group * slots;
  const int rr = s / (D / 4), d = (s - rr * (D / 4)) * 4;
  __shared__ f4_t sums[kJoinThreads];
  __shared__ f2_t stat[kJoinThreads];                    // base and sum
  float m = -__builtin_inff(), l = 0.f;
  f4_t v = {0.f, 0.f, 0.f, 0.f};
  // v, l against m, and another part's against its own
  auto add = [&](float bw, float sw, f4_t o) {
    const bool saw = bw != -__builtin_inff();            // a part that saw nothing has the sum 0, or NaN where a page was out of range
    const float now = fmaxf(m, bw), f = m == now ? 1.f : __builtin_amdgcn_exp2f(m - now), g = saw ? __builtin_amdgcn_exp2f(bw - now) : 0.f;
    m = now;
    l = l * f + (saw ? sw * g : sw);
    v = v * f + o * g;
  };
  if (group < groups) {
    for (int i = group; i < n; i += 4 * groups) {
      float bw[4], sw[4];
      f4_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int part = min(i + k * groups, n - 1);     // (again, where there is none)
        const float *from = parts + (((int64_t)(j.first + part) * 2 + (part == 0 && j.second)) * p.slot_rows + from_row + rr) * (D + 4);
        bw[k] = from[D];
        sw[k] = from[D + 1];
        o[k] = *reinterpret_cast<const f4_t *>(from + d);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * groups < n) add(bw[k], sw[k], o[k]);
    }
    sums[t] = v;
    stat[t] = f2_t{m, l};
  }
  __syncthreads();
  if (group != 0) return;
  for (int k = 1; k < groups; ++k) add(stat[s + k * slots][0], stat[s + k * slots][1], sums[s + k * slots]);
  const int row = j.row + from_row + rr, ri = row / p.G, rh = row - ri * p.G;
  uint16_t *y = p.y + (int64_t)(j.row0 + ri) * p.ldy + (int64_t)(j.head * p.G + rh) * D + d;
  if (l == 0.f) v = f4_t{0.f, 0.f, 0.f, 0.f};
  else v *= 1.f / l;
  *reinterpret_cast<u2_t *>(y) = u2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

template <int DT, int D>
hipError_t launch(const KvAttnParams &p, hipStream_t s) {
  const dim3 grid((uint32_t)p.workgroups), block(kWaves * 64);
  if (p.tile_rows == 16) hipLaunchKernelGGL((rows_kernel<DT, D, 1>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((rows_kernel<DT, D, 2>), grid, block, 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.whole) return e;
  hipLaunchKernelGGL((join_kernel<DT, D>), dim3((uint32_t)p.workgroups, p.tile_rows / 16), dim3(kJoinThreads), 0, s, p);
  return hipGetLastError();
}
template <int DT>
hipError_t by_head(const KvAttnParams &p, hipStream_t s) {
  switch (p.cache.D) {
    case 64: return launch<DT, 64>(p, s);
    case 96: return launch<DT, 96>(p, s);
    case 128: return launch<DT, 128>(p, s);
    case 192: return launch<DT, 192>(p, s);
    default: return launch<DT, 256>(p, s);
  }
}

}  // namespace

KvPlan kv_attn_plan(const KvCache &c, const KvRows &r, int G, int window) {
  KvPlan k{};
  int64_t tokens = (int64_t)r.width << c.shift;
  if (window && tokens > (int64_t)window + r.rows + kStep) tokens = (int64_t)window + r.rows + kStep;
  const int64_t steps = (tokens + kStep - 1) / kStep + 1;
  // at most one short tile for each sequence
  auto tiles = [&](int rows) { return r.starts ? (int64_t)r.rows * G / rows + r.batch : (int64_t)r.batch * ((G + rows - 1) / rows); };
  // Tiles of 32 rows read and expand the cache half as often, where sequences have more than 16 rows and
  // there is work for every CU.
  const int64_t rows = r.starts ? (int64_t)r.rows * G / r.batch : G;
  k.tile_rows = rows > 16 && tiles(32) * c.heads * steps >= (int64_t)resident(c.D, 2) * kCUs * kLeast ? 32 : 16;
  k.items = tiles(k.tile_rows) * c.heads;
  k.slot_rows = r.starts || G > k.tile_rows ? k.tile_rows : G;
  const int64_t most = k.items * steps / kLeast + 1, room = resident(c.D, k.tile_rows / 16) * kCUs;
  k.whole = k.items >= 2 * room || steps <= 32;
  k.workgroups = (int)(k.whole ? k.items : most < room ? most : room);
  k.bytes = k.whole ? 0 : (size_t)k.workgroups * (sizeof(Joint) + (size_t)2 * k.slot_rows * (c.D + 4) * 4);
  return k;
}

hipError_t launch_kv_attn(int dtype, const KvAttnParams &p, hipStream_t s) {
  return dtype == DT_F16 ? by_head<DT_F16>(p, s) : by_head<DT_BF16>(p, s);
}

}  // namespace mnb
