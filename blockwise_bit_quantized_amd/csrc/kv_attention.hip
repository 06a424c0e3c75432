// kv_attention.hip -- attention over the paged FP4 cache, of one row of each sequence or of many.
//
// y = softmax(scale q K^T) V over the tokens a row sees.  A tile is 16 or 32 rows: the query heads that
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
// Items (sequence, tile of rows, head) go to a workgroup each where that is fast enough.  Else they are cut in steps of 32
// tokens, laid end to end and shared out evenly, so a long sequence among short ones does not keep one workgroup; a
// workgroup's first and last item may be parts, which a second kernel joins in their order.  Where items are many, only
// those of long sequences are cut, by workgroups behind the others'.
//
// Few rows are bound by memory and the latencies around it: 32 sequences of up to 4096 (32/8 heads of 128, 85 MB) take 26.8 us, and 4 for
// the second kernel's launch, one of 131072 (143 MB) 29 us, 4.9 TB/s, and 6.6 to join its 768 parts; one of 700 (14/2 heads of 64) 7.4 us.
// Many rows are bound by the issue of vector instructions, 217 a step for 34 matrix instructions at tiles of 32 rows of 128, of
// which the expansion of FP4 is 96: 8192 rows of one sequence 610 us, 0.90 PFLOP/s (770 in the first calls behind a pause, by the clocks).
#include "kv_tile.h"

namespace mnb {
namespace {

// What the second kernel is told of a workgroup: the item that ends in its first part, if it began in another's.
struct Joint {
  int rows;                    // 0: none
  int first, second;           // the workgroup where it began, and whether as its second part
  int row0, row, head;         // first row of the sequence, row of it where the tile begins, key/value head
  int pad[2];
};

constexpr int kLeast = 2 * kWaves;   // steps of a workgroup's share at least

// Workgroups of this kernel that share a CU, by the registers of its tile (a third at 32 rows of 64: 4 x 333 rows over
// 3001 tokens, 14/2 heads, 31.2 to 29.4 us; of 96 and 128 it would spill).
constexpr int resident(int D, int R) { return D <= (R == 1 ? 128 : 64) ? 3 : 2; }

// Tiles of 32 rows read and expand the cache half as often as those of 16.  They are taken where sequences have more than 16
// rows and there is work for every CU, of heads whose tile leaves two waves to a SIMD.  16 against 32: 2048 rows of one
// sequence 77.5 and 66.0 us, 256 rows over 4096 45.9 and 35.8, 8 sequences of 16 rows over 2048 28.9 and 24.9 (32/8 heads
// of 128); with less work 8 of 5 rows over 2001 17.7 and 20.1 (20/4 heads of 96).  Heads of 192 are left out although 2048 rows
// of one sequence (32/8 heads) would take 109 us for 127: their tile needs more registers than a wave has, and the
// copies that the compiler then makes are those it has misplaced (see the queries' loads).
constexpr int kTwoTiles = 128;

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
  const typename T::Offsets offsets(g, r, S);
  float *parts = p.part + (int64_t)p.sharers * (sizeof(Joint) / 4);
  Work work = find_work(p);
  const int sharer = (int)blockIdx.x - p.lone;           // (negative: takes an item alone)
  Joint *joint = reinterpret_cast<Joint *>(p.part) + sharer;
  if (!p.whole && threadIdx.x == 0 && sharer >= 0) joint->rows = 0;
  if (work.end == 0) return;
  int64_t at = work.at, begin = work.begin;
  int b = work.b;
  const bool whole = work.whole;
  bool first_item = true;
  while (at < work.end && b < p.rows.batch) {
    const Cut c = cut_of(p, b);
    const int64_t span = whole ? 1 : c.steps, mine = span * c.tiles * p.cache.heads;
    if (at >= begin + mine) {                            // on to the next sequence
      begin += mine;
      b = next_holder(p, whole, b);
      continue;
    }
    const int item = (int)((at - begin) / span);
    const int64_t item0 = begin + item * span, stop = item0 + span < work.end ? item0 + span : work.end;
    const bool part = !(at == item0 && stop == item0 + span);
    const int s0 = whole ? 0 : (int)(at - item0), s1 = whole ? c.steps : (int)(stop - item0);
    // the last rows, which see most, first
    const int h = item % p.cache.heads, tile = c.tiles - 1 - item / p.cache.heads;

    T x;
    x.clear();
    const int tokens = c.seq.n, row0 = tile * kRows;     // row of the sequence: token row / G, head row % G
    // Rows that the tile does not have take the last token's, as zeros: no load of a step or before it stands under a condition
    // on lanes, so none part while the tile's registers are live.  (Where they did, at 32 rows of 192, whose registers pass
    // a wave's 256, the compiler put its copies of others ahead of the lanes' return.)
#pragma unroll
    for (int w = 0; w < R; ++w) {
      const int row = row0 + 16 * w + r, token = row / p.G, gh = row - token * p.G, i = min(token, tokens - 1);
      const uint32_t real = token < tokens ? 0xffffffffu : 0;
      const u4_t *q = reinterpret_cast<const u4_t *>(p.q + (int64_t)(c.seq.row0 + i) * p.ldq + (int64_t)(h * p.G + gh) * D + g * (D / 4));
#pragma unroll
      for (int k = 0; k < D / 32; ++k) x.q[w][k] = (q[k] ^ p.flip) & real;
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
    auto page_of = [&](int t, bool needed) {
      const int col = t >> p.cache.shift, page = pages[min(col, p.rows.width - 1)];   // (no step is taken where the width is 0)
      const bool there = col < p.rows.width && (uint32_t)page < (uint32_t)p.cache.pages;
      bad |= needed && !there;
      return needed && there ? page : 0;
    };
    // The places of 32 steps of the wave, two a step, a lane each; a step's data is loaded while the one before is used.
    for (int s = f0 + wave; s < f1;) {
      const int ahead = s + (lane >> 1) * kWaves;
      const int token = c.from + ahead * kStep + 16 * (lane & 1);
      const HalfStep at = half_step(p.cache, h, page_of(token, ahead < f1), token);
      auto fetch = [&](typename T::Raw &raw, int n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) T::load(raw, k, p.cache.data, HalfStep{lane_of(at.codes, 2 * n + k), lane_of(at.scales, 2 * n + k)}, offsets);
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
    // steps that some row does not see whole
    auto alone = [&](auto far, int s) {
      const int t0 = c.from + s * kStep;
      typename T::Raw raw;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = t0 + 16 * k;
        T::load(raw, k, p.cache.data, half_step(p.cache, h, page_of(t, t <= pos1 && t + 15 >= any_lo), t), offsets);
      }
      x.template step<true, decltype(far)::value>(raw, p.scale, t0, g, r, any_lo, pos1);
    };
    for (int s = e0 + wave; s < e1; s += kWaves)
      if (s < f0 || s >= f1) alone(std::false_type(), s);
    if constexpr (DT == DT_F16) {
      if (__builtin_expect(__any(x.top >= T::kFar), 0)) {
        x.clear();
#pragma unroll 1
        for (int k = 0; k < 2; ++k)                      // the wave's whole steps, and its others
          for (int s = (k ? e0 : f0) + wave; s < (k ? e1 : f1); s += kWaves)
            if (k == 0 || s < f0 || s >= f1) alone(std::true_type(), s);
      }
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
          float *to = parts + (((int64_t)sharer * 2 + (first_item ? 0 : 1)) * p.slot_rows + 16 * w + rr) * (D + 4);
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
  const float *parts = p.part + (int64_t)p.sharers * (sizeof(Joint) / 4);
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
  if constexpr (D <= kTwoTiles) {
    if (p.tile_rows == 32) hipLaunchKernelGGL((rows_kernel<DT, D, 2>), grid, block, 0, s, p);
  }
  if (p.tile_rows == 16) hipLaunchKernelGGL((rows_kernel<DT, D, 1>), grid, block, 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.whole) return e;
  hipLaunchKernelGGL((join_kernel<DT, D>), dim3((uint32_t)p.sharers, p.tile_rows / 16), dim3(kJoinThreads), 0, s, p);
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
  const int64_t rows = r.starts ? (int64_t)r.rows * G / r.batch : G;
  k.tile_rows = c.D <= kTwoTiles && rows > 16 && tiles(32) * c.heads * steps >= (int64_t)resident(c.D, 2) * kCUs * kLeast ? 32 : 16;
  k.items = tiles(k.tile_rows) * c.heads;
  k.slot_rows = r.starts || G > k.tile_rows ? k.tile_rows : G;
  const int64_t most = k.items * steps / kLeast + 1, room = resident(c.D, k.tile_rows / 16) * kCUs;
  // By these sizes alone items are whole where none can be long against the rounds of them that a place on the card takes: a round
  // takes 6 us or more, a step of a workgroup's four waves 0.15 to 0.2 (one of 700 tokens, 14/2 heads of 64, 7.5 us whole, 13.0
  // cut; 256 sequences of 500 with one of 4096 46 and 40, with one of 8192 63 and 43).  Else the lengths decide, in the kernel: of up
  // to two rounds for all items together, of more for those that are long.
  const int64_t rounds = k.items / room;
  const int short_steps = (int)(rounds < 2 ? 40 : 96 + 32 * rounds);
  k.whole = steps <= short_steps;
  k.lone = !k.whole && rounds >= 2 ? (int)k.items : 0;
  k.least = k.lone ? short_steps : 0;
  k.sharers = (int)(k.lone ? room : k.items > room ? k.items : most < room ? most : room);
  k.workgroups = k.whole ? (int)k.items : k.lone + k.sharers;
  k.bytes = k.whole ? 0 : (size_t)k.sharers * (sizeof(Joint) + (size_t)2 * k.slot_rows * (c.D + 4) * 4);
  return k;
}

hipError_t launch_kv_attn(int dtype, const KvAttnParams &p, hipStream_t s) {
  return dtype == DT_F16 ? by_head<DT_F16>(p, s) : by_head<DT_BF16>(p, s);
}

}  // namespace mnb
