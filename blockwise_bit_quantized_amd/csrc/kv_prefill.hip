// kv_prefill.hip -- attention over the paged FP4 cache for many rows of a sequence at once.
//
// The mathematics is that of kv_tile.h; what differs is who expands the cache.  A workgroup's four waves hold
// neighbouring tiles of rows of one sequence and key/value head, so they use the same keys and values: for each step of 32
// tokens a wave expands a fourth of them into LDS, in the order of the matrix instruction's operands (a lane writes
// and reads 16 bytes beside its neighbours', so no banks meet), while all multiply the step before, out of the other
// half.  One barrier a step.  Steps that some row does not see whole are taken by each wave alone.
#include "kv_tile.h"

namespace mnb {
namespace {

// The largest k below count with wave + 4 k < n, plus 1: how many of n things a wave takes.
constexpr int share(int n) { return (n + kWaves - 1) / kWaves; }

template <int DT, int D, int R>
__global__ __launch_bounds__(kWaves * 64, 2) void prefill_kernel(KvAttnParams p) {
  typedef Parts<D> P;
  typedef Tile<DT, D, R> T;
  constexpr int KS = D / 32, kRows = 16 * R, kFrags = 2 * KS + P::tiles;
  __shared__ u4_t frag[2][kFrags][64];                   // keys [half][KS], then values
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r = lane & 15;
  const uint32_t S = 1u << p.cache.shift;
  const Work work = find_work(p);
  if (work.end == 0) return;
  const Cut c = cut_of(p, work.b);
  const int item = (int)(work.at - work.begin);
  const int h = item % p.cache.heads, group = c.tiles - 1 - item / p.cache.heads;   // the last rows, which see most, first
  const int tokens = c.seq.n, group0 = group * kRows * kWaves, row0 = group0 + wave * kRows;

  T x;
  x.clear();
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const int row = row0 + 16 * w + r, i = row / p.G, gh = row - i * p.G;
    const bool real = i < tokens;
    const uint16_t *q = p.q + (int64_t)(c.seq.row0 + i) * p.ldq + (int64_t)(h * p.G + gh) * D + g * (D / 4);
#pragma unroll
    for (int k = 0; k < KS; ++k) x.q[w][k] = real ? reinterpret_cast<const u4_t *>(q)[k] ^ p.flip : u4_t{0, 0, 0, 0};
    x.pos[w] = real ? c.seq.first() + i : -1;
    x.lo[w] = p.window ? x.pos[w] - p.window + 1 : 0;
  }
  const int first = c.seq.first();
  auto token_of = [&](int row) { return min(tokens - 1, row / p.G); };
  // of this wave's rows, and of the workgroup's: the first and the last position
  const int pos0 = first + token_of(row0), pos1 = first + token_of(row0 + kRows - 1);
  const int all0 = first + token_of(group0), all1 = first + token_of(group0 + kRows * kWaves - 1);
  const int any_lo = p.window ? max(0, pos0 - p.window + 1) : 0;
  // steps that this wave's rows need, and those that all the workgroup's rows see whole
  const bool idle = row0 >= (int64_t)tokens * p.G;
  const int e0 = (any_lo - c.from) / kStep, e1 = c.beyond || idle || pos1 < 0 ? e0 : (pos1 - c.from) / kStep + 1;
  const int all_lo = p.window ? max(0, all1 - p.window + 1) : 0;
  const int f0 = (all_lo - c.from + kStep - 1) / kStep, f1 = c.beyond ? f0 : max(f0, (all0 + 1 - c.from) / kStep);

  bool bad = c.beyond;
  const int32_t *pages = p.rows.pages + (int64_t)work.b * p.rows.ldp;
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

  // This wave's part of a step: fragments of keys f = wave + 4 m, half f / KS and instruction f % KS; pairs of tiles of
  // values u = 3 - wave + 4 m, of two elements a lane of part k.
  constexpr int kKeys = share(2 * KS), kPairs = share(KS);
  uint32_t ko[kKeys], keo[kKeys], vo[kPairs], vso[kPairs], shift[kPairs];
  int tile[kPairs];
#pragma unroll
  for (int m = 0; m < kKeys; ++m) {
    const int f = wave + kWaves * m, i = f % KS;
    ko[m] = r * (D / 2) + g * (D / 8) + 4 * i;
    keo[m] = r * (D / 32) + (g * (D / 4) + 8 * i) / 32;
  }
#pragma unroll
  for (int m = 0; m < kPairs; ++m) {
    const int u = kWaves - 1 - wave + kWaves * m;
    int left = u;
    tile[m] = -1;
    vo[m] = vso[m] = shift[m] = 0;
#pragma unroll
    for (int k = 0; k < P::count; ++k) {
      if (left >= 0 && left < P::nib(k) / 2) {
        vo[m] = (g * (D / 8) + P::word(k, r)) * 16;
        vso[m] = (g * (D / 32) + P::word(k, r) / 4) * 4;
        shift[m] = P::shift(k, r) + 8 * left;
        tile[m] = P::tile0(k) + 2 * left;
      }
      left -= P::nib(k) / 2;
    }
  }
  struct Share {
    uint32_t kw[kKeys], ke[kKeys], vs[2][kPairs];
    u4_t v[2][kPairs];
  };
  auto fetch = [&](Share &s, int page_a, int page_b, int t) {
    const uint8_t *head[2] = {data + (int64_t)page_a * p.cache.page_stride, data + (int64_t)page_b * p.cache.page_stride};
    const uint32_t in[2] = {(uint32_t)t & (S - 1), (uint32_t)(t + 16) & (S - 1)};
#pragma unroll
    for (int m = 0; m < kKeys; ++m) {
      const int f = wave + kWaves * m;
      if (f >= 2 * KS) continue;
      const int half = f / KS;
      s.kw[m] = *reinterpret_cast<const uint32_t *>(head[half] + in[half] * (D / 2) + ko[m]);
      s.ke[m] = (head[half] + (S * D + in[half] * (D / 32)))[keo[m]];
    }
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
      if (tile[m] < 0) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s.v[k][m] = *reinterpret_cast<const u4_t *>(head[k] + (S + in[k]) * (D / 2) + vo[m]);
        s.vs[k][m] = *reinterpret_cast<const uint32_t *>(head[k] + (S * D + (S + in[k]) * (D / 32)) + vso[m]);
      }
    }
  };
  auto expand = [&](const Share &s, u4_t (*to)[64]) {
#pragma unroll
    for (int m = 0; m < kKeys; ++m) {
      const int f = wave + kWaves * m;
      if (f < 2 * KS) to[f][lane] = expand8<DT>(s.kw[m], s.ke[m] << 23);
    }
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
      if (tile[m] < 0) continue;
      uint32_t a[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        a[4 * k] = expand2<DT, 0>(s.v[k][m][0] >> shift[m], scale_of<0>(s.vs[k][m]));
        a[4 * k + 1] = expand2<DT, 0>(s.v[k][m][1] >> shift[m], scale_of<1>(s.vs[k][m]));
        a[4 * k + 2] = expand2<DT, 0>(s.v[k][m][2] >> shift[m], scale_of<2>(s.vs[k][m]));
        a[4 * k + 3] = expand2<DT, 0>(s.v[k][m][3] >> shift[m], scale_of<3>(s.vs[k][m]));
      }
      constexpr uint32_t L = 0x05040100u, H = 0x07060302u;
      to[2 * KS + tile[m]][lane] = u4_t{__builtin_amdgcn_perm(a[1], a[0], L), __builtin_amdgcn_perm(a[3], a[2], L),
                                        __builtin_amdgcn_perm(a[5], a[4], L), __builtin_amdgcn_perm(a[7], a[6], L)};
      to[2 * KS + tile[m] + 1][lane] = u4_t{__builtin_amdgcn_perm(a[1], a[0], H), __builtin_amdgcn_perm(a[3], a[2], H),
                                            __builtin_amdgcn_perm(a[5], a[4], H), __builtin_amdgcn_perm(a[7], a[6], H)};
    }
  };

  // Page numbers of 32 steps, two a step, a lane each.
  for (int s0 = f0; s0 < f1; s0 += 32) {
    const int count = min(32, f1 - s0), ahead = s0 + (lane >> 1);
    const int page = page_of(c.from + ahead * kStep + 16 * (lane & 1), ahead < f1);
    auto get = [&](Share &s, int n) {
      n = min(n, count - 1);                             // (again, behind the last)
      fetch(s, __builtin_amdgcn_readlane(page, 2 * n), __builtin_amdgcn_readlane(page, 2 * n + 1), c.from + (s0 + n) * kStep);
    };
    Share next;
    get(next, 0);
    expand(next, frag[0]);
    get(next, 1);
    __syncthreads();
    for (int n = 0; n < count; ++n) {
      // All of a product's operands are asked for before its first instruction: LDS answers after some hundred
      // cycles, which two at a time would be paid eight times.
      const u4_t(*at)[64] = frag[n & 1];
      u4_t use[2 * KS];
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) use[i] = at[i][lane];
      __builtin_amdgcn_sched_barrier(0);
      f4_t s[R][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int w = 0; w < R; ++w) s[w][half] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int w = 0; w < R; ++w) s[w][half] = mfma16<DT>(use[half * KS + i], x.q[w][i], s[w][half]);
      }
      __builtin_amdgcn_sched_barrier(0);
      static_assert(P::tiles == 2 * KS, "as many operands of values as of keys");
#pragma unroll
      for (int j = 0; j < P::tiles; ++j) use[j] = at[2 * KS + j][lane];
      __builtin_amdgcn_sched_barrier(0);
      expand(next, frag[(n + 1) & 1]);                   // (a copy of the last, behind it)
      get(next, n + 2);
      u4_t prob[R];
      x.soften(s, p.scale, prob);
#pragma unroll
      for (int j = 0; j < P::tiles; ++j)
#pragma unroll
        for (int w = 0; w < R; ++w) x.o[w][j] = mfma16<DT>(use[j], prob[w], x.o[w][j]);
      __syncthreads();
    }
  }
  // the steps that are not whole for all
  const typename T::Offsets offsets(g, r);
  for (int s = e0; s < e1; ++s) {
    if (s == f0 && f0 < f1) s = f1;
    if (s >= e1) break;
    const int t0 = c.from + s * kStep;
    typename T::Raw raw;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = t0 + 16 * k, page = page_of(t, t <= pos1 && t + 15 >= any_lo);
      T::load(raw, k, data + (int64_t)page * p.cache.page_stride, t & (S - 1), S, offsets);
    }
    x.template step<true>(raw, p.scale, t0, g, r, any_lo, pos1);
  }

  const bool nan = __any(bad);
#pragma unroll
  for (int w = 0; w < R; ++w) {
    const int row = row0 + 16 * w + r, i = row / p.G, gh = row - i * p.G;
    if (i >= tokens) continue;
    const float sum = nan ? __builtin_nanf("") : x.sum[w][0];
    // a row that saw nothing: zeros, whatever it holds
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *y = p.y + (int64_t)(c.seq.row0 + i) * p.ldy + (int64_t)(h * p.G + gh) * D;
#pragma unroll
    for (int k = 0; k < P::count; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int n = 0; n < P::nib(k); ++n) v[n] = sum == 0.f ? 0.f : x.o[w][P::tile0(k) + n][j] * inv;
        uint16_t *to = y + P::first(k, 4 * g + j);
        if (P::nib(k) == 8) store8<DT>(to, v);
        else if (P::nib(k) == 4) *reinterpret_cast<u2_t *>(to) = u2_t{round2<DT>(v[0], v[1]), round2<DT>(v[2], v[3])};
        else *reinterpret_cast<uint32_t *>(to) = round2<DT>(v[0], v[1]);
      }
  }
}

template <int DT, int D>
hipError_t launch(const KvAttnParams &p, hipStream_t s) {
  hipLaunchKernelGGL((prefill_kernel<DT, D, kv_prefill_rows(D) / (16 * kWaves)>), dim3((uint32_t)p.workgroups), dim3(kWaves * 64), 0, s, p);
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

hipError_t launch_kv_prefill(int dtype, const KvAttnParams &p, hipStream_t s) {
  return dtype == DT_F16 ? by_head<DT_F16>(p, s) : by_head<DT_BF16>(p, s);
}

}  // namespace mnb
