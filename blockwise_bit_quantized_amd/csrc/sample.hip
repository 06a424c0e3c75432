// sample.hip -- one token for each row of logits, by temperature, top-k, top-p and min-p, from a given number.
//
// With m the largest logit, weights are whole numbers w = rint(2^((x - m) log2(e) / temperature) 2^S) in 64
// bits, S such that a row's sum stays below 2^63: their sums depend on no order, and a token is that of the
// 64-bit definition unless u falls within about 2^-40 of a border between two tokens (sums in 32 bits
// would move one in some thousand rows of a flat distribution).  The power is a polynomial in 64 bits, whose
// instructions run at the rate of 32-bit ones here.
//
// A workgroup of 16 waves takes a row, thread t pieces of 8 logits t, t + 1024, ..., read again (from L2) in
// each pass.  What stays is told by one key: order bits of the number over the complement of the index.
//   A top-k of up to kFewK takes a threshold from the maxima of 256 groups of threads (the k-th largest
//   of them is reached by at least k logits and few more); the logits above it go to LDS, and everything
//   is settled among them by counting, for each, the larger ones.  So do rows of up to kList logits, and a min-p alone.
//   Otherwise the border of top-k or top-p is found by histograms: of counts or weights over equal
//   steps of the exponent (where neighbouring lanes rarely meet in one place), then over the order bits in
//   the step that holds the border, until one number is left; of that, the first few by index stay.
//   The token itself is the place where the running sum passes u times the whole: sums of waves, then of lanes.
#include "decode.h"

namespace mnb {
namespace {

constexpr int kThreads = 1024, kSampleWaves = kThreads / 64;
constexpr int kList = 1024;          // logits settled in LDS
constexpr int kFewK = 180;           // about 310 of 256 groups' logits pass the 180th maximum
constexpr int kBins = 2048;
constexpr int kRound = kThreads * 8; // logits of a round of pieces
constexpr int kRounds = 64;          // rounds whose sums of waves lie in LDS

__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor((unsigned long long)v, d);
  return v;
}
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up((unsigned long long)v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ float order_number(uint32_t u) { return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// 2^a for a in [-100, 0], times 2^S, before rounding: the polynomial interpolates 2^f at the 11 Chebyshev points of
// [-1/2, 1/2] and is off by 2^-51 of its value at most.
__device__ __forceinline__ double power(double a, int S) {
  const double t = a + 0x1.8p52;                       // the nearest whole number in the low bits
  const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
  const double f = a - (t - 0x1.8p52);
  double r = 0x1.e6063f7217bc6p-28;
  r = fma(r, f, 0x1.b675bca4eeebbp-24);
  r = fma(r, f, 0x1.62bfd47773353p-20);
  r = fma(r, f, 0x1.ffcb54062e698p-17);
  r = fma(r, f, 0x1.430913096fd9fp-13);
  r = fma(r, f, 0x1.5d87fe9d7a584p-10);
  r = fma(r, f, 0x1.3b2ab6fba1ddap-7);
  r = fma(r, f, 0x1.c6b08d703ce49p-5);
  r = fma(r, f, 0x1.ebfbdff82c598p-3);
  r = fma(r, f, 0x1.62e42fefa3a19p-1);
  r = fma(r, f, 1.0);
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, r) + ((uint64_t)(uint32_t)(n + S) << 52));
}

struct Scale {
  double m, c, least;      // weights below `least` (min-p) count 0
  int S;
  __device__ __forceinline__ double exponent(float x) const { return fmax(((double)x - m) * c, -100.0); }
  // rounded to a whole number, as a double: sums of a thread stay exact
  __device__ __forceinline__ double weight(float x) const {
    const double r = power(exponent(x), S);
    return r >= least ? (r + 0x1p52) - 0x1p52 : 0.0;
  }
};

struct Shared {
  uint64_t key[kList];               // also sums of waves
  uint64_t amount[kList];
  unsigned long long hist[kBins];
  uint64_t wave[kSampleWaves];
  uint64_t chosen, before;
  float group[256];
  uint32_t bits[kSampleWaves];
  int count;
};

// sum over the workgroup
__device__ __forceinline__ uint64_t block_sum(Shared &s, uint64_t v) {
  v = wave_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kSampleWaves; ++i) v += s.wave[i];
  return v;
}

template <int DT> struct Piece { u4_t v[DT == DT_F32 ? 2 : 1]; };
template <int DT>
__device__ __forceinline__ float piece_at(const Piece<DT> &q, int i) {
  if constexpr (DT == DT_F32) return __builtin_bit_cast(float, (uint32_t)q.v[i >> 2][i & 3]);
  else return to_f32<DT>((uint16_t)(q.v[0][i >> 1] >> (16 * (i & 1))));
}

template <int DT>
struct Row {
  typedef typename Elem<DT>::type T;
  const T *x;
  int V, rounds, off;      // the first piece begins `off` logits before the row, at a 16-byte boundary

  // absent logits are -infinity, which weighs nothing
  __device__ __forceinline__ Piece<DT> load(int j) const {
    constexpr uint32_t absent = DT == DT_F32 ? 0xff800000u : DT == DT_F16 ? 0xfc00fc00u : 0xff80ff80u;
    Piece<DT> p;
    const int e = first(j);
    if (e >= 0 && e + 8 <= V) {
#pragma unroll
      for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) p.v[h] = reinterpret_cast<const u4_t *>(x + e)[h];
      return p;
    }
#pragma unroll
    for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) p.v[h] = u4_t{absent, absent, absent, absent};
    if (e >= V || e + 8 <= 0) return p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e + i < 0 || e + i >= V) continue;
      if constexpr (DT == DT_F32) p.v[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, x[e + i]);
      else p.v[0][i >> 1] = (p.v[0][i >> 1] & (0xffffu << (16 * (1 - (i & 1))))) | (uint32_t)x[e + i] << (16 * (i & 1));
    }
    return p;
  }
  __device__ __forceinline__ int first(int j) const { return j * kRound + (int)threadIdx.x * 8 - off; }
  // f(j, piece) for each round, the next piece on its way meanwhile
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    Piece<DT> now = load(0);
    for (int j = 0; j < rounds; ++j) {
      const Piece<DT> next = j + 1 < rounds ? load(j + 1) : now;
      f(j, now);
      now = next;
    }
  }
};

// What stays of a row: keys at or above `least`.
struct Kept {
  uint32_t order = 0;
  int index = 0x7fffffff;          // of the numbers at `order`, those up to this index
  __device__ __forceinline__ bool holds(uint32_t o, int i) const { return o > order || (o == order && i <= index); }
};

// The first index, in order, at which the running sum of amount(x, index) passes goal(total); -1 where it never does.
template <typename R, typename A, typename G>
__device__ __forceinline__ int find_index(Shared &s, R &row, A amount, G goal) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int per = (row.rounds + kRounds - 1) / kRounds;          // rounds of an entry: 1 but for very long rows
  auto piece_sum = [&](int j, const auto &p) {
    double sum = 0.0;
    const int e = row.first(j);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += amount(piece_at(p, i), e + i);
    return (uint64_t)sum;
  };
  __syncthreads();
  if (per > 1) {
    for (int i = threadIdx.x; i < kRounds * kSampleWaves; i += kThreads) s.key[i] = 0;
    __syncthreads();
  }
  row.each([&](int j, const auto &p) {
    const uint64_t sum = wave_sum64(piece_sum(j, p));
    if (lane != 0) return;
    if (per == 1) s.key[j * kSampleWaves + wave] = sum;
    else atomicAdd(reinterpret_cast<unsigned long long *>(&s.key[j / per * kSampleWaves]), (unsigned long long)sum);
  });
  __syncthreads();
  // every wave scans the entries, 64 at a time, and so finds the same one
  auto scan = [&](int n, uint64_t &target, bool &set, uint64_t &total) -> int {
    uint64_t done = 0;
    for (int i0 = 0; i0 < n; i0 += 64) {
      const uint64_t v = i0 + lane < n ? s.key[i0 + lane] : 0, run = wave_scan64(v) + done;
      if (set) {
        const uint64_t hit = __ballot(run > target);
        if (hit) {
          const int at = __builtin_ctzll(hit);
          target -= __shfl((unsigned long long)(run - v), at);
          return i0 + at;
        }
      }
      done = __shfl((unsigned long long)run, 63);
    }
    total = done;
    return -1;
  };
  uint64_t total = 0, target = 0;
  bool set = false;
  const int entries = per == 1 ? row.rounds * kSampleWaves : kRounds * kSampleWaves;
  scan(entries, target, set, total);
  if (!goal(total, target)) return -1;
  set = true;
  int at = scan(entries, target, set, total);
  if (at < 0) return -1;
  if (per > 1) {                                                  // the rounds of that entry, one sum a wave each
    const int j0 = at / kSampleWaves * per, j1 = min(row.rounds, j0 + per);
    __syncthreads();
    for (int j = j0; j < j1; ++j) {
      const uint64_t sum = wave_sum64(piece_sum(j, row.load(j)));
      if (lane == 0) s.key[(j - j0) * kSampleWaves + wave] = sum;
    }
    __syncthreads();
    at = scan((j1 - j0) * kSampleWaves, target, set, total);
    if (at < 0) return -1;
    at += j0 * kSampleWaves;
  }
  const int j = at / kSampleWaves;
  __syncthreads();
  if (wave == at % kSampleWaves) {
    const auto p = row.load(j);
    const uint64_t mine = piece_sum(j, p), run = wave_scan64(mine);
    if (run > target && run - mine <= target) {
      uint64_t left = target - (run - mine);
      int found = -1;
      const int e = row.first(j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t a = (uint64_t)amount(piece_at(p, i), e + i);
        if (found < 0 && a > left) found = e + i;
        left -= found < 0 ? a : 0;
      }
      s.count = found;
    }
  }
  __syncthreads();
  return s.count;
}

// the place of the histogram where the sum from the largest bin down (bin 0 first) reaches target: before < target <= before + it
__device__ __forceinline__ int find_bin(Shared &s, uint64_t target, uint64_t &before) {
  static_assert(kBins == 2 * kThreads, "two bins a thread");
  __syncthreads();
  const uint64_t a = s.hist[2 * threadIdx.x], b = s.hist[2 * threadIdx.x + 1];
  uint64_t run = wave_scan64(a + b);
  if ((threadIdx.x & 63) == 63) s.wave[threadIdx.x >> 6] = run;
  __syncthreads();
  for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) run += s.wave[i];
  const uint64_t start = run - a - b + before;
  if (start < target && target <= start + a + b) {
    const bool second = target > start + a;
    s.chosen = 2 * threadIdx.x + second;
    s.before = start + (second ? a : 0);
  }
  __syncthreads();
  before = s.before;
  return (int)s.chosen;
}

// Narrows `kept` to the shortest run of largest numbers whose amounts (1, or the weight) reach target, at most
// what `kept` holds in all.
template <typename R>
__device__ __forceinline__ void narrow(Shared &s, R &row, const Scale &scale, bool weights, uint64_t target, Kept &kept) {
  const double steps = (kBins - 1) / (scale.S + 2.0);   // the last bin holds what weighs nothing
  auto clear = [&] {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
    __syncthreads();
  };
  auto bin_of = [&](double a) { return (int)fmin(-a * steps, (double)(kBins - 1)); };
  clear();
  row.each([&](int j, const auto &p) {
    const int e = row.first(j);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = piece_at(p, i);
      if (!kept.holds(number_order(x), e + i)) continue;
      const double a = scale.exponent(x);
      const int bin = bin_of(a);
      if (bin == kBins - 1) continue;
      atomicAdd(&s.hist[bin], weights ? (unsigned long long)((power(a, scale.S) + 0x1p52) - 0x1p52) : 1ull);
    }
  });
  if (threadIdx.x == 0) s.chosen = kBins;
  uint64_t before = 0;
  const int bin = find_bin(s, target, before);
  if (bin == kBins) return;                             // the border is among what weighs nothing: all else stays
  // in that bin: the smallest and the largest number, then a histogram over their order bits, until they are one
  uint32_t lo = 0, hi = 0xffffffffu;
  while (true) {
    uint32_t least = 0xffffffffu, most = 0;
    row.each([&](int j, const auto &p) {
      const int e = row.first(j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = piece_at(p, i);
        const uint32_t o = number_order(x);
        if (o < lo || o > hi || !kept.holds(o, e + i) || bin_of(scale.exponent(x)) != bin) continue;
        least = min(least, o);
        most = max(most, o);
      }
    });
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      least = min(least, (uint32_t)__shfl_xor((int)least, d));
      most = max(most, (uint32_t)__shfl_xor((int)most, d));
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.wave[threadIdx.x >> 6] = (uint64_t)least << 32 | most;
    __syncthreads();
    for (int i = 0; i < kSampleWaves; ++i) {
      least = min(least, (uint32_t)(s.wave[i] >> 32));
      most = max(most, (uint32_t)s.wave[i]);
    }
    lo = least;
    hi = most;
    if (lo >= hi) break;
    const int shift = max(0, 21 - __builtin_clz(hi - lo));       // (hi - lo) >> shift < 2048
    clear();
    row.each([&](int j, const auto &p) {
      const int e = row.first(j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = piece_at(p, i);
        const uint32_t o = number_order(x);
        if (o < lo || o > hi || !kept.holds(o, e + i)) continue;
        atomicAdd(&s.hist[(hi - o) >> shift], weights ? (unsigned long long)((power(scale.exponent(x), scale.S) + 0x1p52) - 0x1p52) : 1ull);
      }
    });
    const uint32_t b = (uint32_t)find_bin(s, target, before);
    const uint32_t top = hi - (b << shift);
    lo = max(lo, top - (uint32_t)min((uint64_t)top, (1ull << shift) - 1));
    hi = top;
  }
  // of the numbers at the border, as many as are missing
  const uint64_t one = weights ? (uint64_t)((power(scale.exponent(order_number(lo)), scale.S) + 0x1p52) - 0x1p52) : 1;
  const uint64_t need = (target - before + one - 1) / one;
  const int old = kept.order == lo ? kept.index : 0x7fffffff;
  const int at = find_index(s, row, [&](float x, int i) { return i >= 0 && i < row.V && number_order(x) == lo ? 1.0 : 0.0; },
                            [&](uint64_t total, uint64_t &goal) { goal = need - 1; return need < total; });
  kept.order = lo;
  kept.index = at < 0 ? old : min(at, old);
}

// u times the whole, rounded down, below the whole
__device__ __forceinline__ uint64_t goal_of(float u, uint64_t all) {
  const double place = (double)u * (double)all;
  const uint64_t g = place <= 0.0 ? 0 : (uint64_t)place;
  return g < all ? g : all - 1;
}

// The row's token from the n logits of s.key, all that may stay: for each, sums over the larger ones and over those before it.
__device__ __forceinline__ void settle(Shared &s, int n, const Scale &scale, int top_k, float top_p, double least, float u, int64_t *token) {
  const int t = threadIdx.x;
  const bool on = t < n;
  const uint64_t key = on ? s.key[t] : 0;
  const double r = on ? power(scale.exponent(order_number((uint32_t)(key >> 32))), scale.S) : 0.0;
  uint64_t w = (uint64_t)((r + 0x1p52) - 0x1p52);
  if (on) s.amount[t] = w;
  __syncthreads();
  int rank = 0;
  uint64_t before = 0;
  if (on) {
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const bool larger = s.key[i] > key;
      rank += larger;
      before += larger ? s.amount[i] : 0;
    }
  }
  bool stays = on && (top_k <= 0 || rank < top_k);
  if (top_p < 1.f) {
    const uint64_t all = block_sum(s, stays ? w : 0);
    const double want = ceil((double)top_p * (double)all);
    stays = stays && (rank == 0 || (want >= 1.0 && before < (uint64_t)want));
  }
  stays = stays && (rank == 0 || r >= least);
  w = stays ? w : 0;
  const uint64_t goal = goal_of(u, block_sum(s, w));              // its barriers also end the reads of s.amount
  if (on) s.amount[t] = w;
  __syncthreads();
  if (w == 0) return;
  uint64_t run = 0;                                               // of those up to this one: larger complements first
  const uint32_t mine = (uint32_t)key;
#pragma unroll 4
  for (int i = 0; i < n; ++i) run += (uint32_t)s.key[i] >= mine ? s.amount[i] : 0;
  if (run > goal && run - w <= goal) *token = (int64_t)(uint32_t)~mine;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleParams p, int fraction) {
  __shared__ Shared s;
  const int64_t at = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, V = p.V;
  typedef typename Elem<DT>::type T;
  Row<DT> row;
  row.x = static_cast<const T *>(p.x) + at * p.ldl;
  row.V = V;
  row.off = (int)((uintptr_t)row.x % 16 / sizeof(T));
  row.rounds = (V + row.off + kRound - 1) / kRound;
  const float u = p.u[at], temperature = p.temperature ? p.temperature[at] : p.temperature_all;
  const float top_p = p.top_p ? p.top_p[at] : p.top_p_all, min_p = p.min_p ? p.min_p[at] : p.min_p_all;
  int top_k = p.top_k ? p.top_k[at] : p.top_k_all;
  if (top_k >= V) top_k = 0;

  // the largest logit, whether all are numbers, and the maxima of 256 groups of four threads
  float m = -__builtin_inff();
  uint32_t bits = 0;                                              // of the largest magnitude: past infinity's for a NaN
  row.each([&](int, const auto &q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = piece_at(q, i);
      m = fmaxf(m, x);
      bits = max(bits, __builtin_bit_cast(uint32_t, x) & 0x7fffffffu);
    }
  });
  float g = fmaxf(m, __shfl_xor(m, 1));
  g = fmaxf(g, __shfl_xor(g, 2));
  if ((t & 3) == 0) s.group[t >> 2] = g;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) bits = max(bits, (uint32_t)__shfl_xor((int)bits, d));
  if (lane == 0) s.bits[wave] = bits;
  if (t == 0) s.count = 0;
  __syncthreads();
  float four[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) four[i] = s.group[lane + 64 * i];
  m = fmaxf(fmaxf(four[0], four[1]), fmaxf(four[2], four[3]));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
#pragma unroll
  for (int i = 0; i < kSampleWaves; ++i) bits = max(bits, s.bits[i]);
  if (bits > 0x7f800000u || __builtin_isinf(m) || !(temperature >= 0.f) || __builtin_isinf(temperature) || u != u || top_p != top_p ||
      min_p != min_p) {
    if (t == 0) p.tokens[at] = -1;
    return;
  }
  if (temperature == 0.f) {                                       // the first of the largest
    const int found = find_index(s, row, [&](float x, int i) { return i >= 0 && i < V && x == m ? 1.0 : 0.0; },
                                 [](uint64_t, uint64_t &goal) { goal = 0; return true; });
    if (t == 0) p.tokens[at] = found;
    return;
  }
  Scale scale;
  scale.m = m;
  scale.c = 1.4426950408889634 / (double)temperature;
  scale.S = fraction;
  scale.least = 0.0;
  const double one = (double)(1ull << fraction), least = fmin((double)min_p, 1.0) * one;

  // a threshold that all that may stay reach, and few others
  float above = __builtin_nanf("");
  if (V <= kList) above = -__builtin_inff();
  else if (top_k > 0 && top_k <= kFewK) {
    uint32_t o[4], found = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = number_order(four[i]) >> 16;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {                         // the largest 16-bit prefix that top_k maxima reach
      const uint32_t test = found | 1u << bit;
      int c = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) c += __popcll(__ballot(o[i] >= test));
      if (c >= top_k) found = test;
    }
    above = found <= number_order(-__builtin_inff()) >> 16 ? -__builtin_inff() : order_number(found << 16);
  } else if (top_k <= 0 && top_p >= 1.f && min_p > 0.f) {
    // a little below the least that stays, whose weight decides
    above = (float)((double)m + log2(fmin((double)min_p, 1.0)) / scale.c);
    above -= fabsf(above) * 0x1p-20f + fabsf(m) * 0x1p-20f;
  }
  if (above == above) {
    row.each([&](int j, const auto &q) {
      const int e = row.first(j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = piece_at(q, i);
        if (x >= above && e + i >= 0 && e + i < V) {
          const int n = atomicAdd(&s.count, 1);
          if (n < kList) s.key[n] = (uint64_t)number_order(x) << 32 | (uint32_t)~(uint32_t)(e + i);
        }
      }
    });
    __syncthreads();
    if (s.count <= kList) {
      settle(s, s.count, scale, top_k, top_p, least, u, p.tokens + at);
      return;
    }
  }

  Kept kept;
  for (int weights = 0; weights < 2; ++weights) {                 // top-k, then top-p
    uint64_t target = (uint64_t)top_k;
    if (weights ? top_p >= 1.f : top_k <= 0) continue;
    if (weights) {
      double mine = 0.0;
      row.each([&](int j, const auto &q) {
        const int e = row.first(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = piece_at(q, i);
          if (kept.holds(number_order(x), e + i)) mine += scale.weight(x);
        }
      });
      const uint64_t all = block_sum(s, (uint64_t)mine);
      const double want = ceil((double)top_p * (double)all);
      target = want < 1.0 ? 1 : (uint64_t)want;
      if (target > all) target = all;
    }
    narrow(s, row, scale, weights != 0, target, kept);
  }
  scale.least = least;
  const int found = find_index(s, row, [&](float x, int i) { return kept.holds(number_order(x), i) ? scale.weight(x) : 0.0; },
                               [&](uint64_t total, uint64_t &goal) { goal = goal_of(u, total); return true; });
  if (t == 0) p.tokens[at] = found;
}

template <int DT>
hipError_t launch(const SampleParams &p, int fraction, hipStream_t s) {
  const dim3 grid((uint32_t)p.M), block(kThreads);
  hipLaunchKernelGGL((sample_kernel<DT>), grid, block, 0, s, p, fraction);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(int dtype, const SampleParams &p, hipStream_t s) {
  int bits = 0;
  while ((1ll << bits) < p.V) ++bits;
  const int fraction = 62 - bits < 46 ? 62 - bits : 46;           // weights and a thread's sums stay whole in 53 bits
  return dtype == DT_F16 ? launch<DT_F16>(p, fraction, s) : dtype == DT_BF16 ? launch<DT_BF16>(p, fraction, s) : launch<DT_F32>(p, fraction, s);
}

}  // namespace mnb
