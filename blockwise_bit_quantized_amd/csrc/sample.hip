// sample.hip -- one token for each row of logits, by temperature, top-k, top-p and min-p, from a given number.
//
// With m the largest logit, weights are whole numbers w = rint(2^((x - m) log2(e) / temperature) 2^S) in 64
// bits, S = min(46, 62 - ceil(log2 V)), so that a row's sum stays below 2^63: their sums depend on no order (sums in 32 bits
// would move one token in some thousand rows of a flat distribution).  How exact they are, in units of 2^-S of the largest
// weight: a running sum rounds that of each eight neighbours once, V / 16 + 1 at most (of up to 1024 collected logits each
// weight, 512); the powers and their exponents are off by 3 2^-52 of a weight, V / 22 in a sum; u times the whole is rounded to 53
// bits, V / 64; and both the whole and the running sum have these errors.  So the token is the definition's where u
// times the whole lies further than V / 4 + 1024 units from every border: 2^-32 at 49152 logits, 2^-20 at 2^22.  The
// sums that find the border of top-p round each weight, V / 2: there it is 5 V / 4 + 1024.  The power is a
// polynomial in 64 bits, whose instructions run at the rate of 32-bit ones here.
//
// A workgroup of 8 or 16 waves takes a row, each wave a run of it, 512 logits a round, read again (from L2) in
// each pass.  What stays is told by one key: order bits of the number over the complement of the index.
//   A top-k of up to kMostK takes a threshold from the maxima of 256 or 1024 groups (the k-th largest
//   of them is reached by at least k logits and not many more); the logits above it go to LDS, are sorted there (or, if they
//   are few, each is compared with all by one wave), and the rest is settled by sums over them.  So do rows of up to kSort logits, and a min-p alone.
//   Otherwise the border of top-k or top-p is found by histograms: of counts or weights over equal
//   steps of the exponent (where neighbouring lanes rarely meet in one place), then in
//   the step that holds the border, whose logits are sorted, or where they are many (equal ones), halved further by
//   histograms over their order bits until one number is left, of which the first few by index stay.
//   The token itself is the place where the running sum passes u times the whole: sums of the waves, of
//   that wave's rounds (taken by all waves), of that round's lanes.
//
// Rows are bound by 64-bit instructions, about 22 a weight, on the one CU that has the row, and single rows by
// the latencies of their passes: 1 x 49152 with all filters 14 us, 1024 x 49152 by temperature 63 to 68 us (1.5 TB/s),
// 64 x 131072, of which some have no filter and some top-p alone (a weight for each logit twice, 116 us for such rows), 128 us.
#include <type_traits>

#include "decode.h"

namespace mnb {
namespace {

constexpr int kCollect = 4096;       // logits collected in LDS
constexpr int kSort = 1024;          // ... and sorted there
constexpr int kFew = 128;            // ... or settled by one wave
constexpr int kMostK = 1000;         // about 3900 logits reach the 1000th of 1024 maxima
constexpr int kFewK = 180;           // about 310 logits reach the 180th of 256 maxima (1 x 49152, 1024 against 256
                                     // groups: top-k 50 19.1 and 15.1 us, 150 33.2 and 29.2, 180 33.6 and 34.2, 250 38.5 and 43.1)
constexpr int kHeld = 6;             // rounds of a wave whose pieces stay in registers for the collection
constexpr int kBins = 2048;
constexpr int kRound = 512;          // logits of a wave's round
constexpr int kMostWaves = 16;
static_assert((1 << 22) / (kRound * 8) < kCollect, "the sums of a wave's rounds lie in LDS");

// lane ^ 1, lane ^ 2, rotated by 4 and 8 in 16 lanes
template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xf, 0xf, true);
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xf, 0xf, true);
  return (uint64_t)b << 32 | a;
}
__device__ __forceinline__ uint64_t lane64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
  v += dpp64<0xB1>(v);
  v += dpp64<0x4E>(v);
  v += dpp64<0x124>(v);
  v += dpp64<0x128>(v);
  return (lane64(v, 0) + lane64(v, 16)) + (lane64(v, 32) + lane64(v, 48));
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

// Numbers the compiler may not put into the instruction stream: a 64-bit literal costs two moves at each use,
// a scalar register pair nothing.
__device__ __forceinline__ double in_scalars(double v) {
  asm("" : "+s"(v));
  return v;
}

// Weights of a row, and their whole numbers of 2^-S.
struct Scale {
  double m, c, unit;       // unit: 2^(52 - S); adding it rounds to whole numbers of 2^-S
  double p[10], magic, low;
  int S;
  __device__ __forceinline__ Scale(double largest, double per, int fraction) {
    m = largest;
    c = per;
    S = fraction;
    unit = in_scalars(__builtin_bit_cast(double, (uint64_t)(1023 + 52 - fraction) << 52));
    magic = in_scalars(0x1.8p52);
    low = in_scalars(-100.0);
    const double q[10] = {0x1.62e42fefa3a19p-1, 0x1.ebfbdff82c598p-3, 0x1.c6b08d703ce49p-5, 0x1.3b2ab6fba1ddap-7, 0x1.5d87fe9d7a584p-10,
                          0x1.430913096fd9fp-13, 0x1.ffcb54062e698p-17, 0x1.62bfd47773353p-20, 0x1.b675bca4eeebbp-24, 0x1.e6063f7217bc6p-28};
#pragma unroll
    for (int i = 0; i < 10; ++i) p[i] = in_scalars(q[i]);
  }
  __device__ __forceinline__ double exponent(float x) const { return fmax(((double)x - m) * c, low); }
  // 2^a for a in [-100, 0]: the polynomial interpolates 2^f at the 11 Chebyshev points of [-1/2, 1/2] and is off
  // by 2^-51 of its value at most
  __device__ __forceinline__ double power(double a) const {
    const double t = a + magic;                        // the nearest whole number in the low bits
    const double f = a - (t - magic);
    double r = p[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) r = fma(r, f, p[i]);
    r = fma(r, f, 1.0);
    const uint64_t b = __builtin_bit_cast(uint64_t, r);
    const u2_t w = {(uint32_t)b, (uint32_t)(b >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, t) << 20)};
    return __builtin_bit_cast(double, w);
  }
  // a sum of weights below 2^(52 - S) as a whole number
  __device__ __forceinline__ uint64_t whole(double sum) const { return __builtin_bit_cast(uint64_t, sum + unit) & ((1ull << 52) - 1); }
  __device__ __forceinline__ uint64_t whole_weight(float x) const { return whole(power(exponent(x))); }
};

struct Shared {
  uint64_t key[kCollect];            // also sums of a wave's rounds
  unsigned long long hist[kBins];
  uint64_t wave[2 * kMostWaves];
  uint64_t chosen, before;
  float group[1024];
  uint32_t bits[kMostWaves];
  int count;
};

// sum over the workgroup
template <int WAVES>
__device__ __forceinline__ uint64_t block_sum(Shared &s, uint64_t v) {
  v = wave_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) v += s.wave[i];
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
  int V, off;              // the first piece begins `off` logits before the row, at a 16-byte boundary
  int rounds, mine;        // of a wave; this wave's first

  const Piece<DT> *edge;   // LDS: the piece with the row's first logits and that with its last, where not whole

  static constexpr uint32_t kAbsent = DT == DT_F32 ? 0xff800000u : DT == DT_F16 ? 0xfc00fc00u : 0xff80ff80u;
  // absent logits are -infinity, which weighs nothing
  __device__ __forceinline__ Piece<DT> load(int j) const { return load_at(first(j)); }
  __device__ __forceinline__ Piece<DT> load_at(int e) const {
    Piece<DT> p;
#pragma unroll
    for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) p.v[h] = u4_t{kAbsent, kAbsent, kAbsent, kAbsent};
    if (e < V) {
      const bool whole = e >= 0 && e + 8 <= V;
      if (whole) {
#pragma unroll
        for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) p.v[h] = reinterpret_cast<const u4_t *>(x + e)[h];
      } else {
        p = edge[e >= 0];
      }
    }
    return p;
  }
  // threads 0..15 write an element each of the two pieces that may not be whole
  __device__ __forceinline__ static void fill_edges(Piece<DT> *to, const T *x, int V, int off) {
    const int t = threadIdx.x, i = t & 7;
    if (t >= 16) return;
    const int e = (t < 8 ? -off : (V + off) / 8 * 8 - off) + i;
    T v;
    if constexpr (DT == DT_F32) v = -__builtin_inff();
    else v = (uint16_t)kAbsent;
    if (e >= 0 && e < V) v = x[e];
    reinterpret_cast<T *>(to + (t >> 3))[i] = v;
  }
  // the first logit of this lane's piece in round j of this wave, in round r of all
  __device__ __forceinline__ int first(int j) const { return first_of(mine + j); }
  __device__ __forceinline__ int first_of(int r) const { return r * kRound + (int)(threadIdx.x & 63) * 8 - off; }
  // f(j, piece) for each round, the next ones on their way meanwhile
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int kAhead = DT == DT_F32 ? 2 : 4;
    Piece<DT> next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i] = load(i);
    for (int j = 0; j < rounds; ++j) {
      const Piece<DT> now = next[0];
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) next[i] = next[i + 1];
      if (j + kAhead < rounds) next[kAhead - 1] = load(j + kAhead);
      f(j, now);
    }
  }
};

// the largest number of a piece
template <int DT>
__device__ __forceinline__ float piece_max(const Piece<DT> &q) {
  if constexpr (DT == DT_F16) {
    const u4_t v = q.v[0];
    const h2_t a = __builtin_elementwise_max(as_h2(v[0]), as_h2(v[1])), b = __builtin_elementwise_max(as_h2(v[2]), as_h2(v[3]));
    const h2_t c = __builtin_elementwise_max(a, b);
    return fmaxf((float)c[0], (float)c[1]);
  } else {
    float m = fmaxf(piece_at<DT>(q, 0), piece_at<DT>(q, 1));
#pragma unroll
    for (int i = 2; i < 8; i += 2) m = fmaxf(m, fmaxf(piece_at<DT>(q, i), piece_at<DT>(q, i + 1)));
    return m;
  }
}

// What stays of a row: keys at or above `least`.
struct Kept {
  uint32_t order = 0;
  int index = 0x7fffffff;          // of the numbers at `order`, those up to this index
  __device__ __forceinline__ bool holds(uint32_t o, int i) const { return (o > order) | ((o == order) & (i <= index)); }
};

// The first index, in order, at which the running sum passes goal(total); -1 where it never does.  amounts(piece, first
// index, out) gives the eight amounts of a piece as doubles, whole(sum) a sum of up to eight, rounded to a whole number:
// what is summed on is a piece's whole.
template <int WAVES, typename R, typename A, typename W, typename G>
__device__ __forceinline__ int find_index(Shared &s, const R &row, A amounts, W whole, G goal) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  auto piece_sum = [&](const auto &p, int e) -> uint64_t {
    double a[8];
    amounts(p, e, a);
#pragma unroll
    for (int i = 1; i < 8; ++i) a[i] += a[i - 1];
    return whole(a[7]);
  };
  const int half = (row.rounds + 1) / 2;
  uint64_t sum = 0, early = 0;                                    // of the second half of the wave's rounds, of the first
  row.each([&](int j, const auto &p) {
    if (j == half) {
      early = sum;
      sum = 0;
    }
    sum += piece_sum(p, row.first(j));
  });
  if (half == row.rounds) {
    early = sum;
    sum = 0;
  }
  early = wave_sum64(early);
  sum = wave_sum64(sum);
  __syncthreads();
  if (lane == 0) {
    s.wave[2 * wave] = early;
    s.wave[2 * wave + 1] = sum;
  }
  if (threadIdx.x == 0) s.count = -1;
  __syncthreads();
  uint64_t total = 0, target = 0;
#pragma unroll
  for (int i = 0; i < 2 * WAVES; ++i) total += s.wave[i];
  if (!goal(total, target) || target >= total) return -1;
  int at = 0;
  while (target >= s.wave[at]) target -= s.wave[at++];           // ends: target is below the sum of all
  // the rounds of that half
  const int from = at / 2 * row.rounds + at % 2 * half, rounds = at % 2 ? row.rounds - half : half;
  for (int j = wave; j < rounds; j += WAVES) {
    const int e = row.first_of(from + j);
    const uint64_t one = wave_sum64(piece_sum(row.load_at(e), e));
    if (lane == 0) s.key[j] = one;
  }
  __syncthreads();
  int j = 0;
  for (int j0 = 0; j0 < rounds; j0 += 64) {
    const uint64_t v = j0 + lane < rounds ? s.key[j0 + lane] : 0, run = wave_scan64(v);
    const uint64_t hit = __ballot(run > target);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      target -= lane64(run - v, l);
      j = j0 + l;
      break;
    }
    target -= lane64(run, 63);
  }
  // that round's lanes
  if (wave == 0) {
    const int e = row.first_of(from + j);
    const auto p = row.load_at(e);
    const uint64_t own = piece_sum(p, e), run = wave_scan64(own);
    if (run > target && run - own <= target) {
      // the same sums as the piece's: the last is its whole
      const uint64_t left = target - (run - own);
      int found = -1;
      double a[8];
      amounts(p, e, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i) a[i] += a[i - 1];
        if (found < 0 && whole(a[i]) > left) found = e + i;
      }
      s.count = found;
    }
  }
  __syncthreads();
  return s.count;
}

// sums over the workgroup's threads up to this one, and of all
template <int WAVES>
__device__ __forceinline__ uint64_t block_scan(Shared &s, uint64_t v, uint64_t &total) {
  v = wave_scan64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    v += i < (int)(threadIdx.x >> 6) ? s.wave[i] : 0;
    total += s.wave[i];
  }
  return v;
}

// The n keys in s.key (n up to kSort) in falling order, zeros behind them up to the power of two that is returned.
template <int WAVES>
__device__ __forceinline__ int sort_keys(Shared &s, int n) {
  int P = 64;
  while (P < n) P *= 2;
  __syncthreads();
  for (int i = n + (int)threadIdx.x; i < P; i += WAVES * 64) s.key[i] = 0;
  __syncthreads();
  for (int size = 2; size <= P; size *= 2) {
    for (int stride = size / 2; stride > 0; stride /= 2) {
      for (int q = threadIdx.x; q < P / 2; q += WAVES * 64) {
        const int i = 2 * q - (q & (stride - 1));
        const uint64_t a = s.key[i], b = s.key[i + stride];
        if ((a < b) == ((i & size) == 0)) {
          s.key[i] = b;
          s.key[i + stride] = a;
        }
      }
      // 64 neighbouring pairs stay among their 128 keys while strides are at most 64: a wave's own
      if (stride > 64 || (stride == 1 && size >= 128)) __syncthreads();
      else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
  __syncthreads();
  return P;
}

// the place of the histogram where the sum from the largest bin down (bin 0 first) reaches target: before < target <= before + it
template <int WAVES>
__device__ __forceinline__ int find_bin(Shared &s, uint64_t target, uint64_t &before) {
  constexpr int kEach = kBins / (WAVES * 64);
  __syncthreads();
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += s.hist[kEach * threadIdx.x + i];
  uint64_t run = wave_scan64(sum);
  if ((threadIdx.x & 63) == 63) s.wave[threadIdx.x >> 6] = run;
  __syncthreads();
  for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) run += s.wave[i];
  uint64_t start = run - sum + before;
  if (start < target && target <= start + sum) {
    int bin = kEach * threadIdx.x;
    while (target > start + s.hist[bin]) start += s.hist[bin++];   // ends: target is at most the sum of the thread's
    s.chosen = bin;
    s.before = start;
  }
  __syncthreads();
  before = s.before;
  return (int)s.chosen;
}

// Adds the keys of the logits of a piece whose bit is set in `mask` to s.key, as far as there is room.
template <typename P>
__device__ __forceinline__ void collect(Shared &s, const P &p, int e, uint32_t mask) {
  if (mask == 0) return;
  int n = atomicAdd(&s.count, __popc(mask));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!(mask >> i & 1)) continue;
    if (n < kCollect) s.key[n] = (uint64_t)number_order(piece_at(p, i)) << 32 | (uint32_t)~(uint32_t)(e + i);
    ++n;
  }
}

// Narrows `kept` to the shortest run of largest numbers whose amounts (1, or the weight) reach target(whole), which is at
// most the whole of what `kept` holds and weighs something.
template <int WAVES, typename R, typename F>
__device__ __forceinline__ void narrow(Shared &s, const R &row, const Scale &scale, bool weights, F target_of, Kept &kept) {
  const double steps = (kBins - 1) / (scale.S + 2.0);   // the last bin holds what weighs nothing
  auto clear = [&] {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += WAVES * 64) s.hist[i] = 0;
    __syncthreads();
  };
  auto bin_of = [&](double a) { return (int)fmin(-a * steps, (double)(kBins - 1)); };
  clear();
  row.each([&](int j, const auto &p) {
    const int e = row.first(j);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = piece_at(p, i);
      const double a = scale.exponent(x);
      const int bin = bin_of(a);
      const unsigned long long v = weights ? (unsigned long long)scale.whole(scale.power(a)) : 1ull;
      if (kept.holds(number_order(x), e + i) && bin != kBins - 1) atomicAdd(&s.hist[bin], v);
    }
  });
  if (threadIdx.x == 0) s.chosen = kBins;
  __syncthreads();
  uint64_t all = 0;
  for (int i = threadIdx.x; i < kBins; i += WAVES * 64) all += s.hist[i];
  const uint64_t target = target_of(block_sum<WAVES>(s, all));
  uint64_t before = 0;
  const int bin = find_bin<WAVES>(s, target, before);
  if (bin == kBins) return;                             // the border is among what weighs nothing: all else stays
  // those in that bin, if they are not too many, in order
  const float below = (float)fmax(scale.m - bin / (steps * scale.c), -0x1p127), from = (float)(scale.m - (bin + 1) / (steps * scale.c));
  const float slack = (fabsf(below) + fabsf((float)scale.m)) * 0x1p-20f;     // whose rounding the bin itself decides
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
  row.each([&](int j, const auto &p) {
    if (!(piece_max(p) >= from - slack)) return;
    const int e = row.first(j);
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = piece_at(p, i);
      mask |= (uint32_t)((x >= from - slack) & (x <= below + slack)) << i;
    }
    if (mask == 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = piece_at(p, i);
      if ((mask >> i & 1) && !(kept.holds(number_order(x), e + i) && bin_of(scale.exponent(x)) == bin)) mask &= ~(1u << i);
    }
    collect(s, p, e, mask);
  });
  __syncthreads();
  const int n = s.count;
  if (n <= kSort) {
    constexpr int kEach = kSort / (WAVES * 64);
    sort_keys<WAVES>(s, n);
    uint64_t w[kEach], sum = 0, total;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int a = threadIdx.x * kEach + i;
      w[i] = a >= n ? 0 : weights ? scale.whole_weight(order_number((uint32_t)(s.key[a] >> 32))) : 1;
      sum += w[i];
    }
    uint64_t run = block_scan<WAVES>(s, sum, total) - sum + before;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (run < target && target <= run + w[i]) s.chosen = s.key[threadIdx.x * kEach + i];
      run += w[i];
    }
    __syncthreads();
    kept.order = (uint32_t)(s.chosen >> 32);
    kept.index = (int)~(uint32_t)s.chosen;
    return;
  }
  // else the smallest and the largest number there, then a histogram over their order bits, until they are one
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
    for (int i = 0; i < WAVES; ++i) {
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
        atomicAdd(&s.hist[(hi - o) >> shift], weights ? (unsigned long long)scale.whole_weight(x) : 1ull);
      }
    });
    const uint32_t b = (uint32_t)find_bin<WAVES>(s, target, before);
    const uint32_t top = hi - (b << shift);
    lo = max(lo, top - (uint32_t)min((uint64_t)top, (1ull << shift) - 1));
    hi = top;
  }
  // of the numbers at the border, as many as are missing
  const uint64_t one = weights ? scale.whole_weight(order_number(lo)) : 1;
  const uint64_t need = (target - before + one - 1) / one;
  const int old = kept.order == lo ? kept.index : 0x7fffffff;
  const int at = find_index<WAVES>(s, row, [&](const auto &q, int e, double *a) {
#pragma unroll
                              for (int i = 0; i < 8; ++i) a[i] = e + i >= 0 && e + i < row.V && number_order(piece_at(q, i)) == lo ? 1.0 : 0.0;
                            },
                            [](double sum) { return (uint64_t)sum; },
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

// Leaves the k largest of the n keys in s.key (n up to kCollect, k < n), in any order: their k-th by 8 bits at a time.
template <int WAVES>
__device__ __forceinline__ void leave_largest(Shared &s, int n, int k) {
  constexpr int kEach = kCollect / (WAVES * 64);
  const int t = threadIdx.x, lane = t & 63;
  uint64_t key[kEach], prefix = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) key[i] = t + i * WAVES * 64 < n ? s.key[t + i * WAVES * 64] : 0;   // no key is 0
  uint32_t *hist = reinterpret_cast<uint32_t *>(s.hist);
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = t; i < 256; i += WAVES * 64) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (key[i] && (shift == 56 || key[i] >> (shift + 8) == prefix >> (shift + 8))) atomicAdd(&hist[255 - (key[i] >> shift & 255)], 1u);
    __syncthreads();
    // every wave: four bins a lane, the largest first
    uint32_t four[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += four[i] = hist[4 * lane + i];
    const uint32_t run = (uint32_t)wave_scan64(sum);
    const int l = __builtin_ctzll(__ballot(run >= (uint32_t)k));
    int bin = 4 * l, left = k - (int)__builtin_amdgcn_readlane((int)(run - sum), l);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = (int)__builtin_amdgcn_readlane((int)four[i], l);
      if (bin == 4 * l + i && left > c) {
        left -= c;
        ++bin;
      }
    }
    prefix |= (uint64_t)(255 - bin) << shift;
    k = left;
    __syncthreads();
  }
  if (t == 0) s.count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (key[i] >= prefix && key[i]) s.key[atomicAdd(&s.count, 1)] = key[i];
  __syncthreads();
}

// The row's token from the n logits of s.key (n up to kFew), among them all that may stay, by one wave: each of a lane's
// logits against all, for its rank and the sum of the larger ones, then for the sum of those before it.
__device__ __forceinline__ void settle_few(Shared &s, int n, const Scale &scale, int top_k, float top_p, double least, float u, int64_t *token) {
  constexpr int kEach = kFew / 64;
  const int lane = threadIdx.x;
  uint64_t *weight = reinterpret_cast<uint64_t *>(s.hist);
  uint64_t key[kEach], w[kEach], before[kEach] = {};
  double r[kEach];
  int rank[kEach] = {};
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int a = lane + 64 * k;
    key[k] = a < n ? s.key[a] : 0;
    r[k] = a < n ? scale.power(scale.exponent(order_number((uint32_t)(key[k] >> 32)))) : 0.0;
    w[k] = scale.whole(r[k]);
    if (a < n) weight[a] = w[k];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const uint64_t other = s.key[i], amount = weight[i];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const bool larger = other > key[k];
      rank[k] += larger;
      before[k] += larger ? amount : 0;
    }
  }
  uint64_t sum = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (top_k > 0 && rank[k] >= top_k) w[k] = 0;
    sum += w[k];
  }
  const double want = top_p < 1.f ? ceil((double)top_p * (double)wave_sum64(sum)) : 0x1p64;
  sum = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (rank[k] != 0 && !((double)before[k] < want && r[k] >= least)) w[k] = 0;
    sum += w[k];
  }
  const uint64_t goal = goal_of(u, wave_sum64(sum));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (lane + 64 * k < n) weight[lane + 64 * k] = w[k];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  uint64_t run[kEach] = {};                                       // larger complements of the index come first
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const uint32_t other = (uint32_t)s.key[i];
    const uint64_t amount = weight[i];
#pragma unroll
    for (int k = 0; k < kEach; ++k) run[k] += other >= (uint32_t)key[k] ? amount : 0;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (w[k] && run[k] > goal && run[k] - w[k] <= goal) *token = (int64_t)(uint32_t)~(uint32_t)key[k];
}

// The row's token from the n logits of s.key (n up to kSort), among them all that may stay: in the order of the numbers, what top-k, top-p and
// min-p leave; then in the order of the index, where the running sum passes.
template <int WAVES>
__device__ __forceinline__ void settle(Shared &s, int n, const Scale &scale, int top_k, float top_p, double least, float u, int64_t *token) {
  constexpr int kEach = kSort / (WAVES * 64);
  const int P = sort_keys<WAVES>(s, n), each = (P + WAVES * 64 - 1) / (WAVES * 64), first = threadIdx.x * each;
  if (top_k > 0 && n > top_k) n = top_k;
  uint64_t key[kEach], w[kEach], sum = 0, all;
  double r[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    w[i] = 0;
    if (i >= each || first + i >= n) continue;
    key[i] = s.key[first + i];
    r[i] = scale.power(scale.exponent(order_number((uint32_t)(key[i] >> 32))));
    sum += w[i] = scale.whole(r[i]);
  }
  uint64_t before = block_scan<WAVES>(s, sum, all) - sum;
  const double want = top_p < 1.f ? ceil((double)top_p * (double)all) : 0x1p64;
  sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i >= each || first + i >= P) continue;
    const bool stays = w[i] && (first + i == 0 || ((double)before < want && r[i] >= least));
    before += w[i];
    // the index counted down over the weight, of S + 1 bits: S and the index's bits are 62
    const uint64_t back = ((1ull << (62 - scale.S)) - 1 - (uint32_t)~(uint32_t)key[i]) << (scale.S + 1);
    s.key[first + i] = stays ? back | w[i] : 0;
    sum += stays ? w[i] : 0;
  }
  const uint64_t goal = goal_of(u, block_sum<WAVES>(s, sum));
  sort_keys<WAVES>(s, P);
  sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i >= each || first + i >= P) continue;
    key[i] = s.key[first + i];
    sum += w[i] = key[i] & ((2ull << scale.S) - 1);
  }
  uint64_t run = block_scan<WAVES>(s, sum, all) - sum;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i >= each || first + i >= P) continue;
    if (run <= goal && goal < run + w[i]) *token = (int64_t)((1ull << (62 - scale.S)) - 1 - (key[i] >> (scale.S + 1)));
    run += w[i];
  }
}

// largest number and largest magnitude's bits (past infinity's for a NaN) of a piece, added to those before
template <int DT>
struct Largest {
  float m = -__builtin_inff();
  uint32_t bits = 0;
  h2_t pair = {(_Float16)-__builtin_inff(), (_Float16)-__builtin_inff()};
  typedef uint16_t us2_t __attribute__((ext_vector_type(2)));
  us2_t pair_bits = {0, 0};
  __device__ __forceinline__ void add(const Piece<DT> &q) {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, piece_at(q, i));
        bits = max(bits, q.v[i >> 2][i & 3] & 0x7fffffffu);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = q.v[0][i];
        pair_bits = __builtin_elementwise_max(pair_bits, __builtin_bit_cast(us2_t, w & 0x7fff7fffu));
        if constexpr (DT == DT_F16) pair = __builtin_elementwise_max(pair, as_h2(w));
        else m = fmaxf(m, fmaxf(__builtin_bit_cast(float, w << 16), __builtin_bit_cast(float, w & 0xffff0000u)));
      }
    }
  }
  __device__ __forceinline__ void finish() {
    if constexpr (DT == DT_F16) m = fmaxf((float)pair[0], (float)pair[1]);
    if constexpr (DT != DT_F32) {
      const uint32_t b = max(pair_bits[0], pair_bits[1]);
      bits = DT == DT_BF16 ? b << 16 : b > 0x7c00u ? 0x7fc00000u : 0;
    }
  }
};

template <int DT, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 4) void sample_kernel(SampleParams p, int fraction) {
  __shared__ Shared s;
  __shared__ Piece<DT> edge[2];
  const int64_t at = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, V = p.V;
  typedef typename Elem<DT>::type T;
  Row<DT> row;
  row.x = static_cast<const T *>(p.x) + at * p.ldl;
  row.V = V;
  row.off = (int)((uintptr_t)row.x % 16 / sizeof(T));
  row.rounds = (V + row.off + WAVES * kRound - 1) / (WAVES * kRound);
  row.mine = __builtin_amdgcn_readfirstlane(wave) * row.rounds;
  row.edge = edge;
  row.fill_edges(edge, row.x, V, row.off);
  __syncthreads();
  const float u = p.u[at], temperature = p.temperature ? p.temperature[at] : p.temperature_all;
  const float top_p = p.top_p ? p.top_p[at] : p.top_p_all, min_p = p.min_p ? p.min_p[at] : p.min_p_all;
  int top_k = p.top_k ? p.top_k[at] : p.top_k_all;
  if (top_k >= V) top_k = 0;

  // the largest logit, whether all are numbers, and the maxima of 1024 lanes, or half lanes with 8 waves
  Piece<DT> held[kHeld];
  const bool holds = row.rounds <= kHeld;
  Largest<DT> all, second;
  if (holds) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (j < row.rounds) held[j] = row.load(j);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j >= row.rounds) continue;
      if (WAVES == 8 && (j & 1)) second.add(held[j]);
      else all.add(held[j]);
    }
  } else {
    row.each([&](int j, const auto &q) {
      if (WAVES == 8 && (j & 1)) second.add(q);
      else all.add(q);
    });
  }
  all.finish();
  s.group[t] = all.m;
  float m = all.m;
  uint32_t bits = all.bits;
  if constexpr (WAVES == 8) {
    second.finish();
    s.group[t + 512] = second.m;
    m = fmaxf(m, second.m);
    bits = max(bits, second.bits);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) bits = max(bits, (uint32_t)__shfl_xor((int)bits, d));
  if (lane == 0) s.bits[wave] = bits;
  if (t == 0) s.count = 0;
  __syncthreads();
  float four[4];                                                  // of 256 groups
#pragma unroll
  for (int i = 0; i < 4; ++i)
    four[i] = fmaxf(fmaxf(s.group[lane + 64 * i], s.group[lane + 64 * i + 256]), fmaxf(s.group[lane + 64 * i + 512], s.group[lane + 64 * i + 768]));
  m = fmaxf(fmaxf(four[0], four[1]), fmaxf(four[2], four[3]));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
#pragma unroll
  for (int i = 0; i < WAVES; ++i) bits = max(bits, s.bits[i]);
  if (bits > 0x7f800000u || __builtin_isinf(m) || !(temperature >= 0.f) || __builtin_isinf(temperature) || u != u || top_p != top_p ||
      min_p != min_p) {
    if (t == 0) p.tokens[at] = -1;
    return;
  }
  if (temperature == 0.f) {                                       // the first of the largest
    const int found = find_index<WAVES>(s, row, [&](const auto &q, int e, double *a) {
#pragma unroll
                                        for (int i = 0; i < 8; ++i) a[i] = e + i >= 0 && e + i < V && piece_at(q, i) == m ? 1.0 : 0.0;
                                 },
                                 [](double sum) { return (uint64_t)sum; },
                                 [](uint64_t, uint64_t &goal) { goal = 0; return true; });
    if (t == 0) p.tokens[at] = found;
    return;
  }
  Scale scale(m, 1.4426950408889634 / (double)temperature, fraction);
  const double least = fmin((double)min_p, 1.0);

  // a threshold that all that may stay reach, and few others
  float above = __builtin_nanf("");
  if (V <= kSort) above = -__builtin_inff();
  else if (top_k > 0 && top_k <= kMostK) {
    // the largest 16-bit prefix of order bits that top_k maxima reach
    uint32_t found = 0;
    auto reach = [&](auto count, auto value) {
      constexpr int N = decltype(count)::value;
      uint32_t o[N];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = number_order(value(i)) >> 16;
      for (int bit = 15; bit >= 0; --bit) {
        const uint32_t test = found | 1u << bit;
        int c = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) c += __popcll(__ballot(o[i] >= test));
        if (c >= top_k) found = test;
      }
    };
    if (top_k <= kFewK) reach(std::integral_constant<int, 4>(), [&](int i) { return four[i]; });
    else reach(std::integral_constant<int, 16>(), [&](int i) { return s.group[lane + 64 * i]; });
    above = found <= number_order(-__builtin_inff()) >> 16 ? -__builtin_inff() : order_number(found << 16);
  } else if (top_k <= 0 && top_p >= 1.f && min_p > 0.f) {
    // a little below the least that stays, whose weight decides
    above = (float)((double)m + log2(fmin((double)min_p, 1.0)) / scale.c);
    above -= fabsf(above) * 0x1p-20f + fabsf(m) * 0x1p-20f;
  }
  if (above == above) {
    auto take = [&](int j, const auto &q) {
      if (!(piece_max(q) >= above)) return;
      const int e = row.first(j);
      uint32_t mask = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mask |= (uint32_t)((piece_at(q, i) >= above) & (e + i >= 0) & (e + i < V)) << i;
      collect(s, q, e, mask);
    };
    if (holds) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (j < row.rounds) take(j, held[j]);
    } else {
      row.each(take);
    }
    __syncthreads();
    int n = s.count;
    __syncthreads();
    if (n <= kFew) {
      if (wave == 0) settle_few(s, n, scale, top_k, top_p, least, u, p.tokens + at);
      return;
    }
    if (n > kSort && n <= kCollect && top_k > 0 && top_k <= kSort) {
      leave_largest<WAVES>(s, n, top_k);
      n = top_k;
    }
    if (n <= kSort) {
      settle<WAVES>(s, n, scale, top_k, top_p, least, u, p.tokens + at);
      return;
    }
  }

  Kept kept;
  for (int weights = 0; weights < 2; ++weights) {                 // top-k, then top-p
    if (weights ? top_p >= 1.f : top_k <= 0) continue;
    narrow<WAVES>(s, row, scale, weights != 0, [&](uint64_t all) -> uint64_t {
      if (!weights) return (uint64_t)top_k;
      const double want = ceil((double)top_p * (double)all);
      return want < 1.0 ? 1 : want < (double)all ? (uint64_t)want : all;
    }, kept);
  }
  const auto goal = [&](uint64_t total, uint64_t &target) { target = goal_of(u, total); return true; };
  const auto whole = [&](double sum) { return scale.whole(sum); };
  int found;
  if (kept.order == 0 && !(least > 0.0)) {
    found = find_index<WAVES>(s, row, [&](const auto &q, int, double *a) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = scale.power(scale.exponent(piece_at(q, i)));
    }, whole, goal);
  } else {
    found = find_index<WAVES>(s, row, [&](const auto &q, int e, double *a) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = piece_at(q, i);
        const double r = scale.power(scale.exponent(x));
        const bool stays = (r >= least) & kept.holds(number_order(x), e + i);
        a[i] = stays ? r : 0.0;
      }
    }, whole, goal);
  }
  if (t == 0) p.tokens[at] = found;
}

template <int DT>
hipError_t launch(const SampleParams &p, int fraction, hipStream_t s) {
  const dim3 grid((uint32_t)p.M);
  // 8 waves leave a CU two rows at a time: 1024 x 49152 by temperature 64.5 us (16 waves: 81.2), with top-p 174 (219); a row
  // alone on its CU is faster with 16: 64 x 131072 with top-p 116 (8 waves: 132)
  if (p.M > kCUs) hipLaunchKernelGGL((sample_kernel<DT, 8>), grid, dim3(512), 0, s, p, fraction);
  else hipLaunchKernelGGL((sample_kernel<DT, 16>), grid, dim3(1024), 0, s, p, fraction);
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
