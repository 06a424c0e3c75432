// sample.hip -- one token for each row of logits, by temperature, top-k, top-p and min-p, from a given number.
//
// With m the largest logit, weights are whole numbers w = rint(2^((x - m) log2(e) / temperature) 2^S) in 64
// bits, S such that a row's sum stays below 2^63: their sums do not depend on an order, and a token is that of the
// 64-bit definition unless u falls within about 2^-40 of a border between two tokens (sums in 32 bits
// would move one in some thousand rows of a flat distribution).
//   top-k  the k-th largest number: its 32 order bits eight at a time, a histogram of counts each;
//   top-p  the same with a histogram of weights;
//   both leave a border number, of which only the first few by index stay.
#include "decode.h"

namespace mnb {
namespace {

constexpr int kThreads = 1024, kSampleWaves = kThreads / 64;

__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor((unsigned long long)v, d);
  return v;
}

struct Row {
  uint64_t *part;                        // LDS, kSampleWaves
  __device__ uint64_t sum(uint64_t v) const {
    v = wave_sum64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kSampleWaves; ++i) v += part[i];
    return v;
  }
  __device__ uint64_t largest(uint64_t v) const {
    v = wave_max64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kSampleWaves; ++i) v = part[i] > v ? part[i] : v;
    return v;
  }
  // sum over the threads up to this one, and of all
  __device__ uint64_t scan(uint64_t v, uint64_t &total) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t o = __shfl_up((unsigned long long)v, d);
      if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) part[wave] = v;
    __syncthreads();
    total = 0;
    for (int i = 0; i < kSampleWaves; ++i) {
      if (i < wave) v += part[i];
      total += part[i];
    }
    return v;
  }
};

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleParams p, int fraction) {
  typedef typename Elem<DT>::type T;
  __shared__ uint64_t part[kSampleWaves];
  __shared__ unsigned long long hist[256];
  __shared__ uint32_t chosen;
  __shared__ uint64_t chosen_before;
  __shared__ int token;
  const Row sum{part};
  const int64_t row = blockIdx.x;
  const int V = p.V, t = threadIdx.x;
  const T *x = static_cast<const T *>(p.x) + row * p.ldl;
  const float u = p.u[row], temperature = p.temperature ? p.temperature[row] : p.temperature_all;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p_all;
  float min_p = p.min_p ? p.min_p[row] : p.min_p_all;
  const int top_k = p.top_k ? p.top_k[row] : p.top_k_all;

  uint64_t best = 0;
  for (int i = t; i < V; i += kThreads) {
    const uint64_t k = (uint64_t)number_order(to_f32<DT>(x[i])) << 32 | (uint32_t)~(uint32_t)i;
    best = k > best ? k : best;
  }
  best = sum.largest(best);
  const uint32_t top = (uint32_t)(best >> 32);
  const float m = __builtin_bit_cast(float, top & 0x80000000u ? top ^ 0x80000000u : ~top);
  if (top == kOrderNan || __builtin_isinf(m) || !(temperature >= 0.f) || __builtin_isinf(temperature) || u != u || top_p != top_p ||
      min_p != min_p) {
    if (t == 0) p.tokens[row] = -1;
    return;
  }
  if (temperature == 0.f) {
    if (t == 0) p.tokens[row] = (int64_t)(uint32_t)~(uint32_t)best;
    return;
  }
  min_p = fminf(min_p, 1.f);
  const double c = 1.4426950408889634 / (double)temperature, one = (double)(1ull << fraction);
  auto weight = [&](float v) -> uint64_t {
    const double e = exp2(((double)v - (double)m) * c);
    return e >= (double)min_p ? (uint64_t)rint(e * one) : 0;
  };
  auto raw_weight = [&](float v) -> uint64_t { return (uint64_t)rint(exp2(((double)v - (double)m) * c) * one); };

  // what stays: numbers above `border` and the first `ties` of those at it
  uint32_t border = 0;
  uint32_t ties = 0xffffffffu;
  // the number where the running sum, from the largest down, of amounts (1 or the weight) passes `target`
  auto descend = [&](uint64_t target, bool weights, uint64_t &before) {
    uint32_t prefix = 0;
    before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = t; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = t; i < V; i += kThreads) {
        const float v = to_f32<DT>(x[i]);
        const uint32_t o = number_order(v);
        if (o < border) continue;
        if (shift < 24 && o >> (shift + 8) != prefix >> (shift + 8)) continue;
        // numbers at an earlier border count as if all stayed: the target is at most what does
        atomicAdd(&hist[o >> shift & 255], weights ? (unsigned long long)raw_weight(v) : 1ull);
      }
      __syncthreads();
      // 256 threads: the sum of the larger ones
      if (t < 256) {
        uint64_t above = before;
        for (int i = 255; i > t; --i) above += hist[i];
        if (above < target && target <= above + hist[t]) {
          chosen = prefix | (uint32_t)t << shift;
          chosen_before = above;
        }
      }
      __syncthreads();
      prefix = chosen;
      before = chosen_before;
      __syncthreads();
    }
    return prefix;
  };
  if (top_k > 0 && top_k < V) {
    uint64_t before;
    border = descend((uint64_t)top_k, false, before);
    ties = (uint32_t)(top_k - before);
  }
  if (top_p < 1.f) {
    uint64_t mine = 0, at = 0;
    for (int i = t; i < V; i += kThreads) {
      const float v = to_f32<DT>(x[i]);
      const uint32_t o = number_order(v);
      if (o > border) mine += raw_weight(v);
      else if (o == border) ++at;
    }
    const uint64_t larger = sum.sum(mine), equal = sum.sum(at);
    const float bv = __builtin_bit_cast(float, border & 0x80000000u ? border ^ 0x80000000u : ~border);
    const uint64_t bw = border ? raw_weight(bv) : 0;
    const uint64_t all = larger + bw * (equal < ties ? equal : ties);
    const double want = ceil((double)top_p * (double)all);
    uint64_t target = want < 1.0 ? 1 : (uint64_t)want;
    if (target > all) target = all;
    uint64_t before;
    const uint32_t at_border = border;
    const uint32_t now = descend(target, true, before);
    const float nv = __builtin_bit_cast(float, now & 0x80000000u ? now ^ 0x80000000u : ~now);
    const uint64_t w = raw_weight(nv), need = (target - before + w - 1) / w;
    ties = now == at_border && need > ties ? ties : (uint32_t)need;
    border = now;
  }
  // the whole of what stays, and the token where the running sum passes u times it
  uint64_t mine = 0, at = 0;
  for (int i = t; i < V; i += kThreads) {
    const float v = to_f32<DT>(x[i]);
    const uint32_t o = number_order(v);
    if (o > border) mine += weight(v);
    else if (o == border) ++at;
  }
  const uint64_t larger = sum.sum(mine), equal = sum.sum(at);
  const float bv = __builtin_bit_cast(float, border & 0x80000000u ? border ^ 0x80000000u : ~border);
  const uint64_t bw = border ? weight(bv) : 0;
  const uint64_t all = larger + bw * (equal < ties ? equal : ties);
  const double place = (double)u * (double)all;
  uint64_t goal = place <= 0.0 ? 0 : (uint64_t)place;     // the first token whose running sum is above
  if (goal >= all) goal = all - 1;
  if (t == 0) token = -1;
  uint64_t done = 0, seen = 0;
  for (int i0 = 0; i0 < V; i0 += kThreads) {
    const int i = i0 + t;
    const float v = i < V ? to_f32<DT>(x[i]) : 0.f;
    const uint32_t o = i < V ? number_order(v) : 0;
    uint64_t total = 0, w = 0;
    const bool tie = i < V && o == border && border;
    const uint64_t before = sum.scan(tie, total) - tie + seen;
    seen += total;
    if (i < V && (o > border || (tie && before < ties))) w = weight(v);
    const uint64_t run = sum.scan(w, total) + done;
    if (w && run > goal && run - w <= goal) token = i;
    done += total;
    if (done > goal) break;
  }
  __syncthreads();
  if (t == 0) p.tokens[row] = token;
}

}  // namespace

hipError_t launch_sample(int dtype, const SampleParams &p, hipStream_t s) {
  int bits = 0;
  while ((1ll << bits) < p.V) ++bits;
  const int fraction = 62 - bits;
  const dim3 grid((uint32_t)p.M), block(kThreads);
  if (dtype == DT_F16) hipLaunchKernelGGL((sample_kernel<DT_F16>), grid, block, 0, s, p, fraction);
  else if (dtype == DT_BF16) hipLaunchKernelGGL((sample_kernel<DT_BF16>), grid, block, 0, s, p, fraction);
  else hipLaunchKernelGGL((sample_kernel<DT_F32>), grid, block, 0, s, p, fraction);
  return hipGetLastError();
}

}  // namespace mnb
