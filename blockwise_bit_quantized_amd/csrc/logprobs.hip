// logprobs.hip -- log probabilities of given tokens, entropy and the largest alternatives of
// each row of logits, in one pass over the data.
//
// With m = max x, S = sum exp(x - m), T = sum exp(x - m) (x - m):
//   logprob = x[token] - m - log S,   entropy = log S - T / S.
// A workgroup holds its part of a row (E pieces of 8 elements a thread) in registers, so
// the logits are read once: the maximum first, then S and T against it.
//
// Alternatives.  An element's key is its order-preserving bits over the complement of its
// index: keys are distinct and order by value, then by the lower index.  The largest key of
// each of 64 groups of threads is known after the maximum pass; the top-th largest of those
// 64 is a threshold that at least `top` elements reach, and few more do (about 64 ln(64 /
// (64 - top)) of an unordered row).  Elements at or above it are collected in LDS and ranked
// by counting larger ones, which does not depend on the order of collection.  If they do not
// fit (rows arranged so that one group holds most large values), the workgroup takes the
// maxima one at a time below the last one taken instead.
//
// Rows longer than one workgroup holds, and calls with few rows, split each row; the parts'
// (m, S, T) and keys go through the workspace and a second kernel joins them in part order.
#include "ops.h"

namespace mnb {
namespace {

constexpr int kCap = 512;       // collected candidates
constexpr float kLog2e = 1.4426950408889634f;

// order-preserving bits: larger number, larger integer; every NaN above +infinity, both
// zeros alike, nothing maps to 0 (the key of an absent element)
__device__ __forceinline__ uint32_t order_bits(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);   // -0 becomes +0
  const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return f != f ? 0xffffffffu : u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);   // 0xffffffff: a NaN
}
__device__ __forceinline__ uint64_t make_key(uint32_t u, uint32_t index) { return (uint64_t)u << 32 | (uint32_t)~index; }

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// one piece of 8 elements as loaded
template <int DT> struct Piece { u4_t v[DT == DT_F32 ? 2 : 1]; };
template <int DT>
__device__ __forceinline__ float piece_at(const Piece<DT> &q, int i) {
  if constexpr (DT == DT_F32) return __builtin_bit_cast(float, (uint32_t)q.v[i >> 2][i & 3]);
  else return to_f32<DT>((uint16_t)(q.v[0][i >> 1] >> (16 * (i & 1))));
}

// the row's results from (m, S, T)
__device__ __forceinline__ void write_row(const LogprobsParams &p, int64_t row, float m, float S, float T, float xt) {
  const float ls = logf(S);
  if (p.tokens) {
    const int64_t tok = p.tokens[row];
    p.logprob[row] = tok < 0 ? 0.f : tok >= p.V ? __builtin_nanf("") : (xt - m) - ls;
  }
  if (p.entropy) p.entropy[row] = ls - T / S;
}
template <int DT>
__device__ __forceinline__ float token_logit(const LogprobsParams &p, int64_t row) {
  if (!p.tokens) return 0.f;
  const int64_t tok = p.tokens[row];
  if (tok < 0 || tok >= p.V) return 0.f;
  return to_f32<DT>(static_cast<const typename Elem<DT>::type *>(p.x)[row * p.ldl + tok]);
}

template <int DT, int WAVES, int E>
__global__ __launch_bounds__(WAVES * 64) void part_kernel(LogprobsParams p) {
  constexpr int THREADS = WAVES * 64;
  typedef typename Elem<DT>::type T;
  __shared__ uint64_t thread_key[THREADS];
  __shared__ uint64_t cand[kCap];
  __shared__ float red[WAVES][2];
  __shared__ uint64_t wave_key[WAVES];
  __shared__ uint64_t threshold;
  __shared__ int count;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t row = blockIdx.x / p.chunks;
  const int part = (int)(blockIdx.x - row * p.chunks);
  const int c0 = part * p.chunk, c1 = min(p.V, c0 + p.chunk);   // this part's elements
  const T *x = static_cast<const T *>(p.x) + row * p.ldl;
  // pieces start at 16-byte boundaries: `skew` elements before c0 are not this part's
  constexpr int kAlign = 16 / (int)sizeof(T);
  const int skew = (int)(((uintptr_t)(x + c0) / sizeof(T)) % kAlign);
  const int first = c0 - skew;

  const float ninf = -__builtin_inff();
  Piece<DT> q[E];
  auto present = [&](int j, int i) {
    const int e = first + (j * THREADS + t) * 8 + i;
    return e >= c0 && e < c1;
  };
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int e = first + (j * THREADS + t) * 8;
    if (e >= c0 && e + 8 <= c1) {
#pragma unroll
      for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) q[j].v[h] = reinterpret_cast<const u4_t *>(x + e)[h];
    } else {
      // at a part's ends: absent elements are -infinity, which adds nothing to any sum
      uint32_t w[DT == DT_F32 ? 8 : 4] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        T v = from_f32<DT>(ninf);
        if (e + i >= c0 && e + i < c1) v = x[e + i];
        if constexpr (DT == DT_F32) w[i] = __builtin_bit_cast(uint32_t, v);
        else w[i >> 1] |= (uint32_t)v << (16 * (i & 1));
      }
#pragma unroll
      for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) q[j].v[h] = u4_t{w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
    }
  }

  // the thread's largest key below `limit`
  auto best_below = [&](uint64_t limit) {
    uint64_t best = 0;
#pragma unroll
    for (int j = 0; j < E; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t k = make_key(order_bits(piece_at<DT>(q[j], i)), (uint32_t)(first + (j * THREADS + t) * 8 + i));
        if (present(j, i) && k < limit && k > best) best = k;
      }
    return best;
  };
  const uint64_t mine = best_below(~0ull);
  const uint64_t wk = wave_max(mine);
  if (lane == 0) wave_key[wave] = wk;
  thread_key[t] = mine;
  if (t == 0) count = 0;
  __syncthreads();
  uint64_t top_key = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) top_key = wave_key[i] > top_key ? wave_key[i] : top_key;
  const float m = order_value((uint32_t)(top_key >> 32));
  // a part of -infinities: shift by 0, so that its terms are 0 and not NaN
  const float shift = m == ninf ? 0.f : m;

  float S = 0.f, Tn = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    float s = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = piece_at<DT>(q[j], i) - shift;
      const float e = __builtin_amdgcn_exp2f(d * kLog2e);
      s += e;
      u += e * fmaxf(d, -1e4f);   // e is 0 there: 0, and not 0 times infinity
    }
    S += s;
    Tn += u;
  }
  S = wave_sum(S);
  Tn = wave_sum(Tn);
  if (lane == 0) {
    red[wave][0] = S;
    red[wave][1] = Tn;
  }

  if (p.top > 0 && wave == 0) {
    // the group of lane l: threads l, l + 64, ...
    uint64_t gk = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) gk = thread_key[i * 64 + lane] > gk ? thread_key[i * 64 + lane] : gk;
    int larger = 0;
    for (int i = 0; i < 64; ++i) {
      const uint64_t o = __shfl((unsigned long long)gk, i);
      larger += o > gk || (o == gk && i < lane);   // groups with nothing share key 0
    }
    if (larger == p.top - 1) threshold = gk;
  }
  __syncthreads();
  S = Tn = 0.f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    S += red[i][0];
    Tn += red[i][1];
  }

  const int64_t slot = row * p.chunks + part;
  const float ls = logf(S);
  auto emit = [&](int rank, uint64_t k) {
    if (p.chunks > 1) p.keys[slot * p.top + rank] = k;
    else {
      p.top_tokens[row * p.top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
      p.top_logprobs[row * p.top + rank] = (order_value((uint32_t)(k >> 32)) - m) - ls;
    }
  };
  if (p.top > 0) {
    const uint64_t thr = threshold;
    if (mine >= thr && mine != 0) {
#pragma unroll
      for (int j = 0; j < E; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t k = make_key(order_bits(piece_at<DT>(q[j], i)), (uint32_t)(first + (j * THREADS + t) * 8 + i));
          if (present(j, i) && k >= thr) {
            const int at = atomicAdd(&count, 1);
            if (at < kCap) cand[at] = k;
          }
        }
    }
    __syncthreads();
    const int n = count;
    if (n <= kCap) {
      for (int a = t; a < n; a += THREADS) {
        const uint64_t k = cand[a];
        int rank = 0;
        for (int o = 0; o < n; ++o) rank += cand[o] > k;
        if (rank < p.top) emit(rank, k);
      }
      // a part with fewer elements than `top`: the rest of its slots are absent
      for (int a = n + t; a < p.top; a += THREADS) emit(a, 0);
    } else {
      uint64_t limit = ~0ull;
      for (int rank = 0; rank < p.top; ++rank) {
        const uint64_t b = wave_max(best_below(limit));
        __syncthreads();
        if (lane == 0) wave_key[wave] = b;
        __syncthreads();
        limit = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) limit = wave_key[i] > limit ? wave_key[i] : limit;
        if (t == 0) emit(rank, limit);
      }
    }
  }
  if (t == 0) {
    if (p.chunks > 1) *reinterpret_cast<f4_t *>(p.part + slot * 4) = f4_t{m, S, Tn, 0.f};
    else write_row(p, row, m, S, Tn, token_logit<DT>(p, row));
  }
}

// joins the parts of a row: one workgroup of 256 threads per row
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(LogprobsParams p) {
  extern __shared__ uint64_t keys[];   // [chunks * top]
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const f4_t *part = reinterpret_cast<const f4_t *>(p.part) + row * p.chunks;
  const int n = p.chunks * p.top;
  for (int i = t; i < n; i += 256) keys[i] = p.keys[row * n + i];
  // every thread joins the sums in part order, so all hold the same values
  float m = -__builtin_inff();
  bool nan = false;
  for (int i = 0; i < p.chunks; ++i) {
    const float mi = part[i][0];
    nan = nan || mi != mi;
    m = fmaxf(m, mi);
  }
  if (nan) m = __builtin_nanf("");
  float S = 0.f, T = 0.f;
  for (int i = 0; i < p.chunks; ++i) {
    const f4_t v = part[i];
    if (v[0] == -__builtin_inff() && v[1] == 0.f) continue;   // nothing but -infinity
    const float d = v[0] - m;
    const float f = __builtin_amdgcn_exp2f(d * kLog2e);
    S += f * v[1];
    if (f != 0.f) T += f * (v[2] + d * v[1]);   // (x - m_i) + (m_i - m)
  }
  const float ls = logf(S);
  if (t == 0) write_row(p, row, m, S, T, token_logit<DT>(p, row));
  __syncthreads();
  for (int a = t; a < n; a += 256) {
    const uint64_t k = keys[a];
    if (k == 0) continue;
    int rank = 0;
    for (int o = 0; o < n; ++o) rank += keys[o] > k;
    if (rank < p.top) {
      p.top_tokens[row * p.top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
      p.top_logprobs[row * p.top + rank] = (order_value((uint32_t)(k >> 32)) - m) - ls;
    }
  }
}

// Elements one workgroup can hold after an unaligned start (up to 7 elements before it).
constexpr int held(int threads, int e) { return threads * e * 8 - 8; }

template <int DT>
hipError_t launch(const LogprobsParams &p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.M * p.chunks));
  if (p.chunk <= held(256, 2)) hipLaunchKernelGGL((part_kernel<DT, 4, 2>), grid, dim3(256), 0, s, p);
  else if (p.chunk <= held(1024, 2)) hipLaunchKernelGGL((part_kernel<DT, 16, 2>), grid, dim3(1024), 0, s, p);
  else hipLaunchKernelGGL((part_kernel<DT, 16, 7>), grid, dim3(1024), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.chunks == 1) return e;
  hipLaunchKernelGGL((join_kernel<DT>), dim3((uint32_t)p.M), dim3(256), (uint32_t)(p.chunks * p.top * sizeof(uint64_t)), s, p);
  return hipGetLastError();
}

}  // namespace

// Parts of a row and their length (a multiple of 8): whole rows of up to 57336 elements when
// the rows fill the chip, else parts short enough for about two workgroups per CU.
int logprobs_chunks(int M, int V, int dtype, int *chunk) {
  (void)dtype;
  const int sizes[] = {held(256, 2), held(1024, 2), held(1024, 7)};
  for (int i = 0; i < 3; ++i) {
    const int64_t parts = ((int64_t)V + sizes[i] - 1) / sizes[i];
    // at most 64 parts, so that the joining kernel's keys fit LDS (64 x 32 x 8 bytes)
    if (i == 2 || (parts <= 32 && (parts == 1 || (int64_t)M * parts <= 4 * kCUs))) {
      *chunk = sizes[i];
      return (int)parts;
    }
  }
  return 1;
}

hipError_t launch_logprobs(int dtype, const LogprobsParams &p, hipStream_t s) {
  return dtype == DT_F16 ? launch<DT_F16>(p, s) : dtype == DT_BF16 ? launch<DT_BF16>(p, s) : launch<DT_F32>(p, s);
}

}  // namespace mnb
