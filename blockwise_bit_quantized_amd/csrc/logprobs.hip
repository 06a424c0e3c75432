// logprobs.hip -- log probabilities of given tokens, entropy and the largest alternatives of
// each row of logits, in one pass over the data.
//
// With m = max x, S = sum exp(x - m), T = sum exp(x - m) (x - m):
//   logprob = x[token] - m - log S,   entropy = log S - T / S.
// A workgroup holds its part of a row (E pieces of 8 elements a thread) in registers, so
// the logits are read once: the maximum first, then S and T against it.
//
// Alternatives.  The maxima of 64 groups of threads come with the maximum pass; the top-th
// largest of them is a threshold that at least `top` elements reach and few more do (about
// 64 ln(64 / (64 - top)) of an unordered row).  Elements at or above it are collected in LDS as
// keys, order-preserving bits over the complement of the index, which are distinct and order by
// value, then by the lower index; each is ranked by counting larger ones, so the order
// of collection does not matter.  Where too many reach the threshold,
//   * equal values (masked tokens at -infinity, say) are taken in index order, only as many
//     as are missing, after the larger ones;
//   * if the larger ones alone are too many (one group holds most large values), or the row holds
//     a NaN or +infinity, the keys are taken one at a time, each the largest below the last.
//
// Bound by memory and vector instructions together for many rows (1024 x 49152 fp16, top 20:
// 101 MB in 27 to 28.5 us, 3.6 TB/s, while the instructions take 40 to 60% of the SIMDs' cycles; bfloat16
// 30.5, fp32 55.7), by the chain of reductions for one row (49152: 7.2 us, bfloat16 8.5, fp32 8.1).
//
// Rows longer than one workgroup holds are split; the parts' (m, S, T) and keys go through the
// workspace and a second kernel joins them in part order (one row of 50257 8.6 us, of 131072 10.6, of 262144
// 10.2; 1024 rows of 131072 fp16 65, fp32 137).  A last part with elements in fewer threads than
// give `top` groups has no threshold and takes its keys one at a time: 1024 rows of 50257, whose
// last parts hold 1105, take 110 us for top 20 (fp32 333).
#include "ops.h"

namespace mnb {
namespace {

constexpr int kCap = 512;       // collected candidates
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// order-preserving bits: larger number, larger integer; every NaN above +infinity, both
// zeros alike.  Nothing maps to 0 (the key of an absent element), and a NaN is not the largest
// integer: at index 0 its key would be all ones, which no search for a key below a limit finds.
constexpr uint32_t kNanBits = 0xfffffffeu;
__device__ __forceinline__ uint32_t order_bits(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);   // -0 becomes +0
  const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return f != f ? kNanBits : u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);   // kNanBits: a NaN
}
__device__ __forceinline__ uint64_t make_key(uint32_t u, uint32_t index) { return (uint64_t)u << 32 | (uint32_t)~index; }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// lane ^ 1, lane ^ 2, mirrored in 8 lanes, rotated by 4 and 8 in 16
constexpr int kQuad1 = 0xB1, kQuad2 = 0x4E, kMirror8 = 0x141, kRor4 = 0x124, kRor8 = 0x128;
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// the maximum of each group of 4, 8 or 16 lanes, in all of them
template <int N>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp<kQuad1>(v));
  v = fmaxf(v, dpp<kQuad2>(v));
  if constexpr (N == 8) v = fmaxf(v, dpp<kMirror8>(v));
  if constexpr (N == 16) {
    v = fmaxf(v, dpp<kRor4>(v));
    v = fmaxf(v, dpp<kRor8>(v));
  }
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  v = group_max<16>(v);
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kQuad1>(v);
  v += dpp<kQuad2>(v);
  v += dpp<kRor4>(v);
  v += dpp<kRor8>(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// How many of n keys in LDS are larger than `k`, counted by 8 neighbouring lanes that share k; the
// 8 lanes run it together.  (One lane alone waits for LDS once a key: 320 keys took 10 us.)
__device__ __forceinline__ int count_larger(const uint64_t *keys, int n, uint64_t k, int lane) {
  int c = 0;
#pragma unroll 4
  for (int o = lane & 7; o < n; o += 8) c += keys[o] > k;
  c += __builtin_amdgcn_update_dpp(0, c, kQuad1, 0xf, 0xf, true);
  c += __builtin_amdgcn_update_dpp(0, c, kQuad2, 0xf, 0xf, true);
  return c + __builtin_amdgcn_update_dpp(0, c, kMirror8, 0xf, 0xf, true);
}

// one piece of 8 elements as loaded
template <int DT> struct Piece { u4_t v[DT == DT_F32 ? 2 : 1]; };
template <int DT>
__device__ __forceinline__ float piece_at(const Piece<DT> &q, int i) {
  if constexpr (DT == DT_F32) return __builtin_bit_cast(float, (uint32_t)q.v[i >> 2][i & 3]);
  else return to_f32<DT>((uint16_t)(q.v[0][i >> 1] >> (16 * (i & 1))));
}

// An empty use: what a later pass computes from the piece is computed again, not carried
// over in registers (the converted values would halve the workgroups per CU).
template <int DT>
__device__ __forceinline__ void forget(Piece<DT> &q) {
  asm volatile("" : "+v"(q.v[0]));
  if constexpr (DT == DT_F32) asm volatile("" : "+v"(q.v[1]));
}
// its largest number (a NaN is passed over unless all are)
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
__global__ __launch_bounds__(WAVES * 64, DT == DT_F32 || WAVES < 8 ? 1 : 4) void part_kernel(LogprobsParams p) {
  constexpr int THREADS = WAVES * 64, GROUP = THREADS / 64;
  typedef typename Elem<DT>::type T;
  __shared__ uint64_t cand[kCap];
  __shared__ float group[64];
  __shared__ int larger[64];             // how many groups have a larger maximum
  __shared__ float red[WAVES][2];
  __shared__ uint64_t wave_key[WAVES];
  __shared__ int wave_count[WAVES];
  __shared__ int count;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t row = blockIdx.x / p.chunks;
  const int part = (int)(blockIdx.x - row * p.chunks);
  const int c0 = part * p.chunk, c1 = min(p.V, c0 + p.chunk);   // this part's elements
  const T *x = static_cast<const T *>(p.x) + row * p.ldl;
  // pieces of 8 from the first 16-byte boundary; the up to 7 elements before it and the up to 7
  // behind the last whole piece go one each to threads 0..15
  constexpr int kAlign = 16 / (int)sizeof(T);
  const int a0 = min(c1, c0 + (int)(-(uintptr_t)(x + c0) / sizeof(T) % kAlign));
  const int a1 = a0 + (c1 - a0) / 8 * 8;
  const int rounds = (a1 - a0 + THREADS * 8 - 1) / (THREADS * 8);   // pieces per thread: uniform
  const int mine0 = a0 + t * 8;          // this thread's first element

  const float ninf = -__builtin_inff();
  Piece<DT> q[E];
#pragma clang loop unroll(full)
  for (int j = 0; j < E; ++j) {
    if (j >= rounds) continue;
    const int e = mine0 + j * (THREADS * 8);
    // absent elements are -infinity, which adds nothing to any sum
    const uint32_t absent = DT == DT_F32 ? 0xff800000u : DT == DT_F16 ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
    for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) {
      q[j].v[h] = u4_t{absent, absent, absent, absent};
      if (e < a1) q[j].v[h] = reinterpret_cast<const u4_t *>(x + e)[h];
    }
  }
  const int edge_at = t < 8 ? c0 + t : a1 + t - 8;
  const bool has_edge = t < 8 ? edge_at < a0 : t < 16 && edge_at < c1;
  const float edge = has_edge ? to_f32<DT>(x[edge_at]) : ninf;

  float mine = fmaxf(edge, ninf);        // (a NaN is passed over)
#pragma clang loop unroll(full)
  for (int j = 0; j < E; ++j) {
    if (j >= rounds) continue;
    mine = fmaxf(mine, piece_max<DT>(q[j]));
  }
  const float gm = group_max<GROUP>(mine);
  if (lane % GROUP == 0) group[t / GROUP] = gm;
  if (t < 64) larger[t] = 0;
  if (t == 0) count = 0;
  __syncthreads();
  const float g = group[lane];            // every wave holds the 64 group maxima
  const float m = wave_max(g);
  // a part of -infinities: shift by 0, so that its terms are 0 and not NaN
  const float shift = m == ninf ? 0.f : m;
  if (p.top > 0) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 64 / WAVES; ++i) {
      const int o = wave * (64 / WAVES) + i;
      const float v = lane_value(g, o);
      n += v > g || (v == g && o < lane);
    }
    atomicAdd(&larger[lane], n);
  }

  // Exponents are x log2(e) - fl(m log2(e)), one fused operation an element; the rounding of the
  // constant, `off`, is the same in all of them and is taken out of the sums.  (Not for the wider
  // types, whose m log2(e) may overflow.)
  constexpr bool kFused = DT == DT_F16;
  const float base = shift * kLog2e, off = kFused && base < 1e30f ? fmaf(shift, kLog2e, -base) : 0.f;
  float S = 0.f, Tn = 0.f;                // Tn in units of log 2
  auto add = [&](float v, float &s, float &u) {
    const float d = kFused ? fmaf(v, kLog2e, -base) : (v - shift) * kLog2e;
    const float e = __builtin_amdgcn_exp2f(d);
    s += e;
    u = fmaf(e, fmaxf(d, -1e4f), u);      // e is 0 there: 0, and not 0 times infinity
  };
  add(edge, S, Tn);
#pragma clang loop unroll(full)
  for (int j = 0; j < E; ++j) {
    if (j >= rounds) continue;
    float s = 0.f, u = 0.f;
    forget<DT>(q[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) add(piece_at<DT>(q[j], i), s, u);
    S += s;
    Tn += u;
  }
  S = wave_sum(S);
  Tn = wave_sum(Tn);
  if (lane == 0) {
    red[wave][0] = S;
    red[wave][1] = Tn;
  }
  __syncthreads();
  S = Tn = 0.f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    S += red[i][0];
    Tn += red[i][1];
  }
  if constexpr (kFused) {
    const float f = __builtin_amdgcn_exp2f(-off);
    Tn = (Tn - off * S) * f;
    S *= f;
  }
  Tn *= kLn2;

  const int64_t slot = row * p.chunks + part;
  const float ls = logf(S);
  if (t == 0) {
    if (p.chunks > 1) *reinterpret_cast<f4_t *>(p.part + slot * 4) = f4_t{m, S, Tn, 0.f};
    else write_row(p, row, m, S, Tn, token_logit<DT>(p, row));
  }
  if (p.top == 0) return;

  auto emit = [&](int rank, uint64_t k) {
    if (p.chunks > 1) p.keys[slot * p.top + rank] = k;
    else {
      p.top_tokens[row * p.top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
      p.top_logprobs[row * p.top + rank] = (order_value((uint32_t)(k >> 32)) - m) - ls;
    }
  };
  // collects the elements above the threshold (and, with `ties`, those equal to it)
  const float thr = lane_value(g, __builtin_ctzll(__ballot(larger[lane] == p.top - 1)));
  auto collect = [&](bool ties) {
    auto offer = [&](float v, int at) {
      if (ties ? v >= thr : v > thr) {
        const int n = atomicAdd(&count, 1);
        if (n < kCap) cand[n] = make_key(order_bits(v), (uint32_t)at);
      }
    };
    if (has_edge) offer(edge, edge_at);
#pragma clang loop unroll(full)
    for (int j = 0; j < E; ++j) {
      if (j >= rounds) continue;
      forget<DT>(q[j]);
      const int e = mine0 + j * (THREADS * 8);
      if (e < a1 && piece_max<DT>(q[j]) >= thr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) offer(piece_at<DT>(q[j], i), e + i);
      }
    }
  };
  auto rank_all = [&](int n) {
    for (int a = t / 8; a < n; a += THREADS / 8) {
      const uint64_t k = cand[a];
      const int rank = count_larger(cand, n, k, lane);
      if ((lane & 7) == 0 && rank < p.top) emit(rank, k);
    }
  };

  int n = 0;
  bool one_by_one = S != S;              // a NaN or +infinity in the row
  if (!one_by_one) {
    if (mine >= thr) collect(true);
    __syncthreads();
    n = count;
    if (n <= kCap) {
      rank_all(n);
      // a part with fewer elements than `top`: the rest of its slots are absent
      for (int a = n + t; a < p.top; a += THREADS) emit(a, 0);
      return;
    }
    __syncthreads();
    if (t == 0) count = 0;
    __syncthreads();
    if (mine > thr) collect(false);
    __syncthreads();
    n = count;
    one_by_one = n > kCap;
  }
  // both rare forms read the logits again, one element per thread
  if (!one_by_one) {
    // all larger ones are in; equal ones in index order until `top` are
    int need = p.top - n;                // at most 0 if the larger ones suffice
    for (int e0 = c0; e0 < c1 && need > 0; e0 += THREADS) {
      const int e = e0 + t;
      const bool eq = e < c1 && to_f32<DT>(x[e]) == thr;
      const uint64_t who = __ballot(eq);
      if (lane == 0) wave_count[wave] = __popcll(who);
      __syncthreads();
      int at = __popcll(who & ((1ull << lane) - 1)), total = 0;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) {
        at += i < wave ? wave_count[i] : 0;
        total += wave_count[i];
      }
      if (eq && at < need) cand[n + at] = make_key(order_bits(thr), (uint32_t)e);
      const int took = min(total, need);
      n += took;
      need -= took;
      __syncthreads();                   // wave_count may be written again, cand read
    }
    rank_all(n);
    return;
  }
  uint64_t limit = ~0ull;
  for (int rank = 0; rank < p.top; ++rank) {
    uint64_t best = 0;
    for (int e = c0 + t; e < c1; e += THREADS) {
      const uint64_t k = make_key(order_bits(to_f32<DT>(x[e])), (uint32_t)e);
      if (k < limit && k > best) best = k;
    }
    best = wave_max(best);
    __syncthreads();
    if (lane == 0) wave_key[wave] = best;
    __syncthreads();
    limit = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) limit = wave_key[i] > limit ? wave_key[i] : limit;
    if (t == 0) emit(rank, limit);
  }
}

// joins the parts of a row: one workgroup per row; LDS holds the row's parts and
// keys, so that the loops over them wait for memory once
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS) void join_kernel(LogprobsParams p) {
  extern __shared__ uint64_t keys[];   // [chunks * top], then the parts
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int n = p.chunks * p.top;
  f4_t *part = reinterpret_cast<f4_t *>(keys + (n + 1) / 2 * 2);
  for (int i = t; i < p.chunks; i += THREADS) part[i] = reinterpret_cast<const f4_t *>(p.part)[row * p.chunks + i];
  for (int i = t; i < n; i += THREADS) keys[i] = p.keys[row * n + i];
  const float xt = t == 0 ? token_logit<DT>(p, row) : 0.f;
  __syncthreads();
  // every thread joins the sums in part order, so all hold the same values
  // (a part's maximum passes a NaN over; its S is NaN then, and so is the row's)
  float m = -__builtin_inff();
  for (int i = 0; i < p.chunks; ++i) m = fmaxf(m, part[i][0]);
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
  if (t == 0) write_row(p, row, m, S, T, xt);
  for (int a = t / 8; a < n; a += THREADS / 8) {
    const uint64_t k = keys[a];
    const int rank = count_larger(keys, n, k, t);
    if ((t & 7) == 0 && k != 0 && rank < p.top) {
      p.top_tokens[row * p.top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
      p.top_logprobs[row * p.top + rank] = (order_value((uint32_t)(k >> 32)) - m) - ls;
    }
  }
}

// Elements one workgroup holds in registers.  With 12 pieces a thread of the 8-wave form three workgroups
// share a CU; 14 or 16 pieces leave two, and everything is slower but what then fits (us, 12 / 14 / 16
// pieces, fp16, top 20: 1024x32000 20.9 / 23.4 / 23.5, 1024x49152 28.4 / 32.0 / 32.5, 1024x131072 64 / 81 / 70,
// 1024x50257 110 / 34 / 34).
constexpr int held(int waves, int e) { return waves * 64 * e * 8; }
constexpr int kSmall = held(4, 2), kMiddle = held(8, 4), kLarge = held(8, 12);
static_assert(kLarge == held(16, 6), "both large forms hold the same part");

template <int DT>
hipError_t launch(const LogprobsParams &p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.M * p.chunks));
  if (p.chunk <= kSmall) hipLaunchKernelGGL((part_kernel<DT, 4, 2>), grid, dim3(256), 0, s, p);
  else if (p.chunk <= kMiddle) hipLaunchKernelGGL((part_kernel<DT, 8, 4>), grid, dim3(512), 0, s, p);
  // 16 waves for one workgroup per CU (one row of 49152 fp16: 7.5 against 8.5 us); with more the 8
  // waves' smaller workgroups overlap (1024 rows: 29.3 against 40.3).  32-bit rows take
  // twice the registers: 6 pieces a thread always.
  else if (DT == DT_F32 || (int64_t)p.M * p.chunks <= kCUs)
    hipLaunchKernelGGL((part_kernel<DT, 16, 6>), grid, dim3(1024), 0, s, p);
  else
    hipLaunchKernelGGL((part_kernel<DT == DT_F32 ? DT_F16 : DT, 8, 12>), grid, dim3(512), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.chunks == 1) return e;
  const uint32_t lds = (uint32_t)((p.chunks * p.top + 1) / 2 * 16 + p.chunks * 16);   // 22.8 KiB at most: 86 parts of 32
  // 16 waves where there are many keys to rank (16 parts of 20: 8.1 us with 4)
  if (p.chunks * p.top > 128) hipLaunchKernelGGL((join_kernel<DT, 1024>), dim3((uint32_t)p.M), dim3(1024), lds, s, p);
  else hipLaunchKernelGGL((join_kernel<DT, 256>), dim3((uint32_t)p.M), dim3(256), lds, s, p);
  return hipGetLastError();
}

}  // namespace

// Parts of a row and their length: whole rows of up to kLarge elements, however few (us, whole / in
// parts and joined, fp16: 1x8000 4.3 / 6.3, 1x20000 5.8 / 7.2, 1x32000 6.1 / 7.4, 1x49152 7.2 / 8.7, 32x20000
// 7.1 / 10.2, 32x49152 9.1 / 11.7, 256x49152 11.6 / 15.9; only 1x49152 bfloat16 goes 8.5 / 8.3), longer rows in
// parts of kLarge when they fill the chip, else in parts short enough for up to four workgroups per CU.
int logprobs_chunks(int M, int V, int dtype, int *chunk) {
  (void)dtype;
  const int sizes[] = {kSmall, kMiddle, kLarge};
  for (int i = 0; i < 3; ++i) {
    const int64_t parts = ((int64_t)V + sizes[i] - 1) / sizes[i];
    if (V <= kLarge ? parts == 1 : i == 2 || (parts <= 32 && (int64_t)M * parts <= 4 * kCUs)) {
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
