// kv_append.hip -- new rows of queries, keys and values on their way into the FP4 cache, and rows of it back.
//
// For each head of q and k: h = x / sqrt(mean(x^2) + eps) * w (where a weight is given), then the first `rot`
// elements turn by the angle of the row's position: (a, b) -> (a cos - b sin, b cos + a sin).
// q is rounded once to 16 bits; keys and values become MX FP4 codes (blocks of 32 along the head).
//
// Keys are computed in 64 bits throughout, so their codes are those of the exact key (32 bits would put
// one element in some thousands on the wrong side of a border of the 4-bit grid).  Queries have their sums of squares
// in 64 bits and the products, at most 5 roundings of 2^-24 before the one to 16 bits, in 32.  A lane holds 8 elements and 8, 16 or 32 lanes a head, so a block of 32 is
// four neighbouring lanes, and nothing goes through LDS.
//
// Many rows are bound by memory: 8192 rows of 32 + 8 + 8 heads of 128 in 51 us are 170 MB at 3.3 TB/s (a large copy: 4.7).
// Few are bound by the chain of loads row -> sequence -> page number and angles: 64 rows 5.1 us, one row 3.3 us.  Reading back
// (8192 rows of 8 heads, 42 MB) takes 12.8 us, 3.3 TB/s.
#include "decode.h"

namespace mnb {
namespace {

// The last sequence whose first row is at or before `row`, found by the whole wave (starts do not fall; if they
// do, some sequence in range).
__device__ __forceinline__ int find_sequence(const KvRows &r, int row) {
  if (!r.starts) return row;
  int count = 0;
  for (int b0 = 0; b0 < r.batch; b0 += 64) {
    const int b = b0 + (threadIdx.x & 63);
    const int c = __popcll(__ballot(b < r.batch && r.starts[b] <= row));
    count += c;
    if (c < 64) break;
  }
  return max(0, count - 1);
}

enum Where { kHeld, kNowhere, kUnreachable, kForeign, kUnturned };   // kForeign: the row of no sequence; kUnturned: past the table
struct Place {
  Where where;
  int pos, page, at;
};
__device__ __forceinline__ Place find_place(const KvCache &c, const KvRows &r, int row) {
  const int b = find_sequence(r, row);
  const KvSeq s = kv_seq(r, b);
  Place p{kForeign, 0, 0, 0};
  if (row < s.row0 || row >= s.row0 + s.n) return p;
  p.pos = s.first() + (row - s.row0);
  if (p.pos < 0) {
    p.where = kNowhere;
    return p;
  }
  p.where = kUnreachable;
  const int col = p.pos >> c.shift;
  if (col >= r.width) return p;
  p.page = r.pages[(int64_t)b * r.ldp + col];
  if ((uint32_t)p.page >= (uint32_t)c.pages) return p;
  p.where = kHeld;
  p.at = p.pos & ((1 << c.shift) - 1);
  return p;
}

template <int LANES>
__device__ __forceinline__ double head_sum(double v) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The angle of a row's position for lane l of a head, the same for all its heads: v' = v c + o s, where o is the pair's other
// element.
struct Turn {
  bool on;
  int other;                   // lane that holds the pairs' other elements (halves turned against each other)
  float c[8], s[8];
};
template <int LANES>
__device__ __forceinline__ Turn find_turn(const KvAppendParams &p, int l, int pos) {
  Turn t;
  t.on = 8 * l < p.rot;
  const int half = p.rot / 2, hl = p.rot / 16;           // elements and lanes of half a turn
  const bool low = l < hl;
  t.other = (threadIdx.x & 63 & ~(LANES - 1)) + (!t.on ? l : low ? l + hl : l - hl);
  if (!t.on) return t;
  const float *row = p.table + (int64_t)pos * p.rot + (p.interleaved ? 4 * l : 8 * (low ? l : l - hl));
  const f4_t c0 = *reinterpret_cast<const f4_t *>(row), s0 = *reinterpret_cast<const f4_t *>(row + half);
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] = c0[i / 2];
      t.s[i] = i & 1 ? s0[i / 2] : -s0[i / 2];
    }
  } else {
    const f4_t c1 = *reinterpret_cast<const f4_t *>(row + 4), s1 = *reinterpret_cast<const f4_t *>(row + half + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.c[i] = c0[i];
      t.c[4 + i] = c1[i];
      t.s[i] = low ? -s0[i] : s0[i];
      t.s[4 + i] = low ? -s1[i] : s1[i];
    }
  }
  return t;
}

// norm and rotation of the 8 elements of a lane of a head, in T; all lanes of the head run it together
template <int DT, int LANES, typename T>
__device__ __forceinline__ void norm_rotate(const KvAppendParams &p, const float *x, T *v, const uint16_t *weight, u4_t w8, const Turn &turn) {
  if (weight) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)x[i], (double)x[i], ss);
    ss = head_sum<LANES>(ss);
    const double r = 1.0 / sqrt(ss / p.cache.D + (double)p.eps);   // (as 32 bits it could pass their range)
    float w[8];
    load8<DT>(reinterpret_cast<const uint16_t *>(&w8), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)(x[i] * r) * (T)w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)x[i];
  }
  if (p.rot == 0) return;
  T o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = p.interleaved ? v[i ^ 1] : __shfl(v[i], turn.other);
  if (turn.on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * (T)turn.c[i] + o[i] * (T)turn.s[i];
  }
}

// the lane's 8 elements as FP4 codes with the scale of its block of four lanes
__device__ __forceinline__ uint32_t quantize8(const float *x, uint32_t &e) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu);
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
  e = mx_scale<MX_FP4>(amax);
  const float inv = mx_inverse(e);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e == 255 ? 0.f : x[i] * inv;
  return fp4_codes(v);
}

// One workgroup a row; heads in the order q, k, v, LANES lanes each.  Heads behind the workgroup's first are loaded while
// the ones before are computed; the row's angles stay in registers.
template <int DT, int LANES>
__global__ __launch_bounds__(1024) void append_kernel(KvAppendParams p) {
  const int row = blockIdx.x, D = p.cache.D, S = 1 << p.cache.shift;
  const int l = threadIdx.x & (LANES - 1);
  const bool in = 8 * l < D;
  const int kv = p.cache.heads, heads = p.q_heads + 2 * kv, step = blockDim.x / LANES;
  auto fetch = [&](int h) {
    const int hk = h - p.q_heads, hv = hk - kv;
    const uint16_t *src = hk < 0   ? p.q + (int64_t)row * p.ldq + (int64_t)h * D
                          : hv < 0 ? p.k + (int64_t)row * p.ldk + (int64_t)hk * D
                                   : p.v + (int64_t)row * p.ldv + (int64_t)hv * D;
    return h < heads && in ? *reinterpret_cast<const u4_t *>(src + 8 * l) : u4_t{0, 0, 0, 0};
  };
  u4_t next = fetch((int)threadIdx.x / LANES);
  const u4_t none = {0, 0, 0, 0};
  const u4_t wq = p.qw && in ? *reinterpret_cast<const u4_t *>(p.qw + 8 * l) : none;
  const u4_t wk = p.kw && in ? *reinterpret_cast<const u4_t *>(p.kw + 8 * l) : none;
  Place at = find_place(p.cache, p.rows, row);
  if (at.where == kForeign) return;
  if (at.where == kHeld && p.rot && at.pos >= p.table_rows) at.where = kUnturned;
  uint8_t *page = p.cache.data + (int64_t)at.page * p.cache.page_stride;
  Turn turn{};
  if (at.where == kHeld) turn = find_turn<LANES>(p, l, at.pos);
  for (int h0 = 0; h0 < heads; h0 += step) {            // uniform, so that the exchanges find all lanes
    const int h = h0 + (int)threadIdx.x / LANES;
    const u4_t now = next;
    next = fetch(h + step);
    const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + kv;
    const int hk = h - p.q_heads - (is_k ? 0 : kv);      // head of the cache, for k and v
    const bool on = h < heads && in;
    uint16_t *out = p.out + (int64_t)row * p.ldo + (int64_t)h * D + 8 * l;
    float x[8];
    load8<DT>(reinterpret_cast<const uint16_t *>(&now), x);
    if (at.where != kHeld) {
      if (is_q && on) {
        const float fill = at.where == kNowhere ? 0.f : __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fill;
        store8<DT>(out, x);
      }
      // what is read at that place later is NaN, not what it held before
      if (at.where == kUnturned && !is_q && on && (l & 3) == 0) {
        uint8_t *head = page + (int64_t)hk * kv_head_bytes(S, D);
        const int key = kv_key_scales(S, D) + at.at * (D / 32) + l / 4;
        head[is_k ? key : kv_value_scales(S, D) + ((at.at >> 2) * (D / 32) + l / 4) * 4 + (at.at & 3)] = 255;
      }
      continue;
    }
    if (is_q) {
      float v[8];
      norm_rotate<DT, LANES, float>(p, x, v, p.qw, wq, turn);
      if (on) store8<DT>(out, v);
      continue;
    }
    if (is_k) {
      double v[8];
      norm_rotate<DT, LANES, double>(p, x, v, p.kw, wk, turn);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = to_odd(v[i]);
    }
    uint32_t e;
    const uint32_t codes = quantize8(x, e);
    if (!on) continue;
    uint8_t *head = page + (int64_t)hk * kv_head_bytes(S, D);
    if (is_k) {
      *reinterpret_cast<uint32_t *>(head + at.at * (D / 2) + 4 * l) = codes;
      if ((l & 3) == 0) head[kv_key_scales(S, D) + at.at * (D / 32) + l / 4] = (uint8_t)e;
    } else {
      const int unit = at.at >> 2, tok = at.at & 3;
      *reinterpret_cast<uint32_t *>(head + kv_value_codes(S, D) + ((unit * (D / 8) + l) * 4 + tok) * 4) = codes;
      if ((l & 3) == 0) head[kv_value_scales(S, D) + (unit * (D / 32) + l / 4) * 4 + tok] = (uint8_t)e;
    }
  }
}

__device__ __forceinline__ void expand8(uint32_t w, uint32_t e, float *v) {
  const f2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const f2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const f2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  const float s = mx_value(e);
  v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  v[4] = c[0] * s; v[5] = c[1] * s; v[6] = d[0] * s; v[7] = d[1] * s;
}

// One workgroup a row; 8 elements a thread of a key and of a value head.
template <int DT>
__global__ __launch_bounds__(256) void read_kernel(KvReadParams p) {
  typedef typename Elem<DT>::type T;
  const int row = blockIdx.x, D = p.cache.D, S = 1 << p.cache.shift, per = D / 8;
  const Place at = find_place(p.cache, p.rows, row);
  if (at.where == kForeign) return;
  const uint8_t *page = p.cache.data + (int64_t)at.page * p.cache.page_stride;
  for (int i = threadIdx.x; i < p.cache.heads * per; i += 256) {
    const int h = i / per, l = i - h * per;
    float k[8], v[8];
    if (at.where == kHeld) {
      const uint8_t *head = page + (int64_t)h * kv_head_bytes(S, D);
      const int unit = at.at >> 2, tok = at.at & 3;
      expand8(*reinterpret_cast<const uint32_t *>(head + at.at * (D / 2) + 4 * l), head[kv_key_scales(S, D) + at.at * (D / 32) + l / 4], k);
      expand8(*reinterpret_cast<const uint32_t *>(head + kv_value_codes(S, D) + ((unit * (D / 8) + l) * 4 + tok) * 4),
              head[kv_value_scales(S, D) + (unit * (D / 32) + l / 4) * 4 + tok], v);
    } else {
      const float fill = at.where == kNowhere ? 0.f : __builtin_nanf("");
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = v[j] = fill;
    }
    if (p.k) store8<DT>(static_cast<T *>(p.k) + (int64_t)row * p.ldk + (int64_t)h * D + 8 * l, k);
    if (p.v) store8<DT>(static_cast<T *>(p.v) + (int64_t)row * p.ldv + (int64_t)h * D + 8 * l, v);
  }
}

template <int DT>
hipError_t append(const KvAppendParams &p, hipStream_t s) {
  const int lanes = p.cache.D <= 64 ? 8 : p.cache.D <= 128 ? 16 : 32;
  const int64_t need = (int64_t)(p.q_heads + 2 * p.cache.heads) * lanes;
  // A workgroup takes its row's heads in as many passes as leave all rows on the card at once (16 waves a CU, by
  // registers), but has at least two waves: with 48 heads of 128, of 1024 threads against the rule's, 512 rows take
  // 8.8 and 7.4 us, 2048 rows 27.7 and 17.3, 8192 rows 98.5 and 50.8; 256 rows of 128 threads 9.0, of 1024 5.6.
  int64_t most = (int64_t)kCUs * 1024 / p.rows.rows / 64 * 64;
  most = most < 128 ? 128 : most > 1024 ? 1024 : most;
  const int threads = (int)(need > most ? most : (need + 63) / 64 * 64);
  const dim3 grid((uint32_t)p.rows.rows), block((uint32_t)threads);
  if (lanes == 8) hipLaunchKernelGGL((append_kernel<DT, 8>), grid, block, 0, s, p);
  else if (lanes == 16) hipLaunchKernelGGL((append_kernel<DT, 16>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((append_kernel<DT, 32>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(int dtype, const KvAppendParams &p, hipStream_t s) {
  return dtype == DT_F16 ? append<DT_F16>(p, s) : append<DT_BF16>(p, s);
}

hipError_t launch_kv_read(int dtype, const KvReadParams &p, hipStream_t s) {
  const dim3 grid((uint32_t)p.rows.rows);
  if (dtype == DT_F16) hipLaunchKernelGGL((read_kernel<DT_F16>), grid, dim3(256), 0, s, p);
  else if (dtype == DT_BF16) hipLaunchKernelGGL((read_kernel<DT_BF16>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((read_kernel<DT_F32>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace mnb
