// kv_append.hip -- new rows of queries, keys and values on their way into the FP4 cache, and rows of it back.
//
// For each head of q and k: h = x / sqrt(mean(x^2) + eps) * w (where a weight is given), then the first `rot`
// elements turn by the angle of the row's position: (a, b) -> (a cos - b sin, b cos + a sin).
// q is rounded once to 16 bits; keys and values become MX FP4 codes (blocks of 32 along the head).
//
// Keys are computed in 64 bits throughout, so their codes are those of the exact key (32 bits would put
// one element in some thousands on the wrong side of a border of the 4-bit grid); sums of squares are
// in 64 bits for queries too.  A lane holds 8 elements and 8, 16 or 32 lanes a head, so a block of 32 is
// four neighbouring lanes, and nothing goes through LDS.
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

enum Where { kHeld, kNowhere, kUnreachable, kForeign };   // kForeign: the row of no sequence
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

// norm and rotation of the 8 elements of lane l of a head, in T; every lane of the wave runs it together
template <int DT, int LANES, typename T>
__device__ __forceinline__ void norm_rotate(const KvAppendParams &p, T *v, const uint16_t *weight, int l, bool in, int pos) {
  const int D = p.cache.D;
  if (weight) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)v[i], (double)v[i], ss);
    ss = head_sum<LANES>(ss);
    const T r = (T)(1.0 / sqrt(ss / D + (double)p.eps));
    float w[8] = {};
    if (in) load8<DT>(weight + 8 * l, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * (T)w[i];
  }
  if (p.rot == 0) return;
  const float *row = p.table + (int64_t)pos * p.rot;
  const int half = p.rot / 2, hl = p.rot / 16;        // elements and lanes of half a turn
  if (p.interleaved) {
    if (8 * l < p.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T c = (T)row[4 * l + i], s = (T)row[half + 4 * l + i], a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = a * c - b * s;
        v[2 * i + 1] = b * c + a * s;
      }
    }
    return;
  }
  const int lane = threadIdx.x & 63, base = lane & ~(LANES - 1);
  const bool low = l < hl;
  const int other = base + (l < 2 * hl ? (low ? l + hl : l - hl) : l);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const T o = __shfl(v[i], other);       // the pair's other half
    if (l < 2 * hl) {
      const int e = 8 * (low ? l : l - hl) + i;
      const T c = (T)row[e], s = (T)row[half + e];
      v[i] = low ? v[i] * c - o * s : v[i] * c + o * s;
    }
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

// One workgroup a row; heads in the order q, k, v, LANES lanes each.
template <int DT, int LANES>
__global__ __launch_bounds__(1024) void append_kernel(KvAppendParams p) {
  const int row = blockIdx.x, D = p.cache.D, S = 1 << p.cache.shift;
  const int l = threadIdx.x & (LANES - 1);
  const bool in = 8 * l < D;
  Place at = find_place(p.cache, p.rows, row);
  if (at.where == kForeign) return;
  if (at.where == kHeld && p.rot && at.pos >= p.table_rows) at.where = kUnreachable;
  const int kv = p.cache.heads, heads = p.q_heads + 2 * kv, step = blockDim.x / LANES;
  uint8_t *page = p.cache.data + (int64_t)at.page * p.cache.page_stride;
  for (int h0 = 0; h0 < heads; h0 += step) {            // uniform, so that the exchanges find all lanes
    const int h = h0 + (int)threadIdx.x / LANES;
    const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + kv;
    const int hk = h - p.q_heads - (is_k ? 0 : kv);      // head of the cache, for k and v
    const bool on = h < heads && in;
    const uint16_t *src = is_q   ? p.q + (int64_t)row * p.ldq + (int64_t)h * D
                          : is_k ? p.k + (int64_t)row * p.ldk + (int64_t)hk * D
                                 : p.v + (int64_t)row * p.ldv + (int64_t)hk * D;
    float x[8] = {};
    if (on) load8<DT>(src + 8 * l, x);
    if (at.where != kHeld) {
      if (is_q && on) {
        const float fill = at.where == kNowhere ? 0.f : __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fill;
        store8<DT>(p.out + (int64_t)row * p.ldo + (int64_t)h * D + 8 * l, x);
      }
      continue;
    }
    if (is_q || is_k) {
      double v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[i];
      norm_rotate<DT, LANES, double>(p, v, is_q ? p.qw : p.kw, l, in, at.pos);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = to_odd(v[i]);
    }
    if (is_q) {
      if (on) store8<DT>(p.out + (int64_t)row * p.ldo + (int64_t)h * D + 8 * l, x);
      continue;
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
  const int threads = (int)(need > 1024 ? 1024 : (need + 63) / 64 * 64);
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
