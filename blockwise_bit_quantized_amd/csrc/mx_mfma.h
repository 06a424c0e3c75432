// mx_mfma.h -- the scaled matrix instruction of the MX product, shared by its kernels.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 weight rows (FP4, the row operand) with 32 X
// rows (the column operand) over 64 k, applying one scale byte per operand row and block of 32.
// Operand layouts (measured on the part): FP4, lane 32 b + r holds row r, k = 32 b .. 32 b + 31
// in 16 bytes; FP8, lane 32 h + r holds row r, k = 16 h .. + 15 in the first 16 bytes and
// k = 32 + 16 h .. in the next; the scale byte of block b of row r comes from lane 32 b + r in
// either case, from byte JW (weights) or JX (X) of the lane's dword.  Value 4 q + e of the
// result's lane 32 h + c is weight row 8 q + 4 h + e of X row c.
//
// Of the two shapes this one runs at 7500 TFLOP/s (FP4 X) and 4250 (FP8 X) on random data
// with one wave per SIMD, the 16 x 16 x 128 one at 4480 and 4050: its two-part encoding takes
// as long to issue as half the FP4 instruction takes to run.
//
// Precision.  With FP4 on both sides the sum of an instruction is exact in these formats'
// range; with FP8 the adder keeps about 12 bits below the sum of the magnitudes where the
// scales of its blocks differ by many octaves (2^-12.6 of it was the largest error found
// over scales of 2^-8 to 2^8), and about 24 where they are alike.
#pragma once

#include <type_traits>

#include "ops.h"

namespace mnb {

typedef f16x_t acc_t;

template <int FMT, int JW, int JX>
__device__ __forceinline__ acc_t mx_mfma(u4_t w, u4_t x0, u4_t x1, acc_t acc, uint32_t sw, uint32_t sx) {
  const i8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i8_t b = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, FMT == MX_FP4 ? 4 : 0, JW, (int)sw, JX, (int)sx);
}

template <int I, int N, typename F>
__device__ __forceinline__ void unroll(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<I + 1, N>(f);
  }
}

// the 16 consecutive columns n.. of row m that a lane holds, with the bias, rounded once
template <int DT>
__device__ __forceinline__ void store_cols(const MxMatmulParams &p, int64_t m, int64_t n, const acc_t &acc) {
  uint16_t *y = p.y + m * p.N + n;
  if (n + 16 <= p.N && (p.N & 7) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8], b[8] = {};
      if (p.bias) load8<DT>(p.bias + n + 8 * h, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = acc[8 * h + e] + b[e];
      store8<DT>(y + 8 * h, v);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (n + e < p.N) y[e] = from_f32<DT>(acc[e] + (p.bias ? to_f32<DT>(p.bias[n + e]) : 0.f));
  }
}

}  // namespace mnb
