// mx_mfma.h -- the scaled matrix instruction of the MX product, shared by its kernels.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 weight rows (FP4, the row operand) with
// 16 X rows (the column operand) over 128 k, applying one scale byte per operand row and
// block of 32.  Operand layouts (measured on the part): FP4, lane 16 b + r holds row r,
// k = 32 b .. 32 b + 31 in 16 bytes; FP8, lane 16 g + r holds row r, k = 16 g .. + 15 in the
// first 16 bytes and k = 64 + 16 g .. in the next; the scale byte of block b of row r comes
// from lane 16 b + r in either case, taken from byte J of the lane's dword.  The result's
// lane 16 g + c holds weight rows 4 g .. 4 g + 3 of X row c.
//
// The 32 x 32 x 64 shape was built and measured too.  In a bare loop it runs FP4 at 7500
// TFLOP/s on random data where this one, with its two-part encoding, issues at 4480 to 5410 (FP8:
// 4250 and 4050 to 4230); in the product it is slower, 8192 x 9728 x 2560 176 against 167 us
// (FP8 X) and 138 against 128 (FP4 X): the part clocks down to 1.5 - 1.9 GHz under this load, and
// that shape moves twice the accumulator bytes per operation.
//
// Precision, in units of the sum of the terms' magnitudes.  With FP4 on both sides the sums are as
// exact as 32 bits (2^-23.4 at most over scales of 2^-8 to 2^8, K up to 9728).  With FP8 the adder
// aligns its terms to the largest and keeps fewer bits: 2^-17.9 at K = 96, 2^-20.6 at 2016 and 2^-21.8 at 9696 with
// scales alike, 2^-16.9, 2^-17.6 and 2^-19.2 with scales of 2^-8 to 2^8, 2^-12.6 the largest found on any data.
// It is the instruction's own; the 16-bit formats would hold FP8 values, at half the rate.
#pragma once

#include <type_traits>

#include "ops.h"

namespace mnb {

template <int FMT, int J>
__device__ __forceinline__ f4_t mx_mfma(u4_t w, u4_t x0, u4_t x1, f4_t acc, uint32_t sw, uint32_t sx) {
  const i8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i8_t b = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, FMT == MX_FP4 ? 4 : 0, J, (int)sw, 0, (int)sx);
}

template <int DT>
__device__ __forceinline__ void store_cols(const MxMatmulParams &p, int64_t m, int64_t n, float v) {
  if (p.bias) v += to_f32<DT>(p.bias[n]);
  p.y[m * p.N + n] = from_f32<DT>(v);
}

}  // namespace mnb
