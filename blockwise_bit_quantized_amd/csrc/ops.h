// ops.h -- types, layouts and launchers shared by the kernels of include/mnb_ops.h (MX
// quantisation and product, RMS norm, log probabilities).
#pragma once

#include "common.h"

namespace mnb {

enum { DT_F16 = 0, DT_BF16 = 1, DT_F32 = 2 };
enum { MX_FP4 = 0, MX_FP8 = 1 };

constexpr int kMxStep = 128;   // k of one matrix instruction (4 blocks)
constexpr int kMxMaxK = 1 << 22;   // K limit of the product; its row distances stay below twice that
constexpr int kMxScaleK = 512; // k of one scale dword per lane (4 steps, one byte each)

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef int i8_t __attribute__((ext_vector_type(8)));

// ---- 16-bit and 32-bit values -------------------------------------------------------------

template <int DT> struct Elem { typedef uint16_t type; };
template <> struct Elem<DT_F32> { typedef float type; };

template <int DT>
__device__ __forceinline__ float to_f32(typename Elem<DT>::type v) {
  if constexpr (DT == DT_F16) return h2f(v);
  else if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, (uint32_t)v << 16);
  else return v;
}
// one rounding, to nearest even (a bfloat16 NaN stays a NaN)
template <int DT>
__device__ __forceinline__ typename Elem<DT>::type from_f32(float v) {
  if constexpr (DT == DT_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  else if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return v;
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)from_f32<DT>(a) | (uint32_t)from_f32<DT>(b) << 16;
}
// 8 consecutive elements at a 16-byte aligned address
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type *p, float *v) {
  if constexpr (DT == DT_F32) {
    const f4_t a = reinterpret_cast<const f4_t *>(p)[0], b = reinterpret_cast<const f4_t *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
    const u4_t w = *reinterpret_cast<const u4_t *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = to_f32<DT>((uint16_t)w[i]);
      v[2 * i + 1] = to_f32<DT>((uint16_t)(w[i] >> 16));
    }
  }
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type *p, const float *v) {
  if constexpr (DT == DT_F32) {
    reinterpret_cast<f4_t *>(p)[0] = f4_t{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f4_t *>(p)[1] = f4_t{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u4_t *>(p) =
        u4_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
  }
}

// ---- MX scales and elements ---------------------------------------------------------------

// E8M0 byte of a block from the bits of its largest |x| (32-bit, finite or not): the
// exponent field is floor(log2) + 127 for normal numbers; below 2^-126 the scale is at its
// lowest value in either format, so the field's 0 needs no further care.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - (FMT == MX_FP4 ? 2 : 8);
  return (amax_bits >> 23) == 255 ? 255u : (uint32_t)(e < 0 ? 0 : e);
}
// 1 / 2^(e - 127), 0 for the NaN scale: NaN and infinity are taken out by the caller
__device__ __forceinline__ float mx_inverse(uint32_t e) {
  return e == 255 ? 0.f : __builtin_bit_cast(float, (254u - e) << 23);
}
// 2^(e - 127) (e = 0: the subnormal 2^-127; 255: NaN)
__device__ __forceinline__ float mx_value(uint32_t e) {
  return __builtin_bit_cast(float, e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
}
// 8 scaled values to codes: 4 bytes (FP4, low nibble first) or 8 (FP8).  The conversion
// instructions round to nearest even; FP4 saturates, FP8 gives NaN past 464, hence the
// clamp (v_med3).
__device__ __forceinline__ uint32_t fp4_codes(const float *v) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
}
__device__ __forceinline__ uint32_t fp8_codes4(const float *v) {
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], -448.f, 448.f);
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], r, true);
}

// ---- division by a launch constant --------------------------------------------------------

// n / d for n < 2^31: with 2^L >= d, m = floor(2^(31 + L) / d) + 1 < 2^32 has
// 0 < m d - 2^(31 + L) <= 2^L, so the error of n m / 2^(31 + L) stays below 1 / d.
struct FastDiv {
  uint32_t m, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  int L = 0;
  while ((1u << L) < d) ++L;
  return FastDiv{(uint32_t)(((1ull << (31 + L)) / d) + 1), (uint32_t)(31 + L), d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
  return (uint32_t)(((uint64_t)n * f.m) >> f.shift);
}

// ---- launch parameter blocks and launchers (each returns hipGetLastError()) ---------------

struct MxQuantParams {
  const void *x;
  uint8_t *codes, *scales;
  int64_t ldx, ldc, lds;
  int M, K;
};
hipError_t launch_mx_quantize(int dtype, int fmt, const MxQuantParams &p, hipStream_t s);

struct MxDequantParams {
  const uint8_t *codes, *scales;
  void *y;
  int64_t ldc, lds, ldy;
  int M, K;
};
hipError_t launch_mx_dequantize(int dtype, int fmt, const MxDequantParams &p, hipStream_t s);

// chunk (group of 64 rows, step of 128 k, operand f, lane): 16 bytes at
// (((group * KS + step) * 4 + f) * 64 + lane) * 16.  Lane 16 b + r of operand f holds block
// b of the step (32 k) of row 64 group + 16 (r / 4) + 4 f + r % 4: a lane of the product's
// result then holds 16 consecutive columns over the four operands.  Scale dwords at
// (((group * KB + k / 512) * 4 + f) * 64 + lane) * 4, byte j for step 4 (k / 512) + j.
struct MxPackParams {
  const uint8_t *codes, *scales;
  uint8_t *wq, *sc;
  int64_t ldc, lds;
  int N, K, NG, KS, KB;
};
hipError_t launch_mx_pack(const MxPackParams &p, hipStream_t s);

struct MxMatmulParams {
  const uint8_t *codes, *scales;   // X
  const uint8_t *wq, *sc;          // W
  const uint16_t *bias;
  uint16_t *y;
  int64_t ldc, lds;
  int M, N, K, NG, KS, KB;
};
constexpr int kMxGemvMaxM = 32;
hipError_t launch_mx_gemv(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s);
hipError_t launch_mx_gemm(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s);
int mx_gemv_operands(int fmt, int M, int N, int K);  // operands of 16 weight rows a wave: 1, 2 or 4
int mx_gemv_ksplit(int fmt, int M, int N, int K);    // waves that share a weight row's K: 1, 2 or 4
int mx_gemm_groups(int fmt, int M, int N, int K);    // groups of waves that share a tile's K: 1 or 2
int mx_gemm_rows(int fmt, int M, int N, int K);      // 256 (two 128 x 256 tiles a CU), 128 or 64

struct NormParams {
  const uint16_t *x, *res, *w;
  uint16_t *hidden, *y;
  uint8_t *codes, *scales;
  int64_t ldx, ldr, ldh, ldy, ldc, lds;
  int M, K;
  float eps;
};
// fmt -1: no codes
hipError_t launch_rmsnorm(int dtype, int fmt, const NormParams &p, hipStream_t s);

struct LogprobsParams {
  const void *x;
  int64_t ldl;
  const int64_t *tokens;
  float *logprob, *entropy, *top_logprobs;
  int64_t *top_tokens;
  int M, V, top;
  int chunks, chunk;      // parts of a row and elements of each
  float *part;            // chunks > 1: [M, chunks, 4] (max, sum, sum of p d, unused)
  uint64_t *keys;         //             [M, chunks, top]
};
hipError_t launch_logprobs(int dtype, const LogprobsParams &p, hipStream_t s);
int logprobs_chunks(int M, int V, int dtype, int *chunk);

}  // namespace mnb
