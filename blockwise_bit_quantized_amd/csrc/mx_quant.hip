// mx_quant.hip -- MX quantisation, its inverse, and the weight layout of the MX product.
//
// Per block of 32: e = clamp(floor(log2 max|x|) - emax, -127, 127), codes = rne(x / 2^e)
// clamped to the format's largest value.  All are bound by memory: 16 bits in and 4 or 8
// out (or the reverse), a few operations per element.  A thread takes 8 elements (16 bytes
// of a 16-bit row), four neighbouring threads share a block's maximum by two lane
// exchanges, so no data goes through LDS and a wave reads 1 KiB of consecutive bytes.
// 49152 x 576 bfloat16 to FP4 takes 14 us and back 13 (72 MB each, 5.1 and 5.5 TB/s; a copy of
// 4 GiB runs at 4.8); 8 x 2048 2.1 us, a launch and one pass of latencies.  8192 x 4096 from 16 bits 17 us
// (FP4) and 20 (FP8), back 14 and 16.5; from 32 bits 26 and 29, back 25 and 32: 4.8 to 6.1 TB/s.
//
// Packing is done once for a weight: 16 bytes a thread, a wave reads 64 bytes of each of 16 rows and
// writes 1 KiB; 4096 x 4096 8.8 us, 49152 x 2048 35.5 (3.0 TB/s), in two launches.
#include "ops.h"

namespace mnb {
namespace {

constexpr int kThreads = 256;
// rows x (K / 8) pieces of one launch: below 2^31, as fast_div needs
constexpr int64_t kMaxPieces = 1ll << 30;

template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(MxQuantParams p, FastDiv per_row, uint32_t pieces) {
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
  if (id >= pieces) return;   // K / 8 is a multiple of 4: the threads of a block leave together
  const uint32_t row = div_by(id, per_row), c = id - row * per_row.d;
  typedef typename Elem<DT>::type T;
  float v[8];
  load8<DT>(static_cast<const T *>(p.x) + (int64_t)row * p.ldx + 8 * c, v);
  // |x| as integers keeps a NaN above every number, so a NaN or infinity shows in the maximum
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
  const uint32_t e = mx_scale<FMT>(amax);
  const float inv = mx_inverse(e);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e == 255 ? 0.f : v[i] * inv;
  uint8_t *out = p.codes + (int64_t)row * p.ldc;
  if constexpr (FMT == MX_FP4) *reinterpret_cast<uint32_t *>(out + 4 * c) = fp4_codes(v);
  else *reinterpret_cast<u2_t *>(out + 8 * c) = u2_t{fp8_codes4(v), fp8_codes4(v + 4)};
  if ((c & 3) == 0) p.scales[(int64_t)row * p.lds + (c >> 2)] = (uint8_t)e;
}

template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(MxDequantParams p, FastDiv per_row, uint32_t pieces) {
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
  if (id >= pieces) return;
  const uint32_t row = div_by(id, per_row), c = id - row * per_row.d;
  typedef typename Elem<DT>::type T;
  const uint8_t *in = p.codes + (int64_t)row * p.ldc;
  const float scale = mx_value(p.scales[(int64_t)row * p.lds + (c >> 2)]);
  float v[8];
  if constexpr (FMT == MX_FP4) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(in + 4 * c);
    const f2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f2_t f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = d[0]; v[5] = d[1]; v[6] = f[0]; v[7] = f[1];
  } else {
    const u2_t w = *reinterpret_cast<const u2_t *>(in + 8 * c);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const f2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      v[4 * i] = a[0]; v[4 * i + 1] = a[1]; v[4 * i + 2] = b[0]; v[4 * i + 3] = b[1];
    }
  }
  // the product is exact in 32 bits (4 significant bits, a power of two), so the store's
  // rounding is the only one
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= scale;
  store8<DT>(static_cast<T *>(p.y) + (int64_t)row * p.ldy + 8 * c, v);
}

__global__ __launch_bounds__(kThreads) void pack_codes_kernel(MxPackParams p, int64_t chunks) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= chunks) return;
  const int lane = (int)(id & 63), f = (int)(id >> 6) & 3;
  const int64_t gs = id >> 8;
  const int g = (int)(gs / p.KS), step = (int)(gs - (int64_t)g * p.KS);
  const int r = lane & 15, b = lane >> 4;
  const int64_t n = 64 * (int64_t)g + 16 * (r >> 2) + 4 * f + (r & 3);
  const int kb = step * 4 + b;
  u4_t w = {0, 0, 0, 0};
  if (n < p.N && kb < p.K / kBlock) w = *reinterpret_cast<const u4_t *>(p.codes + n * p.ldc + (int64_t)kb * 16);
  *reinterpret_cast<u4_t *>(p.wq + id * 16) = w;
}

__global__ __launch_bounds__(kThreads) void pack_scales_kernel(MxPackParams p, int64_t words) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= words) return;
  const int lane = (int)(id & 63), f = (int)(id >> 6) & 3;
  const int64_t gk = id >> 8;
  const int g = (int)(gk / p.KB), kb512 = (int)(gk - (int64_t)g * p.KB);
  const int r = lane & 15, b = lane >> 4;
  const int64_t n = 64 * (int64_t)g + 16 * (r >> 2) + 4 * f + (r & 3);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int kb = (kb512 * 4 + j) * 4 + b;
    if (n < p.N && kb < p.K / kBlock) w |= (uint32_t)p.scales[n * p.lds + kb] << (8 * j);
  }
  reinterpret_cast<uint32_t *>(p.sc)[id] = w;
}

// rows in parts of at most kMaxPieces pieces
template <typename P, typename F>
hipError_t by_rows(const P &p, F launch) {
  const int64_t per_row = p.K / 8;
  const int64_t rows = kMaxPieces / per_row;   // K < 2^31: at least 4 rows
  for (int64_t m0 = 0; m0 < p.M; m0 += rows) {
    const int64_t mc = p.M - m0 < rows ? p.M - m0 : rows;
    const uint32_t pieces = (uint32_t)(mc * per_row);
    const hipError_t e = launch(m0, pieces, (pieces + kThreads - 1) / kThreads);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int FMT>
hipError_t quantize(const MxQuantParams &p, hipStream_t s) {
  return by_rows(p, [&](int64_t m0, uint32_t pieces, uint32_t grid) {
    MxQuantParams q = p;
    q.x = static_cast<const typename Elem<DT>::type *>(p.x) + m0 * p.ldx;
    q.codes += m0 * p.ldc;
    q.scales += m0 * p.lds;
    hipLaunchKernelGGL((quantize_kernel<DT, FMT>), dim3(grid), dim3(kThreads), 0, s, q, fast_div(p.K / 8), pieces);
    return hipGetLastError();
  });
}

template <int DT, int FMT>
hipError_t dequantize(const MxDequantParams &p, hipStream_t s) {
  return by_rows(p, [&](int64_t m0, uint32_t pieces, uint32_t grid) {
    MxDequantParams q = p;
    q.y = static_cast<typename Elem<DT>::type *>(p.y) + m0 * p.ldy;
    q.codes += m0 * p.ldc;
    q.scales += m0 * p.lds;
    hipLaunchKernelGGL((dequantize_kernel<DT, FMT>), dim3(grid), dim3(kThreads), 0, s, q, fast_div(p.K / 8), pieces);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_mx_quantize(int dtype, int fmt, const MxQuantParams &p, hipStream_t s) {
  if (fmt == MX_FP4)
    return dtype == DT_F16    ? quantize<DT_F16, MX_FP4>(p, s)
           : dtype == DT_BF16 ? quantize<DT_BF16, MX_FP4>(p, s)
                              : quantize<DT_F32, MX_FP4>(p, s);
  return dtype == DT_F16    ? quantize<DT_F16, MX_FP8>(p, s)
         : dtype == DT_BF16 ? quantize<DT_BF16, MX_FP8>(p, s)
                            : quantize<DT_F32, MX_FP8>(p, s);
}

hipError_t launch_mx_dequantize(int dtype, int fmt, const MxDequantParams &p, hipStream_t s) {
  if (fmt == MX_FP4)
    return dtype == DT_F16    ? dequantize<DT_F16, MX_FP4>(p, s)
           : dtype == DT_BF16 ? dequantize<DT_BF16, MX_FP4>(p, s)
                              : dequantize<DT_F32, MX_FP4>(p, s);
  return dtype == DT_F16    ? dequantize<DT_F16, MX_FP8>(p, s)
         : dtype == DT_BF16 ? dequantize<DT_BF16, MX_FP8>(p, s)
                            : dequantize<DT_F32, MX_FP8>(p, s);
}

hipError_t launch_mx_pack(const MxPackParams &p, hipStream_t s) {
  const int64_t chunks = (int64_t)p.NG * p.KS * 256, words = (int64_t)p.NG * p.KB * 256;
  hipLaunchKernelGGL(pack_codes_kernel, dim3((uint32_t)(chunks / kThreads)), dim3(kThreads), 0, s, p, chunks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(pack_scales_kernel, dim3((uint32_t)(words / kThreads)), dim3(kThreads), 0, s, p, words);
  return hipGetLastError();
}

}  // namespace mnb
