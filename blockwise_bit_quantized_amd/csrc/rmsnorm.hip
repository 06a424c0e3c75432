// rmsnorm.hip -- y = h / sqrt(mean(h^2) + eps) * w, h = x + residual, with the new residual
// stream h and y in 16 bits or MX as outputs, each rounded once from 32 bits.
//
// The sum of squares and the root are in 64 bits, of h before any rounding (32 bits may lose the
// smaller of x and residual, and bfloat16 rows may have squares past their range).  The
// products are in 32 bits, within 4 units of the last place of the exact y; an MX output is
// nevertheless that of the exact y, as values so near a border of the element grid that 4
// units could cross it are computed again in 64 bits from x and residual (one element in 7000, and
// the only ones whose code or block scale can differ).  So are rows whose norm 32 bits do not hold,
// whatever their outputs, and blocks below 2^-100.  (Two limits of 32 bits stay: a y past their
// range counts as infinite, and an element 2^126 times smaller than its row's norm keeps their
// absolute precision.)  All in 64 bits measured 55.7 us at 8192 x 4096 (bfloat16, residual,
// FP8) against 45.8, in fp16 59.0 against 44.8.
//
// Bound by memory (8192 x 4096, bfloat16, residual, FP8: 236 MB in 45.5 us, 5.2 TB/s; 1 x 2048 2.8 us and
// 333 x 896 3.1, latencies): each input is read once and each output written once.  The aligned
// kernel keeps a row's h in registers between the sum of squares and the outputs (CH pieces
// of 8 elements a thread); rows longer than that read the inputs a second time for the
// pieces past it (from L2).  Rows of other alignment take the element-wise kernel, whose accesses of
// 2 bytes bound it (4096 x 4095 with a residual, 16 bits: 134 MB in 56.8 us, 2.4 TB/s).
#include "ops.h"

namespace mnb {
namespace {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// sum over the workgroup, the same in every thread
template <int WAVES>
__device__ __forceinline__ double block_sum(double v) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    __shared__ double part[WAVES];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += part[i];
  }
  return v;
}

// To 32 bits, inexact values to the neighbour with an odd last bit, among subnormals too: a later
// rounding to fewer bits then gives what one rounding of v would (rounding to nearest first
// would turn values next to an element's border into ties).
__device__ __forceinline__ float to_odd(double v) {
  const float f = (float)v;
  const double g = f;
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  if (g == v || __builtin_isinf(f)) return f;
  return __builtin_bit_cast(float, (fabs(g) > fabs(v) ? b - 1 : b) | 1u);
}

// a piece of 8 elements of x and of the residual (-0 without one, which leaves x as it is)
template <int DT>
struct Inputs {
  u4_t x = {0, 0, 0, 0}, r = {0, 0, 0, 0};
  __device__ __forceinline__ void load(const uint16_t *px, const uint16_t *pr, int64_t c) {
    constexpr uint32_t zeros = 0x80008000u;
    x = *reinterpret_cast<const u4_t *>(px + 8 * c);
    r = pr ? *reinterpret_cast<const u4_t *>(pr + 8 * c) : u4_t{zeros, zeros, zeros, zeros};
  }
  __device__ __forceinline__ static float at(const u4_t &v, int i) { return to_f32<DT>((uint16_t)(v[i >> 1] >> (16 * (i & 1)))); }
  __device__ __forceinline__ float h(int i) const { return at(x, i) + at(r, i); }
  __device__ __forceinline__ double h64(int i) const { return (double)at(x, i) + (double)at(r, i); }
};

// Is the root's inverse so far from 1 that 32 bits do not hold it, or h, in full?  (bfloat16 rows of subnormals with a
// small eps, or near the largest number; a NaN too.)
__device__ __forceinline__ bool far_norm(double rstd) { return !(rstd >= 0x1p-100 && rstd <= 0x1p100); }

// K % 8 == 0, every row 16-byte aligned; with codes K % 32 == 0.  The piece loops run to a
// multiple of THREADS so that the four lanes of a block meet in the exchanges.
// 8 waves a SIMD, so that two rows of 16 waves share a CU (500 x 16384, FP8: 16.0 us, 17.0 with 7 waves).
template <int DT, int FMT, int WAVES, int CH>
__global__ __launch_bounds__(WAVES * 64, CH <= 2 ? 8 : 4) void norm_kernel(NormParams p) {
  constexpr int THREADS = WAVES * 64;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, pieces = p.K / 8;
  const uint16_t *x = p.x + row * p.ldx, *res = p.res ? p.res + row * p.ldr : nullptr;
  Inputs<DT> in[CH];
  float h[CH][8];
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = j * THREADS + t;
    if (c < pieces) in[j].load(x, res, c);
  }
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = in[j].h64(i);
      ss = fma(d, d, ss);
      h[j][i] = in[j].h(i);
    }
  for (int c = CH * THREADS + t; c < pieces; c += THREADS) {
    Inputs<DT> more;
    more.load(x, res, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma(more.h64(i), more.h64(i), ss);
  }
  ss = block_sum<WAVES>(ss);
  const double rstd = 1.0 / sqrt(ss / p.K + (double)p.eps);
  const float r32 = (float)rstd;
  const bool far = far_norm(rstd);

  auto finish = [&](int c, const float *h8) {
    float w[8], v[8];
    load8<DT>(p.w + 8 * (int64_t)c, w);
    uint32_t border = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = h8[i] * r32 * w[i];
      // every border (ties, powers of two) has at least 16 zero bits at its end
      if constexpr (FMT >= 0) border = min(border, (__builtin_bit_cast(uint32_t, v[i]) + 4u) << 16);
    }
    uint32_t amax = 0;            // the largest magnitude: of the thread, then of the block's four
    const auto largest = [&] {
      amax = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = max(amax, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
    };
    bool repeat = far;
    if constexpr (FMT >= 0) {
      largest();
      // below 2^-100 the block may be one whose borders end in fewer zeros, or whose v are subnormal
      repeat = repeat || border <= 8u << 16 || amax - 1 < ((127u - 100) << 23) - 1;
    }
    if (repeat) {   // before hidden is stored, which may be in the place of x or residual
      Inputs<DT> again;
      again.load(x, res, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_odd(again.h64(i) * rstd * (double)w[i]);
      if constexpr (FMT >= 0) largest();
    }
    if (p.hidden) {
      uint16_t *to = p.hidden + row * p.ldh + 8 * (int64_t)c;
      // with MX outputs the next call reads those and not the hidden rows: past the caches
      // 8192 x 4096 takes 45.8 us, not 49.3 (4096 x 8192 with 16-bit outputs 51.4, not 49.9, so not there)
      if constexpr (FMT >= 0)
        __builtin_nontemporal_store(u4_t{pack2<DT>(h8[0], h8[1]), pack2<DT>(h8[2], h8[3]), pack2<DT>(h8[4], h8[5]), pack2<DT>(h8[6], h8[7])},
                                    reinterpret_cast<u4_t *>(to));
      else store8<DT>(to, h8);
    }
    if (p.y) store8<DT>(p.y + row * p.ldy + 8 * (int64_t)c, v);
    if constexpr (FMT >= 0) {
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
      const uint32_t e = mx_scale<FMT>(amax);
      const float inv = mx_inverse(e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e == 255 ? 0.f : v[i] * inv;
      uint8_t *out = p.codes + row * p.ldc;
      if constexpr (FMT == MX_FP4) *reinterpret_cast<uint32_t *>(out + 4 * (int64_t)c) = fp4_codes(v);
      else *reinterpret_cast<u2_t *>(out + 8 * (int64_t)c) = u2_t{fp8_codes4(v), fp8_codes4(v + 4)};
      if ((c & 3) == 0) p.scales[row * p.lds + (c >> 2)] = (uint8_t)e;
    }
  };
  // K % 32 == 0 with codes: the four threads of a block are all inside the row or all past it
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = j * THREADS + t;
    if (c < pieces) finish(c, h[j]);
  }
  for (int c = CH * THREADS + t; c < pieces; c += THREADS) {
    Inputs<DT> more;
    more.load(x, res, c);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = more.h(i);
    finish(c, v);
  }
}

// any K and alignment, 16-bit outputs only: one element at a time, the inputs read twice
template <int DT>
__global__ __launch_bounds__(256) void norm_any_kernel(NormParams p) {
  const int64_t row = blockIdx.x;
  const uint16_t *x = p.x + row * p.ldx, *res = p.res ? p.res + row * p.ldr : nullptr;
  double ss = 0.0;
  for (int k = threadIdx.x; k < p.K; k += 256) {
    const double h = (double)to_f32<DT>(x[k]) + (res ? (double)to_f32<DT>(res[k]) : 0.0);
    ss = fma(h, h, ss);
  }
  ss = block_sum<4>(ss);
  const double rstd = 1.0 / sqrt(ss / p.K + (double)p.eps);
  const float r32 = (float)rstd;
  const bool far = far_norm(rstd);
  for (int k = threadIdx.x; k < p.K; k += 256) {
    const float a = to_f32<DT>(x[k]), b = res ? to_f32<DT>(res[k]) : 0.f, h = a + b, w = to_f32<DT>(p.w[k]);
    if (p.hidden) p.hidden[row * p.ldh + k] = from_f32<DT>(h);
    p.y[row * p.ldy + k] = from_f32<DT>(far ? to_odd(((double)a + (double)b) * rstd * (double)w) : h * r32 * w);
  }
}

bool aligned16(const void *p, int64_t ld) { return !p || (((uintptr_t)p | (uintptr_t)(2 * ld)) & 15) == 0; }

template <int DT, int FMT>
hipError_t launch(const NormParams &p, hipStream_t s) {
  const dim3 grid((uint32_t)p.M);
  if constexpr (FMT < 0) {
    if (p.K % 8 || !aligned16(p.x, p.ldx) || !aligned16(p.res, p.ldr) || !aligned16(p.hidden, p.ldh) ||
        !aligned16(p.y, p.ldy) || !aligned16(p.w, 0)) {
      hipLaunchKernelGGL((norm_any_kernel<DT>), grid, dim3(256), 0, s, p);
      return hipGetLastError();
    }
  }
  // As few pieces a thread as give a workgroup the row, of 4 or 16 waves: with 4 pieces in 4 waves 8192 x 2560
  // (FP4 out, the kernel alone) takes 41.7 us, 8192 x 4096 (FP8) 53.0 and 4096 x 8192 (16 bits) 51.4, so
  // 30.3, 45.8 and 49.9; 16 waves for 2560 and 4096 k take 61.2 and 70.4.
  if (p.K <= 2048) hipLaunchKernelGGL((norm_kernel<DT, FMT, 4, 1>), grid, dim3(256), 0, s, p);
  else if (p.K <= 4096) hipLaunchKernelGGL((norm_kernel<DT, FMT, 4, 2>), grid, dim3(256), 0, s, p);
  else if (p.K <= 8192) hipLaunchKernelGGL((norm_kernel<DT, FMT, 16, 1>), grid, dim3(1024), 0, s, p);
  else if (p.K <= 16384) hipLaunchKernelGGL((norm_kernel<DT, FMT, 16, 2>), grid, dim3(1024), 0, s, p);
  else hipLaunchKernelGGL((norm_kernel<DT, FMT, 16, 4>), grid, dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(int dtype, int fmt, const NormParams &p, hipStream_t s) {
  if (dtype == DT_F16)
    return fmt < 0          ? launch<DT_F16, -1>(p, s)
           : fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s)
                           : launch<DT_F16, MX_FP8>(p, s);
  return fmt < 0          ? launch<DT_BF16, -1>(p, s)
         : fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s)
                         : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
