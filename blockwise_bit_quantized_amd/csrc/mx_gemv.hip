// mx_gemv.hip -- MX product for up to 32 rows: the weight streams once for all of them.
//
// Bound by the weight's bytes.  A wave owns the 32 weight rows of one packed operand and a
// share of K: it loads 1 KiB of codes per step of 64 k straight into the matrix
// instruction's operand (the packed layout is the operand's), four steps and their scale
// dword at a time, the next four while it multiplies, and the X rows (from L2) as the other
// operand.  KSPLIT waves of a workgroup share a row's K when the rows alone give too few
// waves to keep the memory busy; their partial sums meet in LDS in a fixed order.
#include "mx_mfma.h"

namespace mnb {
namespace {

template <int DT, int FMT, int KSPLIT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void gemv_kernel(MxMatmulParams p) {
  constexpr int XB = FMT == MX_FP4 ? 32 : 64;   // X bytes per row and step
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int ks = wave % KSPLIT;
  // units past the end repeat the last one and store nothing
  const int units = p.NG * 2, unit_raw = blockIdx.x * (WAVES / KSPLIT) + wave / KSPLIT;
  const int unit = min(unit_raw, units - 1);
  const int64_t g = unit >> 1;
  const int f = unit & 1;

  const uint8_t *wbase = p.wq + (g * p.KS * 2 + f) * 1024 + lane * 16;
  const uint32_t *sbase = reinterpret_cast<const uint32_t *>(p.sc) + (g * p.KB * 2 + f) * 64 + lane;
  const bool row_ok = r < p.M;
  const uint8_t *xrow = p.codes + (int64_t)(row_ok ? r : 0) * p.ldc;
  const uint8_t *srow = p.scales + (int64_t)(row_ok ? r : 0) * p.lds;
  const int xbytes = FMT == MX_FP4 ? p.K / 2 : p.K, blocks = p.K / kBlock;

  struct Weights {
    u4_t w[4];
    uint32_t s;
  };
  // steps 4 kb .. 4 kb + 3; past K the last step again (its X is 0)
  auto load = [&](Weights &o, int kb) {
    o.s = sbase[(int64_t)kb * 128];
#pragma unroll
    for (int j = 0; j < 4; ++j) o.w[j] = *reinterpret_cast<const u4_t *>(wbase + (int64_t)min(kb * 4 + j, p.KS - 1) * 2048);
  };
  acc_t acc = {};
  auto multiply = [&](const Weights &o, int kb) {
    const u4_t zero = {0, 0, 0, 0};
    u4_t x0[4], x1[4];
    const u2_t sx = *reinterpret_cast<const u2_t *>(srow + kb * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = (kb * 4 + j) * XB + h * 16;   // bytes past the row's end stay 0
      x0[j] = x1[j] = zero;
      if (row_ok && at < xbytes) x0[j] = *reinterpret_cast<const u4_t *>(xrow + at);
      if (FMT == MX_FP8 && row_ok && at + 32 < xbytes) x1[j] = *reinterpret_cast<const u4_t *>(xrow + at + 32);
    }
    unroll<0, 4>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      // rows past M and blocks past K have codes 0; their scale must not be a stray NaN
      const uint32_t s = row_ok && (kb * 4 + j) * 2 + h < blocks ? sx[j / 2] >> (16 * (j & 1) + 8 * h) : 0u;
      acc = mx_mfma<FMT, j, 0>(o.w[j], x0[j], x1[j], acc, o.s, s);
    });
  };
  Weights a, b;
  int kb = ks;
  if (kb < p.KB) load(a, kb);
  for (; kb < p.KB; kb += 2 * KSPLIT) {
    if (kb + KSPLIT < p.KB) load(b, kb + KSPLIT);
    multiply(a, kb);
    if (kb + KSPLIT >= p.KB) break;
    if (kb + 2 * KSPLIT < p.KB) load(a, kb + 2 * KSPLIT);
    multiply(b, kb + KSPLIT);
  }

  if constexpr (KSPLIT > 1) {
    __shared__ acc_t red[WAVES][64];
    if (ks) red[wave][lane] = acc;
    __syncthreads();
    if (ks) return;
#pragma unroll
    for (int i = 1; i < KSPLIT; ++i) acc += red[wave + i][lane];
  }
  if (unit_raw < units && row_ok) store_cols<DT>(p, r, 64 * g + 32 * h + 16 * f, acc);
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  const int ksplit = mx_gemv_ksplit(p.N, p.K), waves = ksplit < 4 ? 4 : ksplit;
  const uint32_t grid = (uint32_t)(((int64_t)p.NG * 2 * ksplit + waves - 1) / waves);
  const dim3 g(grid), b(waves * 64);
  switch (ksplit) {
    case 1: hipLaunchKernelGGL((gemv_kernel<DT, FMT, 1, 4>), g, b, 0, s, p); break;
    case 2: hipLaunchKernelGGL((gemv_kernel<DT, FMT, 2, 4>), g, b, 0, s, p); break;
    case 4: hipLaunchKernelGGL((gemv_kernel<DT, FMT, 4, 4>), g, b, 0, s, p); break;
    default: hipLaunchKernelGGL((gemv_kernel<DT, FMT, 8, 8>), g, b, 0, s, p); break;
  }
  return hipGetLastError();
}

}  // namespace

// the smallest split that gives 8 waves per CU, but not more waves than 256-k parts
int mx_gemv_ksplit(int N, int K) {
  const int64_t units = ((int64_t)N + 63) / 64 * 2;
  const int parts = (K + kMxScaleK - 1) / kMxScaleK;
  int s = 1;
  while (s < 8 && units * s < 8 * kCUs && 2 * s <= parts) s *= 2;
  return s;
}

hipError_t launch_mx_gemv(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s) {
  if (dtype == DT_F16) return fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s) : launch<DT_F16, MX_FP8>(p, s);
  return fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s) : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
