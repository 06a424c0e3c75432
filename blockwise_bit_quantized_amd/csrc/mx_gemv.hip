// mx_gemv.hip -- MX product for up to 16 rows: the weight streams once for all of them.
//
// Bound by the weight's bytes.  A wave owns the 16 weight rows of one packed operand and a
// share of K: it loads 1 KiB of codes per step of 128 k straight into the matrix
// instruction's operand (the packed layout is the operand's), four steps and their scale
// dword at a time, and the X rows (L2) as the other operand.  KSPLIT waves of a workgroup
// share a row's K when the rows alone give too few waves to keep the memory busy; their
// partial sums meet in LDS in a fixed order.
#include "mx_mfma.h"

namespace mnb {
namespace {

constexpr int kWaves = 4;

template <int DT, int FMT, int KSPLIT>
__global__ __launch_bounds__(kWaves * 64) void gemv_kernel(MxMatmulParams p) {
  constexpr int XB = FMT == MX_FP4 ? 64 : 128;   // X bytes per row and step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, b = lane >> 4;
  const int ks = wave % KSPLIT;
  // units past the end repeat the last one and store nothing
  const int units = p.NG * 4, unit_raw = blockIdx.x * (kWaves / KSPLIT) + wave / KSPLIT;
  const int unit = min(unit_raw, units - 1);
  const int64_t g = unit >> 2;
  const int f = unit & 3;

  const uint8_t *wbase = p.wq + (g * p.KS * 4 + f) * 1024 + lane * 16;
  const uint32_t *sbase = reinterpret_cast<const uint32_t *>(p.sc) + (g * p.KB * 4 + f) * 64 + lane;
  const bool row_ok = r < p.M;
  const uint8_t *xrow = p.codes + (int64_t)(row_ok ? r : 0) * p.ldc;
  const uint8_t *srow = p.scales + (int64_t)(row_ok ? r : 0) * p.lds;
  const int xbytes = FMT == MX_FP4 ? p.K / 2 : p.K, blocks = p.K / kBlock;

  f4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = ks; kb < p.KB; kb += KSPLIT) {
    u4_t w[4], x0[4], x1[4];
    const uint32_t sw = sbase[(int64_t)kb * 256];
    const u4_t sx = *reinterpret_cast<const u4_t *>(srow + kb * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int step = kb * 4 + j;
      const u4_t zero = {0, 0, 0, 0};
      w[j] = x0[j] = x1[j] = zero;
      if (step < p.KS) {
        w[j] = *reinterpret_cast<const u4_t *>(wbase + (int64_t)step * 4096);
        const int o = step * XB + b * 16;   // bytes past the row's end stay 0
        if (row_ok && o < xbytes) x0[j] = *reinterpret_cast<const u4_t *>(xrow + o);
        if (FMT == MX_FP8 && row_ok && o + 64 < xbytes) x1[j] = *reinterpret_cast<const u4_t *>(xrow + o + 64);
      }
    }
    // rows past M and blocks past K have codes 0; their scale must not be a stray NaN
    auto xs = [&](int j) { return row_ok && (kb * 4 + j) * 4 + b < blocks ? sx[j] >> (8 * b) : 0u; };
    if (kb * 4 + 0 < p.KS) acc = mx_mfma<FMT, 0>(w[0], x0[0], x1[0], acc, sw, xs(0));
    if (kb * 4 + 1 < p.KS) acc = mx_mfma<FMT, 1>(w[1], x0[1], x1[1], acc, sw, xs(1));
    if (kb * 4 + 2 < p.KS) acc = mx_mfma<FMT, 2>(w[2], x0[2], x1[2], acc, sw, xs(2));
    if (kb * 4 + 3 < p.KS) acc = mx_mfma<FMT, 3>(w[3], x0[3], x1[3], acc, sw, xs(3));
  }

  if constexpr (KSPLIT > 1) {
    __shared__ f4_t red[kWaves][64];
    red[wave][lane] = acc;
    __syncthreads();
    if (ks) return;
#pragma unroll
    for (int i = 1; i < KSPLIT; ++i) acc += red[wave + i][lane];
  }
  if (unit_raw >= units || !row_ok) return;
  const int64_t n = 64 * g + 16 * b + 4 * f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) store_cols<DT>(p, r, n + i, acc[i]);
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  const int ksplit = mx_gemv_ksplit(p.N, p.K);
  const uint32_t grid = (uint32_t)(((int64_t)p.NG * 4 * ksplit + kWaves - 1) / kWaves);
  const dim3 g(grid), b(kWaves * 64);
  if (ksplit == 1) hipLaunchKernelGGL((gemv_kernel<DT, FMT, 1>), g, b, 0, s, p);
  else if (ksplit == 2) hipLaunchKernelGGL((gemv_kernel<DT, FMT, 2>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gemv_kernel<DT, FMT, 4>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace

// the smallest split that gives 8 waves per CU, but not more waves than 512-k parts
int mx_gemv_ksplit(int N, int K) {
  const int64_t units = ((int64_t)N + 63) / 64 * 4;
  const int parts = (K + kMxScaleK - 1) / kMxScaleK;
  int s = 1;
  while (s < kWaves && units * s < 8 * kCUs && 2 * s <= parts) s *= 2;
  return s;
}

hipError_t launch_mx_gemv(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s) {
  if (dtype == DT_F16) return fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s) : launch<DT_F16, MX_FP8>(p, s);
  return fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s) : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
