// mx_gemv.hip -- MX product for up to 32 rows: the weight streams once for all of them.
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

template <int DT, int FMT, int KSPLIT, int CT>
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
  // X row r of column operand c; rows past M are zero and not stored
  bool row_ok[CT];
  const uint8_t *xrow[CT], *srow[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    row_ok[c] = 16 * c + r < p.M;
    xrow[c] = p.codes + (int64_t)(row_ok[c] ? 16 * c + r : 0) * p.ldc;
    srow[c] = p.scales + (int64_t)(row_ok[c] ? 16 * c + r : 0) * p.lds;
  }
  const int xbytes = FMT == MX_FP4 ? p.K / 2 : p.K, blocks = p.K / kBlock;

  f4_t acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = f4_t{0.f, 0.f, 0.f, 0.f};
  for (int kb = ks; kb < p.KB; kb += KSPLIT) {
    u4_t w[4], x0[CT][4], x1[CT][4], sx[CT];
    const u4_t zero = {0, 0, 0, 0};
    const uint32_t sw = sbase[(int64_t)kb * 256];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = zero;
      if (kb * 4 + j < p.KS) w[j] = *reinterpret_cast<const u4_t *>(wbase + (int64_t)(kb * 4 + j) * 4096);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      sx[c] = *reinterpret_cast<const u4_t *>(srow[c] + kb * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = (kb * 4 + j) * XB + b * 16;   // bytes past the row's end stay 0
        x0[c][j] = x1[c][j] = zero;
        if (row_ok[c] && o < xbytes) x0[c][j] = *reinterpret_cast<const u4_t *>(xrow[c] + o);
        if (FMT == MX_FP8 && row_ok[c] && o + 64 < xbytes) x1[c][j] = *reinterpret_cast<const u4_t *>(xrow[c] + o + 64);
      }
    }
    auto step = [&](auto jc) {
      constexpr int j = decltype(jc)::value;
      if (kb * 4 + j >= p.KS) return;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        // rows past M and blocks past K have codes 0; their scale must not be a stray NaN
        const uint32_t s = row_ok[c] && (kb * 4 + j) * 4 + b < blocks ? sx[c][j] >> (8 * b) : 0u;
        acc[c] = mx_mfma<FMT, j>(w[j], x0[c][j], x1[c][j], acc[c], sw, s);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }

  if constexpr (KSPLIT > 1) {
    __shared__ f4_t red[CT][kWaves][64];
#pragma unroll
    for (int c = 0; c < CT; ++c) red[c][wave][lane] = acc[c];
    __syncthreads();
    if (ks) return;
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 1; i < KSPLIT; ++i) acc[c] += red[c][wave + i][lane];
  }
  if (unit_raw >= units) return;
  const int64_t n = 64 * g + 16 * b + 4 * f;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row_ok[c] && n + i < p.N) store_cols<DT>(p, 16 * c + r, n + i, acc[c][i]);
}

template <int DT, int FMT, int CT>
hipError_t launch_rows(const MxMatmulParams &p, hipStream_t s) {
  const int ksplit = mx_gemv_ksplit(p.N, p.K);
  const uint32_t grid = (uint32_t)(((int64_t)p.NG * 4 * ksplit + kWaves - 1) / kWaves);
  const dim3 g(grid), b(kWaves * 64);
  if (ksplit == 1) hipLaunchKernelGGL((gemv_kernel<DT, FMT, 1, CT>), g, b, 0, s, p);
  else if (ksplit == 2) hipLaunchKernelGGL((gemv_kernel<DT, FMT, 2, CT>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gemv_kernel<DT, FMT, 4, CT>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  return p.M <= 16 ? launch_rows<DT, FMT, 1>(p, s) : launch_rows<DT, FMT, 2>(p, s);
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
