// mx_gemv.hip -- MX product for up to 32 rows: the weight streams once for all of them.
//
// Bound by the weight's bytes (1x49152x2048: 10.0 us, 5.4 TB/s out of the caches; 1x8192x2048
// 3.5 us, where a launch and one pass of latencies are most of it).  A wave owns RB operands
// of 16 weight rows and a share of K: it loads 1 KiB of codes per step of 128 k straight into
// the matrix instruction's operand (the packed layout is the operand's), four steps and their
// scale dword at a time, and one or two operands of 16 X rows (L2).  Weight and X loads are
// issued in turn, so that the first step can start while the rest are under way: all weights
// first took 6.2 us where this takes 5.5 (8x49152x576).  KSPLIT waves of a workgroup share a
// row's K when the rows alone give too few waves to keep the memory busy; their partial sums
// meet in LDS in a fixed order.  Two X operands for 17 to 32 rows take 5.9 us at
// 32x8192x2048 and 16.1 at 32x49152x2048, the tiled kernel 7.5 and 21.4.  With FP4 X:
// 1x49152x2048 9.8 us, 8x49152x576 5.3, 32x8192x2048 5.7, 32x49152x2048 14.4, 24x16384x4096 10.3.
//
// Farthest from the weight's bytes are long K and few columns (1x2560x9728 6.4 us with FP8 X, 32x2560x9728
// 13.5, FP4 9.2, for 2.9): N gives 160 workgroups of at most four waves that share a K, and a wave issues a
// 512-k part's loads when it has multiplied the part before.
#include "mx_mfma.h"

namespace mnb {
namespace {

constexpr int kWaves = 4;

template <int DT, int FMT, int KSPLIT, int CT, int RB>
__global__ __launch_bounds__(kWaves * 64) void gemv_kernel(MxMatmulParams p) {
  constexpr int XB = FMT == MX_FP4 ? 64 : 128;   // X bytes per row and step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, b = lane >> 4;
  const int ks = wave % KSPLIT;
  // units past the end repeat the last one and store nothing
  const int units = p.NG * (4 / RB), unit_raw = blockIdx.x * (kWaves / KSPLIT) + wave / KSPLIT;
  const int unit = min(unit_raw, units - 1);
  const int64_t g = unit / (4 / RB);
  const int f = unit % (4 / RB) * RB;

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

  f4_t acc[CT][RB];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int o = 0; o < RB; ++o) acc[c][o] = f4_t{0.f, 0.f, 0.f, 0.f};
  for (int kb = ks; kb < p.KB; kb += KSPLIT) {
    u4_t w[RB][4], x0[CT][4], x1[CT][4], sx[CT];
    uint32_t sw[RB];
    const u4_t zero = {0, 0, 0, 0};
#pragma unroll
    for (int o = 0; o < RB; ++o) sw[o] = sbase[(int64_t)kb * 256 + o * 64];
#pragma unroll
    for (int c = 0; c < CT; ++c) sx[c] = *reinterpret_cast<const u4_t *>(srow[c] + kb * 16);
    // weight and X loads in turn: the first step's operands come first
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int o = 0; o < RB; ++o) {
        w[o][j] = zero;
        if (kb * 4 + j < p.KS)
          w[o][j] = *reinterpret_cast<const u4_t *>(wbase + (int64_t)(kb * 4 + j) * 4096 + o * 1024);
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
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
#pragma unroll
        for (int o = 0; o < RB; ++o) acc[c][o] = mx_mfma<FMT, j>(w[o][j], x0[c][j], x1[c][j], acc[c][o], sw[o], s);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }

  if constexpr (KSPLIT > 1) {
    __shared__ f4_t red[CT * RB][kWaves][64];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int o = 0; o < RB; ++o) red[c * RB + o][wave][lane] = acc[c][o];
    __syncthreads();
    if (ks) return;
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int o = 0; o < RB; ++o)
#pragma unroll
        for (int i = 1; i < KSPLIT; ++i) acc[c][o] += red[c * RB + o][wave + i][lane];
  }
  if (unit_raw >= units) return;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int o = 0; o < RB; ++o) {
      const int64_t n = 64 * g + 16 * b + 4 * (f + o);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row_ok[c] && n + i < p.N) store_cols<DT>(p, 16 * c + r, n + i, acc[c][o][i]);
    }
}

template <int DT, int FMT, int CT, int RB>
hipError_t launch_rows(const MxMatmulParams &p, hipStream_t s) {
  const int ksplit = mx_gemv_ksplit(FMT, p.M, p.N, p.K);
  const uint32_t grid = (uint32_t)(((int64_t)p.NG * (4 / RB) * ksplit + kWaves - 1) / kWaves);
  const dim3 g(grid), b(kWaves * 64);
  if (ksplit == 1) hipLaunchKernelGGL((gemv_kernel<DT, FMT, 1, CT, RB>), g, b, 0, s, p);
  else if (ksplit == 2) hipLaunchKernelGGL((gemv_kernel<DT, FMT, 2, CT, RB>), g, b, 0, s, p);
  else hipLaunchKernelGGL((gemv_kernel<DT, FMT, 4, CT, RB>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int DT, int FMT, int CT>
hipError_t launch_cols(const MxMatmulParams &p, hipStream_t s) {
  switch (mx_gemv_operands(FMT, p.M, p.N, p.K)) {
    case 1: return launch_rows<DT, FMT, CT, 1>(p, s);
    case 2: return launch_rows<DT, FMT, CT, 2>(p, s);
    default: return launch_rows<DT, FMT, CT, 4>(p, s);
  }
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  return p.M <= 16 ? launch_cols<DT, FMT, 1>(p, s) : launch_cols<DT, FMT, 2>(p, s);
}

}  // namespace

// Every wave reads all of X from L2, so with one operand a wave X's bytes pass N / 16 times.
// Where that is much (24 MB, 48 MB) a wave takes 2 or 4 operands and reads X once for them,
// as long as there stay about two waves per CU.  Measured with 1 / 2 / 4 operands, us:
// 32x49152x2048 FP8 28.9 / 18.7 / 16.1, 24x16384x4096 FP8 17.7 / 12.6 / 11.4, 32x8192x2048
// FP8 7.4 / 5.9 / 7.1, 32x49152x576 FP8 9.9 / 8.5 / 10.2 (few steps a wave), 8x49152x576
// FP8 5.4 / 5.7 / 6.0, 32x2560x9728 FP8 13.7 / 15.3 / 17.9 (few waves).
int mx_gemv_operands(int fmt, int M, int N, int K) {
  const int64_t units = ((int64_t)N + 63) / 64 * 4, traffic = units * M * (fmt == MX_FP4 ? K / 2 : K);
  const int parts = (K + kMxScaleK - 1) / kMxScaleK, split = parts < kWaves ? parts : kWaves;
  int rb = traffic < (24 << 20) ? 1 : traffic < (48 << 20) || K < 1024 ? 2 : 4;
  while (rb > 1 && units / rb * split < 600) rb /= 2;
  return rb;
}

// The smallest split that gives 8 waves per CU, as long as it shortens the longest wave's K:
// three 512-k parts over four waves (16x1000x1056) take 3.1 us, over two 3.5.
int mx_gemv_ksplit(int fmt, int M, int N, int K) {
  const int64_t units = ((int64_t)N + 63) / 64 * 4 / mx_gemv_operands(fmt, M, N, K);
  const int parts = (K + kMxScaleK - 1) / kMxScaleK;
  int s = 1;
  while (s < kWaves && units * s < 8 * kCUs && s < parts) s *= 2;
  return s;
}

hipError_t launch_mx_gemv(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s) {
  if (dtype == DT_F16) return fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s) : launch<DT_F16, MX_FP8>(p, s);
  return fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s) : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
