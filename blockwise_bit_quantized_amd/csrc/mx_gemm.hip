// mx_gemm.hip -- MX product for more than 16 rows.
//
// 128 x 128 outputs per workgroup of 4 waves, each 64 x 64 (4 x 4 scaled 16x16x128 matrix
// instructions per step of 128 k).  The X tile goes through LDS (two buffers, the next
// step's loads in registers meanwhile), 16-byte chunks XOR-swizzled so that the 16 rows an
// operand read touches fall on distinct banks; the weights are packed in operand order and
// load straight into registers.
#include "mx_mfma.h"

namespace mnb {
namespace {

constexpr int BM = 128, BN = 128, kThreads = 256;

// LDS byte of 16-byte chunk c of row m: rows of 128 bytes (FP8) or 64 (FP4)
template <int FMT>
__device__ __forceinline__ int x_chunk(int m, int c) {
  return FMT == MX_FP8 ? m * 128 + ((c ^ ((m >> 1) & 7)) << 4) : m * 64 + ((c ^ ((m >> 2) & 3)) << 4);
}

template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void gemm_kernel(MxMatmulParams p) {
  constexpr int XB = FMT == MX_FP4 ? 64 : 128, XC = XB / 16;
  constexpr int LD = BM * XC / kThreads;   // 16-byte loads per thread and step
  __shared__ uint8_t xt[2][BM * XB] __attribute__((aligned(16)));
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int r = lane & 15, b = lane >> 4;
  const int MT = (p.M + BM - 1) / BM;
  const int tile = blockIdx.x;
  const int64_t m0 = (int64_t)(tile % MT) * BM, n0 = (int64_t)(tile / MT) * BN;
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
  const int xbytes = FMT == MX_FP4 ? p.K / 2 : p.K, blocks = p.K / kBlock;

  const int64_t g = min((n0 + wn) / 64, (int64_t)p.NG - 1);   // past the end: a copy, not stored
  const uint8_t *wbase = p.wq + g * p.KS * 4096 + lane * 16;
  const uint32_t *sbase = reinterpret_cast<const uint32_t *>(p.sc) + g * p.KB * 256 + lane;

  const uint8_t *xsrc[LD];
  int xcol[LD], xdst[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int id = i * kThreads + t, m = id / XC, c = id % XC;
    xsrc[i] = p.codes + min(m0 + m, (int64_t)p.M - 1) * p.ldc;
    xcol[i] = c * 16;
    xdst[i] = x_chunk<FMT>(m, c);
  }
  const uint8_t *srow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) srow[i] = p.scales + min(m0 + wm + 16 * i + r, (int64_t)p.M - 1) * p.lds;

  u4_t xr[LD], w[4];
  auto load = [&](int step) {
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int o = step * XB + xcol[i];
      const u4_t zero = {0, 0, 0, 0};
      xr[i] = o < xbytes ? *reinterpret_cast<const u4_t *>(xsrc[i] + o) : zero;
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) w[f] = *reinterpret_cast<const u4_t *>(wbase + (int64_t)step * 4096 + f * 1024);
  };

  f4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[i][f] = f4_t{0.f, 0.f, 0.f, 0.f};

  load(0);
  uint32_t sw[4];
  u4_t sx[4];
  auto step_body = [&](auto jc, int kb) {
    constexpr int J = decltype(jc)::value;
    const int step = kb * 4 + J;
    if (step >= p.KS) return;
    uint8_t *buf = xt[J & 1];   // 4 steps per scale dword: the parity of the step is J's
#pragma unroll
    for (int i = 0; i < LD; ++i) *reinterpret_cast<u4_t *>(buf + xdst[i]) = xr[i];
    u4_t wc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) wc[f] = w[f];
    __syncthreads();
    if (step + 1 < p.KS) load(step + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = wm + 16 * i + r;
      const u4_t x0 = *reinterpret_cast<const u4_t *>(buf + x_chunk<FMT>(m, b));
      u4_t x1 = {0, 0, 0, 0};
      if constexpr (FMT == MX_FP8) x1 = *reinterpret_cast<const u4_t *>(buf + x_chunk<FMT>(m, b + 4));
      const uint32_t s = step * 4 + b < blocks ? sx[i][J] >> (8 * b) : 0u;
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[i][f] = mx_mfma<FMT, J>(wc[f], x0, x1, acc[i][f], sw[f], s);
    }
  };
  for (int kb = 0; kb < p.KB; ++kb) {
#pragma unroll
    for (int f = 0; f < 4; ++f) sw[f] = sbase[(int64_t)kb * 256 + f * 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) sx[i] = *reinterpret_cast<const u4_t *>(srow[i] + kb * 16);
    step_body(std::integral_constant<int, 0>{}, kb);
    step_body(std::integral_constant<int, 1>{}, kb);
    step_body(std::integral_constant<int, 2>{}, kb);
    step_body(std::integral_constant<int, 3>{}, kb);
  }

  const int64_t n = n0 + wn + 16 * b;   // 16 consecutive columns per lane
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + wm + 16 * i + r;
    if (m >= p.M) continue;
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + 4 * f + e < p.N) store_cols<DT>(p, m, n + 4 * f + e, acc[i][f][e]);
  }
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  const int64_t tiles = ((int64_t)p.M + BM - 1) / BM * (((int64_t)p.N + BN - 1) / BN);
  hipLaunchKernelGGL((gemm_kernel<DT, FMT>), dim3((uint32_t)tiles), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int mx_gemm_splits(int M, int N, int K, int fmt) {
  (void)M; (void)N; (void)K; (void)fmt;
  return 1;
}

hipError_t launch_mx_gemm(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s) {
  if (dtype == DT_F16) return fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s) : launch<DT_F16, MX_FP8>(p, s);
  return fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s) : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
