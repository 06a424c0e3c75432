// mx_gemm.hip -- MX product for more rows than the weight-streaming kernel takes.
//
// Bound by the matrix cores where there is enough work: an instruction of 32 x 32 outputs and
// 64 k takes 32 cycles (FP4 X) or 64 (FP8 X).  A workgroup owns BM x BN outputs, a wave MF x
// NF operands of 32 rows and 32 columns.
//
// X goes through LDS in steps of 128 bytes a row (128 k of FP8, 256 of FP4), a ring of
// D + 1 slots filled by direct-to-LDS loads D steps ahead; a row's eight 16-byte chunks are
// XOR-swizzled by the row through the source address (the loads write lanes
// consecutively), so that the 16 rows of an operand read fall on distinct banks.  Weights are
// packed in operand order and load straight into registers, a step ahead (D with PRE).  The X scales of
// up to 4096 k are staged in LDS before the steps ([chunk of 512 k][row][16 bytes], where
// the rows of an operand are consecutive) and read 4 blocks at a time; weight scales are
// one dword per operand and 256 k.  Loads, LDS reads and products are interleaved: a wave whose
// loads wait to be accepted issues nothing.
//
// With PRE the X operands of the next step are read into a second register set during the
// current step, so a single wave per SIMD does not wait for LDS.
#include "mx_mfma.h"

namespace mnb {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane to LDS at dst + 16 lane: address = descriptor base + voff + soff
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 16, voff, soff, 0, 0);
}
// s_waitcnt with vmcnt = N (gfx9 encoding: vmcnt bits 3:0 and 15:14), other counters free
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// LDS accesses done, workgroup barrier; the clobber keeps memory accesses on their side
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));   // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}
// keeps the order of the loads on either side, which the vmcnt waits count
__device__ __forceinline__ void pin() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// the value is computed here (an empty use the compiler cannot move)
__device__ __forceinline__ void keep(acc_t &v) { asm volatile("" : "+v"(v)); }

constexpr int kPanel = 8;    // 512-k chunks of X scales in LDS at a time

template <int DT, int FMT, int BM, int WM, int WN, int NF, int D, bool PRE>
__global__ __launch_bounds__(WM * WN * 64, PRE ? 1 : 2) void gemm_kernel(MxMatmulParams p) {
  constexpr int WAVES = WM * WN, BN = WN * NF * 32, MF = BM / WM / 32;
  constexpr int SUB = FMT == MX_FP4 ? 4 : 2;      // instructions per step, operand pair
  constexpr int SLOTS = D + 1, SLOT = BM * 128;
  constexpr int XQ = BM / 8 / WAVES;              // X loads per wave and step (8 rows each)
  constexpr int WQ = SUB * NF;                    // weight loads per wave and step
  // weight register sets, one instruction's each: without PRE those of a step and half of the
  // next one's, whose other half takes the sets that the step has done with
  constexpr int WS = PRE ? SLOTS * SUB : SUB * 3 / 2, EARLY = SUB / 2;
  constexpr int GROUPS = SUB * MF, OPS = XQ + WQ + NF;   // X operands and loads of a step
  // steps per unrolled loop body: a multiple of the slots, of 4 instructions and of the sets
  constexpr int U = PRE ? 4 : FMT == MX_FP4 ? 3 : 6;
  static_assert(U % SLOTS == 0 && U * SUB % WS == 0 && U * SUB % 4 == 0, "slots, sets and scale bytes are compile-time");
  static_assert(PRE ? D >= 2 : D == 2, "ring depth");
  static_assert(PRE || (EARLY * NF + NF + XQ) * GROUPS / OPS >= EARLY * MF, "late weight loads");
  // loads younger than the ones a step waits for at its start
  constexpr int YOUNGER = PRE ? (D - 2) * (XQ + WQ) + WQ : XQ + (SUB - EARLY) * NF;
  static_assert(XQ >= 1 && 8 * XQ * WAVES == BM, "X rows per wave");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SLOTS * SLOT + kPanel * BM * 16];
  uint8_t *sxl = smem + SLOTS * SLOT;

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);   // uniform: addresses stay scalar
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;
  // workgroup ids are dealt to the 8 XCDs by id modulo 8: each XCD takes a contiguous range of
  // tiles, in bands of 8 tile rows, so that it shares X rows and weight columns in its L2
  const int MT = (p.M + BM - 1) / BM, NT = (p.N + BN - 1) / BN, tiles = MT * NT;
  const int per = (tiles + 7) / 8, xcd = blockIdx.x & 7;
  const int tile = xcd * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || tile >= tiles) return;
  const int band = tile / (8 * NT), rows_in = min(8, MT - band * 8), in = tile - band * 8 * NT;
  const int64_t m0 = (int64_t)(band * 8 + in % rows_in) * BM, n0 = (int64_t)(in / rows_in) * BN;

  const int xbytes = FMT == MX_FP4 ? p.K / 2 : p.K, blocks = p.K / kBlock;
  const int steps = (xbytes + 127) / 128;
  const int tail = (xbytes & 127) >> 4;   // 16-byte chunks of a last step that K ends inside, 0: whole
  const int64_t last_row = (int64_t)min((int64_t)BM, p.M - m0) - 1;   // of this tile; further rows repeat it
  // every address is in range by construction (rows are clamped, offsets stay below 2^31)
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(p.codes + m0 * p.ldc, 0x7fffffffL);
  const __amdgpu_buffer_rsrc_t sr = buffer_rsrc(p.scales + m0 * p.lds, 0x7fffffffL);
  uint32_t xvoff[XQ];
#pragma unroll
  for (int q = 0; q < XQ; ++q) {
    const int row = (wave * XQ + q) * 8 + (lane >> 3);
    xvoff[q] = (uint32_t)(min((int64_t)row, last_row) * p.ldc) + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
  }
  // packed operands: NF = 2 a whole group of 64 rows, NF = 1 half of one
  const int64_t col = n0 + wn * NF * 32;
  const int64_t g = min(col / 64, (int64_t)p.NG - 1);     // past the end: a copy, not stored
  const int f0 = (int)(col % 64) / 32;
  const uint8_t *wbase = p.wq + g * p.KS * 2048 + f0 * 1024 + lane * 16;
  const uint32_t *sbase = reinterpret_cast<const uint32_t *>(p.sc) + (g * p.KB * 2 + f0) * 64 + lane;

  acc_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = acc_t{};

  u4_t w[WS][NF];
  // Load q of a step's X.  Chunks past K in the last step hold the next row's bytes, or nothing:
  // an offset past the descriptor's range reads nothing and puts zeros into LDS.
  const int chunk0 = (lane & 7) ^ (lane >> 4), chunk1 = chunk0 ^ 4;   // this lane's source chunk, q even and odd
  auto load_x = [&](int step, int slot, int q) {
    const uint32_t soff = (uint32_t)min(step, steps - 1) * 128;
    const int limit = step >= steps - 1 && tail ? tail : 8;
    dma16(xr, ((q & 1) ? chunk1 : chunk0) < limit ? xvoff[q] : 0x7fffffffu, soff, smem + slot * SLOT + (wave * XQ + q) * 1024);
  };
  // operands of instruction s of a step into register set `set`
  auto load_w = [&](int step, int s, int set, int f) {
    const uint8_t *src = wbase + (int64_t)min(min(step, steps - 1) * SUB + s, p.KS - 1) * 2048;
    w[set][f] = *reinterpret_cast<const u4_t *>(src + f * 1024);
  };
  // this lane's chunks h, 2 + h, 4 + h, 6 + h of row r of operand 0 in a slot
  const int row0 = wm * MF * 32 + r;
  int xa[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) xa[c] = row0 * 128 + (((2 * c + h) ^ ((row0 >> 1) & 7)) << 4);
  constexpr int XR = FMT == MX_FP8 ? 2 : 1;       // 16-byte pieces of an X operand
  constexpr int SR = SUB / 2;                     // scale dwords of an operand and step
  struct Frag {            // one X operand: 32 rows, one instruction
    u4_t x[XR];
  };
  auto read_x = [&](Frag &o, int i, int s, const uint8_t *xs) {
#pragma unroll
    for (int c = 0; c < XR; ++c) o.x[c] = *reinterpret_cast<const u4_t *>(xs + xa[XR * s + c] + i * 4096);
  };
  // the scales of a step's blocks: byte 0 for instruction 0 (and 2), byte 2 for 1 (and 3)
  auto read_s = [&](uint32_t (&o)[SR], int i, const uint8_t *ss) {
    if constexpr (SR == 1) {
      o[0] = *reinterpret_cast<const uint32_t *>(ss + i * 512) >> (8 * h);
    } else {
      const u2_t v = *reinterpret_cast<const u2_t *>(ss + i * 512);
      o[0] = v[0] >> (8 * h);
      o[1] = v[1] >> (8 * h);
    }
  };
  // X scales of a step, from the panel's first
  auto scales_at = [&](int in_panel) {
    return sxl + (in_panel * SUB / 8 * BM + row0) * 16 + (in_panel * SUB % 8) * 2;
  };
  auto multiply = [&](auto nc, int i, const Frag &x, const uint32_t (&sx)[SR], const uint32_t (&sw)[NF]) {
    constexpr int n = decltype(nc)::value, s = n % SUB;   // instruction index within the loop body, the step
#pragma unroll
    for (int f = 0; f < NF; ++f)
      acc[i][f] = mx_mfma<FMT, n & 3, 2 * (s & 1)>(w[n % WS][f], x.x[0], x.x[XR - 1], acc[i][f], sw[f], sx[s / 2]);
  };

  // K in panels whose X scales fit LDS
  const int pieces = (p.K + kMxScaleRow - 1) / kMxScaleRow;   // 512-k chunks of X scales
  for (int c0 = 0; c0 < pieces; c0 += kPanel) {
    const int chunks = min(kPanel, pieces - c0);
    const int s0 = c0 * 8 / SUB, s1 = min(steps, s0 + chunks * 8 / SUB);   // steps of the panel
    uint32_t sw[NF], sw_next[NF];         // weight scales of this 256 k and the next
    auto load_sw = [&](int kb, int f) { sw_next[f] = sbase[(int64_t)min(kb, p.KB - 1) * 128 + f * 64]; };
#pragma unroll
    for (int f = 0; f < NF; ++f) load_sw(s0 * SUB / 4, f);
    lds_barrier();                        // the panel before has been read
    for (int q = wave; q < chunks * (BM / 64); q += WAVES) {
      const int c = q / (BM / 64), row = (q % (BM / 64)) * 64 + lane;
      dma16(sr, (uint32_t)(min((int64_t)row, last_row) * p.lds), (uint32_t)(c0 + c) * 16,
            sxl + (c * BM + (q % (BM / 64)) * 64) * 16);
    }
    pin();
#pragma unroll
    for (int d = 0; d < D; ++d) {
      pin();
#pragma unroll
      for (int q = 0; q < XQ; ++q) load_x(s0 + d, d, q);
      pin();
      if (!PRE && d) continue;
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f) load_w(s0 + d, s, (d * SUB + s) % WS, f);
    }
    pin();
    const int left = (blocks & 15);
    if (left && c0 + chunks == pieces) {    // scale bytes past K may hold anything, a NaN among it
      wait_vmcnt<0>();
      lds_barrier();
      for (int id = t; id < BM * 16; id += WAVES * 64)
        if ((id & 15) >= left) sxl[(chunks - 1) * BM * 16 + id] = 0;
      lds_barrier();
    }
    constexpr int AHEAD = 2;              // without PRE: operands read ahead
    Frag fr[PRE ? 2 * SUB : 1][PRE ? MF : AHEAD + 1];
    uint32_t sx[PRE ? 2 : 1][MF][SR];
    if constexpr (PRE) {
      wait_vmcnt<(D - 1) * (XQ + WQ)>();
      lds_barrier();
#pragma unroll
      for (int i = 0; i < MF; ++i) read_s(sx[0][i], i, scales_at(0));
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < MF; ++i) read_x(fr[s][i], i, s, smem);
    }
    for (int base = s0; base < s1; base += U) {
      unroll<0, U>([&](auto uc) {
        constexpr int u = decltype(uc)::value;
        const int step = base + u;
        if (step >= s1) return;
        constexpr bool next_chunk = u * SUB % 4 == 0;
        // PRE: the next step's X; else this step's X and first weights.  The count is of the
        // loads younger than the ones needed; more of them only wait longer.
        wait_vmcnt<YOUNGER>();
        lds_barrier();
        if constexpr (next_chunk) {
#pragma unroll
          for (int f = 0; f < NF; ++f) sw[f] = sw_next[f];
        }
        // the operands read during this step: the next step's, or AHEAD further on in this one
        const int rstep = PRE ? min(step + 1, s1 - 1) : step;   // (past the last: read, not used)
        constexpr int ru = PRE ? u + 1 : u;
        const uint8_t *xs = smem + ru % SLOTS * SLOT, *sp = scales_at(rstep - s0);
        if constexpr (!PRE) {
#pragma unroll
          for (int i = 0; i < MF; ++i) read_s(sx[0][i], i, sp);
#pragma unroll
          for (int j = 0; j < AHEAD; ++j) read_x(fr[0][j], j % MF, j / MF, xs);
        }
        unroll<0, GROUPS>([&](auto jc) {
          constexpr int j = decltype(jc)::value, s = j / MF, i = j % MF, n = j + AHEAD;
          pin();
          unroll<j * OPS / GROUPS, (j + 1) * OPS / GROUPS>([&](auto oc) {
            // PRE: X, weights, scales; else early weights, scales, X, late weights
            constexpr int o = decltype(oc)::value, early = PRE ? 0 : EARLY * NF;
            constexpr int sw0 = PRE ? XQ + WQ : early, x0 = PRE ? 0 : early + NF;
            if constexpr (o >= x0 && o < x0 + XQ) load_x(step + D, (u + D) % SLOTS, o - x0);
            else if constexpr (o >= sw0 && o < sw0 + NF) {
              if constexpr (next_chunk) load_sw(step * SUB / 4 + 1, o - sw0);
            } else {
              constexpr int m = PRE ? o - XQ : o < early ? o : o - NF - XQ, sm = m / NF, ahead = PRE ? D : 1;
              load_w(step + ahead, sm, ((u + ahead) * SUB + sm) % WS, m % NF);
            }
          });
          pin();
          if constexpr (PRE) {
            if constexpr (s == 0) read_s(sx[ru & 1][i], i, sp);
            read_x(fr[(ru & 1) * SUB + s][i], i, s, xs);
          } else if constexpr (n < GROUPS) {
            read_x(fr[0][n % (AHEAD + 1)], n % MF, n / MF, xs);
          }
          multiply(std::integral_constant<int, u * SUB + s>{}, i, fr[PRE ? (u & 1) * SUB + s : 0][PRE ? i : j % (AHEAD + 1)],
                   sx[PRE ? u & 1 : 0][i], sw);
          // the products stay between the reads around them (the compiler would sink them
          // past the step's end, holding every operand of the step in registers)
          if constexpr (!PRE) {
#pragma unroll
            for (int f = 0; f < NF; ++f) keep(acc[i][f]);
          }
        });
      });
    }
    wait_vmcnt<0>();   // loads past the last step land before their slots are reused
  }

  // A lane holds 16 consecutive columns of each operand.  Through LDS they become whole rows
  // of the tile, 16 bytes a thread: stores straight from the registers put 16-byte
  // pieces into 64 lines each and ran at 2.2 TB/s.  Chunks XOR-swizzled by the row.
  constexpr int CHUNKS = BN / 8;          // 16-byte chunks of an output row
  static_assert(BM * BN * 2 <= (int)sizeof(smem), "the output tile fits");
  if (p.N & 7) {                          // rows of other alignment
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        if (m0 + row0 + 32 * i < p.M) store_cols<DT>(p, m0 + row0 + 32 * i, col - 32 * f0 + 32 * h + 16 * (f0 + f), acc[i][f]);
    return;
  }
  lds_barrier();                          // every wave has read the last step
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int n = wn * NF * 32 - 32 * f0 + 32 * h + 16 * (f0 + f);   // within the tile
    float bias[16] = {};
    if (p.bias) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (n0 + n + 8 * e < p.N) load8<DT>(p.bias + n0 + n + 8 * e, bias + 8 * e);
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int row = row0 + 32 * i;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = acc[i][f][8 * e + k] + bias[8 * e + k];
        store8<DT>(reinterpret_cast<uint16_t *>(smem + row * (BN * 2) + (((n / 8 + e) ^ (row & (CHUNKS - 1))) << 4)), v);
      }
    }
  }
  lds_barrier();
#pragma unroll
  for (int j = 0; j < BM * CHUNKS / (WAVES * 64); ++j) {
    const int id = j * (WAVES * 64) + t, row = id / CHUNKS, c = id % CHUNKS;
    if (row > last_row || n0 + 8 * c >= p.N) continue;
    *reinterpret_cast<u4_t *>(p.y + (m0 + row) * p.N + n0 + 8 * c) =
        *reinterpret_cast<const u4_t *>(smem + row * (BN * 2) + ((c ^ (row & (CHUNKS - 1))) << 4));
  }
}

template <int DT, int FMT, int BM, int WM, int WN, int NF, int D, bool PRE>
hipError_t launch_tile(const MxMatmulParams &p, hipStream_t s) {
  const int64_t tiles = ((int64_t)p.M + BM - 1) / BM * (((int64_t)p.N + WN * NF * 32 - 1) / (WN * NF * 32));
  hipLaunchKernelGGL((gemm_kernel<DT, FMT, BM, WM, WN, NF, D, PRE>), dim3((uint32_t)((tiles + 7) / 8 * 8)), dim3(WM * WN * 64),
                     0, s, p);
  return hipGetLastError();
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  const int rows = mx_gemm_rows(p.M, p.N);
  if (rows == 256) return launch_tile<DT, FMT, 128, 1, 4, 2, 2, false>(p, s);
  if (rows == 128) return launch_tile<DT, FMT, 128, 1, 4, 1, 3, true>(p, s);
  return launch_tile<DT, FMT, 64, 1, 4, 1, 3, true>(p, s);
}

}  // namespace

int mx_gemm_rows(int M, int N) {
  const int64_t big = ((int64_t)M + 255) / 256 * (((int64_t)N + 255) / 256);
  if (big >= kCUs) return 256;
  const int64_t mid = ((int64_t)M + 127) / 128 * (((int64_t)N + 127) / 128);
  return mid >= kCUs / 2 ? 128 : 64;
}

int mx_gemm_splits(int M, int N, int K, int fmt) {
  (void)M; (void)N; (void)K; (void)fmt;
  return 1;
}

hipError_t launch_mx_gemm(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s) {
  if (dtype == DT_F16) return fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s) : launch<DT_F16, MX_FP8>(p, s);
  return fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s) : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
