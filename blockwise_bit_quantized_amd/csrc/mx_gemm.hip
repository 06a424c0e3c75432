// mx_gemm.hip -- MX product for more rows than the weight-streaming kernel takes.
//
// Bound by the matrix cores where there is enough work: an instruction of 16 x 16 outputs and
// 128 k takes 16 cycles (FP4 X) or 32 (FP8 X).  A workgroup owns BM x BN outputs, a wave
// MF x NF operands of 16 rows and 16 columns.
//
// X goes through LDS in steps of 128 bytes a row (128 k of FP8, 256 of FP4), a ring of
// D + 1 slots filled by direct-to-LDS loads D steps ahead; a row's eight 16-byte chunks are
// XOR-swizzled by the row through the source address (the loads write lanes
// consecutively), so that the 16 rows of an operand read fall on distinct banks.  Weights are
// packed in operand order and load straight into registers, D steps ahead as well: a wave's
// loads complete in order, so neither may run further ahead than the other.  The X scales of
// up to 8192 k are staged in LDS before the steps ([chunk of 512 k][row][16 bytes], where
// the 16 rows of an operand are 256 consecutive bytes) and read one byte per lane, the byte
// the instruction wants; weight scales are one dword per operand and 512 k.
//
// With PRE the X operands of the next step are read into a second register set before the
// current step's instructions are issued, so a single wave per SIMD does not wait for LDS.
// With KG = 2 two groups of waves work on halves of K, each with its own ring and panel; the
// second group's sums join the first's in LDS.
//
// Reached: 8192x9728x2560 150 us with FP8 X (2.7 PFLOP/s), 107 with FP4 (3.8); 4096^3 49 us
// (2.8) and 36 (3.8).  The bare instructions on random data run at 4.25 and 4.5 PFLOP/s: the
// clock falls to 1.5 - 1.9 GHz under them.  A 128 x 256 step of FP8 takes 2134 cycles for
// 2048 of its instructions.
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
__device__ __forceinline__ void keep(f4_t &v) { asm volatile("" : "+v"(v)); }

constexpr int kPanel = 16;   // 512-k chunks of X scales in LDS at a time

template <int I, int N, typename F>
__device__ __forceinline__ void unroll(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<I + 1, N>(f);
  }
}

template <int DT, int FMT, int BM, int WM, int WN, int NF, int D, bool PRE, int KG>
__global__ __launch_bounds__(KG * WM * WN * 64, KG * (PRE ? 1 : 2)) void gemm_kernel(MxMatmulParams p) {
  constexpr int WAVES = WM * WN, BN = WN * NF * 16, MF = BM / WM / 16;
  constexpr int SUB = FMT == MX_FP4 ? 2 : 1;      // instructions per step, operand pair
  constexpr int SLOTS = D + 1, SLOT = BM * 128;
  constexpr int XQ = BM / 8 / WAVES;              // X loads per wave and step (8 rows each)
  constexpr int WQ = SUB * NF;                    // weight loads per wave and step
  constexpr int WS = PRE ? SLOTS * SUB : SUB + 1; // weight register sets, one instruction's each
  constexpr int GROUPS = SUB * MF, OPS = XQ + WQ + NF;   // X operands and loads of a step
  constexpr int U = !PRE && SUB == 2 ? 6 : 4;     // steps per unrolled loop body
  static_assert(U % SLOTS == 0 && U * SUB % WS == 0 && U * SUB % 4 == 0, "slots, sets and scale bytes are compile-time");
  static_assert(PRE || D == 1, "without PRE the weights run one step ahead");
  // FP4 without PRE: the second instruction's weights go into the first one's set, so they are
  // loaded in the second half of the step
  static_assert(PRE || SUB == 1 || (XQ + NF) * GROUPS / OPS >= MF, "second-half weight loads");
  static_assert(XQ >= 1 && 8 * XQ * WAVES == BM, "X rows per wave");
  constexpr int LDS = SLOTS * SLOT + kPanel * BM * 16;   // of one group of waves
  __shared__ __attribute__((aligned(1024))) uint8_t smem_all[KG * LDS];

  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // uniform: addresses stay scalar
  const int wave = wave_all % WAVES, kg = wave_all / WAVES, t = wave * 64 + lane;
  uint8_t *smem = smem_all + kg * LDS, *sxl = smem + SLOTS * SLOT;
  const int r = lane & 15, b = lane >> 4;
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
  // packed operands: NF = 4 a whole group of 64 rows, NF = 2 half of one
  const int64_t col = n0 + wn * NF * 16;
  const int64_t g = min(col / 64, (int64_t)p.NG - 1);     // past the end: a copy, not stored
  const int f0 = (int)(col % 64) / 16;
  const uint8_t *wbase = p.wq + g * p.KS * 4096 + f0 * 1024 + lane * 16;
  const uint32_t *sbase = reinterpret_cast<const uint32_t *>(p.sc) + (g * p.KB * 4 + f0) * 64 + lane;

  f4_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = f4_t{0.f, 0.f, 0.f, 0.f};

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
    const uint8_t *src = wbase + (int64_t)min(min(step, steps - 1) * SUB + s, p.KS - 1) * 4096;
    w[set][f] = *reinterpret_cast<const u4_t *>(src + f * 1024);
  };
  // this lane's chunk addresses in a slot: chunk b and chunk b + 4 of row r of operand 0
  const int row0 = wm * MF * 16 + r;
  const int xa = row0 * 128 + ((b ^ ((row0 >> 1) & 7)) << 4), xb = xa ^ 64;
  constexpr int XR = FMT == MX_FP8 ? 2 : 1;       // 16-byte pieces of an X operand
  struct Frag {            // one X operand: 16 rows, one instruction
    u4_t x[XR];
    uint32_t s;
  };
  // operand i of the instruction whose index mod 4 is `byte`; sub: which of the step's
  auto read_x = [&](Frag &o, int i, int sub, const uint8_t *xs, const uint8_t *ss, int byte) {
    o.x[0] = *reinterpret_cast<const u4_t *>(xs + (sub ? xb : xa) + i * 2048);
    if constexpr (XR == 2) o.x[1] = *reinterpret_cast<const u4_t *>(xs + xb + i * 2048);
    o.s = ss[i * 256 + (byte & 3) * 4];
  };
  auto multiply = [&](auto hc, int i, const Frag &x, const uint32_t (&sw)[NF]) {
    constexpr int h = decltype(hc)::value;        // instruction index within the loop body
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = mx_mfma<FMT, h & 3>(w[h % WS][f], x.x[0], x.x[XR - 1], acc[i][f], sw[f], x.s);
  };

  // K in panels whose X scales fit LDS
  const int share = (p.KB + KG - 1) / KG;   // 512-k chunks of a group; the last group may have fewer, or none
  for (int panel = 0; panel < share; panel += kPanel) {
    const int c0 = kg * share + panel, chunks = max(0, min(min(kPanel, share - panel), p.KB - c0));
    const int s0 = c0 * (4 / SUB), s1 = max(s0, min(steps, s0 + chunks * (4 / SUB)));   // steps of the panel
    // the groups meet at the same barriers: one with fewer steps only waits through the others'
    const int s_end = KG == 1 ? s1 : s0 + min(kPanel, share - panel) * (4 / SUB);
    uint32_t sw[NF], sw_next[NF];         // weight scales of this 512-k chunk and the next
    auto load_sw = [&](int kb, int f) { sw_next[f] = sbase[(int64_t)min(kb, p.KB - 1) * 256 + f * 64]; };
#pragma unroll
    for (int f = 0; f < NF; ++f) load_sw(c0, f);
    lds_barrier();                        // the panel before has been read
    for (int q = wave; q < chunks * (BM / 64); q += WAVES) {
      const int c = q / (BM / 64), row = (q % (BM / 64)) * 64 + lane;
      dma16(sr, (uint32_t)(min((int64_t)row, last_row) * p.lds), (uint32_t)(c0 + c) * 16,
            sxl + (c * BM + (q % (BM / 64)) * 64) * 16);
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      pin();
#pragma unroll
      for (int q = 0; q < XQ; ++q) load_x(s0 + d, d, q);
      pin();
#pragma unroll
      for (int h = 0; h < SUB; ++h)
#pragma unroll
        for (int f = 0; f < NF; ++f) load_w(s0 + d, h, (d * SUB + h) % WS, f);
    }
    pin();
    const int left = (blocks & 15);
    // does the last group end in this panel?  (the same answer in every group: there are barriers inside)
    const int cl = (KG - 1) * share + panel;
    const bool ends = cl < p.KB && min(min(kPanel, share - panel), p.KB - cl) == p.KB - cl;
    if (left && ends) {   // scale bytes past K may hold anything, a NaN among it
      wait_vmcnt<0>();
      lds_barrier();
      if (kg == KG - 1) for (int id = t; id < BM * 16; id += WAVES * 64)
        if ((id & 15) >= left) sxl[(chunks - 1) * BM * 16 + id] = 0;
      lds_barrier();
    }
    const uint8_t *ss = sxl + row0 * 16 + b;
    constexpr int AHEAD = FMT == MX_FP8 ? 2 : 3;  // without PRE: operands read ahead
    Frag fr[PRE ? 2 * SUB : 1][PRE ? MF : AHEAD + 1];
    if constexpr (PRE) {
      wait_vmcnt<(D - 1) * (XQ + WQ)>();
      lds_barrier();
#pragma unroll
      for (int h = 0; h < SUB; ++h)
#pragma unroll
        for (int i = 0; i < MF; ++i) read_x(fr[h][i], i, h, smem, ss, h);
    }
    for (int base = s0; base < s_end; base += U) {
      unroll<0, U>([&](auto uc) {
        constexpr int u = decltype(uc)::value;
        const int step = base + u;
        if (step >= s_end) return;
        constexpr bool next_chunk = u * SUB % 4 == 0;
        // PRE: the next step's X; else this step's.  The count is of the loads younger than the
        // ones needed; more of them only wait longer.
        if constexpr (PRE) wait_vmcnt<(D - 2) * (XQ + WQ) + WQ>();
        else wait_vmcnt<0>();
        lds_barrier();
        if (KG > 1 && step >= s1) return;
        if constexpr (next_chunk) {
#pragma unroll
          for (int f = 0; f < NF; ++f) sw[f] = sw_next[f];
        }
        // the operands read during this step: the next step's, or AHEAD further on in this one
        const int rstep = PRE ? max(s0, min(step + 1, s1 - 1)) : step;   // (past the last: read, not used)
        constexpr int ru = PRE ? u + 1 : u;
        const uint8_t *xs = smem + ru % SLOTS * SLOT, *sp = ss + (rstep - s0) * SUB / 4 * BM * 16;
        if constexpr (!PRE) {
#pragma unroll
          for (int j = 0; j < AHEAD; ++j) read_x(fr[0][j], j % MF, j / MF, xs, sp, u * SUB + j / MF);
        }
        // Loads, operand reads and products interleaved: a wave whose loads wait to be accepted
        // issues nothing, so they go one at a time between the products.
        unroll<0, GROUPS>([&](auto jc) {
          constexpr int j = decltype(jc)::value, h = j / MF, i = j % MF, n = j + AHEAD;
          pin();
          unroll<j * OPS / GROUPS, (j + 1) * OPS / GROUPS>([&](auto oc) {
            constexpr int o = decltype(oc)::value;
            if constexpr (o < XQ) load_x(step + D, (u + D) % SLOTS, o);
            else if constexpr (o < XQ + WQ) load_w(step + D, (o - XQ) / NF, ((u + D) * SUB + (o - XQ) / NF) % WS, (o - XQ) % NF);
            else if constexpr (next_chunk) load_sw(c0 + (step - s0) * SUB / 4 + 1, o - XQ - WQ);
          });
          pin();
          if constexpr (PRE) read_x(fr[(ru & 1) * SUB + h][i], i, h, xs, sp, ru * SUB + h);
          else if constexpr (n < GROUPS) read_x(fr[0][n % (AHEAD + 1)], n % MF, n / MF, xs, sp, u * SUB + n / MF);
          multiply(std::integral_constant<int, u * SUB + h>{}, i, fr[PRE ? (u & 1) * SUB + h : 0][PRE ? i : j % (AHEAD + 1)], sw);
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

  if constexpr (KG == 2) {   // the second group's sums go through LDS to the first, which stores
    static_assert(MF * NF * WAVES * 1024 <= LDS, "the sums fit");
    lds_barrier();           // every wave has read the last step
    f4_t *sums = reinterpret_cast<f4_t *>(smem_all + LDS) + wave * (MF * NF * 64) + lane;
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        if (kg) sums[(i * NF + f) * 64] = acc[i][f];
    lds_barrier();
    if (!kg) {
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[i][f] += sums[(i * NF + f) * 64];
    }
  }

  // A lane holds NF * 4 consecutive columns of each of its rows.  Through LDS they become whole
  // rows of the tile, 16 bytes a thread: stores straight from the registers put their pieces into
  // 16 lines each and ran at 3.9 TB/s, these at 6.3.  Chunks XOR-swizzled by the row.
  constexpr int CHUNKS = BN / 8;          // 16-byte chunks of an output row
  static_assert(BM * BN * 2 <= LDS, "the output tile fits");
  const int nt = wn * NF * 16 - 16 * f0 + 16 * b + 4 * f0;   // this lane's first column within the tile
  if (p.N & 7) {                          // rows of other alignment
    if (kg) return;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int64_t m = m0 + row0 + 16 * i;
      if (m >= p.M) continue;
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + nt + 4 * f + e < p.N) store_cols<DT>(p, m, n0 + nt + 4 * f + e, acc[i][f][e]);
    }
    return;
  }
  lds_barrier();                          // every wave has read the last step
  if (!kg) {
#pragma unroll
  for (int e = 0; e < NF / 2; ++e) {      // two operands: 8 columns
    float bias[8] = {};
    if (p.bias && n0 + nt + 8 * e < p.N) load8<DT>(p.bias + n0 + nt + 8 * e, bias);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int row = row0 + 16 * i;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = acc[i][2 * e + k / 4][k % 4] + bias[k];
      store8<DT>(reinterpret_cast<uint16_t *>(smem + row * (BN * 2) + (((nt / 8 + e) ^ (row & (CHUNKS - 1))) << 4)), v);
    }
  }
  }
  lds_barrier();
  // Stores past the caches leave X and the weights in L2 for the tiles after (8192x9728x2560 FP8
  // 148 us, not 170, FP4 107, not 130; 4096^3 FP4 35.5, not 36.8).  Rows that end inside a line of
  // 128 bytes are slower so (2100x9000x1120 FP4 27.4, not 25.2), and where K is short the stores
  // themselves are the bound and go faster to the last-level cache (4096x8192x512 FP4 24.5, not 22.7).
  const bool past_caches = BM == 128 && (p.N & 63) == 0 && p.K >= 1024;
#pragma unroll
  for (int j = 0; j < BM * CHUNKS / (KG * WAVES * 64); ++j) {
    const int id = (j * KG + kg) * (WAVES * 64) + t, row = id / CHUNKS, c = id % CHUNKS;
    if (row > last_row || n0 + 8 * c >= p.N) continue;
    const u4_t v = *reinterpret_cast<const u4_t *>(smem_all + row * (BN * 2) + ((c ^ (row & (CHUNKS - 1))) << 4));
    u4_t *dst = reinterpret_cast<u4_t *>(p.y + (m0 + row) * p.N + n0 + 8 * c);
    if (past_caches) {
      asm volatile("; past the caches");   // (else the compiler joins the two stores, to a plain one)
      __builtin_nontemporal_store(v, dst);
      asm volatile("");
    } else {
      *dst = v;
    }
  }
}

template <int DT, int FMT, int BM, int WM, int WN, int NF, int D, bool PRE, int KG>
hipError_t launch_tile(const MxMatmulParams &p, hipStream_t s) {
  const int64_t tiles = ((int64_t)p.M + BM - 1) / BM * (((int64_t)p.N + WN * NF * 16 - 1) / (WN * NF * 16));
  hipLaunchKernelGGL((gemm_kernel<DT, FMT, BM, WM, WN, NF, D, PRE, KG>), dim3((uint32_t)((tiles + 7) / 8 * 8)), dim3(KG * WM * WN * 64),
                     0, s, p);
  return hipGetLastError();
}

template <int DT, int FMT>
hipError_t launch(const MxMatmulParams &p, hipStream_t s) {
  const int rows = mx_gemm_rows(FMT, p.M, p.N, p.K);
  if (rows == 256) return launch_tile<DT, FMT, 128, 1, 4, 4, 1, false, 1>(p, s);
  if (rows == 128) return launch_tile<DT, FMT, 128, 1, 4, 2, 3, true, 1>(p, s);
  if (mx_gemm_groups(FMT, p.M, p.N, p.K) == 2) return launch_tile<DT, FMT, 64, 1, 4, 2, 3, true, 2>(p, s);
  return launch_tile<DT, FMT, 64, 1, 4, 2, 3, true, 1>(p, s);
}

bool long_k(int fmt, int K) { return (fmt == MX_FP4 ? K / 2 : K) >= 16 * 128; }   // 16 steps or more

}  // namespace

// The tile with the least time for a whole grid: the rounds that 256 CUs need, times a tile's
// time per step (FP8, 4096 k: 64 x 128 0.34 us alone on a CU, 128 x 128 0.56, 128 x 256 0.93,
// two of them together 1.55; 64 x 128 without the second group of waves shares a CU and takes
// less).  Measured with 64 x 128 / 128 x 128 / 128 x 256, us: 512x4096x4096 FP8 13.7 / 19.2 /
// 28.2, 1024x4096x4096 23.7 / 20.2 / 28.8 and FP4 20.4 / 16.0 / 20.4, 2048x4096x4096 43 / 37 /
// 31, 4096^3 83 / 71 / 49, 1500x2560x2560 18.5 / 14.5 / 20.3, 300x16384x1024 11.1 / 15.4 / 12.2.
// FP4 goes by the same weights, though its times stand to each other differently: 600x9728x2560 takes
// 17.6 with the tile chosen and 16.0 with the next.
int mx_gemm_rows(int fmt, int M, int N, int K) {
  const auto rounds = [&](int bm, int bn) { return (((int64_t)M + bm - 1) / bm * (((int64_t)N + bn - 1) / bn) + kCUs - 1) / kCUs; };
  const int64_t r64 = rounds(64, 128), r128 = rounds(128, 128), r256 = rounds(128, 256);
  const int64_t c64 = r64 * (long_k(fmt, K) ? 5 : 4), c128 = r128 * 9, c256 = r256 * (r256 > 1 ? 12 : 14);
  return c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
}

// A CU draws about 60 GB/s however far ahead its loads run (7 steps ahead instead of 3: no
// change), so a grid of few tiles is bound by its number of CUs.  A second group of waves with
// the other half of K keeps more of them in flight: 64x2560x9728 FP8 28.5 -> 22.3 us,
// 200x2560x4096 FP8 14.3 -> 12.2, FP4 9.9 -> 9.6; under 16 steps the join costs more than it
// gives (64x8192x2048 FP4 6.1 -> 7.0).
int mx_gemm_groups(int fmt, int M, int N, int K) {
  return mx_gemm_rows(fmt, M, N, K) == 64 && long_k(fmt, K) ? 2 : 1;
}

hipError_t launch_mx_gemm(int dtype, int fmt, const MxMatmulParams &p, hipStream_t s) {
  if (dtype == DT_F16) return fmt == MX_FP4 ? launch<DT_F16, MX_FP4>(p, s) : launch<DT_F16, MX_FP8>(p, s);
  return fmt == MX_FP4 ? launch<DT_BF16, MX_FP4>(p, s) : launch<DT_BF16, MX_FP8>(p, s);
}

}  // namespace mnb
