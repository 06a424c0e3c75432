// decode.h -- layouts, launch parameters and device helpers shared by the kernels of
// include/mnb_decode.h (cache append and read, attention over the cache, sampling).
#pragma once

#include "ops.h"

namespace mnb {

// ---- the cache ------------------------------------------------------------------------------

// A page of one head, S tokens of D elements (layout in include/mnb_decode.h).  Keys lie in rows, so that a
// lane's load is a run of one token; values in units of 4 tokens x 8 elements, so that a lane's 16
// bytes hold the same elements of 4 tokens: the tokens are the matrix instruction's inner index.
constexpr int kv_head_bytes(int S, int D) { return S * (D + D / 16); }
constexpr int kv_value_codes(int S, int D) { return S * D / 2; }
constexpr int kv_key_scales(int S, int D) { return S * D; }
constexpr int kv_value_scales(int S, int D) { return S * D + S * D / 32; }

struct KvCache {
  uint8_t *data;
  int64_t page_stride;
  int pages, heads, D, shift;   // page_size = 1 << shift
};
struct KvRows {
  const int32_t *pages;
  int64_t ldp;
  const int32_t *lengths, *starts;
  int batch, width, rows;
};

// The rows of sequence b: first row, their number, and the position of the first (host sizes bound
// them all, whatever the device's numbers are).
struct KvSeq {
  int row0, n, len;
  __device__ __forceinline__ int first() const { return len - n; }   // position of the first row, may be negative
};
__device__ __forceinline__ KvSeq kv_seq(const KvRows &r, int b) {
  KvSeq s;
  s.len = max(0, r.lengths[b]);
  if (!r.starts) {
    s.row0 = b;
    s.n = 1;
  } else {
    s.row0 = min(max(0, r.starts[b]), r.rows);
    s.n = min(max(s.row0, r.starts[b + 1]), r.rows) - s.row0;
  }
  return s;
}

struct KvAppendParams {
  KvCache cache;
  KvRows rows;
  const uint16_t *q, *k, *v, *qw, *kw;
  uint16_t *out;
  const float *table;
  int64_t ldq, ldk, ldv, ldo;
  int q_heads, table_rows, rot, interleaved;
  float eps;
};
hipError_t launch_kv_append(int dtype, const KvAppendParams &p, hipStream_t s);

struct KvReadParams {
  KvCache cache;
  KvRows rows;
  void *k, *v;
  int64_t ldk, ldv;
};
hipError_t launch_kv_read(int dtype, const KvReadParams &p, hipStream_t s);

struct KvAttnParams {
  KvCache cache;
  KvRows rows;
  const uint16_t *q;
  uint16_t *y;
  int64_t ldq, ldy;
  int G;               // query heads of a key/value head
  int window;          // 0: none
  float scale;         // |scale| times log2(e); a negative one turns q's signs by
  uint32_t flip;       // these bits
  int whole;           // every item goes to one workgroup, whatever the lengths are
  int workgroups;      // of the first kernel
  int lone;            // the first of them, which take an item each (0: as the lengths say)
  int sharers;         // those behind, which share out the steps of items that are cut
  int least;           // an item of at most so many steps is not cut
  int tile_rows;       // 16 or 32
  int slot_rows;       // rows of a partial result
  float *part;         // what the second kernel is told of each sharer, then [sharers, 2, slot_rows, D + 4]
};
// The workgroups for these sizes, and whether items may be split over them.
struct KvPlan {
  int workgroups, lone, sharers, least, whole, tile_rows, slot_rows;
  int64_t items;       // at most
  size_t bytes;        // of the workspace
};
KvPlan kv_attn_plan(const KvCache &c, const KvRows &r, int G, int window);
hipError_t launch_kv_attn(int dtype, const KvAttnParams &p, hipStream_t s);

struct SampleParams {
  const void *x;
  int64_t ldl;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
  int64_t *tokens;
  int M, V;
};
hipError_t launch_sample(int dtype, const SampleParams &p, hipStream_t s);

// order-preserving bits of a number: larger number, larger integer; every NaN above +infinity, both zeros
// alike.  Nothing maps to 0.
constexpr uint32_t kOrderNan = 0xfffffffeu;
__device__ __forceinline__ uint32_t number_order(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);   // -0 becomes +0
  const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return f != f ? kOrderNan : u;
}

}  // namespace mnb
