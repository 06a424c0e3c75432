// api_ops.hip -- the exported calls of include/mnb_ops.h: argument validation, workspace
// sizes and kernel launches.
#include <stdio.h>

#include <climits>

#include "checks.h"
#include "mnb_ops.h"
#include "ops.h"

using namespace mnb;

namespace {

int check_mx(int fmt, int K, const void *codes, int64_t ldc, const void *scales, int64_t lds) {
  if (!codes || !scales) return MNB_ERR_INVALID_ARG;
  if (ldc < mx_row(fmt, K) || lds < scale_row(K)) return MNB_ERR_INVALID_ARG;
  if (off16(codes) || off16(scales) || off16(ldc) || off16(lds)) return MNB_ERR_MISALIGNED;
  return MNB_OK;
}

int check_matmul_sizes(int M, int N, int K, int fmt) {
  if (M < 0 || N < 0 || K < 0) return MNB_ERR_INVALID_ARG;
  if (fmt != MNB_MX_FP4 && fmt != MNB_MX_FP8) return MNB_ERR_INVALID_ARG;
  // 32-bit offsets from a tile's first row reach its 128 rows of X
  if (K % kBlock || K >= kMxMaxK) return MNB_ERR_UNSUPPORTED;
  // a launch has fewer than 2^32 threads: 256 per (row group, step) of the packer and at most
  // 512 per tile of 64 x 128 outputs of the product, whose count is rounded up to a multiple of 8
  if (cdiv(N, 64) * cdiv(K, kMxStep) >= 1 << 24) return MNB_ERR_UNSUPPORTED;
  if (cdiv(M, 64) * cdiv(N, 128) > (1 << 23) - 8) return MNB_ERR_UNSUPPORTED;
  return MNB_OK;
}

}  // namespace

extern "C" {

int mnb_ops_version(void) { return 100; }

int mnb_mx_quantize(const void *X, int dtype, int M, int K, int64_t ldx, int fmt, void *codes, int64_t ldc,
                    void *scales, int64_t lds, void *stream) {
  if (M < 0 || K < 0 || bad_dtype(dtype, true) || fmt < MNB_MX_FP4 || fmt > MNB_MX_FP8) return MNB_ERR_INVALID_ARG;
  if (K % kBlock) return MNB_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return MNB_OK;
  if (!X || bad_ld(ldx, K) || bad_ld(ldc, 0) || bad_ld(lds, 0)) return MNB_ERR_INVALID_ARG;
  const int st = check_mx(fmt, K, codes, ldc, scales, lds);
  if (st) return st;
  const int sz = elem_size(dtype);
  if (off16(X) || off16(ldx * sz)) return MNB_ERR_MISALIGNED;
  const Span x{X, M, ldx * sz, (int64_t)K * sz}, c{codes, M, ldc, mx_row(fmt, K)}, e{scales, M, lds, K / kBlock};
  if (overlap(x, c) || overlap(x, e) || overlap(c, e)) return MNB_ERR_ALIAS;
  return status(launch_mx_quantize(dtype, fmt, MxQuantParams{X, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales),
                                                             ldx, ldc, lds, M, K}, as_stream(stream)));
}

int mnb_mx_dequantize(const void *codes, int64_t ldc, const void *scales, int64_t lds, int fmt, int M, int K, void *Y,
                      int dtype, int64_t ldy, void *stream) {
  if (M < 0 || K < 0 || bad_dtype(dtype, true) || fmt < MNB_MX_FP4 || fmt > MNB_MX_FP8) return MNB_ERR_INVALID_ARG;
  if (K % kBlock) return MNB_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return MNB_OK;
  if (!Y || bad_ld(ldy, K) || bad_ld(ldc, 0) || bad_ld(lds, 0)) return MNB_ERR_INVALID_ARG;
  const int st = check_mx(fmt, K, codes, ldc, scales, lds);
  if (st) return st;
  const int sz = elem_size(dtype);
  if (off16(Y) || off16(ldy * sz)) return MNB_ERR_MISALIGNED;
  const Span y{Y, M, ldy * sz, (int64_t)K * sz}, c{codes, M, ldc, mx_row(fmt, K)}, e{scales, M, lds, K / kBlock};
  if (overlap(y, c) || overlap(y, e)) return MNB_ERR_ALIAS;
  return status(launch_mx_dequantize(dtype, fmt, MxDequantParams{static_cast<const uint8_t *>(codes),
                                                                 static_cast<const uint8_t *>(scales), Y, ldc, lds, ldy, M, K},
                                     as_stream(stream)));
}

int mnb_mx_packed_sizes(int N, int K, size_t *wq_bytes, size_t *sc_bytes) {
  const int st = check_matmul_sizes(0, N, K, MNB_MX_FP4);
  if (st) return st;
  const size_t ng = (size_t)cdiv(N, 64);
  if (wq_bytes) *wq_bytes = ng * cdiv(K, kMxStep) * 4096;
  if (sc_bytes) *sc_bytes = ng * cdiv(K, kMxScaleK) * 1024;
  return MNB_OK;
}

int mnb_mx_pack(const void *codes, int64_t ldc, const void *scales, int64_t lds, int N, int K, void *wq, void *sc,
                void *stream) {
  int st = check_matmul_sizes(0, N, K, MNB_MX_FP4);
  if (st) return st;
  if (N == 0 || K == 0) return MNB_OK;
  if (!codes || !scales || !wq || !sc || bad_ld(ldc, K / 2) || bad_ld(lds, K / kBlock)) return MNB_ERR_INVALID_ARG;
  if (off16(codes) || off16(ldc) || off16(wq) || off16(sc)) return MNB_ERR_MISALIGNED;
  size_t wqb = 0, scb = 0;
  mnb_mx_packed_sizes(N, K, &wqb, &scb);
  const Span c{codes, N, ldc, K / 2}, e{scales, N, lds, K / kBlock}, w{wq, 1, 0, (int64_t)wqb}, d{sc, 1, 0, (int64_t)scb};
  if (overlap(c, w) || overlap(c, d) || overlap(e, w) || overlap(e, d) || overlap(w, d)) return MNB_ERR_ALIAS;
  return status(launch_mx_pack(MxPackParams{static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales),
                                            static_cast<uint8_t *>(wq), static_cast<uint8_t *>(sc), ldc, lds, N, K,
                                            (int)cdiv(N, 64), (int)cdiv(K, kMxStep), (int)cdiv(K, kMxScaleK)},
                               as_stream(stream)));
}

int mnb_mx_describe_route(int M, int N, int K, int fmt, char *buf, size_t buf_len) {
  const int st = check_matmul_sizes(M, N, K, fmt);
  if (st) return st;
  if (!buf || buf_len == 0) return MNB_ERR_INVALID_ARG;
  const char *name = fmt == MNB_MX_FP4 ? "fp4" : "fp8";
  if (M == 0 || N == 0) snprintf(buf, buf_len, "noop");
  else if (K == 0) snprintf(buf, buf_len, "fill");
  else if (M <= kMxGemvMaxM) snprintf(buf, buf_len, "mx_gemv_%s operands=%d ksplit=%d", name,
                                        mx_gemv_operands(fmt, M, N, K), mx_gemv_ksplit(fmt, M, N, K));
  else {
    const int rows = mx_gemm_rows(fmt, M, N, K);
    snprintf(buf, buf_len, "mx_gemm_%s tile=%dx%d%s", name, rows == 64 ? 64 : 128, rows == 256 ? 256 : 128,
             mx_gemm_groups(fmt, M, N, K) == 2 ? " groups=2" : "");
  }
  return MNB_OK;
}

int mnb_mx_matmul(const void *codes, int64_t ldc, const void *scales, int64_t lds, int fmt, const void *wq, const void *sc,
                  const void *bias, void *Y, int dtype, int M, int N, int K, void *stream) {
  int st = check_matmul_sizes(M, N, K, fmt);
  if (st) return st;
  if (bad_dtype(dtype, false)) return MNB_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MNB_OK;
  if (!Y) return MNB_ERR_INVALID_ARG;
  if (off16(Y) || off16(bias)) return MNB_ERR_MISALIGNED;
  const Span y{Y, 1, 0, (int64_t)M * N * 2}, bi{bias, 1, 0, (int64_t)N * 2};
  if (overlap(y, bi)) return MNB_ERR_ALIAS;
  if (K == 0)
    return status(launch_fill(static_cast<uint16_t *>(Y), static_cast<const uint16_t *>(bias), M, N, as_stream(stream)));
  if (!wq || !sc || bad_ld(ldc, 0) || bad_ld(lds, 0)) return MNB_ERR_INVALID_ARG;
  st = check_mx(fmt, K, codes, ldc, scales, lds);
  if (st) return st;
  if (ldc > 2 * kMxMaxK || lds > 2 * kMxMaxK) return MNB_ERR_UNSUPPORTED;
  if (off16(wq) || off16(sc)) return MNB_ERR_MISALIGNED;
  size_t wqb = 0, scb = 0;
  mnb_mx_packed_sizes(N, K, &wqb, &scb);
  const Span x{codes, M, ldc, mx_row(fmt, K)}, e{scales, M, lds, scale_row(K)}, w{wq, 1, 0, (int64_t)wqb},
      s{sc, 1, 0, (int64_t)scb};
  if (overlap(y, x) || overlap(y, e) || overlap(y, w) || overlap(y, s)) return MNB_ERR_ALIAS;
  MxMatmulParams p{};
  p.codes = static_cast<const uint8_t *>(codes);
  p.scales = static_cast<const uint8_t *>(scales);
  p.wq = static_cast<const uint8_t *>(wq);
  p.sc = static_cast<const uint8_t *>(sc);
  p.bias = static_cast<const uint16_t *>(bias);
  p.y = static_cast<uint16_t *>(Y);
  p.ldc = ldc;
  p.lds = lds;
  p.M = M;
  p.N = N;
  p.K = K;
  p.NG = (int)cdiv(N, 64);
  p.KS = (int)cdiv(K, kMxStep);
  p.KB = (int)cdiv(K, kMxScaleK);
  if (M <= kMxGemvMaxM) return status(launch_mx_gemv(dtype, fmt, p, as_stream(stream)));
  return status(launch_mx_gemm(dtype, fmt, p, as_stream(stream)));
}

int mnb_rmsnorm(const void *X, int64_t ldx, const void *residual, int64_t ldr, const void *weight, float eps, int dtype,
                int M, int K, void *hidden, int64_t ldh, void *Y, int64_t ldy, int fmt, void *codes, int64_t ldc,
                void *scales, int64_t lds, void *stream) {
  if (M < 0 || K < 0 || bad_dtype(dtype, false) || !(eps >= 0.f)) return MNB_ERR_INVALID_ARG;
  const bool mx = codes != nullptr || scales != nullptr;
  if (mx && (fmt < MNB_MX_FP4 || fmt > MNB_MX_FP8)) return MNB_ERR_INVALID_ARG;
  if (mx && K % kBlock) return MNB_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return MNB_OK;
  if (!X || !weight || (!Y && !mx)) return MNB_ERR_INVALID_ARG;
  if (bad_ld(ldx, K) || (residual && bad_ld(ldr, K)) || (hidden && bad_ld(ldh, K)) || (Y && bad_ld(ldy, K)))
    return MNB_ERR_INVALID_ARG;
  if (((uintptr_t)X | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)hidden | (uintptr_t)Y) & 1) return MNB_ERR_MISALIGNED;
  if (mx) {
    if (bad_ld(ldc, 0) || bad_ld(lds, 0)) return MNB_ERR_INVALID_ARG;
    const int st = check_mx(fmt, K, codes, ldc, scales, lds);
    if (st) return st;
    if (off16(X) || off16(residual) || off16(weight) || off16(hidden) || off16(Y) || off16(2 * ldx) ||
        (residual && off16(2 * ldr)) || (hidden && off16(2 * ldh)) || (Y && off16(2 * ldy)))
      return MNB_ERR_MISALIGNED;
  }
  const int64_t row = (int64_t)K * 2;
  const Span x{X, M, 2 * ldx, row}, r{residual, M, 2 * ldr, row}, w{weight, 1, 0, row}, h{hidden, M, 2 * ldh, row},
      y{Y, M, 2 * ldy, row}, c{mx ? codes : nullptr, M, ldc, mx_row(fmt, K)}, e{mx ? scales : nullptr, M, lds, K / kBlock};
  if (overlap(h, w) || overlap(y, w) || overlap(c, w) || overlap(e, w)) return MNB_ERR_ALIAS;
  if ((overlap(h, x) && !same(h, x)) || (overlap(h, r) && !same(h, r)) || (overlap(y, x) && !same(y, x))) return MNB_ERR_ALIAS;
  if (overlap(y, r) || overlap(y, h) || overlap(c, x) || overlap(c, r) || overlap(c, h) || overlap(c, y)) return MNB_ERR_ALIAS;
  if (overlap(e, x) || overlap(e, r) || overlap(e, h) || overlap(e, y) || overlap(e, c)) return MNB_ERR_ALIAS;
  NormParams p{};
  p.x = static_cast<const uint16_t *>(X);
  p.res = static_cast<const uint16_t *>(residual);
  p.w = static_cast<const uint16_t *>(weight);
  p.hidden = static_cast<uint16_t *>(hidden);
  p.y = static_cast<uint16_t *>(Y);
  p.codes = static_cast<uint8_t *>(codes);
  p.scales = static_cast<uint8_t *>(scales);
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldh = ldh;
  p.ldy = ldy;
  p.ldc = ldc;
  p.lds = lds;
  p.M = M;
  p.K = K;
  p.eps = eps;
  // a launch has fewer than 2^32 threads, up to 1024 per row
  for (int m0 = 0; m0 < M; m0 += 1 << 20) {
    NormParams q = p;
    q.M = M - m0 < 1 << 20 ? M - m0 : 1 << 20;
    q.x += (int64_t)m0 * ldx;
    if (residual) q.res += (int64_t)m0 * ldr;
    if (hidden) q.hidden += (int64_t)m0 * ldh;
    if (Y) q.y += (int64_t)m0 * ldy;
    if (mx) {
      q.codes += (int64_t)m0 * ldc;
      q.scales += (int64_t)m0 * lds;
    }
    const hipError_t err = launch_rmsnorm(dtype, mx ? fmt : -1, q, as_stream(stream));
    if (err != hipSuccess) return MNB_ERR_HIP;
    if (M - m0 <= 1 << 20) break;
  }
  return MNB_OK;
}

static int check_logprobs(int M, int V, int dtype, int top) {
  if (M < 0 || V < 0 || bad_dtype(dtype, true) || top < 0) return MNB_ERR_INVALID_ARG;
  if (top > MNB_LOGPROBS_MAX_TOP || V > (1 << 22)) return MNB_ERR_UNSUPPORTED;
  if (M > 0 && V > 0 && top > V) return MNB_ERR_INVALID_ARG;
  return MNB_OK;
}

size_t mnb_logprobs_workspace_bytes(int M, int V, int dtype, int top) {
  if (check_logprobs(M, V, dtype, top) || M == 0 || V == 0) return 0;
  int chunk = 0;
  const int chunks = logprobs_chunks(M, V, dtype, &chunk);
  return chunks > 1 ? (size_t)M * chunks * (16 + (size_t)top * 8) : 0;
}

int mnb_logprobs(const void *logits, int dtype, int M, int V, int64_t ldl, const int64_t *tokens, int top, float *logprob,
                 float *entropy, float *top_logprobs, int64_t *top_tokens, void *workspace, size_t ws_bytes, void *stream) {
  const int st = check_logprobs(M, V, dtype, top);
  if (st) return st;
  if (M == 0 || V == 0) return MNB_OK;
  if (!logits || bad_ld(ldl, V) || (tokens && !logprob) || (top && (!top_logprobs || !top_tokens))) return MNB_ERR_INVALID_ARG;
  if (!tokens && !entropy && !top) return MNB_ERR_INVALID_ARG;
  const int sz = elem_size(dtype);
  if (((uintptr_t)logits & (sz - 1)) || (((uintptr_t)tokens | (uintptr_t)top_tokens) & 7) ||
      (((uintptr_t)logprob | (uintptr_t)entropy | (uintptr_t)top_logprobs) & 3) || off16(workspace))
    return MNB_ERR_MISALIGNED;
  const size_t need = mnb_logprobs_workspace_bytes(M, V, dtype, top);
  if (need && (!workspace || ws_bytes < need)) return MNB_ERR_WORKSPACE;
  const Span in[] = {{logits, M, ldl * sz, (int64_t)V * sz}, {tokens, 1, 0, (int64_t)M * 8}};
  const Span out[] = {{tokens ? logprob : nullptr, 1, 0, (int64_t)M * 4}, {entropy, 1, 0, (int64_t)M * 4},
                      {top ? top_logprobs : nullptr, 1, 0, (int64_t)M * top * 4},
                      {top ? top_tokens : nullptr, 1, 0, (int64_t)M * top * 8},
                      {need ? workspace : nullptr, 1, 0, (int64_t)need}};
  for (int i = 0; i < 5; ++i) {
    for (const Span &s : in)
      if (overlap(out[i], s)) return MNB_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MNB_ERR_ALIAS;
  }
  LogprobsParams p{};
  p.x = logits;
  p.ldl = ldl;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_logprobs = top_logprobs;
  p.top_tokens = top_tokens;
  p.M = M;
  p.V = V;
  p.top = top;
  p.chunks = logprobs_chunks(M, V, dtype, &p.chunk);
  p.part = static_cast<float *>(workspace);
  p.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + (need ? (size_t)M * p.chunks * 16 : 0));
  // a launch has fewer than 2^32 threads, up to 1024 per part of a row
  const int rows = ((1 << 22) - 1) / p.chunks;
  for (int64_t m0 = 0; m0 < M; m0 += rows) {
    LogprobsParams q = p;
    q.M = (int)(M - m0 < rows ? M - m0 : rows);
    q.x = static_cast<const char *>(logits) + m0 * ldl * sz;
    if (tokens) {
      q.tokens += m0;
      q.logprob += m0;
    }
    if (entropy) q.entropy += m0;
    if (top) {
      q.top_logprobs += m0 * top;
      q.top_tokens += m0 * top;
    }
    if (need) {
      q.part += m0 * p.chunks * 4;
      q.keys += m0 * p.chunks * top;
    }
    const hipError_t err = launch_logprobs(dtype, q, as_stream(stream));
    if (err != hipSuccess) return MNB_ERR_HIP;
  }
  return MNB_OK;
}

}  // extern "C"
