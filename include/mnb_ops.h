/*
 * mnb_ops.h -- the operators beside MatMulNBits that libmnb also exports: microscaled (MX)
 * quantisation, its inverse and the MX product, the root-mean-square norm with the
 * residual's addition, and log probabilities over logits.  One AMD Instinct MI355X (gfx950).
 *
 * Conventions are those of mnb.h (device pointers, status codes, `stream`, the caller owns
 * every buffer, nothing is synchronised, arguments are validated before anything is
 * enqueued), with these differences:
 *  - activations, norms and logits may be binary16, bfloat16 or (where said) binary32:
 *    `dtype` is MNB_F16, MNB_BF16 or MNB_F32;
 *  - rows may be strided: `ld...` arguments are distances between rows, in elements of the
 *    tensor, or in bytes for codes and scales;
 *  - an output shares no byte with an input or another output (MNB_ERR_ALIAS), but where said; rows
 *    between each other's rows, as column ranges of one buffer with one row distance, share none;
 *  - workspaces of these calls need no initialisation and hold nothing between calls.
 * M, N, K, V == 0 (no rows or no columns): nothing is enqueued, MNB_OK, except K == 0 of
 * mnb_mx_matmul, which fills Y with the bias or zeros.
 *
 * MX formats (OCP Microscaling Formats specification v1.0): blocks of 32 along K share a
 * scale byte e (E8M0) that stands for 2^(e - 127), 255 for NaN.  Elements:
 *   MNB_MX_FP4  E2M1, two per byte, even k in the low nibble:   codes [M, K/2] bytes
 *   MNB_MX_FP8  E4M3 (1.4.3, 0x7f / 0xff NaN):                  codes [M, K]   bytes
 * Scales: [M, K/32] bytes with a row distance that is a multiple of 16 and at least
 * 16 * ceil(K / 512), so that a row's scales are read in 16-byte pieces; the bytes past
 * K/32 of a row may hold anything and every row has its full ceil(K/512)*16 bytes.
 */
#ifndef MNB_OPS_H
#define MNB_OPS_H

#include "mnb.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MNB_F16 = 0, MNB_BF16 = 1, MNB_F32 = 2 };
enum { MNB_MX_FP4 = 0, MNB_MX_FP8 = 1 };

/* The largest `top` of mnb_logprobs. */
#define MNB_LOGPROBS_MAX_TOP 32

/*
 * Quantise X [M, K] (any of the three types, K % 32 == 0) to MX.  Per block:
 *   e = clamp(floor(log2(max |x|)) - emax, -127, 127), emax = 2 (FP4) or 8 (FP8);
 *   codes = x / 2^e rounded to nearest even, clamped to +-6 (FP4) or +-448 (FP8);
 *   a block of zeros has scale byte 0; a block that holds an infinity or a NaN has scale
 *   byte 255 (it stands for NaN throughout) and codes 0.
 * X, codes and scales 16-byte aligned, as are their row distances in bytes.
 */
int mnb_mx_quantize(const void *X, int dtype, int M, int K, int64_t ldx, int fmt, void *codes,
                    int64_t ldc, void *scales, int64_t lds, void *stream);

/* The values of an MX tensor as Y [M, K], rounded once to `dtype` (any of the three). */
int mnb_mx_dequantize(const void *codes, int64_t ldc, const void *scales, int64_t lds, int fmt,
                      int M, int K, void *Y, int dtype, int64_t ldy, void *stream);

/*
 * Device layout of an FP4 weight [N, K] for mnb_mx_matmul (K % 32 == 0, K < 2^22,
 * ceil(N / 64) ceil(K / 128) < 2^24, else MNB_ERR_UNSUPPORTED):
 * rows in groups of 64, K in steps of 128; the 4 KiB of a (group, step) hold four matrix
 * operands of 16 rows, each 16 bytes (32 consecutive k of one row) for each of 64 lanes.
 * mnb_mx_packed_sizes (host only) gives the two buffers' bytes.  Rows past N and k past K
 * are written as code 0 with scale byte 0.  scales: as above, or any row distance >= K/32.
 */
int mnb_mx_packed_sizes(int N, int K, size_t *wq_bytes, size_t *sc_bytes);
int mnb_mx_pack(const void *codes, int64_t ldc, const void *scales, int64_t lds, int N, int K,
                void *wq, void *sc, void *stream);

/*
 * Y[M,N] = X . W^T (+ bias), X an MX tensor [M, K] (fmt FP8 or FP4), W an FP4 weight packed
 * by mnb_mx_pack; Y fp16 or bf16 [M, N] row-major, rounded once from the matrix instructions' 32-bit
 * sums; bias [N] of Y's type or NULL.  How exact these sums are depends on X's format (the
 * MX specification leaves it open), in units of sum_k |x| |w| of the result:
 *   FP4 X  as a sum in 32 bits: at most (K / 128 + 1) 2^-23;
 *   FP8 X  fewer bits, as the instruction aligns its terms to the largest: at most 2^-12, measured
 *          2^-16 to 2^-22 (the smaller the longer K) over scales of 2^-8 to 2^8.  Of Y's own size that
 *          is about 2^-17 on random data, where 3 to 8% of fp16 results are a neighbour of what a
 *          32-bit sum would give; results that nearly cancel have no more than that.
 * W's sizes as for mnb_mx_pack, ceil(M / 64) ceil(N / 128) <= 2^23 - 8, ldc and lds at most 2^23, else
 * MNB_ERR_UNSUPPORTED.  A NaN scale or element of X reaches its own row of Y only, one of W its
 * own column.  codes, scales, wq, sc and Y 16-byte aligned, as are ldc and lds; bias 16-byte
 * aligned.  Y must not overlap the inputs.
 *
 * M <= 32 streams the weight once for all rows; more rows run as tiles of 64 or 128 rows.
 */
int mnb_mx_matmul(const void *codes, int64_t ldc, const void *scales, int64_t lds, int fmt,
                  const void *wq, const void *sc, const void *bias, void *Y, int dtype, int M,
                  int N, int K, void *stream);

/* The kernels mnb_mx_matmul would launch, as text (host only), e.g. "mx_gemv_fp8 ...". */
int mnb_mx_describe_route(int M, int N, int K, int fmt, char *buf, size_t buf_len);

/*
 * h = X + residual (residual NULL: h = X);  y = h / sqrt(mean(h^2) + eps) * weight
 * for each row of X [M, K], in 32 bits or more; the norm is that of the unrounded sum.
 * Outputs, each rounded once, each NULL where it is not wanted (one of Y and codes must be):
 *   hidden  h in `dtype` [M, K] (the new residual stream)
 *   Y       y in `dtype` [M, K]
 *   codes, scales   y quantised as by mnb_mx_quantize (K % 32 == 0; aligned as there, and
 *           so are the other tensors then)
 * dtype fp16 or bf16 for X, residual, weight [K], hidden and Y; weight contiguous.  hidden may be
 * residual or X itself, and Y may be X (same address and row distance); any other overlap
 * is refused.
 * Any K and any element alignment without codes.
 */
int mnb_rmsnorm(const void *X, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                float eps, int dtype, int M, int K, void *hidden, int64_t ldh, void *Y, int64_t ldy,
                int fmt, void *codes, int64_t ldc, void *scales, int64_t lds, void *stream);

/*
 * Log probabilities over logits [M, V] (any of the three types, any element alignment):
 *   logprob[m] = logits[m, tokens[m]] - lse(logits[m]), lse the log of the sum of exponentials;
 *                0 where tokens[m] < 0 (padding), NaN where tokens[m] >= V
 *   entropy[m] = -sum_v p log p, terms with p = 0 counting 0
 *   top_tokens [M, top], top_logprobs [M, top]: the `top` largest logits in falling order,
 *                equal ones by the lower index (a NaN ranks above every number)
 * A row whose logits are all -infinity, or that holds a NaN or +infinity, has no
 * distribution: its logprob (of a token >= 0), entropy and top_logprobs are NaN; its
 * top_tokens follow the order above.
 * tokens int64 [M] or NULL (then logprob is not written and may be NULL); entropy may be NULL;
 * 0 <= top <= min(MNB_LOGPROBS_MAX_TOP, V), the top outputs may be NULL for 0.  logprob, entropy and
 * top_logprobs are FP32, top_tokens int64, all contiguous.  V <= 2^22.
 * workspace: at least mnb_logprobs_workspace_bytes bytes, 16-byte aligned (NULL if that is 0).
 */
size_t mnb_logprobs_workspace_bytes(int M, int V, int dtype, int top);
int mnb_logprobs(const void *logits, int dtype, int M, int V, int64_t ldl, const int64_t *tokens,
                 int top, float *logprob, float *entropy, float *top_logprobs, int64_t *top_tokens,
                 void *workspace, size_t ws_bytes, void *stream);

/* Version of this header's calls (major * 100 + minor). */
int mnb_ops_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MNB_OPS_H */
