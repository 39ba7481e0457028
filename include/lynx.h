/*
 * lynx.h -- C ABI of the B200 (sm_100a) RT-Lynx online 2:4 activation-sparse
 * linear layer.
 *
 * The layer (RT-Lynx pages; "qingkeai.online article" = the RT-Lynx article on
 * qingkeai.online, "ai-feeds summary" = the ai-feeds.com summary of the paper):
 *
 *     Y = S(X) W^T + bias + (X A^T) B^T
 *
 *   - S(X): per token row, each group of 4 consecutive K-values keeps its 2
 *     largest magnitudes, ties to the lower position (qingkeai.online article
 *     section 02: Y = S(X) W^T with a 2:4 pattern made at run time; section 03:
 *     Top-K).  The kept values are multiplied by the norm-compensation factor
 *     s = sum|x| / sum|kept| of the row, computed in fp32 (section 03.1; ai-feeds
 *     summary, core module 1), and rounded to bf16.
 *   - (X A^T) B^T: LoRA residual of rank r on the dense X, frozen W (section
 *     03.2; the neuraltrendhub summary gives rank 64, the pages' setting).  Any
 *     r with r % 16 == 0 and 16 <= r <= 256 is accepted.
 *   - skip_sparsify: the layer stays dense, S(X) = X (section 03.3, selective
 *     layer skipping).
 *   - The sparse product runs on sparse tensor cores (tcgen05.mma.sp) with the
 *     compression, metadata layout, sparse GEMM and LoRA residual in CUDA
 *     kernels of this library (section 04).
 *
 * Conventions for every entry point:
 *   - Tensors are bf16 (bfloat16: the upper 16 bits of an IEEE fp32), row-major, contiguous,
 *     given as plain device pointers.  The caller owns and allocates every
 *     buffer; the library never allocates device memory.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Calls only enqueue work and return; nothing synchronises except
 *     lynx_check_error.
 *   - Return value: a lynx_status.  Host-side checks run before anything is
 *     enqueued: on failure nothing is launched and no buffer is touched.
 *     Device-side failures (a bounded wait that gave up) are recorded in a
 *     status word of the stream the call was enqueued on, which
 *     lynx_check_error(stream) reports; a CUDA graph captured from a stream
 *     keeps recording into that stream's word when it is replayed.
 *   - Inputs must be finite; NaN/Inf inputs give unspecified (but memory-safe)
 *     results.
 *   - Shapes: M >= 1 tokens, K >= 64 with K % 64 == 0, N >= 8 with N % 8 == 0,
 *     and, when a LoRA branch is given, 16 <= r <= 256 with r % 16 == 0.
 *     Every pointer 16-byte aligned.
 *   - Thread safety: calls from several host threads on different streams are
 *     safe.  Calls whose device work overlaps must not share output buffers or
 *     a workspace.
 */
#ifndef LYNX_H_
#define LYNX_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LYNX_API __attribute__((visibility("default")))
#else
#define LYNX_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lynx_status {
  LYNX_OK = 0,
  LYNX_ERR_INVALID_ARG = 1,         /* null pointer, A without B, bad flag */
  LYNX_ERR_UNSUPPORTED_SHAPE = 2,   /* M < 1, K % 64, N % 8, r % 16, r > 256, ... */
  LYNX_ERR_MISALIGNED = 3,          /* a pointer not 16-byte aligned */
  LYNX_ERR_WORKSPACE_TOO_SMALL = 4, /* workspace_bytes < lynx_workspace_bytes() */
  LYNX_ERR_CUDA = 5,                /* a CUDA runtime/driver call failed */
  LYNX_ERR_DEVICE_TIMEOUT = 6       /* a kernel gave up a bounded wait */
} lynx_status;

/* Human-readable name of a status code (static storage, never NULL). */
LYNX_API const char* lynx_status_string(int status);

/* ABI version: (major << 16) | minor. */
LYNX_API int lynx_version(void);

/* The LoRA rank the RT-Lynx pages use (64); the bindings' default. */
LYNX_API int lynx_lora_rank(void);

/* 1 if the kernels accept LoRA rank r (r % 16 == 0 and 16 <= r <= 256), else 0.
 * r is the N of the down-projection MMA (M = 128 rows, N a multiple of 16 up to
 * 256) and the K of the up-projection, which runs in steps of 32 (the last one
 * half empty when r % 32 == 16). */
LYNX_API int lynx_lora_rank_supported(int64_t r);

/* ---- sizes ------------------------------------------------------------- */

/* Bytes of the compressed values S(X): M x K/2 bf16 = M*K bytes. */
LYNX_API size_t lynx_vals_bytes(int64_t M, int64_t K);

/* Bytes of the 2:4 metadata in the tcgen05.mma.sp operand layout: one
 * 2048-byte block per 128 rows x 128 dense K; rows are padded to a multiple of
 * 256 (128-row blocks come in pairs, one per CTA of a CTA pair) and K to a
 * multiple of 128: ceil(M/256) * 2 * ceil(K/128) * 2048.
 * Layout: block (mb, kb) at byte (mb * ceil(K/128) + kb) * 2048; inside a
 * block, row m and dense column k (both relative to the block) map to TMEM
 * lane L = (m % 8) + 8 * ((k / 16) % 2) + 16 * (m / 16), 32-bit word
 * w = k / 32 of the lane's 16 bytes, bit b = (k % 16) + 16 * ((m / 8) % 2);
 * each group of 4 owns 4 bits: lo | hi << 2 (lo < hi its kept positions).
 * Padding rows hold the pattern of an all-zero row (lo = 0, hi = 1). */
LYNX_API size_t lynx_meta_bytes(int64_t M, int64_t K);

/* Bytes of the workspace lynx_linear needs (kept values, metadata, row scales,
 * the bf16 LoRA down-projection [M,r], per-range partial sums, one state word
 * per 32-row slice, alignment).  r = 0 (no LoRA) sizes it as for r = 64. */
LYNX_API size_t lynx_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* Where in that workspace the sparse path of lynx_linear, lynx_linear_act and
 * lynx_linear_begin leaves the metadata of S(X) (lynx_meta_bytes(M,K) bytes): a
 * byte offset, the same for every N and r.  Copied from there before the workspace
 * is used again, it is the selection lynx_sparsify_backward_meta takes. */
LYNX_API size_t lynx_workspace_meta_offset(int64_t M, int64_t K);

/* ---- the layer --------------------------------------------------------- */

/* Bytes of the scratch workspace lynx_sparsify needs (per-range partial row
 * sums and, when no row_scale buffer is given, s). */
LYNX_API size_t lynx_sparsify_workspace_bytes(int64_t M, int64_t K);

/* S(X) alone (qingkeai.online article sections 02-03.1; ai-feeds summary,
 * core module 1).
 *   X         [M,K] bf16, input activations (read only)
 *   vals      [M,K/2] bf16, out: kept values after compensation, two per group,
 *             ascending position (lynx_vals_bytes)
 *   meta      out: metadata blocks, lynx_meta_bytes(M,K) bytes (layout above);
 *             padding rows hold the pattern of an all-zero row
 *   row_scale [M] fp32, out: s per row, or NULL
 *   workspace caller-allocated scratch of workspace_bytes >=
 *             lynx_sparsify_workspace_bytes(M,K) */
LYNX_API int lynx_sparsify(const void* X, int64_t M, int64_t K, void* vals, void* meta,
                           float* row_scale, void* workspace, size_t workspace_bytes,
                           void* stream);

/* ---- S(X) without a caller workspace ---------------------------------- */

/* Largest M lynx_sparsify_noalloc accepts. */
#define LYNX_SPARSIFY_NOALLOC_MAX_ROWS 16384

/* lynx_sparsify with its scratch (the per-range partial row sums and, when
 * row_scale is NULL, s) in a fixed device array of the library instead of a
 * caller workspace: LYNX_SPARSIFY_NOALLOC_MAX_ROWS * (8 * 8 + 4) bytes
 * (1.06 MiB) per device.  The RT-Lynx pages have no counterpart of this entry
 * point; it exists for callers that cannot hand out a workspace: code behind a
 * fixed operator signature that receives only its inputs and outputs, and
 * latency-critical loops that must not call cudaMalloc (which can synchronise
 * the whole device) nor go through another runtime's allocator.
 *   Arguments, output layout, results and errors are those of lynx_sparsify.
 *   M > LYNX_SPARSIFY_NOALLOC_MAX_ROWS returns LYNX_ERR_WORKSPACE_TOO_SMALL
 *   before anything is launched.
 *   The call allocates no memory.  The first call on a device looks up the
 *   scratch's device address (cudaGetSymbolAddress) and the device's SM count;
 *   make that first call before any stream capture.
 *   Nothing in the scratch has to start at zero: every call writes all the
 *   partials it reads.
 *   All calls on one device share the one scratch array: two calls whose device
 *   work overlaps (different streams, or different host threads, without an
 *   ordering between them) race on it and give wrong results.  Calls in order
 *   on one stream are safe. */
LYNX_API int lynx_sparsify_noalloc(const void* X, int64_t M, int64_t K, void* vals, void* meta,
                                   float* row_scale, void* stream);

/* LYNX_SPARSIFY_NOALLOC_MAX_ROWS, for callers without the header. */
LYNX_API int64_t lynx_sparsify_noalloc_max_rows(void);

/* Y = S(X) W^T + bias + (X A^T) B^T  (S(X) = X when skip_sparsify != 0).
 *   X [M,K], W [N,K] (frozen backbone weight), bias [N] or NULL,
 *   A [r,K] and B [N,r] (LoRA, both or neither; r % 16 == 0, 16 <= r <= 256),
 *   Y [M,N] out.
 *   workspace: caller-allocated device buffer of workspace_bytes >=
 *   lynx_workspace_bytes(M,N,K,r), used as scratch; at 256-byte aligned
 *   offsets, in this order, it ends up holding the kept values before
 *   compensation [M,K/2] bf16, the metadata, s per row [M] fp32 and T/s [M,r]
 *   bf16 (T = X A^T).  The workspace needs no initial contents: every call
 *   writes what it reads, the GEMM's per-row-block state words included (the
 *   call's first kernel sets them to 0), so calls and replays of a captured
 *   CUDA graph that reuse one workspace in stream order are independent.
 *   The compensation factor s is applied to the fp32 accumulator row, so
 *   Y = bf16(s * (S0 W^T + (T/s) B^T) + bias) with S0 the uncompensated kept
 *   values: the same product as S(X) W^T + T B^T with one rounding fewer. */
LYNX_API int lynx_linear(const void* X, const void* W, const void* bias, const void* A, const void* B,
                int64_t M, int64_t N, int64_t K, int64_t r, int skip_sparsify, void* Y,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---- the layer in two halves ------------------------------------------ */

/* lynx_linear_act split at its one internal hand-off, so that a caller can put
 * the halves on different streams (for example the next layer's pass beside
 * this layer's GEMM, each with its own workspace):
 *   lynx_linear_begin   the sparsify pass (S(X) kept values, metadata, the row
 *                       sums and T partials) into the workspace; on the dense
 *                       path (skip_sparsify) the LoRA-down pass, or nothing;
 *   lynx_linear_finish  the GEMM from that workspace into Y.
 * Both take lynx_linear_act's arguments and check them the same way.  finish
 * must run after begin has completed on the same workspace (the same stream in
 * order, or another stream that waits on an event recorded after begin), with
 * nothing else writing that workspace in between; then the pair computes
 * exactly what lynx_linear_act does (the same Y, bit for bit).  begin reads X
 * and A; finish reads X (dense path only), W, bias, B and the workspace. */
LYNX_API int lynx_linear_begin(const void* X, const void* W, const void* bias, const void* A,
                               const void* B, int64_t M, int64_t N, int64_t K, int64_t r,
                               int skip_sparsify, int act, void* Y, void* workspace,
                               size_t workspace_bytes, void* stream);
LYNX_API int lynx_linear_finish(const void* X, const void* W, const void* bias, const void* A,
                                const void* B, int64_t M, int64_t N, int64_t K, int64_t r,
                                int skip_sparsify, int act, void* Y, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---- an activation applied in the GEMM epilogue ------------------------ */

/* Activations lynx_linear_act applies to the finished output row. */
#define LYNX_ACT_NONE 0
/* GELU, tanh form (Hendrycks & Gimpel, "Gaussian Error Linear Units"):
 * gelu(v) = v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))), the activation
 * between a DiT block's MLP up- and down-projections; the down-projection
 * (MLP.Down, the layer the qingkeai.online article takes as its example in
 * section 02) reads its output as the activation it sparsifies.  Not on the
 * RT-Lynx pages themselves, which fuse the sparsification steps so that no
 * intermediate goes back to memory (same article, section 04); this carries
 * that to the activation pass before the sparsified layer. */
#define LYNX_ACT_GELU_TANH 1

/* Y = act(S(X) W^T + bias + (X A^T) B^T): lynx_linear with the activation
 * applied in fp32 to each finished output value before its one bf16 rounding,
 * inside the GEMM's epilogue.  Saves the separate activation pass over Y (one
 * read and one write of M*N*2 bytes) that the layer feeding a sparsified
 * MLP down-projection otherwise needs.
 *   act: LYNX_ACT_NONE (then the call is lynx_linear) or LYNX_ACT_GELU_TANH;
 *   any other value returns LYNX_ERR_INVALID_ARG before anything is launched.
 *   Every other argument, the workspace and the errors are those of
 *   lynx_linear.  GELU is evaluated as v * sigmoid(2u), u = sqrt(2/pi)
 *   (v + 0.044715 v^3) (the same function: (1 + tanh u)/2 = sigmoid(2u)), with
 *   the hardware base-2 exponential and reciprocal approximations (a few fp32
 *   ulps; values whose magnitude falls below the fp32 normal range may come
 *   out as zero). */
LYNX_API int lynx_linear_act(const void* X, const void* W, const void* bias, const void* A,
                             const void* B, int64_t M, int64_t N, int64_t K, int64_t r,
                             int skip_sparsify, int act, void* Y, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ---- the fully fused variant ------------------------------------------- */

/* Y = act(S(X) W^T + bias + (X A^T) B^T) like lynx_linear_act, with the 2:4
 * selection and compression inside the GEMM (qingkeai.online article, section
 * 04: selection, compression, the sparse operand layout, the sparse GEMM and the
 * LoRA residual fused, no compressed activations written back).  A slim first
 * pass reads X for the two row sums (s) and T = X A^T only; the GEMM then loads
 * the dense X tiles itself, selects and compresses them in shared memory into
 * the tcgen05.mma.sp operand (values and metadata) and multiplies.  The
 * selection is redone for every output tile of 256 columns, so on B200 this
 * variant is slower than lynx_linear whenever N is much more than 256 (the
 * selection work grows with N / 256); lynx_linear is the default path.
 * Results equal lynx_linear's within the same tolerance (the same s, the same
 * kept values).  Arguments, workspace and errors as lynx_linear_act without
 * skip_sparsify; shapes the CTA-pair GEMM does not take (M <= 128, N < 256,
 * K % 128 != 0) run lynx_linear_act. */
LYNX_API int lynx_linear_fused(const void* X, const void* W, const void* bias, const void* A,
                               const void* B, int64_t M, int64_t N, int64_t K, int64_t r, int act,
                               void* Y, void* workspace, size_t workspace_bytes, void* stream);

/* ---- the layer on host-memory activations ------------------------------ */

/* Bytes of the device workspace lynx_linear_host needs: device copies of X and
 * Y plus the layer workspace of one row chunk. */
LYNX_API size_t lynx_linear_host_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* lynx_linear with X [M,K] and Y [M,N] in host memory (page-locked for the copies
 * to run asynchronously); W, bias, A, B stay device pointers.  The rows are
 * processed in up to 8 chunks (multiples of 256 rows): the copy of chunk i+1 into
 * the device, the layer on chunk i and the copy of chunk i-1 back to the host run
 * at the same time, the two copy directions on internal streams of the library.
 * The work is ordered after everything already enqueued on `stream`, and
 * anything enqueued on `stream` afterwards (a synchronize included) sees Y
 * complete in host memory.  Results equal lynx_linear's, row for row.
 *   workspace: device buffer of workspace_bytes >= lynx_linear_host_workspace_bytes.
 *   Errors as lynx_linear.  The first call on a device creates its two streams
 *   and its events.  Enqueues from several host threads are serialised inside
 *   the call; each call needs its own workspace and Y. */
LYNX_API int lynx_linear_host(const void* X_host, const void* W, const void* bias, const void* A,
                              const void* B, int64_t M, int64_t N, int64_t K, int64_t r,
                              int skip_sparsify, void* Y_host, void* workspace,
                              size_t workspace_bytes, void* stream);

/* lynx_linear_host with an activation in the GEMM epilogue (lynx_linear_act's
 * act argument); same workspace and errors. */
LYNX_API int lynx_linear_host_act(const void* X_host, const void* W, const void* bias, const void* A,
                                  const void* B, int64_t M, int64_t N, int64_t K, int64_t r,
                                  int skip_sparsify, int act, void* Y_host, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* The dense path of a layer that selective layer skipping leaves dense
 * (qingkeai.online article section 03.3): Y = X W^T + bias + (X A^T) B^T.
 * Same arguments and workspace as lynx_linear. */
LYNX_API int lynx_linear_dense(const void* X, const void* W, const void* bias, const void* A,
                      const void* B, int64_t M, int64_t N, int64_t K, int64_t r, void* Y,
                      void* workspace, size_t workspace_bytes, void* stream);

/* The sparse product on an S(X) made earlier by lynx_sparsify (or the
 * workspace of lynx_linear):  Y = S(X) W^T + bias + T B^T.
 *   vals [M,K/2] and meta as written by lynx_sparsify; T [M,r] bf16 or NULL,
 *   B [N,r] or NULL (both or neither, r as for lynx_linear); other arguments as
 *   above. */
LYNX_API int lynx_sparse_gemm(const void* vals, const void* meta, const void* T, const void* W,
                     const void* bias, const void* B, int64_t M, int64_t N, int64_t K, int64_t r,
                     void* Y, void* stream);

/* ---- the frozen weight in 4 bits, and the layer for a few tokens -------- */

/* With few tokens the layer's time is the time to read W.  The entry points
 * below keep the frozen weight in 4 bits with one scale per `group` consecutive
 * K-values of a row:
 *
 *     w[n,k] = s[k / group, n] * (q[n,k] - z[k / group, n]),   0 <= q, z <= 15
 *
 *   Wq      [N, K/2] bytes: row n holds its q in 32-bit little-endian words of 8
 *           consecutive k; from the low to the high nibble a word holds
 *           k = 0, 2, 4, 6, 1, 3, 5, 7 (so that one shift and one mask give two
 *           neighbouring k in the two halves of a register)
 *   scales  [K/group, N] bf16
 *   zeros   [K/group, N] bytes, each 0..15 (the low 4 bits are read), or NULL:
 *           z = 8 everywhere
 *   group   32, 64 or 128, with K % group == 0 (else LYNX_ERR_UNSUPPORTED_SHAPE)
 * N and K follow the layer's rules (N % 8 == 0, K % 64 == 0).  None of it is on
 * the RT-Lynx pages, which keep W in bf16.
 *
 * This section, the checkpoints and the backward pass: a buffer that a call writes
 * (the workspace among them) must overlap no other of its buffers, else
 * LYNX_ERR_INVALID_ARG. */

/* Bytes of Wq: N * K / 2. */
LYNX_API size_t lynx_w4_bytes(int64_t N, int64_t K);

/* W [N,K] bf16 -> Wq, scales, zeros (or NULL).  Per row and group:
 *   zeros == NULL:  s = bf16(max|w| / 7), q = clamp(rint(w / s), -8, 7) + 8;
 *   else, with hi = max(w, 0), lo = min(w, 0) over the group:
 *                   s = bf16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15),
 *                   q = clamp(rint(w / s) + z, 0, 15).
 * A group whose s is 0 stands for zeros (q = z).  rint ties to even.  A group with a
 * NaN has s = NaN, one with an infinity (and no NaN) s = infinity, both q = z (z = 0
 * where zero points are made): it stands for NaN throughout, in lynx_w4_dequantize and
 * in the outputs of lynx_linear_w4 that it enters. */
LYNX_API int lynx_w4_quantize(const void* W, int64_t N, int64_t K, int group, void* Wq, void* scales,
                              void* zeros, void* stream);

/* Wq, scales, zeros (or NULL) -> W [N,K] bf16, each value rounded once.  The
 * way to the other entry points (lynx_linear and so on) for many tokens. */
LYNX_API int lynx_w4_dequantize(const void* Wq, const void* scales, const void* zeros, int64_t N,
                                int64_t K, int group, void* W, void* stream);

/* Most rows of X lynx_linear_w4 takes. */
#define LYNX_LINEAR_W4_MAX_ROWS 32

/* LYNX_LINEAR_W4_MAX_ROWS, for callers without the header. */
LYNX_API int64_t lynx_linear_w4_max_rows(void);

/* Bytes of the workspace lynx_linear_w4 needs (T = X A^T in fp32); 0 for r = 0. */
LYNX_API size_t lynx_linear_w4_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* Y = act(X W^T + bias + (X A^T) B^T) with W in 4 bits, for 1 <= M <=
 * LYNX_LINEAR_W4_MAX_ROWS tokens (more: LYNX_ERR_UNSUPPORTED_SHAPE; dequantise
 * the weight and call lynx_linear).  The dense layer: S(X) = X.
 *   X [M,K], bias [N] or NULL, A [r,K] and B [N,r] (both or neither), Y [M,N]
 *   out, act as for lynx_linear_act.  Every sum and T are kept in fp32; Y is
 *   rounded once.  Equal calls give equal bits, and a row's do not depend on the
 *   values in the other rows.  They do depend on M, N, K, r and the device: the
 *   order of the sums goes by them, so the same token among 16 and among 17 rows
 *   may differ in its last bit.
 *   workspace: device scratch of workspace_bytes >=
 *   lynx_linear_w4_workspace_bytes(M,N,K,r); may be NULL without A and B. */
LYNX_API int lynx_linear_w4(const void* X, const void* Wq, const void* scales, const void* zeros,
                            const void* bias, const void* A, const void* B, int64_t M, int64_t N,
                            int64_t K, int64_t r, int group, int act, void* Y, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ---- activation checkpoints in 8 bits ---------------------------------- */

/* X kept for the backward pass in 8 bits: per row, every 32 consecutive values
 * share a power of two, so the values a checkpoint stands for are exact bf16
 * and a product with them needs no further rounding.
 *   q  [M,K] bytes: int8 (LYNX_CKPT8_INT8) or e4m3 (LYNX_CKPT8_E4M3)
 *   e  [M,K/32] bytes: the biased exponent of the block
 *   value = q * 2^(e - 133) for int8 (|q| <= 127), q * 2^(e - 127) for e4m3
 * int8: e = 127 + max(floor(log2 max|x|), -127), q = clamp(rint(x / 2^(e-133)),
 * -127, 127): an absolute error of at most 2^-7 of the block's largest
 * magnitude.  e4m3: e - 127 is the smallest exponent >= -127 with max|x| <= 448
 * * 2^(e-127), q rounded to e4m3: a relative error of at most 2^-4 down to 2^-13
 * of the block's largest magnitude (a block that reaches 2^127 saturates at
 * 240 * 2^120, since 2^128 is no bf16).  All ties to even.  A block with an
 * infinity or a NaN is stored as e = 255, q = 0 and stands for NaN throughout.
 * Shapes: M >= 1, K % 64 == 0.  Not on the RT-Lynx pages, which train the LoRA
 * branch but do not say what is kept for it. */
#define LYNX_CKPT8_INT8 0
#define LYNX_CKPT8_E4M3 1

/* Bytes of e: M * K / 32 (q has M * K). */
LYNX_API size_t lynx_ckpt8_exponent_bytes(int64_t M, int64_t K);

LYNX_API int lynx_ckpt8_store(const void* X, int64_t M, int64_t K, int format, void* q, void* e,
                              void* stream);

/* The values (bf16) the checkpoint stands for. */
LYNX_API int lynx_ckpt8_restore(const void* q, const void* e, int64_t M, int64_t K, int format, void* X,
                                void* stream);

/* ---- the layer's backward pass from a checkpoint ------------------------ */

/* With x the checkpoint's values and dY [M,N] bf16 the gradient of Y (before
 * the activation, if one was applied), W frozen:
 *   the adapter's gradients      lynx_lora_backward
 *   G = dY W                     lynx_linear_dense(dY, W^T laid out once as [K,N])
 *   the gradient of X            lynx_sparsify_backward_meta with the metadata of
 *                                the forward pass (sparse path);
 *                                dense path: lynx_linear_dense(dY, W^T [K,N],
 *                                NULL, B^T [r,N], A^T [K,r])
 * (lynx_linear_dense sums over N there, so N % 64 == 0.) */

/* Bytes of the workspace lynx_lora_backward needs. */
LYNX_API size_t lynx_lora_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* dT = dY B [M,r], dB = dY^T T [N,r], dA = dT^T x [r,K], with T = x A^T computed
 * from the checkpoint.  All outputs bf16, overwritten; dT may be NULL (not
 * wanted).  Sums in fp32 in an order that only the shape fixes (equal calls give
 * equal bits); T and dT enter the second products as the sum of two bf16, off
 * by at most 2^-17 of the value.
 *   dY [M,N], q and e as stored (format says how), A [r,K], B [N,r].
 *   workspace: device scratch of workspace_bytes >=
 *   lynx_lora_backward_workspace_bytes(M,N,K,r). */
LYNX_API int lynx_lora_backward(const void* dY, const void* q, const void* e, const void* A,
                                const void* B, int64_t M, int64_t N, int64_t K, int64_t r, int format,
                                void* dA, void* dB, void* dT, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Bytes of the workspace lynx_sparsify_backward needs (two floats a row). */
LYNX_API size_t lynx_sparsify_backward_workspace_bytes(int64_t M, int64_t K);

/* dX [M,K] bf16 from G = dL/dS(X) [M,K] bf16 at the checkpoint's values x: with
 * m the 2:4 selection of x (ties to the lower position), L = sum|x|,
 * Lk = sum m|x|, s = L / Lk and D = sum m G x of the row,
 *
 *   dX = s m G + sign(x) (D / Lk) (1 - s m) + dT A      (sign(0) = 0)
 *
 * the derivative of S at x where the selection does not change (the bf16 rounding
 * of S(X) passed through).  A row with Lk = 0 has s = 1 and no second term.
 * Rows of any magnitude that a checkpoint holds are in range; D is summed in fp32
 * against x in units of the row's largest block, which takes |G| up to 2^88.
 *   x is not the X of the forward pass, and neither is this m: small values of a
 * block share a code, and ties between codes go to the lower position where X
 * decided otherwise.  On heavy-tailed and on GELU activations 3 to 12 % of the
 * groups are selected otherwise, and dX is 0.17 to 0.35 of its norm away from
 * the gradient of the layer that ran.  lynx_sparsify_backward_meta is the call
 * for that gradient.
 *   dT [M,r] and A [r,K] (both or neither): the LoRA branch's share.
 *   workspace: device scratch of workspace_bytes >=
 *   lynx_sparsify_backward_workspace_bytes(M,K). */
LYNX_API int lynx_sparsify_backward(const void* G, const void* q, const void* e, const void* dT,
                                    const void* A, int64_t M, int64_t K, int64_t r, int format, void* dX,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* The same with m the selection that the forward pass made: `meta` is its
 * metadata (lynx_meta_bytes(M,K) bytes in the layout given there: lynx_sparsify's
 * output, or a copy of what lynx_linear left at lynx_workspace_meta_offset), and
 * must not be NULL.  x, s and D are taken from the checkpoint: on the activations
 * named above dX is within 0.02 (int8) and 0.005 (e4m3) of its norm of the gradient
 * at the forward pass's X at K = 4096 (values stored as 0 have lost their sign, which
 * costs more in shorter rows, as 1 / sqrt(K)).  A row whose kept values are all stored as 0 has
 * s = 1 and no second term.  Everything else as above. */
LYNX_API int lynx_sparsify_backward_meta(const void* G, const void* q, const void* e, const void* meta,
                                         const void* dT, const void* A, int64_t M, int64_t K, int64_t r,
                                         int format, void* dX, void* workspace, size_t workspace_bytes,
                                         void* stream);

/* ---- errors and metadata conversion ----------------------------------- */

/* Synchronises `stream`, then reports (and clears) the status word of that
 * stream on the current device: LYNX_ERR_DEVICE_TIMEOUT if a kernel launched on
 * it gave up a bounded wait since the last check, LYNX_ERR_CUDA if the stream
 * holds a CUDA error, else LYNX_OK.  Errors of calls on other streams stay in
 * their own words.  (A process uses at most 1023 words per device; the streams
 * after those share one more word, which any of them reports and clears.)
 * *device_code (may be NULL) receives the raw device code (0 if none). */
LYNX_API int lynx_check_error(void* stream, uint32_t* device_code);

/* Host-side conversions between the hardware metadata layout (above) and the
 * canonical one: row m owns K/8 bytes, group g is the nibble lo | hi << 2 in
 * byte m*K/8 + g/2, low nibble for even g.  Host pointers; K % 8 == 0.
 * canonical_to_hw fills padding rows with the all-zero-row pattern (lo=0,hi=1)
 * and padding K with zero bits. */
LYNX_API int lynx_meta_hw_to_canonical(const uint8_t* hw, uint8_t* canonical, int64_t M, int64_t K);
LYNX_API int lynx_meta_canonical_to_hw(const uint8_t* canonical, uint8_t* hw, int64_t M, int64_t K);

/* Profiling hook: when `event` (a cudaEvent_t passed as void*) is non-NULL,
 * lynx_linear records it on its stream between the sparsify pass and the GEMM,
 * so a caller can time the two kernels of one call separately with events
 * recorded before and after the call.  NULL (the default) turns it off.
 * While it is set, the GEMM no longer starts (programmatic launch) during the
 * tail of the sparsify pass, so a call takes slightly longer.
 * Process-wide; returns the previous event. */
LYNX_API void* lynx_profile_set_split_event(void* event);

/* Profiling hook: part 1 makes lynx_linear (and lynx_linear_act) enqueue only
 * its first kernel, the sparsify (or, on the dense path, LoRA-down) pass; part
 * 2 only what follows it (the GEMM, after a reset of its per-row-block state
 * words, and the split event, if set, between the two), on a workspace that
 * an earlier full call filled.  0 (the default) runs the whole layer.
 * Process-wide; returns the previous part (-1 for an invalid argument). */
LYNX_API int lynx_profile_set_part(int part);

/* Test hook (not for production use): when nonzero, kernels launched after
 * this call never load their inputs, so their bounded waits run out (about 2 s)
 * and lynx_check_error reports LYNX_ERR_DEVICE_TIMEOUT.  Returns the old value. */
LYNX_API int lynx_debug_set_stall(int enable);

#ifdef __cplusplus
}
#endif

#endif /* LYNX_H_ */
