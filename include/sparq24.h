/*
 * sparq24 — online 2:4 prune-and-compress, dense quantizers and the energy
 * reductions that compare them, for AMD Instinct MI355X (gfx950).
 *
 * The operations follow Xiuyi Qin, "Is 2:4 Sparsity Still Worth It?
 * Semi-Structured Sparsity versus Quantization in LLM Inference"
 * (arXiv 2610.28947) as summarised on the paper-daily.com English page,
 * cited below as [PD §n] (n = the section number on that page).
 *
 * ---------------------------------------------------------------------------
 * Conventions shared by every call
 * ---------------------------------------------------------------------------
 * Operand.  A sparq24_tensor describes B x R vectors of length K along the
 *   GEMM reduction axis ("rows"); the hardware forms its groups of four along
 *   that axis [PD §1].  Element (b, r, k) lives at
 *   data + b*batch_stride + r*row_stride + k*k_stride   (strides in elements).
 *   Two layouts are accepted:
 *     K-contiguous: k_stride == 1 (e.g. X [tokens, hidden], W [out, in],
 *                   Q/K [heads*seq, head_dim], P [heads*q, keys]);
 *     transposed:   row_stride == 1 and k_stride >= R (e.g. V [heads, seq,
 *                   head_dim] pruned along seq: B = heads, R = head_dim,
 *                   K = seq, k_stride = head_dim), R <= 4194240 (65535
 *                   tiles of 64 rows, else SPARQ24_ERR_UNSUPPORTED).
 *                   sparq24_prune_compress reads it directly (16-bit
 *                   magnitude with R % 64 == 0 and K % 256 == 0: 8 x 8
 *                   blocks transposed in registers; otherwise an LDS-tiled
 *                   transpose); the
 *                   other calls (except sparq24_col_l2norm, which rejects it
 *                   with SPARQ24_ERR_UNSUPPORTED) first stage it as dense
 *                   K-contiguous rows in their workspace, which then needs
 *                   B*R*K elements more.
 *   K must be a multiple of 8 (two groups fill one metadata byte).
 * Outputs.  Always dense and K-contiguous, row-major over (b, r):
 *   kept values / kept codes [B][R][K/2], metadata [B][R][K/8],
 *   per-row scales [B][R], dense codes [B][R][K] (or [B][R][K/2] packed).
 * Memory.  Every array pointer is DEVICE memory owned by the caller, which
 *   must keep it alive until the stream work completes.  Inputs and outputs
 *   must not overlap.  The library allocates nothing and keeps no state
 *   between calls apart from device properties it caches on first use (the
 *   compute-unit count per device, each kernel's resident workgroups per CU);
 *   calls are safe from several host threads.
 * Alignment.  data, outputs and workspace must be 16-byte aligned, and
 *   batch_stride/row_stride (K-contiguous) or k_stride/batch_stride
 *   (transposed) times the element size must be multiples of 16 bytes
 *   whenever that dimension has more than one entry.
 * Streams.  Work is enqueued on `stream` (NULL = the default stream) and the
 *   call returns without synchronising.  A fault during execution surfaces at
 *   the caller's next synchronisation.
 * Workspace.  Calls taking (ws, ws_bytes): ws == NULL with ws_bytes != NULL
 *   is a size query: the call stores the bytes it needs in *ws_bytes,
 *   returns SPARQ24_OK and enqueues nothing.  Any other combination runs the
 *   call: if it needs workspace, ws must be non-NULL and *ws_bytes at least
 *   the queried size (else SPARQ24_ERR_WORKSPACE); if it needs none, ws and
 *   ws_bytes may both be NULL.  Workspace contents need no initialisation.
 * Errors.  Arguments are checked on the host before anything is enqueued;
 *   on any error nothing is enqueued.  No call aborts or throws.
 * Rounding.  Every fp32 step named below is one IEEE-754 single-precision
 *   operation (round to nearest even, subnormals kept).
 */
#ifndef SPARQ24_H
#define SPARQ24_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPARQ24_OK = 0,
  SPARQ24_ERR_INVALID = 1,     /* null pointer, negative size, unknown enum value */
  SPARQ24_ERR_UNSUPPORTED = 2, /* dtype / format / bits / layout not offered by this call */
  SPARQ24_ERR_SHAPE = 3,       /* K % 8 (K % 32 for MXFP4, K % 16 for NVFP4), K too large, bad block size */
  SPARQ24_ERR_ALIGN = 4,       /* 16-byte alignment of a pointer or stride */
  SPARQ24_ERR_WORKSPACE = 5,   /* *ws_bytes smaller than required, or ws_bytes == NULL */
  SPARQ24_ERR_DEVICE = 6,      /* no usable HIP device */
  SPARQ24_ERR_LAUNCH = 7       /* the HIP runtime rejected a kernel launch */
} sparq24_status;

typedef enum { SPARQ24_F32 = 0, SPARQ24_BF16 = 1, SPARQ24_F16 = 2 } sparq24_dtype;

typedef struct {
  const void* data;
  int32_t dtype; /* sparq24_dtype */
  int64_t batch, rows, k;
  int64_t batch_stride, row_stride, k_stride; /* in elements */
} sparq24_tensor;

/* Pruning score [PD §2, the 2:4 side's pruners]: magnitude |x|, or Wanda
 * |w| * n_k with n_k the L2 norm of input channel k (an fp32 array of K
 * entries supplied by the caller, e.g. from sparq24_col_l2norm).  The Wanda
 * product is formed exactly (in fp64). */
typedef enum { SPARQ24_SCORE_MAGNITUDE = 0, SPARQ24_SCORE_WANDA = 1 } sparq24_score;

/* Quantization formats [PD §2-§3]:
 *  NONE  keep the storage type (the 2:4 side at 16 bits);
 *  INT   symmetric b-bit round-to-nearest-even, one scale per row,
 *        qmax = 2^(b-1)-1, s = fp32(amax/qmax), code = clamp(rne(fp32(x *
 *        fp32(qmax/amax))), -qmax, qmax); codes int8 for b <= 8, int16 above;
 *  FP8   OCP e4m3 of fp32(x * fp32(448/amax)), RNE, saturating at 448, sign
 *        copied; one fp32 scale s = fp32(amax/448) per row; uint8 codes;
 *  MXFP4 E2M1 codes with one E8M0 scale per 32 elements, 2^e with
 *        e = floor(log2 amax_blk) - 2 clamped to [-127,127];
 *  NVFP4 E2M1 codes with one e4m3 scale per 16 elements plus an fp32 tensor
 *        scale s_t = fp32(T/2688), T the tensor's absolute maximum; block
 *        code = e4m3(fp32(amax_blk * fp32(448/T))), elements are E2M1 of
 *        fp32(x * fp32(1/fp32(bval*s_t))).
 * E2M1 is RNE and saturating at 6 with the sign copied; two codes per byte,
 * element 2j in the low nibble.  A row (INT/FP8) or tensor (NVFP4) whose
 * absolute maximum is below 2^-64 gets scale 0 and zero codes. */
typedef enum {
  SPARQ24_Q_NONE = 0,
  SPARQ24_Q_INT = 1,
  SPARQ24_Q_FP8_E4M3 = 2,
  SPARQ24_Q_MXFP4 = 3,
  SPARQ24_Q_NVFP4 = 4
} sparq24_qfmt;

typedef struct {
  int32_t fmt;                 /* sparq24_qfmt */
  int32_t bits;                /* INT: 2..16; ignored otherwise */
  const float* tensor_amax_in; /* NVFP4: device pointer to T, or NULL to compute T */
} sparq24_qspec;

/* Largest K accepted by the calls that need a whole row at once
 * (prune_quantize, quantize INT/FP8, error_energy, predict_R). */
#define SPARQ24_MAX_ROW_K 32768
/* Largest number of quantizer pairs of one sparq24_predict_R call. */
#define SPARQ24_MAX_PAIRS 16

/* Online 2:4 prune-and-compress [PD §3, the fused online kernel; PD intro:
 * two of every four kept along the reduction axis].
 * In every aligned group of four along K, keep the two elements with the
 * largest score (ties keep the lower position).  values [B][R][K/2] receives
 * the kept elements in the input's storage type, in position order;
 * meta [B][R][K/8] receives per group the nibble (i0 | i1 << 2), group 2j in
 * the low nibble of byte j.  col_norm: NULL for magnitude, [K] fp32 for
 * Wanda.  Reads the operand once and writes each output once. */
sparq24_status sparq24_prune_compress(const sparq24_tensor* x, int32_t score,
                                      const float* col_norm, void* values,
                                      uint8_t* meta, hipStream_t stream);

/* Dense online quantization [PD §2: the quantized side pays its online
 * quantization; PD §3: INT8 with one scale per row, FP8, MXFP4, NVFP4].
 * INT/FP8: codes [B][R][K], scales fp32 [B][R].
 * MXFP4:   codes uint8 [B][R][K/2], scales uint8 E8M0 [B][R][K/32].
 * NVFP4:   codes uint8 [B][R][K/2], scales uint8 e4m3 [B][R][K/16], and
 *          tensor_scale_out (device, 1 fp32) receives s_t.
 * Workspace: NVFP4 without tensor_amax_in needs a few KB; others need none. */
sparq24_status sparq24_quantize(const sparq24_tensor* x, const sparq24_qspec* q,
                                void* codes, void* scales, float* tensor_scale_out,
                                void* ws, size_t* ws_bytes, hipStream_t stream);

/* Fused online prune + compress + quantize of the kept values [PD §4: the
 * 2:4 side quantizes its kept values to 2m bits; PD §5: 2:4 stacked on FP8;
 * PD §3: MXFP4 and NVFP4].  Same selection and metadata as
 * sparq24_prune_compress; the kept values of each row, in compressed order,
 * are quantized as a row of K/2 values:
 *   INT/FP8: codes [B][R][K/2] (int8, int16 above 8 bits, or e4m3 bytes) and
 *            scales fp32 [B][R], one per row from the absolute maximum of
 *            that row's kept values.
 *   MXFP4:   codes uint8 [B][R][K/4] (two E2M1 per byte, low nibble first),
 *            scales E8M0 [B][R][K/64] (one per 32 kept values); K % 64 == 0.
 *   NVFP4:   codes uint8 [B][R][K/4], scales e4m3 [B][R][K/32] (one per 16
 *            kept values), tensor_scale_out (device, 1 fp32) receives s_t;
 *            T is the largest |kept value| of the operand, or
 *            *q->tensor_amax_in.  K % 32 == 0.
 * tensor_scale_out is only read for NVFP4 (NULL otherwise).  Workspace:
 * NVFP4 without tensor_amax_in needs a few KB, a transposed operand its
 * staging copy, others none (pass ws = ws_bytes = NULL).  One read of the
 * operand (plus one for the NVFP4 tensor maximum), one write per output. */
sparq24_status sparq24_prune_quantize(const sparq24_tensor* x, int32_t score,
                                      const float* col_norm, const sparq24_qspec* q,
                                      void* codes, uint8_t* meta, void* scales,
                                      float* tensor_scale_out, void* ws, size_t* ws_bytes,
                                      hipStream_t stream);

/* Error energies of both sides [PD §4].
 * For each block of rows_per_block consecutive rows (flattened over (b, r);
 * 0 = the whole operand; the last block may be shorter), out[blk][4] fp64 =
 *   { sum x^2, sum of dropped x^2, sum over kept elements of (x - xhat)^2
 *     under kept_q, sum over all elements of (x - xhat)^2 under dense_q }.
 * kept_q: NONE, INT, FP8, MXFP4 (K % 64) or NVFP4 (K % 32; T over the kept
 * values of the whole operand), blocked over the compressed row as in
 * sparq24_prune_quantize.  dense_q: INT, FP8, MXFP4 or NVFP4 (NVFP4's T is
 * over the whole operand).  Sums are accumulated in fp64 in a fixed order,
 * so repeated calls give identical bits. */
sparq24_status sparq24_error_energy(const sparq24_tensor* x, int32_t score,
                                    const float* col_norm, const sparq24_qspec* kept_q,
                                    const sparq24_qspec* dense_q, int64_t rows_per_block,
                                    double* out, void* ws, size_t* ws_bytes,
                                    hipStream_t stream);

/* Predicted R [PD §4]: for every block and pair p (kept_q[p] vs dense_q[p]),
 * out[blk][p][5] fp64 = { E_prune, E_qkept, E_2:4, E_dense, R } with
 * E_prune = dropped energy / total, E_qkept = kept error / total,
 * E_2:4 = E_prune + E_qkept (disjoint elements, so the energies add),
 * E_dense = dense error / total and R = sqrt(E_2:4 / E_dense); IEEE fp64
 * division (0/0 = NaN, x/0 = inf).  1 <= npairs <= SPARQ24_MAX_PAIRS.
 * Equal quantizers appearing in several pairs are evaluated once. */
sparq24_status sparq24_predict_R(const sparq24_tensor* x, int32_t score,
                                 const float* col_norm, const sparq24_qspec* kept_q,
                                 const sparq24_qspec* dense_q, int32_t npairs,
                                 int64_t rows_per_block, double* out, void* ws,
                                 size_t* ws_bytes, hipStream_t stream);

/* sparq24_predict_R without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, outputs and errors as
 * sparq24_predict_R, except that the workspace is a static device array of
 * SPARQ24_NOALLOC_SCRATCH_BYTES inside the library: each GPU it runs on holds
 * one copy until the process ends, and the call allocates nothing.  A call
 * whose workspace would exceed that size (as sparq24_predict_R's size query
 * reports it) returns SPARQ24_ERR_WORKSPACE and enqueues nothing.  Every call
 * on one GPU uses that GPU's array, so calls that overlap on one GPU (from
 * several host threads or on several streams) race; serialise them.  The
 * array's contents need no initialisation (each call writes before it reads). */
#define SPARQ24_NOALLOC_SCRATCH_BYTES (8u << 20)
sparq24_status sparq24_predict_R_noalloc(const sparq24_tensor* x, int32_t score,
                                         const float* col_norm, const sparq24_qspec* kept_q,
                                         const sparq24_qspec* dense_q, int32_t npairs,
                                         int64_t rows_per_block, double* out, hipStream_t stream);

/* Pairwise 4:8 prune-and-compress [PD §6: Blackwell's sparse FP4 splits each
 * group of eight into four adjacent pairs and keeps two].  In every aligned
 * group of eight along K the two pairs (2p, 2p+1) with the largest energy
 * fp64(a^2 + b^2) are kept, ties to the lower pair.  values [B][R][K/2]
 * receives the kept pairs in pair order; meta [B][R][K/16] receives per group
 * the nibble (p0 | p1 << 2), group 2j in the low nibble of byte j.
 * K % 16 == 0; K-contiguous operands only. */
sparq24_status sparq24_prune_compress_pairs48(const sparq24_tensor* x, void* values,
                                              uint8_t* meta, hipStream_t stream);

/* Pairwise 4:8 prune + quantize of the kept values [PD §6: with NVFP4 this is
 * Blackwell's sparse FP4 operand].  Selection and meta [B][R][K/16] as
 * sparq24_prune_compress_pairs48; codes, scales, tensor_scale_out, formats,
 * workspace and shape rules as sparq24_prune_quantize (kept values blocked
 * over the compressed row; the INT/FP8 row scale and the NVFP4 tensor
 * maximum come from the kept values, which need not hold the row's largest
 * element).  K % 16 == 0. */
sparq24_status sparq24_prune_quantize_pairs48(const sparq24_tensor* x, const sparq24_qspec* q,
                                              void* codes, uint8_t* meta, void* scales,
                                              float* tensor_scale_out, void* ws,
                                              size_t* ws_bytes, hipStream_t stream);

/* Predicted R of pairwise 4:8 against dense quantizers [PD §4, §6]: same
 * outputs and workspace protocol as sparq24_predict_R, with the pairwise 4:8
 * selection above in place of element-wise 2:4.  K % 16 == 0. */
sparq24_status sparq24_predict_R_pairs48(const sparq24_tensor* x, const sparq24_qspec* kept_q,
                                         const sparq24_qspec* dense_q, int32_t npairs,
                                         int64_t rows_per_block, double* out, void* ws,
                                         size_t* ws_bytes, hipStream_t stream);

/* Sparsity pattern selector of the rotated calls below. */
typedef enum {
  SPARQ24_PATTERN_24 = 0,      /* element-wise 2:4 */
  SPARQ24_PATTERN_PAIRS48 = 1, /* pairwise 4:8 */
  SPARQ24_PATTERN_DENSE = 2    /* no pruning (operator error only) */
} sparq24_pattern;

/* Block Hadamard rotation along K [PD §4: before low-bit quantization the
 * operand is multiplied by a rescaled +-1 orthogonal Hadamard matrix, which
 * spreads outliers over many elements].  Every aligned block of `block`
 * elements (a power of two, 8..4096, dividing K; so a whole row of up to
 * 4096 elements) becomes y = H x / sqrt(block)
 * with H the Sylvester Hadamard matrix (entry (i, j) = (-1)^popcount(i & j)).
 * Precision: the sums S = H x are fp64 butterflies, exact (so independent of
 * their order) whenever a block's values span at most 53 - log2(block) bits
 * from the largest magnitude's leading bit to the lowest set bit of any
 * element; a zero sum is +0; fp64(S * c), c the fp64 1/sqrt(block), is
 * rounded to fp32 and then to the storage type (round-to-nearest-even).
 * out [B][R][K] in x's storage type, K-contiguous.  Workspace: a transposed
 * operand's staging copy, else none.  Errors: block not a power of two in
 * range -> INVALID; K % block -> SHAPE; block > 512 with K > 8192 ->
 * UNSUPPORTED (such blocks are rotated by a whole 256-lane workgroup per
 * row, each lane holding at most four 8-element units of the row in
 * registers, so a row may span at most 256 * 4 * 8 = 8192 elements). */
sparq24_status sparq24_hadamard(const sparq24_tensor* x, int32_t block, void* out, void* ws,
                                size_t* ws_bytes, hipStream_t stream);

/* sparq24_quantize of the rotated operand, the rotation fused into the load
 * (one read of x): identical outputs to sparq24_hadamard followed by
 * sparq24_quantize.  block as sparq24_hadamard (0 is INVALID). */
sparq24_status sparq24_quantize_rot(const sparq24_tensor* x, int32_t block,
                                    const sparq24_qspec* q, void* codes, void* scales,
                                    float* tensor_scale_out, void* ws, size_t* ws_bytes,
                                    hipStream_t stream);

/* Magnitude prune (pattern 2:4 or pairwise 4:8) + quantization of the kept
 * values of the rotated operand, fused: identical outputs to sparq24_hadamard
 * followed by sparq24_prune_quantize (2:4, magnitude) or
 * sparq24_prune_quantize_pairs48. */
sparq24_status sparq24_prune_quantize_rot(const sparq24_tensor* x, int32_t block, int32_t pattern,
                                          const sparq24_qspec* q, void* codes, uint8_t* meta,
                                          void* scales, float* tensor_scale_out, void* ws,
                                          size_t* ws_bytes, hipStream_t stream);

/* Predicted R of the rotated operand ("Is 2:4 Sparsity Still Worth It?",
 * paper-daily.com English summary, §4: the pages report that a Hadamard
 * rotation raises R by about a factor of two on attention Q, K and on
 * linear-layer inputs), magnitude selection with the given pattern:
 * identical outputs to sparq24_hadamard followed by sparq24_predict_R (2:4)
 * or sparq24_predict_R_pairs48, up to the energy tolerance. */
sparq24_status sparq24_predict_R_rot(const sparq24_tensor* x, int32_t block, int32_t pattern,
                                     const sparq24_qspec* kept_q, const sparq24_qspec* dense_q,
                                     int32_t npairs, int64_t rows_per_block, double* out,
                                     void* ws, size_t* ws_bytes, hipStream_t stream);

/* One side of an operator-level comparison: the operand A as a GEMM would
 * consume it.  pattern: SPARQ24_PATTERN_DENSE (q: INT, FP8, MXFP4 or NVFP4
 * over all values, as sparq24_quantize), SPARQ24_PATTERN_24 or
 * SPARQ24_PATTERN_PAIRS48 (magnitude selection; q over the kept values as
 * sparq24_prune_quantize, or NONE to keep them in bf16). */
typedef struct {
  int32_t pattern;
  sparq24_qspec q;
} sparq24_side;

/* Operator-level output error [PD §2: accuracy is the relative error of the
 * operator output against a full-precision reference; PD §4: the energy
 * criterion predicts it].  For Y = A B^T with A [M][K] (the operand under
 * test) and B [N][K] (the unmodified second operand), both bf16 and
 * K-contiguous (batches folded into rows), out[m][0] = sum_n Y[m][n]^2 and
 * out[m][1 + s] = sum_n ((Ahat_s - A) B^T)[m][n]^2 for every side s, fp64
 * [M][1 + nsides].  The relative error energy of side s is the column sum
 * of 1 + s over the column sum of 0; the measured R of two sides is the
 * square root of the ratio of their error energies.
 * Arithmetic: Ahat - A per element is one fp32 FMA (code * scale - x), split
 * into bf16 hi + lo (within 2^-17 relative); products are bf16 MFMAs with
 * fp32 accumulation; per-row energies are fp32 over 128 output columns, then
 * summed in fp64.  K % 64 == 0; 1 <= nsides <= SPARQ24_MAX_PAIRS.
 * Workspace: M * 2K bf16 for one side's residual, (1 + nsides) * M * N/128
 * fp32 partials, NVFP4 partial maxima. */
sparq24_status sparq24_operator_error(const sparq24_tensor* a, const sparq24_tensor* b,
                                      const sparq24_side* sides, int32_t nsides, double* out,
                                      void* ws, size_t* ws_bytes, hipStream_t stream);

/* GEMM on the compressed 2:4 operand [PD §3: the 2:4 side multiplies the
 * pruned, compressed operand with a sparse GEMM]: c [M][N] fp32 (row-major)
 * = A B^T, A given as the output of sparq24_prune_compress (bf16 kept values
 * [M][K/2], metadata [M][K/8]), B a dense bf16 [N][K] K-contiguous operand.
 * gfx950's v_smfmac_f32_16x16x64_bf16 reads the layout as is: per lane 8
 * kept values of 16 logical k and their 16 metadata bits.  Products are
 * exact, sums fp32.  K % 64 == 0; pointers 16-byte aligned. */
sparq24_status sparq24_sparse_gemm(const void* values, const uint8_t* meta, int64_t m, int64_t k,
                                   const sparq24_tensor* b, float* c, hipStream_t stream);

/* The same GEMM tile on a dense bf16 A [M][K] (the comparison the pages
 * draw between a sparse GEMM and its dense rival): c [M][N] fp32 = A B^T. */
sparq24_status sparq24_dense_gemm(const sparq24_tensor* a, const sparq24_tensor* b, float* c,
                                  hipStream_t stream);

/* The dense FP8 rival's GEMM [PD §2: 2:4 with 16-bit values against dense
 * FP8 at equal nominal throughput]: c [M][N] fp32 = (scale_a[m] * scale_b[n])
 * * sum_k a[m][k] b[n][k] with a [M][K] and b [N][K] the e4m3 codes and
 * per-row scales of sparq24_quantize (FP8).  gfx950's
 * v_mfma_f32_16x16x128_f8f6f4; e4m3 products are exact in fp32, sums fp32,
 * then two fp32 scale multiplies.  K % 128 == 0. */
sparq24_status sparq24_fp8_gemm(const uint8_t* a, const float* scale_a, int64_t m,
                                const uint8_t* b, const float* scale_b, int64_t n, int64_t k,
                                float* c, hipStream_t stream);

/* The dense INT8 side's GEMM [PD §2, §3: INT8 with one scale per row]: c
 * [M][N] = (sum_k a[m][k] b[n][k]) * scale_a[m] * scale_b[n] (+ bias[n]) with a
 * [M][K] and b [N][K] the int8 codes and per-row scales of sparq24_quantize
 * (INT, at most 8 bits): one scale per token and one per output channel.  The
 * sums are int32 and exact (codes of -128 too), so no order or split of K
 * changes a bit; then one rounding to fp32, the two fp32 scale multiplies in
 * that order, the bias add (fp32 [N], or NULL for none) and one rounding to
 * c_dtype (sparq24_dtype).  lda and ldb are the bytes between rows (a multiple
 * of 16 where there is more than one row, at least K), ldc the elements
 * between rows of c (at least N).  a, b, c 16-byte aligned; scales and bias
 * 4-byte.  K % 16 == 0 and K <= SPARQ24_MAX_INT8_K (SHAPE); K == 0 gives the
 * bias or zeros, whatever lda and ldb.  Any M and N.  Workspace protocol as above. */
#define SPARQ24_MAX_INT8_K 131056
sparq24_status sparq24_int8_gemm(const int8_t* a, int64_t lda, const float* scale_a, int64_t m,
                                 const int8_t* b, int64_t ldb, const float* scale_b, int64_t n,
                                 int64_t k, const float* bias, int32_t c_dtype, void* c,
                                 int64_t ldc, void* ws, size_t* ws_bytes, hipStream_t stream);

/* The dense MXFP4 side's GEMM [PD §3: MXFP4, one power of two per 32 elements]:
 * c [M][N] = sum_g 2^(scale_a[m][g] + scale_b[n][g] - 254) sum_{k in g} a[m][k]
 * b[n][k] (+ bias[n]) over the groups g of 32 elements along K, with a [M][K/2]
 * and b [N][K/2] the codes and scale_a [M][K/32], scale_b [N][K/32] the E8M0
 * bytes of sparq24_quantize (MXFP4).  gfx950's v_mfma_scale_f32_16x16x128_f8f6f4
 * takes both as they are: products are exact, sums fp32 (of a group and of all,
 * in a fixed order that depends on M, N and K), then the bias add (fp32 [N], or
 * NULL) and one rounding to c_dtype (sparq24_dtype).  A group whose scale byte is
 * 255 (E8M0's NaN) makes its row of a (its column of c, for b) NaN, also where
 * its codes are zeros.  lda and ldb are the bytes between rows of codes (a
 * multiple of 16 where there is more than one row, at least K/2), ldc the
 * elements between rows of c (at least N); scales are dense, at any byte.  a, b,
 * c 16-byte aligned, bias 4-byte.  K % 32 == 0 and K <= SPARQ24_MAX_MXFP4_K
 * (SHAPE); K == 0 gives the bias or zeros.  Any M and N whose tiles one grid holds
 * (UNSUPPORTED otherwise): M and N up to 2^28 with M * N up to 2^34 always fit.
 * Workspace protocol as above. */
#define SPARQ24_MAX_MXFP4_K 131072
sparq24_status sparq24_mxfp4_gemm(const uint8_t* a, int64_t lda, const uint8_t* scale_a, int64_t m,
                                  const uint8_t* b, int64_t ldb, const uint8_t* scale_b, int64_t n,
                                  int64_t k, const float* bias, int32_t c_dtype, void* c,
                                  int64_t ldc, void* ws, size_t* ws_bytes, hipStream_t stream);

/* Root-mean-square norm with the residual's addition, quantized for the next
 * product [PD §2: the quantized side pays its online quantization]: one read of
 * x and residual, one write of each output.  Per row of K elements:
 *   h = x, or with a residual the sum fp32(x + residual) rounded to their type,
 *       which is what `sum` receives and what the norm is taken of;
 *   r = fp32(1 / sqrt(mean + eps)), mean = sum h^2 / K, all fp64 (0 where mean +
 *       eps is 0);
 *   y = fp32(fp32(h * r) * w), not rounded to h's type;
 * then the row y is quantized as sparq24_quantize does (fp32 input): q INT (2..8
 * bits) or FP8: codes [B][R][K], scales fp32 [B][R]; MXFP4 (K % 32 == 0): codes
 * [B][R][K/2], scales E8M0 [B][R][K/32].  A row with an element of h that is
 * infinite or NaN gets zero codes and a NaN scale (bytes 255); so does a row (a
 * group, with MXFP4) with a y that is.  weight: [K] of weight_dtype
 * (sparq24_dtype: fp32, or x's type).  residual and sum: x's type and shape, any
 * strides that x may have; both or neither (NULL).  sum may be residual or x
 * itself (the same rows at the same places), not overlap them otherwise (UNSUPPORTED
 * where the strides are the same; with others the caller sees to it).
 * eps: finite, >= 0.  K <= SPARQ24_MAX_ROW_K, B * R < 2^31 (else UNSUPPORTED).
 * K-contiguous operands only. */
sparq24_status sparq24_rmsnorm_quantize(const sparq24_tensor* x, const sparq24_tensor* residual,
                                        const void* weight, int32_t weight_dtype, float eps,
                                        const sparq24_qspec* q, void* codes, void* scales,
                                        const sparq24_tensor* sum, hipStream_t stream);

/* Paged 8-bit key/value cache: the quantized storage of attention's K and V
 * [PD §1, §2: K and V are operands produced online], one scale per block of
 * tokens and kv head.
 *   k: codes [blocks][heads][tokens][dim], v: codes [blocks][heads][dim][tokens]
 *   (each reduction of attention, q.k along dim and p.v along the tokens, is
 *   contiguous), k_scale and v_scale: fp32 [blocks][heads].
 * fmt: SPARQ24_Q_INT (8 bits: int8, qmax 127) or SPARQ24_Q_FP8_E4M3 (qmax 448).
 * tokens: a power of two, 16..256; dim: 64, 128, 192 or 256; blocks >= 1. */
typedef struct {
  void* k;
  float* k_scale;
  void* v;
  float* v_scale;
  int32_t fmt;
  int64_t blocks, heads, tokens, dim;
} sparq24_kvcache;

/* The sequences of one call.  Sequence b has seq_lens[b] tokens in the cache,
 * the call's new tokens included as its last ones; position p of it lives in
 * block block_table[b * table_stride + p / tokens].  The call's token rows
 * (new keys and values, or queries) are [total]: rows cu_tokens[b] ..
 * cu_tokens[b + 1] - 1 belong to sequence b (device int32 [seqs + 1],
 * ascending), or total / seqs rows each where cu_tokens is NULL.  Sequences
 * may have no rows or no tokens.  Positions at or past max_blocks * tokens (or
 * 2^31 - 256) and entries outside 0 .. blocks - 1 name no storage: nothing is
 * written there and attention sees no token there.  All arrays are device int32. */
typedef struct {
  const int32_t* block_table;
  int64_t max_blocks, table_stride;
  const int32_t* seq_lens;
  const int32_t* cu_tokens;
  int64_t seqs, total;
} sparq24_kvseqs;

/* Appends token rows to the cache.  k and v: batch = total tokens, rows = kv
 * heads, k = dim (any batch and row strides, k_stride 1), fp32, bf16 or fp16,
 * both of one type.  The i-th of a sequence's n rows becomes position
 * seq_lens[b] - n + i.  Per touched block and head, with amax the largest
 * finite |element| that the block receives: cand = fp32(amax / qmax), 0 where
 * amax < 2^-64; the new scale s is cand where the block's first token is among
 * the new ones, else max(old scale, cand); new codes are encode(fp32(x * fp32(1 /
 * s))) (nearest even, saturating, so infinities become +-qmax; NaN, and with s =
 * 0 everything, as 0); where s grew, the codes before the new ones become
 * encode(fp32(code * fp32(old * fp32(1 / s)))), otherwise they stay.  Codes behind
 * the last new token stay as they are.  Calling it again with the same arguments
 * changes nothing.  A block must receive tokens of one sequence only in a call
 * (else its codes and scale are unspecified, those of other blocks are not). */
sparq24_status sparq24_kv_append(const sparq24_kvcache* cache, const sparq24_kvseqs* seqs,
                                 const sparq24_tensor* k, const sparq24_tensor* v,
                                 hipStream_t stream);

/* Attention of query rows over the cached tokens.  q: batch = total tokens,
 * rows = query heads (a multiple of the kv heads; query head h reads kv head
 * h / (rows / heads)), k = dim, bf16 or fp16, any batch and row strides.  The
 * i-th of a sequence's n query tokens is at position seq_lens[b] - n + i.
 * With s_t = scale * <q, K_t>, K_t and V_t the stored codes times their block's
 * scale, out = sum_t exp(s_t) V_t / sum_t exp(s_t) over the visible tokens t:
 * all of the sequence, or with causal = 1 those up to the query's position,
 * and of these the last `window` ones where window > 0 (needs causal).
 * out [total][query heads][dim] in q's type (q itself may be it, where it is
 * laid out so); lse [total][query heads] fp32 (or NULL) receives log sum_t
 * exp(s_t).  A row that sees no token gets zeros and -inf.  Rows of out and lse
 * that belong to no sequence stay as they are.
 * What a row does not see (behind its position or its sequence, before its
 * window) does not reach it, whatever its bits; a visible e4m3 NaN code makes a
 * row NaN (of k) or its elements of that dim (of v).  scale: finite, > 0.
 * Block scales: 0, or 2^-80 to 2^126, in any mixture; an infinite or NaN one
 * makes the rows that see a token of its block NaN, an infinite or NaN query
 * element its row.
 * Arithmetic: codes enter fp16 MFMAs exactly, queries up to elements below 2^-27
 * of their row's largest, which are rounded to 2^-38 of that; the weights exp(s_t)
 * are rounded to fp16 (2^-11), all sums, maxima and scores are fp32.
 * Workspace: partial results of sequences that are split along their tokens and
 * the work list of more than 128 sequences; none for at most 128 where
 * max_blocks * tokens <= 1024.  Concurrent calls, and graphs that may
 * replay at the same time, need workspaces of their own. */
sparq24_status sparq24_kv_attention(const sparq24_kvcache* cache, const sparq24_kvseqs* seqs,
                                    const sparq24_tensor* q, float scale, int32_t causal,
                                    int64_t window, void* out, float* lse, void* ws,
                                    size_t* ws_bytes, hipStream_t stream);

/* Paged 4-bit key/value cache: MXFP4 along the head dim, so a token's codes
 * depend on that token alone.
 *   k and v: codes [blocks][heads][tokens][dim/2], the even dim in the low nibble;
 *   k_scale and v_scale: E8M0 bytes [blocks][heads][dim/32][tokens], so that the
 *   tokens of a group of dims lie side by side.
 * tokens, dim and blocks as in sparq24_kvcache. */
typedef struct {
  uint8_t* k;
  uint8_t* k_scale;
  uint8_t* v;
  uint8_t* v_scale;
  int64_t blocks, heads, tokens, dim;
} sparq24_kvcache_mxfp4;

/* Appends token rows to a 4-bit cache: arguments, positions and refusals of
 * sparq24_kv_append.  Per token, head and 32 dims the codes and the scale byte are
 * those of sparq24_quantize (MXFP4) of the finite elements; infinite elements
 * saturate, NaN is coded as 0.  Nothing else is written, so a block may receive
 * tokens of several sequences in a call, as long as each position of it receives
 * one. */
sparq24_status sparq24_kv_append_mxfp4(const sparq24_kvcache_mxfp4* cache,
                                       const sparq24_kvseqs* seqs, const sparq24_tensor* k,
                                       const sparq24_tensor* v, hipStream_t stream);

/* Attention of query rows over a 4-bit cache: arguments, masks, outputs, refusals
 * and workspace protocol of sparq24_kv_attention, K_t and V_t the stored codes
 * times their scales.  With bf16 queries a visible V scale above 2^96 may make its
 * rows infinite or NaN, and scales of 2^126 and 2^127 (which the append never
 * writes) count as 2^125; with fp16 queries K_t and V_t are rounded to fp16, and
 * scales above 2^13 (which no fp16 element gives) count as 2^13.  A scale byte
 * of 255 in K or V of a token makes the rows that see the token NaN; what a row
 * does not see does not reach it, whatever its bits.  An infinite or NaN query
 * element makes its row NaN; a score above fp32's range does, too, one below it
 * counts as hidden.
 * Arithmetic: K and queries enter the matrix units exactly in the queries' type, V
 * exactly in fp16; the weights exp(s_t) are rounded to fp16 (2^-11 of the weight, or
 * 2^-33 of the largest), all sums, maxima and scores are fp32.  With bf16 queries V and weights are bf16 (2^-8)
 * instead for rows of a sequence and head that meet, among up to 128 that go through
 * the cache together, a V scale outside 2^-23 .. 2^8 of a token that one of them sees
 * and whose codes there are not all zero. */
sparq24_status sparq24_kv_attention_mxfp4(const sparq24_kvcache_mxfp4* cache,
                                          const sparq24_kvseqs* seqs, const sparq24_tensor* q,
                                          float scale, int32_t causal, int64_t window, void* out,
                                          float* lse, void* ws, size_t* ws_bytes,
                                          hipStream_t stream);

/* Wanda's input-channel norms [PD §2]: norms[k] = fp32(sqrt(sum over all
 * (b, r) of x[b][r][k]^2)), the sum in fp64 (fixed order), the square root in
 * fp64, then rounded once.  x is an activation [tokens, channels] given with
 * rows = tokens and k = channels (K-contiguous).  Workspace: a few hundred KB. */
sparq24_status sparq24_col_l2norm(const sparq24_tensor* x, float* norms, void* ws,
                                  size_t* ws_bytes, hipStream_t stream);

/* Plain device copy of `bytes` bytes (16-byte aligned, bytes % 16 == 0): the
 * read-once/write-once bandwidth baseline the prune kernels are compared to. */
sparq24_status sparq24_copy(const void* src, void* dst, size_t bytes, hipStream_t stream);

/* Storage bits per original element [PD §2: values, position indices and
 * scales are all charged].  Host-only arithmetic; no device needed.
 * sparse24 = 0: dense q; = 1: 2:4 with kept values in q (2 position bits per
 * kept value); = 2: pairwise 4:8 (2 bits per kept pair).  Sparse block
 * scales cover kept values, so they cost half as much per original element.
 * row_len: elements sharing one per-row scale (INT/FP8), 0 to leave scales
 * out.  value_bits:
 * width for SPARQ24_Q_NONE.  tensor_elems: NVFP4 tensor size, 0 to leave its
 * scale out.  Returns a negative value for an invalid spec. */
double sparq24_bits_per_element(const sparq24_qspec* q, int32_t sparse24, int64_t row_len,
                                int32_t value_bits, int64_t tensor_elems);

/* Static text for a status code. */
const char* sparq24_status_string(sparq24_status s);

/* Library version as "major.minor.patch". */
const char* sparq24_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SPARQ24_H */
