/*
 * fp8_quant_grouped.h -- C ABI of the MI355X (gfx950) MoE FP8 training hot path.
 *
 * Operations (page titles as printed on the pages they come from):
 *   - "FP8 su GPU AMD: i guadagni di TorchTitan e TorchAO ora sono nel mainline PyTorch"
 *     (ai-radar.it), introduction: MoE FP8 training needs rowwise scales on activations,
 *     columnwise scales on the expert weights and an offset tensor that routes tokens to
 *     experts.  Section "La correttezza del formato viene prima del tuning": AMD's e4m3fnuz
 *     format has 240 as its largest value and no NaN/Inf encoding; scales must be taken
 *     against the maximum of the format actually used.  Section "Il guadagno vero e' nel
 *     movimento dei dati": the chain is absmax per row or column, scale, clamp, cast to FP8;
 *     the backward's transposed operand is written directly (no transpose-copy through HBM);
 *     columnwise outputs are transposed through LDS so that writes coalesce; cross-block
 *     maxima use relaxed-order atomics.
 *   - "AMD Boosts PyTorch FP8 Training on Instinct GPUs" (latestnews.news), third paragraph:
 *     the FNUZ encoding has only finite codes (no NaN/Inf) and a single, unsigned zero;
 *     grouped GEMM for MoE on ROCm.
 *   - "AMD Primus adds FP8/MXFP8 kernels, megakernel fusion and DeepSeek-V3 training at 1024
 *     GPUs" (fosswire.org), section "What Primus adds for MoE training on MI355X": FP8 and
 *     MXFP8 grouped GEMM for expert FFNs.  MXFP8 itself (1x32 blocks, E8M0 power-of-two
 *     shared scale, e4m3 elements) is defined by the OCP Microscaling Formats v1.0 spec.
 *
 * Conventions shared by every entry point:
 *   - Every pointer argument is a DEVICE pointer owned by the caller; the library never
 *     allocates, frees or retains memory.  bf16 tensors are passed as raw 16-bit patterns.
 *   - Every call is asynchronous on `stream` (0 = the null stream) and never synchronises the
 *     host.  Offsets tensors are read on the device only.
 *   - Matrices are row-major with an explicit leading dimension (elements between rows).
 *   - Offsets: int32[groups], the cumulative END row of each group: group g covers rows
 *     [offsets[g-1], offsets[g]) with offsets[-1] = 0.  Non-decreasing, offsets[groups-1] equals
 *     the row count, empty groups allowed.  The quantizers do not check this (violations give
 *     unspecified results); the grouped GEMMs check it on the device and report the result in
 *     their workspace (see fp8_grouped_gemm).  No offsets content makes a kernel access memory
 *     outside its operands.
 *   - Inputs must be finite.  Behaviour on NaN/Inf inputs is unspecified.
 *   - Host-checkable violations (null pointer, negative size, leading dimension too small,
 *     unknown format, workspace too small, a size beyond a kernel's limit) return a status
 *     and launch nothing.  A failed launch returns FP8Q_ERR_HIP.
 *   - Scale semantics: the stored scale is the quantization MULTIPLIER
 *     s = FMAX / max(absmax, 1e-12f), rounded once to fp32; dequantization multiplies by 1/s.
 *     Elements are cast as q = ENC(clamp(RN32(x * s), -FMAX, FMAX)) with round-to-nearest-even
 *     into the FP8 grid.  e4m3fnuz never yields byte 0x80 (its NaN); any value that rounds to
 *     zero gives 0x00.  e4m3fn keeps the sign of zero.
 */
#ifndef FP8_QUANT_GROUPED_H
#define FP8_QUANT_GROUPED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* hipStream_t;

#define FP8Q_ABI_VERSION 2

/* FP8 element encoding.  e4m3fnuz: bias 8, largest value 240, single zero, 0x80 is NaN
 * ("La correttezza del formato viene prima del tuning").  e4m3fn: OCP e4m3, bias 7, largest
 * value 448, signed zero, 0x7F/0xFF are NaN. */
typedef enum { FP8Q_E4M3FNUZ = 0, FP8Q_E4M3FN = 1 } fp8q_format_t;

typedef enum {
    FP8Q_OK = 0,
    FP8Q_ERR_INVALID_ARG = 1,
    FP8Q_ERR_UNSUPPORTED = 2,
    FP8Q_ERR_WORKSPACE = 3,
    FP8Q_ERR_HIP = 4
} fp8q_status_t;

typedef enum { FP8Q_GEMM_FWD_MGROUPED = 0, FP8Q_GEMM_WGRAD_KGROUPED = 1 } fp8q_gemm_mode_t;

/* Element type of a grouped GEMM's output: bf16 (round to nearest even) or fp32. */
typedef enum { FP8Q_OUT_BF16 = 0, FP8Q_OUT_FP32 = 1 } fp8q_out_t;

/* ABI version (FP8Q_ABI_VERSION) and a static text for a status code; the fp8_* names are the
 * same functions. */
int fp8q_abi_version(void);
const char* fp8q_status_string(fp8q_status_t status);
int fp8_abi_version(void);
const char* fp8_status_string(fp8q_status_t status);

/* Rowwise quantization of activations (ai-radar.it, introduction and "Il guadagno vero e' nel
 * movimento dei dati": one scale per token row, chain absmax -> scale -> clamp -> cast, fused
 * into a single pass over HBM).
 *   x       bf16 [rows][ld_x], ld_x >= cols
 *   q       u8   [rows][ld_q], ld_q >= cols: the FP8 bytes of each row
 *   scales  fp32 [rows]: s[r] = FMAX / max(max_k |x[r,k]|, 1e-12f)
 * rows == 0 or cols == 0 is a no-op that still validates its arguments (cols == 0 with
 * rows > 0 writes s = FMAX/1e-12f). */
fp8q_status_t fp8_quant_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                fp8q_format_t fmt, uint8_t* q, int64_t ld_q, float* scales,
                                hipStream_t stream);

/* Rowwise quantization of gathered rows (fosswire.org "AMD Primus adds FP8/MXFP8 kernels ...",
 * section "What Primus adds for MoE training on MI355X": the MegaMoE item fuses the token
 * exchange with the kernels that consume its rows; here the one-GPU half, routed token rows put
 * into expert order and quantized in one pass).  For r in [0, rows):
 *   q[r*ld_q + k] and scales[r] = fp8_quant_rowwise of source row i = row_index[r],
 * with i clamped into [0, src_rows) (an out-of-range index reads the nearest end row; it is
 * never an out-of-bounds access).  A source row may be listed any number of times.
 *   x          bf16 [src_rows][ld_x], ld_x >= cols
 *   row_index  int32 [rows] device
 *   q          u8   [rows][ld_q], ld_q >= cols;  scales fp32 [rows]
 * rows == 0 is a no-op; src_rows == 0 with rows > 0 is FP8Q_ERR_INVALID_ARG. */
fp8q_status_t fp8_quant_rowwise_gather(const uint16_t* x, int64_t src_rows, int64_t cols,
                                       int64_t ld_x, const int32_t* row_index, int64_t rows,
                                       fp8q_format_t fmt, uint8_t* q, int64_t ld_q,
                                       float* scales, hipStream_t stream);

/* Bytes of device workspace fp8_quant_colwise_grouped needs (its cross-block maxima). */
size_t fp8_quant_colwise_grouped_workspace_size(int64_t rows, int64_t cols, int32_t groups);

/* Columnwise quantization per row group with a transposed FP8 output (ai-radar.it,
 * introduction: colwise scales on per-expert weights, token groups from an offset tensor;
 * "Il guadagno vero e' nel movimento dei dati": the backward's transposed operand written
 * directly, output tile transposed through LDS, relaxed atomics for cross-block maxima).
 * For group g (rows [o[g-1], o[g])) and column c:
 *   scales[g*cols + c] = FMAX / max(max_{r in g} |x[r,c]|, 1e-12f)
 *   q_t[c*ld_qt + r]   = ENC(clamp(RN32(x[r,c] * scales[g*cols + c])))  for r in g
 * i.e. q_t is the column-major copy of the whole quantized matrix.  An empty group writes its
 * scales (FMAX/1e-12f) and no bytes.  Weights [E,K,N] viewed as [E*K, N] with offsets
 * K, 2K, ... give per-(expert, output column) scales and the K-contiguous B operand [N, E*K]
 * of the forward grouped GEMM; activations/gradients [M, C] with token offsets give the
 * per-(group, column) operands of the weight-gradient GEMM.
 *   x          bf16 [rows][ld_x]
 *   offsets    int32 [groups] device, groups >= 1
 *   q_t        u8   [cols][ld_qt], ld_qt >= rows
 *   scales     fp32 [groups][cols]
 *   workspace  device, >= fp8_quant_colwise_grouped_workspace_size(rows, cols, groups) bytes,
 *              no initial content required; its content after the call is unspecified.
 * Concurrent calls must use distinct workspaces. */
fp8q_status_t fp8_quant_colwise_grouped(const uint16_t* x, int64_t rows, int64_t cols,
                                        int64_t ld_x, const int32_t* offsets, int32_t groups,
                                        fp8q_format_t fmt, uint8_t* q_t, int64_t ld_qt,
                                        float* scales, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream);

/* Both layouts of an activation or gradient matrix in one call, for the operand that feeds one
 * GEMM along rows and another along columns (activations: the forward and the weight gradient;
 * gradients dY: the data gradient and the weight gradient).  Same results as the two separate
 * calls, bit for bit:
 *   q, s_rows   = fp8_quant_rowwise(x)                        (one scale per row)
 *   q_t, s_cols = fp8_quant_colwise_grouped(x, offsets)       (one scale per (group, column))
 * but x is read twice instead of three times: the maxima pass also records each row's maximum
 * per 64-column tile, and the cast pass writes the row-major and the transposed bytes from the
 * same loads (ai-radar.it, "Il guadagno vero e' nel movimento dei dati": every avoided pass
 * over HBM counts).
 *   x          bf16 [rows][ld_x]
 *   offsets    int32 [groups] device (token groups, as for fp8_quant_colwise_grouped)
 *   q          u8   [rows][ld_q], ld_q >= cols        s_rows fp32 [rows]
 *   q_t        u8   [cols][ld_qt], ld_qt >= rows       s_cols fp32 [groups][cols]
 *   workspace  >= fp8_quant_dual_grouped_workspace_size(rows, cols, groups) bytes, any content,
 *              16-byte aligned (FP8Q_ERR_INVALID_ARG otherwise).
 * Errors as for fp8_quant_colwise_grouped.  cols == 0 is a no-op. */
size_t fp8_quant_dual_grouped_workspace_size(int64_t rows, int64_t cols, int32_t groups);
fp8q_status_t fp8_quant_dual_grouped(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                     const int32_t* offsets, int32_t groups, fp8q_format_t fmt,
                                     uint8_t* q, int64_t ld_q, float* s_rows, uint8_t* q_t,
                                     int64_t ld_qt, float* s_cols, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/* fp8_quant_colwise_grouped without a workspace argument and without any allocation, for
 * callers that cannot allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  Same arguments (minus the workspace), results and
 * errors as fp8_quant_colwise_grouped, bit for bit.  Its cross-block maxima live in a static
 * device array of FP8Q_NOALLOC_SCRATCH_BYTES (8 MiB) per GPU, held until the process ends; a
 * call whose fp8_quant_colwise_grouped_workspace_size(rows, cols, groups) exceeds it returns
 * FP8Q_ERR_WORKSPACE and launches nothing.  Every call on a GPU shares that GPU's array (each
 * call clears what it uses on its stream): calls that overlap on one GPU -- on different
 * streams, or from several host threads -- race and must be serialised by the caller.  The
 * first call on a device looks up the array's device address (hipGetSymbolAddress) and keeps
 * it; a failure there returns FP8Q_ERR_HIP. */
#define FP8Q_NOALLOC_SCRATCH_BYTES (8u << 20)
fp8q_status_t fp8_quant_colwise_grouped_noalloc(const uint16_t* x, int64_t rows, int64_t cols,
                                                int64_t ld_x, const int32_t* offsets,
                                                int32_t groups, fp8q_format_t fmt, uint8_t* q_t,
                                                int64_t ld_qt, float* scales, hipStream_t stream);

/* Expert weights in both layouts at once, for quantizing them once per optimizer step and
 * reusing the bytes across micro-batches (the forward reads W^T per expert with one scale per
 * (expert, output column); the data gradient reads W along N with one scale per (expert, k)).
 * Same results as the two separate calls, bit for bit:
 *   q_rows, s_rows = fp8_quant_rowwise(w)                            (scales along N)
 *   q_t, s_cols    = fp8_quant_colwise_grouped(w, offsets K, 2K, ..) (scales along K)
 * but W is read twice instead of three times and no atomics are used: the rowwise pass also
 * writes each 128-row block's column maxima, which a small kernel reduces per expert before the
 * colwise cast pass (ai-radar.it, "Il guadagno vero e' nel movimento dei dati": fewer passes
 * over HBM; fosswire.org, "What Primus adds for MoE training on MI355X": FP8 expert weights).
 *   w        bf16 [experts*K][ld_w], ld_w >= N; expert e is rows e*K .. e*K+K-1
 *   q_rows   u8 [experts*K][ld_qr], ld_qr >= N      s_rows fp32 [experts*K]
 *   q_t      u8 [N][ld_qt], ld_qt >= experts*K      s_cols fp32 [experts][N]
 *   workspace >= fp8_quant_weights_dual_workspace_size(experts, K, N) bytes, any content.
 * Limits (FP8Q_ERR_UNSUPPORTED, nothing launched): N <= 2048, N, ld_w and ld_qr multiples of 8,
 * w 16-byte and q_rows 8-byte aligned, experts * K < 2^31 and experts * ceil(K/128) < 2^31
 * (128-row blocks along K).  experts == 0, K == 0 or N == 0 is a no-op. */
size_t fp8_quant_weights_dual_workspace_size(int64_t experts, int64_t K, int64_t N);
fp8q_status_t fp8_quant_weights_dual(const uint16_t* w, int64_t experts, int64_t K, int64_t N,
                                     int64_t ld_w, fp8q_format_t fmt, uint8_t* q_rows,
                                     int64_t ld_qr, float* s_rows, uint8_t* q_t, int64_t ld_qt,
                                     float* s_cols, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream);

/* Workspace bytes of the grouped GEMMs (fp8_grouped_gemm, fp8_mx_grouped_gemm and
 * fp8_mx_grouped_gemm_wgrad) for the given problem.  The workspace receives the offsets check
 * (below); its content before the call does not matter. */
size_t fp8_grouped_gemm_workspace_size(fp8q_gemm_mode_t mode, int64_t M, int64_t N, int64_t K,
                                       int32_t groups);

/* Scaled FP8 grouped GEMM with fp32 accumulation on FP8 MFMA and dequantization fused into
 * the epilogue (latestnews.news third paragraph: grouped GEMM for MoE on ROCm; fosswire.org
 * "What Primus adds for MoE training on MI355X": FP8 grouped GEMM for the expert FFNs;
 * ai-radar.it introduction: rowwise activation scales, colwise expert-weight scales, the
 * offset tensor routing token rows to experts).  fmt is the encoding of both operands.
 *
 * mode FP8Q_GEMM_FWD_MGROUPED (forward, groups along M):
 *   a         Xq  u8 [M][lda], lda >= K               a_scales fp32 [M]
 *   b         per group g the matrix b + g*b_group_stride, rows n = 0..N-1 at stride ldb,
 *             K bytes each (K-contiguous) ldb >= K    b_scales fp32 [groups][N]
 *             (weights quantized by fp8_quant_colwise_grouped into [N, E*K]: ldb = E*K,
 *             b_group_stride = K; weights stored [E,N,K]: ldb = K, b_group_stride = N*K)
 *   c         [M][ldc] of out_dtype, ldc >= N
 *   c[m,n] = (sum_k dec(a[m,k]) * dec(b_g[n,k])) * (1/a_scales[m]) * (1/b_scales[g,n])
 *   for m in group g.
 * mode FP8Q_GEMM_WGRAD_KGROUPED (weight gradient, groups along the contraction dimension):
 *   a         XqT u8 [K][lda], lda >= M (column-major quantized activations)
 *   a_scales  fp32 [groups][K]
 *   b         dYqT u8 [N][ldb], ldb >= M              b_scales fp32 [groups][N]
 *   b_group_stride must be 0
 *   c         [groups][K][ldc] of out_dtype, ldc >= N, group stride K*ldc
 *   c[g,k,n] = (sum_{m in g} dec(a[k,m]) * dec(b[n,m])) * (1/a_scales[g,k]) * (1/b_scales[g,n])
 *   An empty group writes zeros.  Only the bytes of tokens [0, M) are used: the padding of
 *   the token dimension (columns M..ld-1) and the bytes of other groups may hold any codes.
 *
 * Offsets check: the kernel writes two int32 words at the start of the workspace:
 *   {FP8Q_OK, -1} for valid offsets, or {FP8Q_ERR_INVALID_ARG, g} where g is the first group
 *   whose end lies below its start or beyond M, or the last group when offsets[groups-1] != M.
 *   The words are written on the stream (read them after it, no host synchronisation is done);
 *   a call with an empty output launches nothing and writes nothing.  With invalid offsets the
 *   kernel still only reads and writes inside the operands (offsets are clamped into [0, M]),
 *   but the results are unspecified.
 *
 * Accuracy: the matrix cores sum each 8 consecutive contraction products in fixed point whose
 * last bit is 2^-13 of 2^E, E the largest exponent sum (exponent of a plus exponent of b) in
 * the 8, each product truncated toward zero, and add those partial sums into an fp32
 * accumulator (measured on gfx950).  So |c - exact| <= sum over the 8-product groups of
 * (nonzero products) * 2^(E-13) / (a_scale * b_scale), plus fp32 accumulation rounding (about
 * 2^-23 of the summed magnitudes), plus the final rounding to out_dtype.  Element bits of c are
 * not specified beyond that bound.
 *
 * Kernel limits (FP8Q_ERR_UNSUPPORTED, nothing launched): forward needs K, lda, ldb and
 * b_group_stride multiples of 16; weight gradient needs lda and ldb multiples of 16 (pad the
 * token dimension); a and b 16-byte aligned; groups <= 2048; M, N, K < 2^31 and 256 * lda,
 * 256 * ldb < 2^31.  Other errors: FP8Q_ERR_WORKSPACE for a null or too small workspace,
 * FP8Q_ERR_INVALID_ARG for an unknown out_dtype or a workspace not 4-byte aligned. */
fp8q_status_t fp8_grouped_gemm(fp8q_gemm_mode_t mode, fp8q_format_t fmt, const uint8_t* a,
                               int64_t lda, const float* a_scales, const uint8_t* b,
                               int64_t ldb, int64_t b_group_stride, const float* b_scales,
                               const int32_t* offsets, int32_t groups, int64_t M, int64_t N,
                               int64_t K, void* c, int64_t ldc, fp8q_out_t out_dtype,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* MXFP8 quantization along rows (OCP MX v1.0; the pages only name MXFP8 kernels for MI355X in
 * "What Primus adds for MoE training on MI355X"): blocks of 32 consecutive elements of a row
 * share one E8M0 scale byte.  For each block: a = max |x|; e = floor(log2 a) - 8 (8 is the
 * exponent of e4m3fn's largest value), clamped to [-127, 127], e = -127 for an all-zero block;
 * e8m0 byte = e + 127; q = ENC_e4m3fn(clamp(x * 2^-e, -448, 448)).  Elements are OCP e4m3fn.
 *   x       bf16 [rows][ld_x], cols % 32 == 0
 *   q       u8   [rows][ld_q]
 *   e8m0    u8   [rows][ld_s], ld_s >= cols/32 */
fp8q_status_t fp8_mx_quant_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                   uint8_t* q, int64_t ld_q, uint8_t* e8m0, int64_t ld_s,
                                   hipStream_t stream);

/* MXFP8 quantization along columns with a transposed output: blocks of 32 consecutive rows of
 * one column share a scale.  Same per-block rule as fp8_mx_quant_rowwise.  Used for weights
 * [E*K, N] (K % 32 == 0) to obtain the K-contiguous B operand [N, E*K] and its scales.
 *   x       bf16 [rows][ld_x], rows % 32 == 0
 *   q_t     u8   [cols][ld_qt], ld_qt >= rows: q_t[c*ld_qt + r]
 *   e8m0    u8   [cols][ld_s], ld_s >= rows/32: e8m0[c*ld_s + r/32] */
fp8q_status_t fp8_mx_quant_colwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                   uint8_t* q_t, int64_t ld_qt, uint8_t* e8m0, int64_t ld_s,
                                   hipStream_t stream);

/* MXFP8 grouped GEMM, forward (groups along M), on gfx950's block-scaled FP8 MFMA:
 *   c[m,n] = sum_kb 2^(ea[m,kb] + eb_g[n,kb]) * sum_{k in kb} dec(a[m,k]) * dec(b_g[n,k])
 * with ea = a_e8m0[m*ld_sa + kb] - 127, eb_g = b_e8m0[g*sb_group_stride + n*ld_sb + kb] - 127,
 * b_g = b + g*b_group_stride (rows n at stride ldb), K % 32 == 0, e4m3fn elements, fp32
 * accumulation.  Weights from fp8_mx_quant_colwise on [E*K, N]: ldb = E*K,
 * b_group_stride = K, ld_sb = E*K/32, sb_group_stride = K/32.
 * c is [M][ldc] of out_dtype; workspace, offsets check and accuracy as for fp8_grouped_gemm
 * (each 8-product group lies inside one 32-element scale block; the E8M0 factors scale the
 * partial sums exactly).  Limits as for the forward FP8 GEMM, plus 256 * ld_sa,
 * 256 * ld_sb < 2^31. */
fp8q_status_t fp8_mx_grouped_gemm(const uint8_t* a, int64_t lda, const uint8_t* a_e8m0,
                                  int64_t ld_sa, const uint8_t* b, int64_t ldb,
                                  int64_t b_group_stride, const uint8_t* b_e8m0, int64_t ld_sb,
                                  int64_t sb_group_stride, const int32_t* offsets,
                                  int32_t groups, int64_t M, int64_t N, int64_t K, void* c,
                                  int64_t ldc, fp8q_out_t out_dtype, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/* MXFP8 grouped GEMM, weight gradient (groups along the token dimension, which is the
 * contraction) -- the MX backward (fosswire.org "AMD Primus adds FP8/MXFP8 kernels ...",
 * section "What Primus adds for MoE training on MI355X": MXFP8 grouped GEMMs for the expert
 * FFNs; block rule of OCP MX v1.0).  The operands are the transposed MX quantizations of X
 * [M, K] and dY [M, N] from fp8_mx_quant_colwise: scale blocks are 32 consecutive tokens counted
 * from token 0, so a block may straddle a group boundary; it keeps its one scale and each group
 * sums only its own tokens:
 *   c[(g*K + k)*ldc + n] = sum_{m in g} dec(a[k,m]) 2^(ea[k, m/32]) dec(b[n,m]) 2^(eb[n, m/32])
 * with ea = a_e8m0[k*ld_sa + m/32] - 127, eb = b_e8m0[n*ld_sb + m/32] - 127; empty groups write
 * zeros.
 *   a       XqT u8 [K][lda], lda >= M;  a_e8m0 [K][ld_sa], ld_sa >= M/32
 *   b       dYqT u8 [N][ldb], ldb >= M; b_e8m0 [N][ld_sb], ld_sb >= M/32
 *   offsets int32 [groups] device (as for the FP8 weight gradient); M % 32 == 0
 *   c       [groups][K][ldc] of out_dtype, ldc >= N
 * Workspace, offsets check and accuracy as for fp8_grouped_gemm.  Limits as for the FP8
 * weight-gradient GEMM, plus 256 * ld_sa, 256 * ld_sb < 2^31. */
fp8q_status_t fp8_mx_grouped_gemm_wgrad(const uint8_t* a, int64_t lda, const uint8_t* a_e8m0,
                                        int64_t ld_sa, const uint8_t* b, int64_t ldb,
                                        const uint8_t* b_e8m0, int64_t ld_sb,
                                        const int32_t* offsets, int32_t groups, int64_t M,
                                        int64_t N, int64_t K, void* c, int64_t ldc,
                                        fp8q_out_t out_dtype, void* workspace,
                                        size_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------------------------
 * Block-scaled FP8: one fp32 factor per block of 128.  Elements are OCP e4m3fn.  For a block
 *   s = 448 / max(absmax, 1e-12f)  and  d = 1 / s   (IEEE quotients, each rounded once to fp32),
 *   q = ENC(clamp(RN32(x * s), -448, 448)), round to nearest even;
 * the STORED factor is d, the one that dequantization multiplies by (x ~ dec(q) * d): the products
 * below use a factor per contraction block inside their sums, where a division has no place.
 * Blocks are counted from index 0 of their matrix; the last one of a row, column or matrix may be
 * shorter.  The quantizers take matrices of fewer than 2^24 tiles of 128 x 128, cut ones counted
 * (FP8Q_ERR_UNSUPPORTED beyond).
 *
 * fp8_block_quant_rowwise: blocks of 1 x 128 along each row (activations of the forward, output
 * gradients of the data gradient).
 *   x       bf16 [rows][ld_x], ld_x >= cols
 *   q       u8   [rows][ld_q], ld_q >= cols
 *   scales  fp32 [ceil(cols/128)][ld_s], ld_s >= rows: scales[b*ld_s + r] is d of row r, columns
 *           128 b .. (a contraction step of the product reads 256 consecutive rows' factors)
 * Any sizes and alignments; 16-byte aligned x, ld_x and cols multiples of 8, and 8-byte aligned q
 * rows take the wide accesses.  rows == 0 or cols == 0 is a no-op. */
fp8q_status_t fp8_block_quant_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                      uint8_t* q, int64_t ld_q, float* scales, int64_t ld_s,
                                      hipStream_t stream);

/* Both layouts from one read of x: blocks of 1 x 128 along rows as above, and blocks of 128 x 1
 * along columns with the bytes transposed (the operands of the weight gradient).
 *   q, s_rows  as q, scales of fp8_block_quant_rowwise, bit for bit; both may be null together, for
 *              the transposed layout alone (ld_q and ld_sr are then ignored)
 *   q_t        u8   [cols][ld_qt], ld_qt >= rows: q_t[c*ld_qt + r]
 *   s_cols     fp32 [ceil(rows/128)][ld_sc], ld_sc >= cols: d of column c, rows 128 b ..
 * Row blocks are counted from row 0 and know nothing of token groups: a block that two groups
 * share keeps its one factor, and the weight gradient sums each group's own rows of it. */
fp8q_status_t fp8_block_quant_dual(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                   uint8_t* q, int64_t ld_q, float* s_rows, int64_t ld_sr,
                                   uint8_t* q_t, int64_t ld_qt, float* s_cols, int64_t ld_sc,
                                   hipStream_t stream);

/* Expert weights in blocks of 128 x 128, both layouts from one read.
 *   w       bf16 [experts*rows][ld_w], ld_w >= cols: experts matrices of rows x cols
 *   q       u8   [experts*rows][ld_q], ld_q >= cols, or null
 *   q_t     u8   [cols][ld_qt], ld_qt >= experts*rows, or null (not both): the matrices'
 *           transposes side by side, expert e at columns e*rows ..
 *   scales  fp32 [experts][ceil(rows/128)][ceil(cols/128)], contiguous; they serve both layouts
 * experts <= 65535 (FP8Q_ERR_UNSUPPORTED beyond). */
fp8q_status_t fp8_block_quant_weights(const uint16_t* w, int64_t experts, int64_t rows, int64_t cols,
                                      int64_t ld_w, uint8_t* q, int64_t ld_q, uint8_t* q_t,
                                      int64_t ld_qt, float* scales, hipStream_t stream);

/* Block-scaled FP8 grouped GEMM.  Operand layouts, groups, offsets check and the modes are those
 * of fp8_grouped_gemm; the factors enter per contraction block:
 *
 * mode FP8Q_GEMM_FWD_MGROUPED:
 *   c[m,n] = sum_kb a_scales[kb*ld_sa + m] * b_scales[g*sb_group_stride + (n/128)*sb_n + kb*sb_k]
 *                   * sum_{k in kb} dec(a[m,k]) * dec(b_g[n,k])        for m in group g
 *   a u8 [M][lda] with a_scales fp32 [ceil(K/128)][ld_sa >= M]; b_g = b + g*b_group_stride, rows n
 *   at stride ldb >= K.  Weights [G][N][K] quantized by fp8_block_quant_weights (rows = N,
 *   cols = K): ldb = K, b_group_stride = N*K, sb_n = ceil(K/128), sb_k = 1,
 *   sb_group_stride = ceil(N/128)*ceil(K/128).  The data gradient dX[m,k] is the same call with N
 *   and K exchanged, b = q_t (ldb = G*N, b_group_stride = N) and sb_n, sb_k exchanged.
 * mode FP8Q_GEMM_WGRAD_KGROUPED:
 *   c[g,k,n] = sum_tb a_scales[tb*ld_sa + k] * b_scales[tb*sb_k + n]
 *                     * sum_{m in g, m in tb} dec(a[k,m]) * dec(b[n,m])
 *   a u8 [K][lda >= M], a_scales [ceil(M/128)][ld_sa >= K]; b u8 [N][ldb >= M], b_scales
 *   [ceil(M/128)][sb_k >= N]; b_group_stride = sb_group_stride = 0, sb_n = 1.  An empty group
 *   writes zeros; bytes of other groups and padding may hold any code.
 *
 * offsets may be null with groups == 1: one group of all M rows.  workspace may be null: the
 * offsets check is then not reported (the kernel uses clamped offsets either way); otherwise
 * fp8_grouped_gemm_workspace_size bytes.  Sums: each block's products on the matrix cores (see
 * Accuracy at fp8_grouped_gemm) from zero, times the factors into an fp32 accumulator.
 * Limits (FP8Q_ERR_UNSUPPORTED): as for fp8_grouped_gemm (M, N, K up to 2^31 - 256), (N/128 + 1) *
 * sb_n <= 2^29, and in the forward groups * ceil(M/128) * ceil(N/128) < 2^31. */
fp8q_status_t fp8_block_grouped_gemm(fp8q_gemm_mode_t mode, const uint8_t* a, int64_t lda,
                                     const float* a_scales, int64_t ld_sa, const uint8_t* b,
                                     int64_t ldb, int64_t b_group_stride, const float* b_scales,
                                     int64_t sb_n, int64_t sb_k, int64_t sb_group_stride,
                                     const int32_t* offsets, int32_t groups, int64_t M, int64_t N,
                                     int64_t K, void* c, int64_t ldc, fp8q_out_t out_dtype,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------------------------
 * A mixture-of-experts layer for a few tokens (decoding): routing, then the experts' SwiGLU
 * feed-forward on block-scaled weights.
 *
 * moe_route: x bf16 [T][ld_x >= H], router bf16 [E][ld_r >= H].
 *   logits[t,e] = sum_h x[t,h] * router[e,h]                                   (fp32 sums)
 *   scores      = softmax over e, or 1 / (1 + exp(-logits))
 *   choice      the top_k experts by scores + bias (bias fp32 [E], or null: by logits), in
 *               descending order; ties go to the lowest index, NaN goes last
 *   weights     the chosen scores (without the bias), divided by their sum if renormalize, times
 *               scale; the quotients keep their precision where the scores leave fp32's range
 *               below (sums under 2^-64 are formed from the logits), and are zeros where every
 *               chosen logit is minus infinity
 *   ids int32 [T][top_k], weights fp32 [T][top_k]; workspace moe_route_workspace_size bytes, any
 *   content, 4-byte aligned; it may be null where that is 0 (small routers).
 * Limits (FP8Q_ERR_UNSUPPORTED): E <= 1024, top_k <= 32, H, ld_x and ld_r multiples of 8, x and
 * router 16-byte aligned, T <= 1048560.  T == 0 is a no-op. */
typedef enum { FP8Q_SCORE_SOFTMAX = 0, FP8Q_SCORE_SIGMOID = 1 } fp8q_scoring_t;
size_t moe_route_workspace_size(int64_t T, int64_t H, int64_t E);
fp8q_status_t moe_route(const uint16_t* x, int64_t T, int64_t H, int64_t ld_x, const uint16_t* router,
                        int64_t E, int64_t ld_r, const float* bias, fp8q_scoring_t scoring,
                        int32_t top_k, int renormalize, float scale, int32_t* ids, float* weights,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* fp8_moe_few_tokens: for every token t
 *   y[t] = sum_j weights[t,j] * W2_e (silu(G_e x_t) * (U_e x_t)),  e = ids[t,j]
 * with e4m3fn weights in blocks of 128 x 128 (fp8_block_quant_weights): [G_e; U_e] = w13[e] is
 * 2I x H (gate rows first), W2_e = w2[e] is H x I.  Nothing is quantized: x stays bf16, and what lies
 * between the two products has 16 significant bits and fp32 range, sums are fp32.  An id
 * outside [0, E) adds nothing (an expert that lives elsewhere); a token with none gives zeros.
 *   x bf16 [T][ld_x >= H]; ids int32, weights fp32 [T][top_k]
 *   w13 rows at stride ld13 >= H, experts at w13_group_stride; w2 rows at ld2 >= I
 *   s13, s2 fp32: the factor of row n and column k of expert e is
 *     s[e*group_stride + (n/128)*s_n + (k/128)*s_k]
 *   y bf16 [T][ld_y >= H]; workspace fp8_moe_few_tokens_workspace_size bytes, any content,
 *   16-byte aligned.
 * Three kernels; every sum has a fixed order.  Limits (FP8Q_ERR_UNSUPPORTED): T <= 128 (the grouped
 * product takes more), E <= 1024, top_k <= 32, H and I multiples of 16, ld_x a multiple of 8, the
 * weights' strides multiples of 16, x, w13 and w2 16-byte aligned, ld13 and ld2 < 2^26, T * ld_x <
 * 2^30, T * top_k * I < 2^29.  T == 0 is a no-op. */
size_t fp8_moe_few_tokens_workspace_size(int64_t T, int64_t H, int64_t I, int32_t top_k);
fp8q_status_t fp8_moe_few_tokens(const uint16_t* x, int64_t T, int64_t H, int64_t ld_x,
                                 const int32_t* ids, const float* weights, int32_t top_k,
                                 const uint8_t* w13, int64_t ld13, int64_t w13_group_stride,
                                 const float* s13, int64_t s13_n, int64_t s13_k,
                                 int64_t s13_group_stride, const uint8_t* w2, int64_t ld2,
                                 int64_t w2_group_stride, const float* s2, int64_t s2_n,
                                 int64_t s2_k, int64_t s2_group_stride, int64_t E, int64_t I,
                                 uint16_t* y, int64_t ld_y, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8_QUANT_GROUPED_H */
