/*
 * gptq.h - C ABI of the MI355X (gfx950) GPTQ layer quantizer.
 *
 * The method (pages cited by title and section):
 *  - "GPTQ" (wikiprompt.org), "Enfoque Técnico": second-order (Hessian)
 *    information of the layer loss; weight columns are quantized one at a
 *    time and the columns not yet quantized receive a closed-form correction
 *    derived from Optimal Brain Quantization; grouped quantization with a
 *    scale per group; 4, 3 and 2 bits.
 *  - "El balance de errores de la inferencia de pocos bits" (auturnal.com),
 *    section 1: uniform affine format with a scale and a zero point; a
 *    format must state its signed range, grouping direction, group size,
 *    scale precision, rounding rule, clipping method and packing layout.
 *  - "Resumen Técnico: GPTQ-intrinsic LoRA" (gist.science 2606.01412),
 *    "Declaración del Problema": the objective ||X W - X W_hat||_F^2 over a
 *    calibration matrix X; "Metodología" 2: standard GPTQ factorises the
 *    regularised Hessian by Cholesky with a parameter lambda, and the
 *    augmented variant appends full-precision columns that are never rounded.
 *
 * Format fixed by this library (the pages leave these open):
 *  - H = 2 X^T X, fp32, full symmetric n x n, row-major.
 *  - lambda = damp * mean(diag H); a zero diagonal entry is replaced by 1
 *    before ordering and damping.
 *  - groups: g consecutive columns of one output row, in processing order;
 *    range = [min(0, min v), max(0, max v)] of the group's current values
 *    when the sweep reaches its first column, (-1, 1) if degenerate; no
 *    clipping search. s = (xmax - xmin) / (2^b - 1) (fp32),
 *    z = rint(-xmin / s) stored as uint8 in [0, 2^b - 1],
 *    q = clamp(rint(w / s) + z, 0, 2^b - 1), rint = round half to even,
 *    reconstruction s * (q - z). Codes are unsigned.
 *  - act_order: columns 0..n_quant-1 processed by descending diag(H)
 *    (stable); columns n_quant..n-1 stay last.
 *  - packing: per row, code k (original column order) occupies bits
 *    [k*b, k*b + b) of an LSB-first stream of little-endian uint32 words;
 *    ceil(n_quant*b/32) words per row; codes may straddle two words.
 *
 * Conventions for every call:
 *  - Matrices are row-major. W is d_out x n (PyTorch Linear layout), X is
 *    T x n. All data pointers are DEVICE pointers owned by the caller; the
 *    library never allocates or frees device memory. Scratch memory is the
 *    caller's ``workspace`` (size from the matching *_workspace_bytes call,
 *    256-byte aligned base).
 *  - ``stream`` is a hipStream_t (NULL = the legacy default stream). Work is
 *    enqueued on it in order.
 *  - Argument errors return GPTQ_EINVAL before anything is enqueued.
 *  - HIP launch or runtime errors return GPTQ_EHIP; gptq_last_error() gives
 *    the text (thread-local).
 */
#ifndef GPTQ_MI355X_H
#define GPTQ_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GPTQ_OK = 0,
  GPTQ_EINVAL = -1,      /* bad argument; nothing enqueued */
  GPTQ_ENOTPD = -2,      /* damped Hessian not positive definite */
  GPTQ_ENONFINITE = -3,  /* NaN/Inf in W or H */
  GPTQ_EHIP = -4,        /* HIP runtime or launch failure */
  GPTQ_EWORKSPACE = -5   /* workspace NULL, misaligned or too small */
} gptq_status;

typedef enum { GPTQ_BF16 = 0, GPTQ_F32 = 1 } gptq_dtype;

typedef struct {
  uint32_t struct_size; /* sizeof(gptq_params); at least offsetof(sym); a
                           field is read only when struct_size covers it */
  int32_t bits;         /* 2, 3 or 4 */
  int32_t group;        /* g >= 8; n_quant % g == 0; g % block == 0 or block % g == 0 */
  float damp;           /* lambda = damp * mean(diag H); >= 0, finite */
  int32_t block;        /* lazy-batch width B: 32, 64 or 128 */
  int32_t act_order;    /* 0 or 1 */
  int64_t n_quant;      /* 1..n; columns n_quant..n-1 receive feedback only */
  int32_t sym;          /* 0: affine grid (scale and zero point per group);
                           1: symmetric alphabet {-A..A}, A = 2^(bits-1) - 1,
                           s = max|v| / A over the group's current values
                           (1 / A for a group of zeros), stored as codes
                           q + A with zeros = A. Read only when struct_size
                           covers it (older callers: 0). ("Resumen Técnico:
                           GPTQ-intrinsic LoRA": a finite integer alphabet of
                           size 2B + 1.) */
  int32_t scale_fp16;   /* 0: scales in fp32; 1: each group's scale is rounded
                           to binary16 (nearest, ties to even; 0 -> 2^-24)
                           before the zero point, the codes and w_hat use it,
                           so the fp32 scales output holds binary16 values
                           that convert exactly. Read only when struct_size
                           covers it (older callers: 0). ("El balance de
                           errores de la inferencia de pocos bits", section
                           1: the precision of the scales is part of the
                           format.) */
  int32_t reserved;     /* 0. (With it the block grew from 40 to 48 bytes, so a
                           caller built before scale_fp16 existed, whose
                           struct_size is 40, never has its padding read.) */
} gptq_params;

typedef struct {
  /* all device pointers, caller-allocated; NULL = not wanted (except where noted) */
  uint32_t *qweight; /* d_out x ceil(n_quant*bits/32) packed codes, original column order */
  uint8_t *codes;    /* d_out x n_quant unpacked codes, original column order */
  float *scales;     /* REQUIRED: d_out x (n_quant/group), group order (processing order) */
  uint8_t *zeros;    /* REQUIRED: d_out x (n_quant/group), integer zero points */
  int32_t *g_idx;    /* n_quant: group index of each original column */
  float *w_hat;      /* d_out x n: s*(q-z) for quantized columns, the fp32
                        feedback-updated values for columns >= n_quant;
                        original column order */
  float *row_loss;   /* d_out: sum over the row's columns of e_j^2,
                        e_j = (w_j - w_hat_j) / U_jj */
} gptq_outputs;

/* ---- Hessian accumulation ------------------------------------------------
 * H (n x n fp32, row-major, ld = n) += 2 X^T X, or H = 2 X^T X when
 * zero_first != 0. X: T x n, row stride ldx >= n elements, dtype xdt
 * (bf16 products are exact in fp32; accumulation is fp32, split over token
 * chunks and summed in a fixed order: results are bitwise reproducible).
 * H stays exactly symmetric. T == 0 only applies zero_first.
 * Asynchronous on ``stream``. Workspace: gptq_hessian_workspace_bytes.
 * ("GPTQ", "Enfoque Técnico": second-order information; factor 2 and fp32
 * storage are this library's convention.) */
gptq_status gptq_hessian_workspace_bytes(int64_t T, int64_t n, gptq_dtype xdt,
                                         size_t *bytes);
gptq_status gptq_accumulate_hessian(void *stream, const void *X, gptq_dtype xdt,
                                    int64_t T, int64_t n, int64_t ldx, float *H,
                                    int zero_first, void *workspace,
                                    size_t workspace_bytes);

/* ---- Layer quantization ----------------------------------------------------
 * GPTQ of W (d_out x n, dtype wdt, row stride ldw >= n) against H (n x n fp32,
 * symmetric, not modified). Steps: dead-column fix and damping, optional
 * act-order, upper Cholesky factor U of (H + lambda I)^-1 (U^T U = H_d^-1),
 * column sweep in blocks of B with in-block error feedback and a lazy-batch
 * trailing update, then un-permutation and packing.
 * Synchronises ``stream`` before returning to read the device status:
 * GPTQ_ENOTPD / GPTQ_ENONFINITE set *fail_col (if fail_col != NULL) to the
 * first offending ORIGINAL column (-1 if unknown); outputs are then
 * unspecified. d_out == 0 is a no-op.
 * Workspace: gptq_workspace_bytes(d_out, n, p) bytes, 256-byte aligned,
 * owned by the caller, not read before it is written (its contents on entry
 * do not matter). It holds the factorisation (two n x n fp32 matrices and
 * U's split-bf16 parts; for n >= 6144 also the bf16 pieces of one
 * 2048-column super-panel, and for the inverse's block products of 1024 or
 * more output tiles the pieces of the largest one's operands: 2.8 GB at
 * n = 28672), the fp32 working weights, one super-block of errors and the
 * processing-order codes.
 * ("GPTQ" (wikiprompt.org), "Enfoque Técnico": the columns are quantized in
 * turn and the columns not yet quantized get the closed-form Optimal Brain
 * Quantization correction, with groups of weights sharing a scale;
 * "El balance de errores de la inferencia de pocos bits", section 1: scale,
 * zero point, rounding and packing fields of the format; "Resumen Técnico:
 * GPTQ-intrinsic LoRA", "Detalles de Implementación": the Cholesky
 * factorisation of the lambda-regularised Hessian; "Metodología" 2: appended
 * columns n_quant..n-1 that absorb the feedback unrounded.) */
gptq_status gptq_workspace_bytes(int64_t d_out, int64_t n, const gptq_params *p,
                                 size_t *bytes);
gptq_status gptq_quantize_layer(void *stream, const void *W, gptq_dtype wdt,
                                int64_t d_out, int64_t n, int64_t ldw,
                                const float *H, const gptq_params *p,
                                void *workspace, size_t workspace_bytes,
                                const gptq_outputs *out, int64_t *fail_col);

/* ---- The factorisation alone (steps 2-3 of quantize_layer) ----------------
 * U_out (n x n fp32 row-major): upper Cholesky factor U of the inverse of
 * the damped, dead-fixed, (optionally) act-order-permuted H, in processing
 * order (U^T U = H_d^-1; strict lower part zero). perm_out (n int32, may be
 * NULL): original column at each processing position. Uses p->damp,
 * p->act_order and p->n_quant only; workspace: gptq_workspace_bytes(0, n, p).
 * Synchronises like quantize_layer.
 * ("Resumen Técnico: GPTQ-intrinsic LoRA", "Detalles de Implementación":
 * Cholesky of the regularised Hessian.) */
gptq_status gptq_factor_hinv(void *stream, const float *H, int64_t n,
                             const gptq_params *p, void *workspace,
                             size_t workspace_bytes, float *U_out,
                             int32_t *perm_out, int64_t *fail_col);

/* ---- Packing (the layout above) -------------------------------------------
 * codes: d_out x n_quant uint8 (values must be < 2^bits; higher bits are
 * masked off), qweight: d_out x ceil(n_quant*bits/32) uint32. Asynchronous. */
gptq_status gptq_pack_codes(void *stream, const uint8_t *codes, int64_t d_out,
                            int64_t n_quant, int32_t bits, uint32_t *qweight);
gptq_status gptq_unpack_codes(void *stream, const uint32_t *qweight,
                              int64_t d_out, int64_t n_quant, int32_t bits,
                              uint8_t *codes);

/* ---- Inference: dequantising product of a packed layer ---------------------
 * Y (M x d_out fp32, row pitch ldy >= d_out) = X W_hat^T for X (M x n, bf16
 * only: xdt must be GPTQ_BF16, row pitch ldx >= n with ldx % 8 == 0, 16-byte
 * aligned base) and W_hat[o][k] = scales[o][k/group] * (q[o][k] -
 * zeros[o][k/group]), the codes q read from qweight in the layout above
 * (d_out x n*bits/32 words, 16-byte aligned base, n_quant = n). Groups must
 * be contiguous in qweight's column order: a layer quantized without
 * act-order as it is, an act-order layer after gptq_repack_act_order (then
 * pass its perm). group must be a positive multiple of 32 that divides n.
 * Products of bf16 activations and the integers q - z are exact in fp32 and
 * each group's sum is scaled once (the weights are never rounded to bf16);
 * sums are fp32 in a fixed order, so results are bitwise reproducible.
 * Workspace: gptq_dequant_matmul_workspace_bytes (the gathered activations
 * when permuted, and fp32 partials when few output tiles split the groups;
 * 0 when neither applies).
 * Asynchronous on ``stream``. M == 0 or d_out == 0 enqueues nothing; n == 0
 * writes zeros.
 * ("El balance de errores de la inferencia de pocos bits", section 6: the
 * saving is realised by a kernel that unpacks, dequantises and multiplies;
 * decode and prefill are separate regimes. Section 1: reconstruction
 * s (q - z).) */
gptq_status gptq_dequant_matmul_workspace_bytes(int64_t M, int64_t n, int64_t d_out,
                                                int32_t bits, int32_t group,
                                                int32_t permuted, size_t *bytes);
/* perm: NULL, or n int32 column indices (see gptq_repack_act_order): the
 * product is then X[:, perm] W_hat^T with qweight, scales and zeros in that
 * column order; X is gathered into the workspace (permuted = 1 in the size
 * call), so its rows need no alignment then. */
gptq_status gptq_dequant_matmul(void *stream, const void *X, int32_t xdt, int64_t M,
                                int64_t n, int64_t ldx, const uint32_t *qweight,
                                const float *scales, const uint8_t *zeros,
                                const int32_t *perm, int64_t d_out, int32_t bits,
                                int32_t group, float *Y, int64_t ldy, void *workspace,
                                size_t ws_bytes);

/* ---- The product without a workspace -----------------------------------------
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, serving loops that must not call hipMalloc, harnesses that
 * forbid it. Same arguments, result and errors as gptq_dequant_matmul (the
 * same kernels, bit-identical Y), but its scratch (the gathered activations
 * of a permuted product, the fp32 partials of a split product) lives in a
 * static device array of GPTQ_NOALLOC_SCRATCH_BYTES that the library holds
 * on every GPU it runs on until the process ends; nothing is allocated or
 * freed. A product whose scratch, gptq_dequant_matmul_workspace_bytes(M, n,
 * d_out, bits, group, perm != NULL), exceeds that size returns GPTQ_EINVAL
 * before anything is enqueued. The array belongs to the current device
 * (hipGetDevice): ``stream`` must be a stream of that device. Every call on
 * one GPU shares that GPU's array, so calls that may overlap on one GPU
 * (concurrent streams, several host threads) race and give wrong results:
 * serialise them. The array keeps the last call's contents; every value a
 * call reads from it was written by the same call. */
#define GPTQ_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
gptq_status gptq_dequant_matmul_noalloc(void *stream, const void *X, int32_t xdt,
                                        int64_t M, int64_t n, int64_t ldx,
                                        const uint32_t *qweight, const float *scales,
                                        const uint8_t *zeros, const int32_t *perm,
                                        int64_t d_out, int32_t bits, int32_t group,
                                        float *Y, int64_t ldy);

/* ---- Act-order layers for the product ---------------------------------------
 * A layer quantized with act-order has, in the original column order, groups
 * that are not contiguous (g_idx). The product is invariant to one
 * permutation of the columns of both X and W_hat, so such a layer is used
 * through the order perm that lists group 0's columns, then group 1's, ...
 * (a stable sort of g_idx): perm_out (n int32) receives it, qweight_out (same
 * size as qweight) the codes repacked in that order, whose groups are then
 * contiguous and match scales and zeros as quantize_layer wrote them. g_idx
 * must give every group exactly `group` columns (as quantize_layer's does);
 * otherwise perm is not a permutation and the product is wrong (entries of a
 * short group stay 0; nothing is read out of bounds). Workspace:
 * gptq_repack_act_order_workspace_bytes (d_out x n bytes of codes).
 * Asynchronous. ("El balance de errores de la inferencia de pocos bits",
 * section 1: the grouping direction is part of the format.) */
gptq_status gptq_repack_act_order_workspace_bytes(int64_t d_out, int64_t n, size_t *bytes);
gptq_status gptq_repack_act_order(void *stream, const uint32_t *qweight,
                                  const int32_t *g_idx, int64_t d_out, int64_t n,
                                  int32_t bits, int32_t group, uint32_t *qweight_out,
                                  int32_t *perm_out, void *workspace, size_t ws_bytes);

/* ---- Mixtures of experts: rows in the order of their experts, and back -------
 * A layer with E experts sends each of T tokens to k of them. The packed
 * products below, and gptq_accumulate_hessian on a slice of rows, want the
 * rows of one expert contiguous. A slot is a pair (t, j), its number
 * i = t k + j; R = T k.
 *
 * gptq_route: expert_ids (T x k int32, row pitch ldi >= k) -> the stable
 * order of the slots by expert. offsets (E + 1 int32): expert e holds the
 * places offsets[e] .. offsets[e + 1] - 1. rows (R int32): the token of each
 * place. inverse (R int32, slot order): each slot's place. Ids outside
 * [0, E) (padding, dropped tokens) hold no place: their inverse is -1, and
 * rows is -1 from offsets[E] on. 1 <= E <= GPTQ_MAX_EXPERTS, 1 <= k,
 * T k <= 2^31 - 65536; T == 0 writes zero offsets. The order does not depend on
 * timing. Workspace: gptq_route_workspace_bytes (0 for up to 4096 slots). */
#define GPTQ_MAX_EXPERTS 1024
gptq_status gptq_route_workspace_bytes(int64_t T, int64_t k, int64_t E, size_t *bytes);
gptq_status gptq_route(void *stream, const int32_t *expert_ids, int64_t ldi, int64_t T, int64_t k, int64_t E,
                       int32_t *offsets, int32_t *rows, int32_t *inverse, void *workspace, size_t ws_bytes);

/* From here on R is the number of rows of Xs, Ys and dYs: T k, or any other
 * number (a capacity). inverse, weights and dweights are in slot order and
 * have T k entries whatever R is.
 *
 * gptq_dispatch: Xs[inverse[t k + j]] = X[t] (bits copied; X: T x n, Xs: R x
 * n, dtype dt, row pitches ldx, lds >= n). Slots whose place is outside
 * [0, R) are skipped, and rows of Xs that no slot names keep what they held.
 * Places inside [0, R) must be distinct.
 *
 * gptq_combine: Y[t] = sum_j weights[t k + j] Ys[inverse[t k + j]], summed in
 * the order of j in fp32 and rounded once (Y: T x n, ydt; Ys: R x n, ysdt;
 * weights: T k fp32, or NULL for weights of one, which makes it the gradient
 * of gptq_dispatch). Slots whose place is outside [0, R) add nothing; a token
 * with none gets zeros.
 *
 * gptq_combine_grad: the gradients of gptq_combine for dY (T x n, dydt):
 * dYs[inverse[i]] = weights[i] dY[t] (R x n, odt; rows that no slot names
 * keep what they held; places inside [0, R) must be distinct) and dweights[i]
 * = <dY[t], Ys[inverse[i]]> (T k fp32, all of them written: 0 for a slot whose
 * place is outside [0, R); fp32 sums in a fixed order).
 *
 * dtypes are GPTQ_BF16 or GPTQ_F32, each argument its own; any alignment and
 * pitch. No output may overlap an input. At most 2^32 - 512 threads start at
 * once: T ceil(n / 8) of them in gptq_combine and gptq_dispatch (fp32: T
 * ceil(n / 4); T n where a row has less than 16 bytes), 256 T in
 * gptq_combine_grad. All asynchronous, no workspace. */
gptq_status gptq_dispatch(void *stream, const void *X, int32_t dt, int64_t T, int64_t n, int64_t ldx, int64_t k,
                          const int32_t *inverse, int64_t R, void *Xs, int64_t lds);
gptq_status gptq_combine(void *stream, const void *Ys, int32_t ysdt, int64_t R, int64_t lds, const int32_t *inverse,
                         const float *weights, int64_t T, int64_t n, int64_t k, void *Y, int32_t ydt, int64_t ldy);
gptq_status gptq_combine_grad(void *stream, const void *dY, int32_t dydt, int64_t ldy, const void *Ys, int32_t ysdt,
                              int64_t R, int64_t lds, const int32_t *inverse, const float *weights, int64_t T,
                              int64_t n, int64_t k, void *dYs, int32_t odt, int64_t ldo, float *dweights);

/* ---- Products of experts' packed weights --------------------------------------
 * E layers of the same shape in the packed layout of gptq_dequant_matmul, one
 * after another: qweight E x d_out x n*bits/32 words (16-byte aligned base),
 * scales and zeros E x d_out x n/group; group a positive multiple of 32 that
 * divides n, groups contiguous (layers quantized without act-order); zero
 * points in 0 .. 2^bits - 1, as gptq_quantize_layer writes them. offsets
 * (E + 1 int32 on the device, as gptq_route writes them) split the R rows
 * into the experts' segments; NULL with E = 1 gives all rows to the one
 * layer. Rows from offsets[E] on are not read, and their outputs keep what
 * they held. The offsets are read on the device (nothing waits for the host),
 * clamped to [0, R] there.
 *
 * gptq_expert_matmul: Y[p] = X[rows[p]] W_hat_e^T for the rows p of expert e
 * (Y: R x d_out, ydt bf16 or fp32, row pitch ldy; X: T x n bf16, row pitch
 * ldx). rows (R int32, as gptq_route writes them; clamped to [0, T)) spares
 * the copy of gptq_dispatch; NULL: X holds the R sorted rows (T >= R).
 * Products of activations and integers are exact in fp32, sums are fp32 in a
 * fixed order, and groups are scaled in fp32: the weights are not rounded.
 * Results are bitwise reproducible. Few rows per expert (R <= 16 E, 16-byte
 * aligned) take a matrix-vector form, which at 4 bits sums x (16 + q) over 128
 * codes: an infinite activation, or one above 2^116, may give NaN or an
 * infinity there where the sum is infinite or still finite. Many (R > 512 E,
 * 4 bits, groups that are multiples of 128, tiles for half of the GPU) keep
 * one running sum in units of the current group's scale; there the weights of
 * a group whose scale is outside 2^-40 .. 2^40 are rounded to bf16, a partial
 * sum above 2^88 may become infinite (in a group of scale 2^-40), and what is
 * below 2^-109 may be lost (scale 2^40).
 *
 * gptq_expert_matmul_grad: dX[p] = dY[p] W_hat_e (dX: R x n, dxdt; dY: R x
 * d_out bf16, row pitch ldy). The scale changes along this sum: with a bf16
 * result each weight's fp32 value s (q - z) is rounded to bf16 once (relative
 * 2^-8 at most; the result's error is about 1.4 times what its own rounding
 * gives); with an fp32 result it is taken in three bf16 pieces, which hold
 * its fp32 value (below 2^-110 to within 2^-134), at three times the matrix
 * work. Sums are fp32 in a fixed order.
 *
 * d_out >= 1, n >= 1; R == 0 enqueues nothing. Rows of X and dY may have any
 * alignment (16-byte aligned rows are faster). Fewer than 2^24 - 16 tiles of
 * 64 or 128 rows x 128 columns, E - 1 rows of tiles more than R needs.
 * Asynchronous. Workspace:
 * gptq_expert_matmul_workspace_bytes / gptq_expert_matmul_grad_workspace_bytes
 * (fp32 partial results when few tiles split the sum; 0 for most sizes).
 * ("El balance de errores de la inferencia de pocos bits", section 6: decode
 * and prefill are separate regimes of one dequantising product.) */
gptq_status gptq_expert_matmul_workspace_bytes(int64_t R, int64_t n, int64_t d_out, int64_t E, int32_t bits,
                                               int32_t group, size_t *bytes);
gptq_status gptq_expert_matmul(void *stream, const void *X, int32_t xdt, int64_t T, int64_t n, int64_t ldx,
                               const int32_t *rows, int64_t R, const int32_t *offsets, int64_t E,
                               const uint32_t *qweight, const float *scales, const uint8_t *zeros, int64_t d_out,
                               int32_t bits, int32_t group, void *Y, int32_t ydt, int64_t ldy, void *workspace,
                               size_t ws_bytes);
gptq_status gptq_expert_matmul_grad_workspace_bytes(int64_t R, int64_t n, int64_t d_out, int64_t E, int32_t bits,
                                                    int32_t group, size_t *bytes);
gptq_status gptq_expert_matmul_grad(void *stream, const void *dY, int32_t dydt, int64_t R, int64_t ldy,
                                    const int32_t *offsets, int64_t E, const uint32_t *qweight, const float *scales,
                                    const uint8_t *zeros, int64_t d_out, int64_t n, int32_t bits, int32_t group,
                                    void *dX, int32_t dxdt, int64_t ldx, void *workspace, size_t ws_bytes);

/* ---- Activations kept in 8 bits for the backward pass -------------------------
 * X (T x n, bf16 or fp32, row pitch ldx) is kept as codes (T x 32 ceil(n / 32)
 * int8, 16-byte aligned base, the columns past n zero) and exps (T x
 * ceil(n / 32) uint8), one byte per group of 32 columns of a row:
 *   exps = max(exponent field of max|x| - 6, 1) (fp32 fields: 127 is 1.0),
 *   step = 2^(exps - 127), code = clamp(rint(x / step), -127, 127),
 *   x_hat = code step.
 * With 2^p <= max|x| < 2^(p + 1) the step is 2^(p - 6): errors are at most
 * half a step, up to a whole one within half a step of 2^(p + 1). x_hat is
 * exact in bf16. A group with an infinity or NaN has exps = 255 and codes 0
 * and comes back as NaN. T ceil(n / 32) is at most 2^30 - 128.
 *
 * gptq_checkpoint_weight_grad: G (E x m x n fp32, contiguous) with
 * G[e] = sum over the rows p of segment e of P[p]^T x_hat[rows[p]] (P: R x m
 * bf16, row pitch ldp): the weight gradient of a linear layer (P = dY), or of
 * an adapter's input factor (P = dY B), from the kept input. offsets, rows
 * and E as above (one kept row per token serves its k places); an empty
 * segment's G is zero. Products are exact, sums fp32 in a fixed order. At
 * most 2^32 - 512 threads start at once: 256 for each 128 columns of 128 rows
 * of one G (of 32 or 64 where m is no more).
 * Workspace: gptq_checkpoint_weight_grad_workspace_bytes (fp32 partial sums
 * when few tiles split the rows). All asynchronous.
 * ("Resumen Técnico: GPTQ-intrinsic LoRA", "Declaración del Problema": the
 * low-rank factors beside the quantized layer, which tuning moves.) */
gptq_status gptq_checkpoint_save(void *stream, const void *X, int32_t dt, int64_t T, int64_t n, int64_t ldx,
                                 int8_t *codes, uint8_t *exps);
gptq_status gptq_checkpoint_restore(void *stream, const int8_t *codes, const uint8_t *exps, int64_t T, int64_t n,
                                    void *X, int32_t dt, int64_t ldx);
gptq_status gptq_checkpoint_weight_grad_workspace_bytes(int64_t R, int64_t E, int64_t m, int64_t n, size_t *bytes);
gptq_status gptq_checkpoint_weight_grad(void *stream, const void *P, int32_t pdt, int64_t R, int64_t m, int64_t ldp,
                                        const int8_t *codes, const uint8_t *exps, int64_t T, int64_t n,
                                        const int32_t *rows, const int32_t *offsets, int64_t E, float *G,
                                        void *workspace, size_t ws_bytes);

/* ---- Packed layers with bias, activation, gate and residual ---------------------
 * gptq_linear: the product of gptq_expert_matmul with what stands behind it in
 * a model, in the same launch: for the rows p of expert e
 *   z = X[rows[p]] W_hat_e^T + bias[e]                 (fp32)
 *   plain:  Y[p] = act(z) + residual[p]
 *   gated:  Y[p] = act(z[0 .. d)) * z[d .. 2 d) + residual[p]
 * d: columns of Y. A gated layer has 2 d packed rows an expert: those of the
 * gate, then those of the other factor (two layers quantized against the same
 * Hessian, one after the other, are one layer of 2 d rows). With m = d (2 d when
 * gated): qweight E x m x n*bits/32, scales and zeros E x m x n/group, bias
 * E x m fp32 or NULL, residual R x d (rdt, row pitch ldr) or NULL, Y R x d (ydt,
 * row pitch ldy), Z R x m (zdt, row pitch ldz) or NULL: where z is kept for
 * gptq_linear_grad. X, rows, offsets, E, R, bits, group and the kernels' numbers
 * are those of gptq_expert_matmul (its matrix-vector form serves up to 48 rows an
 * expert here); the epilogue is computed in fp32 and rounded once. E = 1 and
 * offsets NULL: one dense layer. Rows from offsets[E] on are neither read nor
 * written in any matrix. Y may be the residual (same type and pitch, refused
 * with others); no other output may overlap an input.
 *   act: GPTQ_ACT_NONE z; _RELU max(z, 0) (NaN stays NaN); _GELU z Phi(z);
 * _GELU_TANH z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2; _SILU z / (1 +
 * exp(-z)). Of minus infinity the last three are NaN.
 * Workspace: gptq_linear_workspace_bytes (fp32 partial results; 0 for most
 * sizes). m <= 2^31 - 65536. Asynchronous.
 *
 * gptq_linear_grad: from dY (R x d, dydt bf16 or fp32, row pitch ldy) and Z as
 * gptq_linear kept it (bf16 or fp32),
 *   plain:  dZ[p] = dY[p] act'(z);  gated:  dZ[p] = (dY u act'(g), dY act(g))
 *   dbias[e] = sum over the rows p of segment e of dZ[p]     (fp32, 0 if empty)
 *   dX[p] = dZ[p] W_hat_e                                    (R x n, dxdt)
 * dZ (R x m bf16, row pitch lddz) is rounded to bf16 once, which is what the
 * matrix product takes, and is also P of gptq_checkpoint_weight_grad; dbias sums
 * its values before that rounding, in a fixed order (NULL: not wanted; at most
 * 2^30 - 128 of them an expert). With GPTQ_ACT_NONE and no gate Z is not read
 * and may be NULL, and if dY is bf16 dZ may be NULL too (the product then takes
 * dY). The residual's gradient is dY, the gradient of X by token is gptq_combine
 * of dX. dX takes the weights as
 * gptq_expert_matmul_grad does: of two rounded factors, with a bf16 dX its error
 * is about 1.7 times what its own rounding gives (0.0029 against 0.0017 of it). An
 * fp32 dX takes the weights' whole 24 bits, at three times the work, but the same
 * dZ, whose one rounding is then its error (0.0017, 2^-8 of each term at most): it
 * is no fp32 gradient.
 * act' of relu is 0 at 0. dZ may be Z or, ungated, dY (bf16, same pitch; refused
 * with others).
 * Workspace: gptq_linear_grad_workspace_bytes. Asynchronous.
 * ("El balance de errores de la inferencia de pocos bits", section 6: what a
 * fused kernel saves is the traffic between its parts.) */
typedef enum {
  GPTQ_ACT_NONE = 0,
  GPTQ_ACT_RELU = 1,
  GPTQ_ACT_GELU = 2,
  GPTQ_ACT_GELU_TANH = 3,
  GPTQ_ACT_SILU = 4
} gptq_act;
gptq_status gptq_linear_workspace_bytes(int64_t R, int64_t n, int64_t d, int32_t gated, int64_t E, int32_t bits,
                                        int32_t group, size_t *bytes);
gptq_status gptq_linear(void *stream, const void *X, int32_t xdt, int64_t T, int64_t n, int64_t ldx,
                        const int32_t *rows, int64_t R, const int32_t *offsets, int64_t E, const uint32_t *qweight,
                        const float *scales, const uint8_t *zeros, const float *bias, int64_t d, int32_t bits,
                        int32_t group, int32_t act, int32_t gated, const void *residual, int32_t rdt, int64_t ldr,
                        void *Z, int32_t zdt, int64_t ldz, void *Y, int32_t ydt, int64_t ldy, void *workspace,
                        size_t ws_bytes);
gptq_status gptq_linear_grad_workspace_bytes(int64_t R, int64_t n, int64_t d, int32_t gated, int64_t E, int32_t bits,
                                             int32_t group, size_t *bytes);
gptq_status gptq_linear_grad(void *stream, const void *dY, int32_t dydt, int64_t ldy, const void *Z, int32_t zdt,
                             int64_t ldz, int64_t R, const int32_t *offsets, int64_t E, const uint32_t *qweight,
                             const float *scales, const uint8_t *zeros, int64_t d, int64_t n, int32_t bits,
                             int32_t group, int32_t act, int32_t gated, void *dZ, int64_t lddz, float *dbias, void *dX,
                             int32_t dxdt, int64_t ldx, void *workspace, size_t ws_bytes);

/* ---- A whole layer of experts for a few tokens ----------------------------------
 * gptq_expert_layer: for T tokens with k slots each, in two launches,
 *   h = end(up_e x_t + up_bias[e]),  e = expert_ids[t][j]
 *   Y[t] = residual[t] + sum_j weights[t k + j] (down_e h + down_bias[e])
 * with end(z) = act(z), or act(z[0 .. d)) * z[d .. 2 d) when gated, as in
 * gptq_linear. It is gptq_route, gptq_linear for both layers and gptq_combine
 * (plus the residual), for the tokens of a decoding step. X: T x n bf16, rows
 * 16-byte aligned (ldx % 8 == 0); expert_ids T x k int32, row pitch ldi; ids
 * outside [0, E) add nothing, a token without others gets its residual or 0;
 * an expert may stand more than once in a row. weights: T k fp32, or NULL for
 * ones. up: E layers of m = d (2 d when gated) rows of n codes, down: E layers
 * of n rows of d codes, both with `bits` and `group` (which divides n and d) in
 * the layout of gptq_dequant_matmul, 16-byte aligned; biases fp32 (E x m, E x n)
 * or NULL; residual T x n (rdt, row pitch ldr) or NULL; Y T x n (ydt, row pitch
 * ldy), which may be the residual (same type and pitch).
 * T k <= GPTQ_LAYER_MAX_SLOTS. n and d at most 2^20. More tokens are served by
 * the calls named above.
 * Numbers: both products as gptq_expert_matmul's matrix-vector form has them
 * (at 4 bits activations, and h, up to 2^116). h passes from one launch to the
 * other rounded to bf16 where Y is bf16 (as a bf16 model keeps it; the result's
 * error is then about 1.4 times what its own rounding gives), and in three bf16
 * pieces, which hold its fp32 value, where Y is fp32. Sums are fp32 in a
 * fixed order: results are bitwise reproducible.
 * Workspace: gptq_expert_layer_workspace_bytes. Asynchronous; T == 0 enqueues
 * nothing.
 * ("El balance de errores de la inferencia de pocos bits", section 6: decoding
 * pays for the traffic of the packed weights, and for every launch beside it.) */
#define GPTQ_LAYER_MAX_SLOTS 1024
gptq_status gptq_expert_layer_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t d, int32_t ydt,
                                              size_t *bytes);
gptq_status gptq_expert_layer(void *stream, const void *X, int32_t xdt, int64_t T, int64_t n, int64_t ldx,
                              const int32_t *expert_ids, int64_t ldi, int64_t k, const float *weights, int64_t E,
                              const uint32_t *up_qweight, const float *up_scales, const uint8_t *up_zeros,
                              const float *up_bias, const uint32_t *down_qweight, const float *down_scales,
                              const uint8_t *down_zeros, const float *down_bias, int64_t d, int32_t bits,
                              int32_t group, int32_t act, int32_t gated, const void *residual, int32_t rdt,
                              int64_t ldr, void *Y, int32_t ydt, int64_t ldy, void *workspace, size_t ws_bytes);

/* ---- Distillation from a teacher's top logits -----------------------------------
 * The loss that tuning a quantized model (its adapters, or the layers around
 * its packed weights) against the model before quantization minimises, from
 * the K entries per position that were kept of the teacher.
 *   s = Z[t] / temperature, lse[t] = log sum_v exp(s_v), q_v = exp(s_v - lse)
 *   p: log_probs == 0: softmax over the entries k of teacher[t] / temperature;
 *      log_probs == 1: p_k = exp(teacher[t][k]) as it is (their sum M may be
 *      below 1)
 *   loss[t] = sum_k p_k (log p_k - log q_{ids[t][k]})
 * Z: T x V (zdt bf16 or fp32, row pitch ldz); ids, teacher: T x K, int32 and
 * fp32, contiguous; loss, lse: T fp32. Entries whose id is outside [0, V) do not
 * count; a row without entries, or whose p are all 0 (padding), has loss 0 and
 * gradient 0. An entry with p = 0 adds nothing wherever its logit is. Logits of
 * -infinity (masked entries) have q = 0; a row of nothing else has lse = -infinity
 * and a loss of NaN, unless it is padding. NaN and +infinity make their row NaN.
 * 1 <= K <= GPTQ_DISTILL_MAX_K, V <= 2^31 - 65536, temperature positive and
 * finite, and log2(e) / temperature too. Everything is fp32, in an order that does
 * not depend on timing.
 *
 * gptq_distill_grad: for grad (T fp32: d total / d loss[t]) and lse as
 * gptq_distill gave it,
 *   dZ[t][v] = grad[t] / temperature (M q_v - sum over k with ids = v of p_k)
 * (T x V, dzdt bf16 or fp32, row pitch ldd; an id that stands more than once in
 * a row counts each time). dZ may be Z (same type and pitch). What fp32 rounds
 * off lse is relative in q: rows whose lse is beyond +-128 (2048 where dZ is
 * bf16) form their sum anew and read their logits twice, so that it stays below
 * 2^-18 (2^-14); a row of lowest values is the uniform distribution here as in
 * the loss. Neither needs a
 * workspace; both are asynchronous; T == 0 enqueues nothing. T may be at most 2^24 - 2.
 * ("Resumen Técnico: GPTQ-intrinsic LoRA", "Declaración del Problema": the
 * low-rank factors beside the quantized layer, which tuning moves.) */
#define GPTQ_DISTILL_MAX_K 1024
gptq_status gptq_distill(void *stream, const void *Z, int32_t zdt, int64_t T, int64_t V, int64_t ldz,
                         const int32_t *ids, const float *teacher, int64_t K, float temperature, int32_t log_probs,
                         float *loss, float *lse);
gptq_status gptq_distill_grad(void *stream, const void *Z, int32_t zdt, int64_t T, int64_t V, int64_t ldz,
                              const int32_t *ids, const float *teacher, int64_t K, float temperature,
                              int32_t log_probs, const float *lse, const float *grad, void *dZ, int32_t dzdt,
                              int64_t ldd);

/* ---- EoRA: rank-r compensation of the compression error ----------------------
 * B (d_out x rank fp32, row-major) and A (rank x n fp32, row-major) such that
 * W_hat + B A is the best rank-r correction of W_hat in the layer loss
 * tr((W - W_hat - B A) H (W - W_hat - B A)^T), and sigma (rank fp32,
 * descending) the singular values of the error projected into the
 * eigenspace of H. H == NULL: the plain SVD of W - W_hat (B = U_r Sigma_r,
 * A = V_r^T). W: d_out x n, dtype wdt, row stride ldw >= n; W_hat: d_out x n
 * fp32 (e.g. quantize_layer's w_hat); H: n x n fp32 symmetric (e.g. the
 * Hessian 2 X^T X). 1 <= rank <= min(64, d_out). The r largest eigenpairs of
 * D H D^T (D = W - W_hat) come from iters steps of block subspace iteration
 * (0: 24) on a block of min(rank + 64, 128) columns and a Rayleigh-Ritz
 * step; B A = U_r U_r^T D, B = U_r diag(sigma), A = diag(1/sigma) U_r^T D
 * (a zero sigma gives zero rows of A). Workspace:
 * gptq_eora_workspace_bytes(d_out, n, rank, H != NULL). Synchronises the
 * stream; GPTQ_ENONFINITE if W - W_hat or H is not finite.
 * ("Aumento de la precisión de LLM de 2 bits con EoRA" (7minutos.es), "Bucear
 * en el espacio propio en busca de un adaptador": the error projected by the
 * eigendecomposition of the activation covariance, truncated by SVD and
 * projected back; the plain-SVD adapter B = U Sigma, A = V^T beside it. Any
 * square root of H gives the same product B A as Q Lambda^{1/2}.) */
gptq_status gptq_eora_workspace_bytes(int64_t d_out, int64_t n, int32_t rank, int32_t with_h,
                                      size_t *bytes);
gptq_status gptq_eora(void *stream, const void *W, gptq_dtype wdt, const float *W_hat,
                      int64_t d_out, int64_t n, int64_t ldw, const float *H, int32_t rank,
                      int32_t iters, float *B, float *A, float *sigma, void *workspace,
                      size_t workspace_bytes);

/* ---- OLrC / Bid-Up refinement of a low-precision plus low-rank layer ---------
 * W ~ W_hat + B A with W_hat = s (q - z) the codes on a fixed grid: each of
 * `cycles` cycles first sets B (d_out x rank) and A (rank x n) to the best
 * rank-r correction of W - W_hat (OLrC: the computation of gptq_eora), then
 * runs `passes` Bid-Up passes over the codes for the target W - B A: the
 * columns in order, each code moved to the grid point nearest the minimiser
 * of tr((W - B A - W_hat) H (...)^T) along it, clamped to [0, 2^bits - 1]
 * (columns with H_jj <= 0 unchanged). Every step lowers or keeps the layer
 * error (up to fp32 rounding). codes: d_out x n uint8, in/out (e.g.
 * quantize_layer's codes); scales / zeros: d_out x (n / group) with g_idx (n
 * int32) mapping each column to its group, as quantize_layer writes them;
 * H: n x n fp32; W: d_out x n, dtype wdt, row stride ldw. Outputs B, A and,
 * if w_hat != NULL, the dequantised codes (d_out x n fp32). bits 2..8,
 * 1 <= rank <= min(64, d_out), cycles and passes 1..100. Workspace:
 * gptq_refine_workspace_bytes. Synchronises the stream.
 * ("Resumen Técnico: GPTQ-intrinsic LoRA", "Refinamiento Bid-Up": OLrC
 * optimises L and R for a fixed Q, Bid-Up optimises Q on the fixed grid by
 * coordinate updates; the alternation never increases the layer error.) */
gptq_status gptq_refine_workspace_bytes(int64_t d_out, int64_t n, int32_t rank, size_t *bytes);
gptq_status gptq_refine_lowrank(void *stream, const void *W, gptq_dtype wdt, int64_t d_out,
                                int64_t n, int64_t ldw, const float *H, int32_t bits,
                                int32_t group, const int32_t *g_idx, const float *scales,
                                const uint8_t *zeros, uint8_t *codes, int32_t rank,
                                int32_t cycles, int32_t passes, float *B, float *A,
                                float *w_hat, void *workspace, size_t workspace_bytes);

/* ---- Round-to-nearest on the same grid ---------------------------------------
 * codes (rows x cols uint8), scales / zeros (rows x cols/group fp32 / uint8)
 * and, if x_hat != NULL, x_hat = s (q - z) (rows x cols fp32) for X (rows x
 * cols fp32, row stride ldx): the quantizer's affine grid per group of
 * `group` consecutive columns of a row, with no error feedback. For the
 * low-rank factors of an adapter (B at 8 bits, A at 4 bits) and as the
 * round-to-nearest baseline. bits 2..8; group divides cols; rows <= 65535.
 * Asynchronous. ("Resumen Técnico: GPTQ-intrinsic LoRA", "Resultados
 * Clave": quantizing the low-rank factors L and R to 4 and 8 bits is often
 * lossless; "GPTQ", "Rendimiento y Precisión": round-to-nearest as the
 * baseline.) */
gptq_status gptq_quantize_rtn(void *stream, const float *X, int64_t rows, int64_t cols,
                              int64_t ldx, int32_t bits, int32_t group, uint8_t *codes,
                              float *scales, uint8_t *zeros, float *x_hat);

/* ---- Diagnostics ------------------------------------------------------------ */
const char *gptq_status_string(int status);
const char *gptq_last_error(void); /* thread-local detail of the last failure */

/* Timing with hipEvents recorded on the caller's stream: around the
 * Hessian Gram kernel, around the Hessian reduction, and around a whole
 * quantize_layer call (events are deliberately coarse: an event record
 * between every pair of small kernels costs microseconds of GPU time).
 * enable == 1 starts recording those (and clears what was recorded);
 * enable >= 2 also records the phases of quantize_layer: the factorisation
 * (preparation of H included), the W preparation and the final un-permute /
 * pack, every sweep launch (with its near-field update), every far-field
 * update, and every block product of the factorisation's inverse that runs
 * on the six-product bf16 kernel (the product alone, not its operand
 * splits; those products are also inside the factorisation's interval);
 * that adds a few microseconds per launch and is meant for one untimed
 * breakdown pass. The arrays given to gptq_profile_collect hold
 * GPTQ_PROF_NCLASSES entries. enable == 0 stops. gptq_profile_collect
 * synchronises the recorded events and returns, for class c in
 * [0, GPTQ_PROF_NCLASSES), the summed milliseconds and the number of timed
 * intervals, then clears. */
enum {
  GPTQ_PROF_HESSIAN_SYRK = 0,
  GPTQ_PROF_HESSIAN_REDUCE = 1,
  GPTQ_PROF_QUANTIZE = 2,
  GPTQ_PROF_FACTOR = 3,
  GPTQ_PROF_PREP_FINISH = 4,
  GPTQ_PROF_SWEEP = 5,
  GPTQ_PROF_FARFIELD = 6,
  GPTQ_PROF_INVERSE_X6 = 7,
  GPTQ_PROF_NCLASSES = 8
};
gptq_status gptq_profile_enable(int enable);
gptq_status gptq_profile_collect(double *ms, int64_t *count);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_MI355X_H */
