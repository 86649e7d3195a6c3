/*
 * GPTQ single-layer solver for AMD Instinct MI355X (gfx950): C ABI.
 *
 * The solver quantizes one linear layer's weights W (rows x d, d = input features) to low-bit
 * integer codes with a scale and zero point per group, pushing each column's rounding error onto the
 * columns not yet quantized through the Cholesky factor of the inverse Hessian of the layer's
 * calibration inputs X (tokens x d). The four calls below are its steps, in order:
 *
 *   gptq_hessian_accumulate  H += 2 X_c^T X_c for each token chunk X_c (gptq_hessian_compute:
 *                            H = 2 X_c^T X_c, for the first chunk)
 *   gptq_factor              damping, optional act-order, U = upper Cholesky factor of Hhat^-1
 *   gptq_quantize_layer      the column loop with lazy block updates; codes, scales, zeros, loss
 *   gptq_pack                eight 4-bit codes per 32-bit word (four 8-bit ones)
 *   gptq_pack_dense          the codes as one dense bit stream per row
 *   gptq_pack_ordered        the codes in a column order (act-order layers stored in processing order)
 *   gptq_permute_columns     inputs gathered by the same order
 *
 * the calls that use the stored layer:
 *
 *   gptq_dequant_gemm        y = x W^T for a few input rows, read straight from the packed codes
 *   gptq_lora_gemm           low-rank adapters of many requests added beside it
 *
 * and the attention half of a decoder block:
 *
 *   gptq_norm_rotate         per-head norm of queries and keys with the position rotation
 *   gptq_attention           attention over packed sequences: shared heads, masks, capped scores
 *
 * Sources (web pages on GPTQ): the GPTQ tools page at ozercemkelahmet.com ("How it works",
 * Steps 3-8, "Optional refinements", "A minimal Python sketch", "Memory arithmetic"); "GPTQ
 * Quantization: Complete Technical Guide" (notes.jayaprakash.net; "Quantization Equation",
 * "Computing the Hessian", "Damping Factor", "Configuration Deep Dive"); "Paper breakdown: GPTQ"
 * (ai360xpert.com; "How It Works", lazy batching); "What Is GPTQ?" (ai-tldr.dev; "How it works",
 * Step 3, groups).
 *
 * Conventions for every call:
 *   - Matrices are row-major. Pointers named as device memory must be device memory of the current
 *     HIP device; the caller allocates and owns every buffer and the library allocates no device
 *     memory. The only state it keeps: on first use on a device it creates two helper streams and a
 *     few events there (kept until the process ends), on which parts of a call run concurrently;
 *     and one static device array, the workspace of gptq_factor_noalloc.
 *   - `stream` is a hipStream_t (NULL: the default stream). Work is queued on it and the call returns
 *     without waiting, except gptq_factor, which waits once for its own work (see there). Work a call
 *     places on the helper streams starts after the work queued on `stream` before the call and
 *     ends before the call's later work on `stream`, so the call is ordered on `stream` as a whole.
 *   - Arguments are checked on the host before anything is queued. A rejected call returns a negative
 *     status and has no effect. HIP launch failures return GPTQ_EHIP.
 *   - Calls that share no output buffer may run concurrently on different streams.
 */
#ifndef GPTQ_H
#define GPTQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t gptq_status_t;

enum {
  GPTQ_OK = 0,
  GPTQ_EINVAL = -1,       /* invalid argument (null pointer, bad size, inconsistent settings)   */
  GPTQ_ENOTPD = -2,       /* damped Hessian not positive definite (see gptq_factor's info)      */
  GPTQ_EUNSUPPORTED = -3, /* a setting this library does not implement (e.g. block_size > 128)  */
  GPTQ_EHIP = -4,         /* a HIP runtime call or kernel launch failed                         */
  GPTQ_ENOMEM = -5        /* the workspace passed is smaller than gptq_workspace_bytes asks     */
};

/* Element types of W and X. */
enum { GPTQ_F32 = 0, GPTQ_F16 = 1, GPTQ_BF16 = 2 };

/* Storage layouts of packed codes (gptq_dequant_gemm's `layout`). */
enum {
  GPTQ_LAYOUT_FIELDS = 0, /* gptq_pack: a nibble per code up to 4 bits (8 per word), a byte above    */
  GPTQ_LAYOUT_DENSE = 1   /* gptq_pack_dense: exactly `bits` bits per code in one bit stream per row */
};

/* Workspace kinds for gptq_workspace_bytes. */
enum { GPTQ_WS_HESSIAN = 0, GPTQ_WS_FACTOR = 1, GPTQ_WS_QUANTIZE = 2 };

/* Quantization settings (the configuration surface of the Technical Guide's AutoGPTQ example:
 * bits, group_size, desc_act, damp_percent; the lazy-batch block size of the tools page, Step 7). */
typedef struct {
  int32_t bits;          /* code width, 2..8; codes are unsigned in [0, 2^bits - 1]             */
  int32_t group_size;    /* columns per group (>= 2); <= 0: one group per row. Groups and blocks
                            must nest: block_size % group_size == 0 or group_size % block_size == 0.
                            A group size of 1 is rejected (Technical Guide, "Don'ts").          */
  int32_t block_size;    /* lazy-batch width B, 1..128 (tools page, Step 7: "often 128")        */
  int32_t act_order;     /* 1: process columns by descending diag(H) (tools page, Act-order)     */
  int32_t sym;           /* 0: asymmetric min/max grid, zero = round(-wmin / scale); 1: symmetric
                            grid (tools page, "Optional refinements"): scale = max(2 max|w|, 1e-8)
                            / maxq and zero = 2^(bits-1), the middle code, so value = scale x
                            (code - zero) spans the Technical Guide's signed range [-8, 7] steps
                            at 4 bits. Codes stay unsigned in [0, 2^bits - 1].                  */
  int32_t static_groups; /* 0: a group's grid is taken from the current, error-updated weights
                            when the loop reaches the group's first column (groups are g
                            consecutive processing positions); 1: every grid is fixed before the
                            loop from the original weights of g consecutive original columns,
                            each column uses its original group's grid, and g_idx = k / g also
                            with act-order (the Technical Guide's static_groups setting).        */
  int32_t compact_meta;  /* 1: each grid is what a 16-bit scale and a zero of the code width store
                            (tools page, "Memory arithmetic"), and the loop quantizes with exactly
                            that: the scale rounded to the nearest float16 (the smallest positive
                            float16 if it would round to zero), the zero clamped to [0, maxq].
                            The fp32 scales and int32 zeros written then convert to that storage
                            without loss.                                                      */
  double damp;           /* relative damping >= 0: lambda = damp * mean(diag(H / n)) (Step 4)     */
} gptq_params_t;

/*
 * H += 2 * X^T X over one chunk of calibration tokens (GPTQ tools page, "How it works", Step 3;
 * Technical Guide, "Computing the Hessian": a sum of outer products of the layer inputs).
 *
 *   H      device float[d * d]. Accumulated in place; zero it before the first chunk. Only the
 *          upper triangle (i <= j) is authoritative; entries below the diagonal are left as they
 *          were, except inside 256 x 256 diagonal tiles, where they may take their part of the sum.
 *   d      number of input features, >= 1.
 *   X      device array [n_tok x ld_x] of x_dtype (GPTQ_F32, GPTQ_F16 or GPTQ_BF16), token-major:
 *          row t holds the d features of token t. Not modified. May be NULL when n_tok == 0.
 *   n_tok  tokens in this chunk, >= 0 (0: nothing is queued).
 *   ld_x   row pitch of X in elements, >= d.
 *   work   device workspace of work_bytes bytes, or NULL. With at least
 *          gptq_workspace_bytes(GPTQ_WS_HESSIAN, n_tok, d, NULL) bytes the token range is split
 *          across more workgroups (partial sums are added in token order); with less (or NULL) it
 *          is not split, which sums in another order (same float32 error bound) and may be slower.
 *          The workspace must not be shared with a concurrent call.
 * fp16 / bf16 products are exact in fp32; sums are fp32. The result does not depend on scheduling.
 */
gptq_status_t gptq_hessian_accumulate(float *H, int64_t d, const void *X, int32_t x_dtype, int64_t n_tok,
                                      int64_t ld_x, void *work, size_t work_bytes, void *stream);

/*
 * H = 2 * X^T X over one chunk of calibration tokens: gptq_hessian_accumulate for the first chunk,
 * without zeroing H first (the same source passages). Same arguments and errors as
 * gptq_hessian_accumulate. H's upper triangle (i <= j) is overwritten and H is not read; entries
 * below the diagonal are written inside 256 x 256 diagonal tiles only (their part of the sum, or
 * zero). With n_tok == 0 the whole of H is set to zero. The result is bit for bit that of zeroing H
 * and calling gptq_hessian_accumulate with the same chunk and workspace.
 */
gptq_status_t gptq_hessian_compute(float *H, int64_t d, const void *X, int32_t x_dtype, int64_t n_tok,
                                   int64_t ld_x, void *work, size_t work_bytes, void *stream);

/*
 * Damping, processing order and the upper Cholesky factor of the damped inverse Hessian
 * (GPTQ tools page, "How it works", Steps 4 and 6; "Optional refinements", Act-order).
 *
 *   H        device float[d * d], the accumulated sum of gptq_hessian_accumulate (upper triangle
 *            read). Not modified, unless U == H.
 *   n_total  number of tokens summed into H (> 0); Hhat = H / n_total + lambda I with
 *            lambda = p->damp * mean(diag(H / n_total)).
 *   p        settings; reads damp, act_order, sym, static_groups.
 *   U        device float[d * d], output: upper-triangular U with Hhat_perm^-1 = U^T U, in
 *            processing order (row/column j is original column perm[j]); zeros below the diagonal.
 *            Either U == H (the factor overwrites H in place, with no second d x d buffer) or the
 *            two do not overlap; a partial overlap is GPTQ_EINVAL.
 *   perm     device int32[d], output: the processing order. Identity without act-order; with it,
 *            columns by descending diag(H), equal values by lower index first.
 *   work     device workspace of at least gptq_workspace_bytes(GPTQ_WS_FACTOR, 0, d, p) bytes.
 *   info     host int64 output: 0 on success; k > 0 when the k-th pivot (1-based, in the reversed
 *            order the factorization runs in) was not positive (U is then unspecified).
 * This call waits for the stream once, to read the pivot check. Returns GPTQ_ENOTPD when info != 0
 * (damping "helps but does not fix" a rank-deficient Hessian: retry with a larger damp), GPTQ_EINVAL
 * when mean(diag(H)) is not positive and finite.
 */
gptq_status_t gptq_factor(const float *H, int64_t d, int64_t n_total, const gptq_params_t *p, float *U,
                          int32_t *perm, void *work, size_t work_bytes, int64_t *info, void *stream);

/*
 * gptq_factor for callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation. Same arguments, results and errors as
 * gptq_factor, without `work`: its workspace is a static device array inside the library (about
 * 25 MB, held on each device the library runs on until the process ends), and every launch goes to
 * `stream` (no helper stream or event is created). The call allocates nothing; the caller still
 * passes H, U and perm (U == H allowed, as for gptq_factor).
 *
 *   d  at most GPTQ_FACTOR_NOALLOC_MAX_D; larger d returns GPTQ_EUNSUPPORTED.
 *
 * All calls on one device share that device's array, and each call overwrites it: calls that
 * overlap on one device (on different streams or host threads) race. Like gptq_factor, the call
 * waits for the stream once to read the pivot check.
 */
#define GPTQ_FACTOR_NOALLOC_MAX_D 12288
gptq_status_t gptq_factor_noalloc(const float *H, int64_t d, int64_t n_total, const gptq_params_t *p, float *U,
                                  int32_t *perm, int64_t *info, void *stream);

/*
 * The GPTQ column loop for one layer (GPTQ tools page, "How it works", Steps 5, 7 and 8; the
 * Technical Guide's "Quantization Equation" grid; "What Is GPTQ?", Step 3 groups).
 *
 *   W       device array [rows x ld_w] of w_dtype (GPTQ_F32, GPTQ_F16 or GPTQ_BF16), original column
 *           order. Not modified.
 *   rows    output features, >= 0 (0: only g_idx is written and loss is set to 0).
 *   d       input features, >= 1; ld_w >= d.
 *   U, perm from gptq_factor with the same d and act_order.
 *   p       settings; reads bits, group_size, block_size, sym, static_groups.
 *   codes   device uint8[rows * d], output: codes in [0, 2^bits - 1], original column order.
 *   scales  device float[rows * ngroups], zeros device int32[rows * ngroups], output, with
 *           ngroups = ceil(d / g) and g = group_size (d when group_size <= 0). Group j of a row
 *           covers processing positions [j g, (j+1) g), or original columns [j g, (j+1) g) with
 *           static_groups; dequantized value = scale * (code - zero).
 *   g_idx   device int32[d], output: the group of each original column.
 *   loss    device double[1], output: the sum over rows and columns of err^2, where err is a
 *           column's rounding error divided by the factor's diagonal entry; it equals
 *           sum_r (W - Q)_r Hhat (W - Q)_r^T (the damped layer objective, tools page Step 2).
 *   work    device workspace of at least gptq_workspace_bytes(GPTQ_WS_QUANTIZE, rows, d, p) bytes.
 * Rounding is to nearest, ties to even; the rounding ratios are taken in fp32 with correctly rounded
 * division. Rows are independent: splitting W by rows over calls gives the same results.
 */
gptq_status_t gptq_quantize_layer(const void *W, int32_t w_dtype, int64_t rows, int64_t d, int64_t ld_w,
                                  const float *U, const int32_t *perm, const gptq_params_t *p, uint8_t *codes,
                                  float *scales, int32_t *zeros, int32_t *g_idx, double *loss, void *work,
                                  size_t work_bytes, void *stream);

/*
 * gptq_quantize_layer with a breakdown of where its device time goes (measurement: the same work
 * and results, plus events recorded between its launches). Same arguments, plus:
 *   part_ms  host double[3], output: device milliseconds of the column-loop kernels (the in-block
 *            chain with the lazy updates inside each super-block of up to 512 columns), of the lazy
 *            products that carry each super-block's errors to the later columns (fp32 MFMA GEMMs),
 *            and of the rest (working copy, indices, un-permute, loss). NULL is GPTQ_EINVAL.
 * Unlike gptq_quantize_layer it waits for the stream before returning.
 */
gptq_status_t gptq_quantize_layer_timed(const void *W, int32_t w_dtype, int64_t rows, int64_t d, int64_t ld_w,
                                        const float *U, const int32_t *perm, const gptq_params_t *p, uint8_t *codes,
                                        float *scales, int32_t *zeros, int32_t *g_idx, double *loss, void *work,
                                        size_t work_bytes, double *part_ms, void *stream);

/*
 * Packs codes in fixed fields along the columns (GPTQ tools page, "How it works", Step 8: eight 4-bit
 * codes per 32-bit word): a nibble per code for bits 1..4, a byte per code for bits 5..8.
 *
 *   codes   device uint8[rows * d]; every code must be < 2^bits (bits above the field are dropped).
 *   rows    >= 0; d >= 8 and a multiple of 8; bits in 1..8 (3-bit codes also take a nibble).
 *   packed  device int32[rows * d * f / 32], output, f = 4 or 8: bits f t .. f t + f - 1 of word k of
 *           a row hold column (32 / f) k + t.
 */
gptq_status_t gptq_pack(const uint8_t *codes, int64_t rows, int64_t d, int32_t bits, int32_t *packed,
                        void *stream);

/*
 * Packs codes as one dense bit stream per row, exactly `bits` bits per code, so 3-bit codes take 3
 * bits, not a nibble (the tools page's "Memory arithmetic": storage follows the bit width). At 4 and
 * 8 bits the words equal gptq_pack's.
 *
 *   codes   device uint8[rows * d]; every code must be < 2^bits (higher bits are dropped).
 *   rows    >= 0; d >= 1 with d * bits a multiple of 32; bits in 1..8.
 *   packed  device int32[rows * d * bits / 32], output: code k of a row occupies stream bits
 *           bits k .. bits k + bits - 1, and stream bit t is bit t % 32 of word t / 32 of the row.
 */
gptq_status_t gptq_pack_dense(const uint8_t *codes, int64_t rows, int64_t d, int32_t bits, int32_t *packed,
                              void *stream);

/*
 * Packs the codes in a given column order, in gptq_pack's field layout: column j of the output is
 * column order[j] of the codes. With order = gptq_factor's perm (the act-order processing order), a
 * group's columns are contiguous again (group j / g), so gptq_dequant_gemm can take its fast kernels
 * with g_idx = NULL on inputs gathered by the same order (gptq_permute_columns). The product is the
 * same sum taken in another order. This is the act-order trade-off of the tools page ("Optional
 * refinements"; What Is GPTQ, kernel speed) paid once at storage time instead of in every product.
 *
 *   codes   device uint8[rows * d], original column order (gptq_quantize_layer's codes).
 *   rows    >= 0; d >= 8 and a multiple of 8; bits in 1..8.
 *   order   device int32[d], a permutation of 0..d-1 (values outside [0, d) are clamped into it).
 *   packed  device int32[rows * d * f / 32], output, f = 4 for bits <= 4 and 8 above.
 */
gptq_status_t gptq_pack_ordered(const uint8_t *codes, int64_t rows, int64_t d, int32_t bits, const int32_t *order,
                                int32_t *packed, void *stream);

/*
 * Gathers the columns of a row-major matrix: out[i][j] = in[i][order[j]] (the layer inputs in the
 * order of codes packed by gptq_pack_ordered).
 *
 *   in      device array [m x ld_in] of dtype (GPTQ_F32, GPTQ_F16 or GPTQ_BF16). Not modified.
 *   m       rows, >= 0 (0: nothing is queued); d columns, >= 1; ld_in, ld_out >= d.
 *   order   device int32[d] (values outside [0, d) are clamped into it).
 *   out     device array [m x ld_out] of dtype, output; must not overlap `in`.
 */
gptq_status_t gptq_permute_columns(const void *in, int32_t dtype, int64_t m, int64_t d, int64_t ld_in,
                                   const int32_t *order, void *out, int64_t ld_out, void *stream);

/*
 * The stored layer at inference: y = x W^T for a few rows of inputs x, with W expanded from the packed
 * codes, scales and zeros inside the kernel (GPTQ tools page, "How it works", Step 8: a fused kernel
 * unpacks, scales and multiplies; "What Is GPTQ?", "How it works", Step 3: each group is expanded
 * back to higher precision just in time for the product). Small-batch products like this are bound
 * by reading the weights, about half a byte per weight here.
 *
 *   x       device array [m x ld_x] of x_dtype (GPTQ_F32, GPTQ_F16 or GPTQ_BF16): one row per token,
 *           d features each. Not modified.
 *   m       input rows, >= 0 (0: nothing is queued). Rows are taken eight at a time, and each group
 *           of eight reads the codes once.
 *   ld_x    row pitch of x in elements, >= d.
 *   packed  device int32 codes of rows x d weights in `layout`: GPTQ_LAYOUT_FIELDS is gptq_pack's
 *           (rows * d / 8 words of nibbles for bits <= 4, rows * d / 4 words of bytes above),
 *           GPTQ_LAYOUT_DENSE is gptq_pack_dense's (rows * d * bits / 32 words; d * bits must be
 *           a multiple of 32). Not modified.
 *   bits    the code width, 1..8.
 *   layout  GPTQ_LAYOUT_FIELDS or GPTQ_LAYOUT_DENSE.
 *   scales  device float[rows * ngroups] and zeros device int32[rows * ngroups], as
 *           gptq_quantize_layer writes them, with ngroups = ceil(d / g) and g = group_size (d when
 *           group_size <= 0).
 *   g_idx   device int32[d], the group of each column (gptq_quantize_layer's g_idx, needed after
 *           act-order), or NULL when column k is in group k / g. Entries outside [0, ngroups) are
 *           clamped into it.
 *   rows    weight rows (outputs), >= 0 (0: nothing is queued); d input columns, >= 8, a multiple
 *           of 8.
 *   y       device float[m x ld_y], output, ld_y >= rows: y[i, r] = sum_k x[i, k] W[r, k] with
 *           W[r, k] = scales[r, G] * (code[r, k] - zeros[r, G]) and G the group of column k.
 * Products and sums are fp32 (fp16 x times a code is exact in fp32). Faster kernels run for nibble
 * fields when x is fp16, g_idx is NULL, g is a multiple of 32 or at least d, d is a multiple of 32,
 * and the rows of x and the codes are 16-byte aligned (for 3 or more input rows also g a multiple of
 * 128 and d of 128); otherwise a general one does. Results do not depend on scheduling.
 */
gptq_status_t gptq_dequant_gemm(const void *x, int32_t x_dtype, int64_t m, int64_t ld_x, const int32_t *packed,
                                int32_t bits, int32_t layout, const float *scales, const int32_t *zeros,
                                const int32_t *g_idx, int64_t rows, int64_t d, int32_t group_size, float *y,
                                int64_t ld_y, void *stream);

/*
 * Low-rank adapters of many requests beside a shared projection (the stored layer's product, or any
 * other): row i of x names adapter a = index[i], and
 *   y[i, r] = base[i, r] + scales[a] * sum_k T[i, k] B_a[r, k],   T[i, k] = sum_c x[i, c] A_a[k, c].
 * A row whose index is outside [0, adapters) has no adapter: y[i] = base[i].
 *
 *   x        device array [m x ld_x] of dtype (GPTQ_F32, GPTQ_F16 or GPTQ_BF16), d features a row.
 *            Not modified.
 *   m        input rows, >= 0 (0: nothing is queued); ld_x >= d.
 *   A, B     device arrays of dtype: A [adapters x rank x d], B [adapters x rows x rank], contiguous.
 *   ranks    device int32[adapters], the rank each adapter uses (clamped to [0, rank]; what A's rows and
 *            B's columns hold beyond it takes no part), or NULL: every adapter uses `rank`.
 *   scales   device float[adapters], or NULL: 1.
 *   adapters >= 0; rank 1..256.
 *   index    device int32[m], in any order; rows may share an adapter.
 *   rows     outputs, 0..2^24 (0: nothing is queued); d input features, >= 1.
 *   base     device float[m x ld_base], ld_base >= rows, or NULL: zeros. May be y itself with the same
 *            pitch (added in place), or not overlap it; another overlap is GPTQ_EINVAL.
 *   y        device float[m x ld_y], output, ld_y >= rows. Must not overlap the other arrays.
 *   work     device workspace of at least gptq_lora_workspace_bytes(m, d, rows, adapters, rank) bytes,
 *            not shared with a concurrent call; 16-byte aligned.
 * Products of x and A are exact in fp32 (fp16 and bf16), T and all sums are fp32. Results do not depend
 * on scheduling. Launches on `stream` alone; the call may be captured in a graph.
 */
gptq_status_t gptq_lora_gemm(const void *x, int32_t dtype, int64_t m, int64_t ld_x, const void *A, const void *B,
                             const int32_t *ranks, const float *scales, int64_t adapters, int32_t rank,
                             const int32_t *index, int64_t rows, int64_t d, const float *base, int64_t ld_base,
                             float *y, int64_t ld_y, void *work, size_t work_bytes, void *stream);

/* Workspace bytes for gptq_lora_gemm; 0 for invalid arguments (or m, rows or adapters of 0). */
size_t gptq_lora_workspace_bytes(int64_t m, int64_t d, int64_t rows, int64_t adapters, int32_t rank);

/*
 * Sizes and strides of gptq_norm_rotate. Element (t, h, c) of a tensor x is at t * x_ld + h * x_hp + c:
 * x_ld is the pitch of tokens, x_hp the pitch of heads (head_dim for heads side by side).
 */
typedef struct {
  int64_t n;          /* tokens, >= 0 (0: nothing is queued)                                      */
  int64_t q_ld, q_hp, k_ld, k_hp;                    /* pitches of q and k                        */
  int64_t q_out_ld, q_out_hp, k_out_ld, k_out_hp;    /* pitches of the outputs                    */
  double eps;         /* norm's epsilon, >= 0                                                     */
  int32_t dtype;      /* of q, k and the outputs: GPTQ_F32, GPTQ_F16 or GPTQ_BF16                 */
  int32_t w_dtype;    /* of the norm's weights                                                    */
  int32_t q_heads;    /* 1..65535                                                                 */
  int32_t k_heads;    /* 0..65535 (0: k and k_out are not used)                                   */
  int32_t head_dim;   /* 1..1024                                                                  */
  int32_t rotary_dim; /* rotated columns of each head: even, 0..head_dim (0: no rotation)         */
  int32_t interleaved; /* 0: pair i is columns i and i + rotary_dim / 2; 1: columns 2i and 2i + 1 */
  int32_t axes;       /* rows of positions, 1..64 (time, height, width: 3)                        */
  int32_t norm;       /* 1: each head is divided by the root of its mean square (plus eps); 0: not */
} gptq_norm_rotate_t;

/*
 * Per-head norm of queries and keys and their position rotation in one pass. For each head x of each
 * token: y = x / sqrt(mean(x^2) + eps), times its weights (norm = 0: y = x), and pair i of the first
 * rotary_dim columns, (a, b), becomes (a cos t - b sin t, b cos t + a sin t) with the angle
 * t = positions[axis of pair i][token] * inv_freq[i].
 *
 *   q, k          device arrays, not modified (k is not used with k_heads = 0).
 *   q_weight      device array of w_dtype [head_dim] (k_weight the same), or NULL: ones. With norm = 0
 *                 both must be NULL.
 *   positions     device int32[axes * n], any values; inv_freq device float[rotary_dim / 2].
 *   pair_axis     device int32[rotary_dim / 2], the row of positions each pair takes (clamped into
 *                 [0, axes)), or NULL: row 0. positions, inv_freq and pair_axis are not used with
 *                 rotary_dim = 0.
 *   q_out, k_out  device arrays, output; each may be its input itself with the same pitches (in place).
 *                 Otherwise its address range must be apart from those of q, k and the other output, or
 *                 both be column ranges of one array with one token pitch that do not meet; anything
 *                 else is GPTQ_EINVAL. Heads and tokens of an output must not overlap.
 * The angle is formed in 64 bits, so far positions lose nothing; sums and products are fp32, rounded
 * once to dtype. Finite heads of any size are normed (squares that leave fp32's range are scaled).
 * 16-byte accesses are used where columns, pitches and pointers allow them.
 */
gptq_status_t gptq_norm_rotate(const gptq_norm_rotate_t *a, const void *q, const void *k, const void *q_weight,
                               const void *k_weight, const int32_t *positions, const float *inv_freq,
                               const int32_t *pair_axis, void *q_out, void *k_out, void *stream);

/* Sizes, strides and settings of gptq_attention; pitches as in gptq_norm_rotate_t. */
typedef struct {
  int64_t seqs;       /* sequences, >= 0 (0: nothing is queued)                                   */
  int64_t n_q, n_kv;  /* rows of q and out, rows of k and v; 0..2^30                              */
  int64_t q_ld, q_hp, k_ld, k_hp, v_ld, v_hp, out_ld, out_hp;
  double scale;       /* score scale, finite in fp32 (1 / sqrt(head_dim) as a rule)               */
  double softcap;     /* c >= 1e-37: scores become c tanh(score / c); 0: no cap                   */
  int32_t dtype;      /* of q, k, v and out: GPTQ_F32, GPTQ_F16 or GPTQ_BF16                      */
  int32_t q_heads;    /* 1..65535                                                                 */
  int32_t kv_heads;   /* 1..65535, dividing q_heads: query head h reads head h / (q_heads / kv_heads) */
  int32_t head_dim;   /* 1..1024                                                                  */
  int32_t causal;     /* 1: a query sees the keys up to its own position; 0: all of its sequence's */
} gptq_attention_t;

/*
 * Softmax attention over packed sequences. Sequence s holds rows [q_start[s], q_start[s + 1]) of q and
 * rows [kv_start[s], kv_start[s + 1]) of k and v, lq and lk of them. Its queries are its last tokens:
 * query i has position p = i + lk - lq (one new token against a cache: lq = 1). For key j of the same
 * sequence:
 *   score = scale * q . k_j, capped (softcap), minus slopes[head] * |p - j|
 *   seen  = (j <= p, or j < prefix[s], or causal = 0), and, with documents, q_doc = kv_doc[j] >= 0
 *   out   = sum of v_j exp(score) / sum of exp(score) over the keys that are seen
 * A query that sees no key gets zeros. A key that is not seen takes no part, whatever k and v hold there
 * (infinities and NaN included). Rows of out that belong to no sequence are left as they were.
 *
 *   q, k, v        device arrays, not modified (k and v may be NULL with n_kv = 0).
 *   q_start        device int32[seqs + 1], ascending, or NULL: seqs equal ranges (n_q a multiple of seqs);
 *   kv_start       the same for k and v. Values are clamped so that every access stays inside n_q and
 *                  n_kv rows. Key ranges may overlap; query ranges must not.
 *   slopes         device float[q_heads], or NULL: no distance bias.
 *   q_doc, kv_doc  device int32[n_q] and int32[n_kv], documents of queries and keys in any order, or both
 *                  NULL. A negative document (padding) sees nothing and is not seen.
 *   prefix         device int32[seqs]: the first prefix[s] keys are seen by every query of the sequence
 *                  (with causal = 1; it changes nothing otherwise), or NULL.
 *   out            device array, output; apart from q, k and v as in gptq_norm_rotate (not in place), its
 *                  heads and tokens from each other.
 *   work           device workspace of work_bytes bytes (16-byte aligned), or NULL. With at least
 *                  gptq_attention_workspace_bytes(a) bytes, long key ranges are split across workgroups
 *                  when there are few queries and joined in key order; with less (or NULL) they are not.
 *                  It must not be shared with a concurrent call, two captured graphs included.
 * Scores, the softmax's maximum and sum and the output's sums are fp32, but for two roundings with fp16 and bf16
 * (neither is made with fp32 inputs, nor for head_dim > 256):
 *   - each probability is rounded once to the type before it weighs a value, which moves the output by at most
 *     half a step (fp16 2^-11, bf16 2^-8) of sum p |v|, beside the result's own half step. The probabilities' sum is
 *     of the unrounded ones. Random inputs: 2.4e-4..2.9e-4 off in norm in fp16, 2.1e-3 in bf16 (2.1e-4 and 1.6e-3
 *     for the result's rounding alone).
 *   - with a softcap c up to 256, a capped score is up to 2^-22 c off (6e-5 at 256).
 * Results do not depend on scheduling. Finite values give finite averages (within fp32 roundings of its largest
 * number they may round to infinity). Rows that see infinities or NaN, or whose tiles of keys hold some that they do
 * not see, are right, but computed one by one, as are rows whose weighted sum passes fp32's range: hundreds of
 * times slower (2 x 2048 bf16 tokens, 32 query heads: 29 ms instead of 0.1 with NaN in every padding key and value).
 * Padding is best kept finite.
 * Returns GPTQ_EUNSUPPORTED, before anything is queued, when head_dim <= 256 and
 * (n_q * (q_heads / kv_heads) / 128 + seqs) * kv_heads >= 2^24 (tiles of 128 rows; one launch takes all of them).
 */
gptq_status_t gptq_attention(const gptq_attention_t *a, const void *q, const void *k, const void *v,
                             const int32_t *q_start, const int32_t *kv_start, const float *slopes,
                             const int32_t *q_doc, const int32_t *kv_doc, const int32_t *prefix, void *out, void *work,
                             size_t work_bytes, void *stream);

/* Workspace bytes with which gptq_attention splits key ranges; 0 when it would not (or for invalid arguments). */
size_t gptq_attention_workspace_bytes(const gptq_attention_t *a);

/*
 * One pre-norm decoder block for gptq_quantize_block. The pages fix the order in which a block's
 * layers are solved but not the block itself; this one is RMSNorm -> multi-head causal
 * self-attention (q, k, v, o; no positional rotation) -> residual -> RMSNorm -> SiLU-gated MLP
 * (gate, up, down) -> residual, with no learned norm weights.
 */
typedef struct {
  int64_t hidden;   /* model width, >= 8; q, k, v, o are hidden x hidden                          */
  int64_t heads;    /* attention heads, 1..65535, dividing hidden; heads * seq_len <= 2^31        */
  int64_t inter;    /* MLP width, >= 8; gate and up are inter x hidden, down hidden x inter       */
  int64_t seqs;     /* calibration sequences, >= 1                                                */
  int64_t seq_len;  /* tokens per sequence, >= 1; attention is causal within each sequence        */
  double eps;       /* RMSNorm epsilon, >= 0: y = x / sqrt(mean(x^2) + eps) over each token's row  */
} gptq_block_shape_t;

/* One layer of the block: its weights in, its gptq_quantize_layer outputs out. */
typedef struct {
  const void *W;    /* device [rows x d] of w_dtype, row-major with ld = d; not modified          */
  uint8_t *codes;   /* device uint8[rows x d], original column order                              */
  float *scales;    /* device float[rows x ngroups]                                               */
  int32_t *zeros;   /* device int32[rows x ngroups]                                               */
  int32_t *g_idx;   /* device int32[d]                                                            */
  int32_t *perm;    /* device int32[d]: the processing order used (shared within a stage)         */
  double *loss;     /* device double[1]                                                           */
  int32_t w_dtype;  /* GPTQ_F32, GPTQ_F16 or GPTQ_BF16                                            */
} gptq_block_layer_t;

/* Workspace bytes for gptq_quantize_block (p->block_size is read); 0 for invalid arguments. */
size_t gptq_block_workspace_bytes(const gptq_block_shape_t *shape, const gptq_params_t *p);

/*
 * Quantizes the seven linear layers of one decoder block in the true-sequential order (GPTQ tools
 * page, "How it works", Step 9; the Technical Guide's "true_sequential" setting):
 *   stage 0: q, k, v from the Hessian of the attention input RMSNorm(X);
 *   stage 1: o from the Hessian of the attention output, recomputed through the quantized q, k, v;
 *   stage 2: gate, up from the MLP input RMSNorm(X + attn o^T), through the quantized o;
 *   stage 3: down from silu(x gate^T) * (x up^T), through the quantized gate and up.
 * Each stage forms H = 2 A^T A over all tokens, factors it once (gptq_factor) and runs
 * gptq_quantize_layer for each of its layers with that factor and order. With true_sequential = 0
 * every stage input comes from the block with its original weights (the layers are solved from
 * one unquantized forward pass). Activations are fp32. The projections and each stage's H run on
 * the fp16 matrix cores from operands split into two fp16 halves (hi + lo equals an fp32 value to
 * within 2^-22 relative; weights are scaled by a power of two first), which matches fp32 products
 * to within about their inputs' rounding. Stage inputs must stay below 65504 in magnitude (beyond
 * it H is not finite and the stage's factor fails).
 *
 *   shape   the block and calibration sizes (n = seqs * seq_len tokens).
 *   X       device [n x hidden] of x_dtype, token-major, sequence after sequence. Not modified.
 *   p       the quantization settings of every layer (as gptq_quantize_layer).
 *   layers  host array of 7 descriptors, in the order q, k, v, o, gate, up, down.
 *   Y       device float[n x hidden]: the block output through the quantized weights (the input
 *           of the next block).
 *   hess    NULL, or a host array of 4 pointers (each NULL or device float[d x d] for that stage's
 *           input width d): receives each stage's H (upper triangle authoritative).
 *   work    device workspace of gptq_block_workspace_bytes(shape, p) bytes.
 *   info    host int64[2]: on GPTQ_ENOTPD the failed stage (0..3) and pivot; otherwise {-1, 0}.
 *   stream  HIP stream; the call synchronizes it once per stage (to read each factor's status) and
 *           once per projection (to read the weight's scale): 11 times with true_sequential, 18
 *           without.
 * Returns GPTQ_EINVAL for bad shapes, pointers or settings, GPTQ_ENOMEM for a short workspace,
 * GPTQ_ENOTPD (see info) when a stage's damped Hessian is not positive definite, and the statuses
 * of the calls it makes. Outputs of later stages are undefined after an error.
 */
gptq_status_t gptq_quantize_block(const gptq_block_shape_t *shape, const void *X, int32_t x_dtype,
                                  const gptq_params_t *p, int32_t true_sequential, const gptq_block_layer_t *layers,
                                  float *Y, float *const *hess, void *work, size_t work_bytes, int64_t *info,
                                  void *stream);

/*
 * The attention of a block whose model has more than gptq_quantize_block's: key heads shared by several
 * query heads, a norm of each query and key head, a rotation by position, capped or distance-biased
 * scores, several documents in a sequence, a prefix. Fields as in gptq_norm_rotate_t and gptq_attention_t;
 * head_dim is hidden / heads (at most 1024), and positions, doc and prefix go by the block's tokens and
 * sequences (n = seqs * seq_len).
 */
typedef struct {
  int64_t kv_heads;          /* dividing heads; k and v are (kv_heads * head_dim) x hidden            */
  const void *q_norm;        /* device w_dtype[head_dim] or NULL (ones); only with qk_norm            */
  const void *k_norm;        /* the same for keys                                                     */
  const float *inv_freq;     /* device float[rotary_dim / 2]; with rotary_dim > 0                     */
  const int32_t *positions;  /* device int32[axes * n]; with rotary_dim > 0                           */
  const int32_t *pair_axis;  /* device int32[rotary_dim / 2] or NULL                                  */
  const float *slopes;       /* device float[heads] or NULL                                           */
  const int32_t *doc;        /* device int32[n] or NULL; negative: padding                            */
  const int32_t *prefix;     /* device int32[seqs] or NULL                                            */
  double norm_eps;           /* epsilon of the head norm, >= 0                                        */
  double scale;              /* score scale; 0: 1 / sqrt(head_dim)                                    */
  double softcap;            /* 0: none                                                               */
  int32_t qk_norm;           /* 1: each query and key head is normed                                  */
  int32_t w_dtype;           /* of q_norm and k_norm                                                  */
  int32_t rotary_dim;        /* 0: no rotation                                                        */
  int32_t interleaved;
  int32_t axes;
  int32_t causal;
} gptq_block_attn_t;

/* Workspace bytes for gptq_quantize_block_attn; 0 for invalid arguments, and for more rows than gptq_attention
 * takes (the call itself returns GPTQ_EUNSUPPORTED for them). */
size_t gptq_block_attn_workspace_bytes(const gptq_block_shape_t *shape, const gptq_block_attn_t *attn,
                                       const gptq_params_t *p);

/*
 * gptq_quantize_block with the attention `attn` describes: after the projections, q and k go through
 * gptq_norm_rotate and then, with v, through gptq_attention, in fp32. The other arguments, the order of
 * the solves, the waits and the errors are gptq_quantize_block's; layers k and v have
 * kv_heads * head_dim rows. work: gptq_block_attn_workspace_bytes(shape, attn, p) bytes.
 */
gptq_status_t gptq_quantize_block_attn(const gptq_block_shape_t *shape, const gptq_block_attn_t *attn, const void *X,
                                       int32_t x_dtype, const gptq_params_t *p, int32_t true_sequential,
                                       const gptq_block_layer_t *layers, float *Y, float *const *hess, void *work,
                                       size_t work_bytes, int64_t *info, void *stream);

/*
 * Workspace bytes for a call: kind GPTQ_WS_HESSIAN (a = n_tok of the chunk), GPTQ_WS_FACTOR (a unused)
 * or GPTQ_WS_QUANTIZE (a = rows; p->block_size is read). Returns 0 for invalid arguments.
 */
size_t gptq_workspace_bytes(int32_t kind, int64_t a, int64_t d, const gptq_params_t *p);

/* A static, human-readable name for a status code. */
const char *gptq_status_string(gptq_status_t s);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_H */
