/*
 * lh.h - C ABI of the Local-Hessian NVFP4 weight-scale calibration library
 *        (liblh.so, HIP kernels for AMD Instinct MI355X / gfx950).
 *
 * The method (pages cited by title and section):
 *   "Local-Hessian weight-scale guide" (xxmr.cn/news/266017)
 *     - "What is Local-Hessian": NVFP4 stores FP4 E2M1 values, 16 weights
 *       share one FP8 E4M3 block scale, a block scale maps the block into
 *       the E2M1 range [-6, 6]; the scale sweep tries all 126 positive
 *       non-zero FP8 values.
 *     - "Algorithm principle": linear layer Y = W X with W [C_out x C_in]
 *       and calibration input X [C_in x N]; Q(W, s) = Cast(W / s) * s,
 *       Delta = Q - W; output error E(s) = ||Delta X||_F^2 =
 *       tr(Delta X X^T Delta^T); block-diagonal approximation per 16-weight
 *       block b: E_b(s_b) = Delta_b (X_b X_b^T) Delta_b^T; the sweep kernel
 *       takes weights [N_BLOCKS, 16] in (cout, cin // 16) order, the global
 *       FP32 amax and per-block Hessians [cin // 16, 16, 16], minimises
 *       dw^T H dw over the 126 E4M3 candidates and outputs the per-block
 *       best amax; candidate generation is bit-consistent with fake-quant.
 *     - "Entry API and calibration flow", phase 2: H accumulates the sum of
 *       X^T X over calibration batches; phase 3 passes the normalised
 *       per-block Hessian to the search.
 *     - "Combining with GPTQ": the cast rounds to nearest (RTN).
 *   "ModelOpt overview" (linlog.top/article/1517), "Local-Hessian": 126
 *     candidate scales per block, each block optimised independently.
 *
 * Readings taken where the pages leave a step open:
 *   - candidates: the 126 positive finite OCP E4M3FN values (codes
 *     0x01..0x7E, max 448); candidate index k <-> E4M3 code k + 1;
 *   - S_g = fl32(g / 2688) (2688 = 6 * 448), s_k = fl32(c_k * S_g);
 *   - Cast: x = fl32(|w| / s_k) (IEEE division), nearest E2M1 magnitude
 *     {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, saturation at 6;
 *     Q = fl32(sign(w) * r * s_k), -0 written as +0; s_k = 0 gives Q = 0;
 *   - "normalised" = divided by the token count N (alpha = 1 / N);
 *   - equal errors resolve to the lowest candidate index.
 *
 * Conventions for every entry point:
 *   - all data pointers are DEVICE pointers (hipMalloc'd or a framework's
 *     device tensor); the caller owns and frees every buffer;
 *   - `stream` is a hipStream_t passed as void* (NULL = default stream);
 *     every call only enqueues work on it and returns; the library never
 *     synchronises the device, never allocates, keeps no state between
 *     calls and is safe to call from several host threads;
 *   - arguments are validated on the host before anything is launched; a
 *     non-zero lh_status means nothing was enqueued (LH_ERR_HIP: a launch
 *     failed; lh_last_error_message() holds the HIP error text);
 *   - sizes are element counts; strides / leading dimensions are in
 *     elements of the buffer's own dtype;
 *   - empty problems (a zero size) are valid and enqueue nothing, except the
 *     Hessian with n_tokens = 0, which still applies h = beta * h;
 *   - non-finite inputs give unspecified (but memory-safe) results.
 */
#ifndef LH_H
#define LH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lh_status {
    LH_OK = 0,
    LH_ERR_NULL = 1,      /* a required pointer is NULL                      */
    LH_ERR_SHAPE = 2,     /* negative size, c_in % 16 != 0, ld / stride too small */
    LH_ERR_DTYPE = 3,     /* unknown dtype code                               */
    LH_ERR_LAYOUT = 4,    /* unknown layout code                              */
    LH_ERR_WORKSPACE = 5, /* workspace non-empty but smaller than required    */
    LH_ERR_ARG = 6,       /* other invalid argument (e.g. no output requested) */
    LH_ERR_HIP = 7        /* a HIP launch failed (see lh_last_error_message)  */
} lh_status;

typedef enum lh_dtype {
    LH_DTYPE_F32 = 0,  /* IEEE binary32                                       */
    LH_DTYPE_BF16 = 1, /* bfloat16 (upper half of binary32), RNE-rounded data */
    LH_DTYPE_E4M3 = 2  /* OCP E4M3FN with a power of two per 32 values (only where said) */
} lh_dtype;

typedef enum lh_layout {
    LH_LAYOUT_CHANNEL_MAJOR = 0, /* x[c * ld_x + t]: X as [C_in][N] (the pages' X) */
    LH_LAYOUT_TOKEN_MAJOR = 1    /* x[t * ld_x + c]: X^T as [N][C_in] (hooked activations) */
} lh_layout;

typedef enum lh_rule {
    LH_RULE_SWEEP = 0,         /* all 126 E4M3 candidates (the Local-Hessian sweep) */
    LH_RULE_MAX = 1,           /* max scaling: the block's amax maps to 6           */
    LH_RULE_FOUR_OVER_SIX = 2, /* best of amax -> 6 and amax -> 4                   */
    LH_RULE_AMAX_SEARCH = 3    /* amax multipliers 0.25, 0.35, ..., 3.95            */
} lh_rule;

/* Library ABI version (this header describes version 1). */
int lh_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char *lh_status_string(int status);

/* Message of the last failing call on this host thread ("" if none). */
const char *lh_last_error_message(void);

/*
 * Global amax per group:  amax[g] = max |w[g][r][c]| over r < rows, c < cols.
 * The per-tensor FP32 amax the sweep derives its candidates from ("Algorithm
 * principle": the kernel receives the global FP32 amax).
 *   w        [n_groups] x [rows][ld_w] elements of w_dtype, group stride
 *            group_stride_w (>= 0).
 *   amax     [n_groups] fp32, written (device).
 * ld_w >= cols.  rows, cols, n_groups >= 0 (rows * cols == 0 writes 0).
 * Result is exact (a max), independent of launch shape.
 */
lh_status lh_absmax(const void *w, int w_dtype, int64_t rows, int64_t cols, int64_t ld_w,
                    int64_t n_groups, int64_t group_stride_w, float *amax, void *stream);

/*
 * The normalisation factor that lh_accumulate_hessian and lh_full_hessian
 * apply for a given alpha: alpha itself, or for alpha = NaN the normalised
 * Hessian's factor 1/N of "Entry API and calibration flow", phase 3 (the
 * per-block Hessian normalised by the token count), as fl32(1/n_tokens), and 0
 * for n_tokens <= 0.  Pure host function; lh_calibrate_* use the same factor.
 */
float lh_hessian_alpha(float alpha, int64_t n_tokens);

/*
 * Scratch bytes that let lh_accumulate_hessian split the token dimension of
 * each block over several workgroups and reduce the partial sums in a fixed
 * order (deterministic).  0 bytes is always accepted (one workgroup per
 * block); the value depends only on the three sizes.
 */
size_t lh_hessian_workspace_bytes(int64_t c_in, int64_t n_tokens, int64_t n_groups);

/*
 * Local-Hessian accumulation ("Algorithm principle": local Hessian
 * X_b X_b^T, 16 x 16 per input block; "Entry API and calibration flow",
 * phase 2: H is the sum of X^T X, normalised before the search):
 *
 *   h[g][b][i][j] = beta * h[g][b][i][j]
 *                 + alpha * sum_{t < n_tokens} X[g][16b+i][t] * X[g][16b+j][t]
 *
 * for every group g < n_groups, input block b < c_in / 16, 0 <= i, j < 16.
 * alpha = NaN asks for the normalised Hessian's factor: the library uses
 * lh_hessian_alpha(NaN, n_tokens) = fl32(1/n_tokens) (0 when n_tokens = 0).
 * alpha = 1/n_tokens (or NaN), beta = 0 gives the normalised one-shot
 * Hessian; alpha = 1, beta = 1 streams further token chunks into h.  beta == 0 never
 * reads h (so h may be uninitialised).  Products are exact (bf16 x bf16 or
 * fp32 x fp32 on matrix cores), sums are fp32.
 *   x        activations, x_dtype, `layout` (see lh_layout), leading
 *            dimension ld_x (channel-major: >= n_tokens; token-major:
 *            >= c_in), group stride group_stride_x (>= 0).
 *   h        [n_groups][c_in/16][16][16] fp32, group stride group_stride_h
 *            (>= (c_in/16)*256 when n_groups > 1), read (beta != 0) and written.
 *   workspace, workspace_bytes: NULL/0, or a device buffer of at least
 *            lh_hessian_workspace_bytes(c_in, n_tokens, n_groups) bytes,
 *            4-byte aligned; contents on entry are ignored.
 * c_in % 16 == 0.  Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE,
 * LH_ERR_LAYOUT, LH_ERR_WORKSPACE, LH_ERR_HIP.
 */
lh_status lh_accumulate_hessian(const void *x, int x_dtype, int layout, int64_t c_in,
                                int64_t n_tokens, int64_t ld_x, int64_t n_groups,
                                int64_t group_stride_x, float alpha, float beta, float *h,
                                int64_t group_stride_h, void *workspace, size_t workspace_bytes,
                                void *stream);

/*
 * Scratch bytes lh_accumulate_hessian_ragged can use for its deterministic
 * split of each group's rows (0 = it runs one pass per block).  Depends only
 * on the arguments (max_group_rows as passed to the accumulation).
 */
size_t lh_hessian_ragged_workspace_bytes(int64_t c_in, int64_t n_rows, int64_t n_groups,
                                         int64_t max_group_rows);

/*
 * Ragged / streaming local Hessians ("Entry API and calibration flow",
 * phase 2: forward hooks capture each layer's token-major inputs batch by
 * batch and accumulate X^T X; MoE experts receive only their routed tokens,
 * so their token counts differ and may be zero; phase 3 normalises by the
 * token count).
 *
 * x is token-major, x[t * ld_x + c] for rows t < n_rows; rows
 * token_offsets[g] .. token_offsets[g+1]-1 belong to group g (expert g),
 * n_g = their count.  With S_g[b] = sum over those rows of x_b x_b^T:
 *   token_counts == NULL:  h[g] = S_g / n_g for groups with n_g > 0.
 *   token_counts != NULL:  running mean over calls,
 *                          h[g] = (n_old h[g] + S_g) / (n_old + n_g),
 *                          n_old = token_counts[g]; then token_counts[g] += n_g.
 * A group that receives no row keeps h[g] unchanged (the caller's fallback,
 * e.g. the identity, which makes the sweep the plain weight-error sweep).
 *   x             fp32 or bf16 (x_dtype), ld_x >= c_in.
 *   token_offsets device int64 [n_groups + 1], 8-byte aligned; expected
 *                 non-decreasing within [0, n_rows].  Offsets are clamped to
 *                 [0, n_rows] and a decreasing pair gives an empty group, so
 *                 no offset can make the kernels read outside x.
 *   h             fp32 [n_groups][c_in/16][16][16], group stride
 *                 group_stride_h (>= (c_in/16)*256 when n_groups > 1).
 *   max_group_rows  host-side bound on any group's row count, or 0 if
 *                 unknown.  It only shapes the work split (with it, the rows
 *                 of the largest group spread over many workgroups in 1024-row
 *                 slices; without it, the split follows the average group);
 *                 results are correct whatever it is.
 *   token_counts  NULL, or device int64 [n_groups] (8-byte aligned), read
 *                 and updated on the stream.
 *   workspace     NULL/0, or at least lh_hessian_ragged_workspace_bytes(c_in,
 *                 n_rows, n_groups, max_group_rows) bytes (4-byte aligned).
 * Results are deterministic (fixed reduction order).
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_accumulate_hessian_ragged(const void *x, int x_dtype, int64_t c_in, int64_t ld_x,
                                       int64_t n_rows, const int64_t *token_offsets,
                                       int64_t n_groups, int64_t max_group_rows, float *h,
                                       int64_t group_stride_h,
                                       int64_t *token_counts, void *workspace,
                                       size_t workspace_bytes, void *stream);

/*
 * Scratch bytes that let lh_scale_sweep skip provably worse candidates with a
 * tight per-block certificate (a lower bound on the smallest eigenvalue of
 * the block's correlation matrix, one fp32 per block).  0 bytes is always
 * accepted: the sweep then uses a weaker certificate computed on the fly.
 * Results are identical either way; only the speed differs.
 */
size_t lh_sweep_workspace_bytes(int64_t c_in, int64_t n_groups);

/*
 * Local-Hessian scale sweep ("Algorithm principle": per 16-weight block,
 * all 126 FP8 E4M3 candidate scales derived from the global FP32 amax,
 * minimise dw^T H_b dw with dw = Q(w, s) - w; "ModelOpt overview",
 * "Local-Hessian": blocks are independent).
 *
 * For every group g, output row r < c_out and input block b < c_in/16, with
 * w_b = w[g][r][16b .. 16b+15], H_b = h[g][b] and global amax amax[g]:
 *   k*  = the lowest k in [0, 125] minimising E_k = dw_k^T H_b dw_k
 *   best_idx [g][r][b] = k*              (E4M3 block-scale code = k* + 1)
 *   best_err [g][r][b] = E_k* (fp32)     (optional)
 *   best_amax[g][r][b] = fl32(6 * s_k*)  (optional; the per-block amax)
 * The minimum is exact over all 126 candidates: a candidate is only skipped
 * when a certified lower bound proves it worse than one already evaluated.
 *   w         weights, w_dtype, row stride ld_w >= c_in, group stride
 *             group_stride_w (>= 0).
 *   h         fp32 [n_groups][c_in/16][16][16], 16-byte aligned (any square
 *             matrix is used as given; the output of lh_accumulate_hessian
 *             fits), group stride group_stride_h (>= 0, multiple of 4).
 *   amax      fp32 [n_groups] (device), e.g. from lh_absmax.
 *   best_idx  uint8 [n_groups][c_out][c_in/16], required.
 *   best_err, best_amax  fp32, same shape, NULL to skip.
 *   workspace, workspace_bytes: NULL/0, or a device buffer of at least
 *             lh_sweep_workspace_bytes(c_in, n_groups) bytes, 4-byte
 *             aligned; contents on entry are ignored.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_scale_sweep(const void *w, int w_dtype, int64_t c_out, int64_t c_in, int64_t ld_w,
                         int64_t n_groups, int64_t group_stride_w, const float *h,
                         int64_t group_stride_h, const float *amax, uint8_t *best_idx,
                         float *best_err, float *best_amax, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * The sweep and the fake-quant with its result in one pass ("Algorithm
 * principle": the candidate scales are bit-consistent with fake-quant, and
 * Q(W, s) = Cast(W / s) * s is the path's end product).  Writes exactly what
 * lh_scale_sweep followed by lh_fake_quant_nvfp4 with the chosen indices
 * writes, from one sweep launch that also emits the quantised blocks (each
 * lane quantises the rows it has just swept, so the weights are read again
 * from cache rather than by a second pass over the layer).
 *   Arguments up to workspace_bytes: as lh_scale_sweep (best_idx required).
 *   w_q, packed_e2m1, scale_e4m3, global_scale: as lh_fake_quant_nvfp4
 *             (dense layouts, each optional; w_q 16-byte aligned,
 *             packed_e2m1 8-byte aligned).
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_scale_sweep_fake_quant(const void *w, int w_dtype, int64_t c_out, int64_t c_in,
                                    int64_t ld_w, int64_t n_groups, int64_t group_stride_w,
                                    const float *h, int64_t group_stride_h, const float *amax,
                                    uint8_t *best_idx, float *best_err, float *best_amax,
                                    float *w_q, uint8_t *packed_e2m1, uint8_t *scale_e4m3,
                                    float *global_scale, void *workspace, size_t workspace_bytes,
                                    void *stream);

/*
 * Scratch bytes lh_calibrate_nvfp4 needs: the per-block skip certificates
 * and the Hessian's per-slice partial sums (and partial amax values).
 */
size_t lh_calibrate_workspace_bytes(int64_t c_out, int64_t c_in, int64_t n_tokens, int64_t n_groups);

/*
 * The first half of lh_calibrate_nvfp4: amax and h (as lh_absmax and
 * lh_accumulate_hessian with alpha = fl32(1/N), beta = 0), and the sweep's
 * skip certificates, which stay in the workspace for lh_calibrate_sweep.
 * Arguments as lh_calibrate_nvfp4.  With channel-major X and a contiguous W
 * (ld_w == c_in), both 16-byte aligned, this is two launches (amax and the
 * Hessian's token slices in one, the Hessian's finalisation with the
 * certificates in the other).
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_LAYOUT,
 * LH_ERR_WORKSPACE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_calibrate_prologue(const void *w, int w_dtype, int64_t c_out, int64_t c_in, int64_t ld_w,
                                int64_t n_groups, int64_t group_stride_w, const void *x, int x_dtype,
                                int x_layout, int64_t n_tokens, int64_t ld_x, int64_t group_stride_x,
                                float *amax, float *h, int64_t group_stride_h, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * The second half of lh_calibrate_nvfp4: lh_scale_sweep_fake_quant with the
 * certificates that lh_calibrate_prologue left in the workspace (same
 * workspace, same h and w, in stream order; no other call may write the
 * workspace in between).  Arguments as lh_scale_sweep_fake_quant; the
 * workspace is required.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_calibrate_sweep(const void *w, int w_dtype, int64_t c_out, int64_t c_in, int64_t ld_w,
                             int64_t n_groups, int64_t group_stride_w, const float *h,
                             int64_t group_stride_h, const float *amax, uint8_t *best_idx,
                             float *best_err, float *best_amax, float *w_q, uint8_t *packed_e2m1,
                             uint8_t *scale_e4m3, float *global_scale, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * The whole calibration path for a layer in one call: the global amax of W
 * ("Algorithm principle": the kernel receives the global FP32 amax), the
 * normalised local Hessians H_b = X_b X_b^T / N ("Entry API and calibration
 * flow", phase 3), the 126-candidate sweep and the fake-quant of its result
 * (as lh_scale_sweep_fake_quant).  Every output equals what lh_absmax,
 * lh_accumulate_hessian (alpha = fl32(1/N), beta = 0), lh_scale_sweep and
 * lh_fake_quant_nvfp4 write, bit for bit.
 *   w, w_dtype, c_out, c_in, ld_w, n_groups, group_stride_w: as lh_scale_sweep.
 *   x, x_dtype, x_layout, n_tokens, ld_x, group_stride_x: as
 *             lh_accumulate_hessian (N = n_tokens; N = 0 gives H = 0).
 *   amax      fp32 [n_groups] output.
 *   h         fp32 [n_groups][c_in/16][16][16] output, 16-byte aligned,
 *             group stride group_stride_h (multiple of 4).
 *   best_idx (required), best_err, best_amax, w_q, packed_e2m1, scale_e4m3,
 *   global_scale: as lh_scale_sweep_fake_quant.
 *   workspace: at least lh_calibrate_workspace_bytes(c_out, c_in, n_tokens,
 *             n_groups) bytes, 256-byte aligned, required.
 * It is lh_calibrate_prologue followed by lh_calibrate_sweep: three
 * launches with channel-major X and a contiguous W, both 16-byte aligned;
 * other layouts run the separate calls' kernels in turn.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_LAYOUT,
 * LH_ERR_WORKSPACE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_calibrate_nvfp4(const void *w, int w_dtype, int64_t c_out, int64_t c_in, int64_t ld_w,
                             int64_t n_groups, int64_t group_stride_w, const void *x, int x_dtype,
                             int x_layout, int64_t n_tokens, int64_t ld_x, int64_t group_stride_x,
                             float *amax, float *h, int64_t group_stride_h, uint8_t *best_idx,
                             float *best_err, float *best_amax, float *w_q, uint8_t *packed_e2m1,
                             uint8_t *scale_e4m3, float *global_scale, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * lh_calibrate_nvfp4 for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same arguments without the workspace, the same outputs
 * bit for bit.  Its scratch is a device array inside the library, 32 MiB on
 * each GPU the library runs on, held until the process ends; the call
 * allocates nothing.  Layers whose lh_calibrate_workspace_bytes(c_out, c_in,
 * n_tokens, n_groups) exceeds 32 MiB are rejected with LH_ERR_WORKSPACE
 * before anything is enqueued (mlp-down 5120 x 17408 with 16384 tokens needs
 * 17 MiB).  The stream must belong to the current device.  Every call on a
 * GPU uses that GPU's one array: calls that overlap on one GPU (other
 * streams, other host threads) race and must be ordered by the caller.  No
 * part of the array needs to start at zero: each call writes the scratch it
 * reads before reading it.
 * Errors: as lh_calibrate_nvfp4 (LH_ERR_WORKSPACE: layer too large for the
 * array; LH_ERR_ARG: stream of another device).
 */
lh_status lh_calibrate_nvfp4_noalloc(const void *w, int w_dtype, int64_t c_out, int64_t c_in, int64_t ld_w,
                                     int64_t n_groups, int64_t group_stride_w, const void *x, int x_dtype,
                                     int x_layout, int64_t n_tokens, int64_t ld_x, int64_t group_stride_x,
                                     float *amax, float *h, int64_t group_stride_h, uint8_t *best_idx,
                                     float *best_err, float *best_amax, float *w_q, uint8_t *packed_e2m1,
                                     uint8_t *scale_e4m3, float *global_scale, void *stream);

/*
 * Block-scale selection by rule: the scale rules the Local-Hessian guide
 * compares against ("What is Local-Hessian": max scaling takes the block
 * scale from the block's largest |w|; Four-Over-Six picks one of two
 * candidate scales by the in-block error; the MSE method sweeps all 126
 * positive FP8 values by the weight error; "Entry API and calibration
 * flow": with the 126-value sweep off, the amax is searched from
 * multiplier 0.25 to 4.0 in steps of 0.1).
 *
 * Objective: E_k = dw_k^T H_b dw_k when h is given (the local Hessian),
 * else the plain weight error sum_i dw_i^2 (H = I, the "MSE" rule).
 * Candidate set per block, with a = max |w_b| and S_g = fl32(amax[g]/2688);
 * a wanted scale value t is stored as the nearest positive finite E4M3
 * value (ties to the even code, above 448 -> 448, never zero):
 *   LH_RULE_SWEEP          all 126 candidates (with h: identical to
 *                          lh_scale_sweep; without h: the MSE sweep)
 *   LH_RULE_MAX            t = fl32(fl32(a / 6) / S_g)
 *   LH_RULE_FOUR_OVER_SIX  that t and t = fl32(fl32(a / 4) / S_g)
 *   LH_RULE_AMAX_SEARCH    t_i = fl32(fl32(fl32(m_i a) / 6) / S_g),
 *                          m_i = fl32((25 + 10 i) / 100), i = 0..37
 * Each block gets the candidate of lowest E_k in its set, lowest index on
 * ties; S_g = 0 gives candidate 0.  Outputs, layouts and arguments are
 * those of lh_scale_sweep, except:
 *   rule      an lh_rule value (else LH_ERR_ARG).
 *   h         may be NULL (plain weight error); group_stride_h is then
 *             ignored.
 *   workspace used only by LH_RULE_SWEEP with a Hessian (same contract
 *             as lh_scale_sweep); may be NULL/0.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_select_scales(int rule, const void *w, int w_dtype, int64_t c_out, int64_t c_in,
                           int64_t ld_w, int64_t n_groups, int64_t group_stride_w,
                           const float *h, int64_t group_stride_h, const float *amax,
                           uint8_t *best_idx, float *best_err, float *best_amax, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * NVFP4 fake-quant with chosen block scales ("Algorithm principle":
 * Q(W, s) = Cast(W / s) * s; the candidate scales match the sweep bit for
 * bit; "What is Local-Hessian": two-level format = E2M1 values, E4M3 block
 * scale, FP32 per-tensor scale).  For every weight of block (g, r, b) with
 * s = s_{best_idx[g][r][b]}:
 *   w_q[g][r][c]               = Q(w, s) (fp32, exactly the Q of the sweep)
 *   packed_e2m1[g][r][c/2]     = E2M1 nibble (bit 3 = sign, bits 0-2 =
 *                                magnitude code); low nibble = even column
 *   scale_e4m3[g][r][b]        = best_idx + 1 (OCP E4M3FN byte)
 *   global_scale[g]            = S_g = fl32(amax[g] / 2688)
 * Every output is optional (NULL to skip) but at least one must be given.
 * Output layouts are dense ([n_groups][c_out][c_in], [.][.][c_in/2],
 * [.][.][c_in/16], [n_groups]).  best_idx entries must be < 126.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_fake_quant_nvfp4(const void *w, int w_dtype, int64_t c_out, int64_t c_in,
                              int64_t ld_w, int64_t n_groups, int64_t group_stride_w,
                              const uint8_t *best_idx, const float *amax, float *w_q,
                              uint8_t *packed_e2m1, uint8_t *scale_e4m3, float *global_scale,
                              void *stream);

/*
 * ---------------------------------------------------------------------------
 * Approximation diagnostics ("Algorithm principle": the layer's output error
 * is ||Delta X||_F^2 = tr(Delta X X^T Delta^T), and Local-Hessian keeps only
 * the 16 x 16 diagonal blocks of X X^T; "How scaling reshapes the weight
 * distribution": the histogram of W/s, the values fed to the E2M1 rounding).
 * ---------------------------------------------------------------------------
 */

/*
 * Full Hessian h_full[g] = alpha * X_g X_g^T (C_in x C_in, fp32 accumulation
 * on matrix cores), X channel-major x[g][c * ld_x + t] (fp32 or bf16),
 * h_full[g][i * ld_h + j], ld_h >= c_in, group strides >= 0 (h groups must not
 * overlap).  With alpha = 1/N (or NaN, which the library replaces by
 * lh_hessian_alpha(NaN, n_tokens) = fl32(1/N)) its diagonal 16 x 16 blocks are
 * the local Hessians.  n_tokens = 0 writes zeros.  For bf16 layers with at
 * least 128 output tiles of 256 x 256 (16-byte aligned rows), only the lower
 * triangle of 256 x 256 or 192 x 192 tiles is computed and each off-diagonal
 * tile is also written transposed, so entries outside the diagonal tiles are
 * exact mirrors; otherwise h_full[i][j] and h_full[j][i] are computed
 * separately.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_full_hessian(const void *x, int x_dtype, int64_t c_in, int64_t n_tokens, int64_t ld_x,
                          int64_t n_groups, int64_t group_stride_x, float alpha, float *h_full,
                          int64_t ld_h, int64_t group_stride_h, void *stream);

/* Scratch bytes lh_output_error needs (one fp32 per row and 64-column tile). */
size_t lh_output_error_workspace_bytes(int64_t c_out, int64_t c_in, int64_t n_groups);

/*
 * Layer output error per output row with quantised weights w_q:
 *   err[g][r] = d H d^T,  d = w_q[g][r] - w[g][r] (fp32),  H = h_full[g]
 * (fp32 matrix cores; the row dot and the sum over column tiles run in a
 * fixed order, so results are deterministic).  With h_full = X X^T / N the
 * sum over rows is ||(W_q - W) X||_F^2 / N, to compare with the sum of the
 * sweep's block errors (the block-diagonal part).  H is used as given and
 * must be symmetric (h_full[j][i] stands in for h_full[i][j]).
 *   w (w_dtype, ld_w), w_q fp32 (ld_q), both [n_groups][c_out][.] with group
 *   strides; h_full [n_groups][c_in][ld_h]; err fp32 [n_groups][c_out].
 *   workspace: at least lh_output_error_workspace_bytes(c_out, c_in,
 *   n_groups) bytes, 4-byte aligned, required when there is work.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_output_error(const void *w, int w_dtype, const float *w_q, int64_t c_out, int64_t c_in,
                          int64_t ld_w, int64_t ld_q, int64_t n_groups, int64_t group_stride_w,
                          int64_t group_stride_q, const float *h_full, int64_t ld_h,
                          int64_t group_stride_h, float *err, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * Histogram of W/s: for every weight, x = fl32(|w| / s_k) with its block's
 * candidate k = best_idx (the quotient the cast rounds) and s_k from
 * amax[g]; bin = floor(fl32(x * bins_per_unit)), values at or beyond n_bins
 * go to the overflow bin n_bins; s = 0 gives x = 0.  counts (uint64
 * [n_groups][n_bins + 1], 8-byte aligned) is overwritten.  n_bins in
 * [1, 4096], bins_per_unit positive and finite.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_scaled_histogram(const void *w, int w_dtype, int64_t c_out, int64_t c_in,
                              int64_t ld_w, int64_t n_groups, int64_t group_stride_w,
                              const uint8_t *best_idx, const float *amax, int n_bins,
                              float bins_per_unit, uint64_t *counts, void *stream);

/*
 * ---------------------------------------------------------------------------
 * GPTQ rounding with fixed Local-Hessian scales ("Combining with GPTQ":
 * Local-Hessian sets the block scales, GPTQ then replaces round-to-nearest
 * to minimise the layer output error).  The GPTQ steps are the published
 * method's (Frantar et al., ICLR 2023).  One layer (group) per call.
 * ---------------------------------------------------------------------------
 */

/* Scratch bytes for lh_gptq_prepare (c_in) and lh_gptq_quantize (c_out, c_in). */
size_t lh_gptq_workspace_bytes(int64_t c_out, int64_t c_in);

/*
 * u = the upper Cholesky factor of H'^-1, H' = H + damp * mean(diag H) * I
 * (the identity when the diagonal is all zero): H'^-1 = u^T u, u upper with
 * a positive diagonal, zeros below.  h_full: fp32 [c_in][ld_h] (e.g. from
 * lh_full_hessian; any positive factor gives the same rounding); u: fp32
 * [c_in][ld_u].  The damped Hessian must be numerically positive definite,
 * else u holds non-finite values.  damp = 0.01 is the method's usual value.
 * workspace: lh_gptq_workspace_bytes(c_out, c_in) bytes, 16-byte aligned.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_WORKSPACE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_gptq_prepare(const float *h_full, int64_t c_in, int64_t ld_h, float damp, float *u,
                          int64_t ld_u, void *workspace, size_t workspace_bytes, void *stream);

/*
 * GPTQ quantisation of w [c_out][ld_w] (w_dtype) with the fixed block scales
 * best_idx [c_out][c_in/16] (candidate indices, e.g. from lh_scale_sweep)
 * and the global amax (device fp32 scalar): per row, for i = 0..c_in-1,
 *   q_i = Q(w_i, s_block(i))  (the cast of lh_fake_quant_nvfp4),
 *   e = (w_i - q_i) / u_ii,   w_j = fma(-e, u_ij, w_j) for j > i (fp32),
 * each w_j receiving its updates in increasing i.  w_q [c_out][ld_q] fp32
 * receives the q_i (dequantised values on each block's E2M1 grid; their
 * codes are what lh_fake_quant_nvfp4 would pack).  w is not modified.
 * workspace: lh_gptq_workspace_bytes(c_out, c_in) bytes, 16-byte aligned.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_gptq_quantize(const void *w, int w_dtype, int64_t c_out, int64_t c_in, int64_t ld_w,
                           const uint8_t *best_idx, const float *amax, const float *u,
                           int64_t ld_u, float *w_q, int64_t ld_q, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * What a language model does with the calibrated weights: activations
 * quantised on the fly ("What is Local-Hessian": NVFP4 blocks of 16 with an
 * E4M3 scale; max scaling maps the block's largest value to 6), products with
 * the packed weights and their gradient, and the way of tokens to the experts
 * of an MoE layer and back.
 * ---------------------------------------------------------------------------
 */

/*
 * Activations to NVFP4 in one pass over x [n_groups][rows][ld_x] (fp32 or
 * bf16; c_in % 16 == 0), with the per-tensor amax of the calibration (or of
 * lh_absmax; tokens given as groups get a scale each).  Per 16 values:
 *   code = the E4M3 code of LH_RULE_MAX, r = Cast(x / s), s = fl32(c * S_g),
 * bit for bit as lh_select_scales(LH_RULE_MAX) and lh_fake_quant_nvfp4,
 * wherever the former finds a finite error (it gives other blocks code 1).
 * An infinity takes the largest code and leaves as +-6 times it.  A NaN counts
 * for nothing in its block's maximum and leaves as +-6 times the block's code:
 * E2M1 has none.  With an infinite or NaN amax (lh_absmax of such values)
 * global_scale is infinite or NaN too, and the other outputs mean nothing.
 *   values       v_dtype (fp32 or bf16) [n_groups][rows][c_in]: r * c, the
 *                quantised value in units of S_g, exact in either type (so
 *                Q = values * S_g; lh_linear_nvfp4 takes S_g as x_scale)
 *   packed_e2m1, scale_e4m3, global_scale: as lh_fake_quant_nvfp4.
 * Outputs are dense, each optional, at least one given (where they have any
 * elements); values 16-byte, packed_e2m1 8-byte aligned.  x may have any
 * alignment of its own type.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_quantize_nvfp4(const void *x, int x_dtype, int64_t rows, int64_t c_in, int64_t ld_x,
                            int64_t n_groups, int64_t group_stride_x, const float *amax, void *values,
                            int v_dtype, uint8_t *packed_e2m1, uint8_t *scale_e4m3, float *global_scale,
                            void *stream);

/*
 * Scratch bytes with which lh_linear_nvfp4, lh_linear_nvfp4_grad and their
 * ragged forms run fastest, from the sizes and types alone (n_rows: the rows
 * per group, or all rows of a ragged call; grad: 0 for the product, 1 for the
 * gradient; ragged: 0 or 1; max_group_rows as passed to a ragged call).  0
 * bytes (NULL) is always accepted: other kernels then do the same work.
 */
size_t lh_linear_nvfp4_workspace_bytes(int grad, int ragged, int x_dtype, int64_t n_rows, int64_t c_in,
                                       int64_t c_out, int64_t n_groups, int64_t max_group_rows);

/*
 * Product with NVFP4 weights (Y = W X of "Algorithm principle", token-major):
 *   y[g][t][o] = global_scale[g] * x_scale[g]
 *                * sum_c x[g][t][c] * r[g][o][c] * c[g][o][c / 16]
 * for every group g, token t < n_tokens, output o < c_out; weights as
 * lh_fake_quant_nvfp4 and lh_calibrate_nvfp4 write them (dense
 * packed_e2m1 [n_groups][c_out][c_in/2], low nibble = even column, and
 * scale_e4m3 [n_groups][c_out][c_in/16]; codes 0x01..0x7E).
 * r * c is exact in bf16 and bf16 activations enter as they are; fp32
 * activations as three bf16 values that add up to them exactly (those below
 * 2^-110 but for less than 2^-133).  Products are exact and sums fp32, on
 * matrix cores; for up to two tokens (eight rows in all of a ragged call) the
 * sums of a block's 16 exact products x * r are, which its code then
 * multiplies, with one rounding per block.  One rounding to y_dtype at the end.
 * The order of a sum depends only on the arguments, never on the run.
 *   x            fp32 or bf16, [n_tokens][ld_x] per group, ld_x >= c_in.  bf16
 *                rows that do not start 16-byte aligned take a slower kernel.
 *   global_scale fp32 [n_groups] (S_g).  x_scale: fp32 [n_groups] or NULL
 *                (1): the S_g of activations given as lh_quantize_nvfp4 values.
 *   y            fp32 or bf16, [n_tokens][ld_y] per group, ld_y >= c_out;
 *                must not overlap x.  n_groups > 1: the groups of y must not
 *                overlap (one after the other, or side by side in wide rows).
 *   workspace    NULL/0, or at least lh_linear_nvfp4_workspace_bytes(0, 0,
 *                x_dtype, n_tokens, c_in, c_out, n_groups, 0) bytes, 256-byte
 *                aligned.
 * c_in % 16 == 0, c_out any.  c_in = 0 writes zeros.  A call of more than
 * 2^23 tiles of outputs (8 outputs of a token at least, 256 x 256 at most) may
 * be too large for one launch and is then refused (LH_ERR_SHAPE).
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_linear_nvfp4(const void *x, int x_dtype, int64_t n_tokens, int64_t c_in, int64_t ld_x,
                          int64_t group_stride_x, const uint8_t *packed_e2m1, const uint8_t *scale_e4m3,
                          const float *global_scale, int64_t c_out, int64_t n_groups, const float *x_scale,
                          void *y, int y_dtype, int64_t ld_y, int64_t group_stride_y, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * The product's gradient to its input, the weights being frozen:
 *   dx[g][t][c] = global_scale[g] * sum_o dy[g][t][o] * r[g][o][c] * c[g][o][c / 16]
 * (with activations that went through lh_quantize_nvfp4: the straight-through
 * gradient to them).  dy [n_tokens][ld_dy] with c_out columns, dx
 * [n_tokens][ld_dx] with c_in; types, exactness, aliasing, workspace (grad =
 * 1) and errors as lh_linear_nvfp4.  c_out = 0 writes zeros.
 */
lh_status lh_linear_nvfp4_grad(const void *dy, int dy_dtype, int64_t n_tokens, int64_t c_out, int64_t ld_dy,
                               int64_t group_stride_dy, const uint8_t *packed_e2m1,
                               const uint8_t *scale_e4m3, const float *global_scale, int64_t c_in,
                               int64_t n_groups, void *dx, int dx_dtype, int64_t ld_dx,
                               int64_t group_stride_dx, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * lh_linear_nvfp4 for rows sorted by expert: rows token_offsets[g] ..
 * token_offsets[g+1]-1 of x [n_rows][ld_x] meet the weights of group g, and
 * the result goes to the same rows of y.  Rows of no group are not written.
 *   token_offsets  device int64 [n_groups + 1], 8-byte aligned, expected
 *                  non-decreasing within [0, n_rows]; offsets are clamped
 *                  and a decreasing pair gives an empty group, so that no
 *                  offset can lead outside x or y (as
 *                  lh_accumulate_hessian_ragged).
 *   max_group_rows host bound on any group's rows, or 0 if unknown; it only
 *                  shapes the work split.
 * Everything else as lh_linear_nvfp4 (ragged = 1 in the workspace query).
 */
lh_status lh_linear_nvfp4_ragged(const void *x, int x_dtype, int64_t n_rows, int64_t c_in, int64_t ld_x,
                                 const int64_t *token_offsets, int64_t n_groups, int64_t max_group_rows,
                                 const uint8_t *packed_e2m1, const uint8_t *scale_e4m3,
                                 const float *global_scale, int64_t c_out, const float *x_scale, void *y,
                                 int y_dtype, int64_t ld_y, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* lh_linear_nvfp4_grad for rows sorted by expert, as lh_linear_nvfp4_ragged. */
lh_status lh_linear_nvfp4_ragged_grad(const void *dy, int dy_dtype, int64_t n_rows, int64_t c_out,
                                      int64_t ld_dy, const int64_t *token_offsets, int64_t n_groups,
                                      int64_t max_group_rows, const uint8_t *packed_e2m1,
                                      const uint8_t *scale_e4m3, const float *global_scale, int64_t c_in,
                                      void *dx, int dx_dtype, int64_t ld_dx, void *workspace,
                                      size_t workspace_bytes, void *stream);

typedef enum lh_index {
    LH_INDEX_I32 = 0, /* int32 */
    LH_INDEX_I64 = 1  /* int64 */
} lh_index;

/* Scratch bytes lh_moe_sort needs for n_tokens * top_k assignments (0 for few). */
size_t lh_moe_sort_workspace_bytes(int64_t n_tokens, int64_t top_k, int64_t n_groups);

/*
 * Assignments sorted by expert.  Assignment a = t * top_k + k sends token t to
 * expert expert_ids[a]; an id outside [0, n_groups) means none (dropped, for
 * instance over the expert's capacity).  The sort is stable:
 *   offsets  int64 [n_groups + 1]: expert g owns rows offsets[g] ..
 *            offsets[g+1]-1; offsets[n_groups] = the rows with an expert.
 *   position int32 [n_tokens][top_k]: the row p of assignment a; without an
 *            expert -1 - p, p being its row past offsets[n_groups].
 *   order    int32 [n_tokens * top_k], or NULL: the assignment of row p;
 *            -1 - a for one without an expert.
 * offsets is what lh_accumulate_hessian_ragged and lh_linear_nvfp4_ragged
 * take.  n_groups <= 1024, n_tokens * top_k < 2^31.
 *   expert_ids  ids_type (an lh_index), [n_tokens][top_k], contiguous.
 *   workspace   at least lh_moe_sort_workspace_bytes() bytes, 4-byte aligned
 *               (may be NULL where that is 0).
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_moe_sort(const void *expert_ids, int ids_type, int64_t n_tokens, int64_t top_k,
                      int64_t n_groups, int64_t *offsets, int32_t *position, int32_t *order,
                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * Tokens' rows to their experts: xs[position[t][k]] = x[t] for every
 * assignment with an expert; the rows of the others are set to zero.  Its
 * gradient is lh_moe_combine without weights.
 *   x  [n_tokens][ld_x], xs [n_rows][ld_xs], both dtype (fp32 or bf16) with
 *   `cols` columns (any number), n_rows >= n_tokens * top_k; entries of
 *   position beyond n_rows are ignored, rows that no entry names (past
 *   n_tokens * top_k, with the positions of lh_moe_sort) are not written.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_moe_dispatch(const void *x, int dtype, int64_t n_tokens, int64_t cols, int64_t ld_x,
                          const int32_t *position, int64_t top_k, void *xs, int64_t n_rows, int64_t ld_xs,
                          void *stream);

/*
 * Rows back to their tokens: y[t] = sum_k weights[t][k] * ys[position[t][k]]
 * over the assignments with an expert (a token without any gets zero), fp32
 * sums in the order of k, rounded once.  weights: fp32 [n_tokens][top_k], or
 * NULL for 1.  Sizes, types and errors as lh_moe_dispatch.
 */
lh_status lh_moe_combine(const void *ys, int dtype, int64_t n_rows, int64_t cols, int64_t ld_ys,
                         const int32_t *position, const float *weights, int64_t n_tokens, int64_t top_k,
                         void *y, int64_t ld_y, void *stream);

/*
 * The gradients of lh_moe_combine:
 *   dys[position[t][k]] = weights[t][k] * dy[t]   (zero rows for assignments
 *                         without an expert), dtype, [n_rows][ld_dys]; rows
 *                         that no entry names are not written (their
 *                         gradient is zero)
 *   dweights[t][k]      = <dy[t], ys[position[t][k]]> (0 without an expert),
 *                         fp32 [n_tokens][top_k]
 * Either may be NULL, not both (where they have any elements); weights NULL:
 * 1.  ys may be NULL when dweights is.  dys must not overlap dy or ys.  Sums
 * in a fixed order.
 */
lh_status lh_moe_combine_grad(const void *dy, int dtype, int64_t n_tokens, int64_t cols, int64_t ld_dy,
                              const void *ys, int64_t n_rows, int64_t ld_ys, const int32_t *position,
                              int64_t top_k, const float *weights, void *dys, int64_t ld_dys,
                              float *dweights, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Low-rank adapters beside the frozen projections, for many requests at once,
 * their gradients, and the activations that a backward pass needs kept in 8
 * bits.
 *
 * Rows that follow one another and belong together (a request's tokens, an
 * expert's rows) form a segment; every segment takes one adapter or none.
 * Both factors of adapter g are stored with the rank first, so that product
 * and gradients read whole rows of them: a [n_adapters][rank][c_in], b
 * [n_adapters][rank][c_out] (b is the transpose of a matrix that is applied
 * from the left), dense, fp32 or bf16.  The calls share these arguments:
 *   row_offsets  device int64 [n_segments + 1], 8-byte aligned: segment i has
 *                the rows row_offsets[i] .. row_offsets[i+1]-1; expected
 *                non-decreasing within [0, n_rows].  No offset can lead outside
 *                a buffer; where segments overlap, the first one has the rows
 *                that they share.  NULL: every row is a segment of its own
 *                (n_segments == n_rows), or all rows are one (n_segments == 1).
 *                n_segments and n_adapters are below 2^31.
 *   adapter_ids  ids_type (an lh_index) [n_segments], device; an id outside
 *                [0, n_adapters) means no adapter.  NULL: segment i takes
 *                adapter i (n_segments <= n_adapters; ids_type is ignored).
 *   rank         0 .. 256, the same for all adapters (shorter ones end in
 *                zeros).
 *   scale        fp32 [n_adapters] (device), or NULL (1).  Where x is in units of a
 *                global scale (the values of lh_quantize_nvfp4), that scale belongs
 *                into it, for the product and the factors' gradients.
 * ---------------------------------------------------------------------------
 */

/*
 * Scratch bytes that lh_lora (grad = 0) and lh_lora_grad (grad = 1) need, from
 * the sizes alone.
 */
size_t lh_lora_workspace_bytes(int grad, int64_t n_rows, int64_t n_segments, int64_t c_in, int64_t c_out,
                               int64_t rank);

/*
 * Low-rank adapters beside a projection: for every row t of a segment with
 * adapter g
 *   s[t][r] = sum_c x[t][c] a[g][r][c]
 *   y[t][o] = base[t][o] + scale[g] * sum_r s[t][r] b[g][r][o]
 * Rows of a segment without an adapter get y = base and s = 0; rows of no
 * segment are not written.  Sums are fp32 in an order that depends on the
 * sizes alone, products exact or rounded to fp32; s keeps its 24 bits on the
 * way out, whatever the types.
 * One rounding to y_dtype at the end.  Infinities and NaN follow the formula,
 * in their own row only, those of the factors too (but that an s below 2^-133
 * may count as zero where a bf16 factor is infinite).
 *   x      fp32 or bf16 [n_rows][ld_x], ld_x >= c_in.
 *   base   y_dtype [n_rows][ld_base], ld_base >= c_out, or NULL (0).  It may be
 *          y itself (with ld_base == ld_y): the projection's output is then
 *          added to in place.  Otherwise no buffers may overlap.
 *   y      fp32 or bf16 [n_rows][ld_y], ld_y >= c_out.
 *   s      fp32 [n_rows][rank], dense, or NULL: what lh_lora_weight_grad needs.
 *   workspace  at least lh_lora_workspace_bytes(0, ...) bytes, 256-byte
 *          aligned (may be NULL where that is 0).
 * Rows of any length and alignment of their type; 16-byte aligned ones are
 * fastest.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_lora(const void *x, int x_dtype, int64_t n_rows, int64_t c_in, int64_t ld_x,
                  const int64_t *row_offsets, const void *adapter_ids, int ids_type, int64_t n_segments,
                  const void *a, const void *b, int w_dtype, int64_t n_adapters, int64_t rank,
                  const float *scale, const void *base, int64_t ld_base, int64_t c_out, void *y, int y_dtype,
                  int64_t ld_y, float *s, void *workspace, size_t workspace_bytes, void *stream);

/*
 * lh_lora's gradient to its input, the same with the factors' roles exchanged:
 *   ds[t][r] = sum_o dy[t][o] b[g][r][o]
 *   dx[t][c] = base[t][c] + scale[g] * sum_r ds[t][r] a[g][r][c]
 * base is usually the projection's own gradient (lh_linear_nvfp4_grad).
 * Arguments, workspace (grad = 1) and errors as lh_lora, dy in the place of x
 * and dx of y.
 */
lh_status lh_lora_grad(const void *dy, int dy_dtype, int64_t n_rows, int64_t c_out, int64_t ld_dy,
                       const int64_t *row_offsets, const void *adapter_ids, int ids_type, int64_t n_segments,
                       const void *a, const void *b, int w_dtype, int64_t n_adapters, int64_t rank,
                       const float *scale, const void *base, int64_t ld_base, int64_t c_in, void *dx,
                       int dx_dtype, int64_t ld_dx, float *ds, void *workspace, size_t workspace_bytes,
                       void *stream);

/* Scratch bytes that lh_lora_weight_grad needs, from the sizes alone. */
size_t lh_lora_weight_grad_workspace_bytes(int64_t n_rows, int64_t n_segments, int64_t n_adapters, int64_t rank,
                                           int64_t c_in, int64_t c_out);

/*
 * lh_lora's gradients to the adapters, from what lh_lora (s) and lh_lora_grad
 * (ds) left:
 *   da[g][r][c] = beta * da[g][r][c] + scale[g] * sum_t ds[t][r] x[t][c]
 *   db[g][r][o] = beta * db[g][r][o] + scale[g] * sum_t s[t][r] dy[t][o]
 * over the rows t of all segments with adapter g, each row once (overlapping
 * segments as in the product).  Either output may be NULL,
 * not both (where they have any elements), and so may what only it needs.
 * beta == 0 never reads the outputs; an adapter without rows gets beta times
 * what it had.  fp32 sums in an order that depends on sizes and offsets alone.
 * s, ds and x of rows without an adapter are not read.
 *   x        x_dtype LH_DTYPE_F32, LH_DTYPE_BF16, or LH_DTYPE_E4M3 for a
 *            checkpoint of lh_checkpoint_pack (dense: ld_x == c_in), whose
 *            values enter as lh_checkpoint_unpack gives them in bf16.
 *   x_scale  the checkpoint's scales, or NULL.
 *   dy       fp32 or bf16 [n_rows][ld_dy].
 *   s, ds    fp32 [n_rows][rank], dense.
 *   da, db   out_dtype (fp32 or bf16), [n_adapters][rank][c_in] and
 *            [n_adapters][rank][c_out], dense.
 *   workspace  at least lh_lora_weight_grad_workspace_bytes() bytes, 256-byte
 *            aligned (may be NULL where that is 0).
 * n_adapters <= 1024; n_rows and the leading dimensions below 2^31.  An infinity
 * or NaN in x, dy, s or ds leaves infinities or NaN in its adapter's gradients.
 * Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE, LH_ERR_WORKSPACE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_lora_weight_grad(const void *x, int x_dtype, const uint8_t *x_scale, int64_t c_in, int64_t ld_x,
                              const void *dy, int dy_dtype, int64_t c_out, int64_t ld_dy, const float *s,
                              const float *ds, int64_t n_rows, const int64_t *row_offsets,
                              const void *adapter_ids, int ids_type, int64_t n_segments, int64_t n_adapters,
                              int64_t rank, const float *scale, float beta, void *da, void *db, int out_dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Activations in 8 bits: every 32 values of a row (fewer at its end) share a
 * power of two 2^e, the smallest with e >= -127 and no value beyond 448 2^e,
 * and are rounded to E4M3 after the division by it (nearest, ties to even;
 * the division is exact).
 *   values  uint8 [n_rows][cols]: the OCP E4M3FN codes
 *   scales  uint8 [n_rows][ceil(cols / 32)]: e + 127 (OCP E8M0)
 * A value is off by at most 2^-4 of itself, or 2^-17 of its block's largest
 * where that is more (e = -127 aside).  Infinities and NaN become NaN and count
 * for nothing in their block's maximum.
 *   x  fp32 or bf16 [n_rows][ld_x], ld_x >= cols, any alignment of its type.
 * Outputs are dense.  Errors: LH_ERR_NULL, LH_ERR_SHAPE, LH_ERR_DTYPE,
 * LH_ERR_ARG, LH_ERR_HIP.
 */
lh_status lh_checkpoint_pack(const void *x, int x_dtype, int64_t n_rows, int64_t cols, int64_t ld_x,
                             uint8_t *values, uint8_t *scales, void *stream);

/*
 * The activations back: x[t][c] = E4M3 value * 2^(scales - 127), exact in fp32
 * and bf16 (in bf16 but for values below 2^-133, which are rounded; a block
 * whose largest value was above 1.9375 * 2^127 may give infinities).  A scale
 * byte of 255 is E8M0's NaN.  x fp32 or bf16 [n_rows][ld_x], ld_x >= cols, any
 * alignment of its type.  Errors as lh_checkpoint_pack.
 */
lh_status lh_checkpoint_unpack(const uint8_t *values, const uint8_t *scales, int64_t n_rows, int64_t cols, void *x,
                               int x_dtype, int64_t ld_x, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LH_H */
