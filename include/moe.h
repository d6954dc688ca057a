/*
 * moe.h -- C ABI of the GB300 (sm_103a) fused Mixture-of-Experts layer.
 *
 * The layer is the fused MoE of the AITER walk-through (section 3, "Fused
 * MoE": gating -> token reorder by expert -> expert GEMMs -> weighted
 * combine) built as the two-stage group-GEMM path of the FlyDSL/Mixtral talk
 * (group GEMMs in place of masked dense GEMMs, SwiGLU activation):
 *
 *   route:   logits = x W_router^T (+ bias), top-k per token, softmax over
 *            the k selected logits (the weights sum to 1)
 *   sort:    the T*k (token, slot) pairs grouped by expert, each expert
 *            padded to whole blocks of block_m rows (section 3.1)
 *   stage 1: per block, gathered rows of x times W_gate_up[e]^T, then
 *            h = silu(gate) * up                              (section 3.2)
 *   stage 2: h times W_down[e]^T, each row scaled by its top-k weight
 *   combine: out[t] = sum over j of the weighted rows of token t
 *
 * Conventions for every entry point:
 *  - Pointers marked (device) are CUDA device pointers, (host) are host
 *    pointers.  All matrices are row-major and contiguous.  bf16 is IEEE
 *    bfloat16 bits in a uint16; e4m3 is the OCP FP8 E4M3 byte.
 *  - Weight layouts: W_router [E][H]; W_gate_up [E][2I][H] with rows 0..I-1
 *    the gate projection and rows I..2I-1 the up projection; W_down [E][H][I]
 *    (each expert matrix is N x K with K contiguous).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls are asynchronous on it: no host synchronisation, no
 *    allocation, no exceptions; results are ready when the stream is.
 *  - The caller owns every buffer.  The library keeps no mutable state
 *    that changes what a call computes or launches: only per-device
 *    constants (SM count, how many CTA-pair clusters fit).  Every
 *    choice a caller can make travels in the call's own arguments
 *    (block_m, split_k, and moe_options_t for moe_fused_forward_ex); the
 *    library reads no environment variables.
 *  - Arguments are validated on the host before anything is launched; an
 *    invalid call returns a negative status and launches nothing.  A CUDA
 *    launch error returns MOE_ERR_CUDA.  Kernels that wait on barriers give
 *    up after a bounded time and record MOE_ERR_TIMEOUT in the workspace
 *    status word (read it with moe_workspace_status).
 *
 * Limits: 1 <= k <= min(E, 32); E <= 1024; H and I multiples of 128 (the
 * tile granule of every GEMM kernel here, and the granule the AITER page's
 * stage rules test, inter_dim % 128); T >= 0 (T = 0 is a no-op that
 * returns MOE_OK).
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)
#define MOE_ERR_UNSUPPORTED (-2)
#define MOE_ERR_WORKSPACE (-3)
#define MOE_ERR_CUDA (-4)
#define MOE_ERR_TIMEOUT (-5)

#define MOE_BF16 0          /* bf16 weights and activations, fp32 accumulation */
#define MOE_FP8_BLOCK128 1  /* e4m3 weights (fp32 scale per 128x128 block) and
                               activations (fp32 scale per 1x128 group) */
#define MOE_FP8_TOKEN 2     /* e4m3 weights (fp32 scale per output channel) and
                               activations (fp32 scale per token) */
#define MOE_MXFP4 3         /* E2M1 weights and activations, E8M0 scale per 1x32
                               group */

#define MOE_MODE_GROUPED 0  /* tokens on the MMA M side, 128-row blocks */
#define MOE_MODE_SWAP 1     /* weights on the MMA M side, tokens on N (small T) */

/* Text for a status code.  Never NULL. */
const char *moe_status_string(int status);

/* Library version, major*10000 + minor*100 + patch. */
int moe_version(void);

/*
 * Sizes of the align-sort outputs (AITER page, section 3.1):
 * max_padded = T*k + E*block_m - k entries of sorted_ids / sorted_weights,
 * max_blocks = ceil(max_padded / block_m) entries of sorted_expert_ids.
 * Host only.  Returns MOE_OK or MOE_ERR_INVALID_ARG.
 */
int moe_align_sort_sizes(int T, int k, int E, int block_m, int64_t *max_padded, int64_t *max_blocks);

/*
 * The block-size rule of the AITER page (section 3.3, get_block_size_M):
 * among `candidates` (n entries), the block size with the fewest rounds of
 * tiles over `units` compute units, then the fewest idle units in the last
 * round (a full tie keeps the earlier candidate), where the tile count is
 * the page's tgN * (max_padded + BM - 1) // BM evaluated left to right,
 * (tgN * (max_padded + BM - 1)) / BM, with tgN = ceil(inter_dim/128) and
 * max_padded = token*topk + expert*BM - topk.  Host only; returns the chosen
 * block size or a negative status.
 */
int moe_block_size_m_heuristic(int token, int topk, int expert, int inter_dim, int units,
                               const int *candidates, int n);

/*
 * The K-split rule of the AITER page (section 3.4, get_ksplit), with the
 * page's undefined tgN/tgM read as ceil(inter_dim/128) and
 * ceil(token*topk/block_m).  Returns the split (0 = none) or a negative
 * status.  Host only.
 */
int moe_ksplit_heuristic(int token, int topk, int expert, int inter_dim, int model_dim, int units,
                         int block_m);

/* The plan moe_fused_forward follows for a shape. */
typedef struct moe_plan {
    int mode;           /* MOE_MODE_GROUPED or MOE_MODE_SWAP */
    int block_m;        /* sort block size (rows per padded expert block) */
    int split_k1;       /* K splits of stage 1 (1 = none) */
    int split_k2;       /* K splits of stage 2 (1 = none) */
    int64_t max_padded; /* T*k + E*block_m - k */
    int64_t max_blocks; /* ceil(max_padded / block_m) */
    size_t workspace_bytes;
} moe_plan_t;

/*
 * Choose mode, block size and K splits for a layer shape.  block_m = 0 and
 * split_k = 0 mean automatic; otherwise they are used as given (block_m
 * must be 128 in grouped mode and a multiple of 16 up to 128 in swap mode;
 * split_k splits stage 2's K = I and must divide I/64, I/128 for
 * MOE_FP8_TOKEN or I/256 for MOE_MXFP4; MXFP4 swap mode (T <= 64) takes
 * block_m up to 64).  num_sms = 0 asks
 * the current CUDA device; a positive value plans for that many SMs without
 * touching CUDA.  Returns MOE_OK or a negative status.  Host only.
 */
int moe_plan(int dtype, int T, int H, int I, int E, int k, int block_m, int split_k, int num_sms,
             moe_plan_t *plan);

/*
 * Workspace bytes moe_fused_forward needs for this shape (the plan's
 * workspace_bytes, planned for the current device).  0 on invalid input.
 */
size_t moe_fused_workspace_size(int dtype, int T, int H, int I, int E, int k, int block_m, int split_k);

/*
 * Byte offsets of the intermediate buffers inside the workspace of
 * moe_fused_forward (for inspection and tests; -1 = not present).
 */
typedef struct moe_ws_layout {
    int64_t status;          /* int32 status word (MOE_OK or MOE_ERR_TIMEOUT); word 4 after it:
                                tokens whose tensor-core routing fell back to all
                                fixed-order logits */
    int64_t topk_ids;        /* int32 [T][k] */
    int64_t topk_weights;    /* fp32 [T][k] */
    int64_t sorted_ids;      /* int32 [max_padded] */
    int64_t sorted_weights;  /* fp32 [max_padded] */
    int64_t sorted_expert_ids; /* int32 [max_blocks] */
    int64_t num_tokens_post_padded; /* int32 [1] */
    int64_t expert_counts;   /* int32 [E] */
    int64_t x_sorted;        /* bf16 [max_padded][H] or e4m3 [max_padded][H] */
    int64_t x_scales;        /* fp32 [H/128][max_padded] (FP8 block), [max_padded] (FP8 token) */
    int64_t inter;           /* bf16 [max_padded][I] or e4m3 [max_padded][I] */
    int64_t inter_scales;    /* fp32 [I/128][max_padded] (FP8 block), [max_padded] (FP8 token) */
    int64_t inter_h;         /* bf16 [max_padded][I]: SwiGLU output before its per-token
                                quantisation (FP8 token only) */
    int64_t y;               /* bf16 [T*k][H], weighted rows in slot order (each rounded once
                                from its fp32 value) */
    int64_t router_logits;   /* fp32 router logits: [T][E] from the CUDA-core router, or the
                                tensor-core router's per-slice partial sums
                                [splits][ceil(T/128)*128][E] */
    int64_t total;
} moe_ws_layout_t;

int moe_workspace_layout(int dtype, int T, int H, int I, int E, int k, int block_m, int split_k,
                         moe_ws_layout_t *layout);

/*
 * Read the workspace status word (device) into *status (host).  Synchronises
 * `stream`.  Returns MOE_OK or MOE_ERR_CUDA.
 */
int moe_workspace_status(const void *ws, int *status, void *stream);

/*
 * Router (gating + top-k; AITER page section 3, FlyDSL talk "Mixtral"):
 *   logit[t][e] = sum_h x[t][h] * W_router[e][h]  (+ bias[e])
 * in fp32 in one fixed order -- the H products are dealt to 32 partial sums
 * in chunks of 8 elements (element h to partial (h/8) mod 32), each partial
 * adds in ascending h, then the partials are combined by a butterfly with
 * strides 16, 8, 4, 2, 1 -- so the ids are a deterministic function of the
 * bytes.  topk_ids[t] = the k largest logits, largest first, an equal logit
 * going to the lower expert.  topk_weights[t][j]:
 *   renormalize = 1: exp(l_j - l_0) / sum over the k selected (they sum to 1;
 *                    what moe_fused_forward uses);
 *   renormalize = 0: exp(l_j - l_0) / sum over all E experts (the softmax
 *                    over all experts, evaluated at the selected ones).
 *   x (device) bf16 [T][H]; W_router (device) bf16 [E][H];
 *   bias (device) fp32 [E] or NULL; topk_ids (device) int32 [T][k];
 *   topk_weights (device) fp32 [T][k]; logits (device) fp32 [T][E] or NULL.
 * With logits given and T*E > 4096 the logits are computed by a tiled pass
 * and the top-k by a second pass (faster for large T*E); otherwise one fused
 * launch.  Both give the same bits.  H % 8 == 0.
 */
int moe_route_topk(const void *x, const void *W_router, const float *bias, int T, int H, int E, int k,
                   int renormalize, int32_t *topk_ids, float *topk_weights, float *logits, void *stream);

/* Scratch bytes moe_align_sort needs (device memory passed as ws). */
size_t moe_align_sort_workspace_size(int T, int k, int E);

/*
 * Token sort and alignment by expert (AITER page section 3.1, moe_sorting):
 * slot s = t*k + j.  Expert e's segment lists its slots in ascending s and
 * is padded with the sentinel T*k up to a multiple of block_m; segments
 * follow in ascending e; experts without slots take no block.
 *   topk_ids (device) int32 [T][k]; topk_weights (device) fp32 [T][k];
 *   sorted_ids (device) int32 [max_padded]: slot or T*k (padding / unused);
 *   sorted_weights (device) fp32 [max_padded]: topk weight of the slot, 0 on padding;
 *   sorted_expert_ids (device) int32 [max_blocks]: expert of each block, -1 if unused;
 *   num_tokens_post_padded (device) int32 [1]: sum of the padded segment lengths;
 *   expert_counts (device) int32 [E] or NULL: slots per expert;
 *   ws (device) scratch of moe_align_sort_workspace_size bytes.
 * An id outside [0, E) is a caller error.  The kernels check every id: a
 * slot with a bad id is left out of every segment (nothing outside the
 * output buffers is written) and num_tokens_post_padded is set to
 * MOE_ERR_INVALID_ARG (-1), which no valid result can be; check it when the
 * ids come from untrusted code.
 */
int moe_align_sort(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E, int block_m,
                   int32_t *sorted_ids, float *sorted_weights, int32_t *sorted_expert_ids,
                   int32_t *num_tokens_post_padded, int32_t *expert_counts, void *ws, size_t ws_bytes,
                   void *stream);

/*
 * Block-scaled FP8 quantisation ("per_1x128" on the AITER page):
 * activations per 1x128 group of a row, weights per 128x128 block; each
 * group takes scale = amax / 448 (1 for an all-zero group) and codes
 * e4m3(v / scale), rounded to nearest even and saturated to +-448.
 *   moe_quantize_fp8_act: X (device) bf16 [R][C], C % 128 == 0 ->
 *     q (device) e4m3 [R][C], s (device) fp32 [R][C/128].
 *   moe_quantize_fp8_weights: W (device) bf16 [R][C], R and C % 128 == 0
 *     (an expert stack [E][N][K] is R = E*N, C = K) ->
 *     q (device) e4m3 [R][C], s (device) fp32 [R/128][C/128].
 */
int moe_quantize_fp8_act(const void *X, int64_t R, int C, uint8_t *q, float *s, void *stream);
int moe_quantize_fp8_weights(const void *W, int64_t R, int C, uint8_t *q, float *s, void *stream);

/*
 * Per-row FP8 quantisation ("per_Token" on the AITER page, section 3.2's
 * quantisation types): one scale per row -- a token of the activations or
 * an output channel of a weight stack -- scale = amax of the row / 448 (1
 * for an all-zero row), codes e4m3(v / scale), rounded to nearest even and
 * saturated to +-448.
 *   X (device) bf16 [R][C], C % 16 == 0 -> q (device) e4m3 [R][C],
 *   s (device) fp32 [R].  An expert stack [E][N][K] is R = E*N, C = K.
 */
int moe_quantize_fp8_rows(const void *X, int64_t R, int C, uint8_t *q, float *s, void *stream);

/*
 * MXFP4 quantisation ("per_1x32" on the AITER page; OCP microscaling FP4):
 * each group of 32 consecutive elements of a row shares the power-of-two
 * scale 2^e, e = floor(log2(group amax)) - 2 (0 for an all-zero group),
 * stored as the E8M0 byte e + 127; elements are v * 2^-e rounded to the
 * nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives; ties to the
 * even mantissa), clamped to +-6, as codes sign << 3 | magnitude index.
 *   X (device) bf16 [R][C], C % 32 == 0 -> q (device) [R][C/2] bytes, two
 *   codes per byte (element 2j in the low nibble of byte j);
 *   s (device) E8M0 bytes: tiled = 0 row-major [R][C/32]; tiled = 1 (R and
 *   C multiples of 128; the weight order moe_fused_forward reads)
 *   [R/128][C/128][512], group g of row r of a 128 x 128 tile at byte
 *   (r % 32) * 16 + (r % 128 / 32) * 4 + g % 4.
 */
int moe_quantize_mxfp4(const void *X, int64_t R, int C, uint8_t *q, uint8_t *s, int tiled, void *stream);

/*
 * Per-call choices of moe_fused_forward_ex and the training entries.  Fill
 * one with moe_options_init (the library's defaults) and change the fields
 * you need; a NULL options pointer means the defaults.  These select among
 * kernels that compute the same layer (each within the same tolerance of
 * the definition) or add instrumentation; none changes the workspace size.
 * (No counterpart on the fused-MoE pages: launch choices of this library.)
 */
typedef struct moe_options {
    /* Grouped-mode GEMM kernel for MOE_BF16, MOE_FP8_TOKEN and
     * MOE_FP8_BLOCK128: -1 automatic (CTA pairs when the average expert
     * holds at least one 128-row token block, T*k >= 128 * min(E, T*k): in
     * both stages for bf16, in stage 2 for per-token FP8, never for block
     * FP8, whose pair kernels are bit-identical to its one-SM kernels but
     * slower in stage 1), 0 always the one-SM kernels, 1 CTA pairs (the
     * two-SM tensor core) wherever supported. */
    int gemm_pair;
    /* bf16 swap mode (T <= 128): 1 runs both GEMM stages in one persistent
     * launch ("1-stage", AITER page section 3.2: tiles of both stages claimed
     * from one counter, stage-1 tiles first, the intermediate kept in L2,
     * the token rows fetched from x by the launch itself), 0 two launches
     * with a gather pass before them.  Both give bit-identical results.
     * Default 1. */
    int one_stage;
    /* Programmatic dependent launch: -1 the library's default set of launch
     * boundaries, otherwise a mask of them (bit 0 router -> sort and inside
     * the sort, 1 sort -> gather, 2 -> stage 1, 3 stage 1 -> stage 2, 4 ->
     * combine, 5 logit pass -> top-k pass, 6 preceding work -> router);
     * 0 turns it off.  Default -1 (all, except bits 2 and 3 in grouped mode,
     * where an early-resident persistent GEMM measured slower). */
    int pdl_mask;
    /* NULL, or 7 CUDA events (cudaEvent_t cast to void*, created by the
     * caller) recorded on the call's stream at [0] entry, [1] after routing,
     * [2] after the sort, [3] after the gather (FP8: gather + quantise),
     * [4] after stage 1, [5] after stage 2 (per-token FP8: including the
     * re-quantisation of the intermediate), [6] after the combine.  With the
     * one-launch decode path [3] follows [2] and [5] follows [4] directly.
     * Events between launches stop their overlap: time whole calls without. */
    void *const *stage_events;
    /* Limit, in microseconds, of the one-launch decode path's wait for the
     * intermediate (stage-2 tiles wait for every stage-1 epilogue); 0 = the
     * default of 2 s.  Every other device wait keeps its 2 s limit. */
    unsigned int h_wait_limit_us;
    /* Test of the timeout path only (0 otherwise): 1 makes the one-launch
     * decode path's stage-2 tiles wait for one more stage-1 epilogue than
     * exists, so that wait runs out after h_wait_limit_us; the call then
     * records MOE_ERR_TIMEOUT in the workspace status word and every CTA
     * returns after its copies and MMAs in flight have completed.  The
     * output of such a call is undefined; the next call on the workspace
     * starts clean. */
    int unsatisfiable_h_wait;
    /* MOE_BF16 on CTA pairs: experts with at most 64 tokens take swap-AB
     * pair tiles (the weights on the pair's 256-row MMA side, the expert's
     * tokens, rounded up to 32, on N) instead of a mostly padded 256 x 256
     * tile; light and 256 x 256 tiles are interleaved so that weight
     * streaming and tensor work overlap.  -1 automatic (default: on when I is
     * a multiple of 256, E <= 512 and the average expert that can hold a slot
     * has fewer than 4 blocks of 128 rows), 0 off, 1 on (needs I % 256 == 0
     * and E <= 512, else MOE_ERR_UNSUPPORTED).  Not used by the training
     * forward. */
    int light_tiles;
    /* Router for many experts (E >= 64, E % 32 == 0, T >= 64, k <= 28):
     * -1 automatic / 1: logits on the tensor core, then the k + 4 leading
     * candidates recomputed in the fixed order and the remaining experts
     * checked against a bound on the difference of the two sums (a near tie
     * recomputes all E logits in the fixed order), so the ids and weights are
     * those of the fixed-order router bit for bit; 0: the fixed-order router
     * on CUDA cores for every logit. */
    int tc_router;
} moe_options_t;

/* Set *options to the defaults (gemm_pair -1, one_stage 1, pdl_mask -1, no
 * events, default wait limit, no test switch).  Returns MOE_OK or
 * MOE_ERR_INVALID_ARG (NULL). */
int moe_options_init(moe_options_t *options);

/*
 * moe_fused_forward with per-call options (NULL = defaults).  Everything else
 * as moe_fused_forward.  Returns MOE_ERR_INVALID_ARG for an option outside
 * its range.
 */
int moe_fused_forward_ex(int dtype, const void *x, const void *W_router, const float *router_bias,
                         const void *W_gate_up, const void *w1_scale, const void *W_down, const void *w2_scale,
                         int T, int H, int I, int E, int k, int block_m, int split_k, void *out, void *ws,
                         size_t ws_bytes, const moe_options_t *options, void *stream);

/*
 * The whole layer: route, align-sort, stage 1 (gate/up group GEMM with the
 * SwiGLU epilogue), stage 2 (down group GEMM scaled by the top-k weights),
 * combine.  out (device) bf16 [T][H].
 *   dtype MOE_BF16: W_gate_up / W_down (device) bf16; w1_scale, w2_scale NULL.
 *   dtype MOE_FP8_BLOCK128: W_gate_up / W_down (device) e4m3 with
 *     w1_scale (device) fp32 [E*2I/128][H/128] and w2_scale (device) fp32
 *     [E*H/128][I/128] (as produced by moe_quantize_fp8_weights); x is
 *     quantised per 1x128 group inside the call, the router runs on bf16 x,
 *     and the SwiGLU output is re-quantised per 1x128 group between stages.
 *   dtype MOE_FP8_TOKEN: W_gate_up / W_down (device) e4m3 with w1_scale
 *     (device) fp32 [E*2I] and w2_scale (device) fp32 [E*H], one per output
 *     channel (as produced by moe_quantize_fp8_rows); x is quantised per
 *     token inside the call, the router runs on bf16 x, and the SwiGLU
 *     output (rounded to bf16) is re-quantised per token between stages.
 *   dtype MOE_MXFP4: W_gate_up / W_down (device) E2M1 codes, two per byte
 *     ([E][2I][H/2] and [E][H][I/2] bytes), with w1_scale / w2_scale
 *     (device) the E8M0 scale bytes in the tiled weight order of
 *     moe_quantize_mxfp4 (tiled = 1); x is quantised per 1x32 group inside
 *     the call, the router runs on bf16 x, and the SwiGLU output is
 *     re-quantised per 1x32 group between stages.  H and I multiples of
 *     256 (MOE_ERR_UNSUPPORTED otherwise).
 *   x (device) bf16 [T][H]; W_router (device) bf16 [E][H]; router_bias
 *   (device) fp32 [E] or NULL; block_m / split_k as in moe_plan;
 *   ws (device) of at least moe_fused_workspace_size bytes, 1024-byte aligned.
 * The result is deterministic: no atomics touch floating-point data.
 */
int moe_fused_forward(int dtype, const void *x, const void *W_router, const float *router_bias,
                      const void *W_gate_up, const void *w1_scale, const void *W_down, const void *w2_scale,
                      int T, int H, int I, int E, int k, int block_m, int split_k, void *out, void *ws,
                      size_t ws_bytes, void *stream);

/*
 * Training (bf16; the pages' stated future work for the group-GEMM MoE
 * kernels: backward "dgrad" and "wgrad" passes).
 *
 * moe_train_workspace_size: bytes of the workspace shared by one training
 * forward and its backward (0 on invalid input; I must be a multiple of 256).
 *
 * moe_fused_forward_train: moe_fused_forward for MOE_BF16 that always runs
 * the grouped (128-row block) path and keeps in ws what the backward needs:
 * the routing and sort, the sorted x rows, the pre-activations g | u, the
 * SwiGLU output h and the weighted stage-2 rows.  Same arguments as
 * moe_fused_forward without dtype, scales, block_m and split_k.
 *
 * moe_fused_backward: gradients for loss = sum(dout * out) of the forward
 * that last ran on ws (same x, weights and shape):
 *   dout (device) bf16 [T][H]  ->  dx (device) bf16 [T][H];
 *   dW_gate_up (device) fp32 [E][2I][H], dW_down (device) fp32 [E][H][I],
 *   dW_router (device) fp32 [E][H], dbias (device) fp32 [E] or NULL.
 * The top-k choice is a selection: the gradient reaches the router through
 * the softmax over the chosen k logits.  Experts without tokens get zero
 * weight gradients.  Every sum runs in a fixed order (no atomics), so the
 * gradients are bitwise reproducible.  Returns MOE_OK or a negative status.
 */
size_t moe_train_workspace_size(int T, int H, int I, int E, int k);
int moe_fused_forward_train(const void *x, const void *W_router, const float *router_bias, const void *W_gate_up,
                            const void *W_down, int T, int H, int I, int E, int k, void *out, void *ws,
                            size_t ws_bytes, const moe_options_t *options, void *stream);
int moe_fused_backward(const void *x, const void *W_router, const float *router_bias, const void *W_gate_up,
                       const void *W_down, const void *dout, int T, int H, int I, int E, int k, void *dx,
                       float *dW_gate_up, float *dW_down, float *dW_router, float *dbias, void *ws, size_t ws_bytes,
                       const moe_options_t *options, void *stream);

/*
 * moe_fused_forward with the activations in host memory: x_host (host) bf16
 * [T][H] is copied to the device inside the call and the result is copied
 * back to out_host (host) bf16 [T][H], all on `stream` (pinned host memory
 * keeps the copies asynchronous).  Device staging lives in ws, which must
 * hold moe_fused_workspace_size(...) + moe_host_staging_bytes(T, H) bytes.
 * out_host is valid once the stream has completed.
 */
size_t moe_host_staging_bytes(int T, int H);
int moe_fused_forward_host(int dtype, const void *x_host, const void *W_router, const float *router_bias,
                           const void *W_gate_up, const void *w1_scale, const void *W_down,
                           const void *w2_scale, int T, int H, int I, int E, int k, int block_m,
                           int split_k, void *out_host, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_align_sort without a caller workspace.  (The fused-MoE pages have no
 * counterpart: this entry exists for callers of this library.)
 *
 * For callers that cannot allocate device memory themselves -- code that
 * must not call cudaMalloc because a host framework owns every device
 * allocation through its own pool, runs under a fixed memory budget, or
 * cannot afford the implicit synchronisation of an allocation on its hot
 * path.  They pass the same inputs and outputs as moe_align_sort, but no ws.
 *
 * The scratch is a fixed array of MOE_NOALLOC_SORT_SCRATCH_BYTES in the
 * library's own device memory; every GPU that loads the library holds it
 * until the process exits.  Every call looks up the array's address on the
 * current device (cudaGetSymbolAddress, which allocates nothing; it stays
 * right after a cudaDeviceReset).  The first call on a device may load the
 * library's device code there, so make that first call before any stream
 * capture.  Nothing is allocated, by this library or any library it calls.
 * Shapes whose scratch (one int32 per expert per 1024 slots, plus E+1
 * offsets) does not fit return MOE_ERR_UNSUPPORTED; use moe_align_sort with
 * a workspace for those.  All calls share the one array and it keeps the
 * last call's contents: calls that overlap on the GPU (on different streams,
 * or from different host threads without ordering) race on it and must be
 * serialised by the caller.  Ids are checked as in moe_align_sort.
 */
#define MOE_NOALLOC_SORT_SCRATCH_BYTES (1 << 20)

int moe_align_sort_noalloc(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E,
                           int block_m, int32_t *sorted_ids, float *sorted_weights,
                           int32_t *sorted_expert_ids, int32_t *num_tokens_post_padded,
                           int32_t *expert_counts, void *stream);

/*
 * ------------------------------------------------------------------------
 * Operators around the layer: the token exchange, the block-scaled FP8
 * product and the norms around a block, for blocks that the fused layer does
 * not cover (other expert functions, shared experts, FP8 training).
 *
 * Rows are bf16, fp16 or fp32 (row_type); arithmetic and sums are fp32, each
 * result rounded once.  None of these entries uses floating-point atomics:
 * results are bitwise reproducible.  Rows that start and end on 16-byte
 * boundaries are moved 16 bytes at a time, others element by element.
 * Counts of zero (tokens, rows) are valid; pointers that are not said to be
 * optional are non-null in such a call too, and nothing behind them is read.
 */
#define MOE_ROW_BF16 0
#define MOE_ROW_FP16 1
#define MOE_ROW_FP32 2

/*
 * moe_align_sort that also gives the inverse map: slot_pos (device) int32
 * [T*k], the sorted position of each slot, -1 for a slot left out because its
 * id is outside [0, E).  Everything else as moe_align_sort (same ws): such an
 * id is an error, num_tokens_post_padded = -1 refuses the whole routing, and
 * the entries below that read it then zero no padding and compute no row.
 * Limit: T*k + E*block_m - k < 2^31.
 */
int moe_align_sort_map(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E, int block_m,
                       int32_t *sorted_ids, float *sorted_weights, int32_t *sorted_expert_ids,
                       int32_t *num_tokens_post_padded, int32_t *expert_counts, int32_t *slot_pos, void *ws,
                       size_t ws_bytes, void *stream);

/*
 * moe_align_sort_map for routings that leave slots out on purpose (dropped
 * tokens, masked rows, experts held elsewhere): an id outside [0, E) is no
 * error.  num_tokens_post_padded is the sum of the padded segments of the
 * slots that stay (never -1), and num_left_out (device) int32 [1] the number
 * of slots left out, for callers that expect none.  The entries below then
 * give such a slot nothing and add nothing for it.
 */
int moe_align_sort_drop(const int32_t *topk_ids, const float *topk_weights, int T, int k, int E, int block_m,
                        int32_t *sorted_ids, float *sorted_weights, int32_t *sorted_expert_ids,
                        int32_t *num_tokens_post_padded, int32_t *expert_counts, int32_t *slot_pos,
                        int32_t *num_left_out, void *ws, size_t ws_bytes, void *stream);

/*
 * Rows to the experts' order: xs[slot_pos[t*k + j]] = x[t].
 *   x (device) [T] rows of H elements at a pitch of ld_x >= H elements;
 *   slot_pos (device) int32 [T*k]; a position outside [0, P) is skipped;
 *   xs (device) [P][H].
 * zero_padding = 1 also writes zeros to the padding rows (p <
 * *num_tokens_post_padded with sorted_ids[p] >= T*k; both device pointers,
 * ignored and may be NULL when 0).  Other rows of xs are left as they are.
 * Limits: 1 <= k <= 32, T*k <= 2^30, P < 2^31.
 */
int moe_permute(int row_type, const void *x, int64_t ld_x, const int32_t *slot_pos, const int32_t *sorted_ids,
                const int32_t *num_tokens_post_padded, int T, int k, int H, int64_t P, int zero_padding, void *xs,
                void *stream);

/*
 * The same for bf16 rows, quantised per 1x128 group as moe_quantize_fp8_act
 * does (a negative zero's code is that of zero): q (device) e4m3 [P][H], s
 * (device) fp32 [H/128][P] (by block: the a_scale_by_block = 1 form of
 * moe_gemm_fp8_block).  A padding row that is zeroed has scale 1.  H % 128 == 0, ld_x % 8 == 0, x and q on 16-byte
 * boundaries.
 */
int moe_permute_fp8(const void *x, int64_t ld_x, const int32_t *slot_pos, const int32_t *sorted_ids,
                    const int32_t *num_tokens_post_padded, int T, int k, int H, int64_t P, int zero_padding,
                    uint8_t *q, float *s, void *stream);

/* Gradient of moe_permute: dx[t] = sum over j of dxs[slot_pos[t*k + j]] (j
 * ascending).  dxs (device) [P][H]; dx (device) [T] rows at pitch ld_dx. */
int moe_permute_backward(int row_type, const void *dxs, const int32_t *slot_pos, int T, int k, int H, int64_t P,
                         void *dx, int64_t ld_dx, void *stream);

/*
 * Rows back to the tokens with the weights applied: out[t] = sum over j of
 * topk_weights[t][j] * ys[slot_pos[t*k + j]] (j ascending, one rounding).
 *   ys (device) [P][H]; topk_weights (device) fp32 [T][k], NULL = all 1;
 *   out (device) [T] rows at pitch ld_out >= H.  A token with no position in
 *   [0, P) gets a zero row.
 */
int moe_unpermute(int row_type, const void *ys, const int32_t *slot_pos, const float *topk_weights, int T, int k,
                  int H, int64_t P, void *out, int64_t ld_out, void *stream);

/*
 * Gradient of moe_unpermute: dys[slot_pos[t*k + j]] = topk_weights[t][j] *
 * dout[t] and dweights[t][j] = dout[t] . ys[slot_pos[t*k + j]] (0 for a
 * skipped position).  dout (device) [T] rows at pitch ld_dout; ys, dys
 * (device) [P][H]; dweights (device) fp32 [T][k]; zero_padding as in
 * moe_permute, for dys.  dys may be ys (each row is read before it is
 * written).
 */
int moe_unpermute_backward(int row_type, const void *dout, int64_t ld_dout, const void *ys, const int32_t *slot_pos,
                           const float *topk_weights, const int32_t *sorted_ids,
                           const int32_t *num_tokens_post_padded, int T, int k, int H, int64_t P, int zero_padding,
                           void *dys, float *dweights, void *stream);

/* Bytes of the workspace of moe_gemm_fp8_block and moe_wgrad_fp8_block: a
 * status word that the caller zeroes once before the first call; a call whose
 * wait runs out leaves MOE_ERR_TIMEOUT in it (read with moe_workspace_status). */
#define MOE_GEMM_BLOCK_WS_BYTES 64

/*
 * Matrix product of e4m3 operands with an fp32 scale per block of 128:
 *   D[m][n] = sum over b of a_scale[m, b] * b_scale[e][n/128][b] *
 *             sum over k in [128 b, 128 b + 128) of A[m][k] * B[e][n][k]
 * Dense (sorted_expert_ids and num_tokens_post_padded NULL, E = 1, block_m =
 * 0): all M rows, e = 0.  Grouped: rows in the order of moe_align_sort, e =
 * sorted_expert_ids[m / block_m], rows m < *num_tokens_post_padded (padding
 * rows included; later rows of D are left as they are); block_m 16, 32, 64 or
 * a multiple of 128.
 *   A (device) e4m3 [M][K]; a_scale (device) fp32 [M][ceil(K/128)]
 *   (a_scale_by_block = 0, as moe_quantize_fp8_act gives it) or
 *   [ceil(K/128)][M] (1, as moe_permute_fp8 gives it);
 *   B (device) e4m3 [E][N][K]; b_scale (device) fp32
 *   [E][ceil(N/128)][ceil(K/128)];
 *   D (device) rows of N at a pitch of ld_d, bf16 or fp32 (out_type);
 *   ws (device) MOE_GEMM_BLOCK_WS_BYTES.
 * K % 16 == 0; A and B on 16-byte boundaries; any M and N.  The gradient with
 * respect to A is the same product with B transposed.
 */
int moe_gemm_fp8_block(const uint8_t *A, const float *a_scale, int a_scale_by_block, const uint8_t *B,
                       const float *b_scale, int64_t M, int N, int K, int E, int block_m,
                       const int32_t *sorted_expert_ids, const int32_t *num_tokens_post_padded, int out_type, void *D,
                       int64_t ld_d, void *ws, size_t ws_bytes, void *stream);

/*
 * Weight gradient: for every expert e over its sorted rows p (whole blocks of
 * 128: expert e's rows start after ceil(expert_counts / 128) blocks of each
 * expert before it),
 *   D[e][m][n] (+)= sum over p of a_scale[p/128][m] A[m][p] * b_scale[p/128][n] B[n][p]
 *   A (device) e4m3 [M][P], a_scale (device) fp32 [P/128][M];
 *   B (device) e4m3 [N][P], b_scale (device) fp32 [P/128][N] (both as
 *   moe_quantize_fp8_act_t gives them: padding rows are zero codes);
 *   expert_counts (device) int32 [E], or NULL with E = 1: all P rows.  For
 *   rows sorted with a block_m above 128, pass the counts rounded up to
 *   multiples of block_m (the sort's segments);
 *   D (device) fp32 [E][M][N]; accumulate = 1 adds to D, 0 overwrites it (an
 *   expert without rows gets zeros).
 * P % 128 == 0, N % 4 == 0, E <= 1024, b_scale on a 16-byte boundary.
 */
int moe_wgrad_fp8_block(const uint8_t *A, const float *a_scale, const uint8_t *B, const float *b_scale, int64_t P,
                        int M, int N, int E, const int32_t *expert_counts, float *D, int accumulate, void *ws,
                        size_t ws_bytes, void *stream);

/*
 * Transposing quantiser for moe_wgrad_fp8_block: per column c and 128 rows,
 * scale = amax / 448 (1 if zero) and codes as moe_quantize_fp8_act (a
 * negative zero's code is that of zero).
 *   X (device) bf16 rows of C at a pitch of ld_x; with sorted_ids (device,
 *   int32 [R]) row p is X's row sorted_ids[p] / k, zero where sorted_ids[p] is
 *   outside [0, S) (padding); NULL: row p of X;
 *   num_rows (device) int32 or NULL: rows in use, at most R; rows past it
 *   inside its last block of 128 are zeros, later blocks are not written;
 *   q (device) e4m3 [C] rows at a pitch of ld_q >= ceil(R/128)*128;
 *   s (device) fp32 [ceil(R/128)][C].
 * C % 8 == 0, ld_x % 8 == 0, ld_q % 16 == 0, X and q on 16-byte boundaries.
 */
int moe_quantize_fp8_act_t(const void *X, int64_t ld_x, int64_t R, int C, const int32_t *sorted_ids, int S, int k,
                           const int32_t *num_rows, uint8_t *q, int64_t ld_q, float *s, void *stream);

#define MOE_GATE_NONE 0     /* no gate (1) */
#define MOE_GATE_CHANNEL 1  /* [H]: one value per column */
#define MOE_GATE_TOKEN 2    /* [T]: one value per row */
#define MOE_GATE_FULL 3     /* [T][H] */

/*
 * The norms before and after a block, fused with its gate and residual scale:
 *   n = h * rstd(h) * (w_post + weight_offset)    (n = h if w_post is NULL)
 *   y = residual + scale * gate * n
 *   z = y * rstd(y) * (w_pre + weight_offset)     (no z if w_pre is NULL)
 * with rstd(v) = 1 / sqrt(mean(v^2) + eps) over the row.  h is a block's
 * output, y the residual stream after it, z the next block's input (its
 * w_pre).
 *   h, residual, y, z (device) [T][H] of row_type; gate (device) of row_type,
 *   shaped by gate_kind; w_post, w_pre (device) [H] of row_type; rstd_h,
 *   rstd_y (device) fp32 [T] or NULL: kept for the backward.
 * y may be residual, and z may be h (each row is read before it is written;
 * the backward needs both, so not in training).
 * H <= 16384.
 */
int moe_block_norm(int row_type, const void *h, const void *residual, const void *gate, int gate_kind,
                   const void *w_post, const void *w_pre, int64_t T, int H, float scale, float weight_offset,
                   float eps, void *y, void *z, float *rstd_h, float *rstd_y, void *stream);

/* Workspace bytes of moe_block_norm_backward (0 on invalid input). */
size_t moe_block_norm_workspace_size(int64_t T, int H);

/*
 * Gradients of moe_block_norm for loss = sum(dy * y) + sum(dz * z):
 *   h, residual: the forward's inputs (residual with w_pre only; y is formed
 *   from them again, unrounded); rstd_h, rstd_y as it gave them (each
 *   required with its norm); dy (device) [T][H] or NULL (zero); dz
 *   (device) [T][H], with w_pre only (without it, dy is required);
 *   d_residual, dh (device) [T][H] of row_type;
 *   dgate (device): fp32 [H] or [T], or row_type [T][H]; with a gate only;
 *   dw_post, dw_pre (device) fp32 [H], each with its norm only;
 *   ws (device) moe_block_norm_workspace_size bytes.
 * d_residual may be dy, and dh may be h.
 */
int moe_block_norm_backward(int row_type, const void *h, const void *residual, const void *gate, int gate_kind,
                            const void *w_post, const void *w_pre, const float *rstd_h, const float *rstd_y,
                            const void *dy, const void *dz, int64_t T, int H, float scale, float weight_offset,
                            void *d_residual, void *dh, void *dgate, float *dw_post, float *dw_pre, void *ws,
                            size_t ws_bytes, void *stream);

/*
 * ------------------------------------------------------------------------
 * The rest of a training step: the gated feed-forward block that every token
 * passes, the cross entropy at the end, and the clipping of all gradients.
 *
 * Matrices of the first two are bf16 or fp16 (row_type; MOE_ROW_FP32 is
 * MOE_ERR_UNSUPPORTED) with fp32 sums; they start on 16-byte boundaries, H and
 * I are multiples of 8, and so are the pitches of rows.  T is any number, also
 * 0.  Each workspace starts with a status word that the caller zeroes once
 * before the first call; a call whose wait runs out leaves MOE_ERR_TIMEOUT in
 * it (read with moe_workspace_status).  A workspace serves one call at a time:
 * calls that may overlap on the GPU need one each.  Results are bitwise
 * reproducible.
 *
 * The tensor core drops what lies below the step of its running fp32 sum: of
 * terms of one sign 1.0e-5 of the sum over K = 4096, 7.6e-5 over 16384, 1.7e-4
 * over 32768.  No sum that stays in fp32 is longer than 2048 of K (loss, lse)
 * or 4096 rows (weight gradients) before it is added to others with rounding,
 * and none to a matrix in 16 bits longer than 32768, but for that of a
 * hidden row (gate | up and their gradients, over H; up to 128 tokens also
 * the output's, over I), which is one sum for any H and I.
 */
#define MOE_ACT_SILU 0       /* g sigmoid(g) */
#define MOE_ACT_GELU_TANH 1  /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
#define MOE_ACT_RELU 2       /* max(g, 0) */

/* Workspace bytes of moe_ffn (training = 0) and of moe_ffn_backward and a
 * moe_ffn that is given h (training = 1); 0 on invalid or unsupported sizes. */
size_t moe_ffn_workspace_size(int64_t T, int H, int I, int training);

/*
 * The gated feed-forward block (a shared expert next to the routed ones, or a
 * dense layer):
 *   g = x W_gate^T, u = x W_up^T, h = act(g) * u, out = add + h W_down^T
 *   x (device) [T] rows of H at a pitch of ld_x;
 *   W_gate_up (device) [2I][H], gate rows first; W_down (device) [H][I];
 *   add (device) [T] rows of H at a pitch of ld_add, or NULL (nothing is
 *   added; ld_add is ignored);
 *   out (device) [T] rows of H at a pitch of ld_out; it may be add, with its
 *   pitch, but no other bytes of add (MOE_ERR_INVALID_ARG);
 *   gu (device) [T][2I] (g | u of a row, rounded) and h (device) [T][I]: kept
 *   for the backward; both may be NULL, and gu with h given.
 * h is rounded to row_type before its product.  ws (device)
 * moe_ffn_workspace_size bytes.
 */
int moe_ffn(int row_type, int act, const void *x, int64_t ld_x, const void *W_gate_up, const void *W_down,
            const void *add, int64_t ld_add, int64_t T, int H, int I, void *gu, void *h, void *out, int64_t ld_out,
            void *ws, size_t ws_bytes, void *stream);

/*
 * Gradients of moe_ffn for loss = sum(dout * out) (that of add is dout):
 *   gu, h as the forward kept them; dout (device) [T] rows at a pitch of
 *   ld_dout;
 *   dx (device) [T] rows at a pitch of ld_dx; dW_gate_up (device) [2I][H] and
 *   dW_down (device) [H][I], of grad_type (row_type or MOE_ROW_FP32); each of
 *   the three may be NULL and is then not computed;
 *   accumulate = 1 adds the weight gradients to what is there (one rounding of
 *   the sum), 0 overwrites it;
 *   ws (device) moe_ffn_workspace_size(..., 1) bytes.
 * The gradients of g and u are rounded to row_type before their products; in
 * fp16 they are scaled by a power of two that brings the largest finite |dout|
 * to [1, 2) where it is smaller, so that fp16 holds them (a product dout W_down
 * with its factors of u and act' may then be up to 2^15 times that before it
 * overflows).
 */
int moe_ffn_backward(int row_type, int act, const void *x, int64_t ld_x, const void *W_gate_up, const void *W_down,
                     const void *gu, const void *h, const void *dout, int64_t ld_dout, int64_t T, int H, int I,
                     void *dx, int64_t ld_dx, int grad_type, int accumulate, void *dW_gate_up, void *dW_down, void *ws,
                     size_t ws_bytes, void *stream);

/* Workspace bytes of moe_vocab_loss (piece = 0), or of it and
 * moe_vocab_loss_backward with that piece; 0 on invalid or unsupported sizes.
 * It does not fall as T grows: a workspace for T rows serves fewer as well. */
size_t moe_vocab_loss_workspace_size(int64_t T, int H, int V, int piece);

/*
 * Softmax cross entropy over a vocabulary, from the hidden states:
 *   l = x W^T, lse[t] = log(sum over v of exp(l[t][v])),
 *   loss[t] = lse[t] - l[t][targets[t]]
 * and loss[t] = 0 for a row whose target is outside [0, V) (it is left out;
 * lse is computed for it all the same).  The logits are not kept.
 *   x (device) [T] rows of H at a pitch of ld_x; W (device) [V][H];
 *   targets (device) int32 [T]; loss, lse (device) fp32 [T];
 *   ws (device) moe_vocab_loss_workspace_size bytes.
 * Any V up to 2^24.
 */
int moe_vocab_loss(int row_type, const void *x, int64_t ld_x, const void *W, const int32_t *targets, int64_t T, int H,
                   int V, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream);

/*
 * Gradients of sum over t of dloss[t] * loss[t]:
 *   lse as the forward gave it; dloss (device) fp32 [T] (not read into
 *   anything for a row left out, whose x may be anything too);
 *   piece: columns of the vocabulary at a time, a multiple of 64 (the
 *   workspace grows with T * piece, the time with the number of pieces);
 *   dx (device) [T] rows at a pitch of ld_dx (zeros for a row left out); dW
 *   (device) [V][H] of grad_type (row_type or MOE_ROW_FP32); each may be NULL;
 *   accumulate = 1 adds dW to what is there.
 * The logits' gradients are rounded to row_type (scaled by a power of two so
 * that fp16 holds them) before their products.
 */
int moe_vocab_loss_backward(int row_type, const void *x, int64_t ld_x, const void *W, const int32_t *targets,
                            const float *lse, const float *dloss, int64_t T, int H, int V, int piece, void *dx,
                            int64_t ld_dx, int grad_type, int accumulate, void *dW, void *ws, size_t ws_bytes,
                            void *stream);

/* Workspace bytes of moe_grad_norm and moe_clip_gradients for n tensors. */
#define MOE_CLIP_WS_BYTES(n) ((((size_t)(n) + 511) / 512 + 1) * 9728)

/*
 * The 2-norm of all elements of n tensors: *norm (device fp32) = sqrt(sum of
 * squares), summed so that no square overflows or underflows.
 *   types, grads, numel (host) [n]: MOE_ROW_ type, device address (on a
 *   boundary of its elements) and number of elements of each tensor; they are
 *   read during the call.
 * n <= 65536; n = 0 gives 0.
 */
int moe_grad_norm(int n, const int *types, const void *const *grads, const int64_t *numel, float *norm, void *ws,
                  size_t ws_bytes, void *stream);

/*
 * The same, then out[i] = grads[i] * min(1, max_norm / (norm + eps)), each
 * element rounded once to its tensor's type.  out (host) [n]: device addresses; out[i]
 * may be grads[i], and overlaps no other tensor; nor does norm.  max_norm, eps >= 0.  A norm
 * that is infinite or a NaN scales as the formula says.
 */
int moe_clip_gradients(int n, const int *types, const void *const *grads, void *const *out, const int64_t *numel,
                       float max_norm, float eps, float *norm, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
