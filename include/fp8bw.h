/*
 * fp8bw.h -- C ABI of the blockwise-FP8 Transformer linear layer for NVIDIA B200
 * (sm_100a).
 *
 * The operations follow Puro-2B ("Poor Lab's Qwen2-1.5B Trained on RTX 5090 within
 * $5090", arXiv HTML part 3/7), section 3.2 "FP8 Mixed-Precision Training":
 * Transformer linear layers quantize their BF16 inputs and weights to E4M3
 * immediately before each GEMM.  Activations and their gradients carry a scale for
 * every 128 neighbouring elements in the direction the GEMM sums over, weights a
 * scale for every 128x128 tile; fprop, dgrad and wgrad all run in FP8 and the layer
 * hands a BF16 result back to the model.  Each block scale is the block's absolute
 * maximum divided by 448 (the largest finite E4M3 magnitude) in FP32, and values are
 * divided by it and rounded to nearest-even onto E4M3, saturating at +-448 (the
 * fine-grained recipe section 3.2 says it follows, DeepSeek-V3).
 *
 * Conventions for every entry point
 *   Pointers     Device (or managed) pointers on the calling thread's current CUDA
 *                device, unless stated otherwise; a host pointer or a buffer of
 *                another device returns FP8BW_EINVAL before anything is launched.
 *                The library never changes the current device.  The caller
 *                allocates and owns every buffer; the library never frees caller
 *                memory and keeps no pointer after the call returns.
 *   Layouts      Row-major [rows][cols].  BF16 tensors are IEEE bfloat16.  FP8 codes
 *                are E4M3 ("E4M3FN": bias 7, no infinities, NaN = S.1111.111).
 *                1x128 scale tensors are reduction-block-major, s[kb][row], so one
 *                tile's scales for one reduction block are contiguous.
 *   Sizes        Every dimension must be a positive multiple of 128 and at most
 *                FP8BW_MAX_DIM (else FP8BW_ESHAPE), except a token count: the M of
 *                fp8_quant_act, fp8_quant_act_t, fp8_quant_act_dual and of the FPROP
 *                and DGRAD GEMMs, and the reduction K of the WGRAD GEMM and of
 *                fp8_gemm_wgrad_acc32, which need only be a positive multiple of 16
 *                (the 16-byte row stride of token-major codes).  The last group of
 *                128 tokens may then be partial: its amax and scale are taken over
 *                the tokens present (the result of zero-padding the tokens to a
 *                multiple of 128, restricted to the tokens present), so token-wise
 *                scale arrays have ceil(tokens/128) rows.  The E8M0 entry points
 *                keep whole groups.  The few-token and mixture-of-experts calls state
 *                their own limits on tokens, experts and choices.
 *   Overlap      No output or workspace may share memory with another argument.  The
 *                few-token and mixture-of-experts calls check it (FP8BW_EINVAL).
 *   Alignment    Every pointer must be 16-byte aligned (else FP8BW_EALIGN).
 *   Streams      `stream` is a cudaStream_t (NULL = legacy default stream).  Work is
 *                enqueued asynchronously; no call but fp8bw_last_device_error
 *                synchronizes the stream.  Calls on distinct streams may run
 *                concurrently from different threads.  A call only enqueues
 *                kernels (it allocates nothing and waits for
 *                nothing), so it may be captured into a CUDA graph once its
 *                configuration has run eagerly on the device (the first launch of a
 *                configuration sets its shared-memory limit); fp8bw_last_device_error
 *                must stay outside a capture.
 *   Errors       Every call returns an fp8bw_status and never aborts or throws.
 *                Argument errors are reported before anything is launched.  A failed
 *                launch returns FP8BW_ECUDA.  The GEMMs and the activation quantizers
 *                bound every wait inside their kernels; a wait that runs out sets a
 *                per-device error word that fp8bw_last_device_error() reads.
 *   Inputs       Finite BF16 values.  Non-finite inputs give unspecified codes but
 *                never fault.
 *   Memory       The library allocates no device memory: the per-device error words
 *                are static device variables and TMA descriptors are passed by value.
 */
#ifndef FP8BW_H
#define FP8BW_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8BW_OK = 0,
    FP8BW_EINVAL = 1,      /* null pointer or bad mode; an output that overlaps another argument */
    FP8BW_EALIGN = 2,      /* a pointer is not 16-byte aligned */
    FP8BW_ESHAPE = 3,      /* a size is not a positive multiple of 128 (16 for a token count), or too large */
    FP8BW_ECUDA = 4,       /* a CUDA runtime call or kernel launch failed */
    FP8BW_ETIMEOUT = 5,    /* a bounded in-kernel wait ran out (from fp8bw_last_device_error) */
    FP8BW_EUNSUPPORTED = 6 /* the current device is not sm_100 */
} fp8bw_status;

typedef enum { FP8BW_FPROP = 0, FP8BW_DGRAD = 1, FP8BW_WGRAD = 2 } fp8bw_mode;

#define FP8BW_MAX_DIM (1 << 20)
#define FP8BW_FEW_TOKENS 64    /* most tokens of fp8_linear_few and fp8_moe_few */
#define FP8BW_MAX_EXPERTS 1024 /* most experts of a mixture-of-experts call */
#define FP8BW_MAX_CHOICES 32   /* most experts that one token may choose */

/*
 * fp8_quant_act -- 1x128 groups along the reduction dimension (section 3.2: the
 * scales of activations and of their gradients are taken over runs of 128 adjacent
 * elements in the direction the GEMM sums over).
 *   x  [M][K] BF16 in      q [M][K] E4M3 codes out      s [K/128][M] FP32 out
 * For each row m and block kb: amax = max |x[m][kb*128 .. kb*128+127]|,
 * s[kb][m] = amax / 448 (binary32 division), q = e4m3_rne_sat(x / s) with the
 * quotient rounded to binary32 first.  An all-zero group gets s = 0 and codes 0x00.
 * Used for X before fprop (K = in_features) and dY before dgrad (K = out_features).
 */
int fp8_quant_act(const void *x_bf16, int64_t M, int64_t K, uint8_t *q, float *s,
                  void *stream);

/*
 * fp8_quant_act_t -- the same groups taken along M (the token dimension), the
 * grouping wgrad needs because its reduction runs over tokens (section 3.2: wgrad
 * runs in FP8 on the layer's inputs and output gradients).
 *   x  [M][K] BF16 in      qt [K][M] E4M3 codes out (transposed)      st [ceil(M/128)][K] FP32 out
 * For each column k and block mb: the group is x[mb*128 .. mb*128+127][k];
 * st[mb][k] is its scale and qt[k][mb*128 + i] its codes.  Quantized from the BF16
 * tensor, not from the row-wise FP8 copy.
 */
int fp8_quant_act_t(const void *x_bf16, int64_t M, int64_t K, uint8_t *qt, float *st,
                    void *stream);

/*
 * fp8_quant_act_dual -- both activation layouts from one read of X (section 3.2:
 * wgrad reuses the FP8 copy of the layer input made for fprop; this call produces,
 * in one pass over the BF16 tensor, the row-wise copy fprop/dgrad consume and the
 * token-wise copy wgrad consumes).  Outputs are bit-identical to fp8_quant_act(x, M, K, q, s) and
 * fp8_quant_act_t(x, M, K, qt, st):
 *   x [M][K] BF16 in
 *   q [M][K], s [K/128][M]      1x128 groups along K
 *   qt [K][M], st [ceil(M/128)][K]    1x128 groups along M (codes transposed)
 */
int fp8_quant_act_dual(const void *x_bf16, int64_t M, int64_t K, uint8_t *q, float *s,
                       uint8_t *qt, float *st, void *stream);

/*
 * fp8_quant_weight -- 128x128 blocks (section 3.2: a weight's scales are taken
 * over square 128x128 tiles).
 *   w  [N][K] BF16 in      q [N][K] E4M3 out      s [N/128][K/128] FP32 out
 *   qt_or_null: if not NULL, also writes qt [K][N] = q transposed (same codes; a
 *   128x128 block keeps its one scale under transposition).
 */
int fp8_quant_weight(const void *w_bf16, int64_t N, int64_t K, uint8_t *q, float *s,
                     uint8_t *qt_or_null, void *stream);

/*
 * fp8_gemm_blockwise -- D[M][N] (BF16) = sum over a reduction of length K, with the
 * reduction cut into 128-long blocks kb.  For each kb the FP8 partial product
 * sum_{k in kb} qa*qb is accumulated in FP32 by the tensor cores and then promoted
 * into an FP32 running sum multiplied by (a-scale x b-scale) of that block; the sum
 * is rounded to BF16 (nearest-even) at the end.  Section 3.2: the forward, input-gradient
 * and weight-gradient GEMMs of these layers all run in FP8, and the model receives
 * BF16 results.
 *
 *   FPROP  Y  = X . W^T   a = Qx  [M][K], sa = [K/128][M]   (from fp8_quant_act(X))
 *                         b = Qw  [N][K], sb = [N/128][K/128] (from fp8_quant_weight(W))
 *                         M = tokens, K = in_features, N = out_features
 *   DGRAD  dX = dY . W    a = Qdy [M][K], sa = [K/128][M]   (from fp8_quant_act(dY))
 *                         b = Qw  [K][N], sb = [K/128][N/128] (the weight exactly as
 *                         fp8_quant_weight produced it, [out][in]; read transposed)
 *                         M = tokens, K = out_features, N = in_features
 *   WGRAD  dW = dY^T . X  a = Qdy^T [M][K], sa = [K/128][M] (from fp8_quant_act_t(dY))
 *                         b = Qx^T  [N][K], sb = [K/128][N] (from fp8_quant_act_t(X));
 *                         with K tokens not a multiple of 128, sa and sb have
 *                         ceil(K/128) rows, the last for the partial token group
 *                         M = out_features, K = tokens, N = in_features
 * d_bf16 [M][N] is written, never read.
 */
int fp8_gemm_blockwise(int mode, const uint8_t *a, const float *sa, const uint8_t *b,
                       const float *sb, void *d_bf16, int64_t M, int64_t N, int64_t K,
                       void *stream);

/*
 * fp8_gemm_wgrad_acc32 -- wgrad with FP32 gradient accumulation (the reading notes on
 * the same paper, section 2.3: gradient accumulation stays in FP32).  Same operands
 * and promotion as fp8_gemm_blockwise(FP8BW_WGRAD, ...), but the FP32 running sum is
 * added into dw32 instead of being rounded to BF16:
 *   dw32 [M][N] FP32, read and written: dw32 += sum over the token blocks
 * (M = out_features, N = in_features, K = tokens).  Calls that overlap on the GPU and
 * target the same dw32 may interleave their additions (the sum is the same up to
 * FP32 rounding order).
 */
int fp8_gemm_wgrad_acc32(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb,
                         float *dw32, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * ---- Power-of-two (E8M0) scales: the MXFP8 form of the recipe ----
 * Section 3.2: on the RTX 5090 the 128-blocks run through Transformer Engine's MXFP8
 * path, where every block scale is a power of two stored as an 8-bit exponent.
 * These entry points keep the groupings and code layouts above; each scale is the
 * E8M0 code e + 127 of 2^e, the smallest power of two with amax <= 448 * 2^e (e
 * clamped to [-127, 127]), and each value's code is the round-to-nearest-even of
 * x * 2^-e onto E4M3, which never saturates.  An all-zero group gets code 0 and
 * codes 0x00.
 *
 * Scale layout (the one the tensor cores read scale factors in): 512-byte blocks, one
 * per 128 rows x 128-deep reduction block; in a block the code of row r (0..127)
 * fills bytes 16 (r % 32) + 4 (r / 32) .. +3 (the code repeated four times, once per
 * 32-wide K step of the MMA).
 *   fp8_quant_act_e8m0       x[M][K] -> q[M][K]; s: [M/128][K/128] blocks, rows m
 *   fp8_quant_act_t_e8m0     x[M][K] -> qt[K][M]; st: [K/128][M/128] blocks, the
 *                            columns k of x as rows (the wgrad operand's rows)
 *   fp8_quant_act_dual_e8m0  both, from one read of x
 *   fp8_quant_weight_e8m0    w[N][K] -> q[N][K]; s: [N/128][K/128] blocks, every byte
 *                            of block (nb, kb) the code of that weight block;
 *                            optional qt[K][N]
 * Buffer sizes: M*K/32 bytes of scales for the activation forms, N*K/32 for the
 * weight.  Errors and pointer rules as above (every pointer 16-byte aligned).
 */
int fp8_quant_act_e8m0(const void *x_bf16, int64_t M, int64_t K, uint8_t *q, uint8_t *s_e8m0,
                       void *stream);
int fp8_quant_act_t_e8m0(const void *x_bf16, int64_t M, int64_t K, uint8_t *qt,
                         uint8_t *st_e8m0, void *stream);
int fp8_quant_act_dual_e8m0(const void *x_bf16, int64_t M, int64_t K, uint8_t *q,
                            uint8_t *s_e8m0, uint8_t *qt, uint8_t *st_e8m0, void *stream);
int fp8_quant_weight_e8m0(const void *w_bf16, int64_t N, int64_t K, uint8_t *q,
                          uint8_t *s_e8m0, uint8_t *qt_or_null, void *stream);

/*
 * fp8_gemm_blockwise_e8m0 -- fp8_gemm_blockwise with E8M0 scales (same modes and
 * operand layouts; sa / sb the scale blocks above: FPROP sa from fp8_quant_act_e8m0,
 * sb from fp8_quant_weight_e8m0; DGRAD the same weight blocks, read transposed;
 * WGRAD both from fp8_quant_act_t_e8m0).  The scales are applied
 * by the tensor cores (tcgen05.mma kind::mxf8f6f4.block_scale, each 128-block's
 * scale repeated over its four 32-wide K steps), so the reduction accumulates in one
 * FP32 accumulator and the result is rounded to BF16 once: D = sum_k
 * (qa 2^ea)(qb 2^eb).  d_bf16 [M][N] is written, never read.
 */
int fp8_gemm_blockwise_e8m0(int mode, const uint8_t *a, const uint8_t *sa_e8m0,
                            const uint8_t *b, const uint8_t *sb_e8m0, void *d_bf16, int64_t M,
                            int64_t N, int64_t K, void *stream);

/*
 * ---- Few tokens: the linear of a decode step ----
 *
 * fp8_linear_few -- Y[M][N] = X . W^T for M = 1 .. FP8BW_FEW_TOKENS tokens (any such
 * number): X is quantized within the call exactly as fp8_quant_act would (the same
 * codes and scales), then multiplied as by fp8_gemm_blockwise(FPROP).
 *   x [M][K] BF16     qw [N][K], sw [N/128][K/128] from fp8_quant_weight
 *   y [M][N] BF16, written, never read
 *   workspace: fp8_linear_few_workspace(M, K) bytes (may be NULL if that is 0), not
 *     shared with a call, or a captured graph, that may run at the same time
 * M out of range returns FP8BW_ESHAPE; the size function then returns 0.
 */
int64_t fp8_linear_few_workspace(int64_t M, int64_t K);
int fp8_linear_few(const void *x_bf16, const uint8_t *qw, const float *sw, void *y_bf16,
                   int64_t M, int64_t N, int64_t K, void *workspace, void *stream);

/*
 * ---- Mixture of experts ----
 * T tokens, E experts (1 .. FP8BW_MAX_EXPERTS), k choices per token (1 .. min(E,
 * FP8BW_MAX_CHOICES)); sizes outside these, or T outside 1 .. FP8BW_MAX_DIM, return
 * FP8BW_ESHAPE.  A choice is named by the pair index t * k + j.  An id outside [0, E)
 * marks a choice that is left out.
 *
 * fp8_moe_route -- softmax router.  ids[t][0..k-1] are the experts of the k largest
 * logits of row t, largest first, ties to the lowest expert; weights[t][j] is the
 * softmax of the logits, taken over the chosen experts (renorm != 0) or over all.
 *   logits [T][E] FP32 or (bf16 != 0) BF16      weights [T][k] FP32      ids [T][k] int32
 * A logit of -infinity or NaN is never chosen and has probability zero; a row with
 * fewer than k others gets id -1 and weight 0 in the places left.  +infinity counts as
 * the largest finite value of the logits' type.
 */
int fp8_moe_route(const void *logits, int bf16, int64_t T, int64_t E, int64_t k, int renorm,
                  float *weights, int32_t *ids, void *stream);

/*
 * fp8_moe_route_bwd -- gradient of the logits: with g_j = weights_j dweights_j and
 * G = sum_j g_j,  dlogits = [chosen] g - p G, where p is the softmax over the chosen
 * experts (renorm; zero elsewhere) or over all.  weights, ids and logits are those of
 * the forward call; dlogits [T][E] has the type of logits and is written whole.
 * A choice whose id the caller has since put outside [0, E) takes no part, and nor does its
 * expert's logit in a softmax over the chosen (to drop a choice there, leave its id and
 * give it dweights 0).  The softmax over all is taken from the first choice, which is the
 * largest of the forward call: p = w_0 exp(l - l_0), or anew where that one is left out.
 * With the choices in another order that is as good as w_0 (not if it has underflowed) and
 * exp(l - l_0) are.
 */
int fp8_moe_route_bwd(const float *dweights, const float *weights, const int32_t *ids,
                      const void *logits, int bf16, int64_t T, int64_t E, int64_t k, int renorm,
                      void *dlogits, void *stream);

/*
 * fp8_moe_plan -- lays the pairs out by expert for the grouped GEMMs: expert e gets the
 * blocks of 128 rows seg[e] .. seg[e + 1] - 1 (seg[0] = 0), as many as its pairs need,
 * and its pairs stand there in pair order.
 *   ids [T][k]      seg [E + 1] int32
 *   row [T][k] int32: the row of each pair, -1 for one that is left out
 *   src [rows] int32: the pair of each row, -1 for a row that no pair takes;
 *       rows = fp8_moe_plan_rows(T, E, k) holds any split of the pairs
 *   workspace: fp8_moe_plan_workspace(T, E, k) bytes, not shared with a call that may
 *       run at the same time
 * FP8BW_ESHAPE also if rows exceeds FP8BW_MAX_DIM.  The two size functions return 0 for
 * sizes that the call rejects.
 */
int64_t fp8_moe_plan_rows(int64_t T, int64_t E, int64_t k);
int64_t fp8_moe_plan_workspace(int64_t T, int64_t E, int64_t k);
int fp8_moe_plan(const int32_t *ids, int64_t T, int64_t E, int64_t k, int32_t *seg, int32_t *row,
                 int32_t *src, void *workspace, void *stream);

/*
 * fp8_gemm_grouped -- fp8_gemm_blockwise with one weight per expert.  The tokens (M of
 * FPROP and DGRAD, K of WGRAD; here a multiple of 128) are laid out by expert as above,
 * with zeros in the rows that no pair takes (so that they do not enter WGRAD):
 *   FPROP  a = Qx [M][K], sa = [K/128][M], b = Qw [E][N][K], sb = [E][N/128][K/128],
 *          d [M][N]
 *   DGRAD  a = Qdy [M][K], sa = [K/128][M], b = Qw [E][K][N], sb = [E][K/128][N/128],
 *          d [M][N]
 *   WGRAD  a = Qdy^T [M][K], sa = [K/128][M], b = Qx^T [N][K], sb = [K/128][N],
 *          d [E][M][N]: one weight gradient per expert, zero for one without blocks
 *   seg [E + 1] int32 on the device; entries are clamped to [0, blocks] and to their
 *   predecessors.  Rows of d in blocks that no expert owns are left as they were.
 * E times each of M (WGRAD), N and K (FPROP, DGRAD) must not exceed 2^30.
 */
int fp8_gemm_grouped(int mode, const uint8_t *a, const float *sa, const uint8_t *b,
                     const float *sb, const int32_t *seg, int64_t E, void *d_bf16, int64_t M,
                     int64_t N, int64_t K, void *stream);

/* fp8_gemm_grouped_wgrad_acc32 -- the grouped WGRAD added into FP32 main gradients:
 *   dw32 [E][M][N] FP32, read and written; an expert without blocks is not touched. */
int fp8_gemm_grouped_wgrad_acc32(const uint8_t *a, const float *sa, const uint8_t *b,
                                 const float *sb, const int32_t *seg, int64_t E, float *dw32,
                                 int64_t M, int64_t N, int64_t K, void *stream);

/*
 * fp8_moe_few -- all experts of a SwiGLU layer for T = 1 .. FP8BW_FEW_TOKENS tokens, in
 * two launches: for each token t and chosen expert e
 *   g, u = X[t] . W1_e^T (gate rows first, then up rows),  h = g / (1 + exp(-g)) * u,
 *   y[t] = sum_j weights[t][j] (h . W2_e^T)
 * X and h are quantized per 1x128 group (h from FP32, scale amax/448), each expert's
 * weights are read once, sums are FP32 and y is rounded to BF16 once.
 *   x [T][H] BF16
 *   w1 [E][2I][H], s1 [E][2I/128][H/128]     w2 [E][H][I], s2 [E][H/128][I/128]
 *     (fp8_quant_weight of the matrices stacked by expert; a call of it takes at most
 *     FP8BW_MAX_DIM rows, and its scales and codes of further experts simply follow)
 *   ids, weights [T][k] as from fp8_moe_route; a token that names an expert twice gives
 *     it the sum of the two weights; one whose choices are all left out gets y = 0
 *   y [T][H] BF16, written, never read
 *   workspace: fp8_moe_few_workspace(T, k, H, I) bytes (0 for sizes that the call
 *     rejects); calls that may run at the same time need one each, as do two captured
 *     graphs that may
 * H and I multiples of 128; E * 2I and E * H at most 2^30.
 */
int64_t fp8_moe_few_workspace(int64_t T, int64_t k, int64_t H, int64_t I);
int fp8_moe_few(const void *x_bf16, const uint8_t *w1, const float *s1, const uint8_t *w2,
                const float *s2, const int32_t *ids, const float *weights, void *y_bf16,
                int64_t T, int64_t E, int64_t k, int64_t H, int64_t I, void *workspace,
                void *stream);

/* Human-readable name of a status code (static string). */
const char *fp8bw_status_string(int status);

/* Synchronizes `stream`, then reads and clears the current device's error word:
 * FP8BW_OK, or FP8BW_ETIMEOUT if a bounded in-kernel wait ran out since the last
 * call (the GEMM or quantizer whose wait ran out returned early and its output is
 * undefined). */
int fp8bw_last_device_error(void *stream);

/* Self-test of the failure-detection path (no counterpart in the paper; it checks
 * this library's own bounded waits).  Launches one warp on `stream` that waits, with
 * the GEMM's bounded wait, on a barrier nothing arrives on; after limit_us
 * microseconds (1 .. 1e6, else FP8BW_EINVAL) the wait gives up, records a timeout in
 * the device error word and the kernel returns.  fp8bw_last_device_error() then
 * reports FP8BW_ETIMEOUT once; the device stays usable. */
int fp8bw_selftest_wait_timeout(int64_t limit_us, void *stream);

/* Library version, e.g. "fp8bw 0.1 sm_100a". */
const char *fp8bw_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FP8BW_H */
