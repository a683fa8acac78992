/*
 * spear.h -- C ABI of libspear: a W4A16 linear layer with a per-token gated
 * Error Compensator (EC), written for AMD Instinct MI355X (gfx950).
 *
 * Sources (page title, then section):
 *   "SPEAR: A System for Post-Quantization Error-Adaptive Recovery Enabling
 *   Efficient Low-Bit LLM Serving"
 *     - authors' abstract (fugumt.com record of arXiv 2606.11244): 4-bit
 *       per-channel weights, ECs modulated by per-token gates, the EC fused
 *       into the low-bit GEMM;
 *     - gist.science technical summary, section 2.1 A: the EC maps x to rank r
 *       with A, gates it per token, maps back with B; the effective weight is
 *       W + alpha B diag(gamma) A;
 *     - same summary, section 2.2 A: phase-aware dispatch -- at decode the EC
 *       is fused into the GEMM epilogue (one kernel), at prefill it runs
 *       semi-fused;
 *     - same summary, section 3.1: per-channel 4-bit quantizers (RTN, GPTQ,
 *       AWQ, OmniQuant) -- the layer takes their codes as given.
 *
 * Computation (all shapes row-major; tokens are rows):
 *   x     [M][K]  bf16 activations
 *   W     [N][K]  4-bit codes u (packed, see spear_pack_w4), per-output-channel
 *                 scale s[N] (fp32) and zero point z[N] (uint8; 8 when NULL)
 *   A     [r][K]  bf16 EC down-projection
 *   B     [N][r]  bf16 EC up-projection (alpha folded in)
 *   w_g   [K]     bf16 gate weights, b fp32 gate bias
 *
 *   z_m   = b + sum_k x[m][k] w_g[k]                  (gate logit, fp64 sum)
 *   g_m   = 1 / (1 + exp(-z_m))                       (fp32)
 *   act_m = hard ? (z_m > log(tau / (1 - tau))) : 1   (a tie skips)
 *   u_m[j] = sum_k A[j][k] x[m][k]                     (EC down-projection)
 *   y[m][n] = s_n sum_k x[m][k] (u[n][k] - z_n)
 *           + act_m g_m sum_j B[n][j] u_m[j]
 *
 * Optional vector gate (the summary's diag(gamma(Ax)), gamma a bottleneck MLP
 * on the rank-r projection): with gate_h > 0 the EC term becomes
 *           act_m g_m alpha sum_j B[n][j] gamma_j(u_m) u_m[j],
 *   gamma(u) = sigmoid(W2 relu(W1 u + c1) + c2),  W1 [h][r], c1 [h],
 *   W2 [r][h], c2 [r] (fp32).  With b = +inf (g = 1) and a soft gate this is
 *   the summary's W + alpha B diag(gamma(Ax)) A.
 *
 * Conventions shared by every entry point:
 *   - Data pointers are DEVICE pointers unless stated otherwise.  The caller
 *     allocates and owns all memory, including the workspace.  The library
 *     never allocates device memory.
 *   - State: the workspace carries state from call to call (launch counters
 *     and tagged partial results, see spear_workspace_init), so it is zeroed
 *     once and then left to the library.  The only other state is the
 *     process-wide wait limit (spear_set_wait_limit) and a per-device cache of
 *     the gfx950 check.
 *   - Every call enqueues work on `stream` (a hipStream_t; NULL is the null
 *     stream) and returns without synchronising.  Faults inside a kernel
 *     surface at the caller's next synchronisation.
 *   - Arguments are validated on the host before any HIP call; a call that
 *     fails validation has enqueued nothing.  A call that makes several
 *     launches and returns SPEAR_E_HIP may have enqueued the launches before
 *     the one that failed; the outputs are then unspecified.
 *   - Entry points may be called from several threads at once.  A workspace
 *     must not be shared by calls that may run concurrently (for example on
 *     two streams).
 */
#ifndef SPEAR_H
#define SPEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEAR_ABI_VERSION 2

typedef uint16_t spear_bf16; /* raw bfloat16 bits */
typedef int32_t spear_status;

#define SPEAR_OK            0
#define SPEAR_E_NULL       -1 /* a required pointer is NULL                      */
#define SPEAR_E_SHAPE      -2 /* a size is out of range (see each entry point)   */
#define SPEAR_E_ALIGN      -3 /* a pointer is not aligned as required            */
#define SPEAR_E_ARG        -4 /* an enum is out of range or tau is NaN           */
#define SPEAR_E_WORKSPACE  -5 /* workspace smaller than spear_w4_linear_workspace_size */
#define SPEAR_E_HIP        -6 /* a HIP runtime call or kernel launch failed      */
#define SPEAR_E_DEVICE     -7 /* the current device is not gfx950                */

/* Code kinds accepted by spear_pack_w4. */
#define SPEAR_CODES_S4 0 /* int8 codes q in [-8, 7]; stored offset-binary u = q + 8, zero point 8 */
#define SPEAR_CODES_U4 1 /* uint8 codes u in [0, 15]; zero point per channel */

/* Output element types of spear_w4_linear. */
#define SPEAR_OUT_BF16 0 /* y rounded to bf16 (round to nearest even) */
#define SPEAR_OUT_F32  1 /* y in fp32 */

/* Kernel-path selection of spear_w4_linear_path. */
#define SPEAR_PATH_AUTO          0 /* decode path for M <= 16, prefill path otherwise   */
#define SPEAR_PATH_DECODE        1 /* M <= 16: one launch, EC fused into the epilogue   */
#define SPEAR_PATH_PREFILL       2 /* any M: EC pre-pass, then the MFMA GEMM whose
                                      epilogue applies the EC.  Tiles are 64 x 64
                                      up to 128 tokens, 256 x 128 above.  With few
                                      output tiles K is split and a second launch
                                      adds the slices.  With 64 x 64 tiles or a K
                                      split, and fewer than 2048 tokens, the
                                      pre-pass runs as the first blocks of the
                                      GEMM's launch                                  */
#define SPEAR_PATH_DECODE_2PASS  3 /* M <= 16: EC pre-pass, then the decode kernel      */
#define SPEAR_PATH_PREFILL_LARGE 4 /* any M: EC pre-pass, then the 256 x 128-tile MFMA
                                      GEMM over whole K (the prefill path's choice
                                      when there are enough tiles)                     */

/* Largest EC rank accepted; the rank must also be a multiple of 8. */
#define SPEAR_MAX_RANK 256
/* Largest hidden width of the optional vector gate's MLP. */
#define SPEAR_MAX_GATE_HIDDEN 64

/* Quantised weights (all device pointers). */
typedef struct spear_w4 {
    const uint8_t *packed; /* [N][K/2] from spear_pack_w4; 16-byte aligned          */
    const float *scales;   /* [N] per-channel scale s_n; 4-byte aligned              */
    const uint8_t *zeros;  /* [N] zero points in [0, 15], or NULL for zero point 8   */
    int64_t N;             /* output channels, >= 1                                   */
    int64_t K;             /* input channels, >= 32 and a multiple of 32              */
} spear_w4;

/* Error compensator and gate (device pointers; the *_out fields are optional). */
typedef struct spear_ec {
    const spear_bf16 *A;      /* [r][K]; 16-byte aligned                            */
    const spear_bf16 *B;      /* [N][r]; 16-byte aligned                            */
    const spear_bf16 *w_gate; /* [K]; 16-byte aligned                               */
    float b;                  /* gate bias (-inf gives g = 0)                       */
    float tau;                /* hard-gate threshold on g; must not be NaN          */
    int32_t hard;             /* 0: every token takes the EC; 1: only z_m > logit(tau) */
    int32_t r;                /* rank, a multiple of 8 in [8, SPEAR_MAX_RANK]       */
    float *g_out;             /* optional [M]: g_m                                  */
    int32_t *idx_out;         /* optional [M]: ascending indices of active tokens   */
    int32_t *n_active_out;    /* optional [1]: number of active tokens              */
    /* Optional vector gate (gate_h == 0: none; the other fields are then unused).
       Source: summary section 2.1 A.  All fp32, 4-byte aligned device pointers. */
    int32_t gate_h;           /* hidden width h, 0 or 1 .. SPEAR_MAX_GATE_HIDDEN     */
    float alpha;              /* scale of the vector-gated EC term                  */
    const float *gate_w1;     /* [h][r]                                             */
    const float *gate_c1;     /* [h]                                                */
    const float *gate_w2;     /* [r][h]                                             */
    const float *gate_c2;     /* [r]                                                */
} spear_ec;

/*
 * spear_pack_w4 -- pack 4-bit codes for spear_w4_linear.
 *   codes     [N][K] int8 (SPEAR_CODES_S4) or uint8 (SPEAR_CODES_U4); 16-byte aligned.
 *   packed    [N][K/2] output, 16-byte aligned: each row is a run of little-endian
 *             32-bit words, word w holding u[n][8w .. 8w+7]; nibble position p
 *             (bits 4p .. 4p+3) holds u[n][8w + perm[p]], perm = (0,2,4,6,1,3,5,7):
 *             byte 0 holds codes 0 and 2 (low, high nibble), byte 1 codes 4 and 6,
 *             byte 2 codes 1 and 3, byte 3 codes 5 and 7 (u = q + 8 for signed
 *             codes).  A shift and a mask then give bf16 pairs in natural order.
 *   bad_codes optional device int32 counter; the number of out-of-range codes is
 *             ADDED to it.  Out-of-range codes are packed as their low 4 bits.
 * Shapes: N >= 1, K >= 32, K % 32 == 0.  Source: the summary's section 3.1
 * (per-channel 4-bit codes from any quantizer); the layout is this library's.
 */
spear_status spear_pack_w4(const void *codes, int32_t code_kind, int64_t N, int64_t K,
                           uint8_t *packed, int32_t *bad_codes, void *stream);

/*
 * spear_gate -- the per-token gate and hard-gate token selection alone.
 *   x [M][K] bf16 (16-byte aligned), w_gate [K] bf16 (16-byte aligned).
 *   g        [M] fp32 output, g_m = sigmoid(z_m).
 *   idx      [M] int32 output; entries [0, n_active) are the active tokens in
 *            ascending order, the rest are left unspecified.
 *   n_active [1] int32 output.
 * Shapes: M >= 0 (M == 0 writes n_active = 0), K >= 32, K % 32 == 0.
 * Sources: abstract (per-token gates); summary section 2.1 A (input-dependent gate).
 */
spear_status spear_gate(const spear_bf16 *x, int64_t M, int64_t K, const spear_bf16 *w_gate,
                        float b, float tau, int32_t hard, float *g, int32_t *idx,
                        int32_t *n_active, void *stream);

/*
 * spear_w4_linear_workspace_size -- bytes of workspace spear_w4_linear needs
 * for these sizes (r = 0 when there is no EC).  Host-only, no HIP call.  The
 * size serves every smaller M with the same N, K and r; it is not monotone in
 * N or K (the GEMM's K split depends on the layer's shape), so a workspace
 * shared by layers of several shapes takes the largest of their sizes.
 */
size_t spear_w4_linear_workspace_size(int64_t M, int64_t N, int64_t K, int32_t r);

/*
 * spear_workspace_init -- zero a workspace before its first use (a workspace
 * allocated zero-filled needs no init).  Between calls the workspace holds
 * library state: a launch counter that every fused decode launch advances (its
 * producers tag the partial results they hand to the epilogues with it) and
 * the tagged partials themselves, so it is zeroed once, not per call, and
 * must not be modified by the caller afterwards.  Tags repeat after 2^32
 * fused launches on one workspace; re-initialise it before that.
 * ws: device pointer, 256-byte aligned; bytes >= 256.
 */
spear_status spear_workspace_init(void *ws, size_t bytes, void *stream);

/*
 * spear_w4_linear -- y = x W^T (dequantised) + gated EC; ec == NULL gives the
 * plain W4 linear.  Sources: abstract; summary sections 2.1 A and 2.2 A.
 *   x         [M][K] bf16, 16-byte aligned.  M >= 0 (M == 0 does nothing but
 *             write *n_active_out = 0 when that pointer is given).
 *   w         weights; w->N >= 1, w->K >= 32, w->K % 32 == 0.
 *   ec        EC and gate, or NULL.
 *   y         [M][N] output, fp32 or bf16 per out_dtype; 16-byte aligned.
 *   workspace device scratch of at least spear_w4_linear_workspace_size bytes,
 *             256-byte aligned, zeroed once (see spear_workspace_init).
 * Dispatch: M <= 16 takes the decode path (one launch; the gate, token
 * selection and EC down-projection run in the same kernel as the weight
 * stream, and the EC is applied in its epilogue); M > 16 takes the prefill
 * path (an EC pre-pass, then the MFMA GEMM with the EC in its epilogue).
 * The vector gate is formed where v is formed: in the fused decode kernel's
 * epilogue (ranks up to 32; larger ranks take the pre-pass form of the decode
 * path, two launches), or at the end of the EC pre-pass.
 * The result does not depend on the path beyond fp32 rounding order.
 * SPEAR_E_SHAPE also when a decode path's workspace layout would place the
 * regions its kernels use beyond 4 GiB (their offsets travel as 32-bit values;
 * only layers with billions of channel groups times K ranges come near).
 */
spear_status spear_w4_linear(const spear_bf16 *x, int64_t M, const spear_w4 *w,
                             const spear_ec *ec, void *y, int32_t out_dtype,
                             void *workspace, size_t ws_bytes, void *stream);

/* spear_w4_linear with an explicit SPEAR_PATH_* (the decode paths need M <= 16). */
spear_status spear_w4_linear_path(const spear_bf16 *x, int64_t M, const spear_w4 *w,
                                  const spear_ec *ec, void *y, int32_t out_dtype,
                                  void *workspace, size_t ws_bytes, int32_t path,
                                  void *stream);

/*
 * spear_w4_linear_semifused -- the prefill layer in the summary's semi-fused
 * form (section 2.2 A: at prefill the EC runs as a separate kernel beside the
 * low-bit GEMM, the two joined through the graph of the step).  On
 * `aux_stream`, forked from `stream` by ev_fork: the EC pre-pass (gate logit,
 * selection, v = g u, vector gate) and a ballot compaction of the active
 * tokens.  On `stream`, meanwhile: the plain W4 GEMM into y.  Then `stream`
 * waits for ev_join (recorded on aux_stream after the compaction) and one
 * more kernel adds B v into the rows of the active tokens only.  No kernel
 * waits on another stream's kernel; the fork and the join are event
 * dependencies, which HIP graph capture of `stream` records as graph edges.
 *   Arguments as for spear_w4_linear, except: y is fp32 only ([M][N]); ec may
 *   be NULL (then: the plain GEMM on `stream`, nothing on aux_stream);
 *   aux_stream is a stream other than `stream`; ev_fork and ev_join are
 *   hipEvent_t handles owned by the caller (created with timing disabled is
 *   enough), not used concurrently by other calls.  The workspace is that of
 *   spear_w4_linear (spear_w4_linear_workspace_size).
 */
spear_status spear_w4_linear_semifused(const spear_bf16 *x, int64_t M, const spear_w4 *w,
                                       const spear_ec *ec, float *y, void *workspace,
                                       size_t ws_bytes, void *stream, void *aux_stream,
                                       void *ev_fork, void *ev_join);

/* Activations of spear_epilogue and spear_experts. */
#define SPEAR_ACT_NONE      0 /* t                                                     */
#define SPEAR_ACT_RELU      1 /* max(t, 0)                                             */
#define SPEAR_ACT_SILU      2 /* t / (1 + exp(-t))                                     */
#define SPEAR_ACT_GELU      3 /* t / 2 (1 + erf(t / sqrt 2))                           */
#define SPEAR_ACT_GELU_TANH 4 /* t / 2 (1 + tanh(sqrt(2 / pi) (t + 0.044715 t^3)))     */

/* What follows the layer's output in spear_w4_linear_epilogue (device pointers). */
typedef struct spear_epilogue {
    const float *bias;    /* [N], added to the layer's output (W4 and EC), or NULL; 4-byte aligned */
    const void *residual; /* [M][N], or [M][N/2] with the gated pair, of y's type, added last, or
                             NULL; 16-byte aligned; may be y itself (each element is read before
                             it is written)                                                      */
    int32_t act;          /* SPEAR_ACT_*                                                           */
    int32_t glu;          /* 1: the gated pair below (N even); 0: every channel by itself          */
} spear_epilogue;

/*
 * spear_w4_linear_epilogue -- the layer with bias, activation and residual in
 * its kernels' epilogue, with t the layer's output (W4 and EC, fp32):
 *   glu == 0:  y[m][n] = act(t[m][n] + bias[n]) + residual[m][n]          (N channels)
 *   glu == 1:  y[m][i] = act(t[m][2i] + bias[2i]) (t[m][2i+1] + bias[2i+1])
 *                        + residual[m][i]                                 (N / 2 channels)
 * The gated pair is a decoder's gate and up projection as one layer: row 2i of
 * the weights (codes, scales, zero points, bias, B) is the gate's row i and row
 * 2i + 1 the up projection's, interleaved once before spear_pack_w4.  All of
 * the epilogue is in fp32, rounded once to y's type.  Other arguments, the
 * workspace and the paths are those of spear_w4_linear_path; ep is required.
 * SPEAR_PATH_AUTO with M <= 16, a compensator of rank 64 at most and no gate
 * vector of its own takes the compensator's first half as a launch of its own
 * where the layer is wide (t may then differ from spear_w4_linear's in the order
 * of its sums).
 * An expired wait makes the outputs NaN here too (NaN passes through every
 * activation).
 */
spear_status spear_w4_linear_epilogue(const spear_bf16 *x, int64_t M, const spear_w4 *w,
                                      const spear_ec *ec, const spear_epilogue *ep, void *y,
                                      int32_t out_dtype, void *workspace, size_t ws_bytes,
                                      int32_t path, void *stream);

/* Scores of spear_router. */
#define SPEAR_SCORE_SOFTMAX 0 /* s_e = exp(z_e) / sum exp(z)  */
#define SPEAR_SCORE_SIGMOID 1 /* s_e = 1 / (1 + exp(-z_e))    */
/* Most experts, choices a token, and expert groups. */
#define SPEAR_MAX_EXPERTS 512
#define SPEAR_MAX_TOPK    32
#define SPEAR_MAX_GROUPS  64

/* Router of a mixture of experts (device pointers). */
typedef struct spear_router {
    const spear_bf16 *w;  /* [E][K]; 16-byte aligned                                              */
    const float *bias;    /* [E] added to the scores for the choice alone, or NULL; 4-byte aligned */
    int32_t E;            /* experts, 1 .. SPEAR_MAX_EXPERTS                                       */
    int32_t topk;         /* experts a token takes, 1 .. SPEAR_MAX_TOPK                            */
    int32_t score;        /* SPEAR_SCORE_*                                                         */
    int32_t n_group;      /* groups of E / n_group consecutive experts, 1 .. SPEAR_MAX_GROUPS      */
    int32_t topk_group;   /* groups kept, 1 .. n_group, holding at least topk experts              */
    int32_t group_best;   /* a group counts the sum of its best 1 or 2 choices                     */
    int32_t renorm;       /* 1: the chosen scores are divided by their sum                         */
    float scale;          /* factor of the weights; must not be NaN                                */
} spear_router;

/*
 * spear_route -- which experts each token takes, and with what weights:
 *   z_me = sum_k x[m][k] w[e][k]    s = softmax or sigmoid of z    c = s + bias
 *   kept groups: the topk_group largest by the sum of their group_best largest c
 *   ids[m][0..topk): the experts of the kept groups with the largest c, in
 *     descending order; ties (of experts and of groups) go to the lowest index
 *   weights[m][j] = scale * s[ids[m][j]]  (/ sum_j s with renorm)
 * The choice is the one of logits summed and scores compared in fp64, so it
 * does not hang on an fp32 rounding.  The weights may come of logits summed in
 * fp32: a logit is off by at most (58 + K / 256) 2^-23 |x_m| |w_e| (2-norms),
 * a weight by twice that relative, then one rounding to fp32.  An expert whose
 * c is NaN or -inf (a bias of -inf takes an expert out) is never chosen: a
 * slot left without an expert gets id -1 and weight 0, and takes no part in
 * the sum.  Scores that sum to zero give weights of zero.
 *   x [M][K] bf16, 16-byte aligned; 0 <= M <= 2^27 (0 does nothing); K >= 32,
 *     K % 32 == 0.
 *   weights [M][topk] fp32, ids [M][topk] int32 outputs, 4-byte aligned.
 *   workspace device scratch of spear_route_workspace_size bytes, 256-byte
 *             aligned; needs no zeroing and holds nothing between calls.
 */
size_t spear_route_workspace_size(int64_t M, int32_t E);
spear_status spear_route(const spear_bf16 *x, int64_t M, int64_t K, const spear_router *router,
                         float *weights, int32_t *ids, void *workspace, size_t ws_bytes,
                         void *stream);

/*
 * Experts of a mixture (device pointers): two 4-bit layers an expert, the
 * expert index outermost.  The codes are spear_pack_w4's of [E * NU][K] and
 * [E * N][I]; NU = 2 I with the gated pair (rows 2i and 2i + 1 as in
 * spear_epilogue), else I.
 */
typedef struct spear_experts {
    const uint8_t *up;         /* [E][NU][K/2]; 16-byte aligned           */
    const float *up_scales;    /* [E][NU]                                 */
    const uint8_t *up_zeros;   /* [E][NU], or NULL for zero point 8       */
    const float *up_bias;      /* [E][NU], or NULL                        */
    const uint8_t *down;       /* [E][N][I/2]; 16-byte aligned            */
    const float *down_scales;  /* [E][N]                                  */
    const uint8_t *down_zeros; /* [E][N], or NULL for zero point 8        */
    const float *down_bias;    /* [E][N], or NULL                         */
    int64_t K;                 /* input channels, 32 .. 2^31, a multiple of 32 */
    int64_t I;                 /* inner channels, 32 .. 2^25, a multiple of 32 */
    int64_t N;                 /* output channels, 1 .. 2^25              */
    int32_t E;                 /* 1 .. SPEAR_MAX_EXPERTS                  */
    int32_t act;               /* SPEAR_ACT_* between the two layers      */
    int32_t glu;               /* 1: the gated pair; 0: act alone         */
} spear_experts;

/*
 * spear_w4_experts -- the routed tokens through their experts:
 *   h_mj   = act(up_e x_m + up_bias_e)    (or the gated pair), e = ids[m][j]
 *   y[m]   = residual[m] + sum_j weights[m][j] (down_e h_mj + down_bias_e)
 * with fp32 sums; h is rounded to bf16 (the layers' activation type), y once to
 * bf16.  A slot whose id is outside [0, E) (an expert elsewhere, a padded
 * token, a slot spear_route left empty) adds nothing, whatever its weight; an
 * expert may occur twice in a token.
 *   x [M][K] bf16, ids [M][topk] int32, weights [M][topk] fp32,
 *   residual [M][N] bf16 or NULL (may be y itself), y [M][N] bf16; x, residual
 *   and y 16-byte aligned.  y may not overlap any other input.
 *   M >= 0 (0 does nothing), 1 <= topk <= SPEAR_MAX_TOPK, M topk <= 2^30.
 *   workspace device scratch of spear_w4_experts_workspace_size bytes (0 for
 *             sizes out of range), 256-byte aligned; needs no zeroing and holds
 *             nothing between calls.
 */
size_t spear_w4_experts_workspace_size(int64_t M, int32_t topk, int32_t E, int64_t I, int64_t N);
spear_status spear_w4_experts(const spear_bf16 *x, int64_t M, const spear_experts *w,
                              const int32_t *ids, const float *weights, int32_t topk,
                              const spear_bf16 *residual, spear_bf16 *y, void *workspace,
                              size_t ws_bytes, void *stream);

/*
 * Attention over a cache held in 4 bits: the plan of a serving step, rotary
 * positions, the write into the cache, and the attention that reads it.
 *
 * The cache holds a channel as e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) and
 * one power of two for every block of 32 channels of a token's head.  With a
 * the largest |x| of a block and f = floor(log2 a):
 *   e = f - 2, or f - 1 where a / 2^f >= 1.75 (a rounded to two significant bits
 *       has the next exponent), held within [-125, 125]; a = 0 gives -125
 *   code = x / 2^e rounded to the nearest level, ties to the even code, at most 6
 *       (a rotated key may lie beyond fp32's range, and is finite all the same)
 *   scale byte = e + 127;  a block with a NaN or an infinity: 255, and reads NaN
 * so that a value that is read back is exact in bf16.  Pages of P tokens, a
 * head's tokens side by side (device pointers, each 16-byte aligned):
 */
typedef struct spear_kv4 {
    uint8_t *k_codes;   /* [pages][heads][P][D/2], the lower channel in the low nibble */
    uint8_t *k_scales;  /* [pages][heads][D/32][P]                                      */
    uint8_t *v_codes;   /* as k_codes                                                   */
    uint8_t *v_scales;  /* as k_scales                                                  */
    int64_t pages;      /* 1 .. 2^31 - 1                                                */
    int32_t heads;      /* key heads, 1 .. SPEAR_MAX_HEADS                              */
    int32_t D;          /* channels of a head: 64, 96, 128, 192 or 256                  */
    int32_t P;          /* tokens of a page: 16, 32, 64, 128, 256, 512 or 1024          */
} spear_kv4;

#define SPEAR_MAX_HEADS    1024 /* query or key heads                     */
#define SPEAR_MAX_REQUESTS 4096 /* requests of a step                     */
#define SPEAR_MAX_ROWS     ((int64_t)1 << 23) /* token rows of a step     */
#define SPEAR_MAX_CONTEXT  ((int64_t)1 << 30) /* tokens that a table's row can hold */

/*
 * What spear_kv4_plan makes of a step's lengths (device pointers).
 */
typedef struct spear_kv4_step {
    int32_t *q_start;   /* [B + 1] first row of each request                          */
    int32_t *kv_len;    /* [B] tokens in the cache after the step                     */
    int32_t *positions; /* [T] position of each row in its request                    */
    int64_t *slots;     /* [T] page * P + place in the page; 8-byte aligned           */
    int32_t *n_left;    /* [1] pages left in the free list                            */
    int32_t *status;    /* [2] pages that the free list lacked; pages that the rows of
                           the table have no room for                                  */
} spear_kv4_step;

/*
 * spear_kv4_plan -- block table and slot map of a serving step, from the
 * requests' lengths alone (nothing is read back by the host).
 *   cached [B]  tokens that each request has in the cache (negative: 0)
 *   fresh  [B]  tokens that the step adds to each (negative: 0); 0 is a request
 *               that pauses
 *   table  [B][width]  each request's pages in order, updated in place: the first
 *               ceil(cached / P) entries of a row are read, new pages are written
 *               behind them, the rest of the row is left as it is
 *   free_pages [n_pages]  page ids, a stack of which the first *n_free are free
 *               (clamped to [0, n_pages]); pages are taken from its end, in the
 *               requests' order.  n_free is read, what is left goes to n_left
 *   T           rows of the step (a captured step keeps the largest)
 * The requests' fresh tokens lie in the rows one behind the other.  Fresh tokens
 * past T rows are dropped: q_start, kv_len and the pages count the others.  Rows
 * behind the last token get position 0 and slot -1 (no place in the cache), as
 * do tokens of a page that the free list lacked (its table entry is -1 too) or
 * that the table has no room for; the latter two keep their positions.
 *   0 <= B <= SPEAR_MAX_REQUESTS, 0 <= T <= SPEAR_MAX_ROWS, width >= 1,
 *   width * P <= SPEAR_MAX_CONTEXT; a request's tokens are less than 2^31.
 *   The outputs overlap neither each other nor an input: two steps alternate
 *   between two sets of them.
 */
spear_status spear_kv4_plan(const int32_t *cached, const int32_t *fresh, int32_t B, int32_t *table,
                            int64_t width, const int32_t *free_pages, int64_t n_pages,
                            const int32_t *n_free, int64_t T, int32_t P,
                            const spear_kv4_step *step, void *stream);

/* Which channels of a head a rotation pairs. */
#define SPEAR_ROPE_HALF  0 /* channel i with channel i + rot / 2 */
#define SPEAR_ROPE_PAIRS 1 /* channel 2i with channel 2i + 1     */

/* Rotary positions: the first rot channels of every head, the others as they are. */
typedef struct spear_rotation {
    const double *freqs; /* device [rot / 2]: angle of one position, radians; 8-byte aligned */
    double scale;        /* factor m of the rotated channels (1: none); 0 or 2^-100 <= |m| <= 2^100 */
    int32_t rot;         /* even, 2 .. D                                                       */
    int32_t layout;      /* SPEAR_ROPE_HALF or SPEAR_ROPE_PAIRS                               */
} spear_rotation;

/* How spear_rope_frequencies stretches the positions. */
#define SPEAR_ROPE_PLAIN  0 /* f_i = base^(-2i / rot)                                       */
#define SPEAR_ROPE_LINEAR 1 /* f_i / factor                                                 */
#define SPEAR_ROPE_BASE   2 /* base factor^(rot / (rot - 2)) in place of base: the slowest
                               pair turns factor times slower, the fastest as before        */
#define SPEAR_ROPE_PARTS  3 /* by the turns t = original f_i / 2 pi that a pair makes over the
                               original context: f_i from high turns on, f_i / factor up to
                               low, and g f_i + (1 - g) f_i / factor between them with
                               g = (t - low) / (high - low)                                  */

/*
 * spear_rope_frequencies -- host only, no HIP call: the rot / 2 frequencies of
 * a rotation into freqs (HOST pointer), all in fp64.
 *   rot even, 2 .. 256 (4 at least for SPEAR_ROPE_BASE); base > 1; factor > 0;
 *   original > 0 and low < high for SPEAR_ROPE_PARTS (else unused).
 */
spear_status spear_rope_frequencies(int32_t rot, double base, int32_t kind, double factor,
                                    double original, double low, double high, double *freqs);

/*
 * spear_rope -- y = x with every head rotated to its row's position:
 *   y_a = m (x_a cos t - x_b sin t), y_b = m (x_b cos t + x_a sin t),
 *   t = position * freqs[i], (a, b) the i-th pair, m = scale
 * with angles, cosines and sines in fp64 (far positions lose nothing) and y off from
 * these by 2^-23 |y| + 2^-37 |m| (|x_a| + |x_b|) + 2^-147 before it is rounded to bf16.
 * Infinities and NaN give what the formula gives for them (at position 0 an infinite
 * x_a: y_a infinite, y_b NaN), and no product on the way is cut at fp32's range.
 *   x [T][H][D] bf16, x_stride elements from a row to the next (a multiple of 8,
 *     at least H D); y likewise with y_stride; x and y 16-byte aligned.  y may be
 *     x itself (then with its stride); it overlaps no other input.
 *   positions [T], any int32.
 *   0 <= T <= SPEAR_MAX_ROWS, 1 <= H <= SPEAR_MAX_HEADS, D a multiple of 8 in
 *   [8, 256].
 */
spear_status spear_rope(const spear_bf16 *x, int64_t x_stride, int64_t T, int32_t H, int32_t D,
                        const int32_t *positions, const spear_rotation *rope, spear_bf16 *y,
                        int64_t y_stride, void *stream);

/*
 * spear_rope_kv4_write -- what follows the q/k/v projection, in one launch:
 * q rotated into q_out; k rotated and v as it is, each held in 4 bits in its
 * slot of the cache (k is rounded once, from the fp64 rotation).  rope == NULL
 * rotates nothing (positions is then unused).
 *   q [T][Hq][D], k and v [T][heads][D] bf16, each with a stride from row to row
 *     (a multiple of 8, at least its row); 16-byte aligned.  They may be parts of
 *     one row, and q_out may be q itself (with its stride); otherwise it overlaps
 *     no input.
 *   slots [T]: page * P + place; a row whose slot lies outside the cache is
 *     not written to it (its q is rotated all the same).  No slot may occur twice.
 */
spear_status spear_rope_kv4_write(const spear_bf16 *q, int64_t q_stride, const spear_bf16 *k,
                                  int64_t k_stride, const spear_bf16 *v, int64_t v_stride,
                                  int64_t T, int32_t Hq, const int32_t *positions,
                                  const int64_t *slots, const spear_rotation *rope,
                                  const spear_kv4 *kv, spear_bf16 *q_out, int64_t q_out_stride,
                                  void *stream);

/*
 * spear_kv4_read -- rows of the cache as bf16 (exact): k and v [T][heads][D],
 * either of them NULL if it is not wanted; a row whose slot lies outside the
 * cache is zeros.  k and v 16-byte aligned, slots 8-byte aligned.
 */
spear_status spear_kv4_read(const spear_kv4 *kv, const int64_t *slots, int64_t T, spear_bf16 *k,
                            spear_bf16 *v, void *stream);

/*
 * spear_kv4_attention -- attention of the step's rows over the cache, after
 * their own k and v have been written to it:
 *   row t of request b (q_start[b] <= t < q_start[b + 1]) stands at position
 *     p = kv_len[b] - (q_start[b + 1] - t)
 *   and sees the positions j <= p of its request, with window > 0 those above
 *     p - window only
 *   y[t][h] = sum_j softmax_j(scale q[t][h] . k[j][h / G]) v[j][h / G],  G = Hq / heads
 *   lse[t][h] = log sum_j exp(scale q . k)       (natural; optional)
 * Sums and softmax are in fp32, y is rounded once to bf16.  Probabilities meet v as
 * two bf16 (off by 2^-17 of their size at most), in requests of many rows as one
 * (2^-8).  Products q . k that pass fp32's range only when they are scaled count by
 * their differences (lse is rounded to fp32, an infinity where it lies beyond).
 * Requests of one token, of a few and of long chunks may stand side by side.  A row
 * that sees nothing, or scores of -inf only, gets zeros and lse -inf; one that sees a
 * NaN is NaN; rows behind the last request are left as they were.  A table entry
 * outside [0, pages) (a page that was let go) is as if its tokens were masked; what
 * masked places hold, NaN and infinities among it, does not count.  kv_len is held
 * within [0, width P] and q_start within [0, T].
 *   q [T][Hq][D] bf16 with q_stride elements from row to row (a multiple of 8);
 *     y [T][Hq][D] bf16 without gaps; both 16-byte aligned; y may be q itself if
 *     q has no gaps.  Hq a multiple of heads, G <= 64, T Hq <= 2^27.
 *   table [B][width], q_start [B + 1], kv_len [B] as spear_kv4_plan leaves them.
 *   max_fresh: no request has more rows than that (an upper bound that the host
 *     knows; it chooses kernels and their tiles, the result is right without it).
 *   scale > 0, finite (times log2 e too); window 0 (none) .. 2^30.
 *   workspace device scratch of spear_kv4_attention_workspace_size bytes (0 for
 *     sizes out of range), 256-byte aligned, its first SPEAR_KV4_COUNTER_BYTES zeroed
 *     once (spear_workspace_init): its counters are zero again when a call's work has
 *     ended.  It is not one that other entry points have written to.  The size grows
 *     with T and B and hangs on neither max_fresh nor width, so one for the
 *     largest step serves the others, also between calls of other sizes.
 */
#define SPEAR_KV4_COUNTER_BYTES ((size_t)163840)
size_t spear_kv4_attention_workspace_size(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq,
                                          int32_t heads, int32_t D, int64_t width, int32_t P);
spear_status spear_kv4_attention(const spear_bf16 *q, int64_t q_stride, int64_t T, int32_t Hq,
                                 const spear_kv4 *kv, const int32_t *table, int64_t width,
                                 const int32_t *q_start, const int32_t *kv_len, int32_t B,
                                 int64_t max_fresh, float scale, int32_t window, spear_bf16 *y,
                                 float *lse, void *workspace, size_t ws_bytes, void *stream);

/* Size of the library's own scratch used by spear_w4_linear_noalloc, per GPU. */
#define SPEAR_NOALLOC_MAX_WORKSPACE ((size_t)48 << 20)

/*
 * spear_w4_linear_noalloc -- spear_w4_linear_path without a workspace
 * argument, for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.  The
 * kernels are those of spear_w4_linear_path; the workspace they need is a
 * file-scope device array of SPEAR_NOALLOC_MAX_WORKSPACE bytes inside the
 * library (one per GPU, zero when the library is loaded, held until the
 * process ends).  The call itself allocates nothing: no hipMalloc, no
 * hipFree, no allocating library routine.
 *   Arguments as for spear_w4_linear_path.  A layer whose workspace need
 *   (spear_w4_linear_workspace_size) exceeds SPEAR_NOALLOC_MAX_WORKSPACE is
 *   rejected with SPEAR_E_WORKSPACE before any HIP call.
 * Every call on one GPU uses that GPU's single scratch array, which carries
 * state from call to call (launch counters, tagged partials): calls that may
 * overlap on one GPU (two streams, two threads) race and must not be made.
 * Expired-wait counts of these calls stay inside the scratch (they are not
 * readable through spear_workspace_timeouts); the NaN outputs described below
 * still mark them.
 */
spear_status spear_w4_linear_noalloc(const spear_bf16 *x, int64_t M, const spear_w4 *w,
                                     const spear_ec *ec, void *y, int32_t out_dtype,
                                     int32_t path, void *stream);

/*
 * Some launches wait (bounded) for values that other workgroups of the same
 * launch produce: the fused decode kernel's epilogue (the EC partials), the
 * decode kernel's last K range (the other ranges' sums), the split pre-pass's
 * last slice and, where the pre-pass shares the GEMM's launch, the GEMM
 * epilogue.  If a wait exceeds the limit, every output whose sum it leaves
 * incomplete is written as NaN -- a decode workgroup's channels for all
 * tokens, a pre-pass token group's rows, a GEMM tile -- the affected g_out
 * entries are NaN, *n_active_out is -1, and a counter in the workspace is
 * incremented.  No expired wait ever yields a finite but wrong output.
 * spear_set_wait_limit sets the limit in polling rounds for launches enqueued
 * afterwards, from any thread (0 restores the default, about a second);
 * spear_workspace_timeouts synchronises `stream`, copies the counter to
 * *host_count and clears it.
 */
void spear_set_wait_limit(uint32_t rounds);
spear_status spear_workspace_timeouts(void *workspace, int32_t *host_count, void *stream);

/*
 * EC-aware prefill chunking under an inter-token-latency objective (host
 * only, no HIP call; all pointers are HOST pointers).  Source: the summary's
 * section 2.2 C -- the scheduler takes the largest prefill chunk whose
 * predicted inter-token latency meets the objective, from kernel-latency
 * tables computed ahead of time, and adapts to how many layers carry ECs --
 * and section 3.2 (stable latency objectives with dynamic chunking).
 *
 * The table holds, for each kind of linear call (a weight shape with or
 * without its EC), the measured time of one call at a grid of token counts,
 * and how many calls of that kind one forward step of the model makes (EC
 * density enters through these counts).  One step over m tokens is predicted
 * as overhead_us + sum_k count[k] L_k(m), with L_k the running maximum of the
 * kind's measurements (so the prediction never falls as m grows), linear
 * between grid points, its first value below the grid and its last segment's
 * slope above it.
 */
typedef struct spear_lut {
    int32_t npoints;        /* grid points, >= 1                                   */
    const int32_t *tokens;  /* [npoints] token counts, ascending, tokens[0] >= 1   */
    int32_t nkinds;         /* kinds of linear call, >= 1                          */
    const float *us;        /* [nkinds][npoints] microseconds per call, finite, >= 0 */
    const int32_t *count;   /* [nkinds] calls of each kind per step, >= 0          */
    float overhead_us;      /* fixed time per step outside these calls, >= 0      */
} spear_lut;

/* Predicted time of one step over `tokens` tokens (0 for no tokens). */
spear_status spear_slo_predict(const spear_lut *lut, int32_t tokens, float *us_out);

/*
 * spear_slo_pick_chunk -- the prefill chunk for the next step: the largest c,
 * either `pending` itself or a multiple of `align` below it, such that a step
 * over n_decode + c tokens (the running requests' decode tokens plus the
 * chunk) is predicted within slo_us.  0 when even the smallest chunk does not
 * fit.  *predicted_us (optional) receives the prediction for the chosen c.
 *   n_decode >= 0, pending >= 0 (prompt tokens waiting), align >= 1.
 */
spear_status spear_slo_pick_chunk(const spear_lut *lut, int32_t n_decode, int32_t pending,
                                  int32_t align, float slo_us, int32_t *chunk,
                                  float *predicted_us);

/*
 * spear_stream_read -- measurement helper, not part of the layer: reads every
 * byte of buf once (16-byte loads, four a thread in flight) and writes
 * nothing to *sink in practice (it is written only if the XOR of the data
 * equals a fixed constant, so that the loads cannot be optimised away).  Its
 * rate is the plain read floor that the decode kernel's bandwidth is compared
 * with, for buffers of the layer's size.
 *   buf  device pointer, 16-byte aligned; bytes >= 16 and a multiple of 16.
 *   sink device pointer to one uint32, 4-byte aligned.
 */
spear_status spear_stream_read(const void *buf, size_t bytes, uint32_t *sink, void *stream);

const char *spear_status_string(spear_status s);
int32_t spear_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SPEAR_H */
