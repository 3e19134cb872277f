/*
 * moe_decode.h -- C ABI of the output-centric ("warp decode") MoE decode layer
 * for AMD Instinct MI355X (gfx950).
 *
 * Source of the method: Cursor, "warp decode" blog post.  The MoE FFN of one
 * decode step is two kernels (section "What we changed"):
 *   moe_decode_gate_up  -- section "How the two kernels work", first two
 *       paragraphs: for each token b, routed slot j and intermediate neuron n,
 *       the gate and up rows of expert e = topk_ids[b,j] are streamed, their
 *       MXFP8 values converted to FP32 on the fly and dotted with x[b] in FP32;
 *       the neuron's value SiLU(gate) * up is written once.
 *   moe_decode_down     -- same section, third and fourth paragraphs: for each
 *       token b and output dimension o, the down rows of the token's k routed
 *       experts are streamed against h[b,j,:], each expert's router weight is
 *       folded into one FP32 accumulator, and y[b,o] is written once; the
 *       weighted top-k combine is part of the projection (no padding, no
 *       expert-major gather, no per-expert output buffer, no separate combine:
 *       sections "Stage elimination" and "Eliminating buffers").
 *
 * Number formats.  Weights are MXFP8 (OCP Microscaling v1.0): E4M3 element
 * codes (bias 7, max 448, S.1111.111 = NaN) with one E8M0 scale code
 * (value 2^(v-127), 0xFF = NaN) per 32 consecutive elements along the
 * reduction dimension.  Activations x, the intermediate h and the output y
 * are bf16 (stored as 16-bit patterns); results are rounded to nearest even.
 * Accumulation is FP32 in an unspecified order.  Router weights are FP32 and
 * are used as given (never renormalised).
 *
 * Layouts (all row-major, all contiguous):
 *   x            bf16   [B, H]
 *   topk_ids     int32  [B, k]   expert of slot j of token b
 *   topk_weights fp32   [B, k]   router weight of that slot
 *   w_gate, w_up uint8  [E, I, H]    E4M3 codes, row = one neuron of one expert
 *   s_gate, s_up uint8  [E, I, H/32] E8M0 codes, s[e,n,c/32] scales w[e,n,c]
 *   w_down       uint8  [E, H, I]    E4M3 codes, row = one output dim of one expert
 *   s_down       uint8  [E, H, I/32] E8M0 codes
 *   h            bf16   [B, k, I]    slot order = topk_ids order
 *   y            bf16   [B, H]
 *
 * Ownership and behaviour common to every call:
 *   - Every pointer is a device pointer owned by the caller.  The library
 *     allocates nothing, keeps no pointer after return and never synchronises.
 *   - Work is enqueued on `stream` (a hipStream_t passed as void*; NULL = the
 *     null stream).  The call returns as soon as the launch is enqueued; the
 *     caller synchronises the stream before reading outputs.
 *   - Calls are thread-safe.  The only state the library keeps is set once
 *     per device, before the first launch that needs it on that device, and
 *     is never changed afterwards: each matrix-core kernel's maximum dynamic
 *     LDS, set to the largest size its limits allow, and the device address
 *     of the no-allocation entry point's scratch array (whose concurrent
 *     calls on one device race; see moe_decode_conventional_noalloc).
 *   - Outputs are fully overwritten; every element is written exactly once.
 *   - Outputs must not overlap any input (checked on the host), but where a
 *     call says that an output may be one of its inputs itself.
 *   - B == 0 is a valid no-op.
 *   - topk_ids outside [0, E) are not read through: every output that depends
 *     on such a slot is written as a quiet NaN.  Duplicate ids in one token
 *     are legal and are summed slot by slot.
 *   - E8M0 codes 0x00 (2^-127) and 0xFF (NaN) are honoured.
 * Return value: MOE_OK (0) once the launch is enqueued, else a negative code
 * below.  On any negative return other than MOE_ERR_LAUNCH nothing was
 * launched and no output was touched.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_ERR_NULL (-1)        /* a required pointer is NULL (with B > 0)                    */
#define MOE_ERR_SHAPE (-2)       /* B<0, H/I/E/k<=0, k>E, H or I not a multiple of 32, or a   */
                                 /* shape beyond the supported range (H <= 8192,              */
                                 /* k*I <= 16384, E*I*H < 2^32 bytes per weight tensor)       */
#define MOE_ERR_ALIGN (-3)       /* x, h, w_* not 16-byte aligned; ids/weights not 4-byte     */
#define MOE_ERR_LAUNCH (-4)      /* the HIP runtime reported an error for the launch          */
#define MOE_ERR_ALIAS (-5)       /* an output range overlaps an input range                   */
#define MOE_ERR_ARG (-6)         /* an invalid tuning argument (see the _ex variants)         */
#define MOE_ERR_SCRATCH (-7)     /* the shape needs more scratch than the fixed buffer holds  */
                                 /* (moe_decode_conventional_noalloc only)                   */

/* Gate/up kernel: h[b,j,n] = bf16( SiLU(G) * U ), with
 *   G = sum_c dec(w_gate[e,n,c]) * 2^(s_gate[e,n,c/32]-127) * x[b,c],
 *   U = the same with w_up, s_up,  e = topk_ids[b,j].
 * Reads x [B,H], topk_ids [B,k], w_gate/s_gate/w_up/s_up of the routed experts only;
 * writes h_out [B,k,I]. */
int moe_decode_gate_up(const void *x, const int32_t *topk_ids,
                       const uint8_t *w_gate, const uint8_t *s_gate,
                       const uint8_t *w_up, const uint8_t *s_up,
                       void *h_out,
                       int B, int H, int I, int E, int k, void *stream);

/* Down kernel: y[b,o] = bf16( sum_j topk_weights[b,j] *
 *   sum_i dec(w_down[e_j,o,i]) * 2^(s_down[e_j,o,i/32]-127) * h[b,j,i] ),  e_j = topk_ids[b,j].
 * Reads h [B,k,I], topk_ids and topk_weights [B,k], w_down/s_down of the routed experts only;
 * writes y_out [B,H]. */
int moe_decode_down(const void *h, const int32_t *topk_ids, const float *topk_weights,
                    const uint8_t *w_down, const uint8_t *s_down,
                    void *y_out,
                    int B, int H, int I, int E, int k, void *stream);

/* Kernel variants of the gate/up call.
 *   MOE_GATE_UP_PER_SLOT: one wavefront per (R neurons, token slot) -- the
 *     blog post's organisation, one output set per warp ("How the two kernels
 *     work").  Best while few tokens share an expert.
 *   MOE_GATE_UP_EXPERT_GROUPED: the slots are sorted by expert on the device
 *     (inside the kernel, in LDS) and one wavefront takes R neurons of one
 *     routed expert for every slot routed to it, reading and converting the
 *     expert's rows once (section "Warp decode and Composer training": the
 *     regime where several tokens share an expert).  Same outputs; requires
 *     B*k <= 1024 and E <= 1024.
 *   MOE_GATE_UP_EXPERT_GROUPED_MFMA: the same grouping with the dot products
 *     on the matrix cores (v_mfma_f32_16x16x32_bf16): a workgroup takes 16
 *     neurons of one routed expert for up to 8 or 16 of its slots, streaming the
 *     rows and activations through LDS in 512-element chunks; the E8M0 scale
 *     is folded into the E4M3 -> bf16 conversion.  Same outputs within the
 *     same tolerance; requires H a multiple of 2048 up to 8192, B*k <= 1024,
 *     E <= 1024, and s_gate, s_up 16-byte aligned (MOE_ERR_ALIGN otherwise;
 *     rows_per_wave must be 0 or 16).
 * The plain call takes the matrix-core variant from 0.625 slots per expert
 * on (8*B*k >= 5E), or from half a slot at H >= 4096 (2*B*k >= E), when its
 * limits allow (with unaligned scales it takes the vector-unit grouped
 * variant instead); where they do not, the vector-unit grouped one from one
 * slot per expert on (B*k >= E), or half a slot at H >= 4096; else the
 * per-slot one.  At H = 4096 exactly, the vector-unit grouped variant from
 * 5/16 of a slot per expert up to 7/4 (16*B*k >= 5E, 4*B*k < 7E).  Each
 * choice is the fastest measured there. */
#define MOE_GATE_UP_PER_SLOT 1
#define MOE_GATE_UP_EXPERT_GROUPED 2
#define MOE_GATE_UP_EXPERT_GROUPED_MFMA 3

/* Kernel variants of the down call.
 *   MOE_DOWN_PER_TOKEN: one wavefront per (R output dimensions, token) --
 *     the blog post's organisation ("How the two kernels work").  Best while
 *     few tokens share an expert.
 *   MOE_DOWN_EXPERT_GROUPED: one workgroup per 8 output dimensions (4 for
 *     I > 1024) for every token; its wavefronts share out the routed experts
 *     (sorted on the device, in LDS), read each routed expert's rows once,
 *     and keep each slot's FP32 contribution in LDS until the workgroup adds
 *     every token's k contributions in slot order and writes y once.  No
 *     per-expert output buffer, no combine.  Same outputs; requires
 *     B <= 64, B*k <= 1024, E <= 1024 and I <= 2048.
 *   MOE_DOWN_EXPERT_GROUPED_MFMA: the same organisation (one workgroup per 8
 *     output dimensions for every token, work units of at most 8 slots of one
 *     expert, contributions added in slot order) with the dot products on the
 *     matrix cores (v_mfma_f32_4x4x4_16b_bf16): a wavefront converts its
 *     unit's 8 rows to bf16 once per 4 slots and forms the 8 x 4 dot products
 *     as 16-element chunk products, each scaled by its chunk's E8M0 scale
 *     (exact) before the chunks are summed.  Same outputs within the same
 *     tolerance; requires B*k <= 1024, E <= 1024 and I <= 2048
 *     (rows_per_wave must be 0 or 8).
 * The plain call takes the matrix-core grouped variant once 16*B*k >= 5E
 * (5/16 of a slot per expert on average) and its limits allow it, else the
 * per-token one: the fastest in each measured configuration but one (H =
 * 4096 with 5 tokens of uniform routing, where the per-token kernel is 3.5 %
 * faster; under skewed routing it is 6 % slower there).  The vector-unit
 * grouped variant runs on request only: its limits lie within the
 * matrix-core one's, which is faster wherever both run. */
#define MOE_DOWN_PER_TOKEN 1
#define MOE_DOWN_EXPERT_GROUPED 2
#define MOE_DOWN_EXPERT_GROUPED_MFMA 3

/* Tuning variants of the two calls: the same contract and results within the
 * same tolerance, with the launch shape given explicitly instead of taken
 * from the built-in table.  variant: 0 = the table's choice, else one of the
 * MOE_GATE_UP_* (gate/up) or MOE_DOWN_* (down) values.  rows_per_wave in
 * {1, 2, 4, 8} is the number of neurons (gate/up) or output dimensions (down)
 * one 64-lane wavefront owns (the grouped down kernel: 8 for I <= 1024,
 * else 4); 0 selects
 * the table's choice.  Combinations beyond the register budget (rows x
 * passes of 1024 elements: <= 16 per-slot, <= 8 grouped; per-token down:
 * passes x (5 rows + 8) <= 224), a grouped variant beyond its limits and
 * unknown variants return MOE_ERR_ARG. */
int moe_decode_gate_up_ex(const void *x, const int32_t *topk_ids,
                          const uint8_t *w_gate, const uint8_t *s_gate,
                          const uint8_t *w_up, const uint8_t *s_up,
                          void *h_out,
                          int B, int H, int I, int E, int k,
                          int variant, int rows_per_wave, void *stream);
int moe_decode_down_ex(const void *h, const int32_t *topk_ids, const float *topk_weights,
                       const uint8_t *w_down, const uint8_t *s_down,
                       void *y_out,
                       int B, int H, int I, int E, int k,
                       int variant, int rows_per_wave, void *stream);

/* Router step in front of the layer.  The blog post ("The traditional MoE
 * path") routes each token to a few of many experts (8 of 128 in one layer)
 * and gives no router details; these calls implement the plain top-k router:
 * from logits fp32 [B, E] (row-major, finite values), token b keeps its k
 * largest logits, largest first and the lower expert id first among equal
 * logits (-0 equals +0), so topk_ids[b, j] is its j-th selection; the routing
 * weight topk_weights[b, j] = exp(l_j - l_0) / sum_i exp(l_i - l_0) over the
 * k selections (the softmax over all E renormalised over the kept k), in
 * FP32 with the device's expf.  Ids are always in [0, E), even for logits
 * that are not finite (their weights are then unspecified).
 * Limits: E <= 1024, k <= 64 and k <= E, B*E*4 < 2^31.  Pointers 4-byte
 * aligned; outputs disjoint from each other and from every input.
 *
 *   moe_decode_route: ids and weights only (one 64-lane wavefront per token).
 *   moe_decode_gate_up_routed: gate/up with the router step in front --
 *     reads logits instead of topk_ids, writes h_out as moe_decode_gate_up
 *     would for the ids it selects, and also writes topk_ids_out and
 *     topk_weights_out [B, k] for moe_decode_down.  For E <= 128 and
 *     B*k <= 16 (and whenever the _ex form asks for the per-slot variant
 *     with E <= 128) the selection is the per-slot kernel's prologue: each
 *     workgroup selects its token's experts itself, with no extra launch.
 *     Otherwise the router kernel runs first and the table's (or the asked)
 *     gate/up variant reads the ids it wrote: two launches on `stream`.  The
 *     _ex form takes variant and rows_per_wave as moe_decode_gate_up_ex
 *     does. */
int moe_decode_route(const float *logits, int32_t *topk_ids, float *topk_weights,
                     int B, int E, int k, void *stream);
int moe_decode_gate_up_routed(const void *x, const float *logits,
                              const uint8_t *w_gate, const uint8_t *s_gate,
                              const uint8_t *w_up, const uint8_t *s_up,
                              void *h_out, int32_t *topk_ids_out, float *topk_weights_out,
                              int B, int H, int I, int E, int k, void *stream);
int moe_decode_gate_up_routed_ex(const void *x, const float *logits,
                                 const uint8_t *w_gate, const uint8_t *s_gate,
                                 const uint8_t *w_up, const uint8_t *s_up,
                                 void *h_out, int32_t *topk_ids_out, float *topk_weights_out,
                                 int B, int H, int I, int E, int k,
                                 int variant, int rows_per_wave, void *stream);

/* The launch the built-in table picks for a call (for reports): writes the
 * variant, rows_per_wave and the number of workgroups; returns 0 or a
 * negative code. */
int moe_decode_gate_up_plan(int B, int H, int I, int E, int k, int *variant, int *rows_per_wave, int *workgroups);
int moe_decode_down_plan(int B, int H, int I, int E, int k, int *variant, int *rows_per_wave, int *workgroups);

/* The conventional, expert-centric path, for A/B comparison (blog post,
 * sections "The traditional MoE path", "Stage elimination", "Eliminating
 * buffers" and "Accuracy improvement").  Same layer as gate_up + down, but
 * computed the way an expert-centric pipeline does it, as seven launches on
 * `stream` through caller-provided device workspace: route (per-expert token
 * lists, each padded to a power of two), quantise x to MXFP8 (E4M3 codes and
 * one E8M0 scale 2^(floor(log2 amax) - 8) per 32 along H, saturating at 448),
 * scatter the quantised rows into an expert-major gather buffer, gate/up per
 * row (h = bf16(SiLU(G) * U)), quantise h to MXFP8 (blocks along I), down per
 * row into a bf16 per-expert output buffer, and the weighted combine y[b] =
 * bf16(sum_j w[b,j] * out[b,j]).  Padding rows are computed and discarded.
 * Inputs and y as for the two calls above; `workspace` is device memory of at
 * least the size moe_decode_conventional_workspace() reports, 256-byte
 * aligned, owned by the caller, disjoint from every input and from y, and
 * used only until the launches complete.  Limits: B*k <= 1024, E <= 1024,
 * H and I <= 8192.  Returns MOE_ERR_ARG if the workspace is too small;
 * otherwise the error codes above. */
int moe_decode_conventional_workspace(int B, int H, int I, int E, int k, size_t *bytes);
int moe_decode_conventional(const void *x, const int32_t *topk_ids, const float *topk_weights,
                            const uint8_t *w_gate, const uint8_t *s_gate,
                            const uint8_t *w_up, const uint8_t *s_up,
                            const uint8_t *w_down, const uint8_t *s_down,
                            void *y_out, void *workspace, size_t workspace_bytes,
                            int B, int H, int I, int E, int k, void *stream);

/* The conventional path of moe_decode_conventional for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops
 * and harnesses that forbid hipMalloc.  Same stages, kernels and results, but
 * instead of a caller's workspace the launches use a fixed 32 MiB device
 * buffer inside the library (one per device, resident from module load until
 * the process ends).  Nothing in that buffer needs to start at zero: the route
 * stage writes every entry the later stages read.  The call allocates and
 * frees nothing (no hipMalloc, hipFree or allocating library routine); its
 * first call on a device looks up that device's address of the buffer once.
 * Every call on one device shares that device's buffer and leaves its contents
 * behind, so calls that overlap in time on one device race: the caller orders
 * them (one stream, or events between streams).  Returns MOE_ERR_SCRATCH
 * (before any launch) when the shape's workspace,
 * moe_decode_conventional_workspace(), exceeds 32 MiB; otherwise the codes
 * and limits of moe_decode_conventional. */
int moe_decode_conventional_noalloc(const void *x, const int32_t *topk_ids, const float *topk_weights,
                                    const uint8_t *w_gate, const uint8_t *s_gate,
                                    const uint8_t *w_up, const uint8_t *s_up,
                                    const uint8_t *w_down, const uint8_t *s_down,
                                    void *y_out, int B, int H, int I, int E, int k, void *stream);

/* Training the router: per-expert counts, the balance loss and the z loss, and
 * their gradient with respect to the router's logits.
 *
 * T tokens in G groups of S = T / G consecutive tokens (a group is the unit
 * the balance loss is taken over: the whole batch, G = 1, or one sequence).
 * Token t of group g is valid unless `valid` is given and valid[t] == 0.  With
 * n_g the valid tokens of group g, c_ge the slots of its valid tokens routed to
 * expert e, p_t = softmax(logits_t) and N = sum_g n_g:
 *   losses[0] = 1/G sum_g E / (k n_g) * 1 / n_g * sum_e c_ge sum_t p_te
 *   losses[1] = 1/N sum_t logsumexp(logits_t)^2
 * (sums over valid tokens; a group without one contributes 0 to both, as does
 * N = 0).  The counts are constants to the gradient:
 *   dlogits_te = grad_losses[0] / (G n_g) * p_te (f_ge - sum_j f_gj p_tj)
 *              + grad_losses[1] * 2/N * logsumexp(logits_t) * p_te,
 *   f_ge = E c_ge / (k n_g);  0 for a token that is not valid.
 *
 *   logits       [T, E] of `dtype` (MOE_F32 or MOE_BF16), row t at t * ld elements
 *   topk_ids     int32 [T, k]; ids outside [0, E) are not counted; a repeated
 *                id counts as often as it stands there
 *   valid        uint8 [T] or NULL (every token is valid)
 *   losses       fp32 [2]
 *   counts       int32 [G, E]
 *   tokens       int32 [G + 1]: n_0 .. n_(G-1), then N
 *   grad_losses  fp32 [2], device memory: the factors of the two losses
 *   dlogits      [T, E] of `dtype`, row t at t * ld_d elements
 * A logit of -inf (an expert ruled out) has probability 0; a valid row of -inf
 * only has p = 0 and logsumexp taken as 0.  +inf and NaN give NaN.  The logits
 * of a token that is not valid may hold anything.  Sums are FP32 over at most
 * 32768 tokens, then FP64, always in the same order: the same inputs give the
 * same bits.  Elements between the rows (ld > E) are neither read
 * nor written.
 * Limits: E <= 1024, k <= 64 and k <= E, G divides T, T <= 2^30, T * k < 2^31,
 * G <= 2^19, G * E < 2^26, strides up to 2^30.  `workspace` is device memory of at least
 * moe_decode_balance_workspace() bytes, 256-byte aligned, used until the
 * launches complete (calls that may overlap in time need one each); it need
 * not be cleared, and where that says 0 bytes (one group of up to 256 tokens)
 * it is not looked at.  T == 0 is a valid no-op that writes nothing. */
#define MOE_F32 0
#define MOE_BF16 1
#define MOE_F16 2
int moe_decode_balance_workspace(int T, int E, int k, int G, size_t *bytes);
int moe_decode_balance(const void *logits, long long ld, int dtype, const int32_t *topk_ids, const uint8_t *valid,
                       float *losses, int32_t *counts, int32_t *tokens, void *workspace, size_t workspace_bytes,
                       int T, int E, int k, int G, void *stream);
int moe_decode_balance_backward(const void *logits, long long ld, int dtype, const uint8_t *valid,
                                const int32_t *counts, const int32_t *tokens, const float *grad_losses,
                                void *dlogits, long long ld_d, int T, int E, int k, int G, void *stream);

/* Rows to 8 bits with one scale for each block of 128: the operand of the
 * products below.  For row m and block b of 128 columns (the last one may be
 * shorter), with v the block's values:
 *   scales[m, b] = max(amax |v| / 448, 2^-126),
 *   q[m, c] = E4M3(v_c / scales[m, b])      round to nearest even
 * amax over the block's finite values; both quotients are FP32 divisions,
 * correctly rounded.  MOE_QUANT_POW2 raises each scale to the next power of two.
 * A NaN or an infinity becomes the NaN code 0x7F and leaves its block's other
 * values as they would be without it.
 *   x       [M, K] of `dtype` (MOE_F32, MOE_BF16 or MOE_F16), row m at m * ldx elements;
 *           with MOE_QUANT_SWIGLU [M, 2K] and v_c = SiLU(x[m, c]) * x[m, K + c]
 *           in FP32 (within 6 * 2^-23 of its value; e^-|x| below 2^-126 counts
 *           as 0), not rounded before the quantisation
 *   q       uint8 [M, K] E4M3 codes
 *   scales  fp32 [M, ceil(K / 128)]
 * Limits: M * ceil(K / 128) <= 2^28 - 16, K <= 2^28, ldx up to 2^30.  M == 0 is a valid no-op. */
#define MOE_QUANT_SWIGLU 1
#define MOE_QUANT_POW2 2
int moe_decode_quantize_fp8(const void *x, long long ldx, int dtype, uint8_t *q, float *scales,
                            int M, int K, int flags, void *stream);

/* Products of 8-bit operands with a scale for each block of 128:
 *   y[m, n] = sum_b sx[m, b] * sw[n / 128, b] * sum_{c in block b} x[m, c] * w[n, c]
 * with each block's sum formed on the matrix cores in FP32, scaled (by the
 * product of the two scales, itself an FP32 number) and added in FP32, and one
 * rounding to y.
 *   x   uint8 [M, K] E4M3 codes, row m at m * ldx bytes
 *   sx  fp32 [M, ceil(K / 128)]
 *   w   uint8 [N, K] E4M3 codes
 *   sw  fp32 [ceil(N / 128), ceil(K / 128)]
 *   y   [M, N] of y_dtype (MOE_F32, MOE_BF16 or MOE_F16), row m at m * ldy elements
 * K a multiple of 16, x and w 16-byte aligned, ldx a multiple of 16.
 * The gradient with respect to x is a product of the same kind: of dy, quantised
 * in blocks of 128 along N (N a multiple of 16), with w^T [K, N] and sw^T [ceil(K /
 * 128), ceil(N / 128)], which the caller lays out.  (With experts it is one row for
 * each row of y; a row of x that several of them come from gets their sum.)
 *
 * moe_decode_matmul_fp8_experts: the same for E matrices w [E, N, K], sw [E,
 * ceil(N / 128), ceil(K / 128)] on rows sorted by expert: the first counts[0]
 * rows of y belong to expert 0, the next counts[1] to expert 1, and so on
 * (counts int32 [E], device memory).  moe_decode_balance's counts are those of
 * its valid tokens' slots with ids in [0, E), group by group: with G = 1, or its
 * groups' added up, they go with those slots sorted by expert and the slots of
 * tokens that are not valid, or of other ids, behind them all, where they are not
 * computed.  (Slots of padding sorted in among the others would shift every later
 * expert's rows.)  Row m of y comes from row m of x, or from row x_rows[m] where
 * x_rows (int32 [M]) is given; x and sx have X rows.  A row number outside [0, X)
 * is not read through: its row of y is NaN.  Rows of y behind the last expert's are
 * left as they were; negative counts are taken as 0, and rows beyond M are not
 * computed.
 * Limits: E <= 1024, N * K < 2^31, M < 2^24 (experts) or 2^30, K <= 2^30, strides
 * up to 2^30, and of the tiles that y is cut into fewer than 2^24 (2^22 of
 * ROWS_16 and TILE_256X256).  M == 0 is a valid no-op.
 *
 * Kernel variants (the _ex forms take one; 0 = the built-in choice, by the
 * sizes; moe_decode_matmul_fp8_plan reports it for ordinary strides, E = 0
 * asking about one matrix):
 *   MOE_MATMUL_ROWS_16: 16 rows a workgroup, its wavefronts sharing out K.
 *   MOE_MATMUL_TILE_<rows>X<columns>: a tile of y a workgroup, both operands
 *     through LDS; _STREAM reads w as data that is used once.
 *   MOE_MATMUL_FAR_ROWS: as TILE_64X64 for any stride.
 * A TILE variant needs 32-bit offsets to reach its rows of x (with x_rows all X
 * rows), TILE_256X256 a 16-bit y: MOE_ERR_ARG otherwise.
 *
 * MOE_MATMUL_FP8_SUMS, added to a variant or alone (the built-in choice for it),
 * lets a 16-bit y take its blocks' sums from the FP8 matrix instruction, at up to
 * twice the rate: it adds eight products at a time and cuts them off 2^-13 below
 * the largest, so that a sum of K products is off by at most 2^-10 of the sum of
 * their magnitudes (of its root mean square: 1.5e-5 on normally distributed
 * codes, where a bf16 result's rounding is 1.7e-3 and an FP16 one's 2.1e-4; 7e-5
 * with 1 % of the channels 20 times as large; more where sums cancel).  It changes
 * nothing for an FP32 y and for ROWS_16.  TILE_256X256 has these sums only, with
 * or without it; no other call gets them.
 *
 * The order of the FP32 sums is the variant's (ROWS_16 has one of its own, all
 * others the same), and the built-in choice goes by the sizes: the same row can
 * differ in the last bit from one M to another.  A caller who needs it alike for
 * every M asks for one variant. */
#define MOE_MATMUL_ROWS_16 1
#define MOE_MATMUL_TILE_64X64 2
#define MOE_MATMUL_TILE_64X128 3
#define MOE_MATMUL_TILE_64X128_STREAM 4
#define MOE_MATMUL_TILE_128X128 5
#define MOE_MATMUL_TILE_256X256 6
#define MOE_MATMUL_FAR_ROWS 7
#define MOE_MATMUL_FP8_SUMS 256
int moe_decode_matmul_fp8(const uint8_t *x, long long ldx, const float *sx, const uint8_t *w, const float *sw,
                          void *y, long long ldy, int y_dtype, int M, int N, int K, void *stream);
int moe_decode_matmul_fp8_ex(const uint8_t *x, long long ldx, const float *sx, const uint8_t *w, const float *sw,
                             void *y, long long ldy, int y_dtype, int M, int N, int K, int variant, void *stream);
int moe_decode_matmul_fp8_experts(const uint8_t *x, long long ldx, const float *sx, const int32_t *x_rows,
                                  const int32_t *counts, const uint8_t *w, const float *sw,
                                  void *y, long long ldy, int y_dtype, int X, int M, int N, int K, int E, void *stream);
int moe_decode_matmul_fp8_experts_ex(const uint8_t *x, long long ldx, const float *sx, const int32_t *x_rows,
                                     const int32_t *counts, const uint8_t *w, const float *sw,
                                     void *y, long long ldy, int y_dtype, int X, int M, int N, int K, int E,
                                     int variant, void *stream);
int moe_decode_matmul_fp8_plan(int M, int N, int K, int E, int *variant, int *workgroups);

/* Routing to experts by scores.  From logits [T, E], with s_te = softmax(l_t)_e, or
 * 1 / (1 + e^-l_te) with MOE_ROUTE_SIGMOID, and c_te = s_te + bias_e:
 *   - the experts lie in `groups` groups of E / groups neighbours.  A group's score
 *     is its largest c, or with MOE_ROUTE_GROUP_TOP2 the sum of its two largest (the
 *     one, where one expert alone is not ruled out; of groups of one expert the flag
 *     says nothing).  The top_groups groups with the largest scores stay, the lower
 *     group first among equals.
 *   - of their experts token t takes the k with the largest c, largest first, the
 *     lower id first among equals: topk_ids[t, j].
 *   - topk_weights[t, j] = scale * s of that expert (without the bias), with
 *     MOE_ROUTE_RENORM over the sum of the k (0 where all k are ruled out, or of
 *     sigmoid scores that are 0 in 64 bits too).
 * Choices are those of c in 64 bits; without a bias, experts (and groups by their
 * largest) go by the logits.  Weights are FP32; a score below 2^-126 may count as 0.
 * A logit of -inf rules an expert out: it comes behind all others of the groups that
 * stay, its score is 0, a group of such comes last.  Ids are always different from
 * each other and in [0, E); with a logit of +inf or NaN in the row they and the
 * weights are not specified otherwise.
 *   logits        [T, E] of `dtype` (MOE_F32 or MOE_BF16), row t at t * ld elements
 *   bias          fp32 [E] or NULL (0)
 *   topk_ids      int32 [T, k];  topk_weights  fp32 [T, k]
 * moe_decode_route_experts_backward: dlogits_te = sum_j grad_weights[t, j] *
 * d topk_weights[t, j] / d l_te, with the choices as constants (the bias has no
 * gradient).  topk_ids outside [0, E) contribute nothing; an expert that stands
 * there twice gets both terms.  Of the flags SIGMOID and RENORM matter.
 * Limits: E <= 1024, k <= 64, groups <= 64 and a divisor of E, k <= top_groups * E /
 * groups, T < 2^26, T * k < 2^31, strides up to 2^30.  T == 0 is a valid no-op. */
#define MOE_ROUTE_SIGMOID 1
#define MOE_ROUTE_RENORM 2
#define MOE_ROUTE_GROUP_TOP2 4
int moe_decode_route_experts(const void *logits, long long ld, int dtype, const float *bias,
                             int32_t *topk_ids, float *topk_weights, int T, int E, int k,
                             int groups, int top_groups, int flags, float scale, void *stream);
int moe_decode_route_experts_backward(const void *logits, long long ld, int dtype, const int32_t *topk_ids,
                                      const float *grad_weights, void *dlogits, long long ld_d,
                                      int T, int E, int k, int flags, float scale, void *stream);

/* The slots of topk_ids [T, k] sorted by expert, and by their number t * k + j within
 * an expert: the rows of moe_decode_matmul_fp8_experts, and where the results of a
 * token's slots lie.
 *   counts     int32 [E]     slots of each expert
 *   x_rows     int32 [T * k] the token of each sorted row; -1 behind the last expert's
 *   positions  int32 [T, k]  the sorted row of each slot; -1 where it is not counted
 * Slots of a token with valid[t] == 0 (valid: uint8 [T] or NULL) and ids outside [0,
 * E) are not counted.  Limits: E <= 1024, k <= 64, T * k < 2^24.  `workspace` is
 * device memory of at least moe_decode_sort_slots_workspace() bytes, 256-byte
 * aligned, used until the launches complete (calls that may overlap in time need one
 * each); it need not be cleared, and where that says 0 bytes it is not looked at.
 * T == 0 is a valid no-op that writes nothing: counts, which are then of no slots,
 * keep what they hold (0 in them before the call makes them right for every T). */
int moe_decode_sort_slots_workspace(int T, int E, int k, size_t *bytes);
int moe_decode_sort_slots(const int32_t *topk_ids, const uint8_t *valid, int32_t *counts, int32_t *x_rows,
                          int32_t *positions, void *workspace, size_t workspace_bytes,
                          int T, int E, int k, void *stream);

/* The experts' rows back to their tokens:
 *   y[t, n] = add[t, n] + sum_j weights[t, j] * rows[positions[t, j], n]
 * in FP32, rounded once.  A position outside [0, M) contributes nothing (its weight
 * is not looked at).
 *   rows       [M, N] of `dtype` (MOE_F32, MOE_BF16 or MOE_F16), row m at m * ld_rows
 *   positions  int32 [T, k];  weights  fp32 [T, k] or NULL (1: a sum of rows, as for
 *              the gradient of a token that stands in several sorted rows)
 *   add        [T, N] of `dtype` or NULL (0); it may be y itself, with y's stride
 *   y          [T, N] of `dtype`
 * moe_decode_combine_backward: drows[positions[t, j], n] = weights[t, j] * dy[t, n]
 * and dweights[t, j] = sum_n dy[t, n] * rows[positions[t, j], n] (0 for a position
 * outside [0, M)); the gradient of `add` is dy.  Rows that no slot names are left as
 * they were; no two slots may name the same row (one of their values would be left).
 * dweights NULL: not wanted, rows are not read.
 * Limits: k <= 64, T * k < 2^24, M <= 2^24, T * ceil(N / 2048) < 2^24, N <= 2^28,
 * strides up to 2^30.  T == 0 is a valid no-op. */
int moe_decode_combine(const void *rows, long long ld_rows, int dtype, const int32_t *positions,
                       const float *weights, const void *add, long long ld_add, void *y, long long ld_y,
                       int M, int T, int N, int k, void *stream);
int moe_decode_combine_backward(const void *dy, long long ld_dy, const void *rows, long long ld_rows, int dtype,
                                const int32_t *positions, const float *weights, void *drows, long long ld_d,
                                float *dweights, int M, int T, int N, int k, void *stream);

/* Root-mean-square norm of rows, with the residual's addition in front and 8 bits
 * behind:
 *   r = x + residual, rounded to `dtype` (x itself without a residual)
 *   rstd = 1 / sqrt(mean_c r_c^2 + eps)
 *   v_c = r_c * rstd * weight_c      in FP32
 *   sum = r,  y = v rounded to `dtype`,  q and scales = v as moe_decode_quantize_fp8
 *   makes them of FP32 values (MOE_QUANT_POW2 among its flags)
 * Squares whose sum passes FP32 are added in FP64.  A NaN or an infinity in a row goes
 * where the formula takes it.
 *   x, residual, y, sum  [M, H] of `dtype` (MOE_F32, MOE_BF16 or MOE_F16), each with
 *              its stride; residual, y and sum may be NULL (sum goes with a residual;
 *              y or q is asked for); sum may be the residual itself, with its stride
 *   weight     [H] of weight_dtype: `dtype` or MOE_F32
 *   q          uint8 [M, H] E4M3 codes, scales fp32 [M, ceil(H / 128)], or both NULL
 *   rstd       fp32 [M] or NULL
 *   eps        a positive normal number up to 2^126
 * moe_decode_rms_norm_backward, from dy [M, H], r as it was stored (sum, or x) and
 * rstd, n_c = r_c * rstd:
 *   dx_c = rstd * (dy_c weight_c - n_c * mean_i dy_i weight_i n_i) + dsum_c
 *   dweight_c = sum_m dy_mc n_mc     fp32 [H], the rows' sums in a fixed order
 * dx is the gradient of x and of the residual.  dsum (the gradient that reaches `sum`
 * from elsewhere) may be NULL (0), or dx itself with its stride.  `workspace` is device memory
 * of at least moe_decode_rms_norm_backward_workspace() bytes, 256-byte aligned, used
 * until the launches complete (calls that may overlap in time need one each); it need
 * not be cleared.
 * Limits: H <= 32768; M < 2^26 up to 1024 columns, 2^24 up to 16384, else 2^22;
 * strides up to 2^30.  M == 0 is a valid no-op that writes nothing: dweight, whose sums
 * are then of no rows, keeps what it holds (0 before the call, as for counts above). */
int moe_decode_rms_norm(const void *x, long long ld_x, const void *residual, long long ld_residual, int dtype,
                        const void *weight, int weight_dtype, float eps, void *y, long long ld_y,
                        uint8_t *q, float *scales, void *sum, long long ld_sum, float *rstd,
                        int M, int H, int flags, void *stream);
int moe_decode_rms_norm_backward_workspace(int M, int H, size_t *bytes);
int moe_decode_rms_norm_backward(const void *dy, long long ld_dy, const void *r, long long ld_r, int dtype,
                                 const void *weight, int weight_dtype, const float *rstd,
                                 const void *dsum, long long ld_dsum, void *dx, long long ld_dx, float *dweight,
                                 void *workspace, size_t workspace_bytes, int M, int H, void *stream);

/* Low-rank adapters of many requests beside a projection:
 *   y[m, n] = base[m, n] + scaling[l] * sum_r b[l, n, r] * sum_c a[l, r, c] * x[m, c]
 * with l = row_adapters[m]; a row whose l lies outside [0, L) gets the base alone.
 * Both sums are FP32, the inner ones not rounded to 16 bits between the two (they
 * enter the second as the sum of two 16-bit numbers, to 2^-16 of themselves, in FP16
 * of the row's largest), and the result is rounded once.
 *   x             [M, K] of `dtype` (MOE_BF16 or MOE_F16), row m at m * ld_x elements
 *   row_adapters  int32 [M]
 *   a             [L, R, K];  b  [L, N, R];  scaling  fp32 [L]
 *   base          [M, N] of `dtype`, or NULL (0); it may be y itself, with y's stride
 *   y             [M, N] of `dtype`
 * K, R and ld_x multiples of 8; x, a and b 16-byte aligned.
 * Limits: R <= 256, L <= 1023, M < 2^22, K and N <= 2^20, strides up to 2^30.
 * `workspace` is device memory of at least moe_decode_adapters_workspace() bytes,
 * 256-byte aligned, used until the launches complete (calls that may overlap in time
 * need one each); it need not be cleared, and where that says 0 bytes it is not
 * looked at.  The size never goes down where M grows.  M == 0 is a valid no-op. */
int moe_decode_adapters_workspace(int M, int K, int N, int R, int L, size_t *bytes);
int moe_decode_adapters(const void *x, long long ld_x, int dtype, const int32_t *row_adapters,
                        const void *a, const void *b, const float *scaling,
                        const void *base, long long ld_base, void *y, long long ld_y,
                        void *workspace, size_t workspace_bytes, int M, int K, int N, int R, int L, void *stream);

/* Bandwidth probes that set the denominator of the efficiency figure (blog
 * post, "Hardware efficiency": peak measured with a copy kernel over
 * contiguous memory).  copy: dst[0:bytes) = src[0:bytes); read: reads
 * src[0:bytes) and writes nothing unless an impossible checksum appears
 * (sink: one 4-byte device word).  bytes must be a positive multiple of 16,
 * pointers 16-byte aligned, src and dst disjoint.  Asynchronous on `stream`. */
int moe_decode_copy_peak(const void *src, void *dst, size_t bytes, void *stream);
int moe_decode_read_peak(const void *src, size_t bytes, void *sink, void *stream);

/* Static description of a return code (never NULL). */
const char *moe_decode_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
