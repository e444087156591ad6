/*
 * v4moe.h -- C ABI of libv4moe: the DeepSeek-V4-style MoE layer forward on one
 * MI355X (gfx950), with FP4 (MXFP4) expert weights dequantised losslessly to
 * FP8 E4M3 for FP8 matrix-core contractions.
 *
 * Sources (cited by short tag and section):
 *   P1 = "DeepSeek-V4揭秘：细粒度专家并行隐藏通信时延，FP4量化与TileLang协同优化百万Token上下文"
 *        (itsolotime.com/archives/32374)
 *   P2 = "DeepSeek V4架构学习笔记" (67808.cn/a/484462.html)
 *   P4 = "DeepSeek-V4 的暗线之二：训练一台不会失控的万亿参数机器"
 *        (blog.xieydd.top/deepseek-v4-control-part2)
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller; the library
 *     never allocates, frees or keeps them.  Outputs are fully overwritten.
 *   - Calls are asynchronous on `stream` (a hipStream_t passed as void*; NULL
 *     is the default stream) and never synchronise the host, except
 *     moe_prepack_weights, which is an offline step and synchronises.
 *   - bf16 values travel as uint16_t bit patterns; E4M3 and FP4 as bytes.
 *   - Return value: 0 on success, a negative V4MOE_E* code otherwise (no
 *     exceptions cross the ABI).  A code is returned before anything is
 *     enqueued.  Device faults surface at the caller's next synchronisation.
 *   - T = 0 is a valid no-op: only expert_offsets (E+1 zeros) is written, by
 *     moe_permute and moe_layer_forward; pointers to empty arrays may be NULL.
 *   - Results are deterministic and batch-invariant: a token's outputs do not
 *     depend on the other tokens of the batch nor on run-to-run scheduling
 *     (P1 §3.1 batch invariance, §3.2 determinism).  No atomics accumulate
 *     data; atomics only hand out work and signal readiness.
 *   - Not thread-safe per workspace: concurrent calls must use distinct
 *     workspaces.
 */
#ifndef V4MOE_H
#define V4MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Error codes. */
#define V4MOE_OK               0
#define V4MOE_ENULL           -1   /* a required pointer is NULL                       */
#define V4MOE_EDIMS           -2   /* unsupported or inconsistent dimensions            */
#define V4MOE_EALIGN          -3   /* a pointer is not 16-byte aligned                  */
#define V4MOE_EWORKSPACE      -4   /* workspace too small (see moe_workspace_bytes)     */
#define V4MOE_ELAUNCH         -5   /* a HIP launch or runtime call failed               */
#define V4MOE_ESCALE          -6   /* sub-block scale outside the lossless window       */
#define V4MOE_EDEVICE         -7   /* current device is not a gfx950                    */

/* Layer dimensions.  Requirements: 0 <= T; T*topk <= 2^24; T*H < 2^31;
 * T*topk*I < 2^31; H a multiple of 256 with 256 <= H <= 16384; I a multiple
 * of 128 with 128 <= I <= 16384; 1 <= E <= 1024; 1 <= topk <= min(E, 16). */
typedef struct {
    int32_t T;      /* tokens in the batch                          */
    int32_t H;      /* hidden size (linear1 K, linear2 N)           */
    int32_t I;      /* expert intermediate size (linear1 N, linear2 K) */
    int32_t E;      /* routed experts                               */
    int32_t topk;   /* experts per token                            */
    int32_t act;    /* expert activation, V4MOE_ACT_* (0: SwiGLU)   */
} v4moe_dims;

/* Expert activations.  SwiGLU (P1 §1.4): h = SiLU(gate x) * (up x).  The
 * gate-less ones are the cheap alternative the pages recommend (P1, the
 * hardware suggestions closing §1: an elementwise activation with no
 * exponential or division, and no gate projection so that the intermediate
 * can be wider at the same parameter count; the pages name no function):
 * h = max(up x, 0)^2 or h = max(up x, 0).  Gate-less layers have no gate
 * matrix (its pointers are ignored) and need I % 256 == 0. */
#define V4MOE_ACT_SWIGLU 0
#define V4MOE_ACT_RELU2  1
#define V4MOE_ACT_RELU   2

/* One expert weight matrix for all E experts: N output rows, K inputs.
 * P1 §4 (FP4 quantisation-aware training): FP4 E2M1 elements with a scale per
 * 1x32 sub-block, nested in 128x128 FP8 quantisation blocks.
 *
 * CANONICAL layout (what a checkpoint holds; input of moe_prepack_weights):
 *   fp4  uint8 [E][N][K/2]     K contiguous; element k in the low nibble when k is even
 *   e8m0 uint8 [E][N][K/32]    sub-block scale 2^b stored as the byte 127+b
 *   blk  fp32  [E][N/128][K/128]  scale of each 128x128 block
 * PACKED layout (output of moe_prepack_weights; what every compute entry
 * point reads).  Same byte counts; blk is unchanged.  N must be a multiple
 * of 64 (true for every matrix: N is I or H).
 *   fp4  uint8 [E][N/16][K/128][64][16]  for each expert, 16-row group n16 and
 *        128-wide K chunk c, a 1 KiB record of 64 slots of 16 bytes; slot s
 *        holds row n16*16 + s%16, elements k = c*128 + (s/16)*32 + [0, 32),
 *        in canonical nibble order (element k in byte k/2, low nibble when k
 *        is even);
 *   e8m0 uint8 [E][N/64][K/128][64][4]   for each group of four consecutive
 *        n16 and each chunk c, a 256-byte record; byte t of its dword s is the
 *        sub-block scale of slot s of n16 = 4*group + t;
 *   blk  fp32  [E][N/128][K/128]
 */
typedef struct {
    const void*  fp4;
    const void*  e8m0;
    const float* blk;
} v4moe_mat;

/* The expert weights (P1 §1.4: gate, up and down projections).
 * gate, up: N = I, K = H.  down: N = H, K = I.  gate is ignored (may be all
 * NULL) for the gate-less activations. */
typedef struct {
    v4moe_mat gate;
    v4moe_mat up;
    v4moe_mat down;
} v4moe_experts;

#define V4MOE_ROUTE_LEARNED 0
#define V4MOE_ROUTE_HASH    1

/* Workspace bytes needed by moe_route, moe_permute, moe_expert_ffn and
 * moe_layer_forward for these dimensions (host-only, pure).  Returns 0 for
 * invalid dims.  The workspace is device memory owned by the caller,
 * 16-byte aligned; its contents need no initialisation. */
size_t moe_workspace_bytes(const v4moe_dims* d);

/* Routing (P2, DeepSeekMoE notes: the affinity is sqrt(softplus(.)) in place
 * of V3's sigmoid; the early layers use hash routing).
 *   x         bf16 [T][H]
 *   w_router  fp32 [H][E]
 *   bias      fp32 [E] or NULL: added to the logits (selection and weights)
 *   mode      V4MOE_ROUTE_LEARNED: logits z[t][e] = one fp32 fused
 *             multiply-add chain over h = 0 .. H-1 ascending, starting from
 *             +0 (x exact as fp32), + bias as one fp32 add afterwards; the
 *             topk largest z are taken, ties to the lower expert id, slot j
 *             = j-th pick; a = sqrt(softplus(z)); topk_w = a / sum(a) over
 *             the picks.
 *             V4MOE_ROUTE_HASH: expert_j = splitmix64(id*topk + j) mod E,
 *             stepping +1 mod E past experts already picked; topk_w = 1/topk.
 *   token_ids int64 [T] or NULL (NULL: id = t); hash mode only.
 *   topk_ids  int32 [T][topk]   (out)
 *   topk_w    fp32  [T][topk]   (out)
 *   workspace moe_workspace_bytes(d) bytes (learned mode; may be NULL in hash mode)
 * x, w_router, workspace: 16-byte aligned. */
int moe_route(const v4moe_dims* d, const uint16_t* x, const float* w_router,
              const float* bias, int32_t mode, const int64_t* token_ids,
              int32_t* topk_ids, float* topk_w, void* workspace, size_t ws_bytes,
              void* stream);

/* Dispatch on one GPU (P1 §1.1-1.2: the FP8 dispatch stage becomes a local
 * expert-sorted permutation; P1 §1.4: FP8 dispatch payload).
 *   x              bf16 [T][H]
 *   topk_ids       int32 [T][topk] (as produced by moe_route; ids must be in [0,E))
 *   expert_offsets int32 [E+1]  (out) exclusive scan of per-expert pair counts
 *   sorted_pair    int32 [T*topk] (out) pair ids p = t*topk+j, stably sorted by expert
 *   pair_pos       int32 [T*topk] (out) inverse of sorted_pair
 *   xq             uint8 [T][H]  (out) E4M3 codes of x: per token and 128-channel
 *                  group g, s = fp32(amax/448) (1 if the group is zero) and
 *                  q = E4M3(fp32(x/s)), round to nearest even, saturating
 *   xs             fp32 [T][H/128] (out) the scales s
 * The FP8 rows are gathered by the expert FFN on load: they are never
 * materialised in expert order.  x, xq: 16-byte aligned. */
int moe_permute(const v4moe_dims* d, const uint16_t* x, const int32_t* topk_ids,
                int32_t* expert_offsets, int32_t* sorted_pair, int32_t* pair_pos,
                uint8_t* xq, float* xs, void* workspace, size_t ws_bytes, void* stream);

/* Expert FFN over all experts, unfused schedule (linear1 + SwiGLU for every
 * expert, then linear2 for every expert; P1 §1.1 stage model).
 * For each pair p routed to expert e (rows of e in sorted order):
 *   G, U = per-128-K-chunk FP8 products of xq[t] with the dequantised gate/up
 *          rows, each chunk scaled by xs[t][c] * blk[n/128][c], fp32 accumulation;
 *   h    = SiLU(G) * U  (fp32), requantised to E4M3 per 128 channels like x;
 *   y[p] = bf16 of the same chunked product of h with the down rows.
 *   y    bf16 [T*topk][H] (out), row p = t*topk + j.
 * w: PACKED weights.  xq, y and all weight arrays: 16-byte aligned. */
int moe_expert_ffn(const v4moe_dims* d, const uint8_t* xq, const float* xs,
                   const int32_t* expert_offsets, const int32_t* sorted_pair,
                   const v4moe_experts* w, uint16_t* y,
                   void* workspace, size_t ws_bytes, void* stream);

/* Combine as a weighted un-permute (P1 §1.4: BF16 combine payload; P1 §3.2:
 * no atomics):  out[t] = bf16( sum_{j=0..topk-1} topk_w[t][j] * y[t*topk+j] ),
 * summed in fp32 in increasing j.  y, out: 16-byte aligned. */
int moe_combine(const v4moe_dims* d, const uint16_t* y, const float* topk_w,
                uint16_t* out, void* stream);

/* The whole layer: route, dispatch, then the expert FFN, then the combine.
 * When experts get at most 64 rows per m-tile (weight-streaming batches) the
 * FFN is one persistent kernel that runs the experts in waves of 8 (P1 §1.2
 * and Fig. 5: the compute of wave w overlaps the gather of wave w+1 and the
 * scatter-back of finished experts); with 128-row m-tiles it is the two
 * launches of moe_expert_ffn, which measured faster there.  Same tiles and
 * arithmetic either way, so the output is bit-identical to moe_route +
 * moe_permute + moe_expert_ffn + moe_combine.
 *   topk_ids, topk_w, expert_offsets: outputs exported for checking.
 *   out bf16 [T][H]. */
int moe_layer_forward(const v4moe_dims* d, const uint16_t* x, const float* w_router,
                      const float* bias, int32_t mode, const int64_t* token_ids,
                      const v4moe_experts* w, int32_t* topk_ids, float* topk_w,
                      int32_t* expert_offsets, uint16_t* out,
                      void* workspace, size_t ws_bytes, void* stream);

/* moe_layer_forward without a caller workspace, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same arguments, kernels and results as
 * moe_layer_forward (bit-identical outputs); the workspace is instead a
 * static device array of the library, one per GPU, of
 * moe_noalloc_max_workspace_bytes() bytes (16 MiB: the full decode layer, H =
 * 4096, I = 2048, E = 256, top-8, fits up to T = 189), held by each GPU the
 * library runs on until the process ends.  Nothing is allocated or freed.
 * Errors: V4MOE_EDIMS for unsupported dimensions; V4MOE_EWORKSPACE when
 * moe_workspace_bytes(d) exceeds the array (nothing is enqueued); otherwise
 * as moe_layer_forward.  Every call on one GPU shares the array: calls that
 * overlap on a GPU (other streams, other host threads) race, calls on one
 * stream are ordered.  No contents need to survive between calls. */
size_t moe_noalloc_max_workspace_bytes(void);
int moe_layer_forward_noalloc(const v4moe_dims* d, const uint16_t* x, const float* w_router,
                              const float* bias, int32_t mode, const int64_t* token_ids,
                              const v4moe_experts* w, int32_t* topk_ids, float* topk_w,
                              int32_t* expert_offsets, uint16_t* out, void* stream);

/* FP32 master weights -> FP4 weights (P1 §4 and P4 §4: FP4 quantisation-aware
 * training quantises the FP32 master weights to FP4 in the forward pass;
 * element format and shared-exponent rule per the OCP MX specification the
 * pages cite).
 *   w: device fp32 [E][N][K], row-major, finite values; N % 128 == 0,
 *      K % 128 == 0; 16-byte aligned.
 *   packed: 0 writes the CANONICAL layout (fp4 [E][N][K/2], e8m0
 *      [E][N][K/32]); non-zero writes the PACKED layout the matrix kernels
 *      read, byte for byte what moe_prepack_weights makes of the canonical
 *      output (so a training step needs no separate prepack).
 *   out: device matrix in that layout plus blk [E][N/128][K/128], written in
 *      full.
 * Per 128x128 block, s = max|w| / 384 in fp32 (1 for an all-zero block), so
 * the block's largest magnitude maps to 6 * 2^6, FP4's largest value at the
 * top of the lossless window.  Per 1x32 sub-block of a row, v = w / s in fp32,
 * b = floor(log2(max|v|)) - 2, raised to -8 when below the window (such a
 * sub-block is "clamped": it keeps fewer significant codes), 0 for an
 * all-zero sub-block; each element is the E2M1 code nearest to v * 2^-b,
 * ties to the even code, saturating at 6, sign kept (-0.0 gives code 8).
 * clamped: device uint64 to which the number of clamped sub-blocks is added
 * (the caller clears it), or NULL.  Asynchronous on `stream`; allocates
 * nothing.  The output passes moe_prepack_weights' window check. */
int moe_quantize_weights(int32_t E, int32_t N, int32_t K, const float* w, int32_t packed,
                         const v4moe_mat* out, uint64_t* clamped, void* stream);

/* Offline: canonical -> packed weight layout (both device buffers of equal
 * size; blk pointers of `packed` may alias those of `canonical`).  Checks that
 * every sub-block exponent b lies in the lossless window [-8, 6] (P1 §4: the
 * FP4->FP8 conversion is exact while the sub-block scales of a block stay
 * within a bounded ratio; with E4M3 subnormals that window is b in [-8, 6]).
 * Needs a workspace of at least 256 bytes; synchronises `stream`. */
int moe_prepack_weights(const v4moe_dims* d, const v4moe_experts* canonical,
                        const v4moe_experts* packed, void* workspace, size_t ws_bytes,
                        void* stream);

/* Test export of the weights exactly as the matrix kernels consume them:
 * expert `expert` of the PACKED matrix m (N rows, K inputs; N % 64 == 0,
 * K % 128 == 0) is read through the same block-scaled FP8 x FP4 MFMA path as
 * the GEMMs and written as E4M3 bytes [N][K] in canonical row-major order
 * (P1 §4: inside the window every FP4 value times its sub-block scale is an
 * E4M3 value, so the bytes are exact; a zero keeps its code's sign). */
int moe_dequant_fp8(const v4moe_mat* m, int32_t N, int32_t K, int32_t expert,
                    uint8_t* out, void* stream);

/* ---- Backward (P1 §3 and P4 §3: the MoE backward accumulates in a fixed,
 * token-ordered sequence with no atomics; P1 §4 and P4 §4: gradients are
 * computed with the forward's FP8 weights and go straight to the FP32 master
 * weights, and the transposed weights are the same FP8 values) ---- */

/* Workspace bytes of moe_layer_backward (host-only, pure; 0 for invalid dims).
 * Device memory owned by the caller, 16-byte aligned, no initialisation. */
size_t moe_backward_workspace_bytes(const v4moe_dims* d);

/* The PACKED expert weights as transposed FP8 values, one OCP E4M3 byte each
 * (exact: inside the scale window every E2M1 code times its power-of-two
 * sub-block scale is an E4M3 value, the byte moe_dequant_fp8 gives; a zero
 * keeps its code's sign; the fp32 128x128 block scales are not applied and
 * stay in w):
 *   wt_gu: [E][H][2I] bytes with [e][h][i] = gate(e, i, h), [e][h][I + i] =
 *          up(e, i, h) (gate-less: [E][H][I] of up);
 *   wt_d:  [E][I][H] bytes with [e][i][h] = down(e, h, i).
 * Computed once per weight version and passed to moe_layer_backward (whose
 * matrix products read them as bf16, converted exactly when staged).
 * Asynchronous on `stream`; 16-byte aligned outputs. */
int moe_transpose_weights(const v4moe_dims* d, const v4moe_experts* w, uint8_t* wt_gu,
                          uint8_t* wt_d, void* stream);

/* Gradients of L = sum(dout * out) for the layer forward moe_layer_forward
 * computes on the same inputs (routing, quantisation and the FFN are
 * recomputed here).  The quantisation steps are straight-through, so
 *   dx  [T][H] fp32   = dL/dx (through the FP8 dispatch payload),
 *   dw  [T][topk] fp32 = dL/d(routing weight) = <dout_t, Y_p> (the router
 *                       itself is not differentiated),
 *   dWg, dWu [E][I][H], dWd [E][H][I] fp32 = dL/d(master weights): the
 *                       gradients with respect to the FP8 weight values
 *                       (dWg unused and may be NULL gate-less).
 * Every gradient is written in full (zeros for experts without tokens), by
 * one thread per element, in a fixed order: the result is bitwise
 * deterministic.  Products run on bf16 matrix cores with fp32 accumulation;
 * dout and the row gradients are rounded to bf16 before each product, as are
 * the forward activations (E4M3 code x scale) in the weight gradients.
 *   w: PACKED weights; wt_gu, wt_d: from moe_transpose_weights;
 *   dout: bf16 bits [T][H]; workspace: moe_backward_workspace_bytes(d).
 * Pointers 16-byte aligned. */
int moe_layer_backward(const v4moe_dims* d, const uint16_t* x, const float* w_router,
                       const float* bias, int32_t mode, const int64_t* token_ids,
                       const v4moe_experts* w, const uint8_t* wt_gu, const uint8_t* wt_d,
                       const uint16_t* dout, float* dx, float* dw, float* dWg, float* dWu,
                       float* dWd, void* workspace, size_t ws_bytes, void* stream);

/* ---- Operators next to the layer: gating from given logits, dense FP8
 * products, gradient clipping.  They follow the conventions above, except
 * that pointers need only the alignment stated with each call (V4MOE_EALIGN
 * otherwise) and that matrices may have a leading dimension (in elements)
 * larger than their rows. ---- */

/* Element types. */
#define V4MOE_TYPE_F32  0
#define V4MOE_TYPE_BF16 1

/* Scores of moe_gate. */
#define V4MOE_SCORE_SIGMOID      0   /* 1 / (1 + exp(-z))                  */
#define V4MOE_SCORE_SOFTMAX      1   /* exp(z - max) / sum over the experts */
#define V4MOE_SCORE_SQRTSOFTPLUS 2   /* sqrt(softplus(z))                  */

/* Gate: 0 <= T <= 2^24; 1 <= E <= 1024; 1 <= topk <= 16; 1 <= groups <= 64
 * dividing E; 1 <= topk_groups <= groups; topk <= topk_groups * E / groups. */
typedef struct {
    int32_t T;            /* tokens                                            */
    int32_t E;            /* experts                                           */
    int32_t topk;         /* experts per token                                 */
    int32_t score;        /* V4MOE_SCORE_*                                     */
    int32_t groups;       /* groups of E/groups consecutive experts (1: none)  */
    int32_t topk_groups;  /* groups a token may pick from                      */
    int32_t renorm;       /* non-zero: weights divided by their sum            */
    float   scale;        /* factor of the weights                             */
} v4moe_gate;

/* Routing from given logits; its outputs are what moe_permute and moe_combine
 * take.
 *   logits fp32 or bf16 (type) [T][ld], E used; NaN and values <= -1e30 (so
 *          -inf and the types' lowest values) mask an expert, values above
 *          1e30 count as 1e30
 *   bias   fp32 [E] or NULL, added to the scores for the selection only
 *          (-inf switches an expert off)
 *   topk_ids int32 [T][topk], topk_w fp32 [T][topk] (out)
 * key = score + bias, each one fp32 operation; a group's value is the sum of
 * its two largest keys (masked experts add nothing); of the topk_groups largest
 * groups the topk largest keys are picked in order; ties go to the lower group
 * and expert.  Weights are scale * score, divided by the sum of the picked
 * scores with renorm (0 where that is 0).  A token with fewer than topk
 * unmasked experts fills its slots with the lowest other ids, weight 0, so
 * that ids are distinct and in range in every row.  Pointers: aligned to their
 * element. */
int moe_gate(const v4moe_gate* g, const void* logits, int32_t type, int64_t ld, const float* bias,
             int32_t* topk_ids, float* topk_w, void* stream);

/* Gradient of L with respect to the logits of moe_gate, given dw = dL/dtopk_w
 * fp32 [T][topk] (moe_layer_backward's dw) and moe_gate's outputs; the selection
 * is held fixed, and slots of weight 0 have no gradient.
 *   dlogits [T][ldd] of the logits' type (out), its E columns written in full. */
int moe_gate_backward(const v4moe_gate* g, const void* logits, int32_t type, int64_t ld,
                      const int32_t* topk_ids, const float* topk_w, const float* dw, void* dlogits,
                      int64_t ldd, void* stream);

/* moe_layer_forward and moe_layer_backward with the routing given (moe_gate's
 * outputs: topk_ids int32 [T][topk], distinct per token and in [0, E); topk_w fp32
 * [T][topk], any values) instead of computed from x.  Same kernels, workspaces
 * (moe_workspace_bytes, moe_backward_workspace_bytes) and results as with that routing. */
int moe_routed_forward(const v4moe_dims* d, const uint16_t* x, const int32_t* topk_ids,
                       const float* topk_w, const v4moe_experts* w, int32_t* expert_offsets,
                       uint16_t* out, void* workspace, size_t ws_bytes, void* stream);
int moe_routed_backward(const v4moe_dims* d, const uint16_t* x, const int32_t* topk_ids,
                        const float* topk_w, const v4moe_experts* w, const uint8_t* wt_gu,
                        const uint8_t* wt_d, const uint16_t* dout, float* dx, float* dw, float* dWg,
                        float* dWu, float* dWd, void* workspace, size_t ws_bytes, void* stream);

/* E4M3 codes of x [M][K] (fp32 or bf16) with an fp32 scale for each group of
 * 128: s = fp32(amax / 448) (1 where that is 0), code = E4M3(fp32(x / s)),
 * nearest even, saturating.  A group holding an infinity or NaN gets scale NaN and
 * codes 0: every product it enters is NaN.  Either order, or both in one pass:
 *   q  [M][K16], s  [ceil(K/128)][M]: groups of 128 along a row (K16 = K rounded up
 *      to 16, the columns past K zero)
 *   qt [K][M16], st [ceil(M/128)][K]: the transpose, groups of 128 along a column
 * A pair may be NULL.  0 <= M, K <= 2^22.  q, qt: 16-byte aligned. */
int moe_fp8_quantize(int32_t M, int32_t K, const void* x, int32_t type, int64_t ldx,
                     uint8_t* q, float* s, uint8_t* qt, float* st, void* stream);

/* E4M3 weights: one scale for each 128x128 block, the same codes in both orders.
 *   w [N][K] fp32 or bf16; q [N][K16], qt [K][N16], blk fp32 [ceil(N/128)][ceil(K/128)] */
int moe_fp8_quantize_weights(int32_t N, int32_t K, const void* w, int32_t type, int64_t ldw,
                             uint8_t* q, uint8_t* qt, float* blk, void* stream);

/* Scales of the second operand of moe_fp8_gemm. */
#define V4MOE_SCALE_BLOCK 0   /* one per 128 rows and 128 of K: bs[(n/128)*bs_n + (k/128)*bs_k] */
#define V4MOE_SCALE_ROW   1   /* one per row and 128 of K: bs [ceil(K/128)][N]                  */

/* 0 <= M, N, K, lda, ldb <= 2^22; K, lda, ldb multiples of 16. */
typedef struct {
    int32_t M, N, K;
    int32_t b_scale;      /* V4MOE_SCALE_*                          */
    int32_t c_type;       /* V4MOE_TYPE_*                           */
    int32_t accumulate;   /* non-zero: c = what it holds + result, in fp32, rounded once */
    int64_t lda, ldb, ldc;
    int64_t bs_n, bs_k;   /* V4MOE_SCALE_BLOCK only                 */
} v4moe_gemm;

/* c[m][n] = sum over chunks i of 128 of as[i][m] * bs(n, i) * sum_{k in i} a[m][k] b[n][k].
 *   a uint8 [M][lda], as fp32 [ceil(K/128)][M], b uint8 [N][ldb], c [M][ldc]
 * Chunk sums come from the matrix cores, which align a chunk's products to the
 * largest and drop what lies far below it: a chunk is off by up to 4e-4 of its
 * largest product (measured; 1.0e-5 to 1.4e-5 of the result in the 2-norm for codes
 * of normal numbers, where fp32 products of the same values are off by 1e-7 to 1e-6:
 * an fp32 c holds more digits than it has).  Chunks are added in fp32, in order, in every variant, so a row
 * does not depend on the other rows.  K = 0 writes zeros.  a, b: 16-byte
 * aligned. */
int moe_fp8_gemm(const v4moe_gemm* g, const uint8_t* a, const float* as, const uint8_t* b,
                 const float* bs, void* c, void* stream);

/* A dense weight [N][K] as moe_fp8_quantize_weights writes it.  q is read by the
 * forward, qt by the data gradient. */
typedef struct {
    int32_t N, K;
    const uint8_t* q;
    const uint8_t* qt;
    const float* blk;
} v4moe_fp8mat;

/* Workspace bytes of moe_fp8_linear (backward = 0) and moe_fp8_linear_backward
 * (host-only, pure; 0 for invalid sizes).  16-byte aligned, no initialisation. */
size_t moe_fp8_linear_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t backward);

/* y = x W^T: x [M][K] quantised by rows, then the product. */
int moe_fp8_linear(int32_t M, const void* x, int32_t x_type, int64_t ldx, const v4moe_fp8mat* w,
                   void* y, int32_t y_type, int64_t ldy, void* workspace, size_t ws_bytes, void* stream);

/* Gradients of moe_fp8_linear, quantisation straight-through (as in
 * moe_layer_backward), with dy quantised by rows for dx and by columns for dW:
 *   dx [M][K] = dy W, dW [N][K] (+)= dy^T x.  dx or dw may be NULL.  With M = 0, dw
 * is set to zero (left alone with accumulate). */
int moe_fp8_linear_backward(int32_t M, const void* x, int32_t x_type, int64_t ldx, const void* dy,
                            int32_t dy_type, int64_t lddy, const v4moe_fp8mat* w, void* dx,
                            int32_t dx_type, int64_t lddx, void* dw, int32_t dw_type, int64_t lddw,
                            int32_t accumulate, void* workspace, size_t ws_bytes, void* stream);

/* A gradient of n elements (0 <= n <= 2^36), contiguous, aligned to its
 * element; out NULL or equal to g: in place.  What a call writes must not overlap
 * any other gradient or output of the list (V4MOE_EDIMS). */
typedef struct {
    const void* g;
    void* out;
    int64_t n;
    int32_t type;         /* V4MOE_TYPE_* */
} v4moe_tensor;

/* Workspace bytes of moe_clip_grads for a list of `count` (<= 2^20) tensors. */
size_t moe_clip_workspace_bytes(int32_t count);

/* norm = sqrt(sum of the squares of all elements of all tensors) (squares and
 * sums in fp64, a fixed order), coef = norm > max_norm ? max_norm / norm : 1, and
 * out = g * coef in each tensor's type.  An infinity or NaN among the elements
 * makes the norm that and leaves the gradients unscaled; a norm beyond fp32's
 * range is returned as infinity, and the gradients are scaled by it all the same.
 * Nothing is read back to the host.
 *   tensors: HOST array; norm: device fp32 [1] (out); max_norm >= 0 (infinity: the
 * norm only, and copies where out is not g). */
int moe_clip_grads(int32_t count, const v4moe_tensor* tensors, float max_norm, float* norm,
                   void* workspace, size_t ws_bytes, void* stream);

/* ---- Products grouped by expert, bf16 weights ----
 * Rows are sorted by expert: expert e has the rows offsets[e] <= m < offsets[e + 1]
 * (offsets int32 [E+1] on the device, as moe_permute writes them: ascending, within
 * [0, M]; 1 <= E <= 1024).  w bf16 [E][N][K], contiguous; x, dy, y, dx have leading
 * dimensions.  0 <= M, 1 <= N, K, and leading dimensions of bf16 operands, up to 2^22.
 * Sums are fp32, in an order that depends on the contraction alone: a row's result
 * does not depend on the other rows.  Rows before the first expert's and behind the
 * last one's take no part, and those of outputs are left as they are.  Pointers:
 * aligned to their element.  What a call writes must not overlap what it reads, but
 * for gradients added to (here and in the two sections below, where more is said). */

/* Workspace bytes of the calls below (host-only, pure; 0 for invalid sizes): operands
 * whose rows do not begin at 16 bytes, or are not a multiple of 8 elements long, are
 * copied there first, by every call and as a whole: of w all experts' rows, whether they
 * have rows of x or not.  The pointers are only looked at for that.  16-byte aligned. */
size_t moe_grouped_workspace_bytes(int32_t M, int32_t E, int32_t N, int32_t K, const uint16_t* x,
                                   int64_t ldx, const uint16_t* dy, int64_t lddy, const uint16_t* w,
                                   int32_t backward);

/* y[m] = W[e] x[m] for each row m of each expert e: y [M][ldy] of a type. */
int moe_grouped_linear(int32_t M, int32_t E, int32_t N, int32_t K, const uint16_t* x, int64_t ldx,
                       const uint16_t* w, const int32_t* offsets, void* y, int32_t y_type,
                       int64_t ldy, void* workspace, size_t ws_bytes, void* stream);

/* Its gradients: dx[m] = W[e]^T dy[m], dW[e] (+)= sum over e's rows of dy[m] x[m]^T
 * (dw [E][N][K], contiguous; with accumulate added to in fp32 and rounded once).
 * dx or dw may be NULL.  Experts without rows get a dW of zeros (with accumulate:
 * theirs is left alone). */
int moe_grouped_linear_backward(int32_t M, int32_t E, int32_t N, int32_t K, const uint16_t* x,
                                int64_t ldx, const uint16_t* dy, int64_t lddy, const uint16_t* w,
                                const int32_t* offsets, void* dx, int32_t dx_type, int64_t lddx,
                                void* dw, int32_t dw_type, int32_t accumulate, void* workspace,
                                size_t ws_bytes, void* stream);

/* The tile that a product of these calls takes, for a reader of a profile (host-only, pure):
 * rows << 16 | columns, and V4MOE_TILE_SHARED where both gradients go out in one launch; 0
 * for invalid arguments.  what: V4MOE_PRODUCT_*; both: both gradients are asked for.  Results
 * do not depend on it, in any bit. */
#define V4MOE_PRODUCT_FORWARD 0   /* y; the cross entropy's logits              */
#define V4MOE_PRODUCT_DX      1
#define V4MOE_PRODUCT_DW      2
#define V4MOE_PRODUCT_AGAIN   3   /* the cross entropy's logits in its backward */
#define V4MOE_TILE_SHARED     (1 << 30)
int32_t moe_grouped_tile(int32_t M, int32_t E, int32_t N, int32_t K, int32_t what, int32_t both);

/* ---- Softmax cross entropy over a large vocabulary, from the hidden states ----
 *   z = x W^T (x bf16 [T][ldx], W bf16 [V][ldw], H used of both), never in memory as a whole
 *   lse[t] = log sum_v exp(z[t][v]); loss[t] = lse[t] - z[t][targets[t]]
 * targets int64 [T]: a token whose target is not in [0, V) (-100, say) has loss and lse 0
 * and no gradient, costs no products, and what its row of x holds reaches nothing.
 * 0 <= T, 1 <= H, V, all up to 2^22, leading dimensions of x and W too.  fp32 sums; a
 * token's loss and lse do not depend on the other tokens, in any bit.  Pointers: aligned
 * to their element. */

/* Workspace bytes (host-only, pure; 0 for invalid sizes; W's pointer is looked at for its
 * alignment only: where its rows do not begin at 16 bytes, or H is no multiple of 8, there
 * is room for a copy).  16-byte aligned, no initialisation.  The backward holds the logits'
 * gradient of a piece of the vocabulary in it, at most 256 MiB or 256 columns. */
size_t moe_linear_xent_workspace_bytes(int32_t T, int32_t H, int32_t V, const uint16_t* w,
                                       int64_t ldw, int32_t backward);

/* loss, lse: fp32 [T] (out). */
int moe_linear_xent(int32_t T, int32_t H, int32_t V, const uint16_t* x, int64_t ldx,
                    const uint16_t* w, int64_t ldw, const int64_t* targets, float* loss, float* lse,
                    void* workspace, size_t ws_bytes, void* stream);

/* Gradients of sum_t dloss[t] loss[t], given lse from moe_linear_xent:
 *   d[t][v] = dloss[t] (exp(z[t][v] - lse[t]) - [v = targets[t]])
 *   dx [T][lddx] = d W;  dW [V][lddw] (+)= d^T x (accumulate: added to in fp32, rounded once)
 * dx or dw may be NULL.  dloss fp32, element t at dloss[t * dloss_stride] (0: one for all).
 * d enters the products in bf16 (divided by the largest |dloss| first), but at the targets
 * in 16 bits: fp32 results are good to 1e-5 to 1e-3 of their 2-norm, the first where the
 * probabilities are spread over many columns, the last where a few have them all.
 * accumulate | V4MOE_GRAD_FULL: all of d in 16 bits, for results that are good to about 5e-6
 * (what products in fp32 give), at twice the gradients' products. */
#define V4MOE_GRAD_FULL 2
int moe_linear_xent_backward(int32_t T, int32_t H, int32_t V, const uint16_t* x, int64_t ldx,
                             const uint16_t* w, int64_t ldw, const int64_t* targets, const float* lse,
                             const float* dloss, int64_t dloss_stride, void* dx, int32_t dx_type,
                             int64_t lddx, void* dw, int32_t dw_type, int64_t lddw,
                             int32_t accumulate, void* workspace, size_t ws_bytes, void* stream);

/* As moe_grouped_tile, of a cross entropy's products; those of its backward are of the first
 * piece of the vocabulary.  (dx is cut into slices of the vocabulary for its tile, so that its
 * last bits do depend on it.) */
int32_t moe_linear_xent_tile(int32_t T, int32_t H, int32_t V, int32_t what, int32_t both);

/* ---- Low-rank adapters of many requests beside a shared projection ----
 * Row m uses adapter ids[m] (int32 [M] on the device, in any order; outside [0, L): none)
 *   a bf16 [L][r][K], b bf16 [L][r][N], contiguous; scale fp32 [L]
 *   x, dy bf16 rows [M][ldx], [M][lddy]
 * 0 <= M, 1 <= N, K, leading dimensions of bf16 operands, all up to 2^22; 1 <= r <= 512;
 * 1 <= L <= 65535.  Sums are fp32 in a fixed order, the rank-sized intermediates kept to
 * 16 bits of significand, as two bf16 numbers (an infinite element of x, dy or a factor may
 * give NaN where one product would give an infinity); a row's result does not depend on the
 * other rows.  More than 64 ranks pass in pieces of 64, each over all rows.  Pointers:
 * aligned to their element. */
typedef struct {
    int32_t M;      /* rows                       */
    int32_t N;      /* columns of the projection  */
    int32_t K;      /* its inputs                 */
    int32_t r;      /* rank                       */
    int32_t L;      /* adapters                   */
} v4moe_lora;

/* Workspace bytes of moe_lora_add (backward = 0) and moe_lora_backward (host-only, pure; 0
 * for invalid sizes).  16-byte aligned, no initialisation. */
size_t moe_lora_workspace_bytes(const v4moe_lora* p, int32_t backward);

/* out[m] = y[m] + scale[i] B[i]^T (A[i] x[m]), i = ids[m]; rows without an adapter: out[m] =
 * y[m].  y [M][ldy], out [M][ldo] of one type (V4MOE_TYPE_*); out may be y. */
int moe_lora_add(const v4moe_lora* p, const void* y, int32_t type, int64_t ldy, const uint16_t* x,
                 int64_t ldx, const uint16_t* a, const uint16_t* b, const int32_t* ids,
                 const float* scale, void* out, int64_t ldo, void* workspace, size_t ws_bytes,
                 void* stream);

/* Its gradients, from dy = dL/dout:
 *   dx[m] = base[m] + scale[i] A[i]^T (B[i] dy[m])  (base: what the shared projection's
 *           backward gave, of dx's type; NULL: zeros; may be dx)
 *   da[i] (+)= scale[i] sum over i's rows of (B[i] dy[m]) x[m]^T
 *   db[i] (+)= scale[i] sum over i's rows of (A[i] x[m]) dy[m]^T
 * Any of dx, da, db may be NULL.  Adapters without rows get zeros (with accumulate: theirs are
 * left alone).  accumulate: da and db are added to, in fp32, rounded once. */
int moe_lora_backward(const v4moe_lora* p, const uint16_t* x, int64_t ldx, const uint16_t* dy,
                      int64_t lddy, const uint16_t* a, const uint16_t* b, const int32_t* ids,
                      const float* scale, const void* base, int64_t ldbase, void* dx,
                      int32_t dx_type, int64_t lddx, void* da, int32_t da_type, void* db,
                      int32_t db_type, int32_t accumulate, void* workspace, size_t ws_bytes,
                      void* stream);

/* Profiling hook (no effect on results).  start/stop are hipEvent_t handles
 * created by the caller (or NULL to clear).  The next moe_expert_ffn or
 * moe_layer_forward call made by this host thread records `start` on its
 * stream just before its expert-FFN matrix kernels (after the tile-list
 * build) and `stop` just after them, then forgets both; elapsed time between
 * them is the device time of the FFN kernels alone. */
void moe_time_next_ffn(void* start_event, void* stop_event);

/* Text for an error code. */
const char* moe_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* V4MOE_H */
