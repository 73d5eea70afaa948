/*
 * mol_block.h -- the MoE block around the LoRA path of mol.h, on GB300 (sm_103a).
 *
 * The LoRA stages of mol.h add adapter deltas into the products of a MoE
 * layer. These calls are the rest of that layer at decode widths:
 *
 *   mol_block_norm   the norm after a block, its gate and residual scale, the
 *                    residual add and the norm before the next block;
 *   mol_moe_route    the router's choice: topk expert ids and their weights;
 *   mol_moe_forward  the experts for a few tokens (bf16 or 4-bit weights), in
 *                    two kernels; mol_moe_gate_up and mol_moe_down are its
 *                    halves, each adding the rows of a LoRA stage;
 *   mol_w4_linear    one linear with 4-bit weights and group scales for a few
 *                    tokens.
 *
 * The conventions of mol.h hold: device pointers owned by the caller, calls
 * only enqueue on `stream`, arguments are checked on the host first, nothing
 * is launched on an error status, no size is rejected after a launch. Rows are
 * 16-byte aligned (pointers, and strides in elements a multiple of 8).
 *
 * 4-bit rows ("w4"). A row of K inputs is padded to Kp = ceil(K / 256) * 256 and
 * takes Kp / 2 bytes: 32-bit little-endian words, sixteen to each block of 128
 * inputs. Word 4 * t + i of a block (t, i in 0..3) holds the inputs
 * 32 * i + 8 * t + j, j in 0..7: input j in bits [4 * (j / 2), +4) for even j and
 * [16 + 4 * (j / 2), +4) for odd j (the two halves of a register then hold
 * neighbouring inputs). Its scales are Kp / group bf16 values, group in
 * {32, 64, 128}; the weight is scale[k / group] * (q - 8), q in 0..15. Padding
 * inputs and their scales take no part, whatever they hold.
 */
#ifndef MOL_BLOCK_H_
#define MOL_BLOCK_H_

#include "mol.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOL_NORM_MAX_H 16384      /* widest row of mol_block_norm */
#define MOL_ROUTE_MAX_EXPERTS 1024
#define MOL_ROUTE_MAX_TOPK 32
#define MOL_MOE_MAX_TOKENS 128    /* most tokens of one experts call */
#define MOL_MOE_MAX_PAIRS 1024    /* most (token, slot) pairs of one experts call */
#define MOL_MOE_MAX_EXPERTS 1024
#define MOL_MOE_MAX_WIDTH 65536   /* widest hidden / intermediate size, and K of the linear */
#define MOL_W4_MAX_TOKENS 64      /* most tokens of one mol_w4_linear call */

#define MOL_F32 0
#define MOL_BF16 1

/*
 * Norms before and after a block. With rms(v; w) = v * w / sqrt(mean(v^2) + eps),
 * for each token row:
 *   n            = rms(y; post_weight)          (y itself when post_weight is NULL)
 *   residual_out = residual + residual_scale * gate * n    (gate 1 when NULL)
 *   normed       = rms(residual_out before its rounding; pre_weight)
 * All in fp32, each output rounded to bf16 once.
 *   y, residual   bf16 rows of H at y + t * y_row_stride (elements)
 *   post_weight, pre_weight   bf16 [H] or NULL
 *   gate          bf16 rows at gate + t * gate_row_stride; stride 0: one row for all
 *   residual_out  bf16 rows; may be `residual` itself (same stride)
 *   normed        bf16 rows, or NULL exactly when pre_weight is NULL; may be `y`
 *                 itself (same stride); any other overlap of inputs and outputs
 *                 is outside the contract
 * Contract: 8 <= H <= MOL_NORM_MAX_H, H % 8 == 0, row strides >= H (gate: or 0),
 * 0 <= eps < infinity, num_tokens < 2^31.
 */
int32_t mol_block_norm(const void* y, int64_t y_row_stride, const void* residual,
                       int64_t residual_row_stride, const void* post_weight, const void* gate,
                       int64_t gate_row_stride, float residual_scale, const void* pre_weight,
                       float eps, int64_t num_tokens, int32_t H, void* residual_out,
                       int64_t residual_out_row_stride, void* normed, int64_t normed_row_stride,
                       void* stream);

/*
 * The router's choice. Each row's topk largest logits, the lower index first
 * among equal ones; a logit of -infinity or NaN is never taken.
 *   topk_ids[t, j]     the j-th expert, or -1 when the row has no more to take
 *   topk_weights[t, j] scale * exp(l_j - max) / sum, 0 where the id is -1; the sum
 *                      is over the row's taken experts (renormalize = 1) or over
 *                      all its experts (0); +infinity counts as its row's maximum
 * The ids feed mol_lora_forward, mol_align_block_size (after the remap) and the
 * experts calls below as they are.
 *   logits   MOL_F32 or MOL_BF16 rows at logits + t * row_stride (any alignment
 *            of the element type)
 *   topk_ids int32 [num_tokens, topk], topk_weights fp32 [num_tokens, topk]
 * Contract: 1 <= topk <= min(num_experts, MOL_ROUTE_MAX_TOPK),
 * num_experts <= MOL_ROUTE_MAX_EXPERTS, num_tokens * topk <= MOL_MAX_NUMEL.
 */
int32_t mol_moe_route(const void* logits, int32_t logits_dtype, int64_t row_stride,
                      int64_t num_tokens, int32_t num_experts, int32_t topk, int32_t renormalize,
                      float scale, int32_t* topk_ids, float* topk_weights, void* stream);

/*
 * First half of the experts: for each pair i = (token t, slot) with expert
 * e = topk_ids[i] in [0, num_experts),
 *   v = w[e] . x[t] (+ delta[i]),   act[i, j] = silu(v[j]) * v[inter + j],  j < inter
 * in fp32, rounded to bf16 once. Rows of other pairs (id -1: another device's
 * expert, no expert) are not written.
 *   x        bf16 rows of `hidden` at x + t * x_row_stride
 *   topk_ids int32 [num_tokens, topk]
 *   w        [num_experts, 2 * inter, hidden], gate rows then up rows: bf16 when
 *            group = 0 (w_scales NULL), else w4 rows with w_scales
 *            [num_experts, 2 * inter, Kp / group]
 *   delta    bf16 rows of 2 * inter at delta + i * delta_row_stride, or NULL: what
 *            mol_lora_forward added into a buffer of zeros
 *   act      bf16 [num_tokens * topk, inter]
 * Contract: num_tokens <= MOL_MOE_MAX_TOKENS, num_tokens * topk <=
 * MOL_MOE_MAX_PAIRS, num_experts <= MOL_MOE_MAX_EXPERTS, hidden % 8 == inter % 8
 * == 0, both <= MOL_MOE_MAX_WIDTH, group in {0, 32, 64, 128}. No output may
 * overlap an input.
 */
int32_t mol_moe_gate_up(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                        int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                        int32_t inter, const void* w, const void* w_scales, int32_t group,
                        const void* delta, int64_t delta_row_stride, void* act, void* stream);

/*
 * Second half: out[t] = sum over the slots of t of
 * topk_weights[i] * (w[e] . act[i] (+ delta[i])), pairs without an expert left
 * out, in fp32, rounded to bf16 once. Every row is written (zeros for a token
 * without any expert). The order of the sums, here and in mol_moe_gate_up, is fixed
 * by the sizes and topk_ids: equal inputs give equal bits. A token's row may differ
 * in its last bits when other tokens of the call take other experts.
 *   w        [num_experts, hidden, inter] as above (w_scales [.., hidden, Kp / group])
 *   delta    bf16 rows of `hidden` at delta + i * delta_row_stride, or NULL
 *   out      bf16 rows of `hidden` at out + t * out_row_stride
 */
int32_t mol_moe_down(const void* act, const int32_t* topk_ids, const float* topk_weights,
                     int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                     int32_t inter, const void* w, const void* w_scales, int32_t group,
                     const void* delta, int64_t delta_row_stride, void* out,
                     int64_t out_row_stride, void* stream);

/*
 * Both halves in one call; act is scratch of num_tokens * topk * inter bf16: the
 * first half's values are rounded to bf16 between the halves here too.
 */
int32_t mol_moe_forward(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                        const float* topk_weights, int64_t num_tokens, int32_t topk,
                        int32_t num_experts, int32_t hidden, int32_t inter, const void* w_gate_up,
                        const void* gate_up_scales, const void* w_down, const void* down_scales,
                        int32_t group, void* act, void* out, int64_t out_row_stride, void* stream);

/*
 * mol_moe_down and mol_moe_forward with a workspace, where they take one step more
 * for many pairs: the products of each pair in fp32, then their weighted sums.
 * Same contract and result (a token's pairs are added in the order of its slots
 * then, the deltas after the products).
 *   workspace  device, >= mol_moe_workspace_bytes of the sizes, 16-byte aligned
 *              (may be NULL when that is 0); contents are scratch
 */
size_t mol_moe_workspace_bytes(int64_t num_tokens, int32_t topk, int32_t num_experts,
                               int32_t hidden, int32_t inter, int32_t group);
int32_t mol_moe_down_split(const void* act, const int32_t* topk_ids, const float* topk_weights,
                           int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                           int32_t inter, const void* w, const void* w_scales, int32_t group,
                           const void* delta, int64_t delta_row_stride, void* workspace,
                           size_t workspace_bytes, void* out, int64_t out_row_stride,
                           void* stream);
int32_t mol_moe_forward_split(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                              const float* topk_weights, int64_t num_tokens, int32_t topk,
                              int32_t num_experts, int32_t hidden, int32_t inter,
                              const void* w_gate_up, const void* gate_up_scales,
                              const void* w_down, const void* down_scales, int32_t group,
                              void* act, void* workspace, size_t workspace_bytes, void* out,
                              int64_t out_row_stride, void* stream);

/*
 * out[t, n] = sum_k w[n, k] * x[t, k] in fp32, rounded to bf16 once.
 *   x    bf16 rows of K at x + t * x_row_stride
 *   w    w4 rows [N, Kp / 2 bytes], scales bf16 [N, Kp / group]
 *   out  bf16 rows of N at out + t * out_row_stride (2-byte aligned, any stride >= N)
 * Contract: num_tokens <= MOL_W4_MAX_TOKENS, K % 8 == 0, K <= MOL_MOE_MAX_WIDTH,
 * 1 <= N <= 2^30, group in {32, 64, 128}.
 */
int32_t mol_w4_linear(const void* x, int64_t x_row_stride, int64_t num_tokens, int32_t K, int32_t N,
                      const void* w, const void* scales, int32_t group, void* out,
                      int64_t out_row_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOL_BLOCK_H_ */
