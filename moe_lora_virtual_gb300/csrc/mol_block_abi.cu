// Exported C ABI of the MoE block around the LoRA path (include/mol_block.h).
// Host code only: validation, dispatch to the launchers.

#include <cmath>

#include "mol_block.h"
#include "mol_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A bf16 row operand: at least `width` elements apart, 16-byte aligned rows.
int32_t check_rows(const void* p, int64_t stride, int64_t width) {
  if (!p || stride < width) return MOL_ERR_INVALID_ARG;
  return stride % 8 != 0 || !aligned16(p) ? MOL_ERR_UNSUPPORTED : MOL_OK;
}

int32_t check_weights(const void* w, const void* scales, int32_t group, bool w4_only) {
  if (!w) return MOL_ERR_INVALID_ARG;
  if (group == 0 && !w4_only) return scales ? MOL_ERR_INVALID_ARG
                                            : aligned16(w) ? MOL_OK : MOL_ERR_UNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return MOL_ERR_UNSUPPORTED;
  if (!scales) return MOL_ERR_INVALID_ARG;
  return aligned16(w) && aligned16(scales) ? MOL_OK : MOL_ERR_UNSUPPORTED;
}

int32_t check_moe_shape(int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                        int32_t inter) {
  if (num_tokens < 0 || topk < 1 || num_experts < 1 || hidden < 1 || inter < 1)
    return MOL_ERR_INVALID_ARG;
  if (num_tokens > MOL_MOE_MAX_TOKENS || num_tokens * topk > MOL_MOE_MAX_PAIRS ||
      num_experts > MOL_MOE_MAX_EXPERTS || hidden % 8 != 0 || inter % 8 != 0 ||
      hidden > MOL_MOE_MAX_WIDTH || inter > MOL_MOE_MAX_WIDTH)
    return MOL_ERR_UNSUPPORTED;
  return MOL_OK;
}

int32_t check_delta(const void* delta, int64_t stride, int64_t width) {
  return delta ? check_rows(delta, stride, width) : MOL_OK;
}

int32_t done(cudaError_t e) { return e == cudaSuccess ? MOL_OK : mol::cuda_fail(e); }

#define MOL_TRY(call)              \
  do {                             \
    const int32_t st_ = (call);    \
    if (st_ != MOL_OK) return st_; \
  } while (0)

int32_t check_down(const void* act, const int32_t* topk_ids, const float* topk_weights,
                   int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                   int32_t inter, const void* w, const void* w_scales, int32_t group,
                   const void* delta, int64_t delta_row_stride, const void* out,
                   int64_t out_row_stride) {
  MOL_TRY(check_moe_shape(num_tokens, topk, num_experts, hidden, inter));
  if (num_tokens == 0) return MOL_OK;
  if (!topk_ids || !topk_weights) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_rows(act, inter, inter));
  MOL_TRY(check_weights(w, w_scales, group, false));
  MOL_TRY(check_delta(delta, delta_row_stride, hidden));
  return check_rows(out, out_row_stride, hidden);
}

// Whether the split form is taken, for which the workspace has to do.
int32_t check_workspace(const mol::MoeShape& s, int32_t group, const void* workspace, size_t bytes,
                        bool& split) {
  const size_t need = mol::moe_split_bytes(s, group);
  split = need > 0;
  if (!split) return MOL_OK;
  if (!workspace || bytes < need) return MOL_ERR_CAPACITY;
  return aligned16(workspace) ? MOL_OK : MOL_ERR_UNSUPPORTED;
}

int32_t forward(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                const float* topk_weights, int64_t num_tokens, int32_t topk, int32_t num_experts,
                int32_t hidden, int32_t inter, const void* w_gate_up, const void* gate_up_scales,
                const void* w_down, const void* down_scales, int32_t group, void* act,
                void* workspace, size_t workspace_bytes, bool may_split, void* out,
                int64_t out_row_stride, void* stream) {
  MOL_TRY(check_moe_shape(num_tokens, topk, num_experts, hidden, inter));
  if (num_tokens == 0) return MOL_OK;
  if (!topk_ids || !topk_weights) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_rows(x, x_row_stride, hidden));
  MOL_TRY(check_weights(w_gate_up, gate_up_scales, group, false));
  MOL_TRY(check_weights(w_down, down_scales, group, false));
  MOL_TRY(check_rows(act, inter, inter));
  MOL_TRY(check_rows(out, out_row_stride, hidden));
  const mol::MoeShape s{(int)num_tokens, topk, num_experts, hidden, inter};
  bool split = false;
  if (may_split) MOL_TRY(check_workspace(s, group, workspace, workspace_bytes, split));
  MOL_TRY(mol::ensure_moe_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = mol::launch_moe_gate_up(
      s, x, x_row_stride, topk_ids, mol::WeightRows{w_gate_up, gate_up_scales, hidden, group},
      nullptr, 0, act, st);
  if (e != cudaSuccess) return mol::cuda_fail(e);
  const mol::WeightRows rows{w_down, down_scales, inter, group};
  return done(split ? mol::launch_moe_down_split(s, act, topk_ids, topk_weights, rows, nullptr, 0,
                                                 workspace, out, out_row_stride, true, st)
                    : mol::launch_moe_down(s, act, topk_ids, topk_weights, rows, nullptr, 0, out,
                                           out_row_stride, true, st));
}

}  // namespace

extern "C" {

int32_t mol_block_norm(const void* y, int64_t y_row_stride, const void* residual,
                       int64_t residual_row_stride, const void* post_weight, const void* gate,
                       int64_t gate_row_stride, float residual_scale, const void* pre_weight,
                       float eps, int64_t num_tokens, int32_t H, void* residual_out,
                       int64_t residual_out_row_stride, void* normed, int64_t normed_row_stride,
                       void* stream) {
  if (num_tokens < 0 || H < 1 || !(eps >= 0.f) || std::isinf(eps)) return MOL_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > MOL_NORM_MAX_H || num_tokens >= (int64_t)1 << 31)
    return MOL_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MOL_OK;
  if ((pre_weight == nullptr) != (normed == nullptr)) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_rows(y, y_row_stride, H));
  MOL_TRY(check_rows(residual, residual_row_stride, H));
  MOL_TRY(check_rows(residual_out, residual_out_row_stride, H));
  if (normed) MOL_TRY(check_rows(normed, normed_row_stride, H));
  if (gate) MOL_TRY(check_rows(gate, gate_row_stride, gate_row_stride == 0 ? 0 : H));
  if (!aligned16(post_weight) || !aligned16(pre_weight)) return MOL_ERR_UNSUPPORTED;
  MOL_TRY(mol::ensure_device());
  mol::NormArgs a = {};
  a.y = y;
  a.residual = residual;
  a.post_weight = post_weight;
  a.gate = gate;
  a.pre_weight = pre_weight;
  a.residual_out = residual_out;
  a.normed = normed;
  a.y_stride = y_row_stride;
  a.residual_stride = residual_row_stride;
  a.gate_stride = gate_row_stride;
  a.residual_out_stride = residual_out_row_stride;
  a.normed_stride = normed_row_stride;
  a.rows = num_tokens;
  a.H = H;
  a.residual_scale = residual_scale;
  a.eps = eps;
  return done(mol::launch_block_norm(a, static_cast<cudaStream_t>(stream)));
}

int32_t mol_moe_route(const void* logits, int32_t logits_dtype, int64_t row_stride,
                      int64_t num_tokens, int32_t num_experts, int32_t topk, int32_t renormalize,
                      float scale, int32_t* topk_ids, float* topk_weights, void* stream) {
  if (num_tokens < 0 || num_experts < 1 || topk < 1 || topk > num_experts ||
      (logits_dtype != MOL_F32 && logits_dtype != MOL_BF16) || renormalize < 0 || renormalize > 1 ||
      row_stride < num_experts)
    return MOL_ERR_INVALID_ARG;
  if (num_experts > MOL_ROUTE_MAX_EXPERTS || topk > MOL_ROUTE_MAX_TOPK ||
      num_tokens > MOL_MAX_NUMEL / topk)
    return MOL_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MOL_OK;
  if (!logits || !topk_ids || !topk_weights) return MOL_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (logits_dtype == MOL_F32 ? 4 : 2) != 0)
    return MOL_ERR_UNSUPPORTED;
  MOL_TRY(mol::ensure_device());
  return done(mol::launch_moe_route(logits, logits_dtype == MOL_BF16, row_stride, num_tokens,
                                    num_experts, topk, renormalize != 0, scale, topk_ids,
                                    topk_weights, static_cast<cudaStream_t>(stream)));
}

int32_t mol_moe_gate_up(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                        int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                        int32_t inter, const void* w, const void* w_scales, int32_t group,
                        const void* delta, int64_t delta_row_stride, void* act, void* stream) {
  MOL_TRY(check_moe_shape(num_tokens, topk, num_experts, hidden, inter));
  if (num_tokens == 0) return MOL_OK;
  if (!topk_ids) return MOL_ERR_INVALID_ARG;
  MOL_TRY(check_rows(x, x_row_stride, hidden));
  MOL_TRY(check_weights(w, w_scales, group, false));
  MOL_TRY(check_delta(delta, delta_row_stride, 2 * (int64_t)inter));
  MOL_TRY(check_rows(act, inter, inter));
  MOL_TRY(mol::ensure_moe_device());
  const mol::MoeShape s{(int)num_tokens, topk, num_experts, hidden, inter};
  return done(mol::launch_moe_gate_up(s, x, x_row_stride, topk_ids,
                                      mol::WeightRows{w, w_scales, hidden, group}, delta,
                                      delta_row_stride, act, static_cast<cudaStream_t>(stream)));
}

int32_t mol_moe_down(const void* act, const int32_t* topk_ids, const float* topk_weights,
                     int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                     int32_t inter, const void* w, const void* w_scales, int32_t group,
                     const void* delta, int64_t delta_row_stride, void* out,
                     int64_t out_row_stride, void* stream) {
  MOL_TRY(check_down(act, topk_ids, topk_weights, num_tokens, topk, num_experts, hidden, inter, w,
                     w_scales, group, delta, delta_row_stride, out, out_row_stride));
  if (num_tokens == 0) return MOL_OK;
  MOL_TRY(mol::ensure_moe_device());
  const mol::MoeShape s{(int)num_tokens, topk, num_experts, hidden, inter};
  return done(mol::launch_moe_down(s, act, topk_ids, topk_weights,
                                   mol::WeightRows{w, w_scales, inter, group}, delta,
                                   delta_row_stride, out, out_row_stride, false,
                                   static_cast<cudaStream_t>(stream)));
}

size_t mol_moe_workspace_bytes(int64_t num_tokens, int32_t topk, int32_t num_experts,
                               int32_t hidden, int32_t inter, int32_t group) {
  if (check_moe_shape(num_tokens, topk, num_experts, hidden, inter) != MOL_OK || num_tokens == 0)
    return 0;
  return mol::moe_split_bytes(mol::MoeShape{(int)num_tokens, topk, num_experts, hidden, inter},
                              group);
}

int32_t mol_moe_down_split(const void* act, const int32_t* topk_ids, const float* topk_weights,
                           int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t hidden,
                           int32_t inter, const void* w, const void* w_scales, int32_t group,
                           const void* delta, int64_t delta_row_stride, void* workspace,
                           size_t workspace_bytes, void* out, int64_t out_row_stride,
                           void* stream) {
  MOL_TRY(check_down(act, topk_ids, topk_weights, num_tokens, topk, num_experts, hidden, inter, w,
                     w_scales, group, delta, delta_row_stride, out, out_row_stride));
  if (num_tokens == 0) return MOL_OK;
  const mol::MoeShape s{(int)num_tokens, topk, num_experts, hidden, inter};
  bool split = false;
  MOL_TRY(check_workspace(s, group, workspace, workspace_bytes, split));
  MOL_TRY(mol::ensure_moe_device());
  const mol::WeightRows rows{w, w_scales, inter, group};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(split ? mol::launch_moe_down_split(s, act, topk_ids, topk_weights, rows, delta,
                                                 delta_row_stride, workspace, out, out_row_stride,
                                                 false, st)
                    : mol::launch_moe_down(s, act, topk_ids, topk_weights, rows, delta,
                                           delta_row_stride, out, out_row_stride, false, st));
}

int32_t mol_moe_forward(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                        const float* topk_weights, int64_t num_tokens, int32_t topk,
                        int32_t num_experts, int32_t hidden, int32_t inter, const void* w_gate_up,
                        const void* gate_up_scales, const void* w_down, const void* down_scales,
                        int32_t group, void* act, void* out, int64_t out_row_stride, void* stream) {
  return forward(x, x_row_stride, topk_ids, topk_weights, num_tokens, topk, num_experts, hidden,
                 inter, w_gate_up, gate_up_scales, w_down, down_scales, group, act, nullptr, 0,
                 false, out, out_row_stride, stream);
}

int32_t mol_moe_forward_split(const void* x, int64_t x_row_stride, const int32_t* topk_ids,
                              const float* topk_weights, int64_t num_tokens, int32_t topk,
                              int32_t num_experts, int32_t hidden, int32_t inter,
                              const void* w_gate_up, const void* gate_up_scales,
                              const void* w_down, const void* down_scales, int32_t group,
                              void* act, void* workspace, size_t workspace_bytes, void* out,
                              int64_t out_row_stride, void* stream) {
  return forward(x, x_row_stride, topk_ids, topk_weights, num_tokens, topk, num_experts, hidden,
                 inter, w_gate_up, gate_up_scales, w_down, down_scales, group, act, workspace,
                 workspace_bytes, true, out, out_row_stride, stream);
}

int32_t mol_w4_linear(const void* x, int64_t x_row_stride, int64_t num_tokens, int32_t K, int32_t N,
                      const void* w, const void* scales, int32_t group, void* out,
                      int64_t out_row_stride, void* stream) {
  if (num_tokens < 0 || K < 1 || N < 1 || out_row_stride < N) return MOL_ERR_INVALID_ARG;
  if (num_tokens > MOL_W4_MAX_TOKENS || K % 8 != 0 || K > MOL_MOE_MAX_WIDTH || N > 1 << 30)
    return MOL_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MOL_OK;
  if (!out) return MOL_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(out) % 2 != 0) return MOL_ERR_UNSUPPORTED;
  MOL_TRY(check_rows(x, x_row_stride, K));
  MOL_TRY(check_weights(w, scales, group, true));
  MOL_TRY(mol::ensure_moe_device());
  return done(mol::launch_w4_linear(x, x_row_stride, (int)num_tokens, N,
                                    mol::WeightRows{w, scales, K, group}, out, out_row_stride,
                                    static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
