// Host side of the calls around the expert layer: argument validation and
// launches of the router, the sorted rows and the block norms.
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "kernels.h"

using moe::check_ptr;
using moe::fail;
using moe::launch_status;
using moe::ok;

namespace {

bool valid_dtype(int dt) { return dt >= MOE_DT_BF16 && dt <= MOE_DT_F32; }
size_t elem(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }

moe_status_t check_router(const moe_router_t* p) {
  if (p == nullptr) return fail(MOE_ERR_INVALID_ARG, "router is NULL");
  if (p->num_tokens < 0) return fail(MOE_ERR_INVALID_ARG, "num_tokens < 0 (%d)", p->num_tokens);
  if (p->num_experts < 1 || p->num_experts > 1024)
    return fail(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 1024], got %d", p->num_experts);
  if (p->top_k < 1 || p->top_k > p->num_experts)
    return fail(MOE_ERR_INVALID_ARG, "top_k must be in [1, num_experts], got %d", p->top_k);
  if (p->top_k > 64) return fail(MOE_ERR_UNSUPPORTED, "top_k is limited to 64, got %d", p->top_k);
  if (!valid_dtype(p->dtype)) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  if (p->score != MOE_SCORE_SOFTMAX && p->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, "unknown score %d", p->score);
  if (p->num_groups < 1 || p->num_groups > 64 || p->num_experts % p->num_groups != 0)
    return fail(MOE_ERR_INVALID_ARG, "num_groups must be in [1, 64] and divide num_experts, got %d",
                p->num_groups);
  if (p->topk_groups < 1 || p->topk_groups > p->num_groups)
    return fail(MOE_ERR_INVALID_ARG, "topk_groups must be in [1, num_groups], got %d",
                p->topk_groups);
  if (p->topk_groups * (p->num_experts / p->num_groups) < p->top_k)
    return fail(MOE_ERR_INVALID_ARG, "%d groups of %d experts hold fewer than top_k %d",
                p->topk_groups, p->num_experts / p->num_groups, p->top_k);
  if (p->group_top != 1 && p->group_top != 2)
    return fail(MOE_ERR_INVALID_ARG, "group_top must be 1 or 2, got %d", p->group_top);
  if (!isfinite(p->scale)) return fail(MOE_ERR_INVALID_ARG, "scale must be finite");
  return MOE_OK;
}

moe::RouterArgs router_args(const moe_router_t* p) {
  moe::RouterArgs a{};
  a.T = p->num_tokens;
  a.E = p->num_experts;
  a.k = p->top_k;
  a.groups = p->num_groups;
  a.topk_groups = p->topk_groups;
  a.group_top = p->group_top;
  a.sigmoid = p->score == MOE_SCORE_SIGMOID;
  a.renormalize = p->renormalize != 0;
  a.scale = p->scale;
  return a;
}

moe_status_t check_rows(const moe_rows_t* p) {
  if (p == nullptr) return fail(MOE_ERR_INVALID_ARG, "rows problem is NULL");
  if (p->num_tokens < 0) return fail(MOE_ERR_INVALID_ARG, "num_tokens < 0 (%d)", p->num_tokens);
  if (p->hidden < 1 || p->hidden > 32768)
    return fail(MOE_ERR_UNSUPPORTED, "hidden must be in [1, 32768], got %d", p->hidden);
  if (p->num_experts < 1 || p->num_experts > 1024)
    return fail(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 1024], got %d", p->num_experts);
  if (p->top_k < 1) return fail(MOE_ERR_INVALID_ARG, "top_k must be >= 1, got %d", p->top_k);
  if ((int64_t)p->num_tokens * p->top_k >= (int64_t)1 << 31)
    return fail(MOE_ERR_UNSUPPORTED, "num_tokens * top_k must be < 2^31");
  if (!valid_dtype(p->dtype)) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  // the streaming kernels count their blocks, at most 32 pieces of a row, in 32 bits
  if ((int64_t)p->num_tokens * ((p->hidden + 1023) / 1024) >= (int64_t)1 << 31)
    return fail(MOE_ERR_UNSUPPORTED, "num_tokens * hidden / 1024 must be < 2^31");
  return MOE_OK;
}

int64_t slots(const moe_rows_t* p) { return (int64_t)p->num_tokens * p->top_k; }

size_t permute_ws_bytes(const moe_rows_t* p) {
  const int64_t chunks = (slots(p) + moe::kSortChunk - 1) / moe::kSortChunk;
  return moe::round_up((size_t)std::max<int64_t>(chunks, 1) * p->num_experts * sizeof(int32_t));
}

moe::RowsArgs rows_args(const moe_rows_t* p, const void* in, void* out, const int32_t* slot_row,
                        const float* weights) {
  moe::RowsArgs a{};
  a.in = (const uint8_t*)in;
  a.out = (uint8_t*)out;
  a.slot_row = slot_row;
  a.weights = weights;
  a.T = p->num_tokens;
  a.slots = slots(p);
  a.k = p->top_k;
  a.H = p->hidden;
  return a;
}

moe_status_t check_opt(const void* ptr, const char* name, size_t align) {
  return ptr == nullptr ? MOE_OK : check_ptr(ptr, name, align);
}

moe_status_t check_norm(const moe_block_norm_t* p) {
  if (p == nullptr) return fail(MOE_ERR_INVALID_ARG, "block norm is NULL");
  if (p->num_tokens < 0) return fail(MOE_ERR_INVALID_ARG, "num_tokens < 0 (%d)", p->num_tokens);
  if (p->hidden < 1 || p->hidden > 32768)
    return fail(MOE_ERR_UNSUPPORTED, "hidden must be in [1, 32768], got %d", p->hidden);
  if (!valid_dtype(p->dtype)) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  if (p->weight_dtype != p->dtype && p->weight_dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "weight_dtype must be dtype or fp32, got %d",
                p->weight_dtype);
  if (p->gate < MOE_GATE_NONE || p->gate > MOE_GATE_FULL)
    return fail(MOE_ERR_INVALID_ARG, "unknown gate kind %d", p->gate);
  // below, squares that fp32 flushes would count beside eps
  if (!(p->eps >= 1e-20f && p->eps <= 1e20f))
    return fail(MOE_ERR_INVALID_ARG, "eps must be in [1e-20, 1e20], got %g", (double)p->eps);
  if (!isfinite(p->residual_scale) || !isfinite(p->weight_offset))
    return fail(MOE_ERR_INVALID_ARG, "residual_scale and weight_offset must be finite");
  return MOE_OK;
}

// the block's part of a norm's arguments: y, its weight and its gate
moe_status_t check_block(const moe_block_norm_t* p, const void* y, const void* post_weight,
                         const void* gate, const void* pre_weight) {
  const size_t es = elem(p->dtype), ws = elem(p->weight_dtype);
  CHECK(check_opt(y, "y", es));
  CHECK(check_opt(pre_weight, "pre_weight", ws));
  if (post_weight != nullptr && (y == nullptr || !p->post_norm))
    return fail(MOE_ERR_INVALID_ARG, "post_weight given without a post norm of y");
  CHECK(check_opt(post_weight, "post_weight", ws));
  if (y == nullptr || p->gate == MOE_GATE_NONE) {
    if (gate != nullptr) return fail(MOE_ERR_INVALID_ARG, "gate given for a norm without one");
  } else {
    CHECK(check_ptr(gate, "gate", es));
  }
  return MOE_OK;
}

// the streams of a norm: y comes with the residual_out that it makes
moe_status_t check_norm_streams(const moe_block_norm_t* p, const void* residual, const void* y,
                                const void* post_weight, const void* gate,
                                const void* pre_weight, const void* residual_out) {
  CHECK(check_ptr(residual, "residual", elem(p->dtype)));
  CHECK(check_block(p, y, post_weight, gate, pre_weight));
  if (y != nullptr) return check_ptr(residual_out, "residual_out", elem(p->dtype));
  if (residual_out != nullptr)
    return fail(MOE_ERR_INVALID_ARG, "residual_out given without y");
  return MOE_OK;
}

moe::NormArgs norm_args(const moe_block_norm_t* p, const void* residual, const void* y,
                        const void* post_weight, const void* gate, const void* pre_weight,
                        void* residual_out, void* normed) {
  moe::NormArgs a{};
  a.r = (const uint8_t*)residual;
  a.y = (const uint8_t*)y;
  a.r_out = (uint8_t*)residual_out;
  a.h = (uint8_t*)normed;
  a.w_post = post_weight;
  a.w_pre = pre_weight;
  a.gate = (const uint8_t*)gate;
  a.T = p->num_tokens;
  a.H = p->hidden;
  a.gate_kind = gate != nullptr ? p->gate : moe::kGateNone;
  a.post = p->post_norm != 0;
  a.gate_sigmoid = p->gate_sigmoid != 0;
  a.eps = p->eps;
  a.alpha = p->residual_scale;
  a.offset = p->weight_offset;
  return a;
}

size_t norm_ws_bytes(const moe_block_norm_t* p) {
  const size_t parts = moe::norm_grad_parts(p->num_tokens, p->hidden, p->dtype);
  return moe::round_up(std::max<size_t>(parts, 1) * 3 * p->hidden * sizeof(float));
}

}  // namespace

extern "C" {

moe_status_t moe_router_topk(const moe_router_t* p, const void* logits, const float* bias,
                             const uint8_t* is_padding, int32_t* topk_ids, float* topk_weights,
                             void* stream) {
  CHECK(check_router(p));
  if (p->num_tokens == 0) return ok();
  CHECK(check_ptr(logits, "logits", elem(p->dtype)));
  CHECK(check_opt(bias, "bias", 4));
  CHECK(check_ptr(topk_ids, "topk_ids", 4));
  CHECK(check_ptr(topk_weights, "topk_weights", 4));
  moe::RouterArgs a = router_args(p);
  a.logits = logits;
  a.bias = bias;
  a.is_padding = is_padding;
  a.ids = topk_ids;
  a.weights = topk_weights;
  return launch_status(moe::launch_router_topk(a, p->dtype, (hipStream_t)stream),
                       "moe_router_topk");
}

moe_status_t moe_router_topk_backward(const moe_router_t* p, const void* logits,
                                      const int32_t* topk_ids, const float* grad_topk_weights,
                                      void* grad_logits, void* stream) {
  CHECK(check_router(p));
  if (p->num_tokens == 0) return ok();
  CHECK(check_ptr(logits, "logits", elem(p->dtype)));
  CHECK(check_ptr(topk_ids, "topk_ids", 4));
  CHECK(check_ptr(grad_topk_weights, "grad_topk_weights", 4));
  CHECK(check_ptr(grad_logits, "grad_logits", elem(p->dtype)));
  moe::RouterArgs a = router_args(p);
  a.logits = logits;
  return launch_status(moe::launch_router_grad(a, topk_ids, grad_topk_weights, grad_logits,
                                               p->dtype, (hipStream_t)stream),
                       "moe_router_topk_backward");
}

moe_status_t moe_permute_workspace_size(const moe_rows_t* p, size_t* bytes) {
  CHECK(check_rows(p));
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = permute_ws_bytes(p);
  return ok();
}

moe_status_t moe_permute(const moe_rows_t* p, const void* x, const int32_t* topk_ids,
                         const uint8_t* is_padding, void* rows, int32_t* expert_offsets,
                         int32_t* slot_row, int32_t* row_slot, void* ws, size_t ws_bytes,
                         void* stream) {
  CHECK(check_rows(p));
  CHECK(check_ptr(expert_offsets, "expert_offsets", 4));
  if (p->num_tokens > 0) {
    CHECK(check_ptr(x, "x", elem(p->dtype)));
    CHECK(check_ptr(topk_ids, "topk_ids", 4));
    CHECK(check_ptr(rows, "rows", elem(p->dtype)));
    CHECK(check_ptr(slot_row, "slot_row", 4));
    CHECK(check_ptr(row_slot, "row_slot", 4));
    CHECK(check_ptr(ws, "ws", 4));
    if (ws_bytes < permute_ws_bytes(p))
      return fail(MOE_ERR_WORKSPACE, "permute workspace too small: %zu < %zu bytes", ws_bytes,
                  permute_ws_bytes(p));
  }
  moe::SortArgs s{};
  s.ids = topk_ids;
  s.is_padding = is_padding;
  s.slots = slots(p);
  s.k = p->top_k;
  s.E = p->num_experts;
  s.hist = (int32_t*)ws;
  s.expert_offsets = expert_offsets;
  s.slot_row = slot_row;
  s.row_slot = row_slot;
  const hipError_t err = moe::launch_permute(s, rows_args(p, x, rows, slot_row, nullptr),
                                             p->dtype, (hipStream_t)stream);
  return launch_status(err, "moe_permute");
}

moe_status_t moe_permute_backward(const moe_rows_t* p, const void* grad_rows,
                                  const int32_t* slot_row, void* grad_x, void* stream) {
  CHECK(check_rows(p));
  if (p->num_tokens == 0) return ok();
  CHECK(check_ptr(grad_rows, "grad_rows", elem(p->dtype)));
  CHECK(check_ptr(slot_row, "slot_row", 4));
  CHECK(check_ptr(grad_x, "grad_x", elem(p->dtype)));
  return launch_status(
      moe::launch_combine_rows(rows_args(p, grad_rows, grad_x, slot_row, nullptr), p->dtype,
                               (hipStream_t)stream),
      "moe_permute_backward");
}

moe_status_t moe_unpermute(const moe_rows_t* p, const void* rows, const int32_t* slot_row,
                           const float* topk_weights, void* out, void* stream) {
  CHECK(check_rows(p));
  if (p->num_tokens == 0) return ok();
  CHECK(check_ptr(rows, "rows", elem(p->dtype)));
  CHECK(check_ptr(slot_row, "slot_row", 4));
  CHECK(check_opt(topk_weights, "topk_weights", 4));
  CHECK(check_ptr(out, "out", elem(p->dtype)));
  return launch_status(moe::launch_combine_rows(rows_args(p, rows, out, slot_row, topk_weights),
                                                p->dtype, (hipStream_t)stream),
                       "moe_unpermute");
}

moe_status_t moe_unpermute_backward(const moe_rows_t* p, const void* grad_out, const void* rows,
                                    const int32_t* slot_row, const float* topk_weights,
                                    void* grad_rows, float* grad_topk_weights, void* stream) {
  CHECK(check_rows(p));
  if (p->num_tokens == 0) return ok();
  CHECK(check_ptr(grad_out, "grad_out", elem(p->dtype)));
  CHECK(check_ptr(rows, "rows", elem(p->dtype)));
  CHECK(check_ptr(slot_row, "slot_row", 4));
  CHECK(check_opt(topk_weights, "topk_weights", 4));
  CHECK(check_ptr(grad_rows, "grad_rows", elem(p->dtype)));
  CHECK(check_ptr(grad_topk_weights, "grad_topk_weights", 4));
  return launch_status(
      moe::launch_combine_grad(rows_args(p, grad_out, grad_rows, slot_row, topk_weights), rows,
                               grad_topk_weights, p->dtype, (hipStream_t)stream),
      "moe_unpermute_backward");
}

moe_status_t moe_block_norm(const moe_block_norm_t* p, const void* residual, const void* y,
                            const void* post_weight, const void* gate, const void* pre_weight,
                            void* residual_out, void* normed, void* stream) {
  CHECK(check_norm(p));
  if (p->num_tokens == 0) return ok();
  CHECK(check_norm_streams(p, residual, y, post_weight, gate, pre_weight, residual_out));
  if (y != nullptr) CHECK(check_opt(normed, "normed", elem(p->dtype)));
  else CHECK(check_ptr(normed, "normed", elem(p->dtype)));
  const moe::NormArgs a =
      norm_args(p, residual, y, post_weight, gate, pre_weight, residual_out, normed);
  return launch_status(
      moe::launch_norm(a, p->dtype, p->weight_dtype == MOE_DT_F32, (hipStream_t)stream),
      "moe_block_norm");
}

moe_status_t moe_block_norm_quant(const moe_block_norm_t* p, int32_t act_quant,
                                  const void* residual, const void* y, const void* post_weight,
                                  const void* gate, const void* pre_weight, void* residual_out,
                                  void* normed, void* x_q, void* x_sf, void* stream) {
  CHECK(check_norm(p));
  if (act_quant != MOE_Q_FP8_UE8M0 && act_quant != MOE_Q_FP8_F32 && act_quant != MOE_Q_MXFP8)
    return fail(MOE_ERR_INVALID_ARG, "unknown 8-bit quantization %d", act_quant);
  if (p->hidden % 128 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "hidden must be a multiple of 128, got %d", p->hidden);
  if (p->num_tokens == 0) return ok();
  CHECK(check_norm_streams(p, residual, y, post_weight, gate, pre_weight, residual_out));
  CHECK(check_opt(normed, "normed", elem(p->dtype)));
  CHECK(check_ptr(x_q, "x_q", 16));
  CHECK(check_ptr(x_sf, "x_sf", 4));
  moe::NormArgs a =
      norm_args(p, residual, y, post_weight, gate, pre_weight, residual_out, normed);
  a.quant = act_quant;
  a.q = (uint8_t*)x_q;
  a.q_sf = (uint8_t*)x_sf;
  return launch_status(
      moe::launch_norm_quant(a, p->dtype, p->weight_dtype == MOE_DT_F32, (hipStream_t)stream),
      "moe_block_norm_quant");
}

moe_status_t moe_block_norm_workspace_size(const moe_block_norm_t* p, size_t* bytes) {
  CHECK(check_norm(p));
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = norm_ws_bytes(p);
  return ok();
}

moe_status_t moe_block_norm_backward(const moe_block_norm_t* p, const void* residual_out,
                                     const void* y, const void* post_weight, const void* gate,
                                     const void* pre_weight, const void* grad_normed,
                                     const void* grad_residual_out, void* grad_residual,
                                     void* grad_y, float* grad_pre_weight,
                                     float* grad_post_weight, void* grad_gate, void* ws,
                                     size_t ws_bytes, void* stream) {
  CHECK(check_norm(p));
  const size_t es = elem(p->dtype);
  const bool gated = p->gate != MOE_GATE_NONE && (y != nullptr || p->num_tokens == 0);
  if (p->num_tokens > 0) {
    CHECK(check_ptr(residual_out, "residual_out", es));
    CHECK(check_block(p, y, post_weight, gate, pre_weight));
    CHECK(check_opt(grad_normed, "grad_normed", es));
    CHECK(check_opt(grad_residual_out, "grad_residual_out", es));
    CHECK(check_ptr(grad_residual, "grad_residual", es));
    if (y != nullptr) CHECK(check_ptr(grad_y, "grad_y", es));
    else if (grad_y != nullptr) return fail(MOE_ERR_INVALID_ARG, "grad_y given without y");
    if (grad_post_weight != nullptr && (y == nullptr || !p->post_norm))
      return fail(MOE_ERR_INVALID_ARG, "grad_post_weight given without a post norm of y");
  }
  CHECK(check_opt(grad_pre_weight, "grad_pre_weight", 4));
  CHECK(check_opt(grad_post_weight, "grad_post_weight", 4));
  if (grad_gate != nullptr && !gated)
    return fail(MOE_ERR_INVALID_ARG, "grad_gate given for a norm without a gate");
  CHECK(check_opt(grad_gate, "grad_gate", p->gate == MOE_GATE_FULL ? es : 4));
  float* channel = p->gate == MOE_GATE_CHANNEL ? (float*)grad_gate : nullptr;
  const bool sums = grad_pre_weight != nullptr || grad_post_weight != nullptr ||
                    channel != nullptr;
  if (sums) {
    CHECK(check_ptr(ws, "ws", 4));
    if (ws_bytes < norm_ws_bytes(p))
      return fail(MOE_ERR_WORKSPACE, "block norm workspace too small: %zu < %zu bytes", ws_bytes,
                  norm_ws_bytes(p));
  }
  moe::NormGradArgs a{};
  a.x = (const uint8_t*)residual_out;
  a.y = (const uint8_t*)y;
  a.dh = (const uint8_t*)grad_normed;
  a.dr_in = (const uint8_t*)grad_residual_out;
  a.dr = (uint8_t*)grad_residual;
  a.dy = (uint8_t*)grad_y;
  a.w_post = post_weight;
  a.w_pre = pre_weight;
  a.gate = (const uint8_t*)gate;
  a.d_gate = p->gate == MOE_GATE_CHANNEL ? nullptr : grad_gate;
  a.part = (float*)ws;
  a.want = (grad_pre_weight != nullptr ? 1 : 0) | (grad_post_weight != nullptr ? 2 : 0) |
           (channel != nullptr ? 4 : 0);
  a.T = p->num_tokens;
  a.H = p->hidden;
  a.gate_kind = gate != nullptr ? p->gate : moe::kGateNone;
  a.post = p->post_norm != 0;
  a.gate_sigmoid = p->gate_sigmoid != 0;
  a.eps = p->eps;
  a.alpha = p->residual_scale;
  a.offset = p->weight_offset;
  return launch_status(
      moe::launch_norm_grad(a, p->dtype, p->weight_dtype == MOE_DT_F32, grad_pre_weight,
                            grad_post_weight, channel, (hipStream_t)stream),
      "moe_block_norm_backward");
}

}  // extern "C"
