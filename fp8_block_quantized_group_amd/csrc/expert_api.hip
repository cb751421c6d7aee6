// Host side of the experts' own products: argument validation and launches.
#include <algorithm>

#include "api_common.h"
#include "kernels.h"

using moe::check_ptr;
using moe::fail;
using moe::launch_status;
using moe::ok;

namespace {

constexpr float kSwigluDefaultLimit = 7.0f;

size_t elem(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }

moe_status_t check_opt(const void* ptr, const char* name, size_t align) {
  return ptr == nullptr ? MOE_OK : check_ptr(ptr, name, align);
}

bool gated(int act) {
  return act != MOE_ACT_NONE && (act < MOE_ACT_SILU_NO_MUL || act > MOE_ACT_RELU2_NO_MUL);
}
int wide_of(int out_features, int act) { return out_features * (gated(act) ? 2 : 1); }
float limit_of(int act, float limit) {
  const bool clamps = act == MOE_ACT_SWIGLUOAI || act == MOE_ACT_SWIGLUSTEP;
  return clamps && limit == 0.0f ? kSwigluDefaultLimit : limit;
}

// what every linear layer of rows sorted by expert has
moe_status_t check_sizes(int rows, int in, int out, int experts, int dtype, int act,
                         float limit) {
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "num_rows < 0 (%d)", rows);
  if (in < 1 || in > 32768)
    return fail(MOE_ERR_UNSUPPORTED, "in_features must be in [1, 32768], got %d", in);
  if (out < 1 || out > 32768)
    return fail(MOE_ERR_UNSUPPORTED, "out_features must be in [1, 32768], got %d", out);
  if (experts < 1 || experts > 1024)
    return fail(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 1024], got %d", experts);
  if (dtype < MOE_DT_BF16 || dtype > MOE_DT_F32)
    return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLUSTEP)
    return fail(MOE_ERR_INVALID_ARG, "unknown activation %d", act);
  if (!(limit >= 0.0f) || limit > 3.0e38f)
    return fail(MOE_ERR_INVALID_ARG, "act_limit must be finite and >= 0, got %g", (double)limit);
  if (limit > 0.0f && act != MOE_ACT_SILU && act != MOE_ACT_SWIGLUOAI &&
      act != MOE_ACT_SWIGLUSTEP)
    return fail(MOE_ERR_UNSUPPORTED, "activation %d takes no clamp limit", act);
  // launches count their tiles, of at least 16 x 16 results, in 31 bits
  const int64_t m = (int64_t)rows / 16 + std::min(rows, experts);
  const int64_t n = (std::max(in, wide_of(out, act)) + 15) / 16;
  if (m * n >= (int64_t)1 << 31)
    return fail(MOE_ERR_UNSUPPORTED, "%d rows of %d columns are more than 2^31 tiles", rows,
                std::max(in, out));
  return MOE_OK;
}

moe_status_t check_offsets(const int32_t* offsets, int experts) {
  if (offsets == nullptr && experts != 1)
    return fail(MOE_ERR_INVALID_ARG, "expert_offsets is NULL with %d experts", experts);
  return check_opt(offsets, "expert_offsets", 4);
}

moe_status_t check_linear(const moe_expert_linear_t* p) {
  if (p == nullptr) return fail(MOE_ERR_INVALID_ARG, "expert linear is NULL");
  CHECK(check_sizes(p->num_rows, p->in_features, p->out_features, p->num_experts, p->dtype,
                    p->activation, p->act_limit));
  // an expert's weights are addressed with 32-bit buffer offsets
  const int64_t wide = wide_of(p->out_features, p->activation);
  if (wide * p->in_features * (int64_t)elem(p->dtype) >= (int64_t)0xF0000000u)
    return fail(MOE_ERR_UNSUPPORTED, "one expert's weights must be under 3.75 GiB");
  // and the weights' gradient is tiled expert by expert
  if (((wide + 63) / 64 * ((p->in_features + 63) / 64) + 7) * p->num_experts >=
      (int64_t)1 << 31)
    return fail(MOE_ERR_UNSUPPORTED, "the experts' weights are more than 2^31 tiles");
  return MOE_OK;
}

moe::ExpertGemmArgs gemm_args(const moe_expert_linear_t* p, const int32_t* offsets) {
  moe::ExpertGemmArgs a{};
  a.offsets = offsets;
  a.R = p->num_rows;
  a.K = p->in_features;
  a.N = p->out_features;
  a.wide = wide_of(p->out_features, p->activation);
  a.E = p->num_experts;
  a.act = p->activation;
  a.limit = limit_of(p->activation, p->act_limit);
  a.split = 1;
  return a;
}

// The backward's workspace: d, then the parts' sums of a split gradient.
size_t linear_d_bytes(const moe_expert_linear_t* p) {
  if (p->activation == MOE_ACT_NONE) return 0;
  return moe::round_up((size_t)p->num_rows * wide_of(p->out_features, p->activation) *
                       elem(p->dtype));
}
size_t linear_ws_bytes(const moe_expert_linear_t* p) {
  const moe::ExpertGemmArgs a = gemm_args(p, nullptr);
  const size_t sx = moe::expert_split(a, p->dtype, false), sw = moe::expert_split(a, p->dtype, true);
  const size_t x = sx > 1 ? sx * a.R * a.K * 4 : 0;
  const size_t w = sw > 1 ? sw * a.E * a.wide * a.K * 4 : 0;
  return linear_d_bytes(p) + moe::round_up(std::max(x, w));
}
void split_gradient(moe::ExpertGemmArgs& a, int dtype, bool grad_w, void* parts) {
  a.split = moe::expert_split(a, dtype, grad_w);
  a.part = (float*)parts;
  a.part_size = (grad_w ? (int64_t)a.E * a.wide : a.R) * a.K;
}

moe_status_t check_w4(const moe_expert_linear_w4_t* p) {
  if (p == nullptr) return fail(MOE_ERR_INVALID_ARG, "expert linear is NULL");
  CHECK(check_sizes(p->num_rows, p->in_features, p->out_features, p->num_experts, p->dtype,
                    p->activation, p->act_limit));
  if (p->format < MOE_W4_INT4 || p->format > MOE_W4_MXFP4)
    return fail(MOE_ERR_INVALID_ARG, "unknown 4-bit format %d", p->format);
  if (p->group_size != 32 && p->group_size != 64 && p->group_size != 128)
    return fail(MOE_ERR_UNSUPPORTED, "group_size must be 32, 64 or 128, got %d", p->group_size);
  if (p->format == MOE_W4_MXFP4 && p->group_size != 32)
    return fail(MOE_ERR_UNSUPPORTED, "MXFP4 groups are 32 columns, got %d", p->group_size);
  if (p->in_features % p->group_size != 0)
    return fail(MOE_ERR_UNSUPPORTED, "group_size %d does not divide in_features %d",
                p->group_size, p->in_features);
  if (p->format != MOE_W4_MXFP4 && p->scale_dtype != p->dtype && p->scale_dtype != MOE_DT_F32)
    return fail(MOE_ERR_UNSUPPORTED, "scale_dtype must be dtype or fp32, got %d",
                p->scale_dtype);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_expert_linear(const moe_expert_linear_t* p, const void* x,
                               const int32_t* expert_offsets, const void* weight, void* out,
                               void* pre_act, void* stream) {
  CHECK(check_linear(p));
  if (p->num_rows == 0) return ok();
  const size_t es = elem(p->dtype);
  CHECK(check_ptr(x, "x", es));
  CHECK(check_offsets(expert_offsets, p->num_experts));
  CHECK(check_ptr(weight, "weight", es));
  CHECK(check_ptr(out, "out", es));
  CHECK(check_opt(pre_act, "pre_act", es));
  moe::ExpertGemmArgs a = gemm_args(p, expert_offsets);
  a.a = (const uint8_t*)x;
  a.b = (const uint8_t*)weight;
  a.out = (uint8_t*)out;
  a.pre = (uint8_t*)pre_act;
  return launch_status(moe::launch_expert_out(a, p->dtype, (hipStream_t)stream),
                       "moe_expert_linear");
}

moe_status_t moe_expert_linear_workspace_size(const moe_expert_linear_t* p, size_t* bytes) {
  CHECK(check_linear(p));
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = linear_ws_bytes(p);
  return ok();
}

moe_status_t moe_expert_linear_backward(const moe_expert_linear_t* p, const void* x,
                                        const int32_t* expert_offsets, const void* weight,
                                        const void* pre_act, const void* grad_out, void* grad_x,
                                        void* grad_weight, void* ws, size_t ws_bytes,
                                        void* stream) {
  CHECK(check_linear(p));
  const size_t es = elem(p->dtype);
  const bool act = p->activation != MOE_ACT_NONE;
  CHECK(check_opt(grad_weight, "grad_weight", es));
  if (p->num_rows > 0) {
    CHECK(check_offsets(expert_offsets, p->num_experts));
    CHECK(check_ptr(grad_out, "grad_out", es));
    CHECK(check_opt(grad_x, "grad_x", es));
    if (grad_weight != nullptr) CHECK(check_ptr(x, "x", es));
    if (grad_x != nullptr) CHECK(check_ptr(weight, "weight", es));
    if (act) {
      CHECK(check_ptr(pre_act, "pre_act", es));
    } else if (pre_act != nullptr) {
      return fail(MOE_ERR_INVALID_ARG, "pre_act given without an activation");
    }
    if (const size_t need = linear_ws_bytes(p)) {
      CHECK(check_ptr(ws, "ws", 16));
      if (ws_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "expert linear workspace too small: %zu < %zu bytes",
                    ws_bytes, need);
    }
  }
  const hipStream_t s = (hipStream_t)stream;
  moe::ExpertGemmArgs a = gemm_args(p, expert_offsets);
  a.a = (const uint8_t*)grad_out;
  a.act = MOE_ACT_NONE;
  if (act && p->num_rows > 0 && (grad_x != nullptr || grad_weight != nullptr)) {
    moe::ExpertActGradArgs g{};
    g.pre = (const uint8_t*)pre_act;
    g.grad_out = (const uint8_t*)grad_out;
    g.d = (uint8_t*)ws;
    g.offsets = expert_offsets;
    g.R = p->num_rows;
    g.N = p->out_features;
    g.E = p->num_experts;
    g.act = p->activation;
    g.limit = a.limit;
    CHECK(launch_status(moe::launch_expert_act_grad(g, p->dtype, s),
                        "moe_expert_linear_backward"));
    a.a = (const uint8_t*)ws;
  }
  void* parts = ws == nullptr ? nullptr : (uint8_t*)ws + linear_d_bytes(p);
  if (grad_x != nullptr && p->num_rows > 0) {
    split_gradient(a, p->dtype, false, parts);
    a.b = (const uint8_t*)weight;
    a.out = (uint8_t*)grad_x;
    CHECK(launch_status(moe::launch_expert_grad_x(a, p->dtype, s),
                        "moe_expert_linear_backward"));
  }
  if (grad_weight != nullptr) {
    split_gradient(a, p->dtype, true, parts);
    if (p->num_rows == 0) a.offsets = nullptr;      // R = 0: every expert's range is empty
    a.b = (const uint8_t*)x;
    a.out = (uint8_t*)grad_weight;
    CHECK(launch_status(moe::launch_expert_grad_w(a, p->dtype, s),
                        "moe_expert_linear_backward"));
  }
  return ok();
}

moe_status_t moe_expert_linear_w4(const moe_expert_linear_w4_t* p, const void* x,
                                  const int32_t* expert_offsets, const void* codes,
                                  const void* scales, const void* zeros, void* out,
                                  void* stream) {
  CHECK(check_w4(p));
  if (p->num_rows == 0) return ok();
  const bool mx = p->format == MOE_W4_MXFP4;
  CHECK(check_ptr(x, "x", elem(p->dtype)));
  CHECK(check_offsets(expert_offsets, p->num_experts));
  CHECK(check_ptr(codes, "codes", 1));
  CHECK(check_ptr(scales, "scales", mx ? 1 : elem(p->scale_dtype)));
  if (p->format == MOE_W4_INT4_ZERO) {
    CHECK(check_ptr(zeros, "zeros", 1));
  } else if (zeros != nullptr) {
    return fail(MOE_ERR_INVALID_ARG, "zeros given for a format without them");
  }
  CHECK(check_ptr(out, "out", elem(p->dtype)));
  moe::ExpertW4Args a{};
  a.x = (const uint8_t*)x;
  a.codes = (const uint8_t*)codes;
  a.scales = (const uint8_t*)scales;
  a.zeros = (const uint8_t*)zeros;
  a.out = (uint8_t*)out;
  a.offsets = expert_offsets;
  a.R = p->num_rows;
  a.K = p->in_features;
  a.N = p->out_features;
  a.wide = wide_of(p->out_features, p->activation);
  a.E = p->num_experts;
  a.act = p->activation;
  a.format = p->format;
  a.group = p->group_size;
  a.limit = limit_of(p->activation, p->act_limit);
  const hipStream_t s = (hipStream_t)stream;
  const bool s32 = p->scale_dtype == MOE_DT_F32;
  const hipError_t err = p->dtype == MOE_DT_BF16  ? moe::launch_expert_w4_dt<0>(a, s32, s)
                         : p->dtype == MOE_DT_F16 ? moe::launch_expert_w4_dt<1>(a, s32, s)
                                                  : moe::launch_expert_w4_dt<2>(a, s32, s);
  return launch_status(err, "moe_expert_linear_w4");
}

}  // extern "C"
