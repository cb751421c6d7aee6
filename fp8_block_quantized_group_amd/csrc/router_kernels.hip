// Router: the top-k experts of every token and their weights from the
// router's logits, and the gradient of the logits.
//
// Scores s = softmax(x) over the token's unmasked experts or sigmoid(x); a
// logit of -inf or NaN masks its expert, +inf counts as the largest finite
// fp32.  Experts are chosen by a key: the logit itself, or, with a selection
// bias or a group value of two experts, s + bias in 64 bits (two experts'
// keys can lie closer together than 32-bit scores tell apart, and the choice
// must not depend on which exp an implementation uses).  Groups of
// consecutive experts may limit the choice first.  Ties go to the lowest
// index.
#include <float.h>
#include <limits.h>

#include "kernels.h"
#include "row_vec.h"

namespace moe {

namespace {

constexpr int kRouterWaves = 4;   // tokens per block, one wave each

// The logit as the definition counts it: NaN masks, +inf is clamped.
__device__ __forceinline__ float clean_logit(float x) {
  return x == x ? fminf(x, FLT_MAX) : -INFINITY;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// 1 / (1 + e^-x) without overflow on either side
__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + expf(-x)); }

// The best (key, index) of the wave: the largest key, the lowest index among
// equal ones.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double k2 = __shfl_xor(key, d);
    const int i2 = __shfl_xor(idx, d);
    if (k2 > key || (k2 == key && i2 < idx)) {
      key = k2;
      idx = i2;
    }
  }
}

// lane l holds experts l, l + 64, ... (VPL of them)
template <int DT, int VPL>
__global__ __launch_bounds__(64 * kRouterWaves) void router_topk_kernel(const RouterArgs a) {
  extern __shared__ double lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave;
  if (t >= a.T) return;
  double* wkeys = lds + (int64_t)wave * a.E;
  const int E = a.E, k = a.k;
  const bool pad = a.is_padding != nullptr && a.is_padding[t] != 0;
  float x[VPL];
  double key[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < E && !pad
               ? clean_logit(RowVec<DT>::load_one((const uint8_t*)a.logits, t * E + e))
               : -INFINITY;
    m = fmaxf(m, x[i]);
  }
  m = wave_max(m);
  const bool scored = a.bias != nullptr || a.group_top > 1;
  double total = 0.0;
  if (scored && !a.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (x[i] > -INFINITY) total += exp((double)x[i] - (double)m);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    key[i] = x[i];
    if (scored && x[i] > -INFINITY) {
      key[i] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i]))
                         : exp((double)x[i] - (double)m) / total;
      if (a.bias != nullptr) key[i] += (double)a.bias[e];
    }
  }
  if (a.groups > 1) {
    const int size = E / a.groups;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < E) wkeys[lane + 64 * i] = key[i];
    __builtin_amdgcn_wave_barrier();
    // lane g: the value of group g
    double value = -INFINITY;
    if (lane < a.groups) {
      double best = -INFINITY, second = -INFINITY;
      for (int j = 0; j < size; ++j) {
        const double v = wkeys[lane * size + j];
        if (v > best) {
          second = best;
          best = v;
        } else if (v > second) {
          second = v;
        }
      }
      value = best + (a.group_top > 1 && second > -INFINITY ? second : 0.0);
    }
    uint64_t kept = 0;
    for (int r = 0; r < a.topk_groups; ++r) {
      double b = value;
      int g = lane;
      wave_best(b, g);
      if (b == -INFINITY) break;
      kept |= 1ull << g;
      if (lane == g) value = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / size)) & 1)) key[i] = -INFINITY;
    }
  }
  // the top k, one after the other; lane j keeps the j-th
  int my_id = -1;
  float my_x = -INFINITY;
  for (int j = 0; j < k; ++j) {
    double b = -INFINITY;
    int at = INT_MAX;
    float bx = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > b) {
        b = key[i];
        at = lane + 64 * i;
        bx = x[i];
      }
    const int mine = at;
    wave_best(b, at);
    if (b == -INFINITY) break;
    bx = __shfl(bx, at & 63);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (mine == at && lane + 64 * i == at) key[i] = -INFINITY;
    if (lane == j) {
      my_id = at;
      my_x = bx;
    }
  }
  // the weights of the chosen, in 32 bits
  float w = 0.0f;
  if (a.sigmoid) {
    w = my_id >= 0 ? sigmoid_f32(my_x) : 0.0f;
    if (a.renormalize) w /= wave_sum(w) + 1e-20f;
  } else if (a.renormalize) {
    const float ms = wave_max(my_x);
    w = my_id >= 0 ? expf(my_x - ms) : 0.0f;
    const float sum = wave_sum(w);
    w = my_id >= 0 ? w / sum : 0.0f;
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += x[i] > -INFINITY ? expf(x[i] - m) : 0.0f;
    sum = wave_sum(sum);
    w = my_id >= 0 ? expf(my_x - m) / sum : 0.0f;
  }
  if (lane < k) {
    a.ids[t * k + lane] = my_id;
    a.weights[t * k + lane] = w * a.scale;
  }
}

// One wave per token.  With p the score of the chosen experts and g their
// weights' gradients: softmax over all experts dx_i = s_i c (g_i - sum g p);
// renormalized softmax the same over the chosen alone; sigmoid dx_j = c g_j
// p_j (1 - p_j), renormalized with g_j replaced by (g_j - sum g p / D) / D.
// A repeated id adds its terms in slot order.
template <int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void router_grad_kernel(const RouterArgs a,
                                                                        const int32_t* ids,
                                                                        const float* grad_w,
                                                                        uint8_t* grad_logits) {
  extern __shared__ float ldsf[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave;
  if (t >= a.T) return;
  float* out = ldsf + (int64_t)wave * a.E;
  const int E = a.E, k = a.k;
  const uint8_t* logits = (const uint8_t*)a.logits;
  int id = lane < k ? ids[t * k + lane] : -1;
  if (id < 0 || id >= E) id = -1;
  float x = id >= 0 ? clean_logit(RowVec<DT>::load_one(logits, t * E + id)) : -INFINITY;
  if (x == -INFINITY) id = -1;
  const float g = id >= 0 ? grad_w[t * k + lane] : 0.0f;
  const bool any = __ballot(id >= 0) != 0;
  const bool dense = !a.sigmoid && !a.renormalize && any;
  float d = 0.0f;                         // the chosen experts' gradients
  float m = 0.0f, total = 1.0f, dot = 0.0f;
  if (a.sigmoid) {
    const float s = id >= 0 ? sigmoid_f32(x) : 0.0f;
    // 1 - s as sigmoid(-x): no cancellation for large x
    const float ds = id >= 0 ? s * sigmoid_f32(-x) : 0.0f;
    if (a.renormalize) {
      const float D = wave_sum(s) + 1e-20f;
      d = (g - wave_sum(g * (s / D))) / D * ds;
    } else {
      d = g * ds;
    }
  } else if (a.renormalize) {
    const float mx = wave_max(x);          // every lane takes part
    const float p0 = id >= 0 ? expf(x - mx) : 0.0f;
    const float sum = wave_sum(p0);
    const float p = id >= 0 ? p0 / sum : 0.0f;
    d = p * (g - wave_sum(g * p));
  } else if (any) {
    m = -INFINITY;
    for (int e = lane; e < E; e += 64)
      m = fmaxf(m, clean_logit(RowVec<DT>::load_one(logits, t * E + e)));
    m = wave_max(m);
    total = 0.0f;
    for (int e = lane; e < E; e += 64)
      total += expf(clean_logit(RowVec<DT>::load_one(logits, t * E + e)) - m);
    total = wave_sum(total);
    const float p = id >= 0 ? expf(x - m) / total : 0.0f;
    dot = wave_sum(g * p);
    d = p * g;
  }
  d = id >= 0 ? d * a.scale : 0.0f;
  for (int e = lane; e < E; e += 64) {
    float v = 0.0f;
    if (dense)
      v = -dot * a.scale *
          (expf(clean_logit(RowVec<DT>::load_one(logits, t * E + e)) - m) / total);
    out[e] = v;
  }
  __builtin_amdgcn_wave_barrier();
  for (int j = 0; j < k; ++j) {
    if (lane == j && id >= 0) out[id] += d;
    __builtin_amdgcn_wave_barrier();
  }
  for (int e = lane; e < E; e += 64) RowVec<DT>::store_one(grad_logits, t * E + e, out[e]);
}

template <int DT>
hipError_t topk_dt(const RouterArgs& a, hipStream_t stream) {
  const unsigned grid = (unsigned)((a.T + kRouterWaves - 1) / kRouterWaves);
  const size_t lds = a.groups > 1 ? (size_t)kRouterWaves * a.E * sizeof(double) : 0;
  const int threads = 64 * kRouterWaves;
  if (a.E <= 64) router_topk_kernel<DT, 1><<<grid, threads, lds, stream>>>(a);
  else if (a.E <= 128) router_topk_kernel<DT, 2><<<grid, threads, lds, stream>>>(a);
  else if (a.E <= 256) router_topk_kernel<DT, 4><<<grid, threads, lds, stream>>>(a);
  else if (a.E <= 512) router_topk_kernel<DT, 8><<<grid, threads, lds, stream>>>(a);
  else router_topk_kernel<DT, 16><<<grid, threads, lds, stream>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t grad_dt(const RouterArgs& a, const int32_t* ids, const float* grad_w, void* grad_logits,
                   hipStream_t stream) {
  const unsigned grid = (unsigned)((a.T + kRouterWaves - 1) / kRouterWaves);
  router_grad_kernel<DT><<<grid, 64 * kRouterWaves, (size_t)kRouterWaves * a.E * sizeof(float),
                           stream>>>(a, ids, grad_w, (uint8_t*)grad_logits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_topk(const RouterArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kBf16: return topk_dt<kBf16>(a, stream);
    case kF16: return topk_dt<kF16>(a, stream);
    default: return topk_dt<kF32>(a, stream);
  }
}

hipError_t launch_router_grad(const RouterArgs& a, const int32_t* ids, const float* grad_w,
                              void* grad_logits, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kBf16: return grad_dt<kBf16>(a, ids, grad_w, grad_logits, stream);
    case kF16: return grad_dt<kF16>(a, ids, grad_w, grad_logits, stream);
    default: return grad_dt<kF32>(a, ids, grad_w, grad_logits, stream);
  }
}

}  // namespace moe
