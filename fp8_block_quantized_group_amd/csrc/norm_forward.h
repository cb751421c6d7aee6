// The norms before and after a block, forward: a row stays in registers from its
// first load to its last store.  norm_kernels.hip says what they compute; with
// QUANT the normed row also leaves in 8 bits (norm_quant.hip).
#pragma once

#include <type_traits>

#include "kernels.h"
#include "row_vec.h"

namespace moe {

namespace {

// sums of M values over the BT lanes that share a row; buf: theirs, one per call
template <int BT, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], float (*buf)[16]) {
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = wave_sum(v[m]);
  if (BT == 64) return;
  const int lane = threadIdx.x & 63, wave = (threadIdx.x % BT) >> 6;
  if (lane == 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) buf[m][wave] = v[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < BT / 64; ++w) s += buf[m][w];
    v[m] = s;
  }
}

// Squares of values over about 1e19 pass fp32's range.  A row whose sum of
// squares is above kBig is summed again with its values scaled by kShrink.
constexpr float kBig = 1e38f;
constexpr float kShrink = 0x1p-96f;

// 1 / sqrt(mean + eps) from the sum of the squares of values scaled by f
__device__ __forceinline__ float inv_rms(float sum, int H, float eps, float f) {
  return f / sqrtf(sum / (float)H + eps * f * f);
}

// A vector of weights, of the rows' type or fp32: its loads, then, when it is
// used, o + w, or 1 without a weight (columns past the end: o).
template <class RV, bool W32>
struct Weights {
  static constexpr int N = RV::N;
  static constexpr bool kPair = W32 && N == 8;    // two fp32 vectors
  typedef std::conditional_t<W32 && N == 1, RowOne<kF32>, RV> WV;
  u32x4_t a, b;                                   // kPair
  typename WV::Raw v;

  __device__ __forceinline__ void load(const void* w, int col, int H) {
    if (w == nullptr) return;
    const uint8_t* p = (const uint8_t*)w;
    if constexpr (kPair) {
      const int c = RV::inside(col, H);
      a = RowVec<kF32>::template load_at<false>(p, c);
      b = RowVec<kF32>::template load_at<false>(p, c + 4);
    } else {
      v = WV::template load<false>(p, col, H);
    }
  }
  __device__ __forceinline__ void use(const void* w, int col, int H, float o, float (&f)[N]) {
    if (w == nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = 1.0f;
      return;
    }
    if constexpr (kPair) {
      RowVec<kF32>::unpack(a, f);
      RowVec<kF32>::unpack(b, f + 4);
      const int k = col - RV::inside(col, H);     // shifted into place as rows are
      if (k > 0) {
#pragma unroll
        for (int d = 1; d < 8; d <<= 1)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[i] = (k & d) ? (i + d < 8 ? f[(i + d) & 7] : 0.0f) : f[i];
      }
    } else {
      WV::settle(v, col, H);
      WV::unpack(v, f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] += o;
  }
};
template <class RV, bool W32>
__device__ __forceinline__ void load_weights(const void* w, int col, int H, float o,
                                             float (&f)[RV::N]) {
  Weights<RV, W32> v;
  v.load(w, col, H);
  v.use(w, col, H, o, f);
}

__device__ __forceinline__ float gate_value(float g, bool sigmoid) {
  return sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// What the gate's value g enters as, and its derivative by g.  1 - s taken from
// a rounded s would cancel (the slope off by 5e-4 of itself at a gate of 10, 0
// from 17 on); with e = exp(-|g|) both come from 1 / (1 + e).
struct GateGrad {
  float value, slope;
};
__device__ __forceinline__ GateGrad gate_grad(float g, bool sigmoid) {
  if (!sigmoid) return GateGrad{g, 1.0f};
  const float e = expf(-fabsf(g)), r = 1.0f / (1.0f + e);
  return GateGrad{g >= 0.0f ? r : e * r, e * r * r};
}

// the row's inverse root mean square, its N * VPT values per lane given by f
template <int BT, int VPT, int N, class F>
__device__ __forceinline__ float row_inv_rms(F&& value, int H, float eps, float (*buf)[1][16]) {
  float s[1] = {0.0f}, f = 1.0f, v[N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    value(i, v);
#pragma unroll
    for (int c = 0; c < N; ++c) s[0] = fmaf(v[c], v[c], s[0]);
  }
  row_sums<BT, 1>(s, buf[0]);
  if (s[0] > kBig) {                          // the same for every lane of the row
    f = kShrink;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      value(i, v);
#pragma unroll
      for (int c = 0; c < N; ++c) s[0] = fmaf(v[c] * f, v[c] * f, s[0]);
    }
    row_sums<BT, 1>(s, buf[1]);
  }
  return inv_rms(s[0], H, eps, f);
}

// The normed row in 8 bits, staged as the layer takes it: a group's maximum
// crosses the lanes that share it (16 of 8 columns or 32 of 4, MX 4 or 8), each
// lane stores its codes and the first one the scale.  Rows are whole groups, so
// lanes past the row's end share none with others.  The quantizer is the
// staging's own; what it quantizes has not been rounded to 16 bits first, and NaN
// leaves as NaN (the converter's clamp makes -448 of it).
template <int N>
__device__ __forceinline__ void quantize_vector(const NormArgs& a, const float (&h)[N],
                                                int64_t row, int col) {
  float amax = 0.0f;
#pragma unroll
  for (int c = 0; c < N; ++c) amax = fmaxf(amax, fabsf(h[c]));
  const bool mx = a.quant == kQuantMxfp8;
  if (mx) {
    amax = N == 8 ? quad_max(amax) : row8_max(amax);
  } else {
    amax = row16_max(amax);
    if (N == 4) amax = fmaxf(amax, __shfl_xor(amax, 16));
  }
  if (col >= a.H) return;
  const GroupScale s =
      a.quant == kQuantF32 ? group_scale<false>(amax) : group_scale<true>(amax);
  uint8_t* q = a.q + row * a.H + col;
  uint32_t code[N / 4];
#pragma unroll
  for (int c = 0; c < N / 4; ++c)
    code[c] = f32x4_to_e4m3x4(h[4 * c] * s.recip, h[4 * c + 1] * s.recip, h[4 * c + 2] * s.recip,
                              h[4 * c + 3] * s.recip);
  bool nan = false;
#pragma unroll
  for (int c = 0; c < N; ++c) nan |= __builtin_isnan(h[c] * s.recip);
  if (nan) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      if (__builtin_isnan(h[c] * s.recip)) code[c / 4] |= 0x7Fu << (8 * (c & 3));
  }
  if constexpr (N == 8) *reinterpret_cast<uint2*>(q) = make_uint2(code[0], code[1]);
  else *reinterpret_cast<uint32_t*>(q) = code[0];
  const int group = mx ? 32 : 128, in = col % group;
  const int g = col / group, G = a.H / group;
  if (a.quant == kQuantF32) {
    if (in == 0) reinterpret_cast<uint32_t*>(a.q_sf)[row * G + g] = s.stored;
    return;
  }
  const int pitch = mx ? G : (G + 3) / 4 * 4;
  if (in == 0) a.q_sf[row * pitch + g] = (uint8_t)s.stored;
  // the row's pad bytes, up to three, by the lanes next to the last group's first
  else if (g == G - 1 && G - 1 + in / N < pitch) a.q_sf[row * pitch + G - 1 + in / N] = 0;
}

// Weights and gate are loaded with the row (EARLY: up to two vectors per
// lane), as a load after each of the two sums would be waited for in full;
// with four the registers cost more waves than that gains (1024 x 7168: 13.7
// us, 10.4 without).
template <class RV, bool W32, int BT, int VPT, bool QUANT>
__global__ __launch_bounds__(BT == 64 ? 256 : BT) void norm_kernel(const NormArgs a) {
  constexpr int N = RV::N;
  constexpr bool EARLY = VPT <= 2;
  __shared__ float buf[4][1][16];
  const int64_t row = BT == 64 ? (int64_t)block_index() * 4 + (threadIdx.x >> 6) : block_index();
  if (row >= a.T) return;                       // whole waves (BT 64) or never
  const int first = BT == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int H = a.H;
  const int64_t at = row * H * RV::kSize;
  const void* w_post = a.post ? a.w_post : nullptr;
  const uint8_t* gates = a.gate_kind == kGateFull ? a.gate + at
                         : a.gate_kind == kGateChannel ? a.gate : nullptr;
  typename RV::Raw rv[VPT], yv[VPT], gv[VPT];
  Weights<RV, W32> wpost[VPT], wpre[VPT];
  float x[VPT][N], gt = 1.0f;
  auto load_gate = [&](int i) {
    const int col = (first + i * BT) * N;
    if (gates != nullptr) gv[i] = RV::template load<false>(gates, col, H);
    wpost[i].load(w_post, col, H);
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (first + i * BT) * N;
    rv[i] = RV::template load<true>(a.r + at, col, H);
    if (a.y != nullptr) yv[i] = RV::template load<true>(a.y + at, col, H);
  }
  if (a.gate_kind == kGateToken) gt = RV::load_one(a.gate, row);
  if (EARLY) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      load_gate(i);
      wpre[i].load(a.w_pre, (first + i * BT) * N, H);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (first + i * BT) * N;
    RV::settle(rv[i], col, H);
    RV::unpack(rv[i], x[i]);
    if (a.y != nullptr) RV::settle(yv[i], col, H);
  }
  if (a.y != nullptr) {
    float ys = 1.0f;
    if (a.post)
      ys = row_inv_rms<BT, VPT, N>([&](int i, float* v) { RV::unpack(yv[i], v); }, H,
                                   a.eps, buf);
    if (a.gate_kind == kGateToken) gt = gate_value(gt, a.gate_sigmoid);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (first + i * BT) * N;
      if (!EARLY) load_gate(i);
      float y[N], w[N], g[N];
      RV::unpack(yv[i], y);
      wpost[i].use(w_post, col, H, a.offset, w);
#pragma unroll
      for (int c = 0; c < N; ++c) g[c] = gt;
      if (gates != nullptr) {
        RV::settle(gv[i], col, H);
        RV::unpack(gv[i], g);
#pragma unroll
        for (int c = 0; c < N; ++c) g[c] = gate_value(g[c], a.gate_sigmoid);
      }
#pragma unroll
      for (int c = 0; c < N; ++c)
        x[i][c] = col + c < H ? fmaf(a.alpha * g[c], y[c] * ys * w[c], x[i][c]) : 0.0f;
      RV::template store<true>(a.r_out + at, col, H, RV::pack(x[i]));
    }
  }
  if (!QUANT && a.h == nullptr) return;
  const float xs = row_inv_rms<BT, VPT, N>(
      [&](int i, float* v) {
#pragma unroll
        for (int c = 0; c < N; ++c) v[c] = x[i][c];
      },
      H, a.eps, buf + 2);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (first + i * BT) * N;
    if (!EARLY) wpre[i].load(a.w_pre, col, H);
    float w[N], h[N];
    wpre[i].use(a.w_pre, col, H, a.offset, w);
#pragma unroll
    for (int c = 0; c < N; ++c) h[c] = x[i][c] * xs * w[c];
    if (!QUANT || a.h != nullptr) RV::template store<true>(a.h + at, col, H, RV::pack(h));
    if constexpr (QUANT) quantize_vector<N>(a, h, row, col);
  }
}

template <class R, int B, int V>
struct Shape {
  typedef R RV;
  static constexpr int BT = B, VPT = V;       // lanes per row, vectors per lane
};

// With many rows the lanes fit the row, two vectors each where a block is
// small enough (8192 rows, bf16: 5120 columns 59 us with 320 lanes x 2, 79 with
// 256 x 4; 7168 82 with 448 x 2, 90; 4096 rows of 12288: 77 with 512 x 3, 87
// with 512 x 4, 92 with 768 x 2).  Up to this many rows (two per CU) a row gets
// more lanes: the call's time is one row's.  Measured with / without, bf16: 32
// x 7168 4.6 / 5.9 us, 256 x 2048 3.5 / 5.8, 512 x 7168 7.1 / 7.5, 600 x 7168
// 8.7 / 8.4.
constexpr int kFewRows = 512;

template <int DT, bool W32, bool QUANT>
hipError_t norm_dt(const NormArgs& a, hipStream_t stream) {
  const int nv = (a.H + RowVec<DT>::N - 1) / RowVec<DT>::N;
  auto go = [&](auto shape) {
    constexpr int BT = decltype(shape)::BT, VPT = decltype(shape)::VPT;
    typedef typename decltype(shape)::RV RV;
    const int64_t grid = BT == 64 ? (a.T + 3) / 4 : a.T;
    norm_kernel<RV, W32, BT, VPT, QUANT><<<grid_of(grid), BT == 64 ? 256 : BT, 0, stream>>>(a);
    return hipGetLastError();
  };
  if constexpr (!QUANT) {                     // rows in 8 bits are whole groups
    if (a.H < RowVec<DT>::N) return go(Shape<RowOne<DT>, 64, 1>());
  }
  if (nv <= 64) return go(Shape<RowVec<DT>, 64, 1>());
  if (nv <= 128) return go(Shape<RowVec<DT>, 64, 2>());
  if (a.T <= kFewRows) {
    if (nv <= 256) return go(Shape<RowVec<DT>, 256, 1>());
    if (nv <= 512) return go(Shape<RowVec<DT>, 512, 1>());
    if (nv <= 1024) return go(Shape<RowVec<DT>, 512, 2>());
    if (nv <= 2048) return go(Shape<RowVec<DT>, 1024, 2>());
  }
  if (nv <= 192) return go(Shape<RowVec<DT>, 64, 3>());
  if (nv <= 256) return go(Shape<RowVec<DT>, 64, 4>());
  if (nv <= 384) return go(Shape<RowVec<DT>, 192, 2>());
  if (nv <= 512) return go(Shape<RowVec<DT>, 256, 2>());
  if (nv <= 640) return go(Shape<RowVec<DT>, 320, 2>());
  if (nv <= 768) return go(Shape<RowVec<DT>, 384, 2>());
  if (nv <= 896) return go(Shape<RowVec<DT>, 448, 2>());
  if (nv <= 1024) return go(Shape<RowVec<DT>, 512, 2>());
  if (nv <= 1536) return go(Shape<RowVec<DT>, 512, 3>());
  if (nv <= 2048) return go(Shape<RowVec<DT>, 512, 4>());
  if (nv <= 4096) return go(Shape<RowVec<DT>, 1024, 4>());
  if constexpr (DT == kF32) return go(Shape<RowVec<DT>, 1024, 8>());
  return hipErrorInvalidValue;                // 2-byte rows end at 4096 vectors
}

}  // namespace

}  // namespace moe
