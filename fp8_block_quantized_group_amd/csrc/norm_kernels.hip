// The norms before and after a block, fused with the block's gate, its
// residual scale and the residual add, and their gradients.
//
//   n  = y * rsqrt(mean(y^2) + eps) * (o + w_post)      (or n = y)
//   r' = r + alpha * gate * n
//   h  = r' * rsqrt(mean(r'^2) + eps) * (o + w_pre)
//
// A row stays in registers from its first load to its last store: BT lanes
// hold VPT vectors each, the row sums cross the lanes of a wave in registers
// and, for BT over 64, the waves through LDS.  Everything is fp32; h is made
// from r' before r' is rounded.
//
// Bound by HBM: every stream is read or written once, non-temporal.  MI355X,
// where a 2 GiB copy moves 5.1 TB/s: forward 16381 x 4096 bf16 92 us (537 MB,
// 5.8 TB/s); gradients 4095 x 7168 bf16 75-80 us (352 MB, 4.4-4.7 TB/s: the
// row sums' barriers leave gaps, and the column sums of 256 blocks cost 22 MB
// each way).
#include <type_traits>

#include "norm_forward.h"

namespace moe {

namespace {

// Gradients at the stored r' (x below).  With xs, ys the inverse root means,
// xh = x xs and yh = y ys:
//   D  = dr'_in + xs (dh w_pre - xh mean(dh w_pre xh))       -> grad r
//   dn = alpha gate D,  e = dn w_post
//   dy = ys (e - yh mean(e yh))
//   grad w_pre += dh xh,  grad w_post += dn yh,  grad gate += alpha D n, times
//   the slope of a sigmoid
// Each block walks rows with a stride of the grid and keeps the column sums
// of its rows; they go to part[output][block][H] and are added up in block
// order by grad_sum_kernel, so the result does not depend on timing.

// what a column vector needs of the row's first sums
struct GradRow {
  float xs, xm;       // inverse root mean of x; mean(dh w_pre xh)
  float ys;           // inverse root mean of y (1 without a post norm)
};

// D, e and the addends of the column sums of one column vector, from its
// weights (o + w, or 1) and its gate as it enters the product.  dg is the
// gradient of that value; the sigmoid's slope multiplies it once per gate, after
// the sum where columns or rows share one.
template <int N, bool HAS_Y>
__device__ __forceinline__ void grad_columns(const NormGradArgs& a, const GradRow& r,
                                             const float (&x)[N], const float (&dh)[N],
                                             const float (&y)[N], const float (&wpre)[N],
                                             const float (&wpost)[N], const float (&g)[N],
                                             float (&D)[N], float (&dpre)[N], float (&e)[N],
                                             float (&dpost)[N], float (&dg)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float xh = x[c] * r.xs;
    dpre[c] = dh[c] * xh;
    D[c] = fmaf(r.xs, fmaf(dh[c], wpre[c], -xh * r.xm), D[c]);
  }
  if (!HAS_Y) return;
  // Each product once, as a value: fused into the two sums that dg goes to, its
  // factors stay live, and the fullest shapes spill up to 17 registers.
#pragma unroll
  for (int c = 0; c < N; ++c) {
#pragma clang fp contract(off)
    const float yh = y[c] * r.ys, ad = a.alpha * D[c], adg = ad * g[c];
    dg[c] = ad * (yh * wpost[c]);
    dpost[c] = adg * yh;
    e[c] = adg * wpost[c];
  }
}

// s: sums of x^2, dh w_pre x and y^2, of values scaled by fx and fy
__device__ __forceinline__ GradRow grad_row(const NormGradArgs& a, const float (&s)[3], float fx,
                                            float fy) {
  GradRow r;
  r.xs = inv_rms(s[0], a.H, a.eps, fx);
  r.xm = r.xs / fx * (s[1] / (float)a.H);
  r.ys = a.post ? inv_rms(s[2], a.H, a.eps, fy) : 1.0f;
  return r;
}

// Rows in registers: BT lanes per row, kGradThreads / BT rows side by side
// (one for BT above), each lane with the column sums of its VPT vectors.
//
// One block per CU (two cost more in weights and column sums than they hide:
// 120 us against 100): the column sums and the next row, which is loaded while
// this one is worked on, take the registers (FULL, a gate of the rows' own
// shape, takes the place of the gate's column sums).  The weights and a
// per-channel gate lie in LDS as fp32, so that nothing but rows goes through
// the counter of loads in flight; a plane of four columns of every vector
// after the other, 16 bytes from lane to lane.
constexpr int kGradThreads = 512;
constexpr int grad_groups(int bt) { return bt < kGradThreads ? kGradThreads / bt : 1; }

// Every load is issued whatever the call leaves out: how many loads follow
// one is then known, and waiting for this row's leaves the next row's in
// flight (a null gradient's loads go to x and are dropped).
enum GradForm { kNoBlock, kBlock, kBlockFullGate };

template <class RV, int VPT, GradForm FORM>
struct GradVectors {
  typename RV::Raw x[VPT], dh[VPT], dr[VPT], y[VPT], gate[VPT];
  float gt;                                   // the token's gate as stored

  // the row's vectors of this lane (the last row's for one past it)
  template <int BT>
  __device__ __forceinline__ void load(const NormGradArgs& a, int64_t row, int first) {
    if (row >= a.T) row = a.T - 1;
    const int64_t at = row * a.H * RV::kSize;
    const uint8_t* pdh = a.dh != nullptr ? a.dh : a.x;
    const uint8_t* pdr = a.dr_in != nullptr ? a.dr_in : a.x;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (first + i * BT) * RV::N;
      x[i] = RV::template load<true>(a.x + at, col, a.H);
      dh[i] = RV::template load<true>(pdh + at, col, a.H);
      dr[i] = RV::template load<true>(pdr + at, col, a.H);
      if (FORM != kNoBlock) y[i] = RV::template load<true>(a.y + at, col, a.H);
      if (FORM == kBlockFullGate) gate[i] = RV::template load<true>(a.gate + at, col, a.H);
    }
    if (FORM == kBlock) {
      const bool token = a.gate_kind == kGateToken;
      gt = RV::load_one(token ? a.gate : a.x, token ? row : 0);
    }
  }
  // zeros past the row's h columns (0: a row that is not there) and for what
  // the call leaves out
  template <int BT>
  __device__ __forceinline__ void settle(const NormGradArgs& a, int first, int h) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (first + i * BT) * RV::N;
      if (a.dh == nullptr) dh[i] = typename RV::Raw{};
      if (a.dr_in == nullptr) dr[i] = typename RV::Raw{};
      if (col + RV::N <= h) continue;
      RV::settle(x[i], col, h);
      RV::settle(dh[i], col, h);
      RV::settle(dr[i], col, h);
      if (FORM != kNoBlock) RV::settle(y[i], col, h);
      if (FORM == kBlockFullGate) RV::settle(gate[i], col, h);
    }
  }
};

template <class RV, bool W32, int BT, int VPT, GradForm FORM>
__global__ __launch_bounds__(BT < kGradThreads ? kGradThreads : BT) void norm_grad_kernel(
    const NormGradArgs a) {
  constexpr int N = RV::N, G = grad_groups(BT), NV = BT * VPT;
  constexpr int P = N < 4 ? N : 4;            // columns of a plane
  constexpr bool HAS_Y = FORM != kNoBlock, FULL = FORM == kBlockFullGate;
  constexpr bool AHEAD = BT <= kGradThreads;
  constexpr int THREADS = BT < kGradThreads ? kGradThreads : BT;
  constexpr int SUMS = FORM == kNoBlock ? 1 : FULL ? 2 : 3;   // column sums: pre, post, gate
  __shared__ float buf1[2][G][3][16], buf2[2][G][2][16], buf3[2][G][3][16];
  __shared__ float sums[G][BT * N];
  __shared__ float slope_of[G];               // a token gate's, kept for the lane that writes it
  __shared__ __align__(16) float wlds[SUMS][N / P][NV][P];   // pre, post, gate
  const int sub = threadIdx.x / BT, first = threadIdx.x % BT;
  const int64_t stride = (int64_t)gridDim.x * G;
  const int H = a.H;
  auto read = [&](int o, int i, float (&f)[N]) {
#pragma unroll
    for (int p = 0; p < N / P; ++p)
#pragma unroll
      for (int c = 0; c < P; ++c) f[P * p + c] = wlds[o][p][first + i * BT][c];
  };
  GradVectors<RV, VPT, FORM> cur;
  cur.template load<BT>(a, (int64_t)blockIdx.x * G + sub, first);
  {
    constexpr int IT = (NV + THREADS - 1) / THREADS;
    Weights<RV, W32> w[2][IT];
    typename RV::Raw gv[IT];
    const void* w_post = a.post ? a.w_post : nullptr;
    const bool channel = FORM == kBlock && a.gate_kind == kGateChannel;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int v = threadIdx.x + i * THREADS;
      w[0][i].load(a.w_pre, v * N, H);
      if (HAS_Y) w[1][i].load(w_post, v * N, H);
      if (channel) gv[i] = RV::template load<false>(a.gate, v * N, H);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int v = threadIdx.x + i * THREADS;
      if (v >= NV) continue;
      float f[3][N];
      w[0][i].use(a.w_pre, v * N, H, a.offset, f[0]);
      if (HAS_Y) w[1][i].use(w_post, v * N, H, a.offset, f[1]);
#pragma unroll
      for (int c = 0; c < N; ++c) f[2][c] = 1.0f;
      if (channel) {
        RV::settle(gv[i], v * N, H);
        RV::unpack(gv[i], f[2]);
#pragma unroll
        for (int c = 0; c < N; ++c) f[2][c] = gate_value(f[2][c], a.gate_sigmoid);
      }
#pragma unroll
      for (int o = 0; o < SUMS; ++o)
#pragma unroll
        for (int c = 0; c < N; ++c) wlds[o][c / P][v][c % P] = f[o][c];
    }
  }
  __syncthreads();
  __builtin_amdgcn_s_waitcnt(0);              // the first row, once
  constexpr int VP = SUMS > 1 ? VPT : 1, VG = SUMS > 2 ? VPT : 1;
  float apre[VPT][N], apost[VP][N], agate[VG][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int c = 0; c < N; ++c) apre[i][c] = apost[i % VP][c] = agate[i % VG][c] = 0.0f;
  int turn = 0;
  // every group makes the same number of turns (the sums meet at barriers);
  // one past the last row computes on zeros and stores nothing
  for (int64_t row0 = (int64_t)blockIdx.x * G; row0 < a.T; row0 += stride, turn ^= 1) {
    const int64_t row = row0 + sub;
    const bool live = row < a.T;
    const int h = live ? H : 0;               // columns of the row
    const int64_t at = row * H * RV::kSize;
    GradVectors<RV, VPT, FORM> next;
    if constexpr (AHEAD) next.template load<BT>(a, row + stride, first);
    cur.template settle<BT>(a, first, h);
    float s[3] = {0.0f, 0.0f, 0.0f}, fx = 1.0f, fy = 1.0f;
    auto add_up = [&](auto scaled) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float x[N], dh[N], y[N], w[N];
        RV::unpack(cur.x[i], x);
        RV::unpack(cur.dh[i], dh);
        if (HAS_Y) RV::unpack(cur.y[i], y);
        read(0, i, w);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float xc = scaled ? x[c] * fx : x[c];
          s[0] = fmaf(xc, xc, s[0]);
          s[1] = fmaf(dh[c] * w[c], xc, s[1]);
          if (HAS_Y) {
            const float yc = scaled ? y[c] * fy : y[c];
            s[2] = fmaf(yc, yc, s[2]);
          }
        }
      }
    };
    add_up(std::false_type());
    row_sums<BT, 3>(s, buf1[turn][sub]);
    bool again = s[0] > kBig || s[2] > kBig;
    if (G > 1 && BT > 64) again = __syncthreads_or(again);   // the groups meet in row_sums
    if (again) {
      fx = s[0] > kBig ? kShrink : 1.0f;
      fy = s[2] > kBig ? kShrink : 1.0f;
      s[0] = s[1] = s[2] = 0.0f;
      add_up(std::true_type());
      row_sums<BT, 3>(s, buf3[turn][sub]);
    }
    const GradRow r = grad_row(a, s, fx, fy);
    float gt = 1.0f;
    if (FORM == kBlock && a.gate_kind == kGateToken) {
      const GateGrad one = gate_grad(cur.gt, a.gate_sigmoid);
      gt = one.value;
      if (first == 0) slope_of[sub] = one.slope;
    }
    float e[VPT][N], q[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      __builtin_amdgcn_sched_barrier(0);      // one vector after the other: registers
      const int col = (first + i * BT) * N;
      float x[N], dh[N], D[N], y[N], wpre[N], wpost[N], g[N], dpre[N], dpost[N], dg[N], slope[N];
      RV::unpack(cur.x[i], x);
      RV::unpack(cur.dh[i], dh);
      RV::unpack(cur.dr[i], D);
      read(0, i, wpre);
      if constexpr (HAS_Y) {
        RV::unpack(cur.y[i], y);
        read(1, i, wpost);
        if constexpr (FULL) {
          RV::unpack(cur.gate[i], g);
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const GateGrad one = gate_grad(g[c], a.gate_sigmoid);
            g[c] = one.value;
            slope[c] = one.slope;
          }
        } else {
          read(2, i, g);
#pragma unroll
          for (int c = 0; c < N; ++c) g[c] *= gt;
        }
      }
      grad_columns<N, HAS_Y>(a, r, x, dh, y, wpre, wpost, g, D, dpre, e[i], dpost, dg);
      if (col < h) RV::template store<true>(a.dr + at, col, H, RV::pack(D));
#pragma unroll
      for (int c = 0; c < N; ++c) apre[i][c] += dpre[c];
      if constexpr (!HAS_Y) continue;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        apost[i % VP][c] += dpost[c];
        agate[i % VG][c] += FULL ? 0.0f : dg[c];
        q[0] = fmaf(e[i][c], y[c] * r.ys, q[0]);
        q[1] += dg[c];
        if (FULL) dg[c] *= slope[c];
      }
      if (FULL && a.d_gate != nullptr && col < h)
        RV::template store<true>((uint8_t*)a.d_gate + at, col, H, RV::pack(dg));
    }
    if constexpr (HAS_Y) {
      row_sums<BT, 2>(q, buf2[turn][sub]);
      if (live && a.gate_kind == kGateToken && a.d_gate != nullptr && first == 0)
        ((float*)a.d_gate)[row] = q[1] * slope_of[sub];
      const float ym = a.post ? q[0] / (float)H : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int col = (first + i * BT) * N;
        if (col >= h) continue;
        float y[N], d[N];
        RV::unpack(cur.y[i], y);
#pragma unroll
        for (int c = 0; c < N; ++c) d[c] = r.ys * fmaf(-y[c] * r.ys, ym, e[i][c]);
        RV::template store<true>(a.dy + at, col, H, RV::pack(d));
      }
    }
    if constexpr (AHEAD) cur = next;
    else cur.template load<BT>(a, row + stride, first);
  }
  // the groups' column sums, in group order, as the block's part
#pragma unroll
  for (int o = 0; o < SUMS; ++o) {
    if (!(a.want & (1 << o))) continue;
    float* part = a.part + ((int64_t)o * gridDim.x + blockIdx.x) * H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float* mine = o == 0 ? apre[i] : o == 1 ? apost[i % VP] : agate[i % VG];
      if (G > 1) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < N; ++c) sums[sub][first * N + c] = mine[c];
        __syncthreads();
        if (sub != 0) continue;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          float v = 0.0f;
#pragma unroll
          for (int g = 0; g < G; ++g) v += sums[g][first * N + c];
          mine[c] = v;
        }
      }
      const int col = (first + i * BT) * N;
      if constexpr (N == 1) {
        if (col < H) part[col] = mine[0];
      } else {
#pragma unroll
        for (int c = 0; c < N; c += 4)
          RowVec<kF32>::template store<false>((uint8_t*)part, col + c, H,
                                              RowVec<kF32>::pack(mine + c));
      }
    }
  }
}

// Rows too wide for registers (2-byte types past 8192 columns, fp32 past
// 8192): one block per row, which is read three times (from the caches after
// the first): for its first sums, for its second, and to write.  The block's
// column sums are kept in its part itself.  2048 x 16384 bf16: 440 us, 0.9
// TB/s of what the call has to move; 62 us without a block, in registers.
constexpr int kWideThreads = 1024;

template <class RV, bool W32>
__global__ __launch_bounds__(kWideThreads) void norm_grad_wide_kernel(const NormGradArgs a) {
  constexpr int N = RV::N;
  __shared__ float buf1[2][3][16], buf2[2][2][16], buf3[2][3][16];
  const int H = a.H;
  const bool has_y = a.y != nullptr;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const int64_t at = row * H * RV::kSize;
    float x[N], dh[N], D[N], y[N];
    auto load = [&](int col) {
      auto one = [&](const uint8_t* p, float (&f)[N]) {
        typename RV::Raw v = {};
        if (p != nullptr) v = RV::template load<false>(p + at, col, H);
        RV::settle(v, col, H);
        RV::unpack(v, f);
      };
      one(a.x, x);
      one(a.dh, dh);
      one(a.dr_in, D);
      one(a.y, y);
    };
    float s[3] = {0.0f, 0.0f, 0.0f}, fx = 1.0f, fy = 1.0f;
    auto add_up = [&]() {
      for (int col = threadIdx.x * N; col < H; col += kWideThreads * N) {
        float w[N];
        load(col);
        load_weights<RV, W32>(a.w_pre, col, H, a.offset, w);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float xc = x[c] * fx, yc = y[c] * fy;
          s[0] = fmaf(xc, xc, s[0]);
          s[1] = fmaf(dh[c] * w[c], xc, s[1]);
          s[2] = fmaf(yc, yc, s[2]);
        }
      }
    };
    add_up();
    row_sums<kWideThreads, 3>(s, buf1[turn]);
    if (s[0] > kBig || s[2] > kBig) {
      fx = s[0] > kBig ? kShrink : 1.0f;
      fy = s[2] > kBig ? kShrink : 1.0f;
      s[0] = s[1] = s[2] = 0.0f;
      add_up();
      row_sums<kWideThreads, 3>(s, buf3[turn]);
    }
    float e[N], dpre[N], dpost[N], dg[N], q[2] = {0.0f, 0.0f};
    const GradRow r = grad_row(a, s, fx, fy);
    const bool token = has_y && a.gate_kind == kGateToken;
    const GateGrad gt = token ? gate_grad(RV::load_one(a.gate, row), a.gate_sigmoid)
                              : GateGrad{1.0f, 1.0f};
    auto columns = [&](int col) {
      float wpre[N], wpost[N], g[N], slope[N];
      load(col);
      load_weights<RV, W32>(a.w_pre, col, H, a.offset, wpre);
      load_weights<RV, W32>(a.post ? a.w_post : nullptr, col, H, a.offset, wpost);
#pragma unroll
      for (int c = 0; c < N; ++c) {
        g[c] = gt.value;
        slope[c] = 1.0f;
      }
      if (has_y && (a.gate_kind == kGateChannel || a.gate_kind == kGateFull)) {
        typename RV::Raw gv =
            RV::template load<false>(a.gate + (a.gate_kind == kGateFull ? at : 0), col, H);
        RV::settle(gv, col, H);
        RV::unpack(gv, g);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const GateGrad one = gate_grad(g[c], a.gate_sigmoid);
          g[c] = one.value;
          if (a.gate_kind == kGateFull) slope[c] = one.slope;
        }
      }
      if (has_y) {
        grad_columns<N, true>(a, r, x, dh, y, wpre, wpost, g, D, dpre, e, dpost, dg);
#pragma unroll
        for (int c = 0; c < N; ++c) dg[c] *= slope[c];
      } else {
        grad_columns<N, false>(a, r, x, dh, y, wpre, wpost, g, D, dpre, e, dpost, dg);
      }
    };
    if (has_y) {
      for (int col = threadIdx.x * N; col < H; col += kWideThreads * N) {
        columns(col);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          q[0] = fmaf(e[c], y[c] * r.ys, q[0]);
          q[1] += dg[c];
        }
      }
      row_sums<kWideThreads, 2>(q, buf2[turn]);
      if (a.gate_kind == kGateToken && a.d_gate != nullptr && threadIdx.x == 0)
        ((float*)a.d_gate)[row] = q[1] * gt.slope;
    }
    const float ym = a.post ? q[0] / (float)H : 0.0f;
    const bool begin = row == blockIdx.x;
    for (int col = threadIdx.x * N; col < H; col += kWideThreads * N) {
      columns(col);
      RV::template store<true>(a.dr + at, col, H, RV::pack(D));
      if (has_y) {
        if (a.gate_kind == kGateFull && a.d_gate != nullptr)
          RV::template store<true>((uint8_t*)a.d_gate + at, col, H,
                                           RV::pack(dg));
#pragma unroll
        for (int c = 0; c < N; ++c) e[c] = r.ys * fmaf(-y[c] * r.ys, ym, e[c]);
        RV::template store<true>(a.dy + at, col, H, RV::pack(e));
      }
#pragma unroll
      for (int o = 0; o < 3; ++o) {
        if (!(a.want & (1 << o))) continue;
        float* part = a.part + ((int64_t)o * gridDim.x + blockIdx.x) * H;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (col + c >= H) continue;
          const float v = o == 0 ? dpre[c] : o == 1 ? dpost[c] : dg[c];
          part[col + c] = begin ? v : part[col + c] + v;
        }
      }
    }
  }
}

constexpr int kSumCols = 64, kSumWays = 16, kSumBatch = 16;

// Column c of output o: 16 interleaved runs of the blocks' parts side by
// side, each with 16 loads in flight, then the runs in order.  gate: the
// channel gate behind a sigmoid (else nullptr), whose slope multiplies output 2.
template <int DT>
__global__ __launch_bounds__(kSumCols* kSumWays) void grad_sum_kernel(const float* part,
                                                                     int parts, int H, float* g0,
                                                                     float* g1, float* g2,
                                                                     const uint8_t* gate) {
  __shared__ float run[kSumWays][kSumCols];
  float* out = blockIdx.y == 0 ? g0 : blockIdx.y == 1 ? g1 : g2;
  if (out == nullptr) return;
  part += (int64_t)blockIdx.y * parts * H;
  const int x = threadIdx.x % kSumCols, w = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + x, at = min(c, H - 1);
  float s = 0.0f;
  for (int p0 = w; p0 < parts; p0 += kSumWays * kSumBatch) {
    float v[kSumBatch];
#pragma unroll
    for (int u = 0; u < kSumBatch; ++u)
      v[u] = part[(int64_t)min(p0 + u * kSumWays, parts - 1) * H + at];
#pragma unroll
    for (int u = 0; u < kSumBatch; ++u) s += p0 + u * kSumWays < parts ? v[u] : 0.0f;
  }
  run[w][x] = s;
  __syncthreads();
  if (w != 0 || c >= H) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumWays; ++i) s += run[i][x];
  if (blockIdx.y == 2 && gate != nullptr) s *= gate_grad(RowVec<DT>::load_one(gate, c), true).slope;
  out[c] = s;
}

template <int DT, bool W32>
hipError_t norm_grad_dt(const NormGradArgs& a, int blocks, hipStream_t stream) {
  const int nv = (a.H + RowVec<DT>::N - 1) / RowVec<DT>::N;
  auto go = [&](auto shape) {
    constexpr int BT = decltype(shape)::BT, VPT = decltype(shape)::VPT;
    typedef typename decltype(shape)::RV RV;
    const int threads = BT < kGradThreads ? kGradThreads : BT;
    if (a.y == nullptr)
      norm_grad_kernel<RV, W32, BT, VPT, kNoBlock><<<blocks, threads, 0, stream>>>(a);
    else if (a.gate_kind == kGateFull)
      norm_grad_kernel<RV, W32, BT, VPT, kBlockFullGate><<<blocks, threads, 0, stream>>>(a);
    else
      norm_grad_kernel<RV, W32, BT, VPT, kBlock><<<blocks, threads, 0, stream>>>(a);
    return hipGetLastError();
  };
  if (a.H < RowVec<DT>::N) return go(Shape<RowOne<DT>, 64, 1>());
  if (nv <= 64) return go(Shape<RowVec<DT>, 64, 1>());
  if (nv <= 128) return go(Shape<RowVec<DT>, 128, 1>());
  if (nv <= 256) return go(Shape<RowVec<DT>, 256, 1>());
  if (nv <= 512) return go(Shape<RowVec<DT>, 512, 1>());
  if (nv <= 1024) return go(Shape<RowVec<DT>, 512, 2>());
  // 1024 x 2 vectors: as fp32; of a 2-byte type, with twice the columns, only
  // without a block's sums
  if constexpr (DT == kF32) {
    if (nv <= 2048) return go(Shape<RowVec<DT>, 1024, 2>());
  } else if (nv <= 2048 && a.y == nullptr) {
    norm_grad_kernel<RowVec<DT>, W32, 1024, 2, kNoBlock><<<blocks, 1024, 0, stream>>>(a);
    return hipGetLastError();
  }
  norm_grad_wide_kernel<RowVec<DT>, W32><<<blocks, kWideThreads, 0, stream>>>(a);
  return hipGetLastError();
}

int rows_per_block(int H, int dtype) {
  const int n = 16 / dtype_size(dtype), nv = (H + n - 1) / n;
  return grad_groups(nv <= 64 ? 64 : nv <= 128 ? 128 : nv <= 256 ? 256 : 512);
}

}  // namespace

// blocks of the gradient kernel, each with a part of the column sums
int norm_grad_parts(int64_t T, int H, int dtype) {
  const int per = rows_per_block(H, dtype);
  const int64_t need = (T + per - 1) / per;
  return (int)(need < kNormGradBlocks ? need : kNormGradBlocks);
}

hipError_t launch_norm(const NormArgs& a, int dtype, bool w32, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  switch (dtype) {
    case kBf16: return w32 ? norm_dt<kBf16, true, false>(a, stream)
                        : norm_dt<kBf16, false, false>(a, stream);
    case kF16: return w32 ? norm_dt<kF16, true, false>(a, stream)
                       : norm_dt<kF16, false, false>(a, stream);
    default: return norm_dt<kF32, true, false>(a, stream);
  }
}

hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, bool w32, float* g_pre,
                            float* g_post, float* g_gate, hipStream_t stream) {
  const int blocks = norm_grad_parts(a.T, a.H, dtype);
  hipError_t err = hipSuccess;
  if (blocks > 0) {
    switch (dtype) {
      case kBf16:
        err = w32 ? norm_grad_dt<kBf16, true>(a, blocks, stream)
                  : norm_grad_dt<kBf16, false>(a, blocks, stream);
        break;
      case kF16:
        err = w32 ? norm_grad_dt<kF16, true>(a, blocks, stream)
                  : norm_grad_dt<kF16, false>(a, blocks, stream);
        break;
      default: err = norm_grad_dt<kF32, true>(a, blocks, stream);
    }
  }
  if (err != hipSuccess || (g_pre == nullptr && g_post == nullptr && g_gate == nullptr))
    return err;
  const bool slope = blocks > 0 && a.gate_kind == kGateChannel && a.gate_sigmoid;
  auto sum = [&](auto dt) {
    grad_sum_kernel<decltype(dt)::value>
        <<<dim3((a.H + kSumCols - 1) / kSumCols, 3), kSumCols * kSumWays, 0, stream>>>(
            a.part, blocks, a.H, g_pre, g_post, g_gate, slope ? a.gate : nullptr);
    return hipGetLastError();
  };
  switch (dtype) {
    case kBf16: return sum(std::integral_constant<int, kBf16>());
    case kF16: return sum(std::integral_constant<int, kF16>());
    default: return sum(std::integral_constant<int, kF32>());
  }
}

}  // namespace moe
