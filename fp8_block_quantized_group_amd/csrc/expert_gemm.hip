// Products of rows sorted by expert with the experts' own bf16, fp16 or fp32
// weights, and their gradients:
//
//   out[r, :]  = F(x[r, :] W_e^T)                 e the expert of row r
//   grad_x     = d W_e                            d = F' grad_out (act_grad_kernel)
//   grad_W_e   = sum over the expert's rows of d[r, :]^T x[r, :]
//
// F is the identity or one of the layer's activations; a gated one takes the
// first half of W's rows as gate and the second as up, and a block computes 16
// (or 32) of each side by side, so that a wave holds both when it stores.
//
// One kernel, three forms: a block makes BM x BN of the result in registers
// from LDS tiles of 128 bytes of the reduction, a ring of two to four of them (two
// where the operands' rows are not multiples of 16 bytes: they pass through registers,
// loaded a step ahead).  The MFMA's
// A operand is the side of the result's columns and its B operand that of its
// rows, so a lane holds four consecutive columns of one row.  An operand whose
// memory runs along the reduction (x and W in out, d in grad_x) lies in LDS as
// rows of 128 bytes and is read 16 bytes per lane; one whose memory runs along
// the result (W in grad_x, both in grad_W) lies there as it comes and is read
// transposed by ds_read_b64_tr_b16 (fp32: word by word).  Every product of the
// 16-bit types is exact and sums are fp32; fp32 goes through the fp32 MFMA.
//
// A batch's product waits for its tiles: 32768 rows of 32 experts, 7168 by 2 x 2048, bf16
// with silu and the pre-activations kept, 1.9 ms (0.94 PFLOP/s; a library's dense product
// of that size 1.3 ms), the MFMAs busy 45 % of the cycles at 2.1 GHz, the waves 37 % of
// theirs at waits and barriers.  The ring holds two stages of 64 KB, so a step's barrier
// waits for loads that were issued behind the one before.  Register double buffers, wave
// pairs in turns and more waves in smaller tiles gave nothing.  Products of few rows are
// bound by the weights' bytes.
#include <algorithm>
#include <type_traits>

#include "expert_act.h"
#include "expert_rows.h"
#include "kernels.h"
#include "lds_copy.h"
#include "row_vec.h"

namespace moe {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr uint32_t kOutOfRange = 0xF0000000u;   // past every buffer: reads as zeros
constexpr int kRowB = 128;                      // bytes of the reduction per step
constexpr int kCus = 256;                       // of the card

enum Product { kOut, kGradX, kGradW };

template <int BM_, int BN_, int WM_, int WN_, int PER_CU_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, PER_CU = PER_CU_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles of a wave
  static constexpr int WAVES_PER_EU = PER_CU * NW / 4 > 0 ? PER_CU * NW / 4 : 1;
  static_assert(TN % 2 == 0, "gate and up in one wave");
};

// 16-byte chunk c of LDS row r of an operand that runs along the reduction is
// at chunk c ^ (r & 7).  A ds_read_b128 passes 16 lanes at a time, of the first
// half lanes 0-3, 12-15, 20-23 and 24-27, then the others: rows 0-3 and 12-15 at
// one chunk with rows 4-11 at the next, which land in 16 different bank groups.
// (With the key of passes of 8 consecutive lanes every read took twice its time.)
__device__ __forceinline__ int key_row(int r) { return r & 7; }
// The same for one that runs along the result: row r is a step of the
// reduction.  A transposed read's 16 lanes take 32 bytes of 4 rows, its four
// groups rows 8 apart; fp32 reads 64 bytes of rows 4 apart.
template <int DT>
__device__ __forceinline__ int key_col(int r) {
  return DT == kF32 ? ((r >> 2) & 3) << 2 : ((r & 3) | ((r >> 1) & 4)) << 1;
}

// Four registers of a fragment: 8 16-bit or 4 fp32 values along the reduction.
template <int DT>
__device__ __forceinline__ v4f mma(u32x4_t a, u32x4_t b, v4f c) {
  if constexpr (DT == kBf16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  } else if constexpr (DT == kF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  } else {
    // lane group g holds values 4g .. 4g+3: each MFMA takes one of every group
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c,
                                               0, 0, 0);
    return c;
  }
}

// The fragment of 16 rows (or columns) from `first` for step s of a stage:
// lane l holds row first + l % 16, chunk 4s + l / 16 of the reduction.
template <int DT, bool RED, int COLS>
__device__ __forceinline__ u32x4_t fragment(const uint8_t* tile, int first, int s, int lane) {
  const int i = lane & 15, g = lane >> 4;
  if constexpr (!RED) {
    const int r = first + i;
    return *reinterpret_cast<const u32x4_t*>(tile + r * kRowB +
                                             (((4 * s + g) ^ key_row(r)) << 4));
  } else if constexpr (DT == kF32) {
    u32x4_t v;
    const int c = (first + i) >> 2, sub = ((first + i) & 3) << 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 16 * s + 4 * g + j;
      v[j] = *reinterpret_cast<const uint32_t*>(tile + r * (COLS * 4) +
                                                ((c ^ key_col<DT>(r)) << 4) + sub);
    }
    return v;
  } else {
    // 16 lanes read 4 rows of 16 columns, 4 columns each, and get back 4 rows of
    // one column; rows r and r + 4 have the same key
    const int r = 32 * s + 8 * g + (i >> 2), c = (first >> 3) + ((i & 3) >> 1);
    const uint8_t* p = tile + r * (COLS * 2) + ((c ^ key_col<DT>(r)) << 4) + ((i & 1) << 3);
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * (COLS * 2)));
    u32x4_t v;
    v[0] = __builtin_bit_cast(uint2, lo).x;
    v[1] = __builtin_bit_cast(uint2, lo).y;
    v[2] = __builtin_bit_cast(uint2, hi).x;
    v[3] = __builtin_bit_cast(uint2, hi).y;
    return v;
  }
}

// Where an operand's 16-byte chunks come from.  RED: LDS rows are steps of the
// reduction and chunks run along the result's columns.
template <int DT, bool RED, int ROWS, int THREADS>
struct Slots {
  static constexpr int ES = dtype_size(DT), CE = 16 / ES, BK = kRowB / ES;
  static constexpr int CHUNKS = RED ? ROWS * ES / 16 : 8;     // of an LDS row
  static constexpr int COUNT = ROWS * 8 / THREADS;            // per lane
  static_assert(ROWS * 8 % THREADS == 0 && (!RED || CHUNKS >= 16), "whole instructions");
  static __device__ __forceinline__ int row(int i) {
    return (i * THREADS + (int)threadIdx.x) / CHUNKS;
  }
  static __device__ __forceinline__ int chunk(int i) {
    const int r = row(i), pos = (int)threadIdx.x % CHUNKS;
    return pos ^ (RED ? key_col<DT>(r) : key_row(r));
  }
};

// A chunk at column col of a row of `limit` columns, at any address, zeros past
// the end; in two steps, so that the load is in flight in between.
template <int DT>
__device__ __forceinline__ u32x4_t load_chunk(const uint8_t* row, int col, int limit) {
  constexpr int CE = RowVec<DT>::N;
  if (limit >= CE) return RowVec<DT>::template load<false>(row, col, limit);
  float f[CE];
#pragma unroll
  for (int i = 0; i < CE; ++i) f[i] = col + i < limit ? RowVec<DT>::load_one(row, col + i) : 0.0f;
  return RowVec<DT>::pack(f);
}
template <int DT>
__device__ __forceinline__ void settle_chunk(u32x4_t& v, int col, int limit, bool live) {
  if (!live || col >= limit) v = u32x4_t{0u, 0u, 0u, 0u};
  else if (limit >= RowVec<DT>::N) RowVec<DT>::settle(v, col, limit);
}

template <int DT, Product P, class S, bool DIRECT, bool GATED>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_EU) void expert_gemm_kernel(
    const ExpertGemmArgs p) {
  constexpr int ES = dtype_size(DT), CE = 16 / ES, BK = kRowB / ES;
  constexpr bool AR = P == kGradW, BR = P != kOut;
  constexpr int BM = S::BM, BN = S::BN, TM = S::TM, TN = S::TN;
  constexpr int WNC = TN * 16, OUTC = GATED ? BN / 2 : BN;     // result columns of a block
  constexpr int PITCH = WNC + 4;                               // floats of an epilogue row
  constexpr int EPI = S::NW * 16 * PITCH * 4;
  // Stages of the ring with LIVE of the TM tiles of rows.  What a tile of few rows
  // leaves free of LDS holds more of them, two to four: its few MFMAs do not cover
  // the loads' latency.  Operands in registers on their way (not DIRECT) take two.
  constexpr bool TRIM = !AR;
  constexpr int HALF = TM >= 4 ? TM / 2 : TM, QUARTER = TM >= 8 ? TM / 4 : HALF;
  constexpr auto slot_bytes = [](int live) {
    return ((TRIM ? BM * live / TM : BM) + BN) * kRowB;
  };
  constexpr auto depth = [=](int live) {
    const int fit = 160 * 1024 / S::PER_CU / slot_bytes(live);
    return !DIRECT || fit < 2 ? 2 : fit > 4 ? 4 : fit;
  };
  constexpr auto most = [](int x, int y) { return x > y ? x : y; };
  constexpr int LDS = most(most(EPI, depth(TM) * slot_bytes(TM)),
                           most(depth(HALF) * slot_bytes(HALF),
                                depth(QUARTER) * slot_bytes(QUARTER)));
  static_assert(LDS <= 160 * 1024, "LDS of a CU");
  __shared__ __align__(1024) uint8_t lds[LDS];
  typedef Slots<DT, AR, BM, S::THREADS> SA;
  typedef Slots<DT, BR, BN, S::THREADS> SB;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int ncols = P == kOut ? p.N : p.K;
  const int nts = (ncols + OUTC - 1) / OUTC;

  // this block's tile: result rows [m0, m0 + mrows) of the operand's, columns from n0
  int e, L, mrows;
  int64_t row0;                 // first result row in out (and of x or d where they are rows)
  int n0;
  const uint8_t *a, *b;         // the operands' first elements of the tile
  int a_pitch, b_pitch;         // bytes
  int64_t a_step, b_step;       // bytes per BK of the reduction
  if constexpr (P == kGradW) {
    const int mts = (p.wide + BM - 1) / BM;
    const ExpertTile w = expert_tile_of_block(block_index(), (int64_t)mts * nts, p.E);
    if (w.e < 0) return;
    e = w.e;
    const TileAt at = tile_at(w.t, mts, nts);
    const ExpertRange r = expert_range(p.offsets, p.R, e);
    L = r.n;
    n0 = at.n * OUTC;
    row0 = at.m * BM;
    mrows = min(BM, p.wide - at.m * BM);
    a_pitch = p.wide * ES;
    b_pitch = p.K * ES;
    a = p.a + (int64_t)r.r0 * a_pitch + row0 * ES;
    b = p.b + (int64_t)r.r0 * b_pitch + (int64_t)n0 * ES;
    a_step = (int64_t)BK * a_pitch;
    b_step = (int64_t)BK * b_pitch;
  } else {
    const RowTile t = find_row_tile<BM>(p.offsets, p.R, p.E, nts, block_index());
    if (!t.live) return;
    e = t.e;
    n0 = t.nt * OUTC;
    row0 = (int64_t)t.r0 + t.m * BM;
    mrows = min(BM, t.n - t.m * BM);
    L = P == kOut ? p.K : p.wide;
    a_pitch = L * ES;
    b_pitch = p.K * ES;
    a = p.a + row0 * a_pitch;
    b = p.b + (int64_t)e * p.wide * b_pitch +
        (P == kOut ? (int64_t)n0 * b_pitch : (int64_t)n0 * ES);
    a_step = kRowB;
    b_step = P == kOut ? kRowB : (int64_t)BK * b_pitch;
  }
  // tile row j of W in out: its distance from the first one, or -1
  auto weight_row = [&](int j) {
    if (!GATED) return n0 + j < p.N ? j : -1;
    const int w = j / WNC, q = j % WNC, c = w * (WNC / 2) + q % (WNC / 2);
    return n0 + c < p.N ? (q < WNC / 2 ? c : p.N + c) : -1;
  };
  int steps = (L + BK - 1) / BK;
  if (P != kOut && p.split > 1) {              // this block's part of the reduction
    const int s = blockIdx.z, t0 = (int)((int64_t)steps * s / p.split);
    const int t1 = (int)((int64_t)steps * (s + 1) / p.split);
    a += t0 * a_step;
    b += t0 * b_step;
    L = min(L, t1 * BK) - t0 * BK;
    steps = t1 - t0;
  }

  uint32_t a_off[SA::COUNT], b_off[SB::COUNT];    // DIRECT: from the step's first element
  if constexpr (DIRECT) {
#pragma unroll
    for (int i = 0; i < SA::COUNT; ++i) {
      const int r = SA::row(i), c = SA::chunk(i);
      const bool in = AR ? c * CE < mrows : r < mrows;
      a_off[i] = in ? (uint32_t)r * a_pitch + c * 16 : kOutOfRange;
    }
#pragma unroll
    for (int i = 0; i < SB::COUNT; ++i) {
      const int r = SB::row(i), c = SB::chunk(i);
      if (BR) {
        b_off[i] = n0 + c * CE < ncols ? (uint32_t)r * b_pitch + c * 16 : kOutOfRange;
      } else {
        const int w = weight_row(r);
        b_off[i] = w >= 0 ? (uint32_t)w * b_pitch + c * 16 : kOutOfRange;
      }
    }
  }
  u32x4_t a_reg[DIRECT ? 1 : SA::COUNT], b_reg[DIRECT ? 1 : SB::COUNT];
  const uint32_t lds0 = lds_addr(lds);

  // step t's tiles on their way: into LDS (behind the last step zeros from nowhere, so
  // that as many loads are in flight as ever), or into registers
  auto fetch = [&](auto live, int t, int slot) {
    constexpr int LIVE = decltype(live)::value;
    constexpr int AROWS = TRIM ? BM * LIVE / TM : BM, AC = AROWS * SA::COUNT / BM;
    const uint8_t* at = a + t * a_step;
    const uint8_t* bt = b + t * b_step;
    const int left = L - t * BK;
    if constexpr (DIRECT) {
      const v4i ra = buffer_rsrc(at, kOutOfRange), rb = buffer_rsrc(bt, kOutOfRange);
      const uint32_t to = lds0 + slot * slot_bytes(LIVE) + wave * 1024;
#pragma unroll
      for (int i = 0; i < AC; ++i) {
        const int k = AR ? SA::row(i) : SA::chunk(i) * CE;
        dma16(ra, to + i * S::THREADS * 16, k < left ? a_off[i] : kOutOfRange);
      }
#pragma unroll
      for (int i = 0; i < SB::COUNT; ++i) {
        const int k = BR ? SB::row(i) : SB::chunk(i) * CE;
        dma16(rb, to + AROWS * kRowB + i * S::THREADS * 16, k < left ? b_off[i] : kOutOfRange);
      }
    } else {
      if (left <= 0) return;
      // rows that are not there load the first one's, which is, and are dropped
#pragma unroll
      for (int i = 0; i < AC; ++i) {
        const int r = SA::row(i), c = SA::chunk(i) * CE;
        a_reg[i] = load_chunk<DT>(at + (int64_t)(r < (AR ? left : mrows) ? r : 0) * a_pitch, c,
                                  AR ? mrows : left);
      }
#pragma unroll
      for (int i = 0; i < SB::COUNT; ++i) {
        const int r = SB::row(i), c = SB::chunk(i) * CE;
        const int w = BR ? (r < left ? r : 0) : max(weight_row(r), 0);
        b_reg[i] = load_chunk<DT>(bt + (int64_t)w * b_pitch, c, BR ? ncols - n0 : left);
      }
    }
  };
  auto settle = [&](auto live, int t) {
    if constexpr (!DIRECT) {
      constexpr int LIVE = decltype(live)::value;
      constexpr int AROWS = TRIM ? BM * LIVE / TM : BM, AC = AROWS * SA::COUNT / BM;
      const int left = L - t * BK;
      uint8_t* to = lds + (t & 1) * slot_bytes(LIVE) + threadIdx.x * 16;
#pragma unroll
      for (int i = 0; i < AC; ++i) {
        const int r = SA::row(i), c = SA::chunk(i) * CE;
        settle_chunk<DT>(a_reg[i], c, AR ? mrows : left, r < (AR ? left : mrows));
        *reinterpret_cast<u32x4_t*>(to + i * S::THREADS * 16) = a_reg[i];
      }
#pragma unroll
      for (int i = 0; i < SB::COUNT; ++i) {
        const int r = SB::row(i), c = SB::chunk(i) * CE;
        settle_chunk<DT>(b_reg[i], c, BR ? ncols - n0 : left,
                         BR ? r < left : weight_row(r) >= 0);
        *reinterpret_cast<u32x4_t*>(to + AROWS * kRowB + i * S::THREADS * 16) = b_reg[i];
      }
    }
  };

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // fp32: the products' sums are added up every 8 steps (256 terms), so that a long
  // reduction's error grows with the root of its 256ths: 8192 terms, 2e-6 of the
  // result in one chain.  The 16-bit types' rounding hides a chain's 2^-24 per term.
  constexpr bool BLOCKED = DT == kF32;
  v4f total[BLOCKED ? TM : 1][BLOCKED ? TN : 1];
  if constexpr (BLOCKED) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) total[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  auto add_up = [&](auto live) {
    if constexpr (BLOCKED) {
#pragma unroll
      for (int i = 0; i < decltype(live)::value; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          total[i][j] += acc[i][j];
          acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
  };

  // One barrier per step: behind it this step's tiles are in LDS and the slot read in
  // the step before is free.  The wave rows take 16 rows in turn, so that a tile of
  // few rows is few MFMAs for both: LIVE of the TM.
  auto loop = [&](auto live) {
    constexpr int LIVE = decltype(live)::value, D = depth(LIVE);
    constexpr int AROWS = TRIM ? BM * LIVE / TM : BM;
    constexpr int LOADS = AROWS * SA::COUNT / BM + SB::COUNT;
    if (steps > 0) {
#pragma unroll
      for (int d = 0; d < D - 1; ++d) fetch(live, d, d);
    }
    int slot = 0, next = D - 1;
    for (int t = 0; t < steps; ++t) {
      settle(live, t);
      wait_then_barrier<DIRECT ? (D - 2) * LOADS : 0>();
      fetch(live, t + D - 1, next);
      const uint8_t* ta = lds + slot * slot_bytes(LIVE);
      const uint8_t* tb = ta + AROWS * kRowB;
      slot = slot + 1 == D ? 0 : slot + 1;
      next = next + 1 == D ? 0 : next + 1;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4_t fa[LIVE], fb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j)
          fb[j] = fragment<DT, BR, BN>(tb, wn * WNC + 16 * j, s, lane);
#pragma unroll
        for (int i = 0; i < LIVE; ++i)
          fa[i] = fragment<DT, AR, BM>(ta, (i * S::WM + wm) * 16, s, lane);
#pragma unroll
        for (int i = 0; i < LIVE; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = mma<DT>(fb[j], fa[i], acc[i][j]);
      }
      if (BLOCKED && (t & 7) == 7) add_up(live);
    }
    add_up(live);
    if (DIRECT) wait_loads<0>();              // the zeros behind the last step
  };
  if (QUARTER < HALF && mrows <= BM / 4) loop(std::integral_constant<int, QUARTER>());
  else if (HALF < TM && mrows <= BM / 2) loop(std::integral_constant<int, HALF>());
  else loop(std::integral_constant<int, TM>());

  // 16 rows at a time through the wave's own LDS, so that a lane stores 8
  // consecutive columns and the activation's code is there once.
  __syncthreads();
  float* mine = reinterpret_cast<float*>(lds) + wave * 16 * PITCH;
  const int64_t out_pitch = (int64_t)ncols * ES;
  uint8_t* out = p.out + row0 * out_pitch;
  if (P == kGradW) out += (int64_t)e * p.wide * out_pitch;
  auto store8 = [&](uint8_t* row, int col, int limit, const float (&f)[8]) {
#pragma unroll
    for (int c = 0; c < 8; c += CE)
      if (col + c < limit)
        RowVec<DT>::template store<false>(row, col + c, limit, RowVec<DT>::pack(f + c));
  };
  for (int i = 0; i < TM; ++i) {
    const int first = (i * S::WM + wm) * 16;
    if (first >= mrows) break;
    wave_lds_order();
    with_constant<TM - 1>(i, [&](auto at) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *reinterpret_cast<v4f*>(mine + (lane & 15) * PITCH + 16 * j + (lane >> 4) * 4) =
            BLOCKED ? total[BLOCKED ? decltype(at)::value : 0][BLOCKED ? j : 0]
                    : acc[decltype(at)::value][j];
    });
    wave_lds_order();
    constexpr int LANES = WNC / (GATED ? 2 : 1) / 8;      // that share a row
    for (int at = lane; at < 16 * LANES; at += 64) {
      const int r = at / LANES, q = (at % LANES) * 8;
      if (first + r >= mrows) continue;
      float g[8], u[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        g[c] = mine[r * PITCH + q + c];
        u[c] = GATED ? mine[r * PITCH + WNC / 2 + q + c] : 0.0f;
      }
      const int col = n0 + wn * (WNC / (GATED ? 2 : 1)) + q;
      if (P == kOut && p.pre != nullptr) {
        uint8_t* row = p.pre + (row0 + first + r) * (int64_t)p.wide * ES;
        store8(row, col, p.N, g);
        if (GATED) store8(row + (int64_t)p.N * ES, col, p.N, u);
      }
      if (P == kOut && p.act != kActNone) {
#pragma unroll
        for (int c = 0; c < 8; ++c) g[c] = expert_act(p.act, g[c], u[c], p.limit);
      }
      if (P != kOut && p.split > 1) {          // a part's sums, unrounded
        float* part = p.part + (int64_t)blockIdx.z * p.part_size +
                      (P == kGradW ? (int64_t)e * p.wide : 0) * ncols +
                      (row0 + first + r) * ncols;
#pragma unroll
        for (int c = 0; c < 8; c += 4)
          if (col + c < ncols)
            RowVec<kF32>::template store<false>(reinterpret_cast<uint8_t*>(part), col + c, ncols,
                                                RowVec<kF32>::pack(g + c));
        continue;
      }
      store8(out + (first + r) * out_pitch, col, ncols, g);
    }
  }
}

// d = F'(pre) grad_out for the rows of all experts; bound by HBM.  Rounded to the rows'
// type, which is what the products' MFMAs take: half a step more than the result's own
// rounding (0.0023 of a bf16 gradient for 0.0017, and fp16's range), where a second part
// of d would double their number.
constexpr int kActThreads = 256;

template <class RV>
__global__ __launch_bounds__(kActThreads) void act_grad_kernel(const ExpertActGradArgs p) {
  constexpr int N = RV::N;
  const int per = (p.N + N - 1) / N;
  const int64_t at = (int64_t)block_index() * kActThreads + threadIdx.x;
  const int64_t row = at / per;
  const int rows = p.offsets == nullptr ? p.R : min(max(p.offsets[p.E], 0), p.R);
  if (row >= rows) return;
  const int col = (int)(at - row * per) * N;
  const int wide = p.N * act_width(p.act);
  const uint8_t* pre = p.pre + row * wide * RV::kSize;
  uint8_t* d = p.d + row * wide * RV::kSize;
  const bool gated = act_width(p.act) == 2;
  typename RV::Raw gv = RV::template load<true>(pre, col, p.N), uv = {};
  if (gated) uv = RV::template load<true>(pre + (int64_t)p.N * RV::kSize, col, p.N);
  typename RV::Raw hv = RV::template load<true>(p.grad_out + row * p.N * RV::kSize, col, p.N);
  RV::settle(gv, col, p.N);
  RV::settle(uv, col, p.N);
  RV::settle(hv, col, p.N);
  float g[N], u[N], h[N];
  RV::unpack(gv, g);
  RV::unpack(uv, u);
  RV::unpack(hv, h);
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const ActGrad r = act_grad(p.act, g[c], u[c], p.limit, h[c]);
    g[c] = r.gate;
    u[c] = r.up;
  }
  RV::template store<false>(d, col, p.N, RV::pack(g));
  if (gated) RV::template store<false>(d + (int64_t)p.N * RV::kSize, col, p.N, RV::pack(u));
}

// The parts' sums in their order, rounded once; rows: those that are there.
template <int DT>
__global__ __launch_bounds__(kActThreads) void add_parts_kernel(const ExpertGemmArgs p,
                                                                bool by_rows) {
  const int64_t at = (int64_t)block_index() * kActThreads + threadIdx.x;
  const int rows = p.offsets == nullptr ? p.R : min(max(p.offsets[p.E], 0), p.R);
  if (at >= (by_rows ? (int64_t)rows * p.K : p.part_size)) return;
  float f = 0.0f;
  for (int s = 0; s < p.split; ++s) f += p.part[s * p.part_size + at];
  RowVec<DT>::store_one(p.out, at, f);
}

typedef Tile<64, 128, 1, 4, 2> Tile64;
typedef Tile<128, 128, 2, 2, 2> Tile128;
typedef Tile<256, 256, 2, 4, 1> Tile256;

// Tiles of the result, at most (the rows of an expert are on the device).
template <class S, Product P, bool GATED>
int64_t most_tiles(const ExpertGemmArgs& a) {
  constexpr int OUTC = GATED ? S::BN / 2 : S::BN;
  const int64_t nts = ((P == kOut ? a.N : a.K) + OUTC - 1) / OUTC;
  return nts * (P == kGradW ? (int64_t)((a.wide + S::BM - 1) / S::BM) * a.E
                            : most_row_tiles<S::BM>(a.offsets, a.R, a.E));
}

template <int DT, Product P, class S, bool GATED>
hipError_t launch_shape(const ExpertGemmArgs& a, bool direct, hipStream_t stream) {
  const int64_t tiles = most_tiles<S, P, GATED>(a), per = P == kGradW ? tiles / a.E : tiles;
  dim3 grid = grid_of(blocks_of_tiles(per) * (P == kGradW ? a.E : 1));
  if (P != kOut) grid.z = a.split;
  if (direct)
    expert_gemm_kernel<DT, P, S, true, GATED><<<grid, S::THREADS, 0, stream>>>(a);
  else
    expert_gemm_kernel<DT, P, S, false, GATED><<<grid, S::THREADS, 0, stream>>>(a);
  return hipGetLastError();
}

// 256 x 256 with a tile for every CU and, of rows, 64 of an expert on average (1024 where
// operands pass through registers: half a tile of the larger ones is then dear); 64 rows
// where that makes no more than two tiles per CU; 128 x 128 else.  bf16, out, us in 64 /
// 128 / 256: 512 x 7168 by 2 x 2048 51 / 76 / 168; 16 experts of 62 rows, 4096 by 2 x
// 2048 146 / 125 / 148, of 125 178 / 187 / 137; 60 of 133, 2048 by 2 x 1408 239 / 231 /
// 200; 32 of 512, 4096 by 2 x 2048 - / 731 / 703, of 1024, 7168 - / 2283 / 1963.
// Unaligned, in 128 / 256: 60 experts of 136 rows, 1001 by 2047 133 / 166, their weights'
// gradient 146 / 132; 2049 by 2047, 32 of 256 rows 238 / 224, 16 of 512 183 / 196, of 1024
// 303 / 294; 8 of 4096, 4097 by 2047 1160 / 1023.
template <int DT, Product P, bool GATED>
hipError_t launch_gemm(const ExpertGemmArgs& a, bool direct, hipStream_t stream) {
  if constexpr (P != kOut) {
    if (a.split > 1) {
      const hipError_t err = launch_shape<DT, P, Tile128, GATED>(a, direct, stream);
      if (err != hipSuccess) return err;
      add_parts_kernel<DT><<<grid_of((a.part_size + kActThreads - 1) / kActThreads), kActThreads,
                             0, stream>>>(a, P == kGradX);
      return hipGetLastError();
    }
  }
  if constexpr (DT != kF32) {
    if (most_tiles<Tile256, P, GATED>(a) >= kCus &&
        (P == kGradW || a.R >= (direct ? 64 : 1024) * (int64_t)a.E))
      return launch_shape<DT, P, Tile256, GATED>(a, direct, stream);
  }
  if constexpr (P != kGradW) {
    if (most_tiles<Tile64, P, GATED>(a) <= 2 * kCus)
      return launch_shape<DT, P, Tile64, GATED>(a, direct, stream);
  }
  return launch_shape<DT, P, Tile128, GATED>(a, direct, stream);
}

template <class F>
hipError_t with_dtype(int dtype, F&& f) {
  switch (dtype) {
    case kBf16: return f(std::integral_constant<int, kBf16>());
    case kF16: return f(std::integral_constant<int, kF16>());
    default: return f(std::integral_constant<int, kF32>());
  }
}

// Whether launch_expert_few is the faster one: up to 8 rows of an expert on average
// where the reduction is long enough for its eight waves, or up to 128 of tiles that
// would leave CUs idle.  us, few / tiles: 256 rows of 64 experts, 4096 by 2 x 1024 179 /
// 198, 2048 by 4096 212 / 196; 16 of 8, 4096 by 2 x 2048 44 / 69; 100 x 7168 by 2 x 2048
// 25 / 47, 256 48 / 48; 64 of 256, 2048 by 2 x 512 56 / 47.
bool few_rows(const ExpertGemmArgs& a) {
  const int64_t per = ((int64_t)a.R + a.E - 1) / a.E;
  const int64_t tiles = act_width(a.act) == 2 ? most_tiles<Tile64, kOut, true>(a)
                                              : most_tiles<Tile64, kOut, false>(a);
  return (per <= 8 && a.K >= 4096) || (tiles <= kCus && tiles * per <= 8192);
}

bool aligned16(const void* p, int64_t pitch) { return (((uintptr_t)p | pitch) & 15) == 0; }

}  // namespace

// A gradient whose tiles of 128 x 128 leave half of the CUs or more without one is split
// along its reduction (grad_x: the weights' rows; grad_weight: an expert's rows, of
// which the host knows the average), 8 steps or more to a part, at most two tiles per CU:
// under 512 parts of tiles of 64 KB.  From 48 steps on, as the second launch costs 6 us.
// bf16 and fp16, us whole / split: grad_x of 2 x 98, 2 x 5747 rows of weights 177 / 22, of
// 100 x 1024, 8192 50 / 19, of 1000 rows of 2 experts, 2 x 1024 (32 steps) 25 / 29;
// grad_weight of 8191 rows, 1001 by 2047 200 / 80, of 4000, 2 x 1024 by 1024 52 / 44.
int expert_split(const ExpertGemmArgs& a, int dtype, bool grad_w) {
  const auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const int bk = kRowB / dtype_size(dtype);
  const int64_t nts = up(a.K, 128);
  const int64_t tiles = grad_w ? nts * up(a.wide, 128) * a.E
                               : nts * (a.R / 128 + std::min(a.R, a.E));
  const int64_t steps = up(grad_w ? up(a.R, a.E) : a.wide, bk);
  if (tiles == 0 || tiles > kCus / 2 || steps < 48) return 1;
  return (int)std::max<int64_t>(1, std::min(2 * kCus / tiles, steps / 8));
}

hipError_t launch_expert_out(const ExpertGemmArgs& a, int dtype, hipStream_t stream) {
  const int64_t pitch = (int64_t)a.K * dtype_size(dtype);
  const bool direct = aligned16(a.a, pitch) && aligned16(a.b, pitch);
  if (direct && dtype != kF32 && few_rows(a))
    return launch_expert_few(a, dtype, stream);
  return with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return act_width(a.act) == 2 ? launch_gemm<DT, kOut, true>(a, direct, stream)
                                 : launch_gemm<DT, kOut, false>(a, direct, stream);
  });
}

hipError_t launch_expert_grad_x(const ExpertGemmArgs& a, int dtype, hipStream_t stream) {
  const bool direct = aligned16(a.a, (int64_t)a.wide * dtype_size(dtype)) &&
                      aligned16(a.b, (int64_t)a.K * dtype_size(dtype));
  return with_dtype(dtype, [&](auto dt) {
    return launch_gemm<decltype(dt)::value, kGradX, false>(a, direct, stream);
  });
}

hipError_t launch_expert_grad_w(const ExpertGemmArgs& a, int dtype, hipStream_t stream) {
  const bool direct = aligned16(a.a, (int64_t)a.wide * dtype_size(dtype)) &&
                      aligned16(a.b, (int64_t)a.K * dtype_size(dtype));
  return with_dtype(dtype, [&](auto dt) {
    return launch_gemm<decltype(dt)::value, kGradW, false>(a, direct, stream);
  });
}

hipError_t launch_expert_act_grad(const ExpertActGradArgs& a, int dtype, hipStream_t stream) {
  return with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    auto go = [&](auto rv) {
      typedef decltype(rv) RV;
      const int64_t lanes = (int64_t)a.R * ((a.N + RV::N - 1) / RV::N);
      act_grad_kernel<RV><<<grid_of((lanes + kActThreads - 1) / kActThreads), kActThreads, 0,
                            stream>>>(a);
      return hipGetLastError();
    };
    return a.N < RowVec<DT>::N ? go(RowOne<DT>()) : go(RowVec<DT>());
  });
}

}  // namespace moe
