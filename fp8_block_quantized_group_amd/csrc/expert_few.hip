// Rows sorted by expert times the experts' 16-bit weights where an expert has few
// rows: bound by the weights' bytes, which are read once per 16 (or 32) rows.
//
// A block makes 16 MT rows of 16 (or 8, or 32) result columns; its W waves share the
// columns of the reduction, every W-th run of 64 each, and add their sums up in
// LDS.  What a wave multiplies it loads itself, into a ring of stages of its own
// in LDS: 128 bytes, a whole line, of each of its weight rows and of x's, by loads
// whose neighbouring lanes are neighbours in memory (an MFMA operand's are not, and
// 64 accesses of 16 bytes are what such a load then takes).  No barrier is needed
// until the end.  x is the MFMA's A operand, the weights its B operand.
//
// 256 rows of 64 experts, 4096 by 2 x 1024, bf16 with silu: 166-172 us, 6.3-6.5 TB/s;
// one row x 7168 by 2 x 2048 10.9 us, 59 MB at 5.4 TB/s (62 with the tiles of batches).
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

constexpr uint32_t kOutOfRange = 0xF0000000u;    // past every buffer: reads as zeros
constexpr int kRun = 64;                         // columns of a stage: 128 bytes of a row
constexpr int kWaves = 8;
constexpr int kStrip = 16 * kRun * 2;            // bytes of 16 rows of a stage

template <int DT>
__device__ __forceinline__ v4f mma(u32x4_t a, u32x4_t b, v4f c) {
  if constexpr (DT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Strips of 16 weight rows.  Gated: one strip of gate and one of up rows (NT 2), or
// 8 of each in one (NT 1), which makes twice the blocks.
template <int DT, bool GATED, int MT, int NT>
__global__ __launch_bounds__(64 * kWaves) void expert_few_kernel(const ExpertGemmArgs p) {
  constexpr int BM = 16 * MT, OUTC = GATED ? NT * 8 : NT * 16;
  constexpr int STAGE = (NT + MT) * kStrip, LOADS = (NT + MT) * 2;
  constexpr int FIT = 160 * 1024 / (kWaves * STAGE), D = FIT > 4 ? 4 : FIT;
  static_assert(D >= 2 && NT * MT * 1024 <= D * STAGE, "LDS");
  __shared__ __align__(1024) uint8_t ring[kWaves * D * STAGE];

  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const RowTile t = find_row_tile<BM>(p.offsets, p.R, p.E, (p.N + OUTC - 1) / OUTC,
                                      block_index());
  if (!t.live) return;
  const int n0 = t.nt * OUTC, rows = min(BM, t.n - t.m * BM);
  const int64_t row0 = (int64_t)t.r0 + t.m * BM;
  const int K = p.K, pitch = K * 2, runs = (K + kRun - 1) / kRun;
  const bool stream = t.n <= BM;                 // no other block reads these weights
  uint8_t* my = ring + wave * D * STAGE;
  const uint32_t my_lds = lds_addr(my);

  // A load takes 8 rows of 128 bytes: lane l row l / 8, its chunk at position l % 8
  // being l % 8 ^ l / 8 (fragment reads then hit all banks; the key of row r is r & 7).
  const int lr = lane >> 3, chunk = (lane & 7) ^ lr;
  const v4i rw = buffer_rsrc(p.b + (int64_t)t.e * p.wide * pitch, kOutOfRange);
  const v4i rx = buffer_rsrc(p.a + row0 * pitch, kOutOfRange);
  uint32_t w_off[NT][2], x_off[MT][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * h + lr;                  // of the strip
      const int c = n0 + (GATED ? (NT == 2 ? r : lr) : 16 * n + r);
      const int row = c + (GATED && (NT == 2 ? n : h) ? p.N : 0);
      w_off[n][h] = c < p.N ? (uint32_t)row * pitch + chunk * 16 : kOutOfRange;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = 16 * m + 8 * h + lr;
      x_off[m][h] = r < rows ? (uint32_t)r * pitch + chunk * 16 : kOutOfRange;
    }
  }
  auto fetch = [&](int c, int slot) {
    const bool in = c * kRun + chunk * 8 < K;    // behind the last run: zeros from nowhere
    const uint32_t to = my_lds + slot * STAGE;
    auto at = [&](uint32_t off) {
      return in && off != kOutOfRange ? off + c * (kRun * 2) : kOutOfRange;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lds = to + n * kStrip + h * 1024;
        if (stream) dma16_nt(rw, lds, at(w_off[n][h]));
        else dma16(rw, lds, at(w_off[n][h]));
      }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        dma16(rx, to + (NT + m) * kStrip + h * 1024, at(x_off[m][h]));
  };
  v4f acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (wave < runs) {
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(wave + d * kWaves, d);
    int slot = 0, next = D - 1;
#pragma unroll 1
    for (int c = wave; c < runs; c += kWaves) {
      fetch(c + (D - 1) * kWaves, next);
      wait_loads<(D - 1) * LOADS>();
      const uint8_t* at = my + slot * STAGE;
      auto fragment = [&](int strip, int s) {
        return *reinterpret_cast<const u32x4_t*>(at + strip * kStrip + i16 * 128 +
                                                 (((4 * s + g) ^ (i16 & 7)) << 4));
      };
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4_t w[NT], x[MT];
#pragma unroll
        for (int n = 0; n < NT; ++n) w[n] = fragment(n, s);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = fragment(NT + m, s);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[n][m] = mma<DT>(x[m], w[n], acc[n][m]);
      }
      wait_lds();                                // before a load into what was read
      slot = slot + 1 == D ? 0 : slot + 1;
      next = next + 1 == D ? 0 : next + 1;
    }
  }
  wait_loads<0>();
  __syncthreads();
  // acc[n][m][i] of lane l: strip row l % 16, row 16m + 4 (l / 16) + i
  v4f* red = reinterpret_cast<v4f*>(ring);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[(wave * NT * MT + n * MT + m) * 64 + lane] = acc[n][m];
  __syncthreads();
  const float* flat = reinterpret_cast<const float*>(ring);
  for (int o = threadIdx.x; o < BM * OUTC; o += 64 * kWaves) {
    const int r = o / OUTC, c = o % OUTC;
    if (r >= rows || n0 + c >= p.N) continue;
    auto total = [&](int n, int c16) {
      const int at = (n * MT + r / 16) * 256 + ((r % 16 / 4) * 16 + c16) * 4 + r % 4;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += flat[w * NT * MT * 256 + at];
      return v;
    };
    const float a = GATED ? total(0, c) : total(c / 16, c % 16);
    const float u = GATED ? (NT == 2 ? total(NT - 1, c) : total(0, 8 + c)) : 0.0f;
    const int64_t row = row0 + r;
    if (p.pre != nullptr) {
      RowVec<DT>::store_one(p.pre, row * p.wide + n0 + c, a);
      if (GATED) RowVec<DT>::store_one(p.pre, row * p.wide + p.N + n0 + c, u);
    }
    const float f = p.act == kActNone ? a : expert_act(p.act, a, u, p.limit);
    RowVec<DT>::store_one(p.out, row * p.N + n0 + c, f);
  }
}

template <int DT, bool GATED, int MT, int NT>
hipError_t launch_strips(const ExpertGemmArgs& a, hipStream_t stream) {
  constexpr int OUTC = GATED ? NT * 8 : NT * 16;
  const int64_t tiles =
      most_row_tiles<16 * MT>(a.offsets, a.R, a.E) * ((a.N + OUTC - 1) / OUTC);
  expert_few_kernel<DT, GATED, MT, NT>
      <<<grid_of(blocks_of_tiles(tiles)), 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

template <int DT, bool GATED, int MT>
hipError_t launch_few(const ExpertGemmArgs& a, hipStream_t stream) {
  // one strip per block where two would leave CUs without a block
  const int64_t two = most_row_tiles<16 * MT>(a.offsets, a.R, a.E) *
                      ((a.N + (GATED ? 15 : 31)) / (GATED ? 16 : 32));
  return two < 256 ? launch_strips<DT, GATED, MT, 1>(a, stream)
                   : launch_strips<DT, GATED, MT, 2>(a, stream);
}

template <int DT, bool GATED>
hipError_t launch_rows(const ExpertGemmArgs& a, hipStream_t stream) {
  return a.R <= 16 * (int64_t)a.E ? launch_few<DT, GATED, 1>(a, stream)
                                  : launch_few<DT, GATED, 2>(a, stream);
}

}  // namespace

hipError_t launch_expert_few(const ExpertGemmArgs& a, int dtype, hipStream_t stream) {
  const bool gated = act_width(a.act) == 2;
  if (dtype == kBf16)
    return gated ? launch_rows<kBf16, true>(a, stream) : launch_rows<kBf16, false>(a, stream);
  return gated ? launch_rows<kF16, true>(a, stream) : launch_rows<kF16, false>(a, stream);
}

}  // namespace moe
