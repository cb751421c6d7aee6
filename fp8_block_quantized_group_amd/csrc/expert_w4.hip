// Rows sorted by expert times 4-bit weights with group scales, for decode
// batches: a few rows per expert, bound by the weights' bytes.
//
//   out[r, n] = F(sum over groups b of s[e, n, b] *
//                 sum over k in b of x[r, k] * (q[e, n, k] - z[e, n, b]))
//
// A wave takes NT tiles of 16 weight rows and every W-th run of 128 columns;
// the block's W waves add their sums up in LDS.  A lane's 16 bytes of codes
// are 32 columns of one weight row: four MFMAs of 32 columns, whose B operand
// they are (a lane's accumulators then belong to one weight row and take one
// scale per group), the rows of x the A operand, straight from memory.  The
// codes of a group have to meet in one MFMA: with groups of 128 they do as they
// lie, groups of 64 and 32 swap registers between the lane quarters first.
//
// Codes become 16-bit floats without a conversion each: or-ed into the
// mantissa of 128 (bf16) or 1024 (fp16) they are 128 + q and 1024 + q, two at a
// time, in the order 0 4 1 5 2 6 3 7, which x is brought into.  fp16 subtracts
// 1024 + z exactly; bf16 has no packed subtraction, so the sum over the group
// is corrected: sum x (q - z) = sum x (128 + q) - (128 + z) sum x, the last
// sum by an MFMA with ones.  That adds 2^-24 * 136 of the sum of |x| per group,
// against the 2^-9 that leave with a bf16 result.  e2m1 codes have a conversion
// of their own.  fp32 rows are split into three bf16 parts, 24 bits, which is
// exact, as the products are; their codes are made bf16 numbers q - z.
//
// MOE_W4_DTYPE: the rows' type (one object per type).
#include "expert_act.h"
#include "expert_rows.h"
#include "kernels.h"
#include "row_vec.h"

#ifndef MOE_W4_DTYPE
#error "MOE_W4_DTYPE"
#endif

namespace moe {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;                // of a block, sharing the columns
constexpr int kRun = 128;                // columns of a lane quad's 64 bytes of codes

template <int DT>
__device__ __forceinline__ v4f mma(u32x4_t a, u32x4_t b, v4f c) {
  if constexpr (DT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// 2^(e - 127); 255 is NaN
__device__ __forceinline__ float e8m0(uint32_t e) {
  return e == 255u ? __builtin_nanf("") : __builtin_ldexpf(1.0f, (int)e - 127);
}

// The codes' dwords so that MFMA j takes one group only (GROUP 32, 64), and
// the first of the 8 columns that lane quarter g has in it.
template <int GROUP>
__device__ __forceinline__ void gather_groups(u32x4_t& w) {
  if constexpr (GROUP < 128) {
    auto swap32 = [](uint32_t a, uint32_t b) {
      return __builtin_amdgcn_permlane32_swap(a, b, false, false);
    };
    const auto p = swap32(w[0], w[2]), q = swap32(w[1], w[3]);
    w = u32x4_t{p[0], q[0], p[1], q[1]};
  }
  if constexpr (GROUP < 64) {
    const auto p = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
    w = u32x4_t{p[0], p[1], q[0], q[1]};
  }
}
template <int GROUP>
__device__ __forceinline__ int column_of(int j, int g) {
  if (GROUP == 128) return 32 * g + 8 * j;
  if (GROUP == 64) return 32 * ((j & 2) | (g & 1)) + 8 * ((j & 1) | (g & 2));
  return 32 * j + 8 * g;
}

// 8 codes as the B operand of one MFMA.  z: the zero point, in the form that
// the type wants (fp16: 1024 + z twice; fp32 rows: z).
template <int DT, bool MX>
__device__ __forceinline__ u32x4_t codes_as_values(uint32_t w, uint32_t z16, float z) {
  u32x4_t v;
  if constexpr (MX) {
    auto pair = [&](auto b) {
      if constexpr (DT == kF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(
                                                w, 1.0f, decltype(b)::value));
      else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                                                w, 1.0f, decltype(b)::value));
    };
    v[0] = pair(std::integral_constant<int, 0>());
    v[1] = pair(std::integral_constant<int, 1>());
    v[2] = pair(std::integral_constant<int, 2>());
    v[3] = pair(std::integral_constant<int, 3>());
  } else if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pack_bf16x2((float)((w >> (8 * i)) & 15) - z, (float)((w >> (8 * i + 4)) & 15) - z);
  } else {
    const uint32_t one = DT == kF16 ? 0x64006400u : 0x43004300u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t q = ((w >> (4 * i)) & 0x000F000Fu) | one;
      v[i] = DT == kF16 ? __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, q) -
                                                           __builtin_bit_cast(v2h, z16))
                        : q;
    }
  }
  return v;
}

// x's 8 columns in the order of the codes' pairs
__device__ __forceinline__ u32x4_t paired(u32x4_t x) {
  u32x4_t v;
  v[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
  v[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
  v[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
  v[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
  return v;
}

// fp32 as three bf16 parts that add up to it, each truncated; what is not
// finite is its own first part.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
  const bool fine = fabsf(x) < __builtin_inff();
  p[0] = fine ? __uint_as_float(__float_as_uint(x) & 0xFFFF0000u) : x;
  const float rest = fine ? x - p[0] : 0.0f;
  p[1] = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u);
  p[2] = rest - p[1];
}

template <int DT, bool MX, int GROUP, bool S32, int MT, int NT>
__global__ __launch_bounds__(64 * kWaves) void expert_w4_kernel(const ExpertW4Args p) {
  constexpr int ES = dtype_size(DT), XR = DT == kF32 ? 2 : 1;  // 16-byte loads of 8 columns
  constexpr int PARTS = DT == kF32 ? 3 : 1;
  constexpr int GR = kRun / GROUP;                             // groups of a run
  constexpr bool SUMS = DT == kBf16 && !MX;                    // corrected by sum x
  constexpr int BM = 16 * MT;
  __shared__ __align__(16) v4f red[kWaves][NT * MT][64];

  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const bool gated = p.wide != p.N;
  const int outc = gated ? NT * 8 : NT * 16;                   // result columns of a block
  const RowTile t = find_row_tile<BM>(p.offsets, p.R, p.E, (p.N + outc - 1) / outc,
                                      block_index());
  if (!t.live) return;
  const int n0 = t.nt * outc, rows = min(BM, t.n - t.m * BM);
  const int64_t row0 = (int64_t)t.r0 + t.m * BM;
  const int K = p.K, groups = K / GROUP;

  // this lane's weight rows (the last one for those past the end) and rows of x
  const uint8_t* wp[NT];
  int64_t sp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    int row = gated ? (n < NT / 2 ? 0 : p.N) + min(n0 + 16 * (n % (NT / 2 > 0 ? NT / 2 : 1)) + i16,
                                                   p.N - 1)
                    : min(n0 + 16 * n + i16, p.N - 1);
    const int64_t at = (int64_t)t.e * p.wide + row;
    wp[n] = p.codes + at * (K / 2);
    sp[n] = at * groups;
  }
  const uint8_t* xp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = p.x + (row0 + min(16 * m + i16, rows - 1)) * K * ES;

  v4f acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};

  const int runs = (K + kRun - 1) / kRun;
  for (int c = wave; c < runs; c += kWaves) {
    const int k0 = c * kRun;
    u32x4_t w[NT], x[MT][4][XR];
    float s[NT][GR], z[NT][GR];
    // past the row's end: its first codes, with x and the scales zero
    const int at = k0 + 32 * g < K ? (k0 + 32 * g) / 2 : 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      w[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(wp[n] + at));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int b = 0; b < GR; ++b) {
        const int gi = k0 / GROUP + b;
        const int64_t i = sp[n] + (gi < groups ? gi : 0);
        if constexpr (MX) {
          s[n][b] = e8m0(p.scales[i]);
        } else {
          s[n][b] = RowVec<S32 ? kF32 : DT>::load_one(p.scales, i);
          z[n][b] = p.zeros != nullptr ? (float)p.zeros[i] : 8.0f;
        }
        if (gi >= groups) s[n][b] = 0.0f;
      }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + column_of<GROUP>(j, g);
#pragma unroll
        for (int h = 0; h < XR; ++h) {
          const u32x4_t v = *reinterpret_cast<const u32x4_any*>(
              xp[m] + (int64_t)(k < K ? k : 0) * ES + 16 * h);
          x[m][j][h] = k < K ? v : u32x4_t{0u, 0u, 0u, 0u};
        }
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) gather_groups<GROUP>(w[n]);

    v4f sum[NT][MT], ssum[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = j * GR / 4;                                // the MFMA's group in the run
      const bool first = j % (4 / GR) == 0, last = (j + 1) % (4 / GR) == 0;
      u32x4_t xa[MT][PARTS];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (DT == kF32) {
          float f[8], q[8][3];
          RowVec<kF32>::unpack(x[m][j][0], f);
          RowVec<kF32>::unpack(x[m][j][1], f + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) split3(f[i], q[i]);
#pragma unroll
          for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) xa[m][h][i] = pack_bf16x2(q[2 * i][h], q[2 * i + 1][h]);
        } else {
          xa[m][0] = MX ? x[m][j][0] : paired(x[m][j][0]);
        }
        if (SUMS) ssum[m] = mma<DT>(xa[m][0], ones, first ? none : ssum[m]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t z16 = 0;
        if (DT == kF16 && !MX)
          z16 = 0x64006400u + (uint32_t)z[n][b] * 0x00010001u;
        const u32x4_t v = codes_as_values<DT, MX>(w[n][j], z16, MX ? 0.0f : z[n][b]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          v4f d = first ? none : sum[n][m];
#pragma unroll
          for (int h = 0; h < PARTS; ++h) d = mma<DT>(xa[m][h], v, d);
          sum[n][m] = d;
          if (last) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float f = SUMS ? fmaf(-128.0f - z[n][b], ssum[m][i], d[i]) : d[i];
              acc[n][m][i] = fmaf(s[n][b], f, acc[n][m][i]);
            }
          }
        }
      }
    }
  }

  // acc[n][m][i] of lane l: weight row 16n + l % 16, row 16m + 4 (l / 16) + i
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[wave][n * MT + m][lane] = acc[n][m];
  __syncthreads();
  const float* flat = reinterpret_cast<const float*>(red);
  constexpr int WAVE = NT * MT * 256;
  for (int o = threadIdx.x; o < BM * outc; o += 64 * kWaves) {
    const int r = o / outc, c = o % outc;
    if (r >= rows || n0 + c >= p.N) continue;
    auto total = [&](int n, int c16) {
      const int at = (n * MT + r / 16) * 256 + ((r % 16 / 4) * 16 + c16) * 4 + r % 4;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += flat[w * WAVE + at];
      return v;
    };
    const float a = total(c / 16, c % 16);
    const float u = gated ? total(NT / 2 + c / 16, c % 16) : 0.0f;
    const float f = p.act == kActNone ? a : apply_act(p.act, a, u, p.limit);
    RowVec<DT>::store_one(p.out, (row0 + r) * p.N + n0 + c, f);
  }
}

template <int DT, bool MX, int GROUP, bool S32, int MT, int NT>
hipError_t launch_tile(const ExpertW4Args& a, hipStream_t stream) {
  const int outc = a.wide != a.N ? NT * 8 : NT * 16;
  const int64_t tiles =
      most_row_tiles<16 * MT>(a.offsets, a.R, a.E) * ((a.N + outc - 1) / outc);
  expert_w4_kernel<DT, MX, GROUP, S32, MT, NT>
      <<<grid_of((tiles + 7) / 8 * 8), 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

// ---- few rows per expert -------------------------------------------------------
// Up to 16 rows of x stay in registers, a wave's RW runs of 128 columns each,
// while the block walks over tiles of weight rows: x is read once per block, and
// the next tile's codes and scales are on their way while this one is worked on.

// The raw codes, scales and zero points of one weight row's run.
template <int FMT, int GROUP, int SB>
struct RawRun {
  static constexpr int GR = kRun / GROUP;
  static constexpr int SW = GR * SB >= 4 ? GR * SB / 4 : 1;    // words of scales
  u32x4_t w;
  uint32_t s[SW], z;

  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales,
                                       const uint8_t* zeros) {
    w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(codes));
    typedef uint32_t __attribute__((aligned(1))) word;
    typedef uint16_t __attribute__((aligned(1))) half;
    if constexpr (GR * SB == 2) {
      s[0] = *reinterpret_cast<const half*>(scales);
    } else {
#pragma unroll
      for (int i = 0; i < SW; ++i) s[i] = reinterpret_cast<const word*>(scales)[i];
    }
    if constexpr (FMT == kW4Int4Zero)
      z = GR == 1   ? *zeros
          : GR == 2 ? *reinterpret_cast<const half*>(zeros)
                    : *reinterpret_cast<const word*>(zeros);
    else
      z = 0x08080808u;
  }
  template <int DT>
  __device__ __forceinline__ float scale(int b) const {
    if constexpr (FMT == kW4Mxfp4) return e8m0((s[0] >> (8 * b)) & 255u);
    else if constexpr (SB == 4) return __uint_as_float(s[b]);
    else if constexpr (DT == kBf16) return __uint_as_float((s[b / 2] >> (16 * (b & 1))) << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)(s[b / 2] >> (16 * (b & 1))));
  }
  __device__ __forceinline__ uint32_t zero(int b) const { return (z >> (8 * b)) & 255u; }
};

// waves of a SIMD: registers for four where they hold everything (two blocks per CU)
constexpr int few_waves(int fmt, int rw) { return rw <= 2 || (rw == 4 && fmt == kW4Mxfp4) ? 4 : 2; }

template <int DT, int FMT, int GROUP, bool S32, int RW, bool GATED>
__global__ __launch_bounds__(64 * kWaves, few_waves(FMT, RW)) void expert_w4_few_kernel(const ExpertW4Args p,
                                                                    int per_block) {
  constexpr bool MX = FMT == kW4Mxfp4;
  constexpr int GR = kRun / GROUP, SB = MX ? 1 : S32 ? 4 : 2;
  constexpr bool SUMS = DT == kBf16 && !MX;
  constexpr int NT = GATED ? 2 : 1;
  typedef RawRun<FMT, GROUP, SB> Raw;
  __shared__ __align__(16) v4f red[2][kWaves][NT][64];

  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int tiles = (p.N + 15) / 16;
  const RowTile t = find_row_tile<16>(p.offsets, p.R, p.E, (tiles + per_block - 1) / per_block,
                                      block_index());
  if (!t.live) return;
  const int rows = min(16, t.n - t.m * 16);
  const int64_t row0 = (int64_t)t.r0 + t.m * 16;
  const int K = p.K, groups = K / GROUP, runs = K / kRun;

  u32x4_t xa[RW][4];
  const uint8_t* xp = p.x + (row0 + min(i16, rows - 1)) * K * 2;
#pragma unroll
  for (int j = 0; j < RW; ++j) {
    const int c = wave * RW + j;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      xa[j][q] = *reinterpret_cast<const u32x4_any*>(
          xp + (int64_t)((c < runs ? c : 0) * kRun + column_of<GROUP>(q, g)) * 2);
  }
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};

  // 16 weight rows, of the gate's half or the up one's; runs that are not there
  // load the first one's, against zeros of x
  auto fetch = [&](int tile, int half, Raw (&r)[RW]) {
    const int64_t at = (int64_t)t.e * p.wide + half * p.N + min(tile * 16 + i16, p.N - 1);
    const uint8_t* codes = p.codes + at * (K / 2) + 16 * g;
    const int64_t sp = at * groups;
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int c = wave * RW + j, k = c < runs ? c : 0;
      const int64_t s = sp + k * GR;
      r[j].load(codes + k * (kRun / 2), p.scales + s * SB, p.zeros + s);
    }
  };
  auto product = [&](Raw (&r)[RW]) {
    v4f acc = none;
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      gather_groups<GROUP>(r[j].w);
      v4f sum, ssum;
      // The sums of x are the same for every tile, and kept: but 7 runs leave no
      // registers for them.
      u32x4_t one = ones;
      if (RW > 4) asm volatile("" : "+v"(one));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int b = q * GR / 4;
        const bool begin = q % (4 / GR) == 0, last = (q + 1) % (4 / GR) == 0;
        const uint32_t z = r[j].zero(b);
        if (SUMS) ssum = mma<DT>(xa[j][q], one, begin ? none : ssum);
        const u32x4_t v =
            codes_as_values<DT, MX>(r[j].w[q], 0x64006400u + z * 0x00010001u, 0.0f);
        sum = mma<DT>(xa[j][q], v, begin ? none : sum);
        if (last) {
          const float s = r[j].template scale<DT>(b), zf = -128.0f - (float)z;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = SUMS ? fmaf(zf, ssum[i], sum[i]) : sum[i];
            acc[i] = fmaf(s, f, acc[i]);
          }
        }
      }
    }
    return acc;
  };
  // The waves' sums of a tile.  Two buffers in turn: what is written was read two
  // tiles ago.  The barrier is for LDS alone, the next loads stay in flight.
  auto finish = [&](int tile, int buf, v4f a, v4f u) {
    red[buf][wave][0][lane] = a;
    if constexpr (GATED) red[buf][wave][NT - 1][lane] = u;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (threadIdx.x >= 256) return;
    const float* flat = reinterpret_cast<const float*>(red[buf]);
    const int r16 = threadIdx.x >> 4, c = threadIdx.x & 15;
    const int at = ((r16 / 4) * 16 + c) * 4 + r16 % 4;
    float f = 0.0f, h = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f += flat[w * NT * 256 + at];
      if (GATED) h += flat[w * NT * 256 + 256 + at];
    }
    if (r16 < rows && tile * 16 + c < p.N) {
      if (p.act != kActNone) f = apply_act(p.act, f, h, p.limit);
      RowVec<DT>::store_one(p.out, (row0 + r16) * p.N + tile * 16 + c, f);
    }
  };

  Raw ra[RW], rb[RW];
  int tile = t.nt * per_block;
  const int end = min(tile + per_block, tiles);
  fetch(tile, 0, ra);
#pragma unroll
  for (int j = 0; j < RW; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (wave * RW + j >= runs) xa[j][q] = u32x4_t{0u, 0u, 0u, 0u};
      if (!MX) xa[j][q] = paired(xa[j][q]);
    }
  if constexpr (GATED) {
    int buf = 0;
    for (; tile + 1 < end; ++tile, buf ^= 1) {
      fetch(tile, 1, rb);
      const v4f a = product(ra);
      fetch(tile + 1, 0, ra);
      finish(tile, buf, a, product(rb));
    }
    fetch(tile, 1, rb);
    const v4f a = product(ra);
    finish(tile, buf, a, product(rb));
  } else {
    for (; tile + 2 < end; tile += 2) {
      fetch(tile + 1, 0, rb);
      finish(tile, 0, product(ra), none);
      fetch(tile + 2, 0, ra);
      finish(tile + 1, 1, product(rb), none);
    }
    if (tile + 1 < end) {
      fetch(tile + 1, 0, rb);
      finish(tile, 0, product(ra), none);
      finish(tile + 1, 1, product(rb), none);
    } else {
      finish(tile, 0, product(ra), none);
    }
  }
}

template <int DT, int FMT, int GROUP, bool S32, int RW>
hipError_t launch_few(const ExpertW4Args& a, hipStream_t stream) {
  const int tiles = (a.N + 15) / 16;
  const int64_t row_tiles = most_row_tiles<16>(a.offsets, a.R, a.E);
  int per = 8;
  while (per > 1 && row_tiles * ((tiles + per - 1) / per) < 512) per /= 2;
  const dim3 grid = grid_of((row_tiles * ((tiles + per - 1) / per) + 7) / 8 * 8);
  if (a.wide != a.N)
    expert_w4_few_kernel<DT, FMT, GROUP, S32, RW, true>
        <<<grid, 64 * kWaves, 0, stream>>>(a, per);
  else
    expert_w4_few_kernel<DT, FMT, GROUP, S32, RW, false>
        <<<grid, 64 * kWaves, 0, stream>>>(a, per);
  return hipGetLastError();
}

template <int DT, int FMT, int GROUP, bool S32>
hipError_t launch_rows(const ExpertW4Args& a, hipStream_t stream) {
  constexpr bool MX = FMT == kW4Mxfp4;
  constexpr int MOST = DT == kF32 ? 2 : 4;
  const bool few = a.R <= 16 * (int64_t)a.E;
  if constexpr (DT != kF32) {
    if (few && a.K % kRun == 0) {
      const int runs = a.K / kRun;
      if (runs <= 2 * kWaves) return launch_few<DT, FMT, GROUP, S32, 2>(a, stream);
      if (runs <= 4 * kWaves) return launch_few<DT, FMT, GROUP, S32, 4>(a, stream);
      if (runs <= 7 * kWaves) return launch_few<DT, FMT, GROUP, S32, 7>(a, stream);
    }
  }
  if (few) return launch_tile<DT, MX, GROUP, S32, 1, 2>(a, stream);
  return launch_tile<DT, MX, GROUP, S32, MOST, 2>(a, stream);
}

}  // namespace

template <int DT>
hipError_t launch_expert_w4_dt(const ExpertW4Args& a, bool s32, hipStream_t stream) {
  if (a.format == kW4Mxfp4) return launch_rows<DT, kW4Mxfp4, 32, false>(a, stream);
  auto group = [&](auto format, auto wide_scales) {
    constexpr int FMT = decltype(format)::value;
    constexpr bool S32 = decltype(wide_scales)::value;
    switch (a.group) {
      case 32: return launch_rows<DT, FMT, 32, S32>(a, stream);
      case 64: return launch_rows<DT, FMT, 64, S32>(a, stream);
      default: return launch_rows<DT, FMT, 128, S32>(a, stream);
    }
  };
  auto scales = [&](auto format) {
    if constexpr (DT != kF32) {
      if (!s32) return group(format, std::false_type());
    }
    return group(format, std::true_type());
  };
  if (a.format == kW4Int4Zero) return scales(std::integral_constant<int, kW4Int4Zero>());
  return scales(std::integral_constant<int, kW4Int4>());
}

template hipError_t launch_expert_w4_dt<MOE_W4_DTYPE>(const ExpertW4Args&, bool, hipStream_t);

}  // namespace moe
