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
// scale per group), the rows of x the A operand.  The codes of a group have to
// meet in one MFMA: the lane quarters exchange registers first.
//
// Codes, scales and zeros come as whole lines by loads into a ring of LDS stages
// that each wave keeps for itself, two or three stages ahead, with no barrier; x
// stays in registers where it fits and is streamed beside them where it does not
// (launch_rows has the sizes and their times).  512 rows of 128 experts, 4096
// by 2 x 2048, MXFP4: 184 us, 1147 MB of codes and scales at 6.2 TB/s.  One row x
// 7168 by 4096: 6.9 us; four of every six loads are of x's 16 rows, of which one is
// there.  Past 16 rows of an expert the conversion of the codes, once for every tile of
// up to 64 rows, and x's way through the ring bound it: 37 rows x 14336 by 4096, 33 MB,
// 27.6 us; 4096 rows x 4096 by 4096 750 us.  fp32 rows, 512 of 128 experts as above, 830
// us.  Columns or pointers that lines do not fit take the simple kernel, which loads from
// memory into registers, 16 rows at a time.
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
#include "lds_copy.h"
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

// A lane quarter g holds 32 consecutive codes, columns 32g on: after this, dword
// j holds columns 32j + 8g on in every quarter, so that MFMA j takes 32
// consecutive columns, which are of one group, and x's operand for it is 64
// consecutive bytes of a row.  (Groups of 64 could do with half the exchange, groups
// of 128 with none; x's lanes would then lie 64 bytes apart.)
__device__ __forceinline__ void gather_groups(u32x4_t& w) {
  const auto p = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto q = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  const auto s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  w = u32x4_t{r[0], r[1], s[0], s[1]};
}
__device__ __forceinline__ int column_of(int j, int g) { return 32 * j + 8 * g; }

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

// x's 8 columns of one MFMA as its A operand: as they are (e2m1 codes come in
// order), in the order of the codes' pairs, or, of fp32, in three parts.
template <int DT, bool MX, int LOADS, int PARTS>
__device__ __forceinline__ void x_operand(const u32x4_t (&x)[LOADS], u32x4_t (&a)[PARTS]) {
  if constexpr (DT == kF32) {
    float f[8], q[8][3];
    RowVec<kF32>::unpack(x[0], f);
    RowVec<kF32>::unpack(x[1], f + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(f[i], q[i]);
#pragma unroll
    for (int h = 0; h < 3; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[h][i] = pack_bf16x2(q[2 * i][h], q[2 * i + 1][h]);
  } else {
    a[0] = MX ? x[0] : paired(x[0]);
  }
}

// The waves' sums of a tile added up, activated and stored.  Of wave w, weight
// tile n and row tile m, lane l's four values belong to weight row 16n + l % 16
// and rows 16m + 4 (l / 16) + i.
template <int DT, int MT, int NT, int W>
__device__ __forceinline__ void store_tile(const ExpertW4Args& p, const float* flat,
                                           int64_t row0, int rows, int n0, int outc,
                                           bool gated) {
  constexpr int WAVE = NT * MT * 256;
  for (int o = threadIdx.x; o < 16 * MT * outc; o += 64 * W) {
    const int r = o / outc, c = o % outc;
    if (r >= rows || n0 + c >= p.N) continue;
    auto total = [&](int n, int c16) {
      const int at = (n * MT + r / 16) * 256 + ((r % 16 / 4) * 16 + c16) * 4 + r % 4;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += flat[w * WAVE + at];
      return v;
    };
    const float a = total(c / 16, c % 16);
    const float u = gated ? total(NT / 2 + c / 16, c % 16) : 0.0f;
    const float f = p.act == kActNone ? a : expert_act(p.act, a, u, p.limit);
    RowVec<DT>::store_one(p.out, (row0 + r) * p.N + n0 + c, f);
  }
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
        const int k = k0 + column_of(j, g);
#pragma unroll
        for (int h = 0; h < XR; ++h) {
          const u32x4_t v = *reinterpret_cast<const u32x4_any*>(
              xp[m] + (int64_t)(k < K ? k : 0) * ES + 16 * h);
          x[m][j][h] = k < K ? v : u32x4_t{0u, 0u, 0u, 0u};
        }
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) gather_groups(w[n]);

    v4f sum[NT][MT], ssum[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = j * GR / 4;                                // the MFMA's group in the run
      const bool first = j % (4 / GR) == 0, last = (j + 1) % (4 / GR) == 0;
      u32x4_t xa[MT][PARTS];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        x_operand<DT, MX>(x[m][j], xa[m]);
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

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[wave][n * MT + m][lane] = acc[n][m];
  __syncthreads();
  store_tile<DT, MT, NT, kWaves>(p, reinterpret_cast<const float*>(red), row0, rows, n0, outc, gated);
}

template <int DT, bool MX, int GROUP, bool S32, int MT, int NT>
hipError_t launch_tile(const ExpertW4Args& a, hipStream_t stream) {
  const int outc = a.wide != a.N ? NT * 8 : NT * 16;
  const int64_t tiles =
      most_row_tiles<16 * MT>(a.offsets, a.R, a.E) * ((a.N + outc - 1) / outc);
  expert_w4_kernel<DT, MX, GROUP, S32, MT, NT>
      <<<grid_of(blocks_of_tiles(tiles)), 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

// ---- streamed ------------------------------------------------------------------
// An MFMA operand's neighbouring lanes hold different rows, and loads of theirs are
// not joined: 64 accesses of 16 bytes for an instruction (measured: with codes,
// scales and x loaded so, the address unit was busy all the time, 280 us for 128
// experts of 2 x 2048 x 4096, 46 for 37 rows x 14336 by 4096).  So everything
// that is streamed goes to LDS, in a wave's own ring of stages, by loads whose
// neighbouring lanes are neighbours in memory, and is read from there as operands.
// No barrier is needed for the ring: a wave reads what it loaded itself.

constexpr uint32_t kOutOfRange = 0xF0000000u;    // past every buffer: reads as zeros

// A stage's part for 16 weight rows and H runs: a row's 64 H bytes of codes one
// after the other, its 16-byte chunk c at c ^ key; then each row's DW words of
// scales and, with them, ZW of zero points.  A ds_read_b128 passes 16 lanes at a
// time, rows 0-3 and 12-15 at one chunk with rows 4-11 at the next: the keys put
// them into 16 different bank groups.
template <int H>
__device__ __forceinline__ int key_codes(int r) {
  if (H == 1) return (((r >> 1) ^ (r >> 2)) & 2) | (r >> 3);
  return r & 7;
}

template <int FMT, int GROUP, int SB, int H>
struct Strip {
  static constexpr bool MX = FMT == kW4Mxfp4, ZERO = FMT == kW4Int4Zero;
  static constexpr int GR = kRun / GROUP, CH = 4 * H, CODES = H;   // loads of codes
  // a stage's scales and zero points in bytes of a row; less than a word: its part
  static constexpr int SBY = H * GR * SB, ZBY = H * GR;
  static constexpr int DW = SBY >= 4 ? SBY / 4 : 1, ZW = ZERO ? (ZBY >= 4 ? ZBY / 4 : 1) : 0;
  static constexpr int SL = (16 * DW + 63) / 64, ZL = ZERO ? 1 : 0;
  static constexpr int SCALES = 1024 * H, ZEROS = SCALES + 64 * DW;
  static constexpr int BYTES = ZEROS + 64 * ZW;
  static constexpr int LOADS = CODES + SL + ZL;
  static_assert(16 * ZW <= 64, "one load");

  // Where the expert's data is, and this lane's offsets in it (of weight row 0).
  v4i codes, scales, zeros;
  uint32_t at_codes, at_scales, at_zeros;
  int pitch, spitch, zpitch, lane;
  bool stream;                   // no other block reads these weights

  __device__ __forceinline__ Strip() {}
  __device__ __forceinline__ Strip(const ExpertW4Args& p, int e, bool alone) {
    stream = alone;
    lane = threadIdx.x & 63;
    const int64_t rows = (int64_t)e * p.wide, groups = p.K / GROUP;
    pitch = p.K / 2;
    spitch = (int)groups * SB;
    zpitch = (int)groups;
    codes = buffer_rsrc(p.codes + rows * pitch, kOutOfRange);
    scales = buffer_rsrc(p.scales + rows * spitch, kOutOfRange);
    zeros = buffer_rsrc(ZERO ? p.zeros + rows * zpitch : p.codes, kOutOfRange);
    const int r = lane / CH;
    at_codes = (uint32_t)r * pitch;
    at_scales = (uint32_t)(lane / DW) * spitch + (lane % DW) * 4;
    at_zeros = ZERO ? (uint32_t)(lane / (ZW + !ZERO)) * zpitch + (lane % (ZW + !ZERO)) * 4 : 0;
  }
  // weight rows from `row` (those from `last` on read as zeros), stage c of H runs
  __device__ __forceinline__ void fetch(uint32_t lds, int row, int last, int c) const {
#pragma unroll
    for (int i = 0; i < CODES; ++i) {
      const int r = i * (64 / CH) + lane / CH;
      const int chunk = (lane % CH) ^ key_codes<H>(r);
      const bool in = row + r < last && (H == 1 || c * CH + chunk < pitch / 16);
      const uint32_t from = at_codes + (uint32_t)(row + i * (64 / CH)) * pitch +
                            (c * CH + chunk) * 16;
      if (stream) dma16_nt(codes, lds + i * 1024, in ? from : kOutOfRange);
      else dma16(codes, lds + i * 1024, in ? from : kOutOfRange);
    }
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int l = i * 64 + lane;
      if (SL == 1 && l >= 16 * DW) continue;
      const int word = (c * SBY & ~3) + (l % DW) * 4;
      const uint32_t at =
          at_scales + (uint32_t)(row + i * (64 / DW)) * spitch + (c * SBY & ~3);
      dma4(scales, lds + SCALES + i * 256,
           row + l / DW < last && word < spitch ? at : kOutOfRange);
    }
    if constexpr (ZERO) {
      if (lane < 16 * ZW) {
        const int word = (c * ZBY & ~3) + (lane % ZW) * 4;
        const uint32_t at = at_zeros + (uint32_t)row * zpitch + (c * ZBY & ~3);
        dma4(zeros, lds + ZEROS, row + lane / ZW < last && word < zpitch ? at : kOutOfRange);
      }
    }
  }
  // what of run h of it is this lane's: weight row lane % 16
  static constexpr int RW = GR * SB >= 4 ? GR * SB / 4 : 1;    // a run's words of scales
  u32x4_t w;
  uint32_t s[RW], z;
  __device__ __forceinline__ void read(const uint8_t* lds, int c, int h) {
    const int i = lane & 15, g = lane >> 4;
    w = *reinterpret_cast<const u32x4_t*>(lds + i * (64 * H) +
                                          (((4 * h + g) ^ key_codes<H>(i)) << 4));
    // a run's scales or zero points may be half or a quarter of a word
    const int sb = (c * SBY & 3) + h * GR * SB, zb = (c * ZBY & 3) + h * GR;
#pragma unroll
    for (int d = 0; d < RW; ++d)
      s[d] = *reinterpret_cast<const uint32_t*>(lds + SCALES + i * DW * 4 + (sb & ~3) + d * 4);
    if (GR * SB < 4) s[0] >>= 8 * (sb & 3);
    if constexpr (ZERO) {
      z = *reinterpret_cast<const uint32_t*>(lds + ZEROS + i * ZW * 4 + (zb & ~3));
      if (GR < 4) z >>= 8 * (zb & 3);
    }
  }
  template <int DT>
  __device__ __forceinline__ float scale(int b) const {
    if constexpr (MX) return e8m0((s[0] >> (8 * b)) & 255u);
    else if constexpr (SB == 4) return __uint_as_float(s[b]);
    else if constexpr (DT == kBf16) return __uint_as_float((s[b / 2] >> (16 * (b & 1))) << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)(s[b / 2] >> (16 * (b & 1))));
  }
  __device__ __forceinline__ uint32_t zero(int b) const {
    return ZERO ? (z >> (8 * b)) & 255u : 8u;
  }
};

// One run's MFMAs of NT strips with MT tiles of 16 rows.  operand(m, q, a): x's
// operand; the sums of x are made here too where the codes carry an offset.  KEEP:
// the compiler may find them the same for every tile and hold on to them.
template <int DT, int PARTS, bool KEEP, int FMT, int GROUP, int SB, int NT, int MT, int H,
          class X>
__device__ __forceinline__ void run_product(Strip<FMT, GROUP, SB, H> (&r)[NT], X&& operand,
                                            v4f (&acc)[NT][MT]) {
  constexpr bool MX = FMT == kW4Mxfp4, SUMS = DT == kBf16 && !MX;
  constexpr int GR = kRun / GROUP;
  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
  u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  if (!KEEP) asm volatile("" : "+v"(ones));
#pragma unroll
  for (int n = 0; n < NT; ++n) gather_groups(r[n].w);
  v4f sum[NT][MT], ssum[MT];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int b = q * GR / 4;
    const bool begin = q % (4 / GR) == 0, last = (q + 1) % (4 / GR) == 0;
    u32x4_t xa[MT][PARTS];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      operand(m, q, xa[m]);
      if (SUMS) ssum[m] = mma<DT>(xa[m][0], ones, begin ? none : ssum[m]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t z = r[n].zero(b);
      const u32x4_t v =
          codes_as_values<DT, MX>(r[n].w[q], 0x64006400u + z * 0x00010001u, (float)z);
      const float s = r[n].template scale<DT>(b), zf = -128.0f - (float)z;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        v4f d = begin ? none : sum[n][m];
#pragma unroll
        for (int h = 0; h < PARTS; ++h) d = mma<DT>(xa[m][h], v, d);
        sum[n][m] = d;
        if (last) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = SUMS ? fmaf(zf, ssum[m][i], d[i]) : d[i];
            acc[n][m][i] = fmaf(s, f, acc[n][m][i]);
          }
        }
      }
    }
  }
}

// Up to 16 rows: x stays in registers, a wave's RW runs of it, while the block
// walks over tiles of 16 weight rows (gated: 16 of the gate's and 16 of the up's).

// Stages are pairs of runs, whole lines of 128 bytes of codes.
template <int DT, int FMT, int GROUP, bool S32, int W, int RW, bool GATED>
__global__ __launch_bounds__(64 * W, 4) void expert_w4_few_kernel(
    const ExpertW4Args p, int per_block) {
  constexpr bool MX = FMT == kW4Mxfp4;
  constexpr int SB = MX ? 1 : S32 ? 4 : 2, NT = GATED ? 2 : 1;
  typedef Strip<FMT, GROUP, SB, 2> S;
  constexpr int RED = W * NT * 1024;
  constexpr int FIT = (158 * 1024 / (16 / W) - RED) / (W * S::BYTES);
  constexpr int D = FIT > 8 ? 8 : FIT;           // stages of a wave's ring
  constexpr bool kKeep = RW * S::GR <= 8;        // the sums of x: four registers a group
  static_assert(D >= 2 && D * S::LOADS < 60, "ring");
  static_assert(D * S::BYTES >= 4096, "a run of x passes through the ring");
  __shared__ __align__(1024) uint8_t ring[W][D * S::BYTES];
  __shared__ __align__(16) v4f red[W][NT][64];

  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int tiles = (p.N + 15) / 16;
  const RowTile t = find_row_tile<16>(p.offsets, p.R, p.E, (tiles + per_block - 1) / per_block,
                                      block_index());
  if (!t.live) return;
  const int rows = min(16, t.n - t.m * 16);
  const int64_t row0 = (int64_t)t.r0 + t.m * 16;
  const int K = p.K, runs = K / kRun;
  const int c0 = wave * RW, mine = min(max(runs - c0, 0), RW);   // this wave's runs,
  const int pairs = (mine + 1) / 2;                              // and stages
  uint8_t* my = ring[wave];
  const uint32_t my_lds = lds_addr(my);

  // x: 4 rows of a run per load, 16 lanes a row, then through LDS to operands
  u32x4_t xa[RW][4];
  {
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.x + row0 * K * 2), 0, kOutOfRange, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < RW; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 4 * q + g;
        const uint32_t at = (uint32_t)r * K * 2 + (c0 + j) * (kRun * 2) + i16 * 16;
        xa[j][q] = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         rs, r < rows && j < mine ? at : kOutOfRange, 0, 0));
      }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      wave_lds_order();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 4 * q + g;
        *reinterpret_cast<u32x4_t*>(my + r * 256 + ((i16 ^ r) << 4)) = xa[j][q];
      }
      wave_lds_order();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(
            my + i16 * 256 + (((4 * q + g) ^ i16) << 4));
        xa[j][q] = MX ? v : paired(v);
      }
    }
    wait_lds();
  }

  const int first = t.nt * per_block, end = min(first + per_block, tiles);
  S strip[1] = {S(p, t.e, t.n <= 16)};
  // The ring is filled in the order it is read: tiles, halves, runs; behind the last
  // tile with zeros from nowhere, so that as many loads are in flight as ever.
  int f_tile = first, f_half = 0, f_j = 0, f_slot = 0;
  auto fetch = [&]() {
    strip[0].fetch(my_lds + f_slot * S::BYTES, f_half * p.N + f_tile * 16,
                   f_tile < end ? (f_half + 1) * p.N : 0, c0 / 2 + f_j);
    f_slot = f_slot + 1 == D ? 0 : f_slot + 1;
    if (++f_j < pairs) return;
    f_j = 0;
    if (GATED && f_half == 0) {
      f_half = 1;
      return;
    }
    f_half = 0;
    ++f_tile;
  };
  if (mine > 0) {
#pragma unroll 1
    for (int d = 0; d < D; ++d) fetch();
  }
  int slot = 0;
  auto product = [&]() {
    v4f acc[1][1] = {{v4f{0.0f, 0.0f, 0.0f, 0.0f}}};
#pragma unroll
    for (int j = 0; j < RW / 2; ++j) {
      if (j < pairs) {
        wait_loads<(D - 1) * S::LOADS>();        // all but the D - 1 stages after this one
        S second = strip[0];
        strip[0].read(my + slot * S::BYTES, c0 / 2 + j, 0);
        second.read(my + slot * S::BYTES, c0 / 2 + j, 1);
        wait_lds();
        fetch();
        slot = slot + 1 == D ? 0 : slot + 1;
        run_product<DT, 1, kKeep>(
            strip, [&](int, int q, u32x4_t (&a)[1]) { a[0] = xa[2 * j][q]; }, acc);
        strip[0].w = second.w;
        strip[0].z = second.z;
#pragma unroll
        for (int d = 0; d < S::RW; ++d) strip[0].s[d] = second.s[d];
        run_product<DT, 1, kKeep>(
            strip, [&](int, int q, u32x4_t (&a)[1]) { a[0] = xa[2 * j + 1][q]; }, acc);
      }
    }
    return acc[0][0];
  };
#pragma unroll 1
  for (int tile = first; tile < end; ++tile) {
    // the waves' sums meet in LDS, where the last tile's have been read by now
    const v4f a = product(), u = GATED ? product() : v4f{};
    lds_barrier();
    red[wave][0][lane] = a;
    if constexpr (GATED) red[wave][NT - 1][lane] = u;
    lds_barrier();
    if (threadIdx.x >= 256) continue;
    const float* flat = reinterpret_cast<const float*>(red);
    const int r16 = threadIdx.x >> 4, c = threadIdx.x & 15;
    const int at = ((r16 / 4) * 16 + c) * 4 + r16 % 4;
    float f = 0.0f, h = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f += flat[w * NT * 256 + at];
      if (GATED) h += flat[w * NT * 256 + 256 + at];
    }
    if (r16 < rows && tile * 16 + c < p.N) {
      if (p.act != kActNone) f = expert_act(p.act, f, h, p.limit);
      RowVec<DT>::store_one(p.out, (row0 + r16) * p.N + tile * 16 + c, f);
    }
  }
  wait_loads<0>();                               // nothing lands in LDS behind the block's end
}

// More rows, or more columns than registers hold: x goes through the ring too, 16
// MT rows of a run beside the codes; a wave takes every W-th run.
template <int DT, int FMT, int GROUP, bool S32, int MT, bool GATED, int NT, int W>
__global__ __launch_bounds__(64 * W) void expert_w4_runs_kernel(const ExpertW4Args p) {
  constexpr bool MX = FMT == kW4Mxfp4;
  constexpr int SB = MX ? 1 : S32 ? 4 : 2, ES = dtype_size(DT);
  constexpr int BM = 16 * MT, OUTC = GATED ? NT * 8 : NT * 16;
  constexpr int XROW = kRun * ES, CH = XROW / 16, PER = 64 / CH;   // x: rows of a load
  constexpr int PARTS = DT == kF32 ? 3 : 1, XL = DT == kF32 ? 2 : 1;
  typedef Strip<FMT, GROUP, SB, 1> S;
  constexpr int STAGE = NT * S::BYTES + BM * XROW, LOADS = NT * S::LOADS + BM / PER;
  constexpr int FIT = 160 * 1024 / (W * STAGE), D = FIT > 3 ? 3 : FIT;   // stages of a ring
  static_assert(D >= 2 && NT * MT * 1024 <= D * STAGE, "LDS");
  static_assert(D * LOADS < 60, "loads in flight");
  __shared__ __align__(1024) uint8_t ring[W * D * STAGE];

  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const RowTile t = find_row_tile<BM>(p.offsets, p.R, p.E, (p.N + OUTC - 1) / OUTC,
                                      block_index());
  if (!t.live) return;
  const int n0 = t.nt * OUTC, rows = min(BM, t.n - t.m * BM);
  const int64_t row0 = (int64_t)t.r0 + t.m * BM;
  const int K = p.K, runs = K / kRun;
  uint8_t* my = ring + wave * D * STAGE;
  const uint32_t my_lds = lds_addr(my);

  const v4i rx = buffer_rsrc(p.x + row0 * K * ES, kOutOfRange);
  uint32_t x_off[BM / PER];
#pragma unroll
  for (int i = 0; i < BM / PER; ++i) {
    const int r = i * PER + lane / CH;
    x_off[i] = r < rows ? (uint32_t)r * K * ES + (((lane % CH) ^ (r & 15)) << 4) : kOutOfRange;
  }
  S strip[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) strip[n] = S(p, t.e, false);
  auto fetch = [&](int c, int slot) {
    const uint32_t to = my_lds + slot * STAGE;
    const bool live = c < runs;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = GATED ? n * p.N + n0 : n0 + 16 * n;
      strip[n].fetch(to + n * S::BYTES, row, live ? GATED ? (n + 1) * p.N : p.N : 0, c);
    }
#pragma unroll
    for (int i = 0; i < BM / PER; ++i)
      dma16(rx, to + NT * S::BYTES + i * 1024,
            live && x_off[i] != kOutOfRange ? x_off[i] + c * XROW : kOutOfRange);
  };
  v4f acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // Every step issues a stage, behind the last run one of zeros from nowhere: how
  // many loads are in flight is then always the same.
  if (wave < runs) {
#pragma unroll 1
    for (int d = 0; d < D - 1; ++d) fetch(wave + d * W, d);
    int slot = 0, next = D - 1;
#pragma unroll 1
    for (int c = wave; c < runs; c += W) {
      fetch(c + (D - 1) * W, next);
      wait_loads<(D - 1) * LOADS>();
      const uint8_t* at = my + slot * STAGE;
#pragma unroll
      for (int n = 0; n < NT; ++n) strip[n].read(at + n * S::BYTES, c, 0);
      const uint8_t* x = at + NT * S::BYTES;
      run_product<DT, PARTS, true>(
          strip,
          [&](int m, int q, u32x4_t (&a)[PARTS]) {
            u32x4_t v[XL];
#pragma unroll
            for (int h = 0; h < XL; ++h)
              v[h] = *reinterpret_cast<const u32x4_t*>(
                  x + (16 * m + i16) * XROW + ((((4 * q + g) * XL + h) ^ i16) << 4));
            x_operand<DT, MX>(v, a);
          },
          acc);
      wait_lds();                                // before a load into what was read
      slot = slot + 1 == D ? 0 : slot + 1;
      next = next + 1 == D ? 0 : next + 1;
    }
  }
  wait_loads<0>();
  __syncthreads();
  v4f* red = reinterpret_cast<v4f*>(ring);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[(wave * NT * MT + n * MT + m) * 64 + lane] = acc[n][m];
  __syncthreads();
  store_tile<DT, MT, NT, W>(p, reinterpret_cast<const float*>(ring), row0, rows, n0, OUTC, GATED);
}

template <int DT, int FMT, int GROUP, bool S32, int W, int RW>
hipError_t launch_few(const ExpertW4Args& a, hipStream_t stream) {
  const int tiles = (a.N + 15) / 16;
  const int64_t row_tiles = most_row_tiles<16>(a.offsets, a.R, a.E);
  int per = 16;
  while (per > 1 && row_tiles * ((tiles + per - 1) / per) < 512) per /= 2;
  const dim3 grid = grid_of(blocks_of_tiles(row_tiles * ((tiles + per - 1) / per)));
  if (a.wide != a.N)
    expert_w4_few_kernel<DT, FMT, GROUP, S32, W, RW, true><<<grid, 64 * W, 0, stream>>>(a, per);
  else
    expert_w4_few_kernel<DT, FMT, GROUP, S32, W, RW, false><<<grid, 64 * W, 0, stream>>>(a, per);
  return hipGetLastError();
}

template <int DT, int FMT, int GROUP, bool S32, int MT, int W>
hipError_t launch_runs(const ExpertW4Args& a, hipStream_t stream) {
  const int64_t row_tiles = most_row_tiles<16 * MT>(a.offsets, a.R, a.E);
  const dim3 grid = grid_of(blocks_of_tiles(row_tiles * ((a.N + 15) / 16)));
  // eight waves where two stages of each fit
  constexpr int W1 = MT == 2 && DT != kF32 ? 8 : W;
  if (a.wide != a.N)
    expert_w4_runs_kernel<DT, FMT, GROUP, S32, MT, true, 2, W><<<grid, 64 * W, 0, stream>>>(a);
  else
    expert_w4_runs_kernel<DT, FMT, GROUP, S32, MT, false, 1, W1><<<grid, 64 * W1, 0, stream>>>(a);
  return hipGetLastError();
}

// Rows of 16-byte chunks and scales in whole words, as the streamed kernels load
// them.
template <int SB>
bool streams(const ExpertW4Args& a) {
  const int groups = a.K / a.group;
  const uintptr_t wide = (uintptr_t)a.x | (uintptr_t)a.codes;
  return a.K % kRun == 0 && wide % 16 == 0 && (uintptr_t)a.scales % 4 == 0 &&
         groups * SB % 4 == 0 &&
         (a.format != kW4Int4Zero || ((uintptr_t)a.zeros % 4 == 0 && groups % 4 == 0));
}

// Up to 16 rows per expert on average: x in registers, by columns 8 x 2, 8 x 4 or 16
// x 4 runs (bf16, 512 rows of 128 experts, 2 x 2048 columns, MXFP4, us: 2048 columns
// 108, 124 with 8 x 4; 4096: 202, 213 with 16 x 2; 7168: 387, 438 with 8 x 8, and
// 660 streamed).  Past 4096 columns a few tiles are done sooner streamed (one row x
// 7168 by 4096: 7.1, 9.5 in registers; by 16384: 24.3 and 24.8), past 8192 all are.
// More rows are streamed in tiles of 16 MT: up to 4 (fp32: 2).
template <int DT, int FMT, int GROUP, bool S32>
hipError_t launch_rows(const ExpertW4Args& a, hipStream_t stream) {
  constexpr int SB = FMT == kW4Mxfp4 ? 1 : S32 ? 4 : 2;
  if (!streams<SB>(a)) return launch_tile<DT, FMT == kW4Mxfp4, GROUP, S32, 1, 2>(a, stream);
  const int64_t per = ((int64_t)a.R + a.E - 1) / a.E;          // rows of an expert
  if constexpr (DT != kF32) {
    const int runs = a.K / kRun;
    const int64_t tiles = most_row_tiles<16>(a.offsets, a.R, a.E) * ((a.N + 15) / 16);
    if (per <= 16) {
      if (runs <= 16) return launch_few<DT, FMT, GROUP, S32, 8, 2>(a, stream);
      if (runs <= 32) return launch_few<DT, FMT, GROUP, S32, 8, 4>(a, stream);
      if (runs <= 64 && tiles > 1024) return launch_few<DT, FMT, GROUP, S32, 16, 4>(a, stream);
      return launch_runs<DT, FMT, GROUP, S32, 1, 8>(a, stream);
    }
    if (per <= 32) return launch_runs<DT, FMT, GROUP, S32, 2, 4>(a, stream);
    if (per <= 48) return launch_runs<DT, FMT, GROUP, S32, 3, 4>(a, stream);
    return launch_runs<DT, FMT, GROUP, S32, 4, 4>(a, stream);
  } else {
    if (per <= 16) return launch_runs<DT, FMT, GROUP, S32, 1, 4>(a, stream);
    return launch_runs<DT, FMT, GROUP, S32, 2, 4>(a, stream);
  }
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
