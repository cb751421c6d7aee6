// Rows of bf16, fp16 or fp32 values in 16-byte vectors, for the kernels
// around the expert layer (rows of any width, starting at any element).
//
// A vector holds 8 (bf16, fp16) or 4 (fp32) consecutive columns.  Rows of an
// odd width start at odd addresses: gfx950 loads and stores 16 bytes at any
// address, so one form serves every width, and only a row's last, partial
// vector goes element by element.
#pragma once

#include "device_common.h"

namespace moe {

// element types (values match moe_dtype_t)
constexpr int kBf16 = 0;
constexpr int kF16 = 1;
constexpr int kF32 = 2;
constexpr int dtype_size(int dt) { return dt == kF32 ? 4 : 2; }

typedef u32x4_t __attribute__((aligned(2))) u32x4_any;   // 16 bytes at any 2-byte address

template <int DT>
struct RowVec {
  static constexpr int kSize = dtype_size(DT);
  static constexpr int N = 16 / kSize;             // columns of a vector

  // columns [col, col + N) of a row of H; those past the row's end are 0
  template <bool NT>
  static __device__ __forceinline__ u32x4_t load(const uint8_t* row, int col, int H) {
    const uint8_t* p = row + (int64_t)col * kSize;
    if (col + N <= H) {
      const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p);
      return NT ? __builtin_nontemporal_load(q) : *q;
    }
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (col + i >= H) continue;
      if (kSize == 4) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else v[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
    return v;
  }
  template <bool NT>
  static __device__ __forceinline__ void store(uint8_t* row, int col, int H, u32x4_t v) {
    uint8_t* p = row + (int64_t)col * kSize;
    if (col + N <= H) {
      u32x4_any* q = reinterpret_cast<u32x4_any*>(p);
      if (NT) __builtin_nontemporal_store(v, q);
      else *q = v;
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (col + i >= H) continue;
      if (kSize == 4) reinterpret_cast<uint32_t*>(p)[i] = v[i];
      else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }

  static __device__ __forceinline__ void unpack(const u32x4_t v, float f[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (DT == kF32) {
        f[i] = __uint_as_float(v[i]);
      } else if (DT == kBf16) {
        f[i] = (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
      } else {
        f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[i / 2] >> (16 * (i & 1))));
      }
    }
  }
  // one rounding, to nearest even, to the rows' type
  static __device__ __forceinline__ u32x4_t pack(const float f[N]) {
    u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (DT == kF32) {
        v[i] = __float_as_uint(f[i]);
      } else if (DT == kBf16) {
        if ((i & 1) == 0) v[i / 2] = pack_bf16x2(f[i], f[i + 1]);
      } else {
        v[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[i]) << (16 * (i & 1));
      }
    }
    return v;
  }
  static __device__ __forceinline__ float load_one(const uint8_t* base, int64_t i) {
    if (DT == kF32) return reinterpret_cast<const float*>(base)[i];
    const uint16_t h = reinterpret_cast<const uint16_t*>(base)[i];
    if (DT == kBf16) return __uint_as_float((uint32_t)h << 16);
    return (float)__builtin_bit_cast(_Float16, h);
  }
  static __device__ __forceinline__ void store_one(uint8_t* base, int64_t i, float f) {
    if (DT == kF32) reinterpret_cast<float*>(base)[i] = f;
    else if (DT == kBf16) reinterpret_cast<uint16_t*>(base)[i] = (uint16_t)f32_to_bf16_bits(f);
    else reinterpret_cast<uint16_t*>(base)[i] = __builtin_bit_cast(uint16_t, (_Float16)f);
  }
};

// Reductions over the 64 lanes of a wave, the same in every lane, in a fixed
// order: four steps shift inside the rows of 16 lanes, two carry a row's
// result to the next ones (DPP operands of the adds themselves, where a
// shuffle would go through LDS), and lane 63's value is read back.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL,
                                                    ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_or<0x111, 0xF>(0.0f, v);      // row_shr:1, 2, 4, 8
  v += dpp_or<0x112, 0xF>(0.0f, v);
  v += dpp_or<0x114, 0xF>(0.0f, v);
  v += dpp_or<0x118, 0xF>(0.0f, v);
  v += dpp_or<0x142, 0xA>(0.0f, v);      // row_bcast:15 into rows 1 and 3
  v += dpp_or<0x143, 0xC>(0.0f, v);      // row_bcast:31 into rows 2 and 3
  return last_lane(v);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOE_STEP(ctrl, rows) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false))
  MOE_STEP(0x111, 0xF);
  MOE_STEP(0x112, 0xF);
  MOE_STEP(0x114, 0xF);
  MOE_STEP(0x118, 0xF);
  MOE_STEP(0x142, 0xA);
  MOE_STEP(0x143, 0xC);
#undef MOE_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// fp32 values as integers of the same order; 0 is below every one of them
__device__ __forceinline__ uint32_t ordered_bits(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);          // -0 and +0 are equal
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ float wave_max(float v) {
  return from_ordered(wave_max(ordered_bits(v)));
}

}  // namespace moe
