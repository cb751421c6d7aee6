// Rows of bf16, fp16 or fp32 values in 16-byte vectors, for the kernels
// around the expert layer (rows of any width, starting at any element).
//
// A vector holds N = 8 (bf16, fp16) or 4 (fp32) consecutive columns.  Rows of
// an odd width start at odd addresses: gfx950 loads and stores 16 bytes at
// any address, so one form serves every width.  A row's last vector, where it
// is partial, is loaded from the row's last N columns and shifted into place
// when it is used (settle), so that no load depends on a branch and all of a
// lane's loads are in flight together: a branch per load with the elements
// one by one on its other side made the compiler wait after each.  Rows
// narrower than a vector go element by element (RowOne).
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
  static constexpr int kDt = DT;
  static constexpr int kSize = dtype_size(DT);
  static constexpr int N = 16 / kSize;             // columns of a vector
  typedef u32x4_t Raw;

  // the first column of a vector moved so that it ends inside the row (H >= N)
  static __device__ __forceinline__ int inside(int col, int H) { return min(col, H - N); }

  template <bool NT>
  static __device__ __forceinline__ Raw load_at(const uint8_t* row, int c) {
    const u32x4_any* q = reinterpret_cast<const u32x4_any*>(row + (int64_t)c * kSize);
    return NT ? __builtin_nontemporal_load(q) : *q;
  }
  template <bool NT>
  static __device__ __forceinline__ void store_at(uint8_t* row, int c, Raw v) {
    u32x4_any* q = reinterpret_cast<u32x4_any*>(row + (int64_t)c * kSize);
    if (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
  }
  // columns [col, col + N) of a row of H, once settled
  template <bool NT>
  static __device__ __forceinline__ Raw load(const uint8_t* row, int col, int H) {
    return load_at<NT>(row, inside(col, H));
  }
  // all bits but those of the first k columns
  static __device__ __forceinline__ Raw mask_from(int k) {
    Raw m;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = kSize == 4 ? (i >= k ? ~0u : 0u)
                        : (2 * i >= k ? 0xFFFFu : 0u) | (2 * i + 1 >= k ? 0xFFFF0000u : 0u);
    return m;
  }
  // columns past the row's end become 0
  static __device__ __forceinline__ void settle(Raw& v, int col, int H) {
    const int k = col + N - H;                     // columns past the end
    if (k <= 0) return;
    if (kSize == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = (k & 1) ? (v[i] >> 16) | (i < 3 ? v[(i + 1) & 3] << 16 : 0u) : v[i];
    }
    const int w = kSize == 2 ? k >> 1 : k;         // whole words
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (w & 1) ? (i < 3 ? v[(i + 1) & 3] : 0u) : v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (w & 2) ? (i < 2 ? v[(i + 2) & 3] : 0u) : v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = k >= N ? 0u : v[i];
  }
  template <bool NT>
  static __device__ __forceinline__ void store(uint8_t* row, int col, int H, Raw v) {
    if (col + N <= H) {
      store_at<NT>(row, col, v);
      return;
    }
    uint8_t* p = row + (int64_t)col * kSize;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (col + i >= H) return;
      if (kSize == 4) reinterpret_cast<uint32_t*>(p)[i] = v[i];
      else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }

  // columns [v0, c + N) of the vector at c, c <= v0
  template <bool NT>
  static __device__ __forceinline__ void store_tail(uint8_t* row, int c, int v0, Raw v) {
    if (c == v0) {
      store_at<NT>(row, c, v);
      return;
    }
    uint8_t* p = row + (int64_t)c * kSize;
#pragma unroll
    for (int i = 1; i < N; ++i) {
      if (c + i < v0) continue;
      if (kSize == 4) reinterpret_cast<uint32_t*>(p)[i] = v[i & 3];
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

// The same for rows narrower than a vector: one column at a time.
template <int DT>
struct RowOne {
  static constexpr int kDt = DT;
  static constexpr int kSize = dtype_size(DT);
  static constexpr int N = 1;
  typedef uint32_t Raw;
  static __device__ __forceinline__ int inside(int col, int H) { return min(col, H - 1); }
  template <bool NT>
  static __device__ __forceinline__ Raw load_at(const uint8_t* row, int c) {
    return __float_as_uint(RowVec<DT>::load_one(row, c));
  }
  template <bool NT>
  static __device__ __forceinline__ void store_at(uint8_t* row, int c, Raw v) {
    RowVec<DT>::store_one(row, c, __uint_as_float(v));
  }
  template <bool NT>
  static __device__ __forceinline__ Raw load(const uint8_t* row, int col, int H) {
    return load_at<NT>(row, inside(col, H));
  }
  static __device__ __forceinline__ Raw mask_from(int k) { return k > 0 ? 0u : ~0u; }
  static __device__ __forceinline__ void settle(Raw& v, int col, int H) {
    if (col >= H) v = 0u;
  }
  template <bool NT>
  static __device__ __forceinline__ void store(uint8_t* row, int col, int H, Raw v) {
    if (col < H) store_at<NT>(row, col, v);
  }
  template <bool NT>
  static __device__ __forceinline__ void store_tail(uint8_t* row, int c, int, Raw v) {
    store_at<NT>(row, c, v);
  }
  static __device__ __forceinline__ void unpack(const Raw v, float f[1]) {
    f[0] = __uint_as_float(v);
  }
  static __device__ __forceinline__ Raw pack(const float f[1]) { return __float_as_uint(f[0]); }
  static __device__ __forceinline__ float load_one(const uint8_t* base, int64_t i) {
    return RowVec<DT>::load_one(base, i);
  }
};

// Grids in two dimensions: a dimension holds fewer than 2^32 lanes, 2^22
// blocks of 1024.  A kernel compares its block's index (at most 2^31 blocks,
// rounded up to rows of the grid) with what there is.
constexpr int64_t kGridX = 1 << 20;
inline dim3 grid_of(int64_t blocks) {
  return dim3((unsigned)(blocks < kGridX ? blocks : kGridX),
              (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ uint32_t block_index() {
  return blockIdx.y * (uint32_t)kGridX + blockIdx.x;
}

// Between a wave's stores to LDS and other lanes' loads: LDS takes a wave's
// accesses in order, the compiler has to as well.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

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
