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
//
// One wave per token; lane l holds the VPL consecutive experts from l * VPL.
// Bound by vector instructions: about 520 per token of 256 experts, top 8 of
// 4 of 8 groups.  So reductions are lane exchanges in registers (with shuffles
// through LDS and 64-bit keys throughout 16384 such tokens took 60 us, now
// 18), a lane's keys are sorted once, nothing is in 64 bits that 32 can tell,
// and large batches put four tokens into a wave (router_rows_kernel, 15 us,
// 17 with 5 % padding; the bytes would take 3.5): about 220 per token, then
// bound by the steps that follow one another in a wave.
//
// The choice runs on 32-bit keys as ordered integers, k rounds of a wave
// maximum; 64-bit keys are computed only for a token where two keys that
// decide something lie within the 32-bit keys' error (kNear*: some tokens in
// a thousand), those of all its experts where more keys than a wave has lanes
// do (saturated scores, or scores that drown in a bias).
#include <float.h>
#include <limits.h>

#include <type_traits>

#include "kernels.h"
#include "row_vec.h"

namespace moe {

namespace {

constexpr int kRouterWaves = 4;   // tokens per block, one wave each

// The logit as the definition counts it: NaN masks, +inf is clamped.
__device__ __forceinline__ float clean_logit(float x) {
  return x == x ? fminf(x, FLT_MAX) : -INFINITY;
}

// 1 / (1 + e^-x) without overflow on either side
__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + expf(-x)); }

// Errors of the 32-bit keys.  A sigmoid from v_exp and v_rcp is off by less
// than 2^-22: its argument's rounding moves it by s (1 - s) |x| 2^-24 at most,
// exp and reciprocal add a step of s each.  A softmax adds the rounding of
// its sum, below 2^-19 of s for 1024 terms, and no s is above 1 / total.
// near is twice that error; adding the bias rounds once more, kNearRound.
// Two keys further apart than near + kNearRound |key| are in the order of
// their 64-bit values; so are two groups' values v1 > v2 with v1 - E1 above v2
// + E2, E = near + kNearRound * the magnitudes added up (they may cancel).
constexpr float kNearSigmoid = 0x1p-20f;
constexpr float kNearSoftmax = 0x1p-18f;    // * 1 / total
constexpr float kNearRound = 0x1p-22f;

// whether the larger key `b` and the smaller `c` (0: none) may change places
__device__ __forceinline__ bool near_keys(uint32_t b, uint32_t c, float near) {
  const float fb = from_ordered(b);
  return fb - from_ordered(c) <= fmaf(kNearRound, fabsf(fb), near);
}

// 2, 4 or 8 bytes at any 2-byte address
template <int BYTES>
struct Few;
template <>
struct Few<2> {
  typedef uint16_t Any;
};
template <>
struct Few<4> {
  typedef uint32_t __attribute__((aligned(2))) Any;
};
template <>
struct Few<8> {
  typedef uint32_t __attribute__((ext_vector_type(2))) __attribute__((aligned(2))) Any;
};

// the VPL logits of a lane as the definition counts them; past E: masked
template <int DT, int VPL, bool NT>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int e0,
                                            float (&x)[VPL]) {
  const uint8_t* row = (const uint8_t*)logits + t * E * RowVec<DT>::kSize;
  constexpr int N = RowVec<DT>::N;
  if constexpr (VPL % N == 0) {             // E > 64: at least one vector
    u32x4_t v[VPL / N];
#pragma unroll
    for (int i = 0; i < VPL / N; ++i) v[i] = RowVec<DT>::template load<NT>(row, e0 + i * N, E);
#pragma unroll
    for (int i = 0; i < VPL / N; ++i) {
      RowVec<DT>::settle(v[i], e0 + i * N, E);
      RowVec<DT>::unpack(v[i], x + i * N);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < E ? clean_logit(x[i]) : -INFINITY;
  } else {
    float f[VPL];
    if (E % VPL == 0) {                     // one load per lane
      typedef Few<VPL * RowVec<DT>::kSize> F;
      const typename F::Any v =
          *reinterpret_cast<const typename F::Any*>(row + min(e0, E - VPL) * RowVec<DT>::kSize);
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = RowVec<DT>::load_one((const uint8_t*)&v, i);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = RowVec<DT>::load_one(row, min(e0 + i, E - 1));
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < E ? clean_logit(f[i]) : -INFINITY;
  }
}

// larger and second of two pairs, each in order
__device__ __forceinline__ void merge_top2(uint32_t& b, uint32_t& s, uint32_t b2, uint32_t s2) {
  s = max(min(b, b2), max(s, s2));
  b = max(b, b2);
}
template <int CTRL>
__device__ __forceinline__ void merge_lanes(uint32_t& b, uint32_t& s) {
  merge_top2(b, s, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, true),
             (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, CTRL, 0xF, 0xF, true));
}

// the value of a group from its two best ordered keys, ordered again
__device__ __forceinline__ uint32_t group_value(uint32_t b, uint32_t s, int group_top) {
  if (b == 0u || s == 0u || group_top == 1) return b;
  return ordered_bits(from_ordered(b) + from_ordered(s));
}

// fp64 values as integers of the same order; 0 is below every one of them
__device__ __forceinline__ uint64_t ordered_bits64(double f) {
  const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double from_ordered64(uint64_t u) {
  return __longlong_as_double((long long)((u >> 63) ? u & ~(1ull << 63) : ~u));
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int l) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}

// the softmax's sum in 64 bits (1 for a sigmoid)
template <int VPL>
__device__ double exact_total(const RouterArgs& a, const float (&x)[VPL], float m) {
  if (a.sigmoid) return 1.0;
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (x[i] > -INFINITY) total += exp((double)x[i] - (double)m);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  return total;
}
__device__ double exact_key(const RouterArgs& a, float x, float m, double total, float bias) {
  const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x))
                             : exp((double)x - (double)m) / total;
  return s + (double)bias;
}

// the 64-bit keys of a lane as ordered integers; 0: masked
template <int VPL>
__device__ __forceinline__ void exact_keys(const RouterArgs& a, const float (&x)[VPL], float m,
                                           uint64_t (&key)[VPL]) {
  const double total = exact_total<VPL>(a, x, m);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0;
    if (x[i] > -INFINITY) {
      const double f = exact_key(a, x[i], m, total,
                                 a.bias != nullptr ? a.bias[(threadIdx.x & 63) * VPL + i] : 0.0f);
      if (f > -INFINITY) key[i] = ordered_bits64(f);           // NaN masks
    }
  }
}

// Sets the keys of all but the kept groups to 0; keep: of the lane's group
// where groups are whole lanes, else of group `lane`.
template <int VPL, class K>
__device__ __forceinline__ void drop_groups(const RouterArgs& a, bool keep, K (&key)[VPL]) {
  if (a.group_lanes_log >= 0) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = keep ? key[i] : 0u;
  } else {
    const uint64_t kept = __ballot(keep);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((kept >> (((threadIdx.x & 63) * VPL + i) / a.group_size & 63)) & 1)) key[i] = 0u;
  }
}

// Which groups are kept, by 64-bit keys (see drop_groups).
template <int VPL>
__device__ bool keep_exactly(const RouterArgs& a, const uint64_t (&key)[VPL], uint64_t* wkeys) {
  const int lane = threadIdx.x & 63;
  const int size = a.group_size;
  const bool by_lanes = a.group_lanes_log >= 0;
  uint64_t best = 0, second = 0;
  int group = lane, pitch = 1;
  if (by_lanes) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      second = max(second, min(best, key[i]));
      best = max(best, key[i]);
    }
    pitch = 1 << a.group_lanes_log;
    for (int d = 1; d < pitch; d <<= 1) {
      const uint64_t b = __shfl_xor((unsigned long long)best, d);
      const uint64_t s = __shfl_xor((unsigned long long)second, d);
      second = max(min(best, b), max(second, s));
      best = max(best, b);
    }
    group = lane >> a.group_lanes_log;
  } else {
    wave_lds_order();                       // what lay there has been read
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i < a.E) wkeys[lane * VPL + i] = key[i];
    wave_lds_order();
    if (lane < a.groups) {
#pragma unroll 8
      for (int j = 0; j < size; ++j) {
        const uint64_t v = wkeys[lane * size + j];
        second = max(second, min(best, v));
        best = max(best, v);
      }
    }
  }
  if (a.group_top > 1 && second != 0)
    best = ordered_bits64(from_ordered64(best) + from_ordered64(second));
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    const uint64_t o = read_lane(best, g * pitch);
    better += (o > best || (o == best && g < group)) ? 1 : 0;
  }
  return better < a.topk_groups && group < a.groups;
}

// Drops the keys (sets them to 0) of all but the topk_groups best groups,
// where two groups' values lie too close to tell by their 64-bit keys.
template <int VPL>
__device__ __forceinline__ void keep_groups(const RouterArgs& a, uint32_t (&key)[VPL],
                                            const float (&x)[VPL], float m, uint64_t* lds,
                                            float near) {
  uint32_t* wkeys = (uint32_t*)lds;
  const int lane = threadIdx.x & 63;
  const int size = a.group_size;
  // groups of 1, 2, 4, 8 or 16 whole lanes meet by lane exchanges; others
  // through LDS, lane g walking group g
  const bool by_lanes = a.group_lanes_log >= 0;
  uint32_t b = 0, s = 0;
  int group = lane, pitch = 1;
  if (by_lanes) {
    const int lanes = 1 << a.group_lanes_log;
#pragma unroll
    for (int i = 0; i < VPL; ++i) merge_top2(b, s, key[i], 0);
    if (lanes > 1) merge_lanes<0xB1>(b, s);       // quad_perm [1,0,3,2]
    if (lanes > 2) merge_lanes<0x4E>(b, s);       // quad_perm [2,3,0,1]
    if (lanes > 4) merge_lanes<0x141>(b, s);      // row_half_mirror
    if (lanes > 8) merge_lanes<0x140>(b, s);      // row_mirror
    group = lane >> a.group_lanes_log;
    pitch = lanes;
  } else {
    wave_lds_order();                     // what lay there, of the token before, has been read
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i < a.E) wkeys[lane * VPL + i] = key[i];
    wave_lds_order();
    if (lane < a.groups)
      for (int j = 0; j < size; ++j) merge_top2(b, s, wkeys[lane * size + j], 0);
  }
  const uint32_t v = group < a.groups ? group_value(b, s, a.group_top) : 0u;
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)v, g * pitch);
    better += (o > v || (o == v && g < group)) ? 1 : 0;
  }
  bool keep = better < a.topk_groups && group < a.groups;
  if (near > 0.0f) {                      // the least of those kept, the best one dropped
    const float fv = from_ordered(v);
    float mag = fabsf(from_ordered(b));
    if (a.group_top > 1 && s != 0u) mag += fabsf(from_ordered(s));
    const float err = fminf(fmaf(kNearRound, mag, near), FLT_MAX);
    const uint32_t dropped = wave_max(keep || v == 0u ? 0u : ordered_bits(fv + err));
    const uint32_t kept = ~wave_max(keep && v != 0u ? ~ordered_bits(fv - err) : 0u);
    if (kept <= dropped) {
      uint64_t exact[VPL];
      exact_keys<VPL>(a, x, m, exact);
      keep = keep_exactly<VPL>(a, exact, lds);
    }
  }
  drop_groups<VPL>(a, keep, key);
}

// The n candidates, one per lane, ordered by their 64-bit keys.  Every
// expert outside is clearly below the last of them.
template <int VPL>
__device__ int rank_exactly(const RouterArgs& a, const float (&x)[VPL], float m, float my_x,
                            float bias, int my_id, int n) {
  const int lane = threadIdx.x & 63;
  const double total = exact_total<VPL>(a, x, m);
  const uint64_t key =
      my_id >= 0 ? ordered_bits64(exact_key(a, my_x, m, total, bias)) : 0;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t o = read_lane(key, j);
    const int oid = __builtin_amdgcn_readlane(my_id, j);
    rank += (o > key || (o == key && oid < my_id)) ? 1 : 0;
  }
  // a permutation: the lanes past the candidates stay where they are
  return __builtin_amdgcn_ds_permute((my_id >= 0 ? rank : lane) * 4, my_id);
}

// The choice from 64-bit keys: lane j gets the j-th expert (-1: none left).
template <int VPL>
__device__ int choose_exactly(const RouterArgs& a, const float (&x)[VPL], float m,
                              uint64_t* wkeys) {
  const int lane = threadIdx.x & 63;
  uint64_t key[VPL];
  exact_keys<VPL>(a, x, m, key);
  if (a.groups > 1) drop_groups<VPL>(a, keep_exactly<VPL>(a, key, wkeys), key);
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    uint64_t b = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) b = max(b, key[i]);
    const uint64_t top = wave_max64(b);
    if (top == 0) break;
    const int l = __builtin_ctzll(__ballot(b == top));
    int at = 0;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) at = key[i] == top ? i : at;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = lane == l && at == i ? 0 : key[i];
    const int e = __builtin_amdgcn_readlane(lane * VPL + at, l);
    my_id = lane == j ? e : my_id;
  }
  return my_id;
}

// The keys of a lane's experts that are still to choose from.  Up to four are
// kept in order (equal ones by index: neighbours swap only when the second is
// larger), so that a round looks at one key and shifts the others up; more
// are searched when one of them has won.
template <int VPL>
struct LaneKeys {
  static constexpr bool kSorted = VPL <= 4;
  uint32_t key[VPL];
  int id[VPL];

  __device__ __forceinline__ void init(const uint32_t (&k)[VPL], int e0) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = k[i];
      id[i] = e0 + i;
    }
    if (!kSorted) return;
#pragma unroll
    for (int n = VPL - 1; n > 0; --n) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const bool swap = key[i + 1] > key[i];
        const uint32_t a = key[i], b = key[i + 1];
        const int ia = id[i], ib = id[i + 1];
        key[i] = swap ? b : a;
        key[i + 1] = swap ? a : b;
        id[i] = swap ? ib : ia;
        id[i + 1] = swap ? ia : ib;
      }
    }
  }
  __device__ __forceinline__ uint32_t head() const {
    uint32_t b = key[0];
    if (!kSorted) {
#pragma unroll
      for (int i = 1; i < VPL; ++i) b = max(b, key[i]);
    }
    return b;
  }
  // takes lane l's key b, its head, away; returns its expert
  __device__ __forceinline__ int pop(uint32_t b, int l) {
    const bool win = (int)(threadIdx.x & 63) == l;
    if (kSorted) {
      const int e = __builtin_amdgcn_readlane(id[0], l);
#pragma unroll
      for (int i = 0; i + 1 < VPL; ++i) {
        key[i] = win ? key[i + 1] : key[i];
        id[i] = win ? id[i + 1] : id[i];
      }
      key[VPL - 1] = win ? 0u : key[VPL - 1];
      return e;
    }
    int at = 0;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) at = key[i] == b ? i : at;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = win && at == i ? 0u : key[i];
    return __builtin_amdgcn_readlane(id[0] + at, l);
  }
};

// One token, by a whole wave; wkeys: LDS of E 64-bit keys, with groups.
template <int DT, int VPL>
__device__ __forceinline__ void route_token(const RouterArgs& a, int64_t t, uint64_t* wkeys) {
  const int lane = threadIdx.x & 63;
  const int E = a.E, k = a.k, e0 = lane * VPL;
  const bool pad = a.is_padding != nullptr && a.is_padding[t] != 0;
  if (pad) {
    if (lane < k) {
      a.ids[t * k + lane] = -1;
      a.weights[t * k + lane] = 0.0f;
    }
    return;
  }
  float x[VPL];
  load_logits<DT, VPL, true>(a.logits, t, E, e0, x);
  const bool scored = a.bias != nullptr || a.group_top > 1;
  float m = 0.0f, total = 1.0f;             // of the softmax over all experts
  const bool over_all = !a.sigmoid && (scored || !a.renormalize);
  if (over_all) {
    m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = wave_max(m);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += x[i] > -INFINITY ? expf(x[i] - m) : 0.0f;
    total = wave_sum(total);
  }
  const float near = !scored ? 0.0f : a.sigmoid ? kNearSigmoid : kNearSoftmax / total;
  float f[VPL];
  if (scored) {
    float bias[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      bias[i] = a.bias != nullptr && e0 + i < E ? a.bias[e0 + i] : 0.0f;
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        f[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i])) + bias[i];
    } else {
      const float inv_total = 1.0f / total;
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = fmaf(expf(x[i] - m), inv_total, bias[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) f[i] = x[i];
  }
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)           // a bias of NaN or -inf masks its expert too
    key[i] = x[i] > -INFINITY && f[i] > -INFINITY ? ordered_bits(f[i]) : 0u;
  if (a.groups > 1) keep_groups<VPL>(a, key, x, m, wkeys, near);
  // lane j keeps the j-th largest key and its expert
  int my_id = -1;
  uint32_t my_key = 0;
  LaneKeys<VPL> mine;
  mine.init(key, e0);
  uint32_t last = 0;
  int n = 0;
  while (n < 64) {
    const uint32_t head = mine.head();
    const uint32_t b = wave_max(head);
    if (b == 0u) break;
    // k of them; where keys have an error, as many more as the last may have
    // to be told from
    if (n >= k && (!scored || !near_keys(last, b, near))) break;
    const int l = __builtin_ctzll(__ballot(head == b));       // lowest lane first
    const int e = mine.pop(b, l);
    my_id = lane == n ? e : my_id;
    my_key = lane == n ? b : my_key;
    last = b;
    ++n;
  }
  // all lanes are taken: what is left may still belong before the last of them
  bool more = false;
  if (scored && n == 64) {
    const uint32_t b = wave_max(mine.head());
    more = b != 0u && near_keys(last, b, near);
  }
  const uint8_t* logits = (const uint8_t*)a.logits;
  float my_x = -INFINITY;
  if (my_id >= 0) my_x = clean_logit(RowVec<DT>::load_one(logits, t * E + my_id));
  if (scored) {
    // neighbours too close to tell, unless equal logits and biases say which
    const float bias = a.bias != nullptr && my_id >= 0 ? a.bias[my_id] : 0.0f;
    const uint32_t prev = __shfl_up((int)my_key, 1);
    const float prev_x = __shfl_up(my_x, 1), prev_bias = __shfl_up(bias, 1);
    const bool unclear = lane > 0 && my_id >= 0 && near_keys(prev, my_key, near) &&
                         !(prev_x == my_x && prev_bias == bias);
    if (more || __ballot(unclear) != 0) {
      // (where no key that is left is near the last one, every expert that may
      // be among the chosen has a lane)
      if (more) my_id = choose_exactly<VPL>(a, x, m, wkeys);
      else my_id = rank_exactly<VPL>(a, x, m, my_x, bias, my_id, n);
      my_x = -INFINITY;
      if (my_id >= 0) my_x = clean_logit(RowVec<DT>::load_one(logits, t * E + my_id));
    }
    if (lane >= k) {
      my_id = -1;
      my_x = -INFINITY;
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
    w = my_id >= 0 ? expf(my_x - m) / total : 0.0f;
  }
  if (lane < k) {
    a.ids[t * k + lane] = my_id;
    a.weights[t * k + lane] = w * a.scale;
  }
}

template <int DT, int VPL>
__global__ __launch_bounds__(64 * kRouterWaves) void router_topk_kernel(const RouterArgs a) {
  extern __shared__ uint64_t lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)block_index() * kRouterWaves + wave;
  if (t >= a.T) return;
  route_token<DT, VPL>(a, t, lds + (int64_t)wave * a.E);
}

// Reductions over the 16 lanes of a row, the same in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, rotated<0x128>(v));         // row_ror:8, 4, 2, 1
  v = max(v, rotated<0x124>(v));
  v = max(v, rotated<0x122>(v));
  return max(v, rotated<0x121>(v));
}
__device__ __forceinline__ float row_max(float v) {
  return from_ordered(row_max(ordered_bits(v)));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(rotated<0x128>(__float_as_uint(v)));
  v += __uint_as_float(rotated<0x124>(__float_as_uint(v)));
  v += __uint_as_float(rotated<0x122>(__float_as_uint(v)));
  return v + __uint_as_float(rotated<0x121>(__float_as_uint(v)));
}

// N keys in descending order: odd-even merges
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&key)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int i = 0; i + q < N; ++i) {
        const int first = q % p;
        if (i < first || ((i - first) / q) % 2 != 0 || i / (2 * p) != (i + q) / (2 * p)) continue;
        const uint32_t hi = max(key[i], key[i + q]);
        key[i + q] = min(key[i], key[i + q]);
        key[i] = hi;
      }
    }
  }
}

// Four tokens per wave, a row of 16 lanes each, for batches that fill the
// chip: what a wave spends beside the experts' scores it spends once for
// four.  Lane l of a row holds the VPL experts from l * VPL, their ordered
// keys with the place in the lane in the low bits, sorted once: a round takes
// the row's largest head, whose lane shifts its keys up.  What the low bits
// carried, or two keys' errors, leave open sends a token to the whole wave, as
// a router_topk_kernel wave takes it.  Keys that are 2-byte logits are exact
// in the bits above.
//
// A group's two keys and their sum lose less than 16 steps each: kNearPlaces of
// their magnitudes, and of subnormal ones, whose step is 2^-149, kNearLeast.
constexpr float kNearPlaces = 0x1p-17f;
constexpr float kNearLeast = 0x1p-143f;  // 64 such steps

template <int DT, int VPL, int WAVE_VPL>
__global__ __launch_bounds__(64 * kRouterWaves) void router_rows_kernel(const RouterArgs a) {
  extern __shared__ uint64_t lds[];
  __shared__ uint2 taken[kRouterWaves][4][16];
  const int lane = threadIdx.x & 63, row = lane >> 4, l = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = ((int64_t)block_index() * kRouterWaves + wave) * 4;
  if (t0 >= a.T) return;
  const int64_t t = t0 + row;
  const int E = a.E, k = a.k, e0 = l * VPL;
  const int64_t at = t < a.T ? t : a.T - 1;
  const bool live = t < a.T && (a.is_padding == nullptr || a.is_padding[at] == 0);
  float x[VPL];
  load_logits<DT, VPL, false>(a.logits, at, E, e0, x);   // a row's vectors share lines
  const bool scored = a.bias != nullptr || a.group_top > 1;
  const bool exact = !scored && DT != kF32;
  float m = 0.0f, total = 1.0f;             // of the softmax over all experts
  if (!a.sigmoid && (scored || !a.renormalize)) {
    m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = row_max(m);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += x[i] > -INFINITY ? expf(x[i] - m) : 0.0f;
    total = row_sum(total);
  }
  const float near = !scored ? 0.0f : a.sigmoid ? kNearSigmoid : kNearSoftmax / total;
  uint32_t key[VPL];
  if (scored) {
    float f[VPL];
    if (a.bias == nullptr) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = 0.0f;
    } else if (E % VPL == 0) {
      const int first = min(e0, E - VPL);
#pragma unroll
      for (int i = 0; i < VPL; i += 4)
        RowVec<kF32>::unpack(RowVec<kF32>::template load_at<false>((const uint8_t*)a.bias, first + i),
                             f + i);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = a.bias[min(e0 + i, E - 1)];
    }
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] += __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
    } else {
      const float inv_total = 1.0f / total;
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = fmaf(expf(x[i] - m), inv_total, f[i]);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      key[i] = x[i] > -INFINITY && f[i] > -INFINITY ? ordered_bits(f[i]) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = x[i] > -INFINITY ? ordered_bits(x[i]) : 0u;
  }
  constexpr uint32_t PLACE = VPL - 1;
#pragma unroll
  for (int i = 0; i < VPL; ++i)             // equal keys: the lower place is the larger
    key[i] = live && key[i] != 0u ? (key[i] & ~PLACE) | (PLACE - i) : 0u;
  sort_descending<VPL>(key);
  bool unclear = false;
  if (a.groups > 1) {                       // of 1, 2, 4, 8 or 16 whole lanes
    const int lanes = 1 << a.row_lanes_log;
    uint32_t b = key[0] & ~PLACE, s = key[1] & ~PLACE;
    if (lanes > 1) merge_lanes<0xB1>(b, s);       // quad_perm [1,0,3,2]
    if (lanes > 2) merge_lanes<0x4E>(b, s);       // quad_perm [2,3,0,1]
    if (lanes > 4) merge_lanes<0x141>(b, s);      // row_half_mirror
    if (lanes > 8) merge_lanes<0x140>(b, s);      // row_mirror
    const int group = l >> a.row_lanes_log;
    // the group in the low bits: values differ, and the lower group's is larger
    const uint32_t v = group < a.groups
                           ? (group_value(b, s, a.group_top) & ~15u) | (uint32_t)(15 - group) : 0u;
    int better = 0;                         // lanes of better groups
#define MOE_STEP(d) \
  if ((d & (lanes - 1)) == 0) better += rotated<0x120 + d>(v) > v ? 1 : 0
    MOE_STEP(1); MOE_STEP(2); MOE_STEP(3); MOE_STEP(4); MOE_STEP(5);
    MOE_STEP(6); MOE_STEP(7); MOE_STEP(8); MOE_STEP(9); MOE_STEP(10);
    MOE_STEP(11); MOE_STEP(12); MOE_STEP(13); MOE_STEP(14); MOE_STEP(15);
#undef MOE_STEP
    const bool keep = better < a.topk_groups && group < a.groups;
    if (!exact) {
      const bool some = v > 15u;
      const float fv = from_ordered(v);
      float mag = fabsf(from_ordered(b));
      if (a.group_top > 1 && s != 0u) mag += fabsf(from_ordered(s));
      const float err = fminf(fmaf(kNearPlaces, mag, near + kNearLeast), FLT_MAX);
      const uint32_t dropped = row_max(keep || !some ? 0u : ordered_bits(fv + err));
      const uint32_t kept = ~row_max(keep && some ? ~ordered_bits(fv - err) : 0u);
      unclear = kept <= dropped;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = keep ? key[i] : 0u;
  }
  // k rounds, and one for the best key that is left
  const int rounds = min(k + 1, 16);
  const uint32_t below = ((1u << l) - 1u) << (row & 1) * 16;
  for (int j = 0; j < rounds; ++j) {
    const uint32_t head = key[0] & ~PLACE;
    const uint64_t best = __ballot(head == row_max(head));
    const uint32_t half = row < 2 ? (uint32_t)best : (uint32_t)(best >> 32);
    if (((half >> (lane & 31)) & 1u) != 0u && (half & below) == 0u) {   // the lowest lane
      taken[wave][row][j] = make_uint2(key[0], (uint32_t)e0);
#pragma unroll
      for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
      key[VPL - 1] = 0u;
    }
  }
  wave_lds_order();
  const uint2 mine = taken[wave][row][min(l, rounds - 1)];
  uint32_t my_key = l < rounds ? mine.x : 0u;
  int my_id = my_key != 0u ? (int)(mine.y + (PLACE - (my_key & PLACE))) : -1;
  my_key &= ~PLACE;
  float my_x = -INFINITY;
  if (my_id >= 0) my_x = clean_logit(RowVec<DT>::load_one((const uint8_t*)a.logits, at * E + my_id));
  if (!exact) {
    // The chosen in order by their whole keys, unless equal logits and biases
    // say why not; then the last of them against all that is left, which is
    // no larger than the best place of the next key.
    const float bias = a.bias != nullptr && my_id >= 0 ? a.bias[my_id] : 0.0f;
    float f = my_x;
    if (scored)
      f = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-my_x)) + bias
                    : fmaf(expf(my_x - m), 1.0f / total, bias);
    const float prev = __uint_as_float(rotated<0x111>(__float_as_uint(f)));    // row_shr:1
    const float prev_x = __uint_as_float(rotated<0x111>(__float_as_uint(my_x)));
    const float prev_bias = __uint_as_float(rotated<0x111>(__float_as_uint(bias)));
    const bool close = l > 0 && my_id >= 0 &&
                       prev - (l == k ? from_ordered(my_key | PLACE) : f) <=
                           (scored ? fmaf(kNearRound, fabsf(prev), near) : 0.0f);
    unclear |= close && (l == k || !(prev_x == my_x && prev_bias == bias));
  }
  if (l >= k) {
    my_id = -1;
    my_x = -INFINITY;
  }
  float w = 0.0f;
  if (a.sigmoid) {
    w = my_id >= 0 ? sigmoid_f32(my_x) : 0.0f;
    if (a.renormalize) w /= row_sum(w) + 1e-20f;
  } else if (a.renormalize) {
    const float ms = row_max(my_x);
    w = my_id >= 0 ? expf(my_x - ms) : 0.0f;
    const float sum = row_sum(w);
    w = my_id >= 0 ? w / sum : 0.0f;
  } else {
    w = my_id >= 0 ? expf(my_x - m) / total : 0.0f;
  }
  const uint64_t open = __ballot(unclear);
  if (l < k && t < a.T && ((open >> (row * 16)) & 0xFFFFu) == 0) {
    a.ids[t * k + l] = my_id;
    a.weights[t * k + l] = w * a.scale;
  }
  for (int r = 0; r < 4; ++r)
    if (((open >> (r * 16)) & 0xFFFFu) != 0)
      route_token<DT, WAVE_VPL>(a, t0 + r, lds + (int64_t)wave * E);
}

// One wave per token.  With p the score of the chosen experts and g their
// weights' gradients: softmax over all experts dx_i = s_i c (g_i - sum g p);
// renormalized softmax the same over the chosen alone; sigmoid dx_j = c g_j
// p_j (1 - p_j), renormalized with g_j replaced by (g_j - sum g p / D) / D.
// A repeated id adds its terms in slot order.  A stream of T * E written
// (and read, for the softmax over all): 8191 x 128 bf16 5.4 us, nearly all
// of it latency.
template <int DT, int VPL>
__global__ __launch_bounds__(64 * kRouterWaves) void router_grad_kernel(
    const RouterArgs a, const int32_t* __restrict__ ids, const float* __restrict__ grad_w,
    uint8_t* __restrict__ grad_logits) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)block_index() * kRouterWaves + wave;
  if (t >= a.T) return;
  const int E = a.E, k = a.k, e0 = lane * VPL;
  const bool dense = !a.sigmoid && !a.renormalize;
  float out[VPL], xs[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) out[i] = 0.0f;
  if (dense) load_logits<DT, VPL, true>(a.logits, t, E, e0, xs);
  int id = lane < k ? ids[t * k + lane] : -1;
  if (id < 0 || id >= E) id = -1;
  // the chosen experts' gradients: of their logits, or, for a softmax over all
  // experts, still of their weights (no load then waits for the ids)
  float d = lane < k ? grad_w[t * k + lane] : 0.0f;
  if (id < 0) d = 0.0f;
  if (!dense && __ballot(id >= 0) != 0) {
    float x = -INFINITY;
    if (id >= 0) x = clean_logit(RowVec<DT>::load_one((const uint8_t*)a.logits, t * E + id));
    if (x == -INFINITY) {
      id = -1;
      d = 0.0f;
    }
    const float g = d;
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
    } else {
      const float mx = wave_max(x);         // every lane takes part
      const float p0 = id >= 0 ? expf(x - mx) : 0.0f;
      const float p = p0 / wave_sum(p0);
      d = p * (g - wave_sum(g * p));
    }
    d = id >= 0 ? d * a.scale : 0.0f;
  }
  for (int j = 0; j < k; ++j) {             // slot order: a repeated id adds up
    const int ej = __builtin_amdgcn_readlane(id, j) - e0;
    const float dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j));
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] += ej == i ? dj : 0.0f;
  }
  if (dense) {
    float m = xs[0], total = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, xs[i]);
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      xs[i] = xs[i] > -INFINITY ? expf(xs[i] - m) : 0.0f;
      if (xs[i] == 0.0f) out[i] = 0.0f;     // masked: whatever its weight's gradient
      total += xs[i];
      dot = fmaf(xs[i], out[i], dot);
    }
    total = wave_sum(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    dot = wave_sum(dot) * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      out[i] = xs[i] == 0.0f ? 0.0f : xs[i] * inv * a.scale * (out[i] - dot);
  }
  uint8_t* row = grad_logits + t * E * RowVec<DT>::kSize;
  constexpr int N = RowVec<DT>::N;
  if constexpr (VPL % N == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += N)
      if (e0 + i < E) RowVec<DT>::template store<true>(row, e0 + i, E, RowVec<DT>::pack(out + i));
  } else if (E % VPL == 0) {
    typedef Few<VPL * RowVec<DT>::kSize> F;
    typename F::Any v;
#pragma unroll
    for (int i = 0; i < VPL; ++i) RowVec<DT>::store_one((uint8_t*)&v, i, out[i]);
    if (e0 < E) *reinterpret_cast<typename F::Any*>(row + e0 * RowVec<DT>::kSize) = v;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i < E) RowVec<DT>::store_one(row, e0 + i, out[i]);
  }
}

// VPL, the experts per lane: the smallest power of two that covers E
template <class F>
hipError_t per_lane(int E, F&& go) {
  if (E <= 64) return go(std::integral_constant<int, 1>());
  if (E <= 128) return go(std::integral_constant<int, 2>());
  if (E <= 256) return go(std::integral_constant<int, 4>());
  if (E <= 512) return go(std::integral_constant<int, 8>());
  return go(std::integral_constant<int, 16>());
}

// the log of the lanes of vpl experts that hold a group, -1 when they are not
// 2^0..2^4 whole lanes
int group_lanes(int group_size, int vpl) {
  for (int l = 0; l <= 4; ++l)
    if (group_size == vpl << l) return l;
  return -1;
}

// Tokens from which a wave takes four.  Where keys have errors, some token of
// nearly every large batch goes to a whole wave after that, and the kernel
// ends with the last.  Measured one / four per wave, 128 experts, top 8, bf16
// softmax: 2048 tokens 4.0 / 3.9 us, 4096 4.5 / 3.9, 16384 10.0 / 5.9, 65536
// 32 / 17; 256 experts, top 8 of 4 of 8 groups, fp32 sigmoid with a bias: 4096
// 8.7 / 11.3, 8192 10.4 / 11.0, 16384 17.9 / 15.0, 65536 60 / 38.
constexpr int kRowsTokens = 4096, kRowsTokensScored = 10240;

template <int DT>
hipError_t topk_dt(RouterArgs a, hipStream_t stream) {
  const size_t lds = a.groups > 1 ? (size_t)kRouterWaves * a.E * sizeof(uint64_t) : 0;
  a.group_size = a.E / a.groups;
  const bool scored = a.bias != nullptr || a.group_top > 1;
  return per_lane(a.E, [&](auto vpl) {
    constexpr int VPL = decltype(vpl)::value;
    a.group_lanes_log = group_lanes(a.group_size, VPL);
    if constexpr (VPL <= 4) {
      constexpr int RVPL = 4 * VPL;         // experts per lane of a row
      a.row_lanes_log = group_lanes(a.group_size, RVPL);
      if (a.T >= (scored ? kRowsTokensScored : kRowsTokens) && a.E > 16 && a.k < 16 && (a.groups == 1 || a.row_lanes_log >= 0)) {
        const dim3 grid = grid_of((a.T + 4 * kRouterWaves - 1) / (4 * kRouterWaves));
        router_rows_kernel<DT, RVPL, VPL><<<grid, 64 * kRouterWaves, lds, stream>>>(a);
        return hipGetLastError();
      }
    }
    const dim3 grid = grid_of((a.T + kRouterWaves - 1) / kRouterWaves);
    router_topk_kernel<DT, VPL><<<grid, 64 * kRouterWaves, lds, stream>>>(a);
    return hipGetLastError();
  });
}

template <int DT>
hipError_t grad_dt(const RouterArgs& a, const int32_t* ids, const float* grad_w, void* grad_logits,
                   hipStream_t stream) {
  const dim3 grid = grid_of((a.T + kRouterWaves - 1) / kRouterWaves);
  return per_lane(a.E, [&](auto vpl) {
    router_grad_kernel<DT, decltype(vpl)::value>
        <<<grid, 64 * kRouterWaves, 0, stream>>>(a, ids, grad_w, (uint8_t*)grad_logits);
    return hipGetLastError();
  });
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
