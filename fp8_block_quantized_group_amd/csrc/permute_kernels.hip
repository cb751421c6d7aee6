// Token rows sorted by expert and combined back, with their gradients.
//
// The routed slots (t, j) -- an id in [0, E), a token that is no padding --
// get the rows of their experts in expert order, within an expert in
// ascending slot order, as moe_stage lays them out.
//   permute            rows[slot_row[t, j]] = x[t]
//   its gradient       grad_x[t] = sum_j grad_rows[slot_row[t, j]]
//   unpermute          out[t] = sum_j w[t, j] rows[slot_row[t, j]]
//   its gradients      grad_rows[r] = w grad_out[t], grad_w[t, j] = <grad_out[t], rows[r]>
// Sums run over j ascending in fp32 and are rounded once.  Every kernel is a
// stream over the rows: one 16-byte vector per lane and row.
#include "kernels.h"
#include "row_vec.h"

namespace moe {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortRounds = kSortChunk / kSortThreads;

__device__ __forceinline__ int routed_id(const int32_t* ids, const uint8_t* pad, int64_t slot,
                                         int k, int E) {
  const int id = ids[slot];
  if (id < 0 || id >= E) return -1;
  if (pad != nullptr && pad[slot / k] != 0) return -1;
  return id;
}

// 1: per chunk of slots, how many go to each expert
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const SortArgs a) {
  extern __shared__ int32_t h[];
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) h[e] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t slot = (int64_t)blockIdx.x * kSortChunk + r * kSortThreads + threadIdx.x;
    if (slot >= a.slots) continue;
    const int id = routed_id(a.ids, a.is_padding, slot, a.k, a.E);
    if (id >= 0) atomicAdd(&h[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads)
    a.hist[(int64_t)blockIdx.x * a.E + e] = h[e];
}

// 2: one block; thread e turns its expert's counts into the chunks' first
// rows and the experts' offsets
__global__ __launch_bounds__(1024) void sort_scan_kernel(const SortArgs a, int chunks) {
  __shared__ int wave_total[16];
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
  int count = 0;
  if (e < a.E)
    for (int b = 0; b < chunks; ++b) count += a.hist[(int64_t)b * a.E + e];
  int incl = count;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_total[wave] = incl;
  __syncthreads();
  for (int w = 0; w < wave; ++w) incl += wave_total[w];
  if (e < a.E) {
    int base = incl - count;
    a.expert_offsets[e] = base;
    if (e == a.E - 1) a.expert_offsets[a.E] = incl;
    for (int b = 0; b < chunks; ++b) {
      const int n = a.hist[(int64_t)b * a.E + e];
      a.hist[(int64_t)b * a.E + e] = base;
      base += n;
    }
  }
}

// 3: the row of every slot: the chunk's first row of its expert plus the
// slots of that expert before it in the chunk
__global__ __launch_bounds__(kSortThreads) void sort_rank_kernel(const SortArgs a) {
  extern __shared__ int32_t next[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < a.E; e += kSortThreads)
    next[e] = a.hist[(int64_t)blockIdx.x * a.E + e];
  __syncthreads();
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t slot = (int64_t)blockIdx.x * kSortChunk + r * kSortThreads + threadIdx.x;
    const int id = slot < a.slots ? routed_id(a.ids, a.is_padding, slot, a.k, a.E) : -1;
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < 10; ++b) {
      const uint64_t m = __ballot((id >> b) & 1);
      same &= ((id >> b) & 1) ? m : ~m;
    }
    const int before = __popcll(same & below);
    for (int w = 0; w < kSortThreads / 64; ++w) {
      if (wave == w && id >= 0) {
        const int row = next[id] + before;
        if (before == 0) next[id] = row + __popcll(same);
        a.slot_row[slot] = row;
        a.row_slot[row] = (int)slot;
      }
      __syncthreads();
    }
    if (id < 0 && slot < a.slots) a.slot_row[slot] = -1;
  }
}

// Lanes of a block in (token, vector) form: `width` lanes (a power of two)
// side by side on one token's row, 256 / width tokens per block.
struct Place {
  int64_t t;
  int v;          // vector of the row
};
__device__ __forceinline__ Place place(int log_width, int pieces) {
  const int64_t b = blockIdx.x;
  const int64_t piece = b % pieces;
  const int64_t group = b / pieces;
  return Place{(group << (8 - log_width)) + (threadIdx.x >> log_width),
               (int)(piece << log_width) + (int)(threadIdx.x & ((1 << log_width) - 1))};
}

// A lane's column where its vector would pass the row's end: the row's last
// N columns.  The columns that the lane before it has too come out the same
// from both.

// 4: the rows themselves: a token's vector is read once and written to the
// rows of its routed slots
template <class RV>
__global__ __launch_bounds__(256) void permute_rows_kernel(const RowsArgs a, int log_width,
                                                           int pieces) {
  const Place p = place(log_width, pieces);
  if (p.t >= a.T || p.v * RV::N >= a.H) return;
  const int col = RV::inside(p.v * RV::N, a.H);
  const int64_t pitch = (int64_t)a.H * RV::kSize;
  const typename RV::Raw v = RV::template load_at<true>(a.in + p.t * pitch, col);
  for (int j = 0; j < a.k; ++j) {
    const int r = a.slot_row[p.t * a.k + j];
    if (r >= 0 && r < a.slots) RV::template store_at<true>(a.out + r * pitch, col, v);
  }
}

// the sum of a token's rows, weighted when weights are given
template <class RV>
__global__ __launch_bounds__(256) void combine_rows_kernel(const RowsArgs a, int log_width,
                                                           int pieces) {
  constexpr int N = RV::N;
  const Place p = place(log_width, pieces);
  if (p.t >= a.T || p.v * N >= a.H) return;
  const int col = RV::inside(p.v * N, a.H);
  const int64_t pitch = (int64_t)a.H * RV::kSize;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    int r[8];
    float w[8];
    typename RV::Raw v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      r[u] = -1;
      w[u] = 1.0f;
      if (j0 + u < a.k) {
        r[u] = a.slot_row[p.t * a.k + j0 + u];
        if (r[u] >= a.slots) r[u] = -1;
        if (a.weights != nullptr) w[u] = a.weights[p.t * a.k + j0 + u];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (r[u] >= 0) v[u] = RV::template load_at<true>(a.in + r[u] * pitch, col);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (r[u] < 0) continue;
      float f[N];
      RV::unpack(v[u], f);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(w[u], f[i], acc[i]);
    }
  }
  RV::template store_at<true>(a.out + p.t * pitch, col, RV::pack(acc));
}

// Gradients of the weighted sum, WIDTH lanes (a wave or the block) per
// token: for 8 slots at a time, the row's gradient is written and its
// product with the token's gradient summed as the rows go by.
template <class RV, int WIDTH>
__global__ __launch_bounds__(256) void combine_grad_kernel(const RowsArgs a,
                                                           const uint8_t* __restrict__ rows,
                                                           float* __restrict__ grad_w) {
  constexpr int N = RV::N;
  __shared__ float part[4][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * (256 / WIDTH) + (WIDTH == 64 ? wave : 0);
  if (t >= a.T) return;                  // whole waves (WIDTH 64) or never
  const int first = WIDTH == 64 ? lane : (int)threadIdx.x;
  const int64_t pitch = (int64_t)a.H * RV::kSize;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    int r[8];
    float w[8], dot[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      r[u] = -1;
      w[u] = 1.0f;
      dot[u] = 0.0f;
      if (j0 + u < a.k) {
        r[u] = a.slot_row[t * a.k + j0 + u];
        if (r[u] >= a.slots) r[u] = -1;
        if (a.weights != nullptr) w[u] = a.weights[t * a.k + j0 + u];
      }
    }
    for (int v0 = first * N; v0 < a.H; v0 += WIDTH * N) {
      const int col = RV::inside(v0, a.H);
      // columns that the lane before has too stay out of the products
      const typename RV::Raw mine = RV::mask_from(v0 - col);
      float g[N], own[N];
      RV::unpack(RV::template load_at<false>(a.in + t * pitch, col), g);
      typename RV::Raw v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (r[u] >= 0) v[u] = RV::template load_at<true>(rows + r[u] * pitch, col);
#pragma unroll
      for (int i = 0; i < N; ++i) own[i] = col + i >= v0 ? g[i] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (r[u] < 0) continue;
        float f[N], d[N];
        RV::unpack(v[u] & mine, f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot[u] = fmaf(own[i], f[i], dot[u]);
          d[i] = w[u] * g[i];
        }
        RV::template store_at<true>(a.out + r[u] * pitch, col, RV::pack(d));
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) dot[u] = wave_sum(dot[u]);
    if (WIDTH == 256) {
      __syncthreads();
      if (lane == 0) {
#pragma unroll
        for (int u = 0; u < 8; ++u) part[wave][u] = dot[u];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 8; ++u) dot[u] = part[0][u] + part[1][u] + part[2][u] + part[3][u];
    }
    if (first == 0) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < a.k) grad_w[t * a.k + j0 + u] = r[u] >= 0 ? dot[u] : 0.0f;
    }
  }
}

// lanes per token and pieces per row of the streaming kernels
void split_row(int H, int N, int* log_width, int* pieces) {
  const int nv = (H + N - 1) / N;
  *log_width = 0;
  while (*log_width < 8 && (1 << *log_width) < nv) ++*log_width;
  *pieces = (nv + (1 << *log_width) - 1) >> *log_width;
}

template <class RV>
hipError_t stream_rows(const RowsArgs& a, bool permute, hipStream_t stream) {
  int log_width, pieces;
  split_row(a.H, RV::N, &log_width, &pieces);
  const int per_block = 256 >> log_width;
  const int64_t grid = (a.T + per_block - 1) / per_block * pieces;
  if (grid >= (int64_t)1 << 31) return hipErrorInvalidValue;
  if (permute) permute_rows_kernel<RV><<<(unsigned)grid, 256, 0, stream>>>(a, log_width, pieces);
  else combine_rows_kernel<RV><<<(unsigned)grid, 256, 0, stream>>>(a, log_width, pieces);
  return hipGetLastError();
}

template <int DT>
hipError_t rows_dt(const RowsArgs& a, bool permute, hipStream_t stream) {
  return a.H < RowVec<DT>::N ? stream_rows<RowOne<DT>>(a, permute, stream)
                             : stream_rows<RowVec<DT>>(a, permute, stream);
}

template <int DT>
hipError_t combine_grad_dt(const RowsArgs& a, const uint8_t* rows, float* grad_w,
                           hipStream_t stream) {
  const unsigned waves = (unsigned)((a.T + 3) / 4);
  if (a.H < RowVec<DT>::N)
    combine_grad_kernel<RowOne<DT>, 64><<<waves, 256, 0, stream>>>(a, rows, grad_w);
  else if (a.H <= 256 * RowVec<DT>::N)
    combine_grad_kernel<RowVec<DT>, 64><<<waves, 256, 0, stream>>>(a, rows, grad_w);
  else
    combine_grad_kernel<RowVec<DT>, 256><<<(unsigned)a.T, 256, 0, stream>>>(a, rows, grad_w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sort(const SortArgs& a, hipStream_t stream) {
  const int chunks = (int)((a.slots + kSortChunk - 1) / kSortChunk);
  if (chunks > 0)
    sort_count_kernel<<<chunks, kSortThreads, a.E * sizeof(int32_t), stream>>>(a);
  sort_scan_kernel<<<1, 1024, 0, stream>>>(a, chunks);
  if (chunks > 0)
    sort_rank_kernel<<<chunks, kSortThreads, a.E * sizeof(int32_t), stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_permute_rows(const RowsArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kBf16: return rows_dt<kBf16>(a, true, stream);
    case kF16: return rows_dt<kF16>(a, true, stream);
    default: return rows_dt<kF32>(a, true, stream);
  }
}

hipError_t launch_combine_rows(const RowsArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kBf16: return rows_dt<kBf16>(a, false, stream);
    case kF16: return rows_dt<kF16>(a, false, stream);
    default: return rows_dt<kF32>(a, false, stream);
  }
}

hipError_t launch_combine_grad(const RowsArgs& a, const void* rows, float* grad_w, int dtype,
                               hipStream_t stream) {
  switch (dtype) {
    case kBf16: return combine_grad_dt<kBf16>(a, (const uint8_t*)rows, grad_w, stream);
    case kF16: return combine_grad_dt<kF16>(a, (const uint8_t*)rows, grad_w, stream);
    default: return combine_grad_dt<kF32>(a, (const uint8_t*)rows, grad_w, stream);
  }
}

}  // namespace moe
