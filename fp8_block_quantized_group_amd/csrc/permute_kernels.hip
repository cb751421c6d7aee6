// Token rows sorted by expert and combined back, with their gradients.
//
// The routed slots (t, j) -- an id in [0, E), a token that is no padding --
// get the rows of their experts in expert order, within an expert in
// ascending slot order, as moe_stage lays them out.
//   permute            rows[slot_row[t, j]] = x[t]
//   its gradient       grad_x[t] = sum_j grad_rows[slot_row[t, j]]
//   unpermute          out[t] = sum_j w[t, j] rows[slot_row[t, j]]
//   its gradients      grad_rows[r] = w grad_out[t], grad_w[t, j] = <grad_out[t], rows[r]>
// Sums run over j ascending in fp32 and are rounded once.
//
// The rows' kernels are streams, bound by HBM: one 16-byte vector per lane
// and row, a token's rows all in flight together.  Rows are read and written
// once and are larger than the caches: non-temporal, both ways (loads through
// the caches: 204 us against 188 for the combine below); a permuted token was
// just written by the kernel before and is read through the caches (108 us
// with non-temporal loads, 91 without).  MI355X, where a 2 GiB copy moves
// 5.1 TB/s: permute 4096 x 8 rows of 7168 bf16 columns 84 us (528 MB, 6.3
// TB/s), combine 16384 x 8 x 4096 bf16 188 us (1.15 GB, 6.1 TB/s), its
// gradients 417 us (2.17 GB, 5.2 TB/s).
#include <type_traits>

#include "kernels.h"
#include "row_vec.h"

namespace moe {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortRounds = kSortChunk / kSortThreads;
// Up to this many chunks every ranking block adds up the chunks before it, 16
// loads in flight; above, one block turns the counts into first rows for all
// of them (at 32 chunks, 256 experts: 5.9 us here, 11.4 + 5.5 in two kernels).
// That block goes chunk by chunk: 16384 x 8 slots of 256 experts 17 us, 65536 x
// 8 63 us, beside 103 and 424 us of rows of 2048 bf16 columns.
constexpr int kSortInline = 64;

// the slot's expert, -1 when it is unrouted
__device__ __forceinline__ int routed_id(const int32_t* ids, const uint8_t* pad, int64_t slot,
                                         int k, int E) {
  const int id = ids[slot];
  if (id < 0 || id >= E) return -1;
  if (pad != nullptr && pad[(uint32_t)slot / (uint32_t)k] != 0) return -1;   // slots < 2^31
  return id;
}

// Slots are ranked in chunks by a block each: latency, not bytes (4096 x 8
// slots: 4.6 us to count, 5.9 to rank).

// per chunk of slots, how many go to each expert
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

// exclusive scan of one value per thread over the block
__device__ __forceinline__ int block_exclusive_scan(int v, int* wave_total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wave_total[wave] = incl;
  __syncthreads();
  for (int w = 0; w < wave; ++w) incl += wave_total[w];
  return incl - v;
}

// One block: thread e turns its expert's counts into the chunks' first rows
// and the experts' offsets.
__global__ __launch_bounds__(1024) void sort_scan_kernel(const SortArgs a, int chunks) {
  __shared__ int wave_total[16];
  const int e = threadIdx.x;
  int count = 0;
  if (e < a.E) {
#pragma unroll 16
    for (int b = 0; b < chunks; ++b) count += a.hist[(int64_t)b * a.E + e];
  }
  int base = block_exclusive_scan(count, wave_total);
  if (e >= a.E) return;
  a.expert_offsets[e] = base;
  if (e == a.E - 1) a.expert_offsets[a.E] = base + count;
  for (int b = 0; b < chunks; ++b) {
    const int n = a.hist[(int64_t)b * a.E + e];
    a.hist[(int64_t)b * a.E + e] = base;
    base += n;
  }
}

// The row of every slot of a chunk: the first row of its expert in the chunk
// plus the slots of that expert before it.  A wave ranks 256 consecutive
// slots, 64 at a time: lanes with the same expert find each other by ballots
// over its bits, and the wave's own counter per expert carries the rest;
// then the threads turn the waves' counts into first rows.  SCANNED: hist holds
// the chunk's first rows; else the counts, which every block adds up itself.
template <bool SCANNED, int PER>
__global__ __launch_bounds__(kSortThreads) void sort_rank_kernel(const SortArgs a, int chunks) {
  extern __shared__ int32_t counts[];       // [kSortWaves][E]
  __shared__ int wave_total[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E;
  int32_t* mine = counts + wave * E;
  for (int e = lane; e < E; e += 64) mine[e] = 0;
  wave_lds_order();
  const int64_t slot0 = (int64_t)blockIdx.x * kSortChunk + wave * (64 * kSortRounds) + lane;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  int id[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t slot = slot0 + 64 * r;
    id[r] = slot < a.slots ? routed_id(a.ids, a.is_padding, slot, a.k, E) : -1;
  }
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    uint64_t same = __ballot(id[r] >= 0);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const uint64_t m = __ballot((id[r] >> b) & 1);
      same &= ((id[r] >> b) & 1) ? m : ~m;
    }
    const int before = __popcll(same & below);
    rank[r] = 0;
    if (id[r] >= 0) {
      rank[r] = mine[id[r]] + before;
      wave_lds_order();
      if (before == 0) mine[id[r]] = rank[r] + __popcll(same);
    }
    wave_lds_order();
  }
  __syncthreads();
  // a thread per PER consecutive experts: the first row of the chunk's slots
  // of each, then of each wave's (an expert past the last reads the last one's
  // counts: no load behind a branch)
  const int e0 = threadIdx.x * PER;
  int total[PER] = {}, prior[PER] = {}, sum = 0;
  if (!SCANNED) {
    int at[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) at[i] = min(e0 + i, E - 1);
    if (chunks == 1) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) total[i] += counts[w * E + at[i]];
    } else {
      constexpr int kBatch = 16;              // chunks whose counts load together
      for (int b0 = 0; b0 < chunks; b0 += kBatch) {
        int n[kBatch][PER];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int i = 0; i < PER; ++i)
            n[u][i] = a.hist[(int64_t)min(b0 + u, chunks - 1) * E + at[i]];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            prior[i] += b0 + u < (int)blockIdx.x ? n[u][i] : 0;
            total[i] += b0 + u < chunks ? n[u][i] : 0;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += e0 + i < E ? total[i] : 0;
  }
  int first = SCANNED ? 0 : block_exclusive_scan(sum, wave_total);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i;
    if (e >= E) continue;
    int base = SCANNED ? a.hist[(int64_t)blockIdx.x * E + e] : first + prior[i];
    if (!SCANNED && blockIdx.x == 0) {
      a.expert_offsets[e] = first;
      if (e == E - 1) a.expert_offsets[E] = first + total[i];
    }
    first += total[i];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = counts[w * E + e];
      counts[w * E + e] = base;
      base += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t slot = slot0 + 64 * r;
    if (slot >= a.slots) continue;
    const int row = id[r] >= 0 ? mine[id[r]] + rank[r] : -1;
    a.slot_row[slot] = row;
    if (row >= 0) a.row_slot[row] = (int)slot;
  }
}

// The streaming kernels' lanes in (token, vector) form: `blocks` blocks share
// `tokens` tokens, each with `pitch` lanes, a power of two or whole blocks;
// where that leaves an eighth of the lanes or more idle, as many lanes as a
// row has vectors, vector after vector over up to 16 blocks.  Whole calls with
// pitches alone / so: 11598 x 3 rows of 531 fp16 columns (67 vectors) combined
// 16.1 / 12.1 us, 4096 x 8 x 7168 bf16 (896) permuted, the sort with it, 104 / 100
// and combined 94 / 87; with 118 of 128 lanes in use it would cost 5 %.
struct Split {
  int tokens, blocks;
  int vectors;           // of a row
  int pitch;
  float inv;             // 1 / pitch
};
struct Place {
  int64_t t;
  int v;                 // vector of the row
};
// t = T when the lane has none
__device__ __forceinline__ Place place(const Split& s, int64_t T) {
  const uint32_t b = block_index();
  const uint32_t group = b / (uint32_t)s.blocks;
  const int flat = (int)(b - group * (uint32_t)s.blocks) * 256 + (int)threadIdx.x;
  // exact: flat is below 2^14, (flat + 0.5) / pitch 0.5 / pitch off an integer
  const int local = (int)(((float)flat + 0.5f) * s.inv);
  const int v = flat - local * s.pitch;
  return Place{local < s.tokens && v < s.vectors ? (int64_t)group * s.tokens + local : T, v};
}

// A lane's column where its vector would pass the row's end: the row's last
// N columns.  The columns that the lane before it has too come out the same
// from both.

// the rows themselves: a token's vector is read once and written to the rows
// of its routed slots
template <class RV>
__global__ __launch_bounds__(256) void permute_rows_kernel(const RowsArgs a, const Split s) {
  const Place p = place(s, a.T);
  if (p.t >= a.T) return;
  const int col = RV::inside(p.v * RV::N, a.H);
  const int64_t pitch = (int64_t)a.H * RV::kSize;
  const typename RV::Raw v = RV::template load_at<false>(a.in + p.t * pitch, col);
  for (int j = 0; j < a.k; ++j) {
    const int r = a.slot_row[p.t * a.k + j];
    if (r >= 0 && r < a.slots) RV::template store_at<true>(a.out + r * pitch, col, v);
  }
}

// Sort and rows in one launch, for few slots: a block per 256 vectors of a
// token finds the rows of the token's slots by comparing each with all slots
// (lanes hold slots, a ballot counts 64 comparisons), and copies.  The blocks
// of a token's first vectors write its slots' rows; the waves share out the
// offsets, each the count of the slots of lower experts.
constexpr int kSmallBatch = 256;            // slots compared per loop turn

template <class RV>
__global__ __launch_bounds__(256) void permute_small_kernel(const RowsArgs a, const SortArgs s,
                                                            int pieces) {
  extern __shared__ int32_t lds[];          // ids [ids], then rows [k]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = (int)a.slots, k = a.k;
  const int ids = (n + kSmallBatch - 1) / kSmallBatch * kSmallBatch;
  int32_t* rows = lds + ids;
  const int t = blockIdx.x / pieces, piece = blockIdx.x - t * pieces;
  const int v0 = (piece * 256 + threadIdx.x) * RV::N;
  const int col = RV::inside(min(v0, a.H - 1), a.H);
  const int64_t pitch = (int64_t)a.H * RV::kSize;
  const typename RV::Raw v = RV::template load_at<false>(a.in + t * pitch, col);
  for (int i = threadIdx.x; i < ids; i += 256)
    lds[i] = i < n ? routed_id(s.ids, s.is_padding, i, k, s.E) : -1;
  __syncthreads();
  // how many slots go before (id, slot): those of lower experts, and of the
  // same one those with a lower slot
  auto before = [&](int id, int slot) {
    int c = 0;
    for (int i = 0; i < ids; i += kSmallBatch) {
#pragma unroll
      for (int u = 0; u < kSmallBatch; u += 64) {
        const int o = lds[i + u + lane];
        c += __popcll(__ballot(o >= 0 && (o < id || (o == id && i + u + lane < slot))));
      }
    }
    return c;
  };
  for (int j = wave; j < k; j += 4) {
    const int slot = t * k + j;
    const int id = __builtin_amdgcn_readfirstlane(lds[slot]);
    const int row = id >= 0 ? before(id, slot) : -1;
    if (lane == 0) {
      rows[j] = row;
      if (piece == 0) {
        s.slot_row[slot] = row;
        if (row >= 0) s.row_slot[row] = slot;
      }
    }
  }
  for (int e = blockIdx.x * 4 + wave; e <= s.E; e += gridDim.x * 4) {
    const int c = before(e, 0);
    if (lane == 0) s.expert_offsets[e] = c;
  }
  __syncthreads();
  if (v0 >= a.H) return;
  for (int j = 0; j < k; ++j)
    if (rows[j] >= 0) RV::template store_at<true>(a.out + rows[j] * pitch, col, v);
}

// the sum of a token's rows, weighted when weights are given
template <class RV>
__global__ __launch_bounds__(256) void combine_rows_kernel(const RowsArgs a, const Split s) {
  constexpr int N = RV::N;
  const Place p = place(s, a.T);
  if (p.t >= a.T) return;
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
// product with the token's gradient summed as the rows go by.  The rows may be
// overwritten by their gradients: a lane writes the columns that it alone
// reads (the last vector's first ones may still be waited for by another wave).
template <class RV, int WIDTH>
__global__ __launch_bounds__(256) void combine_grad_kernel(const RowsArgs a,
                                                           const uint8_t* rows,
                                                           float* __restrict__ grad_w) {
  constexpr int N = RV::N;
  __shared__ float part[4][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)block_index() * (256 / WIDTH) + (WIDTH == 64 ? wave : 0);
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
        RV::template store_tail<true>(a.out + r[u] * pitch, col, v0, RV::pack(d));
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

Split split_rows(int H, int N) {
  const int nv = (H + N - 1) / N;
  Split s{1, (nv + 255) / 256, nv, 0, 0.0f};
  s.pitch = 256 * s.blocks;
  for (; s.pitch / 2 >= nv && s.tokens < 256; s.pitch /= 2) s.tokens *= 2;
  if (8 * nv <= 7 * s.pitch) {
    s.tokens = 1;                          // the fewest that fill their blocks best
    for (int n = 2; n * nv <= 4096; ++n) {
      const int blocks = (n * nv + 255) / 256;
      if (n * s.blocks > s.tokens * blocks) s.tokens = n, s.blocks = blocks;
    }
    s.pitch = nv;
  }
  s.inv = 1.0f / (float)s.pitch;
  return s;
}

hipError_t launch_sort(const SortArgs& a, hipStream_t stream) {
  const int64_t chunks = (a.slots + kSortChunk - 1) / kSortChunk;
  const size_t lds = kSortWaves * a.E * sizeof(int32_t);
  const bool scan = chunks == 0 || chunks > kSortInline;
  if (chunks > 1)
    sort_count_kernel<<<(unsigned)chunks, kSortThreads, a.E * sizeof(int32_t), stream>>>(a);
  if (scan) sort_scan_kernel<<<1, 1024, 0, stream>>>(a, (int)chunks);
  if (chunks == 0) return hipGetLastError();
  auto rank = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    if (scan)
      sort_rank_kernel<true, PER><<<(unsigned)chunks, kSortThreads, lds, stream>>>(a, (int)chunks);
    else
      sort_rank_kernel<false, PER><<<(unsigned)chunks, kSortThreads, lds, stream>>>(a, (int)chunks);
    return hipGetLastError();
  };
  if (a.E <= kSortThreads) return rank(std::integral_constant<int, 1>());
  if (a.E <= 2 * kSortThreads) return rank(std::integral_constant<int, 2>());
  return rank(std::integral_constant<int, 4>());
}

// One launch for the sort and the rows up to this many slots and comparisons
// per block (a token's slots times all slots).  Measured in one launch and in
// two or three, 256 experts: 64 tokens x 8 slots of 7168 columns 6.4 / 8.5
// us, 256 x 8 12.4 / 14.2, 500 x 8 27.1 / 18.9; 2000 x 1 of 1024 columns 7.7
// / 11.1, 4000 x 1 21.0 / 12.1.
constexpr int64_t kSmallSlots = 2048, kSmallCompares = 16384;

// sort != nullptr: permute, after the sort; else combine
template <class RV>
hipError_t stream_rows(const RowsArgs& a, const SortArgs* sort, hipStream_t stream) {
  const Split split = split_rows(a.H, RV::N);
  const dim3 grid = grid_of((a.T + split.tokens - 1) / split.tokens * split.blocks);
  if (sort == nullptr) {
    combine_rows_kernel<RV><<<grid, 256, 0, stream>>>(a, split);
  } else if (a.slots <= kSmallSlots && a.k * a.slots <= kSmallCompares) {
    const size_t lds = (size_t)(a.slots + kSmallBatch - 1 + a.k) * sizeof(int32_t);
    const int pieces = (split.vectors + 255) / 256;
    permute_small_kernel<RV><<<(unsigned)(a.T * pieces), 256, lds, stream>>>(a, *sort, pieces);
  } else {
    const hipError_t err = launch_sort(*sort, stream);
    if (err != hipSuccess) return err;
    permute_rows_kernel<RV><<<grid, 256, 0, stream>>>(a, split);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t rows_dt(const RowsArgs& a, const SortArgs* sort, hipStream_t stream) {
  return a.H < RowVec<DT>::N ? stream_rows<RowOne<DT>>(a, sort, stream)
                             : stream_rows<RowVec<DT>>(a, sort, stream);
}

template <int DT>
hipError_t combine_grad_dt(const RowsArgs& a, const uint8_t* rows, float* grad_w,
                           hipStream_t stream) {
  const dim3 waves = grid_of((a.T + 3) / 4);
  if (a.H < RowVec<DT>::N)
    combine_grad_kernel<RowOne<DT>, 64><<<waves, 256, 0, stream>>>(a, rows, grad_w);
  else if (a.H <= 256 * RowVec<DT>::N)
    combine_grad_kernel<RowVec<DT>, 64><<<waves, 256, 0, stream>>>(a, rows, grad_w);
  else
    combine_grad_kernel<RowVec<DT>, 256><<<grid_of(a.T), 256, 0, stream>>>(a, rows, grad_w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_permute(const SortArgs& sort, const RowsArgs& a, int dtype,
                          hipStream_t stream) {
  if (a.T == 0) return launch_sort(sort, stream);        // the offsets alone
  switch (dtype) {
    case kBf16: return rows_dt<kBf16>(a, &sort, stream);
    case kF16: return rows_dt<kF16>(a, &sort, stream);
    default: return rows_dt<kF32>(a, &sort, stream);
  }
}

hipError_t launch_combine_rows(const RowsArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kBf16: return rows_dt<kBf16>(a, nullptr, stream);
    case kF16: return rows_dt<kF16>(a, nullptr, stream);
    default: return rows_dt<kF32>(a, nullptr, stream);
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
