// Rows to their experts and back: the stable sort of (token, rank) pairs by expert, the
// gather of token rows into that order, the weighted sum of the experts' rows, and the
// gradients.
//
//   slot(p) = starts[e(p)] + #{p' < p : e(p') = e(p)}        pairs p = t k + j
//   dispatch       rows[slot(t, j)] = x[t]                    dx[t] = sum_j drows[slot(t, j)]
//   combine        y[t] = sum_j w[t, j] rows[slot(t, j)]      drows[slot] = w[t, j] dy[t]
//                                                             dw[t, j] = dy[t] . rows[slot]
//
// The rows' bytes bound all of it (a row moves once each way); the sort is a few
// microseconds in front.  No atomics order anything: a pair's slot follows from counts.
//   16384 tokens of 2048, eight experts of 256 each:  98 us, 93 % of the copy's rate (the
//   gather 89; the order alone 7 us);  to codes 61 us (85 %)
//   11 tokens to codes 3.4 us, one launch;  weighted back: 16384 tokens 91 us (100 %), one 2.6
//   the gather's gradient, 5003 tokens of 2560, four of six pairs each: 24 us (79 %)
#include "rows_device.cuh"

namespace moe {

namespace {

// Experts of a pair outside [0, E) have no slot.
__device__ __forceinline__ bool there(int e, int E) { return (unsigned)e < (unsigned)E; }

// Exclusive prefix over v[0..E) in place, by one warp; v[E] = the total.
__device__ __forceinline__ void scan_experts(int* v, int E) {
  const int lane = threadIdx.x & 31;
  int loc[kMaxExperts / 32], sum = 0;
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    const int e = (kMaxExperts / 32) * lane + i;
    loc[i] = e < E ? v[e] : 0;
    sum += loc[i];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  int run = incl - sum;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    const int e = (kMaxExperts / 32) * lane + i;
    if (e < E) v[e] = run;
    run += loc[i];
  }
  if (lane == 31) v[E] = incl;
}

// Rows t0 .. t0 + n - 1 of x to their slots (slots[(t - t0) k + j], -1: none), by the
// whole block.
template <bool kCodes>
__device__ __forceinline__ void gather_rows(const bf16* x, int64_t x_stride, int width, int t0,
                                            int n, int k, const int* slots, const RowsOut& out) {
  if constexpr (kCodes) {
    const int groups = groups_of(width), sub = threadIdx.x & 7;
    const int units = n * groups, per = blockDim.x >> 3;
    for (int u0 = 0; u0 < units; u0 += per) {  // the same for the whole block
      const int u = u0 + (threadIdx.x >> 3);
      const int i = u / groups, c = (u - i * groups) * kGroup + 16 * sub;
      const bool on = u < units;
      float v[16], s;
      unpack16(load16(x + (int64_t)(t0 + i) * x_stride, c, width, on), v);
      const uint4 q = quant16<true>(v, &s);
      if (!on || c >= width) continue;
      for (int j = 0; j < k; ++j) {
        const int slot = slots[i * k + j];
        if (slot < 0) continue;
        *reinterpret_cast<uint4*>(out.codes + (size_t)slot * width + c) = q;
        if (sub == 0) out.scales[(size_t)slot * groups + c / kGroup] = s;
      }
    }
  } else {
    const int vecs = width / 8, all = n * vecs;
    for (int u = threadIdx.x; u < all; u += blockDim.x) {
      const int i = u / vecs, c = 8 * (u - i * vecs);
      const uint4 v = *reinterpret_cast<const uint4*>(x + (int64_t)(t0 + i) * x_stride + c);
      for (int j = 0; j < k; ++j) {
        const int slot = slots[i * k + j];
        if (slot >= 0) *reinterpret_cast<uint4*>(out.v + (int64_t)slot * out.stride + c) = v;
      }
    }
  }
}

// ---- few pairs: one launch --------------------------------------------------------
// Every block counts all pairs itself (in front of its own tokens and in all), so that no
// block waits for another; then it places its tokens' pairs and gathers their rows.
// Up to 1536 tokens of eight pairs, near where both ways take as long (order, and rows of
// 2048, this way and the other: 64 tokens 3.1 and 5.8 us, 1024 8.9 and 11.4, 1500 11.9 and
// 13.2, 2048 17.4 and 16.2, 4096 38.8 and 31.0).
constexpr int kSmallThreads = 512;
constexpr int kSmallPairs = 12288;

template <bool kCodes>
__global__ void __launch_bounds__(kSmallThreads) k_dispatch_small(OrderArgs o, const int* idx,
                                                                  const bf16* x, int64_t x_stride,
                                                                  int width, RowsOut out,
                                                                  int per_block) {
  __shared__ int all[kMaxExperts + 1], before[kMaxExperts];
  extern __shared__ int own[];  // [per_block k] experts, then their slots
  const int P = o.T * o.k, tid = threadIdx.x;
  const int t0 = blockIdx.x * per_block, n = min(per_block, o.T - t0);
  const int p0 = t0 * o.k, np = n * o.k;
  for (int e = tid; e <= o.E; e += kSmallThreads) {
    all[e] = 0;
    if (e < o.E) before[e] = 0;
  }
  __syncthreads();
#pragma unroll 4
  for (int p = tid; p < P; p += kSmallThreads) {
    const int e = __ldg(idx + p);
    if (there(e, o.E)) {
      atomicAdd(&all[e], 1);
      if (p < p0) atomicAdd(&before[e], 1);
    }
    if (p >= p0 && p < p0 + np) own[p - p0] = e;
  }
  __syncthreads();
  if (tid < 32) scan_experts(all, o.E);
  __syncthreads();
  int* slots = own + per_block * o.k;
  for (int i = tid; i < np; i += kSmallThreads) {
    const int e = own[i];
    int slot = -1;
    if (there(e, o.E)) {
      slot = all[e] + before[e];
      for (int q = 0; q < i; ++q) slot += own[q] == e;
      o.pair_of_slot[slot] = p0 + i;
    }
    slots[i] = slot;
    o.slot_of_pair[p0 + i] = slot;
  }
  if (blockIdx.x == 0)
    for (int e = tid; e <= o.E; e += kSmallThreads) o.starts[e] = all[e];
  for (int p = all[o.E] + blockIdx.x * kSmallThreads + tid; p < P; p += gridDim.x * kSmallThreads)
    o.pair_of_slot[p] = -1;
  if (!x) return;
  __syncthreads();
  gather_rows<kCodes>(x, x_stride, width, t0, n, o.k, slots, out);
}

// ---- many pairs: count, place, gather -----------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
static_assert(kSortPairs == 2 * kSortThreads, "two pairs to a thread");

__global__ void __launch_bounds__(kSortThreads) k_sort_count(OrderArgs o, const int* idx,
                                                             int* hist) {
  __shared__ int n[kMaxExperts];
  for (int e = threadIdx.x; e < o.E; e += kSortThreads) n[e] = 0;
  __syncthreads();
  const int P = o.T * o.k;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = blockIdx.x * kSortPairs + i * kSortThreads + threadIdx.x;
    const int e = p < P ? __ldg(idx + p) : -1;
    if (there(e, o.E)) atomicAdd(&n[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < o.E; e += kSortThreads) hist[blockIdx.x * o.E + e] = n[e];
  pdl_trigger();
}

// The lanes whose expert this lane's is, bit by bit (__match_any_sync takes a turn for each
// expert among the lanes: 1.2 us more).
__device__ __forceinline__ unsigned same_expert(int e, bool in) {
  unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
  for (int b = 1; b < kMaxExperts; b <<= 1) {
    const unsigned set = __ballot_sync(0xffffffffu, e & b);
    same &= e & b ? set : ~set;
  }
  return same;
}

// Warp w takes the block's pairs 64 w .. 64 w + 63.  A pair's place among its expert's is
// the count of the blocks in front, of the warps in front, and of the lanes in front.
__global__ void __launch_bounds__(kSortThreads) k_sort_place(OrderArgs o, const int* idx,
                                                             const int* hist, int blocks) {
  __shared__ int all[kMaxExperts + 1], base[kMaxExperts];
  __shared__ unsigned short of_warp[kSortWarps][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = o.T * o.k;
  for (int e = tid; e <= kMaxExperts; e += kSortThreads) {
    all[e] = 0;
    if (e < kMaxExperts) base[e] = 0;
  }
  for (int i = tid; i < kSortWarps * kMaxExperts; i += kSortThreads) (&of_warp[0][0])[i] = 0;
  __syncthreads();
  int e[2], rank[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = blockIdx.x * kSortPairs + 64 * warp + 32 * i + lane;
    e[i] = p < P ? __ldg(idx + p) : -1;
    const bool in = there(e[i], o.E);
    const unsigned same = same_expert(e[i], in);
    const unsigned lower = same & ((1u << lane) - 1);
    rank[i] = __popc(lower) + (in ? of_warp[warp][e[i]] : 0);
    __syncwarp();
    if (in && lower == 0) of_warp[warp][e[i]] += (unsigned short)__popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int c = tid; c < o.E; c += kSortThreads) {  // the warps' counts -> those in front
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = of_warp[w][c];
      of_warp[w][c] = (unsigned short)run;
      run += n;
    }
  }
  pdl_wait();
  pdl_trigger();
  // the blocks' counts: in all and in front, by up to four threads to an expert
  const int split = kSortThreads / kMaxExperts, c = tid % kMaxExperts, part = tid / kMaxExperts;
  if (c < o.E) {
    int sum = 0, front = 0;
#pragma unroll 8
    for (int b = part; b < blocks; b += split) {
      const int n = __ldcg(hist + b * o.E + c);
      sum += n;
      front += b < (int)blockIdx.x ? n : 0;
    }
    atomicAdd(&all[c], sum);
    atomicAdd(&base[c], front);
  }
  __syncthreads();
  if (warp == 0) scan_experts(all, o.E);
  __syncthreads();
  const int kept = all[o.E];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = blockIdx.x * kSortPairs + 64 * warp + 32 * i + lane;
    if (p >= P) continue;
    int slot = -1;
    if (there(e[i], o.E)) {
      slot = all[e[i]] + base[e[i]] + of_warp[warp][e[i]] + rank[i];
      o.pair_of_slot[slot] = p;
    }
    o.slot_of_pair[p] = slot;
    if (p >= kept) o.pair_of_slot[p] = -1;
  }
  if (blockIdx.x == 0)
    for (int i = tid; i <= o.E; i += kSortThreads) o.starts[i] = all[i];
}

constexpr int kGatherThreads = 256;

template <bool kCodes>
__global__ void __launch_bounds__(kGatherThreads) k_gather(OrderArgs o, const bf16* x,
                                                           int64_t x_stride, int width,
                                                           RowsOut out) {
  pdl_wait();
  const int t = blockIdx.x;
  gather_rows<kCodes>(x, x_stride, width, t, 1, o.k, o.slot_of_pair + (size_t)t * o.k, out);
}

// ---- back ----------------------------------------------------------------------------
constexpr int kBackThreads = 256;

// The slot of pair p, -1 where it has none (a slot outside the rows is reported).
__device__ __forceinline__ int slot_of(const OrderArgs& o, int p, int* status) {
  const int s = __ldg(o.slot_of_pair + p);
  if (s < o.T * o.k) return s < 0 ? -1 : s;
  atomicOr(status, kOpsBadOrder);
  return -1;
}

// A block takes up to 256 vectors of 8 columns of a token, a thread one of them: its rows'
// loads go out together, four rows at a time, and the products are added in rank order.
// (16384 tokens of eight rows of 2048: 91 us, the bytes' floor 90; with eight rows at a time
// and four blocks to an SM 98, without a bound on registers 125.)
__global__ void __launch_bounds__(kBackThreads, 6) k_combine(OrderArgs o, const bf16* rows,
                                                             int64_t rows_stride, const float* w,
                                                             int width, bf16* y, int64_t y_stride,
                                                             int* status) {
  const int t = blockIdx.x, c = 8 * (int)(blockIdx.y * blockDim.x + threadIdx.x);
  if (c >= width) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  constexpr int kAhead = 4;
  for (int j0 = 0; j0 < o.k; j0 += kAhead) {
    int slot[kAhead];
    float wt[kAhead];
    uint4 v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      slot[j] = j0 + j < o.k ? slot_of(o, t * o.k + j0 + j, status) : -1;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (slot[j] >= 0) v[j] = ld_stream16(rows + (int64_t)slot[j] * rows_stride + c);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) wt[j] = w && j0 + j < o.k ? __ldg(w + t * o.k + j0 + j) : 1.0f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (slot[j] < 0) continue;
      float x[8];
      unpack8(v[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(wt[j], x[i], acc[i]);
    }
  }
  *reinterpret_cast<uint4*>(y + (int64_t)t * y_stride + c) = pack8(acc);
}

// A warp takes a pair: the dot product of dy with its row, and the row's gradient.  4099 tokens
// of eight rows of 2048 in bf16: 44 us, 96 % of the copy's rate; to codes 45 us, 73 %: the
// quotients keep the schedulers busy in two thirds of the cycles, and the next columns are
// asked for behind them.  (Five blocks to an SM; 60 us without a bound on
// registers; a block to a token, with dy and its groups' magnitudes kept for all of its pairs,
// 52.)
template <bool kCodes>
__global__ void __launch_bounds__(kBackThreads, 5) k_combine_grad(OrderArgs o, const bf16* dy,
                                                               int64_t dy_stride, const bf16* rows,
                                                               int64_t rows_stride, const float* w,
                                                               int width, RowsOut out, float* dw,
                                                               int* status) {
  const int p = blockIdx.x * (kBackThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (p >= o.T * o.k) return;
  const int slot = slot_of(o, p, status);
  if (slot < 0) {
    if (lane == 0) dw[p] = 0.0f;
    return;
  }
  const bf16* d = dy + (int64_t)(p / o.k) * dy_stride;
  const bf16* r = rows + (int64_t)slot * rows_stride;
  const float wt = __ldg(w + p);
  float dot = 0.0f;
#pragma unroll 1
  for (int c0 = 0; c0 < width; c0 += 512) {
    const int c = c0 + 16 * lane;
    const Vec16 rd = load16(d, c, width, true), rr = load16(r, c, width, true);
    float v[16], x[16];
    unpack16(rd, v);
    unpack16(rr, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      dot = fmaf(v[i], x[i], dot);
      v[i] *= wt;
    }
    put16<kCodes, false>(out, slot, c, width, true, v);
  }
  dot = warp_sum(dot);
  if (lane == 0) dw[p] = dot;
}

}  // namespace

cudaError_t launch_dispatch(const OrderArgs& o, const int* idx, const bf16* x, int64_t x_stride,
                            int width, const RowsOut& out, int* hist, int sm_count,
                            cudaStream_t s) {
  const int P = o.T * o.k;
  const bool codes = out.codes != nullptr;
  if (P <= kSmallPairs) {
    const int per = (o.T + sm_count - 1) / sm_count, grid = (o.T + per - 1) / per;
    const size_t smem = (size_t)2 * per * o.k * sizeof(int);
    if (codes)
      k_dispatch_small<true><<<grid, kSmallThreads, smem, s>>>(o, idx, x, x_stride, width, out,
                                                               per);
    else
      k_dispatch_small<false><<<grid, kSmallThreads, smem, s>>>(o, idx, x, x_stride, width, out,
                                                                per);
    return cudaGetLastError();
  }
  const int blocks = (P + kSortPairs - 1) / kSortPairs;
  k_sort_count<<<blocks, kSortThreads, 0, s>>>(o, idx, hist);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_pdl(k_sort_place, dim3(blocks), dim3(kSortThreads), 0, s, true, o, idx, hist,
                   blocks);
  if (e == cudaSuccess && x)
    e = launch_pdl(codes ? k_gather<true> : k_gather<false>, dim3(o.T), dim3(kGatherThreads), 0, s,
                   true, o, x, x_stride, width, out);
  return e;
}

cudaError_t launch_combine_rows(const OrderArgs& o, const bf16* rows, int64_t rows_stride,
                                const float* w, int width, bf16* y, int64_t y_stride, int* status,
                                cudaStream_t s) {
  const int vecs = width / 8, chunks = (vecs + kBackThreads - 1) / kBackThreads;
  const int threads = ((vecs + chunks - 1) / chunks + 31) & ~31;
  k_combine<<<dim3(o.T, chunks), threads, 0, s>>>(o, rows, rows_stride, w, width, y, y_stride,
                                                  status);
  return cudaGetLastError();
}

cudaError_t launch_combine_grad(const OrderArgs& o, const bf16* dy, int64_t dy_stride,
                                const bf16* rows, int64_t rows_stride, const float* w, int width,
                                const RowsOut& out, float* dw, int* status, cudaStream_t s) {
  const int per = kBackThreads / 32, grid = (o.T * o.k + per - 1) / per;
  if (out.codes)
    k_combine_grad<true><<<grid, kBackThreads, 0, s>>>(o, dy, dy_stride, rows, rows_stride, w,
                                                       width, out, dw, status);
  else
    k_combine_grad<false><<<grid, kBackThreads, 0, s>>>(o, dy, dy_stride, rows, rows_stride, w,
                                                        width, out, dw, status);
  return cudaGetLastError();
}

}  // namespace moe
