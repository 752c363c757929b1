// The block-FP8 product for few rows of a group, bounded by the weights' bytes and, for a
// single row, by latency: one launch, rows quantised where they are used, no shared operand.
//
// A CTA takes 16 outputs of up to eight rows of a group.  Its eight warps share the blocks of
// 128 along the contraction: a warp loads a block's 16 x 128 weights straight into the
// fragments of warp MMAs (m16n8k32, the order of K relabelled alike on both sides, see
// mma_e4m3_k64), so that all of a CTA's weights are on their way at once and nothing waits
// for a barrier before the sums of the warps are added, in warp order, at the end.  The lanes
// of a row's fragment hold 32 of its 128 values each, so a group's largest is two shuffles
// away and a bf16 row needs no launch in front that quantises it.
//
// One bf16 row x 2048 x 2560 takes 3.9 us (5.2 MB of weights: 0.8 us at HBM's rate; launch, one
// round of loads, the sums' exchange), 4.8 where the weights come from HBM; eight rows 4.3;
// eight rows of eight experts of 1024 x 2048 5.9.  With 16 rows to a CTA (two products of each
// fragment) the same sizes took 6.3, 6.7 and 8.8 us: twice the quantisation in each warp.
#include "rows_device.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBatch = 2;   // blocks whose weights a warp has on their way
constexpr int kRows = 8;    // rows of a group to a CTA

// The tile of rows with this number: its group, first row and rows (0: there is none).
struct RowTile {
  int g, row0, n;
};

__device__ __forceinline__ RowTile row_tile(const LinArgs& a, int item, RowTile* s) {
  if (!a.starts) return RowTile{0, item * kRows, min(kRows, a.rows - item * kRows)};
  if (threadIdx.x < 32) {
    constexpr int kPer = kMaxExperts / 32;
    const int lane = threadIdx.x;
    int start[kPer], count[kPer], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = kPer * lane + i;
      start[i] = count[i] = 0;
      if (g < a.groups) {
        const int s0 = __ldg(a.starts + g), s1 = __ldg(a.starts + g + 1);
        start[i] = min(max(s0, 0), a.rows);
        const int end = min(max(s1, start[i]), a.rows);
        count[i] = end - start[i];
        bad |= start[i] != s0 || end != s1;
      }
      sum += (count[i] + kRows - 1) / kRows;
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kOpsBadOrder);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31 && item >= incl) *s = RowTile{0, 0, 0};
    int at = item - (incl - sum);  // among this lane's groups' tiles
    if (at >= 0 && at < sum) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int tiles = (count[i] + kRows - 1) / kRows;
        if (at >= 0 && at < tiles)
          *s = RowTile{kPer * lane + i, start[i] + kRows * at, min(kRows, count[i] - kRows * at)};
        at -= tiles;
      }
    }
  }
  __syncthreads();
  return *s;
}

// 32 values of a block of a bf16 row (16 from each half of the block, for the lane's
// quarter) as codes, with the block's scale.
__device__ __forceinline__ void quant32(const bf16* row, int c, int width, bool on, uint4 (&b)[2],
                                        float* scale) {
  float v[2][16], m = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    unpack16(load16(row, c + 64 * h, width, on), v[h]);
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[h][i]));
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  *scale = quant_codes<2, true>(v, m, b);
}

template <bool kCodes>
__global__ void __launch_bounds__(kThreads) k_linear_rows(const __grid_constant__ LinArgs a,
                                                          const bf16* x, int64_t x_stride,
                                                          const uint8_t* codes, const uint8_t* w) {
  __shared__ RowTile s_tile;
  __shared__ float red[kWarps][kRows][17];  // (17: rows apart by other banks)
  const RowTile t = row_tile(a, blockIdx.y, &s_tile);
  if (t.n <= 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q = lane & 3;
  const int n0 = 16 * blockIdx.x, blocks = groups_of(a.inner);
  const uint8_t* w0 = w + ((size_t)t.g * a.outer + n0 + r) * a.inner;
  const uint8_t* w8 = w0 + (size_t)8 * a.inner;
  const float* sw = a.sw + ((size_t)t.g * groups_of(a.outer) + n0 / kGroup) * blocks;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool on = r < t.n;                      // lane's row, of the B fragments
  const int64_t row = t.row0 + (on ? r : 0);
  for (int b0 = warp; b0 < blocks; b0 += kBatch * kWarps) {
    uint4 lo[kBatch][2], hi[kBatch][2];
    float ws[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int b = b0 + k * kWarps;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = b * kGroup + 64 * h + 16 * q;
        lo[k][h] = hi[k][h] = make_uint4(0u, 0u, 0u, 0u);
        if (c < a.inner) {
          lo[k][h] = ld_stream16(w0 + c);
          hi[k][h] = ld_stream16(w8 + c);
        }
      }
      ws[k] = b < blocks ? __ldg(sw + b) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int b = b0 + k * kWarps;
      if (b >= blocks) break;
      const int c = b * kGroup + 16 * q;
      uint4 v[2];
      float s;
      if constexpr (kCodes) {
        const uint8_t* p = codes + row * a.inner;
        v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u);
        if (on && c < a.inner) v[0] = __ldg(reinterpret_cast<const uint4*>(p + c));
        if (on && c + 64 < a.inner) v[1] = __ldg(reinterpret_cast<const uint4*>(p + c + 64));
        s = __ldg(a.sx + row * blocks + b);
      } else {
        quant32(x + row * x_stride, c, a.inner, on, v, &s);
      }
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma_e4m3_k64(d, lo[k][0], hi[k][0], v[0]);
      mma_e4m3_k64(d, lo[k][1], hi[k][1], v[1]);
      // columns 2q and 2q + 1 of the products are the rows of lanes 8q and 8q + 4
      const float s0 = ws[k] * __shfl_sync(0xffffffffu, s, 8 * q);
      const float s1 = ws[k] * __shfl_sync(0xffffffffu, s, 8 * q + 4);
      acc[0] = fmaf(d[0], s0, acc[0]);
      acc[1] = fmaf(d[1], s1, acc[1]);
      acc[2] = fmaf(d[2], s0, acc[2]);
      acc[3] = fmaf(d[3], s1, acc[3]);
    }
  }
  red[warp][2 * q][r] = acc[0];
  red[warp][2 * q + 1][r] = acc[1];
  red[warp][2 * q][r + 8] = acc[2];
  red[warp][2 * q + 1][r + 8] = acc[3];
  __syncthreads();
  const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
  if (m < t.n) {
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) y += red[i][m][n];
    a.y[(t.row0 + m) * a.y_stride + n0 + n] = __float2bfloat16_rn(y);
  }
}

}  // namespace

cudaError_t launch_linear_rows(const LinArgs& a, const bf16* x, int64_t x_stride,
                               const uint8_t* codes, const uint8_t* w, cudaStream_t s) {
  // (the most there can be; a tile that is not there ends at once)
  const int tiles = a.starts ? a.rows / kRows + (a.groups < a.rows ? a.groups : a.rows)
                             : (a.rows + kRows - 1) / kRows;
  const dim3 grid(a.outer / 16, tiles);
  if (codes)
    k_linear_rows<true><<<grid, kThreads, 0, s>>>(a, x, x_stride, codes, w);
  else
    k_linear_rows<false><<<grid, kThreads, 0, s>>>(a, x, x_stride, codes, w);
  return cudaGetLastError();
}

}  // namespace moe
