// The block-FP8 product on the tcgen05 tensor cores: rows of e4m3 codes with a scale for
// each 128 values, times e4m3 weights with a scale for each 128 x 128 block, dense or each
// row by its group's weights.
//
//   y[r][n] = sum_b  sx[r][b] sw[n / 128][b]  sum_{c in block b} x[r][c] W[n][c]
//   trans:    sx[r][b] sw[b][n / 128]  sum_{c in block b} x[r][c] W[c][n]
//
// A tile is 128 rows by 256 outputs.  The scales change with every block of 128 along the
// contraction, so the MMAs of a block (four of K = 32) write a fresh product into one of two
// TMEM buffers, and eight warps add it, times its scale, to fp32 sums in registers while the
// tensor cores fill the other.  With the rows along the TMEM lanes a thread has one row and
// the columns of one weight block: one scale to a thread and block of the contraction, and
// one FMA to a product.  (The weights along the lanes, as the layer's own products have
// them, want a scale from shared memory for every column.)
//
// Warps: 0-7 the sums and the store (warp w: lanes 32 (w % 4) and on, columns 128 (w / 4)
// and on), 8 the TMA loads, 9 the MMAs.  Persistent: a CTA takes tiles blockIdx.x,
// + gridDim.x, ..; the tiles of a group's 128 rows lie next to each other.
#include "attn_tc.cuh"
#include "ops_internal.cuh"

namespace moe {

namespace {

constexpr int kBM = 128, kBN = 256, kKB = 128;
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kSumWarps + 2);
constexpr int kWarpTma = kSumWarps, kWarpMma = kSumWarps + 1;
constexpr int kABytes = kBM * kKB, kBBytes = kBN * kKB, kStageBytes = kABytes + kBBytes;
constexpr int kStages = 4;
constexpr int kSmallBox = 32;                  // rows of a small box of x
constexpr int kOutBytes = 32 * 32 * 2;         // a warp's piece of the output: 32 x 32
constexpr uint32_t kIdescBMajorN = 1u << 16;

struct LinSmem {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int abort;
  int pre[kMaxExperts + 1];    // row tiles in front of each group
  int start[kMaxExperts + 1];  // the group's first row
  int count[kMaxExperts];
};
constexpr size_t kSmemBytes =
    1024 + (size_t)kStages * kStageBytes + kSumWarps * kOutBytes + sizeof(LinSmem);
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

struct Tile {
  int g, f, row0, n;  // group, column tile, first row, rows
};

__device__ __forceinline__ Tile tile_of(const LinSmem& sm, int groups, int cols, int w) {
  const int t = w / cols;
  int lo = 0, hi = groups;  // the last group with pre <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sm.pre[mid] <= t) lo = mid; else hi = mid;
  }
  const int j = t - sm.pre[lo];
  return Tile{lo, w - t * cols, sm.start[lo] + kBM * j, min(kBM, sm.count[lo] - kBM * j)};
}

// Clamped bounds of every group's rows and the prefix of their row tiles, by the block.
__device__ __forceinline__ void group_tiles(const LinArgs& a, LinSmem& sm) {
  for (int g = threadIdx.x; g < a.groups; g += kThreads) {
    int r0 = 0, r1 = a.rows;
    if (a.starts) {
      const int s0 = __ldg(a.starts + g), s1 = __ldg(a.starts + g + 1);
      r0 = min(max(s0, 0), a.rows);
      r1 = min(max(s1, r0), a.rows);
      if ((r0 != s0 || r1 != s1) && blockIdx.x == 0) atomicOr(a.status, kOpsBadOrder);
    }
    sm.start[g] = r0;
    sm.count[g] = r1 - r0;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    constexpr int kPer = kMaxExperts / 32;
    const int lane = threadIdx.x;
    int loc[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = kPer * lane + i;
      loc[i] = g < a.groups ? (sm.count[g] + kBM - 1) / kBM : 0;
      sum += loc[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = kPer * lane + i;
      if (g < a.groups) sm.pre[g] = run;
      run += loc[i];
    }
    if (lane == 31) sm.pre[a.groups] = incl;
  }
  __syncthreads();
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, LinSmem& sm,
                                         int* status) {
  const bool ok = tc::wait_bounded(bar, parity, &sm.abort, status);
  return !__any_sync(0xffffffffu, !ok);
}

// A warp's 32 x 32 outputs (lane: row) through its piece of shared memory, so that stores
// cover 64 bytes of each of eight rows.  16-byte units of a row are permuted by its number.
__device__ __forceinline__ void store_piece(uint8_t* piece, const float* v, bf16* y,
                                            int64_t y_stride, int rows, int cols) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(piece + 64 * lane + 16 * ((c ^ (lane >> 1)) & 3)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  const int c = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 q = *reinterpret_cast<const uint4*>(piece + 64 * r + 16 * ((c ^ (r >> 1)) & 3));
    if (r < rows && 8 * c < cols) *reinterpret_cast<uint4*>(y + (int64_t)r * y_stride + 8 * c) = q;
  }
  __syncwarp();
}

template <bool kTrans>
__global__ void __launch_bounds__(kThreads, 1) k_linear(const __grid_constant__ LinArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* pieces = stages + kStages * kStageBytes;
  LinSmem& sm = *reinterpret_cast<LinSmem*>(pieces + kSumWarps * kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.tfull[i], 1);
      tc::mbar_init(&sm.tempty[i], kSumWarps);
    }
    sm.abort = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch_map(&a.x);
    tc::tma_prefetch_map(&a.xs);
    tc::tma_prefetch_map(&a.w);
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  pdl_wait();
  tc::fence_before_sync();
  group_tiles(a, sm);
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const int cols = (a.outer + kBN - 1) / kBN, blocks = (a.inner + kKB - 1) / kKB;
  const int tiles = sm.pre[a.groups] * cols;

  if (warp == kWarpTma) {
    uint32_t st = 0, ph = 0;
    int issued = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < tiles && ok; w += gridDim.x) {
      const Tile t = tile_of(sm, a.groups, cols, w);
      // more than half a tile of rows in one box (rows behind the group's do no harm: each
      // row's products are its own), fewer in small boxes
      const int boxes = 2 * t.n > kBM ? 0 : (t.n + kSmallBox - 1) / kSmallBox;
      // the second half of the tile's columns, where there are any
      const int halves = a.outer - t.f * kBN > kBN / 2 ? 2 : 1;
      const uint32_t bytes =
          (boxes ? boxes * kSmallBox * kKB : kABytes) + halves * (kBBytes / 2);
      for (int b = 0; b < blocks; ++b) {
        if (!wait_all(&sm.empty[st], ph ^ 1u, sm, a.status)) {
          ok = false;
          break;
        }
        uint8_t* sa = stages + st * kStageBytes;
        uint8_t* sb = sa + kABytes;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&sm.full[st], bytes);
          if (boxes == 0)
            tc::tma_load_2d(sa, &a.x, b * kKB, t.row0, &sm.full[st]);
          else
            for (int i = 0; i < boxes; ++i)
              tc::tma_load_2d(sa + i * kSmallBox * kKB, &a.xs, b * kKB, t.row0 + i * kSmallBox,
                              &sm.full[st]);
          for (int h = 0; h < halves; ++h) {
            const int n0 = t.f * kBN + h * (kBN / 2);
            tc::tma_load_3d(sb + h * (kBBytes / 2), &a.w, kTrans ? n0 : b * kKB,
                            kTrans ? b * kKB : n0, t.g, &sm.full[st]);
          }
        }
        __syncwarp();
        ++issued;
        if (++st == kStages) { st = 0; ph ^= 1u; }
      }
    }
    if (!ok && lane == 0) {
      // copies in flight land before the CTA leaves
      const unsigned long long t0 = tc::global_ns();
      for (int i = 1; i <= kStages && i <= issued; ++i) {
        const int k = issued - i;
        while (!tc::mbar_try_wait(&sm.full[k % kStages], (uint32_t)((k / kStages) & 1)) &&
               tc::global_ns() - t0 < tc::kWaitLimitNs) {
        }
      }
    }
  } else if (warp == kWarpMma) {
    const uint32_t leader = lane == 0;
    const tc::Desc da = tc::desc_of(tc::smem_u32(stages), true);
    const tc::Desc db = tc::desc_of(tc::smem_u32(stages + kABytes), true,
                                    kTrans ? kBBytes / 2 : 16);
    uint32_t st = 0, ph = 0, tb = 0, tph = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < tiles && ok; w += gridDim.x) {
      const int left = a.outer - (w % cols) * kBN;
      const uint32_t idesc = tc::idesc_f8(kBM, left > kBN / 2 ? kBN : kBN / 2) |
                             (kTrans ? kIdescBMajorN : 0u);
      for (int b = 0; b < blocks; ++b) {
        ok = wait_all(&sm.tempty[tb], tph ^ 1u, sm, a.status) &&
             wait_all(&sm.full[st], ph, sm, a.status);
        if (!ok) break;
        tc::fence_after_sync();
        const tc::Desc xa = da + st * kStageBytes, xb = db + st * kStageBytes;
#pragma unroll
        for (int k = 0; k < kKB / 32; ++k)
          // 32 values along a row of 128 bytes; 32 rows of them where the rows run along N
          tc::mma_ss<true>(tmem + tb * kBN, xa + 32 * k, xb + (kTrans ? 32 * kKB : 32) * k, idesc,
                           k > 0, leader);
        tc::commit_by(&sm.empty[st], leader);
        tc::commit_by(&sm.tfull[tb], leader);
        if (++st == kStages) { st = 0; ph ^= 1u; }
        if ((tb ^= 1u) == 0) tph ^= 1u;
      }
    }
  } else {
    const int q = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * (kBN / 2);
    uint8_t* piece = pieces + warp * kOutBytes;
    const int nb_out = (a.outer + kGroup - 1) / kGroup;
    uint32_t tb = 0, tph = 0;
    for (int w = blockIdx.x; w < tiles; w += gridDim.x) {
      const Tile t = tile_of(sm, a.groups, cols, w);
      const int r = 32 * q + lane;               // this thread's row of the tile
      const int c0 = t.f * kBN + half * (kBN / 2);  // this warp's first column
      const bool live = 32 * q < t.n && c0 < a.outer;  // any output in this warp
      const float* sx = a.sx + (size_t)(t.row0 + min(r, t.n - 1)) * blocks;
      const float* sw = a.sw + (size_t)t.g * nb_out * blocks;
      const int cb = min(c0 / kGroup, nb_out - 1);
      sw += kTrans ? cb : cb * blocks;
      const int sw_step = kTrans ? nb_out : 1;
      float acc[kBN / 2];
#pragma unroll
      for (int i = 0; i < kBN / 2; ++i) acc[i] = 0.0f;
      float next = __ldg(sx) * __ldg(sw);
      for (int b = 0; b < blocks; ++b) {
        const float s = next;
        if (b + 1 < blocks) next = __ldg(sx + b + 1) * __ldg(sw + (size_t)(b + 1) * sw_step);
        // (a wait that gave up leaves the sums undefined; the loop still ends)
        tc::wait_bounded(&sm.tfull[tb], tph, &sm.abort, a.status);
        __syncwarp();
        tc::fence_after_sync();
        if (live) {
#pragma unroll
          for (int i = 0; i < kBN / 2; i += 32) {
            uint32_t v[32];
            tc::tmem_ld_async(lanes + tb * kBN + i, v);
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[i + j] = fmaf(__uint_as_float(v[j]), s, acc[i + j]);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.tempty[tb]);
        if ((tb ^= 1u) == 0) tph ^= 1u;
      }
      if (!live || sm.abort) continue;
      bf16* y = a.y + (int64_t)(t.row0 + 32 * q) * a.y_stride + c0;
#pragma unroll
      for (int i = 0; i < kBN / 2; i += 32)
        store_piece(piece, acc + i, y + i, a.y_stride, t.n - 32 * q, a.outer - c0 - i);
    }
  }
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t setup_linear() {
  const cudaError_t e = cudaFuncSetAttribute(
      k_linear<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_linear<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kSmemBytes);
}

cudaError_t launch_linear(const LinArgs& a, bool trans, int sm_count, bool pdl, cudaStream_t s) {
  const long long cols = (a.outer + kBN - 1) / kBN;
  // at most a part tile for each group that has rows
  const long long tiles =
      ((long long)a.rows / kBM + (a.groups < a.rows ? a.groups : a.rows)) * cols;
  const int grid = (int)(tiles < sm_count ? tiles : sm_count);
  return launch_pdl(trans ? k_linear<true> : k_linear<false>, dim3(grid), dim3(kThreads),
                    kSmemBytes, s, pdl, a);
}

}  // namespace moe
