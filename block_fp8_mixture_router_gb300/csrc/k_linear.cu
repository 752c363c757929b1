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
// and on), 8 the TMA loads, 9 and 10 the MMAs, 11 the scales.  Persistent: a CTA takes tiles blockIdx.x,
// + gridDim.x, ..; the tiles of a group's 128 rows lie next to each other.
#include "attn_tc.cuh"
#include "ops_internal.cuh"

namespace moe {

namespace {

constexpr int kBM = 128, kBN = 256, kKB = 128;
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kSumWarps + 4);
constexpr int kWarpTma = kSumWarps, kWarpMma = kSumWarps + 1, kWarpScale = kSumWarps + 3;
// Registers of a thread: twelve warps start with 168 (65536 / 384, by eights); the two
// warpgroups that hold 128 sums and 64 products on their way give and take with the third.
constexpr int kSumRegs = 208, kOtherRegs = 88;
static_assert(2 * kSumRegs + kOtherRegs <= 3 * 168, "no more registers than at launch");
constexpr int kABytes = kBM * kKB, kBBytes = kBN * kKB, kStageBytes = kABytes + kBBytes;
constexpr int kStages = 3;
constexpr int kSmallBox = 32;                  // rows of a small box of x
constexpr int kOutBytes = 32 * 128 * 2;        // a warp's piece of the output: 32 x 128
constexpr uint32_t kIdescBMajorN = 1u << 16;

struct Tile {
  int g, f, row0, n;  // group, column tile, first row, rows
};

struct LinSmem {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int abort;
  Tile tile[4];                // tiles j, j + 1, .. of this CTA, by j % 4
  float scale[2][2][kBM];      // of a buffer's products, by column half and row
  int pre[kMaxExperts + 1];    // row tiles in front of each group
  int start[kMaxExperts + 1];  // the group's first row
  int count[kMaxExperts];
};
constexpr size_t kSmemBytes =
    1024 + (size_t)kStages * kStageBytes + kSumWarps * kOutBytes + sizeof(LinSmem);
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

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

template <int kRegs>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}

// Waits for this warp's TMEM loads.  The registers are operands so that no use of them
// moves in front of the wait.
__device__ __forceinline__ void wait_ld_of(uint32_t (&v)[32]) {
#define MOE_IO8(o)                                                                       \
  "+r"(v[o + 0]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]),        \
      "+r"(v[o + 5]), "+r"(v[o + 6]), "+r"(v[o + 7])
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : MOE_IO8(0), MOE_IO8(8), MOE_IO8(16), MOE_IO8(24)::"memory");
#undef MOE_IO8
}

__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], float s) {
#pragma unroll
  for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(v[j]), s, acc[j]);
}

// A warp's 32 x 128 outputs (lane: row) to its piece of shared memory, as two boxes of 64
// columns under the 128-byte swizzle.
__device__ __forceinline__ void stage_piece(uint8_t* piece, const float (&v)[128]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(piece + (c >> 3) * 4096 + 128 * lane + 16 * ((c ^ lane) & 7)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x,
                                             int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n" ::
                   "l"(reinterpret_cast<uint64_t>(map)),
               "r"(tc::smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

// The staged piece to rows row .. row + 31 of y (the first `rows` of them) from column c0 on.
// Whole pieces go by TMA, which cuts off columns behind the last one; a piece that ends
// inside has its rows copied, since the rows behind are another group's.
__device__ __forceinline__ void send_piece(const LinArgs& a, const uint8_t* piece, int row,
                                           int rows, int c0) {
  const int lane = threadIdx.x & 31, cols = a.outer - c0;
  if (rows >= 32) {
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&a.out, piece, c0, row);
      if (cols > 64) tma_store_2d(&a.out, piece + 4096, c0 + 64, row);
      asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
    }
    return;
  }
  __syncwarp();
  bf16* y = a.y + (int64_t)row * a.y_stride + c0;
  const int c = lane & 7;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = 4 * (i & 7) + (lane >> 3), h = i >> 3;
    if (r < rows && 64 * h + 8 * c < cols)
      *reinterpret_cast<uint4*>(y + (int64_t)r * a.y_stride + 64 * h + 8 * c) =
          *reinterpret_cast<const uint4*>(piece + 4096 * h + 128 * r + 16 * ((c ^ r) & 7));
  }
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
      tc::mbar_init(&sm.tfull[i], 2);  // the MMAs' commit and the scale warp
      tc::mbar_init(&sm.tempty[i], kSumWarps);
    }
    sm.abort = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch_map(&a.x);
    tc::tma_prefetch_map(&a.xs);
    tc::tma_prefetch_map(&a.w);
    tc::tma_prefetch_map(&a.out);
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

  if (warp >= kSumWarps) fewer_regs<kOtherRegs>();
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
  } else if (warp < kWarpScale && warp >= kWarpMma) {
    // Two warps take the blocks in turn, one for each buffer: an issuing warp waits for the
    // tensor cores to take its MMAs, then pays for two commits and two barrier waits, and
    // the other's MMAs run meanwhile.
    const uint32_t leader = lane == 0, tb = warp - kWarpMma;
    const tc::Desc da = tc::desc_of(tc::smem_u32(stages), true);
    const tc::Desc db = tc::desc_of(tc::smem_u32(stages + kABytes), true,
                                    kTrans ? kBBytes / 2 : 16);
    uint32_t st = tb % kStages, ph = 0, tph = 0, turn = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < tiles && ok; w += gridDim.x) {
      const int left = a.outer - (w % cols) * kBN;
      const uint32_t idesc = tc::idesc_f8(kBM, left > kBN / 2 ? kBN : kBN / 2) |
                             (kTrans ? kIdescBMajorN : 0u);
      for (int b = 0; b < blocks; ++b, turn ^= 1u) {
        if (turn != tb) continue;
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
        tc::commit_by(&sm.tfull[tb], leader);
        tc::commit_by(&sm.empty[st], leader);
        tph ^= 1u;
        st += 2;
        if (st >= kStages) { st -= kStages; ph ^= 1u; }
      }
    }
  } else if (warp == kWarpScale) {
    // Scales: a lane has rows lane, + 32, + 64 and + 96 of every tile.  Those of two blocks
    // are loaded while the two in front of them are written.
    constexpr int kAhead = 2;
    const int nb_out = (a.outer + kGroup - 1) / kGroup;
    const int sw_step = kTrans ? nb_out : 1;
    uint32_t tb = 0, tph = 0;
    bool ok = true;
    int j = 0;
    for (int w = blockIdx.x; w < tiles && ok; w += gridDim.x, ++j) {
      const Tile t = tile_of(sm, a.groups, cols, w);
      if (lane == 0) sm.tile[j & 3] = t;
      const float* sx[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        sx[r] = a.sx + (size_t)(t.row0 + min(lane + 32 * r, t.n - 1)) * blocks;
      const int cb = 2 * t.f, cb1 = min(cb + 1, nb_out - 1);
      const float* sw = a.sw + (size_t)t.g * nb_out * blocks;
      const float* sw0 = sw + (kTrans ? cb : cb * blocks);
      const float* sw1 = sw + (kTrans ? cb1 : cb1 * blocks);
      float nx[kAhead][4], nw[kAhead][2];
      const auto load = [&](int b0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int b = min(b0 + k, blocks - 1);
#pragma unroll
          for (int r = 0; r < 4; ++r) nx[k][r] = __ldg(sx[r] + b);
          nw[k][0] = __ldg(sw0 + (size_t)b * sw_step);
          nw[k][1] = __ldg(sw1 + (size_t)b * sw_step);
        }
      };
      load(0);
      for (int b0 = 0; b0 < blocks && ok; b0 += kAhead) {
        float p[kAhead][2][4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            p[k][0][r] = nx[k][r] * nw[k][0];
            p[k][1][r] = nx[k][r] * nw[k][1];
          }
        if (b0 + kAhead < blocks) load(b0 + kAhead);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (b0 + k >= blocks || !ok) break;
          ok = wait_all(&sm.tempty[tb], tph ^ 1u, sm, a.status);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sm.scale[tb][0][lane + 32 * r] = p[k][0][r];
            sm.scale[tb][1][lane + 32 * r] = p[k][1][r];
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.tfull[tb]);
          if ((tb ^= 1u) == 0) tph ^= 1u;
        }
      }
    }
  } else {
    more_regs<kSumRegs>();
    const int q = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * (kBN / 2);
    uint8_t* piece = pieces + warp * kOutBytes;
    uint32_t tb = 0, tph = 0;
    int j = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < tiles && ok; w += gridDim.x, ++j) {
      float acc[kBN / 2];
#pragma unroll
      for (int i = 0; i < kBN / 2; ++i) acc[i] = 0.0f;
      Tile t = {0, 0, 0, 0};
      for (int b = 0; b < blocks; ++b) {
        if (!wait_all(&sm.tfull[tb], tph, sm, a.status)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (b == 0) t = sm.tile[j & 3];
        const float s = sm.scale[tb][half][32 * q + lane];
        if (32 * q < t.n && t.f * kBN + half * (kBN / 2) < a.outer) {  // any output here
          const uint32_t from = lanes + tb * kBN;
          uint32_t v0[32], v1[32];
          tc::tmem_ld_async(from, v0);
          wait_ld_of(v0);
          tc::tmem_ld_async(from + 32, v1);
          add_scaled(acc, v0, s);
          wait_ld_of(v1);
          tc::tmem_ld_async(from + 64, v0);
          add_scaled(acc + 32, v1, s);
          wait_ld_of(v0);
          tc::tmem_ld_async(from + 96, v1);
          add_scaled(acc + 64, v0, s);
          wait_ld_of(v1);
          // the buffer is free: the last products are in registers
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.tempty[tb]);
          add_scaled(acc + 96, v1, s);
        } else {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.tempty[tb]);
        }
        if ((tb ^= 1u) == 0) tph ^= 1u;
      }
      const int c0 = t.f * kBN + half * (kBN / 2), rows = t.n - 32 * q;
      if (!ok || rows <= 0 || c0 >= a.outer) continue;
      // the piece is free once the TMA has read the tile before
      asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
      __syncwarp();
      stage_piece(piece, acc);
      send_piece(a, piece, t.row0 + 32 * q, rows, c0);
    }
    asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
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
