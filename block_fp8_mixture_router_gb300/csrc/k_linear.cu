// The block-FP8 product on the tcgen05 tensor cores: rows of e4m3 codes with a scale for
// each 128 values, times e4m3 weights with a scale for each 128 x 128 block, dense or each
// row by its group's weights.
//
//   y[r][n] = sum_b  sx[r][b] sw[n / 128][b]  sum_{c in block b} x[r][c] W[n][c]
//   trans:    sx[r][b] sw[b][n / 128]  sum_{c in block b} x[r][c] W[c][n]
//
// The scales change with every block of 128 along the contraction, so the MMAs of a block
// (four of K = 32) write fresh products into TMEM, and eight warps add them, times their
// scale, to fp32 sums in registers.  With the rows along the TMEM lanes a thread has one row
// and columns of one weight block at a time: one scale to a thread, and one FMA to a product.
// (The weights along the lanes, as the layer's own products have them, want a scale from
// shared memory for every column.)
//
// A tile is 128 rows by 256 columns.  Each block's MMAs (512 cycles) fill one of two TMEM
// buffers while the warps empty the other: copy 32 columns to registers, multiply the 32 in
// front of them, and give the buffer back before the last 32 are multiplied.
//
// 16384 rows x 2048 x 4096 take 109 us, 2.5 PFLOP/s, and the gradient of 131072 rows of 256
// experts of 1024 x 2048 308 us (1.8 PFLOP/s, 3.8 TB/s).  About 900 cycles a block: the
// buffers' exchange (a block's MMAs with their issue and commit take 800 to be seen done,
// its products 400 to be read and 70 to be given back) and the 768 that 48 KB of a block take
// at the 64 bytes a clock that an SM gets from L2 bind it together.  Without the FMAs it is no
// faster, with two thirds of the bytes 3 %, with a quarter of the MMAs 10 %, without all
// three 16 %.  Measured and not kept: pairs of CTAs that share their columns' weights
// (cta_group::2, 256 x 256): no faster (113 us both ways then), and 126 instead of 96 for 1024
// tokens' rows of 256 experts; four buffers of 128 columns: 163 us; clusters that share a
// tile's contraction where tiles are few: 100 rows x 2048 x 2560 13.4 us and more against 12.4.
//
// Warps: 0-7 the sums (warp w: lanes 32 (w % 4) and on, columns 128 (w / 4) and on), 8 the TMA
// loads, 9 and 10 the MMAs, 11 the scales, 12-15 the stores.  Persistent: a CTA takes tiles
// blockIdx.x, + gridDim.x, ..; the tiles of a group's 128 rows lie next to each other.
#include "attn_tc.cuh"
#include "ops_internal.cuh"

namespace moe {

namespace {

constexpr int kBM = 128, kBN = 256, kKB = 128;   // rows, columns and depth of a CTA's tile
constexpr int kSumWarps = 8;
constexpr int kWarpTma = kSumWarps, kWarpMma = kSumWarps + 1, kWarpScale = kSumWarps + 3;
constexpr int kWarpStore = kSumWarps + 4, kStoreWarps = 4;
constexpr int kThreads = 32 * (kWarpStore + kStoreWarps);
// Registers of a thread: sixteen warps start with 128; the two warpgroups that hold 128 sums
// and 64 products on their way take what the others give.
constexpr int kSumRegs = 216, kOtherRegs = 40;
static_assert(2 * kSumRegs + 2 * kOtherRegs <= 4 * 128, "no more registers than at launch");
constexpr int kABytes = kBM * kKB, kBBytes = kBN * kKB, kStageBytes = kABytes + kBBytes;
constexpr int kStages = 3;
constexpr int kHalf = kBN / 2;                   // columns of a box of weights
constexpr int kBufs = 512 / kBN;                 // TMEM buffers of a block's products: 2
constexpr int kSmallBox = 32;                    // rows of a small box of x
constexpr int kOutBytes = 32 * 128 * 2;          // a warp's piece of the output: 32 x 128
constexpr uint32_t kIdescBMajorN = 1u << 16;

struct Tile {
  int g, f, row0, n;  // group, column tile, first row, rows
};

// The scales' warp is at most kBufs + 1 tiles ahead of the sums, and they two ahead of the
// stores.
constexpr int kTiles = 8;
struct LinSmem {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[kBufs], tempty[kBufs];
  uint64_t ofull[kSumWarps], ofree[kSumWarps];  // a warp's piece of the output
  uint32_t tmem;
  int abort;
  Tile tile[kTiles];           // tiles j, j + 1, .. of this CTA, by j % kTiles
  float scale[kBufs][2][kBM];  // of a buffer's products, by column half and row
  unsigned short pre[kMaxExperts + 1];  // row tiles in front of each group
};
// (The dynamic shared memory of a kernel without any static begins at a multiple of 1024
// bytes, which the swizzled tiles need; the kernel checks it.)
constexpr size_t kSmemBytes =
    (size_t)kStages * kStageBytes + kSumWarps * kOutBytes + sizeof(LinSmem);
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

// First row and rows of a group, clamped to the rows there are.
__device__ __forceinline__ int2 group_rows(const LinArgs& a, int g, bool* bad = nullptr) {
  if (!a.starts) return make_int2(0, a.rows);
  const int s0 = __ldg(a.starts + g), s1 = __ldg(a.starts + g + 1);
  const int r0 = min(max(s0, 0), a.rows), r1 = min(max(s1, r0), a.rows);
  if (bad) *bad |= r0 != s0 || r1 != s1;
  return make_int2(r0, r1 - r0);
}

__device__ __forceinline__ Tile tile_of(const LinArgs& a, const LinSmem& sm, int cols, int w) {
  const int t = w / cols;
  int lo = 0, hi = a.groups;  // the last group with pre <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sm.pre[mid] <= t) lo = mid; else hi = mid;
  }
  const int skip = kBM * (t - sm.pre[lo]);
  const int2 r = group_rows(a, lo);
  return Tile{lo, w - t * cols, r.x + skip, min(kBM, r.y - skip)};
}

// The prefix of the groups' row tiles, by the block.
__device__ __forceinline__ void group_tiles(const LinArgs& a, LinSmem& sm) {
  if (threadIdx.x < 32) {
    constexpr int kPer = kMaxExperts / 32;
    const int lane = threadIdx.x;
    int loc[kPer], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = kPer * lane + i;
      loc[i] = 0;
      if (g < a.groups) {
        loc[i] = (group_rows(a, g, &bad).y + kBM - 1) / kBM;
        sum += loc[i];
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && blockIdx.x == 0 && lane == 0) atomicOr(a.status, kOpsBadOrder);
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
      if (g < a.groups) sm.pre[g] = (unsigned short)run;
      run += loc[i];
    }
    // groups that overlap may have any number of tiles: such a call does nothing
    if (lane == 31) sm.pre[a.groups] = (unsigned short)(bad ? 0 : incl);
  }
  __syncthreads();
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, LinSmem& sm,
                                         int* status) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
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

// Two FMAs in one instruction.
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, float s) {
  asm volatile("{\n .reg .b64 a, v, t;\n mov.b64 a, {%0, %1};\n mov.b64 v, {%2, %3};\n"
      " mov.b64 t, {%4, %4};\n fma.rn.f32x2 a, v, t, a;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "r"(v0), "r"(v1), "f"(s));
}

__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], float s) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) fma2(acc[j], acc[j + 1], v[j], v[j + 1], s);
}

// A warp's 32 x 64 outputs of a half (lane: row) to shared memory, as a box under the
// 128-byte swizzle.
__device__ __forceinline__ void stage_piece(uint8_t* piece, const float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(piece + 128 * lane + 16 * ((c ^ lane) & 7)) =
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
  if (rows <= 0 || cols <= 0) return;
  if (rows >= 32) {
    if (lane == 0) tma_store_2d(&a.out, piece, c0, row);
    return;
  }
  bf16* y = a.y + (int64_t)row * a.y_stride + c0;
  const int c = lane & 7;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    if (r < rows && 8 * c < cols)
      *reinterpret_cast<uint4*>(y + (int64_t)r * a.y_stride + 8 * c) =
          *reinterpret_cast<const uint4*>(piece + 128 * r + 16 * ((c ^ r) & 7));
  }
}

template <bool kTrans>
__global__ void __launch_bounds__(kThreads, 1) k_linear(const __grid_constant__ LinArgs a) {
  extern __shared__ __align__(1024) uint8_t stages[];
  uint8_t* pieces = stages + kStages * kStageBytes;
  LinSmem& sm = *reinterpret_cast<LinSmem*>(pieces + kSumWarps * kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(stages) & 1023u) {  // the same for every CTA
    if (threadIdx.x == 0) atomicOr(a.status, kOpsBadBase);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      tc::mbar_init(&sm.tfull[i], 2);  // the MMAs' commit and the scale warp
      tc::mbar_init(&sm.tempty[i], kSumWarps);
    }
    for (int i = 0; i < kSumWarps; ++i) {
      tc::mbar_init(&sm.ofull[i], 1);
      tc::mbar_init(&sm.ofree[i], 1);
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
  const int first = blockIdx.x, step = gridDim.x;
  const int mine = first < tiles ? (tiles - first + step - 1) / step : 0;  // this CTA's tiles

  if (warp >= kSumWarps) fewer_regs<kOtherRegs>();
  if (warp == kWarpTma) {
    uint32_t st = 0, ph = 0;
    int issued = 0;
    bool ok = true;
    for (int w = first; w < tiles && ok; w += step) {
      const Tile t = tile_of(a, sm, cols, w);
      // rows: more than half a tile of them in one box (rows behind the group's do no harm:
      // each row's products are its own), fewer in small boxes; columns: the halves there are
      const int boxes = 2 * t.n > kBM ? 0 : (t.n + kSmallBox - 1) / kSmallBox;
      const int halves = a.outer - t.f * kBN > kHalf ? 2 : 1;
      const uint32_t bytes =
          (boxes ? boxes * kSmallBox * kKB : kABytes) + halves * (kHalf * kKB);
      // this lane's copy: lanes 0-3 the rows, 4 and 5 the weights
      const CUtensorMap* map = nullptr;
      int place = 0, x0 = 0, y0 = 0, g = 0;
      bool along = true;  // the contraction runs along the box's rows of 128 bytes
      if (lane < 4) {
        if (boxes == 0 ? lane == 0 : lane < boxes) map = boxes == 0 ? &a.x : &a.xs;
        place = lane * kSmallBox * kKB;
        y0 = t.row0 + lane * kSmallBox;
      } else if (lane < 4 + halves) {
        map = &a.w;
        place = kABytes + (lane - 4) * (kHalf * kKB);
        x0 = y0 = t.f * kBN + (lane - 4) * kHalf;
        g = t.g;
        along = !kTrans;
      }
      for (int b = 0; b < blocks; ++b) {
        if (!wait_all(&sm.empty[st], ph ^ 1u, sm, a.status)) {
          ok = false;
          break;
        }
        // every lane with a copy issues it at once: one lane after the other's takes the warp
        // 150 cycles each
        if (lane == 0) tc::mbar_arrive_expect_tx(&sm.full[st], bytes);
        __syncwarp();
        if (map) {
          uint8_t* to = stages + st * kStageBytes + place;
          const int at = b * kKB;
          tc::tma_load_3d(to, map, along ? at : x0, along ? y0 : at, g, &sm.full[st]);
        }
        __syncwarp();
        ++issued;
        if (++st == kStages) { st = 0; ph ^= 1u; }
      }
    }
    // every stage's last commits have arrived before the CTA leaves
    for (int i = 0; i < kStages && ok; ++i) {
      ok = wait_all(&sm.empty[st], ph ^ 1u, sm, a.status);
      if (++st == kStages) { st = 0; ph ^= 1u; }
    }
    if (!ok && lane == 0) {
      // and after a wait that gave up, copies in flight have landed
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
                                    kTrans ? kHalf * kKB : 16);
    uint32_t st = tb, ph = 0, tph = 0, turn = 0;
    bool ok = true;
    for (int w = first; w < tiles && ok; w += step) {
      const int left = a.outer - (w % cols) * kBN;
      const uint32_t idesc = tc::idesc_f8(kBM, left > kHalf ? kBN : kHalf) |
                             (kTrans ? kIdescBMajorN : 0u);
      for (int b = 0; b < blocks; ++b, turn ^= 1u) {
        if (turn != tb) continue;
        // (in this order: a stage's phases go to the two warps in turn, and only the buffer's
        // return says that the other's was over, without which its parity means nothing)
        ok = wait_all(&sm.tempty[tb], tph ^ 1u, sm, a.status) &&
             wait_all(&sm.full[st], ph, sm, a.status);
        if (!ok) break;
        tc::fence_after_sync();
        const tc::Desc xa = da + st * kStageBytes, xb = db + st * kStageBytes;
#pragma unroll
        for (int k = 0; k < kKB / 32; ++k) {
          // 32 values along a row of 128 bytes; 32 rows of them where the rows run along N
          const tc::Desc ka = xa + 32 * k, kb = xb + (kTrans ? 32 * kKB : 32) * k;
          tc::mma_ss<true>(tmem + tb * kBN, ka, kb, idesc, k > 0, leader);
        }
        tc::commit_by(&sm.tfull[tb], leader);
        tc::commit_by(&sm.empty[st], leader);
        tph ^= 1u;
        st += 2;
        if (st >= kStages) { st -= kStages; ph ^= 1u; }
      }
    }
  } else if (warp == kWarpScale) {
    // Scales: a lane has rows lane, + 32, + 64 and + 96 of every tile.  Those of the next
    // block, of the next tile's first after a tile's last, are loaded while one is written: a
    // tile that began with its loads would hold the sums up for their latency.
    const int nb_out = (a.outer + kGroup - 1) / kGroup;
    const int sw_step = kTrans ? nb_out : 1;
    uint32_t tb = 0, tph = 0;
    bool ok = true;
    unsigned sx[4], sw0 = 0, sw1 = 0;  // where the tile's scales begin
    float nx[4], nw0 = 0.0f, nw1 = 0.0f;
    const auto begin = [&](int w, int j) {
      const Tile t = tile_of(a, sm, cols, w);
      if (lane == 0) sm.tile[j % kTiles] = t;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        sx[r] = (unsigned)(t.row0 + min(lane + 32 * r, t.n - 1)) * blocks;
      const int cb = 2 * t.f, cb1 = min(cb + 1, nb_out - 1);
      const unsigned sw = (unsigned)t.g * nb_out * blocks;
      sw0 = sw + (kTrans ? cb : cb * blocks);
      sw1 = sw + (kTrans ? cb1 : cb1 * blocks);
    };
    const auto load = [&](int b) {
#pragma unroll
      for (int r = 0; r < 4; ++r) nx[r] = a.sx[sx[r] + b];  // (of the launch in front: no ldg)
      nw0 = __ldg(a.sw + (sw0 + b * sw_step));
      nw1 = __ldg(a.sw + (sw1 + b * sw_step));
    };
    int w = first, j = 0, b = 0;
    if (w < tiles) {
      begin(w, 0);
      load(0);
    }
    while (w < tiles && ok) {
      float p[2][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p[0][r] = nx[r] * nw0;
        p[1][r] = nx[r] * nw1;
      }
      if (++b == blocks) {
        b = 0;
        w += step;
        if (w < tiles) begin(w, ++j);
      }
      if (w < tiles) load(b);
      ok = wait_all(&sm.tempty[tb], tph ^ 1u, sm, a.status);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        sm.scale[tb][0][lane + 32 * r] = p[0][r];
        sm.scale[tb][1][lane + 32 * r] = p[1][r];
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.tfull[tb]);
      if ((tb ^= 1u) == 0) tph ^= 1u;
    }
  } else if (warp >= kWarpStore) {
    // Stores: a warp has the pieces of sums' warps i and i + 4.
    bool ok = true;
    for (int j = 0; j < mine && ok; ++j) {
#pragma unroll 1
      for (int p = warp - kWarpStore; p < kSumWarps && ok; p += kStoreWarps) {
        ok = wait_all(&sm.ofull[p], j & 1, sm, a.status);
        if (!ok) break;
        tc::fence_async_smem();  // the sums' writes before the TMA's reads
        const Tile t = sm.tile[j % kTiles];
        const int c0 = t.f * kBN + (p >> 2) * kHalf, row = 32 * (p & 3);
        uint8_t* piece = pieces + p * kOutBytes;
        send_piece(a, piece, t.row0 + row, t.n - row, c0);
        send_piece(a, piece + kOutBytes / 2, t.row0 + row, t.n - row, c0 + 64);
        asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
        // the piece is free once the TMA has read it: the one in front's, by now
        if (p >= kStoreWarps) {
          asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(&sm.ofree[p - kStoreWarps]);
            tc::mbar_arrive(&sm.ofree[p]);
          }
        }
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  } else {
    more_regs<kSumRegs>();
    const int q = warp & 3, half = warp >> 2;   // this warp's lanes and columns
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * kHalf;
    uint8_t* piece = pieces + warp * kOutBytes;
    uint32_t n = 0;  // blocks in front
    for (int j = 0; j < mine; ++j) {
      float acc[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf; ++i) acc[i] = 0.0f;
#pragma unroll 1
      for (int b = 0; b < blocks; ++b, ++n) {
        // (a wait that gave up has set the abort flag, which is seen behind the loop; lanes and
        // columns without outputs add up what is there, and drop it)
        const uint32_t tb = n & 1u;
        tc::wait_bounded(&sm.tfull[tb], (n >> 1) & 1u, &sm.abort, a.status);
        __syncwarp();
        tc::fence_after_sync();
        const uint32_t from = lanes + tb * kBN;
        uint32_t v0[32], v1[32];
        tc::tmem_ld_async(from, v0);
        const float s = sm.scale[tb][half][32 * q + lane];
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
        // the last products are in registers: the buffer goes back
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.tempty[tb]);
        add_scaled(acc + 96, v1, s);
      }
      // sums of a tile with a wait that gave up, any warp's, are not handed on
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&sm.abort))) break;
      // the warp's piece, once the tile before has left it
      if (!wait_all(&sm.ofree[warp], (j & 1) ^ 1u, sm, a.status)) break;
      stage_piece(piece, acc);
      stage_piece(piece + kOutBytes / 2, acc + 64);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.ofull[warp]);
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
