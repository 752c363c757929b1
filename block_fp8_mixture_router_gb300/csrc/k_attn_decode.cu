// Attention over the 8-bit paged cache for few rows of a sequence (single
// tokens, frames): commit "the Drama 3 text backbone on CUDA" (full attention
// with shared key heads); the cache's format is this library's.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale q . k_j
//
// in one pass over the keys with a running maximum m and sum.  A row tile is R
// rows (8 or 16): the g query heads of a key head times R/g tokens.
//
// A value is code c x its page's scale 2^lambda, and what the tensor cores sum are codes,
// weighted by 2^(s_j + lambda_j - r) against a reference r of their own, the running maximum
// of s_j + lambda_j over the keys that the row sees:
//
//   out = 2^(r - m) sum_j 2^(s_j + lambda_j - r) c_j / sum_j 2^(s_j - m).
//
// Each row so has weights of its own range, whatever scales other rows' keys have and
// however far apart its own are (2 us of the 107 below, against one scale reference for
// all rows of a tile).  The lower sum takes its terms from the weights, times
// 2^(r - m - lambda), so that a score costs one exponential; where that factor passes
// 2^kSpread, keys that count could have weights below fp32's range, and the terms get
// exponentials of their own.
//
// The cache's bytes bound it, so the codes go to the tensor cores as they are
// stored, keys and values as the operand with M = 128 and the few rows as N:
//
//   S^T [128 keys x 2R] = K [128 keys x D] . (Qhi | Qlo)^T,
//   O^T [D x 4R]       += V^T [D x 128 keys] . (P1 | P2 | P3 | P4)^T,
//
// all in kind::f8f6f4 with fp32 sums.  A query of 8 significant bits is two e4m3
// values of 4, Qhi + Qlo; a weight is four e5m2 values of 3, each part scaled by 2^3 of
// the one before it and summed in columns of its own: 11 bits, over e5m2's thirty
// powers of two.  V's tile is read M-major, just as the pages hold it.  (Warp MMAs
// need both operands widened to fp16 in registers: 600 instructions per warp and
// 32 keys, against about 300 per warp and 128 keys here.)
//
// A CTA has four softmax warps (a thread per key of the tile), a warp that issues
// the MMAs and one that keeps a ring of key tiles (128 keys and their values, 32 KB
// at head_dim 128) filled by TMA; two CTAs share an SM (one at head_dim 256).
//
// Measured: 64 rows of 32 heads over 590 MB of codes, 107 us (5.6 TB/s, where a plain
// copy reaches 6.8); one row of 16 heads over 262143 tokens, 51 us (5.3 TB/s); one row
// over 4096 tokens, 9.2 us: 5 us of dependent steps in a CTA (finding its tiles 1.2,
// queries and first tile 1.6, softmax 1.2, products and the result 1.1), the rest launches
// and the join.
#include "attn_tc.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192;       // four softmax warps, the MMA warp, the TMA warp
constexpr int kSoftmax = 128;
constexpr int kMmaWarp = 4;
constexpr int kTmaWarp = 5;
// A weight is stored as p x 2^12, and p taken against a reference that may lag the
// row's maximum by kLag powers of two: sums are only scaled again when a score
// outgrows that, and 2^(12 + kLag) is where e5m2's last binade begins.
constexpr float kShiftLog = 12.0f;
constexpr float kLag = 3.0f;
// The sum of 2^(s - m) is fp32 and takes a lag of kSumLag.  s + lambda is within kLag of r, so
// s - m can only pass that for a page with r - m - lambda above kSpread, and only then
// are the scores held against m at all.  A weight below 2^-126 then is a term below
// 2^(kSpread - 126).  (What a row does depends on its own scores and scales alone.)
constexpr float kSumLag = 64.0f;
constexpr float kSpread = kSumLag - kLag - 1.0f;
constexpr int kParts = 4;

template <int D>
struct Dec {
  static constexpr bool kWide = D >= 128;              // 128-byte rows and swizzle
  static constexpr int kRowBytes = kWide ? 128 : 64;
  static constexpr int kPanels = D / kRowBytes;        // pieces of a row
  static constexpr int kPanelBytes = kAttnKeys * kRowBytes;
  static constexpr int kTileBytes = kAttnKeys * D;     // keys or values of a stage
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr uint32_t kTmemCols = D == 256 ? 256 : 128;
};

// What a CTA works on: row tile `t` of sequence `s` for key head h.
struct Unit {
  int s, h, t;
  SeqView v;
  int tok0;       // first token of the tile among the sequence's rows
  int rows;       // valid rows (tokens x g)
  int lo, hi;     // keys [lo, hi) that any row of the tile can see
  int kt0, kt1;   // the key tiles of kAttnKeys that cover them (at least one)
};

template <int R>
__device__ __forceinline__ void unit_range(const AttnArgs& a, Unit& u) {
  const int tq = R / a.g;
  u.tok0 = u.t * tq;
  const int toks = min(tq, u.v.n - u.tok0);
  u.rows = toks * a.g;
  u.hi = max(min(u.v.len, u.v.first + u.tok0 + toks), 0);
  u.lo = a.window ? max(0, u.v.first + u.tok0 - a.window + 1) : 0;
  u.lo = min(u.lo, u.hi);
  u.kt0 = u.lo / kAttnKeys;
  u.kt1 = max((int)(((long long)u.hi + kAttnKeys - 1) / kAttnKeys), u.kt0 + 1);
}

// One CTA's shared memory behind the ring (which begins on 1024 bytes).
template <int D>
struct DecSmem {
  uint8_t p[kParts * 16 * 128];  // weight parts: [4R rows][128 keys], swizzled atoms of 8 rows
  uint8_t q[32 * D];       // query parts: [2R rows][D] in panels of kRowBytes, swizzled
  alignas(32) float fac[16];  // a row's score factor, but for the key's scale
  int pos[16];             // a row's position
  alignas(32) float ref[16];  // a row's reference for score + log2(value scale), r above
  alignas(32) float m[16];    // and for the score
  // what is added to a row's scores, 12 - r or 12 where r is -inf, and 2^(r - m), or 0, over the
  // weights' 2^12
  alignas(16) float2 base[16];
  alignas(16) float2 alpha[16];  // what new references multiply its two sums by
  float gap[16];                 // r - m, or -inf
  float spread;                  // the largest of them
  int top[2][4][16];       // the warps' row maxima (r's and m's), as ordered integers
  float l[4][16];          // the warps' row sums
  uint32_t odd[4];         // rows of which a warp's columns hold a NaN
  float2 meta[Dec<D>::kStages][kAttnKeys / 16];  // scales of 16 keys and their values
  uint64_t full[Dec<D>::kStages], empty[Dec<D>::kStages];
  uint64_t q_full, s_full[2], s_empty[2], p_full, pv_done;
  uint32_t tmem;
  int abort, seq, tile;
  long long front;
  long long scan[kThreads / 32];
};

template <int D>
constexpr size_t dec_smem_bytes() {
  return 1024 + (size_t)Dec<D>::kStages * 2 * Dec<D>::kTileBytes + sizeof(DecSmem<D>);
}

__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(kSoftmax) : "memory");
}

// Whether any softmax thread's flag is set (all of them call).
__device__ __forceinline__ bool softmax_any(bool flag) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)flag), "n"(kSoftmax)
      : "memory");
  return r != 0;
}

// Floats as integers of the same order, for the integer warp reduction.
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float from_ordered(int b) {
  return __int_as_float(b >= 0 ? b : b ^ 0x7FFFFFFF);
}

// Byte of (row, byte b of the row) in a [rows][128] or [rows][64] operand under its
// swizzle.
template <bool kWide>
__device__ __forceinline__ int swz(int row, int b) {
  const int col = b >> 4;
  return kWide ? row * 128 + ((col ^ (row & 7)) << 4) + (b & 15)
               : row * 64 + ((col ^ ((row >> 1) & 3)) << 4) + (b & 15);
}

// Eight consecutive floats of shared memory (32-byte aligned).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ uint32_t e5m2x2_of(float lo, float hi) {
  uint16_t w;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(w) : "f"(hi), "f"(lo));
  return w;
}

// The queries of a tile as e4m3 operands.  A row's values are scaled by the power
// of two that brings its largest into [128, 256) and split into a rounded part and
// the rest, hi + lo: exact down to 1/4 (2^-9 of the row's largest), and to 2^-10,
// e4m3's half step (2^-17 of the largest), below.
template <int D, int R>
__device__ __forceinline__ void stage_queries(const AttnArgs& a, const Unit& u, const bf16* q,
                                              int64_t q_stride, DecSmem<D>& sm) {
  using C = Dec<D>;
  constexpr int kPer = D / 8;
  const int c = threadIdx.x % kPer, sub = threadIdx.x / kPer;
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += kSoftmax / kPer) {
    const int r = r0 + sub;  // (at head_dim 64 the lanes pass R)
    const bool on = r < u.rows;
    const int tok = r / a.g;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (on)
      raw = *reinterpret_cast<const uint4*>(q + (int64_t)(u.v.row0 + u.tok0 + tok) * q_stride +
                                            (u.h * a.g + r - tok * a.g) * D + 8 * c);
    float x[8];
    unpack8(raw, x);
    float mx = 0.0f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      odd |= !is_finite(x[i]);
      mx = fmaxf(mx, fabsf(x[i]));
    }
    if (odd) mx = __int_as_float(0x7F800000);
#pragma unroll
    for (int o = kPer / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    uint2 hi = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), lo = make_uint2(0, 0);  // NaN scores
    float f = 0.0f;
    if (is_finite(mx)) {
      const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
      f = __uint_as_float((uint32_t)(127 - 7 + e) << 23) * a.scale;
      uint32_t w[2], z[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = x[4 * i + k] * up;
        w[i] = e4m3x4(y[0], y[1], y[2], y[3]);
        uint32_t h01, h23;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h01) : "h"((uint16_t)w[i]));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h23) : "h"((uint16_t)(w[i] >> 16)));
        const float2 b01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
        const float2 b23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
        z[i] = e4m3x4(y[0] - b01.x, y[1] - b01.y, y[2] - b23.x, y[3] - b23.y);
      }
      hi = make_uint2(w[0], w[1]);
      lo = make_uint2(z[0], z[1]);
    }
    if (r < R) {
      const int panel = 8 * c / C::kRowBytes, b = 8 * c % C::kRowBytes;
      uint8_t* at = sm.q + panel * 2 * R * C::kRowBytes;
      *reinterpret_cast<uint2*>(at + swz<C::kWide>(r, b)) = hi;
      *reinterpret_cast<uint2*>(at + swz<C::kWide>(R + r, b)) = lo;
      if (c == 0) {
        sm.fac[r] = f;
        sm.pos[r] = u.v.first + u.tok0 + tok;
        sm.ref[r] = sm.m[r] = sm.gap[r] = -INFINITY;
        sm.base[r] = make_float2(kShiftLog, 0.0f);
      }
    }
  }
}

// A ring's (or a double buffer's) next slot and the parity of its barriers.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// The TMA warp's part of key tiles [t0, t1): a lane for each box (a page's share
// of a tile) of up to 32 looks up page and scales, then each tile's lanes copy their
// boxes once its stage is free.
template <int D>
__device__ __forceinline__ void produce(const AttnArgs& a, const Unit& u, int t0, int t1,
                                        const CUtensorMap* kmap, const CUtensorMap* vmap,
                                        uint8_t* ring, DecSmem<D>& sm, Ring& r) {
  using C = Dec<D>;
  const int lane = threadIdx.x & 31;
  const int box_rows = 1 << a.page_shift;
  const int per_tile = kAttnKeys / box_rows;
  const int batch = 32 / per_tile;  // tiles of a batch of boxes
  for (int kt0 = t0; kt0 < t1; kt0 += batch) {
    const int tiles = min(batch, t1 - kt0);
    const int key = kt0 * kAttnKeys + lane * box_rows;
    bool on = lane < tiles * per_tile && key < u.hi && key + box_rows > u.lo;
    int page = 0;
    float ks = -1.0f, vs = 1.0f;  // keys of a page that is not copied count as absent
    if (on) {
      page = page_at(a, u.s, key >> a.page_shift);
      if (page < 0) {
        atomicOr(a.status, kAttnBadBatch);
        on = false;
      } else {
        ks = a.ks[(size_t)page * a.Hkv + u.h];  // used after the first copies are out
        vs = a.vs[(size_t)page * a.Hkv + u.h];
      }
    }
    const int y = u.h << a.page_shift;
    for (int i = 0; i < tiles; ++i) {
      tc::wait_bounded(&sm.empty[r.stage], r.phase ^ 1, &sm.abort, a.status);
      if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) return;
      const int sub = lane - i * per_tile;  // this lane's box in the tile
      const bool mine = sub >= 0 && sub < per_tile;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine && on));
      if (mine && on) {
        uint8_t* k = ring + (size_t)r.stage * 2 * C::kTileBytes + sub * box_rows * C::kRowBytes;
#pragma unroll
        for (int p = 0; p < C::kPanels; ++p) {
          tc::tma_load_3d(k + p * C::kPanelBytes, kmap, p * 128, y, page, &sm.full[r.stage]);
          tc::tma_load_3d(k + C::kTileBytes + p * C::kPanelBytes, vmap, p * 128, y, page,
                          &sm.full[r.stage]);
        }
      }
      // the stage's one arrival, with the bytes to expect, follows the scales
      if (mine)
        for (int g = sub * box_rows / 16; g < (sub + 1) * box_rows / 16; ++g)
          sm.meta[r.stage][g] = make_float2(ks, vs);
      __syncwarp();  // all lanes' scales before lane 0's arrival
      if (lane == 0) tc::mbar_arrive_expect_tx(&sm.full[r.stage], boxes * box_rows * D * 2);
      r.next(C::kStages);
    }
  }
}

// Barrier parities that the MMA warp and the softmax warps carry along.
struct Phases {
  Ring ring;      // stages
  Ring s;         // score buffers
  uint32_t q = 0, p = 0, pv = 0;
};

// The MMA warp's part: the next tile's scores are issued before the tile's values,
// so that the tensor cores work on them while the softmax warps take this tile's.
template <int D, int R>
__device__ __forceinline__ void issue(const AttnArgs& a, int t0, int t1, uint32_t ring,
                                      uint32_t tmem, DecSmem<D>& sm, Phases& ph) {
  using C = Dec<D>;
  constexpr uint32_t id_s = tc::idesc_f8(128, 2 * R);
  constexpr uint32_t id_o =
      tc::idesc_f8(128, kParts * R) | tc::kIdescAMajorM | tc::kIdescBE5m2;
  const uint32_t sq = tc::smem_u32(sm.q), sp = tc::smem_u32(sm.p);
  int* abort = &sm.abort;
  tc::wait_bounded(&sm.q_full, ph.q, abort, a.status);
  ph.q ^= 1;
  Ring load = ph.ring;
  const auto scores = [&]() {
    tc::wait_bounded(&sm.full[load.stage], load.phase, abort, a.status);
    tc::wait_bounded(&sm.s_empty[ph.s.stage], ph.s.phase ^ 1, abort, a.status);
    tc::fence_after_sync();
    const uint32_t k = ring + load.stage * 2 * C::kTileBytes;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int panel = 32 * i / C::kRowBytes, b = 32 * i % C::kRowBytes;
      tc::mma_warp<true>(tmem + ph.s.stage * 32,
                         tc::swz_desc(k + panel * C::kPanelBytes + b, C::kWide),
                         tc::swz_desc(sq + panel * 2 * R * C::kRowBytes + b, C::kWide), id_s,
                         i > 0);
    }
    tc::commit_warp(&sm.s_full[ph.s.stage]);
    load.next(C::kStages);
    ph.s.next(2);
  };
  scores();
  for (int kt = t0; kt < t1; ++kt) {
    if (kt + 1 < t1) scores();
    tc::wait_bounded(&sm.p_full, ph.p, abort, a.status);
    ph.p ^= 1;
    tc::fence_after_sync();
    const uint32_t v = ring + ph.ring.stage * 2 * C::kTileBytes + C::kTileBytes;
#pragma unroll
    for (int panel = 0; panel < C::kPanels; ++panel) {
      const uint32_t d = tmem + 64 + panel * 64;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // at head_dim 64 the rows behind a value's 64 repeat it and are not read
        const uint64_t va = tc::swz_desc(v + panel * C::kPanelBytes + 32 * i * C::kRowBytes,
                                         C::kWide, 0);
        tc::mma_warp<true>(d, va, tc::swz_desc(sp + 32 * i, true), id_o, kt > t0 || i > 0);
      }
    }
    tc::commit_warp(&sm.empty[ph.ring.stage]);
    tc::commit_warp(&sm.pv_done);
    ph.ring.next(C::kStages);
  }
}

// a / b for a, b >= 0: a 32-bit division wherever both fit.
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The softmax warps' part of key tiles [t0, t1) of a unit.  whole: they are all of
// the unit's, and the output is written; else the partial result goes to slot
// `slot` for k_attn_merge.
template <int D, int R>
__device__ __forceinline__ void soften(const AttnArgs& a, const Unit& u, int t0, int t1,
                                       bool whole, int slot, const bf16* q, int64_t q_stride,
                                       bf16* out, int64_t out_stride, const AttnSplit& sp,
                                       uint8_t* ring, uint32_t tmem_base, DecSmem<D>& sm,
                                       Phases& ph) {
  using C = Dec<D>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t tmem = tmem_base + ((uint32_t)(warp * 32) << 16);  // this warp's lanes
  int* abort = &sm.abort;
  softmax_sync();  // the last segment's sums have been read
  stage_queries<D, R>(a, u, q, q_stride, sm);
  tc::fence_async_smem();
  softmax_sync();
  if (tid == 0) tc::mbar_arrive(&sm.q_full);
  const int pos0 = u.v.first + u.tok0;                      // earliest row
  const int pos1 = pos0 + (u.rows - 1) / a.g;               // latest row
  float l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) l[r] = 0.0f;
  float spread = -INFINITY;
  // where this thread's weight goes in a part's row n: row * 128 + the swizzled key
  uint8_t* const pw = sm.p + (tid & 15);
  const int col = (tid >> 4) << 4;

  for (int kt = t0; kt < t1; ++kt) {
    tc::wait_bounded(&sm.full[ph.ring.stage], ph.ring.phase, abort, a.status);
    const float2 sc = sm.meta[ph.ring.stage][tid >> 4];
    float lv;  // (a scale of a cache that other code filled may be anything)
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(lv) : "f"(clamp_scale(sc.y)));
    const int key = kt * kAttnKeys + tid;
    const bool live = key >= u.lo && key < u.hi && sc.x >= 0.0f;
    const bool edge = kt * kAttnKeys + kAttnKeys - 1 > pos0 || kt * kAttnKeys < u.lo ||
                      (a.window && kt * kAttnKeys <= pos1 - a.window) || !live;
    uint32_t seen = (1u << R) - 1;
    bool poison = false;
    if (edge) {
      seen = 0;
      if (live)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (key <= sm.pos[r] && (!a.window || key > sm.pos[r] - a.window)) seen |= 1u << r;
      // an unseen key's weight is 0, but 0 x NaN is not: values that do not exist become
      // zeros, NaN codes too, and the rows that do see such a key get a NaN weight
      uint8_t* v = ring + (size_t)ph.ring.stage * 2 * C::kTileBytes + C::kTileBytes;
#pragma unroll
      for (int p = 0; p < C::kPanels; ++p)
#pragma unroll
        for (int b = 0; b < C::kRowBytes; b += 16) {
          uint4* at = reinterpret_cast<uint4*>(v + p * C::kPanelBytes + swz<C::kWide>(tid, b));
          if (!live) {
            *at = make_uint4(0, 0, 0, 0);
          } else {
            uint4 w = *at;
            const uint32_t n[4] = {e4m3_nan_bytes(w.x), e4m3_nan_bytes(w.y), e4m3_nan_bytes(w.z),
                                   e4m3_nan_bytes(w.w)};
            if (n[0] | n[1] | n[2] | n[3]) {
              poison = true;
              w.x &= ~((n[0] >> 7) * 0xFFu);
              w.y &= ~((n[1] >> 7) * 0xFFu);
              w.z &= ~((n[2] >> 7) * 0xFFu);
              w.w &= ~((n[3] >> 7) * 0xFFu);
              *at = w;
            }
          }
        }
    }
    tc::wait_bounded(&sm.s_full[ph.s.stage], ph.s.phase, abort, a.status);
    tc::fence_after_sync();
    __syncwarp();
    float s[R];              // s + lambda
    float peak = -INFINITY;  // the largest of them over their rows' references
#pragma unroll
    for (int h = 0; h < R; h += 8) {
      uint32_t hi[8], lo[8];
      tc::tmem_ld_async(tmem + ph.s.stage * 32 + h, hi);
      tc::tmem_ld_async(tmem + ph.s.stage * 32 + R + h, lo);
      float fac[8], ref[8];
      load8(sm.fac + h, fac);
      load8(sm.ref + h, ref);
      tc::wait_ld();
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        s[h + r] = fmaf(__uint_as_float(hi[r]) + __uint_as_float(lo[r]), fac[r] * sc.x, lv);
        if (seen & (1u << (h + r))) peak = fmaxf(peak, s[h + r] - ref[r]);
      }
    }
    bool outgrown = peak > kLag;
    if (spread - lv > kSpread)
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (seen & (1u << r)) outgrown |= s[r] - lv - sm.m[r] > kSumLag;
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.s_empty[ph.s.stage]);
    ph.s.next(2);
    if (softmax_any(outgrown)) {
      // new references, the running maxima, for the rows that have outgrown theirs
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // (a NaN score raises nothing)
        const float x = (seen & (1u << r)) && s[r] == s[r] ? s[r] : -INFINITY;
        const int t = __reduce_max_sync(0xffffffffu, ordered(x));
        const int u = __reduce_max_sync(0xffffffffu, ordered(x - lv));
        if (lane == 0) sm.top[0][warp][r] = t, sm.top[1][warp][r] = u;
      }
      softmax_sync();
      if (tid < R) {
        const auto top = [&](int i) {
          return from_ordered(max(max(sm.top[i][0][tid], sm.top[i][1][tid]),
                                  max(sm.top[i][2][tid], sm.top[i][3][tid])));
        };
        float ref = sm.ref[tid], m = sm.m[tid];
        float2 alpha = make_float2(1.0f, 1.0f);
        const float ref_top = top(0), m_top = top(1);
        if (ref_top - ref > kLag || m_top - m > kSumLag) {
          const float ref_new = fmaxf(ref, ref_top), m_new = fmaxf(m, m_top);
          alpha = make_float2(exp2_approx(ref - ref_new), exp2_approx(m - m_new));
          sm.ref[tid] = ref = ref_new;
          sm.m[tid] = m = m_new;
          sm.base[tid] = make_float2(kShiftLog - ref, exp2_approx(ref - m - kShiftLog));
          sm.gap[tid] = ref - m;
        }
        sm.alpha[tid] = alpha;
        const int most = __reduce_max_sync((1u << R) - 1, ordered(sm.gap[tid]));
        if (tid == 0) sm.spread = from_ordered(most);
      }
      softmax_sync();
      spread = sm.spread;
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] *= sm.alpha[r].y;
      if (kt > t0) {
        tc::wait_bounded(&sm.pv_done, ph.pv ^ 1, abort, a.status);
        tc::fence_after_sync();
        __syncwarp();
#pragma unroll
        for (int panel = 0; panel < C::kPanels; ++panel) {
#pragma unroll
          for (int h = 0; h < kParts; h += 2) {  // two parts at a time
            const uint32_t d = tmem + 64 + panel * 64 + h * R;
            uint32_t x[2 * R];
            tc::tmem_ld_async(d, x);
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float f = sm.alpha[r].x;
              x[r] = __float_as_uint(__uint_as_float(x[r]) * f);
              x[R + r] = __float_as_uint(__uint_as_float(x[R + r]) * f);
            }
            tc::tmem_st(d, x);
          }
        }
        tc::wait_st();
      }
    }
    // the weights carry the page's scale in their exponent, and the sum of them is
    // freed of it again
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(clamp_scale(sc.y)));
    if (spread - lv > kSpread) {  // of some row at least: the sums here, all rows' in its way
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (seen & (1u << r)) {
          const float2 base = sm.base[r];
          l[r] = sm.gap[r] - lv > kSpread
                     ? l[r] + exp2_approx(s[r] - lv - sm.m[r])
                     : fmaf(exp2_approx(s[r] + base.x), inv * base.y, l[r]);
        }
      inv = 0.0f;
    }
    // the parts' rows are free once the last tile's values are done
    if (kt > t0) tc::wait_bounded(&sm.pv_done, ph.pv ^ 1, abort, a.status);
    ph.pv ^= 1;
#pragma unroll
    for (int r = 0; r < R; r += 2) {
      const float4 base = *reinterpret_cast<const float4*>(sm.base + r);
      float rest[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float p = exp2_approx(s[r + k] + (k ? base.z : base.x));
        if (edge) {
          if (poison) p = __int_as_float(0x7FFFFFFF);
          if (!(seen & (1u << (r + k)))) p = 0.0f;
        }
        l[r + k] = fmaf(p, inv * (k ? base.w : base.y), l[r + k]);
        rest[k] = p;
      }
      // three bits from the top, then three of the rest each time; the first part leaves
      // what e5m2 only holds as a subnormal to the second (the others' are below 2^-32
      // of a weight of one), the last is rounded
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        float part[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          part[k] = i + 1 < kParts ? __uint_as_float(__float_as_uint(rest[k]) & 0xFFE00000u)
                                   : rest[k];
          if (i == 0 && rest[k] < 0x1p-14f) part[k] = 0.0f;
          rest[k] = (rest[k] - part[k]) * 8.0f;
        }
        const uint32_t w2 = e5m2x2_of(part[0], part[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int n = i * R + r + k;
          pw[n * 128 + (col ^ ((n & 7) << 4))] = (uint8_t)(w2 >> (8 * k));
        }
      }
    }
    tc::fence_async_smem();
    tc::fence_before_sync();
    tc::mbar_arrive(&sm.p_full);
    ph.ring.next(C::kStages);
  }

  // the sums of the rows over the threads' keys
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float t = warp_sum(l[r]);
    if (lane == 0) sm.l[warp][r] = t;
  }
  softmax_sync();
  tc::wait_bounded(&sm.pv_done, ph.pv ^ 1, abort, a.status);
  tc::fence_after_sync();
  __syncwarp();
  const auto out_at = [&](int r, int d) {
    const int tok = r / a.g;
    return out + (int64_t)(u.v.row0 + u.tok0 + tok) * out_stride +
           (u.h * a.g + r - tok * a.g) * D + d;
  };
  const auto part_at = [&](int r, int d) {
    return sp.o + ((size_t)slot * kAttnSlotRows + r) * D + d;
  };
  uint32_t odd = 0;  // rows of which this thread's columns hold a NaN
#pragma unroll
  for (int panel = 0; panel < C::kPanels; ++panel) {
    const uint32_t dt = tmem + 64 + panel * 64;
    uint32_t x[2 * R], y[2 * R];
    tc::tmem_ld_async(dt, x);
    tc::tmem_ld_async(dt + 2 * R, y);
    tc::wait_ld();
    const int d = panel * 128 + tid;
    if (tid < C::kRowBytes) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r < u.rows) {
          const float o = (__uint_as_float(x[r]) + __uint_as_float(x[R + r]) * 0x1p-3f +
                           __uint_as_float(y[r]) * 0x1p-6f +
                           __uint_as_float(y[R + r]) * 0x1p-9f);
          if (o != o) odd |= 1u << r;
          if (whole) {
            const float sum = sm.l[0][r] + sm.l[1][r] + sm.l[2][r] + sm.l[3][r];
            const float inv = sum == 0.0f ? 0.0f : __fdividef(sm.base[r].y, sum);
            *out_at(r, d) = __float2bfloat16_rn(o * inv);
          } else {
            __stcg(part_at(r, d), o * 0x1p-12f);
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  // A NaN value of a tile that all rows see reaches its own column only: the row is NaN all
  // the same, as where the rows' masks made its weight NaN.
  if (softmax_any(odd != 0)) {
    odd = __reduce_or_sync(0xffffffffu, odd);
    if (lane == 0) sm.odd[warp] = odd;
    softmax_sync();
    odd = sm.odd[0] | sm.odd[1] | sm.odd[2] | sm.odd[3];
    for (int d = tid; d < D; d += kSoftmax)
      for (int r = 0; r < u.rows; ++r)
        if ((odd >> r) & 1) {
          if (whole) *out_at(r, d) = __float2bfloat16_rn(__int_as_float(0x7FFFFFFF));
          else __stcg(part_at(r, d), __int_as_float(0x7FFFFFFF));
        }
  }
  if (!whole && tid < u.rows)
    __stcg(sp.sums + (size_t)slot * kAttnSlotRows + tid,
           make_float4(sm.ref[tid], sm.m[tid],
                       sm.l[0][tid] + sm.l[1][tid] + sm.l[2][tid] + sm.l[3][tid], 0.0f));
}

// kSplit: the key tiles of all units, in unit order, are dealt to the CTAs in
// equal runs, whatever the sequences' lengths are.  Of a unit that several CTAs
// share, the first CTA's part lies in its second slot and the others' in their first,
// and the first CTA names the unit to k_attn_merge (sp.shared).  Else a CTA per unit.
// All roles walk the same run.
template <int D, int R, bool kSplit>
// (the bounds ask for 128 registers: with more, two CTAs' six warps do not fit an SM)
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2)
    k_attn_decode(const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const AttnArgs a, const bf16* q,
                  int64_t q_stride, bf16* out, int64_t out_stride, const AttnSplit sp) {
  using C = Dec<D>;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  DecSmem<D>& sm =
      *reinterpret_cast<DecSmem<D>*>(ring + (size_t)C::kStages * 2 * C::kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int tq = R / a.g;
  Unit u;
  long long begin = 0, end = 0, per = 1, f = 0;
  if constexpr (!kSplit) {
    int u0;
    const int unit = blockIdx.x / a.Hkv;
    u.h = blockIdx.x % a.Hkv;
    u.s = unit_seq(a, tq, 1, unit, &u0);
    u.v = seq_view(a, u.s);
    if (!u.v.ok && tid == 0) atomicOr(a.status, kAttnBadBatch);
    u.t = unit - u0;
    if (u.t < 0 || u.t * tq >= u.v.n) {
      pdl_wait();  // (what ends before the kernel in front does not wait for it)
      return;
    }
    unit_range<R>(a, u);
    // this unit alone: a run that is exactly its tiles
    begin = (long long)u.h * (u.kt1 - u.kt0);
    end = begin + (u.kt1 - u.kt0);
    per = 0x7FFFFFFFFFFFll;
  } else {
    // each thread's run of sequences, their key tiles, and the tiles in front
    const int per_thread = (a.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(tid * per_thread, a.n_seqs), s1 = min(s0 + per_thread, a.n_seqs);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
      u.v = seq_view(a, s);
      if (!u.v.ok) atomicOr(a.status, kAttnBadBatch);
      for (u.t = 0; u.t * tq < u.v.n; ++u.t) {
        unit_range<R>(a, u);
        mine += (long long)(u.kt1 - u.kt0) * a.Hkv;
      }
    }
    const int lane = tid & 31;
    long long run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) sm.scan[warp] = run;
    __syncthreads();
    long long total = 0, front = run - mine;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) front += sm.scan[w];
      total += sm.scan[w];
    }
    if (total == 0) {
      pdl_wait();
      if (tid == 0) sp.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    per = div_ll(total + gridDim.x - 1, gridDim.x);
    begin = per * blockIdx.x;
    end = min(begin + per, total);
    if (begin >= end) {
      pdl_wait();
      if (tid == 0) sp.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    // the thread whose run holds the first tile finds its unit
    if (mine > 0 && front <= begin && begin < front + mine) {
      bool found = false;
      f = front;
      for (int s = s0; s < s1 && !found; ++s) {
        u.v = seq_view(a, s);
        for (u.t = 0; u.t * tq < u.v.n && !found; ++u.t) {
          unit_range<R>(a, u);
          const long long w = (long long)(u.kt1 - u.kt0) * a.Hkv;
          if (begin < f + w) {
            sm.seq = s;
            sm.tile = u.t;
            sm.front = f;
            found = true;
          } else {
            f += w;
          }
        }
      }
    }
  }
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.s_empty[i], kSoftmax / 32);
    }
    tc::mbar_init(&sm.q_full, 1);
    tc::mbar_init(&sm.p_full, kSoftmax);
    tc::mbar_init(&sm.pv_done, 1);
    sm.abort = 0;
    tc::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::tmem_alloc(&sm.tmem, C::kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == kTmaWarp && (tid & 31) == 0) {
    tc::tma_prefetch_map(&kmap);
    tc::tma_prefetch_map(&vmap);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  if constexpr (kSplit) {
    u.s = sm.seq;
    u.t = sm.tile;
    f = sm.front;  // tiles in front of (sequence, row tile)
    u.v = seq_view(a, u.s);
    unit_range<R>(a, u);
    u.h = (int)div_ll(begin - f, u.kt1 - u.kt0);
  }
  pdl_wait();
  pdl_trigger();  // the merge may take its places and wait
  Phases ph;
  int4 shared = make_int4(0, 0, 0, 0);
  long long at = begin;
  while (at < end) {
    const int w = u.kt1 - u.kt0;
    const long long u_first = f + (long long)u.h * w;  // the unit's first tile
    const long long stop = min(end, u_first + w);
    const int t0 = u.kt0 + (int)(at - u_first), t1 = u.kt0 + (int)(stop - u_first);
    if (warp == kTmaWarp) {
      produce<D>(a, u, t0, t1, &kmap, &vmap, ring, sm, ph.ring);
    } else if (warp == kMmaWarp) {
      issue<D, R>(a, t0, t1, tc::smem_u32(ring), tmem, sm, ph);
    } else {
      const bool first = at == u_first, whole = first && stop == u_first + w;
      if (first && !whole)  // parts, valid rows, first row, key head
        shared = make_int4((int)(div_ll(u_first + w - 1, per) - blockIdx.x) + 1, u.rows,
                           u.v.row0 + u.tok0, u.h);
      soften<D, R>(a, u, t0, t1, whole, 2 * (int)blockIdx.x + (first ? 1 : 0), q, q_stride, out,
                   out_stride, sp, ring, tmem, sm, ph);
    }
    at = stop;
    if (at >= end) break;
    if (++u.h == a.Hkv) {
      u.h = 0;
      f += (long long)w * a.Hkv;
      ++u.t;
      while (u.t * tq >= u.v.n) {
        u.t = 0;
        u.v = seq_view(a, ++u.s);
      }
      unit_range<R>(a, u);
    }
  }
  if (kSplit && tid == 0) sp.shared[blockIdx.x] = shared;
  if (warp >= kMmaWarp && *(volatile int*)&sm.abort) {
    // a wait gave up: time for this CTA's copies and MMAs in flight to end before its
    // memory goes back
    const unsigned long long t = tc::global_ns();
    while (tc::global_ns() - t < 2000000ull) {
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of the units that CTAs of a split launch shared: block (c, row)
// looks at the unit that CTA c was the first to work on.  Parts are weighted by
// their references and added in a fixed order: kRuns interleaved runs, then those.  Bound
// by the latency of its loads: the parts' sums are on their way with their references.
template <int D>
__global__ void __launch_bounds__(2 * D)
    k_attn_merge(AttnSplit sp, int g, bf16* out, int64_t out_stride) {
  constexpr int kThreadsM = 2 * D, kCols = D / 4, kRuns = 8, kWarps = kThreadsM / 32;
  constexpr int kAhead = 8;             // parts of a run that are loaded at once
  __shared__ float s_w[kAttnMaxCtas];   // the parts' weights
  __shared__ float s_ref[kWarps], s_m[kWarps], s_l[kWarps];
  __shared__ float4 s_x[kRuns - 1][kCols];
  const int c0 = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  const int4 unit = __ldcg(sp.shared + c0);
  const int parts = unit.x;
  if (row >= unit.y || parts == 0) return;
  const auto slot = [&](int p) {
    return (size_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)) * kAttnSlotRows + row;
  };
  const int col = tid % kCols, run = tid / kCols;
  float4 y[kAhead];
  const auto load = [&](int p0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = p0 + run + k * kRuns;
      y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < parts) y[k] = __ldcg(reinterpret_cast<const float4*>(sp.o + slot(p) * D) + col);
    }
  };
  // the first parts' references and sums; more parts than threads are read again
  float4 own = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
  if (tid < parts) own = __ldcg(sp.sums + slot(tid));
  load(0);
  float ref = own.x, m = own.y;
  for (int p = tid + kThreadsM; p < parts; p += kThreadsM) {
    const float4 more = __ldcg(sp.sums + slot(p));
    ref = fmaxf(ref, more.x), m = fmaxf(m, more.y);
  }
  ref = warp_max(ref), m = warp_max(m);
  if ((tid & 31) == 0) s_ref[tid >> 5] = ref, s_m[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, s_ref[w]), m = fmaxf(m, s_m[w]);
  float l = 0.0f;
  for (int p = tid; p < parts; p += kThreadsM) {
    if (p >= kThreadsM) own = __ldcg(sp.sums + slot(p));
    const bool none = own.y == -INFINITY;  // (of a row that saw no key its sums are 0, or NaN)
    s_w[p] = none ? 1.0f : exp2_approx(own.x - ref);
    l = fmaf(own.z, none ? 1.0f : exp2_approx(own.y - m), l);
  }
  l = warp_sum(l);
  if ((tid & 31) == 0) s_l[tid >> 5] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) l += s_l[w];
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0;;) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = p0 + run + k * kRuns;
      if (p < parts) {
        const float f = s_w[p];
        x = make_float4(fmaf(y[k].x, f, x.x), fmaf(y[k].y, f, x.y), fmaf(y[k].z, f, x.z),
                        fmaf(y[k].w, f, x.w));
      }
    }
    p0 += kAhead * kRuns;
    if (p0 >= parts) break;
    load(p0);
  }
  if (run > 0) s_x[run - 1][col] = x;
  __syncthreads();
  if (run > 0) return;
#pragma unroll
  for (int i = 0; i < kRuns - 1; ++i) {
    const float4 z = s_x[i][col];
    x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
  }
  const float up = m == -INFINITY ? 1.0f : exp2_approx(ref - m);
  const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l) * up;
  const int tok = row / g;
  const __nv_bfloat162 y0 = __floats2bfloat162_rn(x.x * inv, x.y * inv);
  const __nv_bfloat162 y1 = __floats2bfloat162_rn(x.z * inv, x.w * inv);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&y0);
  w.y = *reinterpret_cast<const uint32_t*>(&y1);
  *reinterpret_cast<uint2*>(out + (int64_t)(unit.z + tok) * out_stride +
                            (unit.w * g + row - tok * g) * D + 4 * col) = w;
}

template <int D, int R>
cudaError_t setup_dr() {
  cudaError_t e = cudaFuncSetAttribute(k_attn_decode<D, R, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)dec_smem_bytes<D>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_attn_decode<D, R, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dec_smem_bytes<D>());
  return e;
}

template <int D>
cudaError_t setup_d() {
  const cudaError_t e = setup_dr<D, 8>();
  return e == cudaSuccess ? setup_dr<D, 16>() : e;
}

template <int D, int R>
cudaError_t launch_dr(const AttnArgs& a, const AttnMaps& m, const bf16* q, int64_t q_stride,
                      bf16* out, int64_t out_stride, const AttnSplit& sp, int grid, bool split,
                      bool pdl, cudaStream_t s) {
  auto* kernel = split ? k_attn_decode<D, R, true> : k_attn_decode<D, R, false>;
  const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kThreads), dec_smem_bytes<D>(), s, pdl,
                                   m.k, m.v, a, q, q_stride, out, out_stride, sp);
  // (one CTA shares no unit)
  if (e != cudaSuccess || !split || grid == 1) return e;
  return launch_pdl(k_attn_merge<D>, dim3(grid, R), dim3(2 * D), 0, s, true, sp, a.g, out,
                    out_stride);
}

}  // namespace

cudaError_t setup_attn_decode(int D) {
  return D == 64 ? setup_d<64>() : D == 128 ? setup_d<128>() : setup_d<256>();
}

// Two CTAs of up to 113 KB, 128 registers and 128 TMEM columns share an SM (the
// occupancy query counts one for a kernel that allocates tensor memory; measured, 64 rows
// over 590 MB of keys and values take 142 us with one and 107 with two).
int attn_decode_slots(int D, int sm_count) { return D == 256 ? sm_count : 2 * sm_count; }

cudaError_t launch_attn_decode(int D, int tile_rows, const AttnArgs& a, const AttnMaps& m,
                               const bf16* q, int64_t q_stride, bf16* out, int64_t out_stride,
                               const AttnSplit& sp, int grid, bool split, bool pdl,
                               cudaStream_t s) {
  if (tile_rows == 8) {
    auto* f = D == 64 ? launch_dr<64, 8> : D == 128 ? launch_dr<128, 8> : launch_dr<256, 8>;
    return f(a, m, q, q_stride, out, out_stride, sp, grid, split, pdl, s);
  }
  auto* f = D == 64 ? launch_dr<64, 16> : D == 128 ? launch_dr<128, 16> : launch_dr<256, 16>;
  return f(a, m, q, q_stride, out, out_stride, sp, grid, split, pdl, s);
}

}  // namespace moe
