// Attention over the 8-bit paged cache for many rows of a sequence (prompts and
// chunks of them): commit "the Drama 3 text backbone on CUDA" (full attention with
// shared key heads); the cache's format is this library's.
//
//   S = Q K^T,  P = 2^(scale S + lambda - r),  O += P C,  out = 2^(r - m) O / sum 2^(scale S - m)
//
// in one pass over the keys with V = C 2^lambda, C the codes and 2^lambda their pages' scales,
// and for each row two running references, r of S + lambda and m of S, and a sum (see
// k_attn_decode.cu for why two).  Bound by the tensor cores and the shared memory that feeds them.  A CTA holds 256 rows
// (128 at head_dim 256): row tiles of 128, the g query heads of a key head times 128/g
// tokens, and takes the keys 64 at a time (128 at head_dim 256).
//
// - S: kind::f8f6f4 on the keys' codes as they are stored; a query of 8 significant
//   bits is two e4m3 values, Qhi + Qlo, multiplied in two passes at twice the
//   16-bit rate: the same time as one 16-bit product, without converting K.
// - P V: kind::f16; four warps widen V's codes to fp16 once for all the CTA's rows, P
//   goes to tensor memory as fp16 over the scores it came from.  (P through shared
//   memory would free the scores' place sooner, but the operands' traffic, 400 KB for
//   256 rows x 128 keys, then takes longer than the products.)
// - A row tile has two score buffers: while its softmax warps work on one, the tensor
//   cores fill the other, so that neither waits for the other's round trip.  Two row
//   tiles' buffers have room for 64 keys each, although an MMA with N = 64 takes as long
//   as one with N = 128.
//
// Measured: a prompt of 16384 rows, 16 heads of 128, 914 us (1203 TFLOP/s of two products,
// 62 % of what a plain 16-bit matrix product reaches); 1024 rows over 8192 keys at head_dim
// 256, 133 us (970); frames of 11 rows, 8 sequences over 1500 keys, 19 us, by their
// latency.  A step of 64 keys and 256 rows takes 1780 clocks, of which the MMAs take 1660:
// those of the scores, with N = 64, twice their share.
//
// Slower at 16384 rows, 16 heads of 128, beside 969 us at the time: one buffer of 128 keys per row
// tile, 1048 us (the row tiles fall into step, and both work while the tensor cores
// idle); the same with the row tiles' softmax warps taking turns, 1161 us (reads of
// tensor memory take twice as long beside running MMAs); a row's scores held in 192
// registers, 1070 us; one warp for all MMAs, 1202 us.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles (a thread per row), 8-11 widen V (at
// head_dim 256, with one row tile, 4-11), 12 and 13 issue a row tile's MMAs each, 14
// copies by TMA.
#include "attn_tc.cuh"

namespace moe {

namespace {

constexpr int kPThreads = 480;
constexpr int kMmaWarp = 12, kTmaWarp = 14;
constexpr int kKeys = 128;          // keys of a tile
constexpr int kChunk = 64;          // keys of a piece of V
// Weights as p x 2^5 in fp16, p against a reference that may lag the row's maximum by kLag
// powers of two: sums are scaled again only when a score outgrows that, or the sum's
// reference by kSumLag.  What is lost of a weight is 2^-12 of it, or 2^-30 of the row's
// largest.  (Each row decides for itself, so that no token it does not see changes it; with
// 2^7 and a lag of 8 a chunk's row tiles are scaled so often that 1024 rows at head_dim 256 take
// 144 us and not 134.)
constexpr float kShiftLog = 5.0f;
constexpr float kLag = 10.0f;
constexpr float kSumLag = 14.0f;
// The row's sum takes its terms 2^(s - m) from the weights 2^(s + lambda - r + 5), so that a
// score costs one exponential.  For a page far below the row's largest the weights are
// taken no smaller than 2^(s - m - kLeast): as fp16 they are 0 all the same, s - m being at
// most kSumLag, and the terms stay within fp32.
constexpr float kLeast = kSumLag + 26.0f;

template <int D>
struct Pr {
  static constexpr int kTiles = D == 256 ? 1 : 2;      // row tiles of a CTA
  static constexpr int kStep = D == 256 ? 128 : 64;    // keys of a score buffer
  static constexpr int kConvWarp = 4 * kTiles;         // first warp that widens V
  static constexpr int kConvWarps = kMmaWarp - kConvWarp;
  static constexpr int kPer = kKeys / kStep;           // steps of a key tile
  static constexpr bool kWide = D >= 128;
  static constexpr int kRowBytes = kWide ? 128 : 64;
  static constexpr int kPanels = D / kRowBytes;
  static constexpr int kPanelBytes = kKeys * kRowBytes;
  static constexpr int kTileBytes = kKeys * D;         // keys of a tile, as stored
  static constexpr int kQBytes = 128 * D;              // one part of a row tile's queries
  static constexpr int kKStages = D == 256 ? 2 : 3;
  static constexpr int kVStages = D == 256 ? 2 : 4;    // pieces of V, as stored
  static constexpr int kVPanelBytes = kChunk * kRowBytes;
  static constexpr int kVBytes = kChunk * D;
  static constexpr int kCStages = D == 256 ? 2 : 4;    // pieces of V, widened
  static constexpr int kCBytes = kChunk * D * 2;
  // tiles whose scales are kept: the softmax warps read a tile's when the TMA warp writes
  // those of the fourth behind it (two stages of keys) or the fifth (three) at the latest
  static constexpr int kMeta = 6;
};

// What the softmax warps need of a tile's pages, for each of its 16-key groups.
struct alignas(16) Meta {
  float ks[kKeys / 16];       // key scales
  float log_vs[kKeys / 16];   // value scales: log2, and one over
  float inv_vs[kKeys / 16];
  uint32_t absent;            // groups whose page does not exist (or is not needed)
};

template <int D>
struct PrSmem {
  static constexpr int kMeta = Pr<D>::kMeta;
  float fac[Pr<D>::kTiles * 128]; // score factors of the rows, but for the key's scale
  Meta meta[kMeta];
  uint32_t poison[kMeta][4];     // keys of a tile that have a NaN value
  uint64_t k_full[3], k_empty[3], v_full[4], v_empty[4], c_full[4], c_empty[4];
  uint64_t meta_full[kMeta], poison_full[kMeta];
  uint64_t q_full[2], s_full[4], p_full[4], pv_done[4];  // [row tile][buffer]
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr size_t pr_smem_bytes() {
  using C = Pr<D>;
  return 1024 + (size_t)C::kTiles * 2 * C::kQBytes +
         (size_t)C::kKStages * C::kTileBytes + (size_t)C::kVStages * C::kVBytes +
         (size_t)C::kCStages * C::kCBytes + sizeof(PrSmem<D>);
}

static_assert(pr_smem_bytes<64>() <= 232448 && pr_smem_bytes<128>() <= 232448 &&
                  pr_smem_bytes<256>() <= 232448,
              "a CTA's shared memory");

// Byte of (row, byte b) in a [rows][128] or [rows][64] operand under its swizzle.
template <bool kWide>
__device__ __forceinline__ int swz(int row, int b) {
  const int col = b >> 4;
  return kWide ? row * 128 + ((col ^ (row & 7)) << 4) + (b & 15)
               : row * 64 + ((col ^ ((row >> 1) & 3)) << 4) + (b & 15);
}

__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}

__device__ __forceinline__ uint32_t widen(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)w));
  return h;
}

// a * b + c and a + b on pairs of floats (one instruction each).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ __nv_bfloat162 abs2(uint32_t w) {
  w &= 0x7FFF7FFFu;
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      phase ^= 1;
    }
  }
};

// A CTA's rows and keys.
struct Work {
  int s, h;
  SeqView v;
  int tq;          // tokens of a row tile
  int tok0;        // first token
  int toks;        // tokens of the CTA (all row tiles)
  int tiles;       // row tiles that hold any
  int lo, hi;      // keys that any row can see
  int t0, t1;      // key tiles of this CTA
  int part, parts; // its share of the key tiles
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort, int* status) {
  return tc::wait_bounded(bar, parity, abort, status);
}

// The queries of one row tile as e4m3 parts (see k_attn_decode.cu), by its softmax
// warps.
template <int D>
__device__ __forceinline__ void stage_queries(const AttnArgs& a, const Work& w, int tile,
                                              const bf16* q, int64_t q_stride, uint8_t* sq,
                                              float* fac) {
  using C = Pr<D>;
  constexpr int kPer = D / 8;
  const int t = threadIdx.x & 127;
  const int c = t % kPer, sub = t / kPer;
  const int valid = min(w.tq, w.toks - tile * w.tq) * a.g;
  constexpr int kStep = 128 / kPer, kBatch = 8;  // rows of a pass; passes loaded at once
  const uint32_t per_g = 65536u / a.g + 1;       // r / g = r per_g >> 16 for r below 128
  // (with a pass's loads behind the pass before, 1024 rows at head_dim 256 took 15 us)
#pragma unroll 1
  for (int r0 = 0; r0 < 128; r0 += kBatch * kStep) {
    uint4 raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kStep + sub, tok = r * per_g >> 16;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (r < valid)
        raw[i] = *reinterpret_cast<const uint4*>(
            q + (int64_t)(w.v.row0 + w.tok0 + tile * w.tq + tok) * q_stride +
            (w.h * a.g + r - tok * a.g) * D + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kStep + sub;
      // the row's largest magnitude, NaN if it has one
      __nv_bfloat162 top = __hmax2_nan(__hmax2_nan(abs2(raw[i].x), abs2(raw[i].y)),
                                       __hmax2_nan(abs2(raw[i].z), abs2(raw[i].w)));
#pragma unroll
      for (int o = kPer / 2; o > 0; o >>= 1)
        top = __hmax2_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mx = __bfloat162float(__hmax_nan(__low2bfloat16(top), __high2bfloat16(top)));
      uint2 hi = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), lo = make_uint2(0, 0);  // NaN scores
      float f = 0.0f;
      if (is_finite(mx)) {
        const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
        f = __uint_as_float((uint32_t)(127 - 7 + e) << 23) * a.scale;
        float x[8];
        unpack8(raw[i], x);
        uint32_t p[2], z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) y[n] = x[4 * k + n] * up;
          p[k] = e4m3x4(y[0], y[1], y[2], y[3]);
          const uint32_t h01 = widen(p[k]), h23 = widen(p[k] >> 16);
          const float2 b01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
          const float2 b23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
          z[k] = e4m3x4(y[0] - b01.x, y[1] - b01.y, y[2] - b23.x, y[3] - b23.y);
        }
        hi = make_uint2(p[0], p[1]);
        lo = make_uint2(z[0], z[1]);
      }
      const int panel = 8 * c / C::kRowBytes, b = 8 * c % C::kRowBytes;
      uint8_t* at = sq + panel * 128 * C::kRowBytes + swz<C::kWide>(r, b);
      *reinterpret_cast<uint2*>(at) = hi;
      *reinterpret_cast<uint2*>(at + C::kQBytes) = lo;
      if (c == 0) fac[r] = f;
    }
  }
}

// ---- the TMA warp ------------------------------------------------------------
template <int D>
__device__ __forceinline__ void copy_tiles(const AttnArgs& a, const Work& w,
                                           const CUtensorMap* kmap, const CUtensorMap* vmap,
                                           uint8_t* sk, uint8_t* sv, PrSmem<D>& sm) {
  using C = Pr<D>;
  const int lane = threadIdx.x & 31;
  const int box = 1 << a.page_shift;
  const int per_tile = kKeys / box;
  const int batch = 32 / per_tile;
  const int y = w.h << a.page_shift;
  const int vbox = min(box, kChunk), v_per = kChunk / vbox;  // boxes of a piece of V
  Ring rk, rv;
  // keys of tile kt + 1 go out before the values of tile kt: they are needed first
  int page = 0, page_next = 0;
  bool on = false, on_next = false;
  float ks = -1.0f, vs = 1.0f, log_vs = 0.0f;
  int base = w.t0;                 // first tile of the lanes' boxes
  const auto look_up = [&](int kt0) {
    const int tiles = min(batch, w.t1 - kt0);
    const int key = kt0 * kKeys + lane * box;
    on_next = lane < tiles * per_tile && key < w.hi && key + box > w.lo;
    ks = -1.0f;
    vs = 1.0f;
    page_next = 0;
    if (on_next) {
      page_next = page_at(a, w.s, key >> a.page_shift);
      if (page_next < 0) {
        atomicOr(a.status, kAttnBadBatch);
        on_next = false;
      } else {
        ks = a.ks[(size_t)page_next * a.Hkv + w.h];
        vs = clamp_scale(a.vs[(size_t)page_next * a.Hkv + w.h]);
      }
    }
    log_vs = __log2f(vs);
  };
  int v_page = 0, v_sub = -1;
  bool v_on = false;
  for (int kt = w.t0; kt <= w.t1; ++kt) {
    int sub = -1;
    uint32_t boxes = 0;
    if (kt < w.t1) {
      if ((kt - w.t0) % batch == 0) {
        base = kt;
        look_up(kt);
        page = page_next;
        on = on_next;
      }
      sub = lane - (kt - base) * per_tile;
      const bool mine = sub >= 0 && sub < per_tile;
      boxes = __popc(__ballot_sync(0xffffffffu, mine && on));
      const int slot = (kt - w.t0) % C::kMeta;
      // (the softmax warps are at most a few tiles behind the keys' copies)
      if (mine)
        for (int g = sub * box / 16; g < (sub + 1) * box / 16; ++g)
        {
          sm.meta[slot].ks[g] = ks;
          sm.meta[slot].log_vs[g] = log_vs;
          sm.meta[slot].inv_vs[g] = __fdiv_rn(1.0f, vs);
        }
      const uint32_t absent = __reduce_or_sync(
          0xffffffffu, mine && !on ? ((1u << (box / 16)) - 1) << (sub * box / 16) : 0u);
      if (lane == 0) sm.meta[slot].absent = absent;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.meta_full[slot]);
      wait(&sm.k_empty[rk.i], rk.phase ^ 1, &sm.abort, a.status);
      if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) return;
      if (lane == 0) tc::mbar_arrive_expect_tx(&sm.k_full[rk.i], boxes * box * D);
      __syncwarp();
      if (mine && on)
#pragma unroll
        for (int p = 0; p < C::kPanels; ++p)
          tc::tma_load_3d(sk + (size_t)rk.i * C::kTileBytes + p * C::kPanelBytes +
                              sub * box * C::kRowBytes,
                          kmap, p * 128, y, page, &sm.k_full[rk.i]);
      rk.next(C::kKStages);
    }
    if (kt > w.t0) {
      for (int c = 0; c < kKeys / kChunk; ++c) {
        // (a page of 128 tokens has a box in both pieces)
        const int at = box > kChunk ? 0 : v_sub - c * v_per;
        const bool mine = v_on && at >= 0 && at < v_per;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, mine));
        wait(&sm.v_empty[rv.i], rv.phase ^ 1, &sm.abort, a.status);
        if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) return;
        if (lane == 0) tc::mbar_arrive_expect_tx(&sm.v_full[rv.i], n * vbox * D);
        __syncwarp();
        if (mine)
#pragma unroll
          for (int p = 0; p < C::kPanels; ++p)
            tc::tma_load_3d(sv + (size_t)rv.i * C::kVBytes + p * C::kVPanelBytes +
                                at * vbox * C::kRowBytes,
                            vmap, p * 128, y + (box > kChunk ? c * kChunk : 0), v_page,
                            &sm.v_full[rv.i]);
        rv.next(C::kVStages);
      }
    }
    v_on = sub >= 0 && sub < per_tile && on;
    v_sub = sub;
    v_page = page;
  }
}

// Whether a tile needs its keys looked at one by one: some row of [pos0, pos1] does
// not see all of them.
__device__ __forceinline__ bool edge_tile(const AttnArgs& a, const Work& w, int kt, int pos0,
                                          int pos1) {
  const int key0 = kt * kKeys;
  return key0 + kKeys - 1 > pos0 || key0 < w.lo || (a.window && key0 <= pos1 - a.window);
}

// ---- the warps that widen V -----------------------------------------------------
template <int D>
__device__ __forceinline__ void widen_tiles(const AttnArgs& a, const Work& w, const uint8_t* sv,
                                            uint8_t* sc, PrSmem<D>& sm) {
  using C = Pr<D>;
  constexpr int kShares = C::kConvWarps / 2;  // of a key's values
  const int t = threadIdx.x - C::kConvWarp * 32, lane = t & 31, warp = t >> 5;
  const int k = t & 63, h = t >> 6;           // key of a piece, share of its values
  const int pos0 = w.v.first + w.tok0, pos1 = pos0 + w.toks - 1;
  Ring rv, rc;
  for (int kt = w.t0; kt < w.t1; ++kt) {
    const int n = kt - w.t0, slot = n % C::kMeta;
    wait(&sm.meta_full[slot], (n / C::kMeta) & 1, &sm.abort, a.status);
    const bool whole = !edge_tile(a, w, kt, pos0, pos1) && sm.meta[slot].absent == 0;
    if (!whole) {
      if (t < 4) sm.poison[slot][t] = 0;
      asm volatile("bar.sync 2, %0;\n" ::"n"(32 * C::kConvWarps) : "memory");
    }
    for (int c = 0; c < 2; ++c) {
      wait(&sm.v_full[rv.i], rv.phase, &sm.abort, a.status);
      wait(&sm.c_empty[rc.i], rc.phase ^ 1, &sm.abort, a.status);
      const uint8_t* v = sv + (size_t)rv.i * C::kVBytes;
      uint8_t* out = sc + (size_t)rc.i * C::kCBytes;
      const int key = c * kChunk + k;
      bool live = true, poison = false;
      if (!whole)
        live = kt * kKeys + key >= w.lo && kt * kKeys + key < w.hi &&
               !((sm.meta[slot].absent >> (key >> 4)) & 1);
#pragma unroll
      for (int i = 0; i < D / 16 / kShares; ++i) {
        const int b = h * (D / kShares) + 16 * i;  // first of 16 values
        uint4 x = *reinterpret_cast<const uint4*>(v + b / C::kRowBytes * C::kVPanelBytes +
                                                  swz<C::kWide>(k, b % C::kRowBytes));
        if (!whole) {
          // values that do not exist become zeros, and NaN codes too: the rows that do see
          // such a key get a NaN weight instead (0 x NaN would reach the others)
          if (!live) x = make_uint4(0, 0, 0, 0);
          const uint32_t n0 = e4m3_nan_bytes(x.x), n1 = e4m3_nan_bytes(x.y),
                         n2 = e4m3_nan_bytes(x.z), n3 = e4m3_nan_bytes(x.w);
          if (n0 | n1 | n2 | n3) {
            poison = true;
            x.x &= ~((n0 >> 7) * 0xFFu);
            x.y &= ~((n1 >> 7) * 0xFFu);
            x.z &= ~((n2 >> 7) * 0xFFu);
            x.w &= ~((n3 >> 7) * 0xFFu);
          }
        }
        uint8_t* row = out + b / 64 * (kChunk * 128);
        const int col = (b % 64) / 8;              // 16-byte column of eight fp16
        *reinterpret_cast<uint4*>(row + k * 128 + ((col ^ (k & 7)) << 4)) =
            make_uint4(widen(x.x), widen(x.x >> 16), widen(x.y), widen(x.y >> 16));
        *reinterpret_cast<uint4*>(row + k * 128 + (((col + 1) ^ (k & 7)) << 4)) =
            make_uint4(widen(x.z), widen(x.z >> 16), widen(x.w), widen(x.w >> 16));
      }
      if (!whole) {
        const uint32_t bits = __ballot_sync(0xffffffffu, poison);
        if (lane == 0 && bits) atomicOr(&sm.poison[slot][2 * c + (warp & 1)], bits);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sm.c_full[rc.i]);
        tc::mbar_arrive(&sm.v_empty[rv.i]);
      }
      rc.next(C::kCStages);
      rv.next(C::kVStages);
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.poison_full[slot]);
  }
}

// ---- the MMA warps: one for each row tile ---------------------------------------
// Step j is kStep keys; its scores go to the row tile's buffer j & 1.
template <int D>
__device__ __forceinline__ void issue(const AttnArgs& a, const Work& w, int m, uint32_t sq,
                                      uint32_t sk, uint32_t sc, uint32_t tmem, PrSmem<D>& sm) {
  using C = Pr<D>;
  constexpr uint32_t id_s = tc::idesc_f8(128, C::kStep);
  constexpr uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                            ((uint32_t)(128 >> 4) << 24);  // fp16, B stored N-major
  int* abort = &sm.abort;
  const uint32_t leader = (threadIdx.x & 31) == 0;
  const int n = C::kPer * (w.t1 - w.t0);
  const uint32_t t_s = tmem + m * 128, t_o = tmem + 256 + m * D;
  const tc::Desc dq = tc::desc_of(sq + 2 * m * C::kQBytes, C::kWide);
  const tc::Desc dk = tc::desc_of(sk, C::kWide);
  const tc::Desc dv = tc::desc_of(sc, true, kChunk * 128);
  Ring rc, rk;
  wait(&sm.q_full[m], 0, abort, a.status);

  const auto scores = [&](int j) {
    const int part_of = j % C::kPer;  // of its key tile
    if (part_of == 0) wait(&sm.k_full[rk.i], rk.phase, abort, a.status);
    // the buffer's weights of two steps ago have been multiplied
    if (j >= 2) wait(&sm.pv_done[2 * m + (j & 1)], ((j >> 1) - 1) & 1, abort, a.status);
    tc::fence_after_sync();
    const tc::Desc k = dk + (rk.i * C::kTileBytes + part_of * C::kStep * C::kRowBytes);
    const uint32_t to = t_s + (j & 1) * C::kStep;
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int panel = 32 * i / C::kRowBytes, b = 32 * i % C::kRowBytes;
        tc::mma_ss<true>(to, dq + (part * C::kQBytes + panel * 128 * C::kRowBytes + b),
                         k + (panel * C::kPanelBytes + b), id_s, part > 0 || i > 0, leader);
      }
    tc::commit_by(&sm.s_full[2 * m + (j & 1)], leader);
    if (part_of == C::kPer - 1) {
      tc::commit_by(&sm.k_empty[rk.i], leader);
      rk.next(C::kKStages);
    }
  };

  scores(0);
  if (n > 1) scores(1);
  for (int j = 0; j < n; ++j) {
#pragma unroll
    for (int c = 0; c < C::kStep / kChunk; ++c) {
      wait(&sm.c_full[rc.i], rc.phase, abort, a.status);
      if (c == 0) wait(&sm.p_full[2 * m + (j & 1)], (j >> 1) & 1, abort, a.status);
      tc::fence_after_sync();
      const tc::Desc v = dv + rc.i * C::kCBytes;
#pragma unroll
      for (int i = 0; i < kChunk / 16; ++i)
        // 16 keys: two groups of eight rows of 1024 bytes; blocks of 64 values behind
        tc::mma_ts_f16(t_o, t_s + (j & 1) * C::kStep + c * 32 + i * 8, v + i * 2048, id_o,
                       j > 0 || c > 0 || i > 0, leader);
      tc::commit_by(&sm.c_empty[rc.i], leader);
      rc.next(C::kCStages);
    }
    tc::commit_by(&sm.pv_done[2 * m + (j & 1)], leader);
    if (j + 2 < n) scores(j + 2);
  }
}

// ---- the softmax warps --------------------------------------------------------------
// What a row does not see of 64 keys becomes minus infinity, and keys that it sees whose
// values hold a NaN become NaN weights.  Done to the scores themselves, so that what
// follows is the same for tiles with and without an edge: as compares at each use an edge
// took 3.7 us of a CTA, now less than one.
struct RowMask {
  unsigned long long seen, nan;
};

// low, high: the columns [low, high] that the row sees; absent: 16-key groups that it does
// not; poison: columns with a NaN value.
__device__ __forceinline__ RowMask row_mask(int low, int high, uint32_t absent,
                                            unsigned long long poison) {
  RowMask mk;
  mk.seen = high < 0 ? 0 : high >= 63 ? ~0ull : (2ull << high) - 1;
  mk.seen &= low <= 0 ? ~0ull : low > 63 ? 0 : ~0ull << low;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    if ((absent >> g) & 1) mk.seen &= ~(0xFFFFull << (16 * g));
  mk.nan = mk.seen & poison;
  return mk;
}

__device__ __forceinline__ void hide64(uint32_t (&v)[2][32], const RowMask& mk) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t seen = (uint32_t)(mk.seen >> (32 * h));
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((seen >> c) & 1)) v[h][c] = 0xFF800000u;
  }
  if (__any_sync(0xffffffffu, mk.nan != 0)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t nan = (uint32_t)(mk.nan >> (32 * h));
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if ((nan >> c) & 1) v[h][c] = 0x7FFFFFFFu;
    }
  }
}

// The largest of a row's 64 scores, in log2 units, with their pages' scales (x) and without
// (y); NaN scores do not count.
__device__ __forceinline__ float2 peak64(const uint32_t (&v)[2][32], const float* f,
                                         const float* lvs) {
  float2 peak = make_float2(-INFINITY, -INFINITY);
  const float4 lv = *reinterpret_cast<const float4*>(lvs);
  const float log_vs[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float x[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(v[g >> 1][16 * (g & 1) + c]);
    float y[5];
#pragma unroll
    for (int c = 0; c < 5; ++c) y[c] = max3(x[3 * c], x[3 * c + 1], x[3 * c + 2]);
    const float m = fmaxf(max3(y[0], y[1], y[2]), max3(y[3], y[4], x[15])) * f[g];
    peak.x = fmaxf(peak.x, m + log_vs[g]);
    peak.y = fmaxf(peak.y, m);
  }
  return peak;
}

// Weights of a row's 64 keys (16-key groups group0 on of the tile),
// 2^(s f + lambda - r_base) by groups of 16, as fp16 to tensor memory, and no group's with an
// exponent below s f + least; returns their sum freed of the pages' value scales and times `up`.
__device__ __forceinline__ float weigh64(const uint32_t (&v)[2][32], uint32_t t_p, const float* f,
                                         const Meta& me, int group0, float r_base, float up,
                                         float least) {
  float sum = 0.0f;
  const float4 lv = *reinterpret_cast<const float4*>(me.log_vs + group0);
  const float4 iv = *reinterpret_cast<const float4*>(me.inv_vs + group0);
  const float log_vs[4] = {lv.x, lv.y, lv.z, lv.w}, inv_vs[4] = {iv.x, iv.y, iv.z, iv.w};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[16];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int g = 2 * h + q;
      const float base = fmaxf(log_vs[g] - r_base, least);
      const float inv = fminf(inv_vs[g] * up, 0x1p40f);  // 2^kLeast
      const float2 ff = make_float2(f[g], f[g]), bb = make_float2(base, base);
      float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 x = fma2(make_float2(__uint_as_float(v[h][16 * q + 2 * i]),
                                    __uint_as_float(v[h][16 * q + 2 * i + 1])),
                        ff, bb);
        x.x = exp2_approx(x.x);
        x.y = exp2_approx(x.y);
        acc[i & 1] = add2(acc[i & 1], x);
        p[8 * q + i] = f16x2_of(x.x, x.y);
      }
      const float2 t = add2(acc[0], acc[1]);
      sum = fmaf(t.x + t.y, inv, sum);
    }
    tc::tmem_st(t_p + 16 * h, p);
  }
  return sum;
}

template <int D>
__device__ __forceinline__ void soften(const AttnArgs& a, const Work& w, int tile, uint32_t tmem,
                                       const float* fac_of, PrSmem<D>& sm, float& r_out,
                                       float& m_out, float& l_out) {
  using C = Pr<D>;
  const int row = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)(row & 96) << 16;
  const uint32_t t_o = tmem + lanes + 256 + tile * D;
  int* abort = &sm.abort;
  const int first = w.v.first + w.tok0 + tile * w.tq;        // earliest row of the tile
  const int toks = min(w.tq, w.toks - tile * w.tq);
  const int pos = first + min(row / a.g, toks - 1);
  // tiles are looked at key by key, and their NaN values taken out of V, by what the
  // CTA's rows see: a row tile that sees all keys has to know of those values too
  const int pos0 = w.v.first + w.tok0, pos1 = pos0 + w.toks - 1;
  const float fac = fac_of[row];
  float r = -INFINITY, m = -INFINITY, l = 0.0f;
  float up = 0.0f;  // 2^(r - m), over the weights' 2^5
  const int n = C::kPer * (w.t1 - w.t0);
  for (int j = 0; j < n; ++j) {
    const int i = j / C::kPer, kt = w.t0 + i, slot = i % C::kMeta, buf = 2 * tile + (j & 1);
    const int part = j % C::kPer, group0 = part * (C::kStep / 16);
    if (part == 0) wait(&sm.meta_full[slot], (i / C::kMeta) & 1, abort, a.status);
    const Meta& me = sm.meta[slot];
    const bool edge = edge_tile(a, w, kt, pos0, pos1) || me.absent != 0;
    RowMask mk[C::kStep / 64];
    if (edge) {
      if (part == 0) wait(&sm.poison_full[slot], (i / C::kMeta) & 1, abort, a.status);
      const int key0 = kt * kKeys + part * C::kStep;
      const int high = min(pos - key0, kKeys);
      const int low = a.window ? pos - a.window + 1 - key0 : -1;
#pragma unroll
      for (int c = 0; c < C::kStep / 64; ++c) {
        const uint32_t* bits = sm.poison[slot] + group0 / 2 + 2 * c;
        mk[c] = row_mask(low - 64 * c, high - 64 * c, me.absent >> (group0 + 4 * c),
                         bits[0] | (unsigned long long)bits[1] << 32);
      }
    }
    float f[C::kStep / 16];
#pragma unroll
    for (int k = 0; k < C::kStep / 16; k += 4) {
      const float4 ks = *reinterpret_cast<const float4*>(me.ks + group0 + k);
      f[k] = fac * ks.x, f[k + 1] = fac * ks.y, f[k + 2] = fac * ks.z, f[k + 3] = fac * ks.w;
    }
    if (edge)  // (minus infinity times a factor that has become zero would be NaN)
#pragma unroll
      for (int k = 0; k < C::kStep / 16; ++k) f[k] = fmaxf(f[k], 0x1p-126f);
    wait(&sm.s_full[buf], (j >> 1) & 1, abort, a.status);
    tc::fence_after_sync();
    __syncwarp();
    const uint32_t t_s = tmem + lanes + tile * 128 + (j & 1) * C::kStep;
    uint32_t v[2][32];
    const auto load = [&](int c) {
      tc::tmem_ld_async(t_s + c * 64, v[0]);
      tc::tmem_ld_async(t_s + c * 64 + 32, v[1]);
      tc::wait_ld();
      if (edge) hide64(v, mk[c]);
    };
    float2 peak = make_float2(-INFINITY, -INFINITY);
#pragma unroll
    for (int c = 0; c < C::kStep / 64; ++c) {
      load(c);
      const float2 x = peak64(v, f + 4 * c, me.log_vs + group0 + 4 * c);
      peak = make_float2(fmaxf(peak.x, x.x), fmaxf(peak.y, x.y));
    }
    const bool outgrown = peak.x > r + kLag || peak.y > m + kSumLag;
    if (__any_sync(0xffffffffu, outgrown)) {
      // new references for those of the warp's rows, and their sums brought to them (a row
      // that has not outgrown its own stays as it is, whatever the others see)
      float alpha = 1.0f;
      if (outgrown) {
        const float r_new = fmaxf(r, peak.x), m_new = fmaxf(m, peak.y);
        alpha = exp2_approx(r - r_new);
        l *= exp2_approx(m - m_new);
        r = r_new;
        m = m_new;
        up = exp2_approx(r - m - kShiftLog);
      }
      if (j > 0) {
        wait(&sm.pv_done[buf ^ 1], ((j - 1) >> 1) & 1, abort, a.status);
        tc::fence_after_sync();
        __syncwarp();
#pragma unroll 1
        for (int b = 0; b < D; b += 16) {
          uint32_t o[16];
          tc::tmem_ld_async(t_o + b, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tc::tmem_st(t_o + b, o);
        }
      }
    }
    const float r_base = (r == -INFINITY ? 0.0f : r) - kShiftLog;
    const float least = (m == -INFINITY ? 0.0f : -m) - kLeast;
#pragma unroll
    for (int c = 0; c < C::kStep / 64; ++c) {
      if (C::kStep > 64) load(c);  // (64 scores are still in registers)
      l += weigh64(v, t_s + 32 * c, f + 4 * c, me, group0 + 4 * c, r_base, up, least);
    }
    tc::wait_st();
    tc::fence_before_sync();
    tc::mbar_arrive(&sm.p_full[buf]);
  }
  wait(&sm.pv_done[2 * tile + ((n - 1) & 1)], ((n - 1) >> 1) & 1, abort, a.status);
  tc::fence_after_sync();
  __syncwarp();
  r_out = r;
  m_out = m;
  l_out = l;
}

template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
    k_attn_prompt(const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const AttnArgs a, const bf16* q,
                  int64_t q_stride, bf16* out, int64_t out_stride, const AttnSplit sp, int units,
                  int splits) {
  using C = Pr<D>;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* sq = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sk = sq + (size_t)C::kTiles * 2 * C::kQBytes;
  uint8_t* sv = sk + (size_t)C::kKStages * C::kTileBytes;
  uint8_t* sc = sv + (size_t)C::kVStages * C::kVBytes;
  PrSmem<D>& sm = *reinterpret_cast<PrSmem<D>*>(sc + (size_t)C::kCStages * C::kCBytes);
  const int tid = threadIdx.x, warp = tid >> 5;
  // late rows of a prompt see the most keys: they go first
  Work w;
  w.part = blockIdx.x % splits;
  w.parts = splits;
  const int uh = blockIdx.x / splits;
  w.h = uh % a.Hkv;
  const int unit = units - 1 - uh / a.Hkv;
  w.tq = 128 / a.g;
  const int per = C::kTiles * w.tq;
  int u0;
  w.s = unit_seq(a, per, 1, unit, &u0);
  w.v = seq_view(a, w.s);
  if (!w.v.ok && tid == 0) atomicOr(a.status, kAttnBadBatch);
  w.tok0 = (unit - u0) * per;
  const bool none = unit < u0 || w.tok0 >= w.v.n;
  if (none) {
    pdl_wait();  // (what ends before the kernel in front does not wait for it)
    if (splits > 1 && tid == 0) sp.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  w.toks = min(per, w.v.n - w.tok0);
  w.tiles = (w.toks + w.tq - 1) / w.tq;
  w.hi = max(min(w.v.len, w.v.first + w.tok0 + w.toks), 0);
  w.lo = a.window ? max(0, w.v.first + w.tok0 - a.window + 1) : 0;
  w.lo = min(w.lo, w.hi);
  {
    const int k0 = w.lo / kKeys;
    const int k1 = max((int)(((long long)w.hi + kKeys - 1) / kKeys), k0 + 1);
    const int n = k1 - k0;
    w.t0 = k0 + (int)((long long)n * w.part / splits);
    w.t1 = k0 + (int)((long long)n * (w.part + 1) / splits);
  }
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(&sm.k_full[i], 1);
      tc::mbar_init(&sm.k_empty[i], w.tiles);
    }
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.q_full[i], 128);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.p_full[i], 128);
      tc::mbar_init(&sm.pv_done[i], 1);
      tc::mbar_init(&sm.v_full[i], 1);
      tc::mbar_init(&sm.v_empty[i], C::kConvWarps);
      tc::mbar_init(&sm.c_full[i], C::kConvWarps);
      tc::mbar_init(&sm.c_empty[i], w.tiles);
    }
    for (int i = 0; i < C::kMeta; ++i) {
      tc::mbar_init(&sm.meta_full[i], 1);
      tc::mbar_init(&sm.poison_full[i], C::kConvWarps);
    }
    sm.abort = 0;
    tc::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::tmem_alloc(&sm.tmem, 512);
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
  pdl_wait();
  pdl_trigger();
  const bool any = w.t0 < w.t1;  // (a share of fewer tiles than shares may be empty)
  if (warp == kTmaWarp) {
    if (any) copy_tiles<D>(a, w, &kmap, &vmap, sk, sv, sm);
  } else if (warp >= kMmaWarp) {
    if (any && warp - kMmaWarp < w.tiles)
      issue<D>(a, w, warp - kMmaWarp, tc::smem_u32(sq), tc::smem_u32(sk), tc::smem_u32(sc), tmem,
               sm);
  } else if (warp >= C::kConvWarp) {
    if (any) widen_tiles<D>(a, w, sv, sc, sm);
  } else if (warp / 4 < w.tiles) {
    const int tile = warp / 4, row = tid & 127;
    float* fac = sm.fac + tile * 128;
    stage_queries<D>(a, w, tile, q, q_stride, sq + (size_t)tile * 2 * C::kQBytes, fac);
    tc::fence_async_smem();
    tc::mbar_arrive(&sm.q_full[tile]);
    asm volatile("bar.sync %0, 128;\n" ::"r"(3 + tile) : "memory");  // fac is complete
    float r = -INFINITY, m = -INFINITY, l = 0.0f;
    if (any) soften<D>(a, w, tile, tmem, fac, sm, r, m, l);
    const int tok = row / a.g, toks = min(w.tq, w.toks - tile * w.tq);
    const bool valid = tok < toks;
    const uint32_t t_o = tmem + ((uint32_t)(row & 96) << 16) + 256 + tile * D;
    float scale = 0x1p-5f;
    if (splits == 1)
      scale = l == 0.0f ? 0.0f
                        : __fdividef(m == -INFINITY ? 1.0f : exp2_approx(r - m - kShiftLog), l);
    bf16* to = out + (int64_t)(w.v.row0 + w.tok0 + tile * w.tq + tok) * out_stride +
               (w.h * a.g + row - tok * a.g) * D;
    const size_t slot = (size_t)blockIdx.x * kAttnPromptRows + tile * 128;
    bool odd = false;  // the row holds a NaN
#pragma unroll 1
    for (int b = 0; b < D; b += 32) {
      uint32_t v[32];
      if (any) {
        __syncwarp();
        tc::tmem_ld_async(t_o + b, v);
        tc::wait_ld();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = 0;
      }
      if (!valid) continue;
#pragma unroll
      for (int k = 0; k < 32; ++k) odd |= __uint_as_float(v[k]) != __uint_as_float(v[k]);
      if (splits == 1) {
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[k + e]) * scale;
          *reinterpret_cast<uint4*>(to + b + k) = pack8(x);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          __stcg(reinterpret_cast<float4*>(sp.o + slot * D + (b + k) * 128 + 4 * row),
                 make_float4(__uint_as_float(v[k]) * scale, __uint_as_float(v[k + 1]) * scale,
                             __uint_as_float(v[k + 2]) * scale,
                             __uint_as_float(v[k + 3]) * scale));
      }
    }
    if (odd) {
      // a NaN value of a tile that all rows see reaches its own column only: the row is NaN
      // all the same, as where its mask made the weight NaN
      const float nan = __int_as_float(0x7FFFFFFF);
      for (int b = 0; b < D; b += 4)
        if (splits == 1)
          *reinterpret_cast<uint2*>(to + b) = make_uint2(0x7FFF7FFFu, 0x7FFF7FFFu);
        else
          __stcg(reinterpret_cast<float4*>(sp.o + slot * D + b * 128 + 4 * row),
                 make_float4(nan, nan, nan, nan));
    }
    if (splits > 1 && valid) __stcg(sp.sums + slot + row, make_float4(r, m, l, 0.0f));
  }
  if (splits > 1 && tid == 0)  // parts, tokens, first row, key head
    sp.shared[blockIdx.x] =
        w.part == 0 ? make_int4(splits, w.toks, w.v.row0 + w.tok0, w.h) : make_int4(0, 0, 0, 0);
  if (warp >= C::kConvWarp && *(volatile int*)&sm.abort) {
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
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a unit's rows, which CTAs of a launch that splits keys left as
// [row tile][4 columns][row] (a row for each thread that writes: 16 bytes of 32 rows side
// by side; row after row the writes took 3 us of a 1024-row chunk's 67).  A thread has four
// columns of a row; kRuns of them take interleaved shares of the parts and are added in
// order.  Bound by the latency of its loads, so the sums of kAhead parts are on their way
// at once: one part after the other made 128 rows over 50000 keys, 148 parts, 145 us; now
// 30.
constexpr int kMergeFew = 16;  // parts up to which a thread takes all

template <int D, bool kFew>
struct Merge {
  static constexpr int kRows = kFew ? 8 : 4, kRuns = kFew ? 1 : 4;
  static constexpr int kThreads = D / 4 * kRows * kRuns;
  static constexpr int kMost = kFew ? kMergeFew : kAttnPromptParts, kAhead = kFew ? 2 : 8;
  static constexpr int kBlocks = Pr<D>::kTiles * 128 / kRows;
};

template <int D, bool kFew>
__global__ void __launch_bounds__(kFew ? 2 * D : 4 * D)
    k_prompt_merge(AttnSplit sp, int g, int splits, bf16* out, int64_t out_stride) {
  using M = Merge<D, kFew>;
  constexpr int kRowThreads = D / 4 * M::kRows;
  __shared__ float4 s_sums[M::kMost][M::kRows];
  __shared__ float4 s_x[M::kRuns][kRowThreads];
  __shared__ float s_l[M::kRuns][kRowThreads];
  pdl_wait();
  const int c0 = blockIdx.x * splits, tid = threadIdx.x;
  const int4 unit = __ldcg(sp.shared + c0);
  const int parts = unit.x, tq = 128 / g;
  const int row0 = blockIdx.y * M::kRows;  // of the unit's row tiles
  const int tile = row0 >> 7;
  // (the block's rows are one tile's: none counts where the first does not)
  if (parts == 0 || (row0 & 127) / g >= tq || tile * tq + (row0 & 127) / g >= unit.y) return;
  const int i = tid % kRowThreads, run = tid / kRowThreads;
  const int row = row0 + i % M::kRows, col = i / M::kRows;
  const int r = row & 127, in = r / g, tok = tile * tq + in;
  const bool on = in < tq && tok < unit.y;
  const float4* o = reinterpret_cast<const float4*>(sp.o) +
                    ((size_t)c0 * kAttnPromptRows + tile * 128) * (D / 4) + col * 128 + r;
  float4 y[M::kAhead];
  const auto load = [&](int p0) {
#pragma unroll
    for (int k = 0; k < M::kAhead; ++k) {
      const int p = p0 + k * M::kRuns;
      y[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (on && p < parts) y[k] = __ldcg(o + (size_t)p * (kAttnPromptRows * (D / 4)));
    }
  };
  load(run);
  for (int e = tid; e < parts * M::kRows; e += M::kThreads) {
    const int p = e / M::kRows, k = e % M::kRows;
    s_sums[p][k] = __ldcg(sp.sums + (size_t)(c0 + p) * kAttnPromptRows + row0 + k);
  }
  __syncthreads();
  float ref = -INFINITY, m = -INFINITY, l = 0.0f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float4 x = s_sums[p][i % M::kRows];
    ref = fmaxf(ref, x.x), m = fmaxf(m, x.y);
  }
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p0 = run;;) {
#pragma unroll
    for (int k = 0; k < M::kAhead; ++k) {
      const int p = p0 + k * M::kRuns;
      if (p < parts) {
        const float4 own = s_sums[p][i % M::kRows];
        const bool none = own.y == -INFINITY;  // (of a row that saw no key its sums are 0, or NaN)
        const float f = none ? 1.0f : exp2_approx(own.x - ref);
        l = fmaf(own.z, none ? 1.0f : exp2_approx(own.y - m), l);
        x = make_float4(fmaf(y[k].x, f, x.x), fmaf(y[k].y, f, x.y), fmaf(y[k].z, f, x.z),
                        fmaf(y[k].w, f, x.w));
      }
    }
    p0 += M::kAhead * M::kRuns;
    if (p0 >= parts) break;
    load(p0);
  }
  if constexpr (M::kRuns > 1) {
    s_x[run][i] = x;
    s_l[run][i] = l;
    __syncthreads();
    if (run > 0) return;
#pragma unroll
    for (int k = 1; k < M::kRuns; ++k) {
      const float4 z = s_x[k][i];
      l += s_l[k][i];
      x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
    }
  }
  if (!on) return;
  const float inv =
      l == 0.0f ? 0.0f : __fdividef(m == -INFINITY ? 1.0f : exp2_approx(ref - m), l);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * inv, x.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(x.z * inv, x.w * inv);
  uint2 v;
  v.x = *reinterpret_cast<const uint32_t*>(&lo);
  v.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(out + (int64_t)(unit.z + tok) * out_stride +
                            (unit.w * g + r - in * g) * D + 4 * col) = v;
}

template <int D>
cudaError_t launch_d(const AttnArgs& a, const AttnMaps& m, const bf16* q, int64_t q_stride,
                     bf16* out, int64_t out_stride, const AttnSplit& sp, int units, int splits,
                     bool pdl, cudaStream_t s) {
  const int heads = units * a.Hkv;
  const cudaError_t e =
      launch_pdl(k_attn_prompt<D>, dim3(heads * splits), dim3(kPThreads), pr_smem_bytes<D>(), s,
                 pdl, m.k, m.v64, a, q, q_stride, out, out_stride, sp, units, splits);
  if (e != cudaSuccess || splits == 1) return e;
  const auto join = [&](auto* kernel, int blocks, int threads) {
    return launch_pdl(kernel, dim3(heads, blocks), dim3(threads), 0, s, true, sp, a.g, splits, out,
                      out_stride);
  };
  return splits <= kMergeFew ? join(k_prompt_merge<D, true>, Merge<D, true>::kBlocks, 2 * D)
                             : join(k_prompt_merge<D, false>, Merge<D, false>::kBlocks, 4 * D);
}

}  // namespace

int attn_prompt_tokens(int D, int g) { return (D == 256 ? 1 : 2) * (128 / g); }

cudaError_t setup_attn_prompt(int D) {
  const auto set = [](auto* kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  };
  return D == 64    ? set(k_attn_prompt<64>, pr_smem_bytes<64>())
         : D == 128 ? set(k_attn_prompt<128>, pr_smem_bytes<128>())
                    : set(k_attn_prompt<256>, pr_smem_bytes<256>());
}

cudaError_t launch_attn_prompt(int D, const AttnArgs& a, const AttnMaps& m, const bf16* q,
                               int64_t q_stride, bf16* out, int64_t out_stride,
                               const AttnSplit& sp, int units, int splits, bool pdl,
                               cudaStream_t s) {
  auto* f = D == 64 ? launch_d<64> : D == 128 ? launch_d<128> : launch_d<256>;
  return f(a, m, q, q_stride, out, out_stride, sp, units, splits, pdl, s);
}

}  // namespace moe
