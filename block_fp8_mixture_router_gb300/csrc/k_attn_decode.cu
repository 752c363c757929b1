// Attention over the 8-bit paged cache for few rows of a sequence (single
// tokens, frames): commit "the Drama 3 text backbone on CUDA" (full attention
// with shared key heads); the cache's format is this library's.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale q . k_j
//
// in one pass over the keys with a running maximum m and sum.  A row tile is 16
// rows: the g query heads of a key head times 16/g tokens.
//
// Bound by the cache's bytes: a CTA has a producer warp that keeps a ring of
// kStages key tiles (128 keys and their values, 32 KB at head_dim 128) filled by
// TMA, and four consumer warps that take 32 keys of a tile each; at head_dim 256
// a second set of four takes the other half of the output.  The tiles lie in
// shared memory with the TMA's swizzle, and a lane's keys are chosen (key_row) so
// that the eight lanes of a shared-memory phase read eight different 16-byte
// columns, of keys and of values alike.
#include "attn_device.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kTileRows = 16;
constexpr int kPair = 2;            // groups of 16 keys that a warp takes of a tile
// Weights are held as p x 2^10 in fp16, and p is taken against a maximum that may
// lag the true one by kLag powers of two: a row's sums are only scaled again where its
// scores outgrow that, and 2^(10 + kLag) is still half of fp16's range.  fp16's
// smallest step is then 2^-34 of a weight of one.
constexpr float kPShift = 1024.0f;
constexpr float kLag = 5.0f;

template <int D>
struct Dec {
  static constexpr int kHalves = D == 256 ? 2 : 1;     // consumer sets, each with its output half
  static constexpr int kConsumers = 128 * kHalves;     // threads
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kDO = D / kHalves;              // output values of a consumer set
  static constexpr int kSlices = D / 64;               // 64-byte slices of a key row
  static constexpr int kOut = kDO / 8;                 // n8 output tiles of a warp
  static constexpr int kVBytes = kDO / 8;              // a lane's bytes of a value row
  static constexpr int kRowBytes = D < 128 ? D : 128;  // a stored row (of a half) and its swizzle
  static constexpr int kHalfBytes = kAttnKeys * kRowBytes;
  static constexpr int kTileBytes = kAttnKeys * D;     // keys or values of a stage
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr int kQStride = 2 * D + 16;          // staged query rows: eight lanes' pieces
                                                       // in eight 16-byte columns
  static constexpr bool kQInRegs = D == 64;
};

// Key of the n8 score tile n that lane group jj's column stands for: columns 2c,
// 2c+1 of tiles 0, 1 are keys 2c, (2c^4)+8, 2c+1, (2c^4)+9 of a warp's sixteen.
__device__ __forceinline__ int key_row(int n, int jj) {
  return ((2 * (jj >> 1)) ^ ((jj & 1) * 4)) + (jj & 1) * 8 + n;
}

// Byte of 16-byte column `col` of row `row` under the TMA's swizzle.
template <int D>
__device__ __forceinline__ int swz(int row, int col) {
  return D == 64 ? row * 64 + ((col ^ ((row >> 1) & 3)) << 4)
                 : row * 128 + ((col ^ (row & 7)) << 4);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)w));
  return h;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}

// What a CTA works on: row tile `t` of sequence `s` for key head h.
struct Unit {
  int s, h, t;
  SeqView v;
  int tok0;       // first token of the tile among the sequence's rows
  int rows;       // valid rows (tokens x g)
  int lo, hi;     // keys [lo, hi) that any row of the tile can see
  int kt0, kt1;   // the key tiles of kAttnKeys that cover them (at least one)
};

__device__ __forceinline__ int tile_tokens(int g) { return kTileRows / g; }

__device__ __forceinline__ void unit_range(const AttnArgs& a, Unit& u) {
  const int tq = tile_tokens(a.g);
  u.tok0 = u.t * tq;
  const int toks = min(tq, u.v.n - u.tok0);
  u.rows = toks * a.g;
  u.hi = max(min(u.v.len, u.v.first + u.tok0 + toks), 0);
  u.lo = a.window ? max(0, u.v.first + u.tok0 - a.window + 1) : 0;
  u.lo = min(u.lo, u.hi);
  u.kt0 = u.lo / kAttnKeys;
  u.kt1 = max((int)(((long long)u.hi + kAttnKeys - 1) / kAttnKeys), u.kt0 + 1);
}

// The queries of a tile as fp16 operands.  A row's values are scaled by the power
// of two that brings its largest into [2^14, 2^15): a bf16 value's 8 bits then fit
// fp16's 11 down to 2^-29 of the row's largest.  (Warp MMAs on e4m3 codes as stored,
// with the queries split into two e4m3 parts, take longer: sm_103a runs them as fp16
// MMAs behind conversions of both operands, 440 instructions a step of 16 keys
// against 300.)
// Layout: [16 rows][kQStride bytes]; factor[row] = the score's factor but for the
// key's scale.
template <int D>
__device__ __forceinline__ void stage_queries(const AttnArgs& a, const Unit& u, const bf16* q,
                                              int64_t q_stride, uint8_t* sq, float* factor) {
  constexpr int kPer = D / 8;
  const int c = threadIdx.x % kPer, sub = threadIdx.x / kPer;
  for (int r = sub; r < kTileRows; r += Dec<D>::kConsumers / kPer) {
    const bool on = r < u.rows;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (on) {
      const int row = u.v.row0 + u.tok0 + r / a.g;
      raw = *reinterpret_cast<const uint4*>(q + (int64_t)row * q_stride +
                                            (u.h * a.g + r % a.g) * D + 8 * c);
    }
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
    uint4 w = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);  // NaN scores
    float f = 0.0f;
    if (is_finite(mx)) {
      const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      f = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * a.scale;
      w = make_uint4(f16x2(x[0] * up, x[1] * up), f16x2(x[2] * up, x[3] * up),
                     f16x2(x[4] * up, x[5] * up), f16x2(x[6] * up, x[7] * up));
    }
    *reinterpret_cast<uint4*>(sq + r * Dec<D>::kQStride + 16 * c) = w;
    if (c == 0) factor[r] = f;
  }
}

// One CTA's shared memory behind the ring.
template <int D>
struct DecSmem {
  uint8_t q[kTileRows * Dec<D>::kQStride];
  float o[kTileRows][D];
  float factor[kTileRows];
  float m[4][kTileRows], l[4][kTileRows];
  float2 meta[Dec<D>::kStages][kAttnKeys / 16];  // scales of 16 keys and their values
  uint64_t full[Dec<D>::kStages], empty[Dec<D>::kStages];
  int last, abort, seq, tile;
  long long front;
  long long scan[Dec<D>::kThreads / 32];
};

template <int D>
constexpr size_t dec_smem_bytes() {
  return 1024 + (size_t)Dec<D>::kStages * 2 * Dec<D>::kTileBytes + sizeof(DecSmem<D>);
}

// A warp's running state over its keys: rows j and j + 8 (j = lane / 4).
template <int D>
struct Acc {
  float o[Dec<D>::kOut][4];
  float m[2], l[2];
  float vref;  // values are held as multiples of it
  float up;    // kPShift / vref
};

// The first operand of the score product over 64 values: the lane's 16 values of
// rows j and j + 8.
struct QFrag {
  uint4 lo[2], hi[2];  // rows j, j + 8; first and second eight
};

template <int D>
__device__ __forceinline__ QFrag load_q(const uint8_t* sq, int j, int c, int t) {
  const uint8_t* p = sq + j * Dec<D>::kQStride + 128 * t + 32 * c;
  QFrag f;
  f.lo[0] = *reinterpret_cast<const uint4*>(p);
  f.hi[0] = *reinterpret_cast<const uint4*>(p + 16);
  f.lo[1] = *reinterpret_cast<const uint4*>(p + 8 * Dec<D>::kQStride);
  f.hi[1] = *reinterpret_cast<const uint4*>(p + 8 * Dec<D>::kQStride + 16);
  return f;
}

// Scores of 64 values: the order of a dot product is free, so the lane's 16 key
// bytes serve as four MMAs' labels 2c, 2c+1, 2c+8, 2c+9 in turn, and the queries'
// values alike.
__device__ __forceinline__ void mma_q_k64(float (&d)[4], const QFrag& f, const uint4& k) {
  mma_f16(d, f.lo[0].x, f.lo[1].x, f.lo[0].y, f.lo[1].y, e4m3x2_to_f16x2(k.x),
          e4m3x2_to_f16x2(k.x >> 16));
  mma_f16(d, f.lo[0].z, f.lo[1].z, f.lo[0].w, f.lo[1].w, e4m3x2_to_f16x2(k.y),
          e4m3x2_to_f16x2(k.y >> 16));
  mma_f16(d, f.hi[0].x, f.hi[1].x, f.hi[0].y, f.hi[1].y, e4m3x2_to_f16x2(k.z),
          e4m3x2_to_f16x2(k.z >> 16));
  mma_f16(d, f.hi[0].z, f.hi[1].z, f.hi[0].w, f.hi[1].w, e4m3x2_to_f16x2(k.w),
          e4m3x2_to_f16x2(k.w >> 16));
}

// Weighted values of 16 keys: V's fragments straight from its rows, a pair of keys'
// bytes interleaved and widened for each MMA.
template <int D>
__device__ __forceinline__ void add_values(Acc<D>& acc, const uint32_t (&p16)[4],
                                           const uint32_t (&vw)[4][Dec<D>::kVBytes / 4]) {
#pragma unroll
  for (int i = 0; i < Dec<D>::kVBytes / 4; ++i) {
    const uint32_t a01 = __byte_perm(vw[0][i], vw[1][i], 0x5140);
    const uint32_t a23 = __byte_perm(vw[0][i], vw[1][i], 0x7362);
    const uint32_t b01 = __byte_perm(vw[2][i], vw[3][i], 0x5140);
    const uint32_t b23 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
    mma_f16(acc.o[4 * i], p16[0], p16[1], p16[2], p16[3], e4m3x2_to_f16x2(a01),
            e4m3x2_to_f16x2(b01));
    mma_f16(acc.o[4 * i + 1], p16[0], p16[1], p16[2], p16[3], e4m3x2_to_f16x2(a01 >> 16),
            e4m3x2_to_f16x2(b01 >> 16));
    mma_f16(acc.o[4 * i + 2], p16[0], p16[1], p16[2], p16[3], e4m3x2_to_f16x2(a23),
            e4m3x2_to_f16x2(b23));
    mma_f16(acc.o[4 * i + 3], p16[0], p16[1], p16[2], p16[3], e4m3x2_to_f16x2(a23 >> 16),
            e4m3x2_to_f16x2(b23 >> 16));
  }
}

// kPair groups of 16 keys (each of one page), warp-wide: scores, weights, and the
// weighted values.  key0: position of the first; kp, vp: the stage's key rows and the
// rows of the warp's half of the values; sc: the groups' scales.  kEdge: some keys
// are unseen by some rows, lie behind the cache's last token, or belong to a page that
// does not exist (there: bit g of `there` clear).
template <int D, bool kEdge>
__device__ __forceinline__ void warp_keys(const AttnArgs& a, const Unit& u, Acc<D>& acc,
                                          const QFrag* qf, const uint8_t* sq,
                                          const float (&fac)[2], int key0, const uint8_t* kp,
                                          const uint8_t* vp, const float2 (&sc)[kPair],
                                          uint32_t there) {
  const int lane = threadIdx.x & 31, j = lane >> 2, c = lane & 3;
  constexpr int S = Dec<D>::kSlices;
  float s[kPair][2][4];
#pragma unroll
  for (int g = 0; g < kPair; ++g)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[g][n][i] = 0.0f;
#pragma unroll
  for (int t = 0; t < S; ++t) {
    const QFrag f = Dec<D>::kQInRegs ? qf[t] : load_q<D>(sq, j, c, t);
#pragma unroll
    for (int g = 0; g < kPair; ++g)
#pragma unroll
      for (int n = 0; n < 2; ++n)
        mma_q_k64(s[g][n], f,
                  *reinterpret_cast<const uint4*>(kp + (t >> 1) * Dec<D>::kHalfBytes +
                                                  g * 16 * Dec<D>::kRowBytes +
                                                  swz<D>(key_row(n, j), 4 * (t & 1) + c)));
  }
  // the rows' factors to log2 units; which keys they see; whether a score outgrew
  // the row's reference, or a page's scale the largest so far
  uint32_t seen[2] = {~0u, ~0u};  // bits 4 g + k of rows j, j + 8
  float f[kPair][2], mx[2] = {-INFINITY, -INFINITY}, top = 0.0f;
#pragma unroll
  for (int g = 0; g < kPair; ++g) {
    if (!kEdge || ((there >> g) & 1)) top = fmaxf(top, sc[g].y);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      f[g][r] = fac[r] * sc[g].x;
      float m = -INFINITY;
      if constexpr (kEdge) {
        const int pos = u.v.first + u.tok0 + (j + 8 * r) / a.g;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = key0 + 16 * g + key_row(k >> 1, 2 * c + (k & 1));
          const bool on = ((there >> g) & 1) && key <= pos && key < u.v.len &&
                          (!a.window || key > pos - a.window);
          if (on) m = fmaxf(m, s[g][k >> 1][2 * r + (k & 1)]);
          else seen[r] &= ~(1u << (4 * g + k));
        }
      } else {
        m = fmaxf(fmaxf(s[g][0][2 * r], s[g][0][2 * r + 1]),
                  fmaxf(s[g][1][2 * r], s[g][1][2 * r + 1]));
      }
      if (m != -INFINITY) mx[r] = fmaxf(mx[r], m * f[g][r]);
    }
  }
  const bool grow = top > acc.vref || mx[0] > acc.m[0] + kLag || mx[1] > acc.m[1] + kLag;
  if (__any_sync(0xffffffffu, grow)) {
    // new references: the rows' running maxima, and the largest page scale so far
    const float vf = top > acc.vref ? __fdiv_rn(acc.vref, top) : 1.0f;
    acc.vref = fmaxf(acc.vref, top);
    acc.up = __fdiv_rn(kPShift, acc.vref);
    float corr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], o));
      const float m_new = fmaxf(acc.m[r], mx[r]);
      const float alpha = m_new == -INFINITY ? 1.0f : exp2_approx(acc.m[r] - m_new);
      acc.m[r] = m_new;
      acc.l[r] *= alpha;
      corr[r] = alpha * vf;
    }
#pragma unroll
    for (int t = 0; t < Dec<D>::kOut; ++t) {
      acc.o[t][0] *= corr[0];
      acc.o[t][1] *= corr[0];
      acc.o[t][2] *= corr[1];
      acc.o[t][3] *= corr[1];
    }
  }
#pragma unroll
  for (int g = 0; g < kPair; ++g) {
    // value rows of the lane's four keys: key_row(0, 2c), (0, 2c+1), (1, 2c), (1, 2c+1)
    constexpr int W = Dec<D>::kVBytes / 4;
    const int limit = !kEdge ? 16 : ((there >> g) & 1) ? u.v.len - key0 - 16 * g : 0;
    uint32_t vw[4][W];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int key = key_row(k >> 1, 2 * c + (k & 1));
      const bool on = !kEdge || key < limit;
      const uint8_t* p = vp + g * 16 * Dec<D>::kRowBytes;
      if constexpr (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + swz<D>(key, j >> 1) + 8 * (j & 1));
        vw[k][0] = on ? x.x : 0;
        vw[k][1] = on ? x.y : 0;
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p + swz<D>(key, j));
        vw[k][0] = on ? x.x : 0;
        vw[k][1] = on ? x.y : 0;
        vw[k][2] = on ? x.z : 0;
        vw[k][3] = on ? x.w : 0;
      }
    }
    uint32_t poison = 0;  // bit k: the lane's k-th key has a NaN value
    if constexpr (kEdge) {
      // an unseen key's weight is 0, but 0 x NaN is not: NaN codes become zeros here,
      // and the rows that do see the key get a NaN weight instead
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t bad = e4m3_nan_bytes(vw[k][i]);
          if (bad) {
            poison |= 1u << k;
            vw[k][i] &= ~((bad >> 7) * 0xFFu);
          }
        }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) poison |= __shfl_xor_sync(0xffffffffu, poison, o);
    }
    // the weights carry the page's scale in their exponent, and the sum of them is
    // freed of it again; a page below 2^-70 of the largest adds no value that counts
    const float w = fmaxf(sc[g].y * acc.up, 0x1p-60f);
    float lw, w_inv;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(lw) : "f"(w));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(w_inv) : "f"(w));
    uint32_t p16[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float base = acc.m[r] == -INFINITY ? lw : lw - acc.m[r];
      float p[4], sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = exp2_approx(fmaf(s[g][k >> 1][2 * r + (k & 1)], f[g][r], base));
        if constexpr (kEdge) {
          if (poison & (1u << k)) p[k] = __int_as_float(0x7FFFFFFF);
          if (!(seen[r] & (1u << (4 * g + k)))) p[k] = 0.0f;
        }
        sum += p[k];
      }
      acc.l[r] = kEdge && !((there >> g) & 1) ? acc.l[r] : fmaf(sum, w_inv, acc.l[r]);
      p16[r] = f16x2(p[0], p[1]);
      p16[2 + r] = f16x2(p[2], p[3]);
    }
    add_values<D>(acc, p16, vw);
  }
}

// Output of one row piece: 4 values of head row r of the tile.
template <int D>
__device__ __forceinline__ void store_out(const AttnArgs& a, const Unit& u, bf16* out,
                                          int64_t out_stride, int r, int d, const float4& x) {
  const int row = u.v.row0 + u.tok0 + r / a.g;
  const __nv_bfloat162 p0 = __floats2bfloat162_rn(x.x, x.y), p1 = __floats2bfloat162_rn(x.z, x.w);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&p0);
  w.y = *reinterpret_cast<const uint32_t*>(&p1);
  *reinterpret_cast<uint2*>(out + (int64_t)row * out_stride + (u.h * a.g + r % a.g) * D + d) = w;
}

// a / b for a, b >= 0: a 32-bit division wherever both fit.
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Barrier of the consumer warps.
template <int D>
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(Dec<D>::kConsumers) : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}

// The ring's next stage and the parity of its barriers.
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

// The producer warp's part of key tiles [t0, t1): a lane for each box (a page's
// share of a tile) of up to 32 looks up page and scales, then each tile's lanes copy
// their boxes once its stage is free.
template <int D>
__device__ __forceinline__ void produce(const AttnArgs& a, const Unit& u, int t0, int t1,
                                        const CUtensorMap* kmap, const CUtensorMap* vmap,
                                        uint8_t* ring, DecSmem<D>& sm, Ring& r) {
  using C = Dec<D>;
  const int lane = threadIdx.x & 31;
  const int box_rows = min(1 << a.page_shift, kAttnKeys);
  const int per_tile = kAttnKeys / box_rows;
  const int batch = 32 / per_tile;  // tiles of a batch of boxes
  for (int kt0 = t0; kt0 < t1; kt0 += batch) {
    const int tiles = min(batch, t1 - kt0);
    const int key = kt0 * kAttnKeys + lane * box_rows;
    bool on = lane < tiles * per_tile && key < u.hi && key + box_rows > u.lo;
    int page = 0;
    float ks = 0.0f, vs = 0.0f;
    if (on) {
      page = page_at(a, u.s, key >> a.page_shift);
      if (page < 0) {
        atomicOr(a.status, kAttnBadBatch);
        on = false;
        ks = -1.0f;  // its keys count as absent
      } else {
        ks = a.ks[(size_t)page * a.Hkv + u.h];  // used after the first copies are out
        vs = a.vs[(size_t)page * a.Hkv + u.h];
      }
    }
    const int y = (u.h << a.page_shift) + (key & ((1 << a.page_shift) - 1));
    for (int i = 0; i < tiles; ++i) {
      tc::wait_bounded(&sm.empty[r.stage], r.phase ^ 1, &sm.abort, a.status);
      if (*(volatile int*)&sm.abort) return;
      const int sub = lane - i * per_tile;  // this lane's box in the tile
      const bool mine = sub >= 0 && sub < per_tile;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine && on));
      if (mine && on) {
        uint8_t* k = ring + (size_t)r.stage * 2 * C::kTileBytes + sub * box_rows * C::kRowBytes;
#pragma unroll
        for (int half = 0; half < D / C::kRowBytes; ++half) {
          tma_load_3d(k + half * C::kHalfBytes, kmap, half * 128, y, page, &sm.full[r.stage]);
          tma_load_3d(k + C::kTileBytes + half * C::kHalfBytes, vmap, half * 128, y, page,
                      &sm.full[r.stage]);
        }
      }
      // the stage's one arrival, with the bytes to expect, follows the scales
      if (mine)
        for (int g = sub * box_rows / 16; g < (sub + 1) * box_rows / 16; ++g)
          sm.meta[r.stage][g] = make_float2(ks, vs);
      __syncwarp();
      if (lane == 0)
        tc::mbar_arrive_expect_tx(&sm.full[r.stage], boxes * box_rows * D * 2);
      r.next(C::kStages);
    }
  }
}

// The consumers' part of key tiles [t0, t1) of a unit.  whole: they are all of
// the unit's, and the output is written; else the partial result goes to slot
// `slot`, and the last of the `parts` CTAs to arrive at counter `c0` merges them all
// in order (the first part lies in slot 2 c0 + 1, the others in 2 (c0 + i)).
template <int D>
__device__ __forceinline__ void consume(const AttnArgs& a, const Unit& u, int t0, int t1,
                                        bool whole, int slot, int c0, int parts, const bf16* q,
                                        int64_t q_stride, bf16* out, int64_t out_stride,
                                        const AttnSplit& sp, const uint8_t* ring, DecSmem<D>& sm,
                                        Ring& r) {
  using C = Dec<D>;
  const int tid = threadIdx.x, lane = tid & 31, j = lane >> 2, c = lane & 3;
  const int grp = (tid >> 5) & 3, half = tid >> 7;  // keys of a tile, output half
  consumer_sync<D>();  // shared memory is free again
  stage_queries<D>(a, u, q, q_stride, sm.q, sm.factor);
  consumer_sync<D>();
  const float fac[2] = {sm.factor[j], sm.factor[j + 8]};
  QFrag qf[C::kQInRegs ? C::kSlices : 1];
  if constexpr (C::kQInRegs)
#pragma unroll
    for (int t = 0; t < C::kSlices; ++t) qf[t] = load_q<D>(sm.q, j, c, t);
  Acc<D> acc;
#pragma unroll
  for (int t = 0; t < C::kOut; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc.o[t][i] = 0.0f;
  acc.m[0] = acc.m[1] = -INFINITY;
  acc.l[0] = acc.l[1] = 0.0f;
  acc.vref = 0x1p-126f;  // any page's scale replaces it
  acc.up = 0.0f;
  const int pos0 = u.v.first + u.tok0;                      // earliest row
  const int pos1 = pos0 + (u.rows - 1) / a.g;               // latest row
  for (int kt = t0; kt < t1; ++kt) {
    tc::wait_bounded(&sm.full[r.stage], r.phase, &sm.abort, a.status);
    const int key0 = kt * kAttnKeys + grp * 16 * kPair;
    if (key0 < u.hi && key0 + 16 * kPair > u.lo) {
      float2 sc[kPair];
      uint32_t there = 0;
#pragma unroll
      for (int g = 0; g < kPair; ++g) {
        sc[g] = sm.meta[r.stage][kPair * grp + g];
        const int k = key0 + 16 * g;
        if (k < u.hi && k + 16 > u.lo && sc[g].x >= 0.0f) there |= 1u << g;
      }
      const uint8_t* kp =
          ring + (size_t)r.stage * 2 * C::kTileBytes + grp * 16 * kPair * C::kRowBytes;
      const uint8_t* vp = kp + C::kTileBytes + half * C::kHalfBytes;
      const bool edge = key0 + 16 * kPair - 1 > pos0 ||
                        (a.window && key0 <= pos1 - a.window) || there != (1u << kPair) - 1;
      if (edge)
        warp_keys<D, true>(a, u, acc, qf, sm.q, fac, key0, kp, vp, sc, there);
      else
        warp_keys<D, false>(a, u, acc, qf, sm.q, fac, key0, kp, vp, sc, there);
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.empty[r.stage]);
    r.next(C::kStages);
  }
  // join the warps: l over the lanes of a row, then rows scaled to one maximum and
  // added in the order of the warps
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) acc.l[i] += __shfl_xor_sync(0xffffffffu, acc.l[i], o);
    if (c == 0 && half == 0) {
      sm.m[grp][j + 8 * i] = acc.m[i];
      sm.l[grp][j + 8 * i] = acc.l[i];
    }
  }
  consumer_sync<D>();
  float g[2];
  bool none[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, sm.m[w][j + 8 * i]);
    const float f = acc.m[i] == -INFINITY ? 0.0f : exp2_approx(acc.m[i] - m);
    g[i] = f * (acc.vref * (1.0f / kPShift));
    // a warp that saw no key of the row adds nothing; one that only saw NaN, NaN
    none[i] = acc.m[i] == -INFINITY && acc.l[i] == acc.l[i];
  }
  for (int w = 0; w < 4; ++w) {
    if (w == grp) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < C::kOut; t += 4) {
            float4* at = reinterpret_cast<float4*>(
                &sm.o[j + 8 * i][half * C::kDO + (2 * c + h) * C::kVBytes + t]);
            float4 x = make_float4(acc.o[t][2 * i + h] * g[i], acc.o[t + 1][2 * i + h] * g[i],
                                   acc.o[t + 2][2 * i + h] * g[i], acc.o[t + 3][2 * i + h] * g[i]);
            if (none[i]) x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (w > 0) {
              const float4 y = *at;
              x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
            }
            *at = x;
          }
    }
    consumer_sync<D>();
  }
  const int rows = u.rows;
  for (int i = tid; i < rows * (D / 4); i += C::kConsumers) {
    const int row = i / (D / 4), d = (i % (D / 4)) * 4;
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, sm.m[w][row]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float mw = sm.m[w][row], lw = sm.l[w][row];
      l += mw == -INFINITY ? lw : lw * exp2_approx(mw - m);
    }
    const float4 x = *reinterpret_cast<const float4*>(&sm.o[row][d]);
    if (whole) {
      const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
      store_out<D>(a, u, out, out_stride, row, d,
                   make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    } else {
      const size_t at = (size_t)slot * kTileRows + row;
      __stcg(reinterpret_cast<float4*>(sp.o + at * D + d), x);
      if (d == 0) __stcg(sp.ml + at, make_float2(m, l));
    }
  }
  if (whole) return;
  __threadfence();
  consumer_sync<D>();
  if (tid == 0) {
    const int n = atomicAdd(sp.arrived + c0, 1);
    sm.last = n == parts - 1;
    if (sm.last) sp.arrived[c0] = 0;
  }
  consumer_sync<D>();
  if (!sm.last) return;
  __threadfence();
  // the parts' loads are independent: the maximum first, then the weighted sum
  for (int i = tid; i < rows * (D / 4); i += C::kConsumers) {
    const int row = i / (D / 4), d = (i % (D / 4)) * 4;
    const auto at = [&](int p) {
      return (size_t)(p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)) * kTileRows + row;
    };
    float m = -INFINITY, l = 0.0f;
#pragma unroll 8
    for (int p = 0; p < parts; ++p) m = fmaxf(m, __ldcg(&sp.ml[at(p)].x));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const float2 ml = __ldcg(sp.ml + at(p));
      const float4 y = __ldcg(reinterpret_cast<const float4*>(sp.o + at(p) * D + d));
      const float f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - m);
      l = fmaf(ml.y, f, l);
      x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
    }
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
    store_out<D>(a, u, out, out_stride, row, d,
                 make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  }
}

// kSplit: the key tiles of all units, in unit order, are dealt to the CTAs in
// equal runs, whatever the sequences' lengths are; a unit that several CTAs share
// is merged by the last of them.  Else a CTA per unit.  The producer and the
// consumers walk the same run.
template <int D, bool kSplit>
__global__ void __launch_bounds__(Dec<D>::kThreads, D == 256 ? 1 : 2)
    k_attn_decode(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const AttnArgs a, const bf16* q, int64_t q_stride, bf16* out, int64_t out_stride,
                  const AttnSplit sp) {
  using C = Dec<D>;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  DecSmem<D>& sm =
      *reinterpret_cast<DecSmem<D>*>(ring + (size_t)C::kStages * 2 * C::kTileBytes);
  const int tid = threadIdx.x;
  const int tq = tile_tokens(a.g);
  const bool producer = tid >= C::kConsumers;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], C::kConsumers / 32);
    }
    sm.abort = 0;
    tc::fence_barrier_init();
  }
  if (producer && (tid & 31) == 0) {
    tc::tma_prefetch_map(&kmap);
    tc::tma_prefetch_map(&vmap);
  }
  Ring r;
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
    if (u.t < 0 || u.t * tq >= u.v.n) return;
    unit_range(a, u);
    // this unit alone: a run that is exactly its tiles
    f = 0;
    begin = (long long)u.h * (u.kt1 - u.kt0);
    end = begin + (u.kt1 - u.kt0);
    per = 0x7FFFFFFFFFFFll;
    __syncthreads();
  } else {
    // each thread's run of sequences, their key tiles, and the tiles in front
    const int per_thread = (a.n_seqs + C::kThreads - 1) / C::kThreads;
    const int s0 = min(tid * per_thread, a.n_seqs), s1 = min(s0 + per_thread, a.n_seqs);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
      u.v = seq_view(a, s);
      if (!u.v.ok) atomicOr(a.status, kAttnBadBatch);
      for (u.t = 0; u.t * tq < u.v.n; ++u.t) {
        unit_range(a, u);
        mine += (long long)(u.kt1 - u.kt0) * a.Hkv;
      }
    }
    const int lane = tid & 31, warp = tid >> 5;
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
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) front += sm.scan[w];
      total += sm.scan[w];
    }
    if (total == 0) return;
    per = div_ll(total + gridDim.x - 1, gridDim.x);
    begin = per * blockIdx.x;
    end = min(begin + per, total);
    if (begin >= end) return;
    // the thread whose run holds the first tile finds its unit
    if (mine > 0 && front <= begin && begin < front + mine) {
      bool found = false;
      f = front;
      for (int s = s0; s < s1 && !found; ++s) {
        u.v = seq_view(a, s);
        for (u.t = 0; u.t * tq < u.v.n && !found; ++u.t) {
          unit_range(a, u);
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
    __syncthreads();
    u.s = sm.seq;
    u.t = sm.tile;
    f = sm.front;  // tiles in front of (sequence, row tile)
    u.v = seq_view(a, u.s);
    unit_range(a, u);
    u.h = (int)div_ll(begin - f, u.kt1 - u.kt0);
  }
  pdl_wait();
  long long at = begin;
  while (at < end) {
    const int w = u.kt1 - u.kt0;
    const long long u_first = f + (long long)u.h * w;  // the unit's first tile
    const long long stop = min(end, u_first + w);
    const int t0 = u.kt0 + (int)(at - u_first), t1 = u.kt0 + (int)(stop - u_first);
    if (producer) {
      produce<D>(a, u, t0, t1, &kmap, &vmap, ring, sm, r);
    } else {
      const bool whole = at == u_first && stop == u_first + w;
      const int c0 = (int)div_ll(u_first, per), c1 = (int)div_ll(u_first + w - 1, per);
      const int slot = at == u_first ? 2 * c0 + 1 : 2 * (int)blockIdx.x;
      consume<D>(a, u, t0, t1, whole, slot, c0, c1 - c0 + 1, q, q_stride, out, out_stride, sp, ring,
                 sm, r);
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
      unit_range(a, u);
    }
  }
  if (producer && *(volatile int*)&sm.abort) {
    // a wait gave up: let this CTA's copies land before its memory goes back
    for (int i = 0; i < C::kStages; ++i)
      for (int k = 0; k < 100000 && !tc::mbar_try_wait(&sm.full[i], 0) &&
                      !tc::mbar_try_wait(&sm.full[i], 1);
           ++k) {
      }
  }
}

template <int D>
cudaError_t setup_d() {
  cudaError_t e = cudaFuncSetAttribute(k_attn_decode<D, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)dec_smem_bytes<D>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_attn_decode<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dec_smem_bytes<D>());
  return e;
}

template <int D>
int slots_d(int sm_count) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_attn_decode<D, true>, Dec<D>::kThreads,
                                                    dec_smem_bytes<D>()) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  return sm_count * (n > 0 ? n : 1);
}

template <int D>
cudaError_t launch_d(const AttnArgs& a, const AttnMaps& m, const bf16* q, int64_t q_stride,
                     bf16* out, int64_t out_stride, const AttnSplit& sp, int grid, bool split,
                     bool pdl, cudaStream_t s) {
  auto* kernel = split ? k_attn_decode<D, true> : k_attn_decode<D, false>;
  return launch_pdl(kernel, dim3(grid), dim3(Dec<D>::kThreads), dec_smem_bytes<D>(), s, pdl, m.k,
                    m.v, a, q, q_stride, out, out_stride, sp);
}

}  // namespace

cudaError_t setup_attn_decode(int D) {
  return D == 64 ? setup_d<64>() : D == 128 ? setup_d<128>() : setup_d<256>();
}

int attn_decode_slots(int D, int sm_count) {
  return D == 64 ? slots_d<64>(sm_count) : D == 128 ? slots_d<128>(sm_count)
                                                    : slots_d<256>(sm_count);
}

cudaError_t launch_attn_decode(int D, const AttnArgs& a, const AttnMaps& m, const bf16* q,
                               int64_t q_stride, bf16* out, int64_t out_stride,
                               const AttnSplit& sp, int grid, bool split, bool pdl,
                               cudaStream_t s) {
  auto* f = D == 64 ? launch_d<64> : D == 128 ? launch_d<128> : launch_d<256>;
  return f(a, m, q, q_stride, out, out_stride, sp, grid, split, pdl, s);
}

}  // namespace moe
