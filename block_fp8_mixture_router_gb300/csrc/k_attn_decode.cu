// Attention over the 8-bit paged cache for few rows of a sequence (single
// tokens, frames): commit "the Drama 3 text backbone on CUDA" (full attention
// with shared key heads); the cache's format is this library's.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale q . k_j
//
// in one pass over the keys with a running maximum m and sum.  A row tile is 16
// rows: the g query heads of a key head times 16/g tokens.
#include "attn_device.cuh"

namespace moe {

namespace {

constexpr int kDecThreads = 128;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kTileRows = 16;
constexpr float kPShift = 1024.0f;  // weights are held as p x 2^10 in fp16

template <int D>
struct Dec {
  static constexpr int kSlices = D / 64;           // 64-byte slices of a key row
  static constexpr int kOut = D / 8;               // n8 output tiles
  static constexpr int kVBytes = D / 8;            // a lane's bytes of a value row
};

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

// The queries of a tile as e4m3 operands.  A row's values are scaled by the power
// of two that brings its largest into [128, 256) and split into a rounded part
// and the rest, hi + lo: a bf16 value has 8 bits and each part 4, so the two hold
// it exactly down to 1/4 (2^-9 of the row's largest), and to 2^-10, e4m3's half
// step (2^-17 of the largest), below.  The tensor cores then take the keys' codes
// as they are stored.
// Layout: [hi | lo][16 rows][D bytes]; factor[row] = the score's factor but for
// the key's scale.
template <int D>
__device__ __forceinline__ void stage_queries(const AttnArgs& a, const Unit& u, const bf16* q,
                                              int64_t q_stride, uint8_t* sq, float* factor) {
  constexpr int kPer = D / 8;
  const int c = threadIdx.x % kPer, sub = threadIdx.x / kPer;
  for (int r = sub; r < kTileRows; r += kDecThreads / kPer) {
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
    uint2 hi, lo;
    float f = 0.0f;
    if (!is_finite(mx)) {
      hi = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);  // NaN scores
      lo = hi;
    } else {
      const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
      f = __uint_as_float((uint32_t)(127 - 7 + e) << 23) * a.scale;
      uint32_t w[2], z[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x0 = x[4 * i] * up, x1 = x[4 * i + 1] * up, x2 = x[4 * i + 2] * up,
                    x3 = x[4 * i + 3] * up;
        w[i] = e4m3x4(x0, x1, x2, x3);
        const uint32_t h01 = e4m3x2_to_f16x2(w[i]), h23 = e4m3x2_to_f16x2(w[i] >> 16);
        const float2 b01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
        const float2 b23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
        z[i] = e4m3x4(x0 - b01.x, x1 - b01.y, x2 - b23.x, x3 - b23.y);
      }
      hi = make_uint2(w[0], w[1]);
      lo = make_uint2(z[0], z[1]);
    }
    *reinterpret_cast<uint2*>(sq + r * D + 8 * c) = hi;
    *reinterpret_cast<uint2*>(sq + (kTileRows + r) * D + 8 * c) = lo;
    if (c == 0) factor[r] = f;
  }
}

// One CTA's shared memory.
template <int D>
struct DecSmem {
  uint8_t q[2 * kTileRows * D];
  float factor[kTileRows];
  float m[kDecWarps][kTileRows], l[kDecWarps][kTileRows];
  float o[kDecWarps][kTileRows][D];
  int last;
  long long scan[kDecWarps];
};

// A warp's running state over its keys: rows j and j + 8 (j = lane / 4).
template <int D>
struct Acc {
  float o[Dec<D>::kOut][4];
  float m[2], l[2];
  float vref;  // values are held as multiples of it
};

// 16 keys of one page, warp-wide: scores, weights, and the weighted values.
// key0: position of the first; kp, vp: their code rows.  kEdge: some keys are
// unseen by some rows (or lie behind the cache's last token).
template <int D, bool kEdge>
__device__ __forceinline__ void warp_keys(const AttnArgs& a, const Unit& u, Acc<D>& acc,
                                          const uint8_t* sq, const float (&fac)[2], int key0,
                                          const uint8_t* kp, const uint8_t* vp, float ksc,
                                          float vsc) {
  const int lane = threadIdx.x & 31, j = lane >> 2, c = lane & 3;
  constexpr int S = Dec<D>::kSlices;
  // the lane's keys of the second product: 2c, 2c+1, 2c+8, 2c+9
  const int limit = u.v.len - key0;  // keys of this step that exist
  uint4 kq[2][S];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int t = 0; t < S; ++t)
      kq[n][t] = (!kEdge || 8 * n + j < limit)
                     ? *reinterpret_cast<const uint4*>(kp + (8 * n + j) * D + 64 * t + 16 * c)
                     : make_uint4(0, 0, 0, 0);
  float s[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
#pragma unroll
  for (int t = 0; t < S; ++t) {
    const uint8_t* p = sq + j * D + 64 * t + 16 * c;
    const uint4 h0 = *reinterpret_cast<const uint4*>(p);
    const uint4 h1 = *reinterpret_cast<const uint4*>(p + 8 * D);
    const uint4 l0 = *reinterpret_cast<const uint4*>(p + kTileRows * D);
    const uint4 l1 = *reinterpret_cast<const uint4*>(p + (kTileRows + 8) * D);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      mma_e4m3_k64(s[n], h0, h1, kq[n][t]);
      mma_e4m3_k64(s[n], l0, l1, kq[n][t]);
    }
  }
  // value rows of the lane's four keys
  constexpr int W = Dec<D>::kVBytes / 4;
  uint32_t vw[4][W];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int key = 2 * c + (k & 1) + (k & 2) * 4;
    const uint8_t* p = vp + key * D + j * Dec<D>::kVBytes;
    const bool on = !kEdge || key < limit;
    if constexpr (W == 2) {
      const uint2 x = on ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
      vw[k][0] = x.x;
      vw[k][1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 x = on ? *reinterpret_cast<const uint4*>(p + 4 * i) : make_uint4(0, 0, 0, 0);
        vw[k][i] = x.x;
        vw[k][i + 1] = x.y;
        vw[k][i + 2] = x.z;
        vw[k][i + 3] = x.w;
      }
    }
  }
  uint32_t poison = 0;  // bit k: the lane's k-th key has a NaN value
  if constexpr (kEdge) {
    // an unseen key's weight is 0, but 0 x NaN is not: NaN codes become zeros here,
    // and the rows that do see the key get a NaN score instead
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
  // scores in log2 units, masked
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float f = fac[r] * ksc;
    const int row = j + 8 * r;
    const int pos = u.v.first + u.tok0 + row / a.g;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x = s[k >> 1][2 * r + (k & 1)] * f;
      if constexpr (kEdge) {
        const int key = key0 + 2 * c + (k & 1) + (k & 2) * 4;
        const bool seen = key <= pos && key < u.v.len && (!a.window || key > pos - a.window);
        if (poison & (1u << k)) x = __int_as_float(0x7FFFFFFF);
        x = seen ? x : -INFINITY;
      }
      s[k >> 1][2 * r + (k & 1)] = x;
      mx[r] = fmaxf(mx[r], x);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], o));
  }
  // values are held relative to the largest page scale so far
  float vf = 1.0f;
  if (vsc > acc.vref) {
    vf = acc.vref / vsc;
    acc.vref = vsc;
  }
  const float w = __fdividef(vsc, acc.vref) * kPShift;
  float corr[2];
  uint32_t p16[4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float m_new = fmaxf(acc.m[r], mx[r]);
    const float base = m_new == -INFINITY ? 0.0f : m_new;
    const float alpha = exp2_approx(acc.m[r] - base);
    acc.m[r] = m_new;
    float p[4], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      p[k] = exp2_approx(s[k >> 1][2 * r + (k & 1)] - base);
      sum += p[k];
    }
    acc.l[r] = acc.l[r] * alpha + sum;
    corr[r] = alpha * vf;
    p16[r] = f16x2(p[0] * w, p[1] * w);
    p16[2 + r] = f16x2(p[2] * w, p[3] * w);
  }
  if (corr[0] != 1.0f || corr[1] != 1.0f) {
#pragma unroll
    for (int t = 0; t < Dec<D>::kOut; ++t) {
      acc.o[t][0] *= corr[0];
      acc.o[t][1] *= corr[0];
      acc.o[t][2] *= corr[1];
      acc.o[t][3] *= corr[1];
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
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

// Key tiles [t0, t1) of a unit by one CTA.  whole: they are all of the unit's,
// and the output is written; else the partial result goes to slot `slot`, and
// the last of the `parts` CTAs to arrive at counter `c0` merges them all in
// order (the first part lies in slot 2 c0 + 1, the others in 2 (c0 + i)).
template <int D>
__device__ __forceinline__ void run_segment(const AttnArgs& a, const Unit& u, int t0, int t1,
                                            bool whole, int slot, int c0, int first_slot,
                                            int parts, const bf16* q, int64_t q_stride, bf16* out,
                                            int64_t out_stride, const AttnSplit& sp,
                                            DecSmem<D>& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane >> 2, c = lane & 3;
  __syncthreads();  // shared memory is free again
  stage_queries<D>(a, u, q, q_stride, sm.q, sm.factor);
  __syncthreads();
  const float fac[2] = {sm.factor[j], sm.factor[j + 8]};
  Acc<D> acc;
#pragma unroll
  for (int t = 0; t < Dec<D>::kOut; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc.o[t][i] = 0.0f;
  acc.m[0] = acc.m[1] = -INFINITY;
  acc.l[0] = acc.l[1] = 0.0f;
  acc.vref = 0x1p-126f;
  const int P = 1 << a.page_shift;
  const int pos0 = u.v.first + u.tok0;                      // earliest row
  const int pos1 = pos0 + (u.rows - 1) / a.g;               // latest row
  for (int kt = t0; kt < t1; ++kt) {
    const int key0 = kt * kAttnKeys + warp * 16;
    if (key0 >= u.hi || key0 + 16 <= u.lo) continue;
    const int page = page_at(a, u.s, key0 >> a.page_shift);
    if (page < 0) {
      if (lane == 0) atomicOr(a.status, kAttnBadBatch);
      continue;
    }
    const size_t block = (size_t)page * a.Hkv + u.h;
    const size_t at = (block * P + (key0 & (P - 1))) * D;
    const float ksc = a.ks[block], vsc = a.vs[block];
    const bool edge = key0 + 15 > pos0 || (a.window && key0 <= pos1 - a.window);
    if (edge)
      warp_keys<D, true>(a, u, acc, sm.q, fac, key0, a.kc + at, a.vc + at, ksc, vsc);
    else
      warp_keys<D, false>(a, u, acc, sm.q, fac, key0, a.kc + at, a.vc + at, ksc, vsc);
  }
  // join the warps: l over the lanes of a row, then rows scaled to one maximum
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], o);
    if (c == 0) {
      sm.m[warp][j + 8 * r] = acc.m[r];
      sm.l[warp][j + 8 * r] = acc.l[r];
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = j + 8 * r;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, sm.m[w][row]);
    const float f = acc.m[r] == -INFINITY ? 0.0f : exp2_approx(acc.m[r] - m);
    const float g = f * (acc.vref * (1.0f / kPShift));
    // lane's values of the row: 2c kVBytes + t and (2c + 1) kVBytes + t
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < Dec<D>::kOut; t += 4) {
        float4 x = make_float4(acc.o[t][2 * r + h] * g, acc.o[t + 1][2 * r + h] * g,
                               acc.o[t + 2][2 * r + h] * g, acc.o[t + 3][2 * r + h] * g);
        // a warp that saw no key of the row adds nothing, NaN or not
        if (acc.m[r] == -INFINITY && !(acc.l[r] != acc.l[r])) x = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(&sm.o[warp][row][(2 * c + h) * Dec<D>::kVBytes + t]) = x;
      }
  }
  __syncthreads();
  const int rows = u.rows;
  for (int i = tid; i < rows * (D / 4); i += kDecThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, sm.m[w][r]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float mw = sm.m[w][r], lw = sm.l[w][r];
      l += mw == -INFINITY ? lw : lw * exp2_approx(mw - m);
      const float4 y = *reinterpret_cast<const float4*>(&sm.o[w][r][d]);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    if (whole) {
      const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
      store_out<D>(a, u, out, out_stride, r, d,
                   make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    } else {
      const size_t at = (size_t)slot * kTileRows + r;
      __stcg(reinterpret_cast<float4*>(sp.o + at * D + d), x);
      if (d == 0) __stcg(sp.ml + at, make_float2(m, l));
    }
  }
  if (whole) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const int n = atomicAdd(sp.arrived + c0, 1);
    sm.last = n == parts - 1;
    if (sm.last) sp.arrived[c0] = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  for (int i = tid; i < rows * (D / 4); i += kDecThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    float m = -INFINITY, l = 0.0f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < parts; ++p) {
      const size_t at = (size_t)(p == 0 ? first_slot : 2 * (c0 + p)) * kTileRows + r;
      const float2 ml = __ldcg(sp.ml + at);
      const float4 y = __ldcg(reinterpret_cast<const float4*>(sp.o + at * D + d));
      const float mn = fmaxf(m, ml.x);
      const float fo = m == -INFINITY ? 1.0f : exp2_approx(m - mn);
      const float fn = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - mn);
      m = mn;
      l = l * fo + ml.y * fn;
      x = make_float4(x.x * fo + y.x * fn, x.y * fo + y.y * fn, x.z * fo + y.z * fn,
                      x.w * fo + y.w * fn);
    }
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
    store_out<D>(a, u, out, out_stride, r, d,
                 make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  }
}

// kSplit: the key tiles of all units, in unit order, are dealt to the CTAs in
// equal runs, whatever the sequences' lengths are; a unit that several CTAs share
// is merged by the last of them.  Else a CTA per unit.
template <int D, bool kSplit>
__global__ void __launch_bounds__(kDecThreads)
    k_attn_decode(AttnArgs a, const bf16* q, int64_t q_stride, bf16* out, int64_t out_stride,
                  AttnSplit sp) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DecSmem<D>& sm = *reinterpret_cast<DecSmem<D>*>(smem_raw);
  const int tid = threadIdx.x;
  const int tq = tile_tokens(a.g);
  if constexpr (!kSplit) {
    pdl_wait();
    Unit u;
    int u0;
    const int unit = blockIdx.x / a.Hkv;
    u.h = blockIdx.x % a.Hkv;
    u.s = unit_seq(a, tq, 1, unit, &u0);
    u.v = seq_view(a, u.s);
    if (!u.v.ok && tid == 0) atomicOr(a.status, kAttnBadBatch);
    u.t = unit - u0;
    if (u.t < 0 || u.t * tq >= u.v.n) return;
    unit_range(a, u);
    run_segment<D>(a, u, u.kt0, u.kt1, true, 0, 0, 0, 1, q, q_stride, out, out_stride, sp, sm);
    return;
  } else {
    // each thread's run of sequences, their key tiles, and the tiles in front
    const int per_thread = (a.n_seqs + kDecThreads - 1) / kDecThreads;
    const int s0 = min(tid * per_thread, a.n_seqs), s1 = min(s0 + per_thread, a.n_seqs);
    long long mine = 0;
    Unit u;
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
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) front += sm.scan[w];
      total += sm.scan[w];
    }
    if (total == 0) return;
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    const long long begin = per * blockIdx.x, end = min(begin + per, total);
    if (begin >= end) return;
    // the thread whose run holds the first tile finds its unit
    __shared__ int s_seq, s_t;
    __shared__ long long s_front;
    if (mine > 0 && front <= begin && begin < front + mine) {
      long long f = front;
      bool found = false;
      for (int s = s0; s < s1 && !found; ++s) {
        u.v = seq_view(a, s);
        for (u.t = 0; u.t * tq < u.v.n && !found; ++u.t) {
          unit_range(a, u);
          const long long w = (long long)(u.kt1 - u.kt0) * a.Hkv;
          if (begin < f + w) {
            s_seq = s;
            s_t = u.t;
            s_front = f;
            found = true;
          } else {
            f += w;
          }
        }
      }
    }
    __syncthreads();
    u.s = s_seq;
    u.t = s_t;
    long long f = s_front;  // tiles in front of (sequence, row tile)
    u.v = seq_view(a, u.s);
    unit_range(a, u);
    u.h = (int)((begin - f) / (u.kt1 - u.kt0));
    pdl_wait();
    long long at = begin;
    while (at < end) {
      const int w = u.kt1 - u.kt0;
      const long long u_first = f + (long long)u.h * w;  // the unit's first tile
      const long long stop = min(end, u_first + w);
      const bool whole = at == u_first && stop == u_first + w;
      const int c0 = (int)(u_first / per), c1 = (int)((u_first + w - 1) / per);
      // a unit that begins with a CTA's run lies in the CTA's first slot when
      // the CTA only works on it
      const int first_slot = 2 * c0 + 1;
      const int slot = at == u_first ? first_slot : 2 * (int)blockIdx.x;
      run_segment<D>(a, u, u.kt0 + (int)(at - u_first), u.kt0 + (int)(stop - u_first), whole, slot, c0,
                     first_slot, c1 - c0 + 1, q, q_stride, out, out_stride, sp, sm);
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
  }
}

template <int D>
cudaError_t setup_d() {
  cudaError_t e = cudaFuncSetAttribute(k_attn_decode<D, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(DecSmem<D>));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_attn_decode<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(DecSmem<D>));
  return e;
}

template <int D>
int slots_d(int sm_count) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_attn_decode<D, true>, kDecThreads,
                                                    sizeof(DecSmem<D>)) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  return sm_count * (n > 0 ? n : 1);
}

template <int D>
cudaError_t launch_d(const AttnArgs& a, const bf16* q, int64_t q_stride, bf16* out,
                     int64_t out_stride, const AttnSplit& sp, int grid, bool split, bool pdl,
                     cudaStream_t s) {
  return split ? launch_pdl(k_attn_decode<D, true>, dim3(grid), dim3(kDecThreads),
                            sizeof(DecSmem<D>), s, pdl, a, q, q_stride, out, out_stride, sp)
               : launch_pdl(k_attn_decode<D, false>, dim3(grid), dim3(kDecThreads),
                            sizeof(DecSmem<D>), s, pdl, a, q, q_stride, out, out_stride, sp);
}

}  // namespace

cudaError_t setup_attn_decode(int D) {
  return D == 64 ? setup_d<64>() : D == 128 ? setup_d<128>() : setup_d<256>();
}

int attn_decode_slots(int D, int sm_count) {
  return D == 64 ? slots_d<64>(sm_count) : D == 128 ? slots_d<128>(sm_count)
                                                    : slots_d<256>(sm_count);
}

cudaError_t launch_attn_decode(int D, const AttnArgs& a, const bf16* q, int64_t q_stride,
                               bf16* out, int64_t out_stride, const AttnSplit& sp, int grid,
                               bool split, bool pdl, cudaStream_t s) {
  auto* f = D == 64 ? launch_d<64> : D == 128 ? launch_d<128> : launch_d<256>;
  return f(a, q, q_stride, out, out_stride, sp, grid, split, pdl, s);
}

}  // namespace moe
