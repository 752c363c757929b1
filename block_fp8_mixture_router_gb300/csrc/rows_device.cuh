// Device helpers of kernels that work through rows of bf16 values 16 to a lane: loads,
// stores, and the quantisation of a group of 128 by eight lanes.
#pragma once

#include "moe_device.cuh"
#include "ops_internal.cuh"

namespace moe {

__device__ __forceinline__ void unpack8(const uint4& r, float* v) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Columns c .. c + 15 of a row of `width` values (a multiple of 8) as two vectors; zeros
// behind its end.
struct Vec16 {
  uint4 a, b;
};

__device__ __forceinline__ Vec16 load16(const bf16* row, int c, int width, bool on) {
  Vec16 v = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (on && c < width) v.a = *reinterpret_cast<const uint4*>(row + c);
  if (on && c + 8 < width) v.b = *reinterpret_cast<const uint4*>(row + c + 8);
  return v;
}

__device__ __forceinline__ void unpack16(const Vec16& r, float (&v)[16]) {
  unpack8(r.a, v);
  unpack8(r.b, v + 8);
}

__device__ __forceinline__ void store16(bf16* row, int c, int width, const Vec16& v) {
  if (c < width) *reinterpret_cast<uint4*>(row + c) = v.a;
  if (c + 8 < width) *reinterpret_cast<uint4*>(row + c + 8) = v.b;
}

__device__ __forceinline__ Vec16 pack16(const float (&v)[16]) { return {pack8(v), pack8(v + 8)}; }

// v / s rounded to nearest even, given y = RN(1 / s): a quotient within an ulp of v / s
// takes an exact remainder, and one more step from it rounds correctly (Markstein's theorem
// on division by a correctly rounded reciprocal).  v y is within two ulps; the first step
// leaves less than one.  Holds while no remainder falls below the smallest subnormal:
// quotients below e4m3's smallest half step, 2^-10, may be off (they are zeros either way),
// the others' remainders are multiples of 2^-56 s.
// kShort: the first step alone, for what e4m3 makes of the quotient of a bf16 value by a
// bf16 value's 448th.  That step is off where v / s lies within 2^-46 of the middle between
// two floats, and that matters only beside a midpoint c of e4m3 (five bits), half an ulp
// from it: v - s c, a multiple of 2^-28 of the leading bit, would have to be s / 2^25 to
// 2^-21 of it, and s a multiple of 1/8 as nearly, while a seventh of an 8-bit number is a
// multiple (then every product is exact) or 1/56 away from the nearest.
template <bool kShort = false>
__device__ __forceinline__ float div_by(float v, float s, float y) {
  float q = v * y;
  q = fmaf(-fmaf(q, s, -v), y, q);  // (the remainder negated: a zero keeps its sign so)
  return kShort ? q : fmaf(-fmaf(q, s, -v), y, q);
}

// Codes of kN x 16 values of a group whose largest magnitude is m: quant4's codes, without its
// test of every value for a quotient that the product leaves open.  Quotients of bf16 values
// often lie on e4m3's midpoints, where that test sends whole warps to the long division
// (134 M values: 160 us that way, 68 this).  kBf16: the values and m are bf16's.  Returns the
// group's scale.
template <int kN, bool kBf16>
__device__ __forceinline__ float quant_codes(const float (&v)[kN][16], float m, uint4 (&code)[kN]) {
  m = m == 0.0f ? 448.0f : m;  // a group of zeros has the scale 1
  if (m >= 0x1p-80f && m <= 0x1p100f) {
    const float s = div_by(m, 448.0f, 0x1.24924ap-9f);  // RN(1 / 448)
    const float y = __frcp_rn(s);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      float q[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = div_by<kBf16>(v[k][i], s, y);
      code[k] = make_uint4(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]),
                           e4m3x4(q[8], q[9], q[10], q[11]), e4m3x4(q[12], q[13], q[14], q[15]));
    }
    return s;
  }
  const float s = group_scale(m);
#pragma unroll
  for (int k = 0; k < kN; ++k)
    code[k] = make_uint4(quant4(v[k][0], v[k][1], v[k][2], v[k][3], s),
                         quant4(v[k][4], v[k][5], v[k][6], v[k][7], s),
                         quant4(v[k][8], v[k][9], v[k][10], v[k][11], s),
                         quant4(v[k][12], v[k][13], v[k][14], v[k][15], s));
  return s;
}

// Codes and scale of a group of 128 values, 16 in each of eight neighbouring lanes (the
// whole warp calls).
template <bool kBf16>
__device__ __forceinline__ uint4 quant16(const float (&v)[16], float* scale) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  uint4 code[1];
  *scale = quant_codes<1, kBf16>(reinterpret_cast<const float(&)[1][16]>(v), m, code);
  return code[0];
}

// Columns c .. c + 15 of row r of the output, whole groups of eight lanes at a time (the
// whole warp calls; `on` is the same for the lanes of a group).  kBf16: the values are bf16's.
template <bool kCodes, bool kBf16>
__device__ __forceinline__ void put16(const RowsOut& out, size_t r, int c, int width, bool on,
                                      const float (&v)[16]) {
  if constexpr (kCodes) {
    float s;
    const uint4 q = quant16<kBf16>(v, &s);
    if (on && c < width) {
      *reinterpret_cast<uint4*>(out.codes + r * width + c) = q;
      if ((threadIdx.x & 7) == 0) out.scales[r * groups_of(width) + c / kGroup] = s;
    }
  } else if (on) {
    store16(out.v + (int64_t)r * out.stride, c, width, pack16(v));
  }
}

}  // namespace moe
