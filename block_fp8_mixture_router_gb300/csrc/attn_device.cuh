// Device helpers of the attention kernels.
#pragma once

#include "attn_internal.cuh"
#include "moe_device.cuh"

namespace moe {

// Rows and lengths of one sequence, clamped so that no address taken from them
// leaves the caller's buffers.
struct SeqView {
  int row0;   // first row
  int n;      // rows
  int len;    // tokens in the cache
  int first;  // position of the first row (negative: rows in front of the cache)
  bool ok;
};

__device__ __forceinline__ SeqView seq_view(const AttnArgs& a, int s) {
  SeqView v;
  const int r0 = a.row_start[s], r1 = a.row_start[s + 1], len = a.kv_len[s];
  const int cap = (int)min((long long)a.pages_stride << a.page_shift, (long long)kAttnMaxTokens);
  v.row0 = min(max(r0, 0), a.rows);
  v.n = min(max(r1, v.row0), a.rows) - v.row0;
  v.len = min(max(len, 0), cap);
  v.first = v.len - v.n;
  v.ok = v.row0 == r0 && v.row0 + v.n == r1 && v.len == len;
  return v;
}

// The page that holds tokens j << page_shift and on, or -1 where the table
// names none of the cache's (the caller reports it).
__device__ __forceinline__ int page_at(const AttnArgs& a, int s, int j) {
  const int p = a.pages[(size_t)s * a.pages_stride + j];
  return (unsigned)p < (unsigned)a.n_pages ? p : -1;
}

// Work units are numbered without a table of prefix sums: sequence s's units
// begin at row_start[s] / per + extra * s, which leaves room for the
// rows / per + extra it can need.  Returns the sequence of unit u (all
// threads of the block call; u is block-uniform) and its first unit.
__device__ __forceinline__ int unit_seq(const AttnArgs& a, int per, int extra, int u, int* first) {
  int below = 0;  // sequences s >= 1 whose units begin at or before u
  for (int b = 1; b < a.n_seqs; b += blockDim.x) {
    const int s = b + (int)threadIdx.x;
    const bool in = s < a.n_seqs && min(max(a.row_start[s], 0), a.rows) / per + extra * s <= u;
    below += __syncthreads_count(in);
  }
  *first = min(max(a.row_start[below], 0), a.rows) / per + extra * below;
  return below;
}

// The same by each warp on its own, without a barrier: for few sequences.
__device__ __forceinline__ int unit_seq_warp(const AttnArgs& a, int per, int extra, int u,
                                             int* first) {
  const int lane = threadIdx.x & 31;
  int below = 0;
  for (int b = 1; b < a.n_seqs; b += 32) {
    const int s = b + lane;
    const bool in = s < a.n_seqs && min(max(a.row_start[s], 0), a.rows) / per + extra * s <= u;
    below += __popc(__ballot_sync(0xffffffffu, in));
  }
  *first = min(max(a.row_start[below], 0), a.rows) / per + extra * below;
  return below;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Cosine and sine (times the amplitude) of pair i at a position.  The angle in turns is
// the top 32 bits of position x turns[i] modulo 2^64, off by at most 1.25 x 2^-32 of a turn
// (the bits below them, and the entry's rounding).  Its nearest quarter turn is taken out in
// integers, and what is left, at most an eighth, goes as x + y, y the part below x's last
// bit, into Taylor's series to x^9 and x^10, whose next terms stay below 2^-29: in all good
// to 2^-23.  (With the fast functions, good to 2^-21, one stored key in a million came out
// on the other side of a rounding.)
__device__ __forceinline__ float2 rope_cs(const RopeArgs& r, int i, int pos) {
  constexpr float kUnit = 0x1.921fb6p-30f;            // 2 pi / 2^32, and what it leaves
  constexpr float kUnitLow = -0x1.777a5cp-55f;
  const unsigned long long t = (unsigned long long)(long long)pos * r.turns[i];
  const uint32_t u = (uint32_t)(t >> 32) + 0x20000000u;
  const uint32_t quarter = u >> 30;
  const int left = (int)(u & 0x3FFFFFFFu) - 0x20000000;
  const float n = (float)left;
  const float x = n * kUnit;
  const float y = fmaf(n, kUnit, -x) + fmaf(n, kUnitLow, (float)(left - (int)n) * kUnit);
  const float x2 = x * x;
  const float p = fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6);
  const float s0 = x + fmaf(x * x2, p, y);
  const float q = fmaf(
      x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24),
      -0.5f);
  const float c0 = 1.0f + fmaf(x2, q, -x * y);
  const float c = quarter & 1 ? s0 : c0, s = quarter & 1 ? c0 : s0;
  return make_float2((quarter + 1) & 2 ? -c * r.amp : c * r.amp,
                     quarter & 2 ? -s * r.amp : s * r.amp);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool is_finite(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// A value scale as a number between the append's smallest and largest, so that its logarithm
// is one too.
__device__ __forceinline__ float clamp_scale(float x) {
  return fminf(fmaxf(x, __uint_as_float((uint32_t)(127 + kScaleMinExp) << 23)),
               __uint_as_float((uint32_t)(127 + kScaleMaxExp) << 23));
}

// 0x80 in every byte of w that is an e4m3 NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t e4m3_nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

}  // namespace moe
