// What happens to the projection's rows before attention: rotary positions
// (with the norm of query and key heads in front), and the append of keys and
// values to the 8-bit paged cache.
//
// Q/K norm and partial rotary positions: commit "the Drama 3 text backbone on
// CUDA"; one prologue launch norms, rotates and caches a row (PR #925, commit
// list).  The cache's format is this library's.
//
// Both are bound by their bytes for many rows and by the launch for few.  A head
// row belongs to D/8 neighbouring lanes, 16 bytes each: loads and stores are
// whole 16-byte pieces, the norm's sum and the half layout's partner values
// travel by shuffles, and since no lane reads another's memory the rotation can
// run in place.  Measured: 20 heads of 128 of 16384 rows rotated in 32.5 us (5.2 TB/s,
// where a plain copy reaches 6.8), of one row in 3.2 us; 10600 rows of keys and values of
// 4 heads in three prompts appended in 10.9 us, a row for each of 64 sequences in 5.7.
#include <algorithm>

#include "attn_device.cuh"

namespace moe {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRopeUnroll = 4;      // head rows per lane group in flight
constexpr int kSmemSeqs = 1024;     // row starts searched in shared memory

template <int D>
struct Lanes {
  static constexpr int kPer = D / 8;                  // lanes of a head row
  static constexpr int kRows = kRowThreads / kPer;    // head rows of a block pass
};

// v *= gamma / sqrt(mean(v^2) + eps) over a head's lanes.
template <int D>
__device__ __forceinline__ void norm_head(float (&v)[8], const bf16* gamma, float eps, int c) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int o = Lanes<D>::kPer / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = __frsqrt_rn(ss * (1.0f / D) + eps);
  float g[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(gamma) + c), g);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * g[i];
}

// Rotates a head held by its lanes (lane c: values 8c..8c+7); cs(i) gives pair
// i's cosine and sine.  All lanes of the warp call.
template <int D, typename Cs>
__device__ __forceinline__ void rotate_head(float (&v)[8], const RopeArgs& r, int c, float* swap,
                                            Cs cs) {
  if (r.rot == 0) return;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if (8 * c + i < r.rot) {
        const float2 w = cs(4 * c + i / 2);
        const float x = v[i], y = v[i + 1];
        v[i] = x * w.x - y * w.y;
        v[i + 1] = y * w.x + x * w.y;
      }
    }
    return;
  }
  const int half = r.rot >> 1;
  float p[8];
  if ((half & 7) == 0) {
    // a lane's eight partners are another lane's eight values
    const int step = half >> 3;
    const int lane = threadIdx.x & 31;
    const int from = c < step ? lane + step : c < 2 * step ? lane - step : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, v[i], from);
  } else {
    float* mine = swap + (threadIdx.x & ~31) * 8 + ((threadIdx.x & 31) - c) * 8;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[8 * c + i] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * c + i;
      p[i] = e < r.rot ? mine[e < half ? e + half : e - half] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 8 * c + i;
    if (e < half) {
      const float2 w = cs(e);
      v[i] = v[i] * w.x - p[i] * w.y;
    } else if (e < r.rot) {
      const float2 w = cs(e - half);
      v[i] = v[i] * w.x + p[i] * w.y;
    }
  }
}

// Head rows [first, first + count) of `heads` per row, starting at row row0,
// with the rows' cosines and sines in `table` [rows][rot/2].  `prepare` fills
// the table and synchronises; the first loads are issued before it.
template <int D, typename Prepare>
__device__ __forceinline__ void rope_items(const bf16* x, int64_t x_stride, int heads, int row0,
                                           int first, int count, const bf16* gamma, float eps,
                                           bf16* y, int64_t y_stride, const RopeArgs& r,
                                           const float2* table, float* swap, Prepare prepare) {
  using L = Lanes<D>;
  const int c = threadIdx.x % L::kPer, sub = threadIdx.x / L::kPer;
  const int half = r.rot >> 1;
  bool ready = false;
  for (int base = 0; base < count; base += kRopeUnroll * L::kRows) {
    uint4 raw[kRopeUnroll];
    int row[kRopeUnroll], head[kRopeUnroll];
#pragma unroll
    for (int k = 0; k < kRopeUnroll; ++k) {
      const int it = base + k * L::kRows + sub;
      raw[k] = make_uint4(0, 0, 0, 0);
      row[k] = (first + it) / heads;
      head[k] = (first + it) - row[k] * heads;
      if (it < count)
        raw[k] = *reinterpret_cast<const uint4*>(x + (int64_t)(row0 + row[k]) * x_stride +
                                                 head[k] * D + 8 * c);
    }
    if (!ready) prepare();
    ready = true;
#pragma unroll
    for (int k = 0; k < kRopeUnroll; ++k) {
      const int it = base + k * L::kRows + sub;
      if (base + k * L::kRows >= count) break;  // the same for the whole block
      const bool on = it < count;
      float v[8];
      unpack8(raw[k], v);
      if (gamma) norm_head<D>(v, gamma, eps, c);
      const float2* t = table + (on ? row[k] : 0) * half;
      rotate_head<D>(v, r, c, swap, [&](int i) { return t[i]; });
      if (on)
        *reinterpret_cast<uint4*>(y + (int64_t)(row0 + row[k]) * y_stride + head[k] * D + 8 * c) =
            pack8(v);
    }
  }
}

// A block takes `block_rows` rows (all of their heads, or one of gridDim.y
// shares of them); the rows' sines are computed once for all heads.
template <int D>
__global__ void __launch_bounds__(kRowThreads, 6)
    k_rope(const bf16* x, int64_t x_stride, int heads, const int* positions, const bf16* gamma,
           float eps, int rows, bf16* y, int64_t y_stride, RopeArgs r, int block_rows) {
  extern __shared__ float2 s_table[];
  __shared__ float s_swap[kRowThreads * 8];
  const int row0 = blockIdx.x * block_rows;
  const int nr = min(block_rows, rows - row0);
  const int items = nr * heads;
  const int share = (items + gridDim.y - 1) / gridDim.y;
  const int first = share * blockIdx.y;
  const int half = r.rot >> 1;
  rope_items<D>(x, x_stride, heads, row0, first, min(share, items - first), gamma, eps, y,
                y_stride, r, s_table, s_swap, [&] {
#pragma unroll 1
                  for (int i = threadIdx.x; i < nr * half; i += kRowThreads)
                    s_table[i] = rope_cs(r, i % half, __ldg(positions + row0 + i / half));
                  __syncthreads();
                });
}

// Scale of a block of values from its largest finite magnitude: the smallest
// 2^k with 448 * 2^k >= amax, 448 = 1.75 * 2^8.  A power of two keeps every
// bit of a code when a later, larger scale makes the older codes of the page
// round again (but for e4m3's subnormal end), and loses none of e4m3's
// relative precision.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  k = max(k, kScaleMinExp);
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

// Four e4m3 codes times f, rounded to e4m3 again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h0) : "h"((uint16_t)w));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h1) : "h"((uint16_t)(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  return e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// One (page, head, K or V) of the call's rows: the values wait in registers
// while the block agrees on the page's scale, so they are read once.
template <int D, int kMost, bool kStep>
__device__ __forceinline__ void append_unit(const AttnArgs& a, const AppendArgs& p, int unit,
                                            int h, bool is_v, float2* table, float* swap) {
  using L = Lanes<D>;
  __shared__ float s_max[kRowThreads / 32];
  const int P = 1 << a.page_shift;
  int u0;
  const int s = a.n_seqs <= 128 ? unit_seq_warp(a, P, 2, unit, &u0) : unit_seq(a, P, 2, unit, &u0);
  const SeqView v = seq_view(a, s);
  if (!v.ok && threadIdx.x == 0) atomicOr(a.status, kAttnBadBatch);
  if (v.n == 0 || v.len == 0 || unit < u0) return;
  const int start = max(v.first, 0);
  const int j = (start >> a.page_shift) + (unit - u0);
  const long long t0 = (long long)j << a.page_shift;
  const int lo = (int)max((long long)start, t0);
  const int hi = (int)min((long long)v.len, t0 + P);
  if (lo >= hi) return;
  const int slot0 = lo - (int)t0, m = hi - lo;
  const int row0 = v.row0 + (lo - v.first);
  const int c = threadIdx.x % L::kPer, sub = threadIdx.x / L::kPer;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const bf16* src = (is_v ? p.v : p.k) + (int64_t)row0 * stride + h * D + 8 * c;
  // the rows are on their way while the page is looked up
  uint4 raw[kMost];
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int i = k * L::kRows + sub;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (i < m) raw[k] = *reinterpret_cast<const uint4*>(src + i * stride);
  }
  const int page = page_at(a, s, j);
  if (page < 0) {
    if (threadIdx.x == 0) atomicOr(a.status, kAttnBadBatch);
    return;
  }
  const size_t block = (size_t)page * a.Hkv + h;
  float* scale_at = (is_v ? a.vs : a.ks) + block;
  const float old = slot0 > 0 ? *scale_at : 0.0f;
  float amax = 0.0f;
  uint32_t bad = 0;  // passes whose row holds an infinity or NaN
  const uint32_t my_lanes = (L::kPer == 32 ? 0xffffffffu : ((1u << (L::kPer & 31)) - 1u))
                            << ((threadIdx.x & 31) - c);
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (k * L::kRows >= m) break;  // the same for the whole block
    float x[8];
    unpack8(raw[k], x);
    if constexpr (kStep) {
      if (!is_v) {
        const int pos = lo + min(k * L::kRows + sub, m - 1);
        if (p.k_gamma) norm_head<D>(x, p.k_gamma, p.eps, c);
        // a row's sines by its lanes, which are one warp's
        float2* cs = table + sub * (D / 2);
        __syncwarp();
        for (int i = c; i < p.rope.rot >> 1; i += L::kPer) cs[i] = rope_cs(p.rope, i, pos);
        __syncwarp();
        rotate_head<D>(x, p.rope, c, swap, [&](int i) { return cs[i]; });
        raw[k] = pack8(x);
        unpack8(raw[k], x);
      }
    }
    bool odd = false;
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      odd |= !is_finite(x[i]);
      mx = fmaxf(mx, fabsf(x[i]));
    }
    const bool row_bad = (__ballot_sync(0xffffffffu, odd) & my_lanes) != 0;
    if (row_bad) bad |= 1u << k;
    else if (k * L::kRows + sub < m) amax = fmaxf(amax, mx);
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  const float fresh = block_scale(amax);
  const float scale = slot0 > 0 ? fmaxf(fresh, old) : fresh;

  uint8_t* codes = (is_v ? a.vc : a.kc) + block * ((size_t)P * D);
  if (slot0 > 0 && scale > old) {
    const float f = __fdiv_rn(old, scale);
    uint4* w = reinterpret_cast<uint4*>(codes);
    for (int i = threadIdx.x; i < slot0 * (D / 16); i += kRowThreads) {
      uint4 q = w[i];
      q.x = rescale4(q.x, f);
      q.y = rescale4(q.y, f);
      q.z = rescale4(q.z, f);
      q.w = rescale4(q.w, f);
      w[i] = q;
    }
  }
  // a power of two divides by an exact product
  const bool whole = (__float_as_uint(scale) & 0x807FFFFFu) == 0 && scale < 0x1p126f;
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int i = k * L::kRows + sub;
    if (i >= m) break;
    float x[8];
    unpack8(raw[k], x);
    uint2 q;
    if (bad & (1u << k)) {
      q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    } else if (whole) {
      q.x = e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      q.y = e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
    } else {  // (a scale of other code's)
      q.x = quant4(x[0], x[1], x[2], x[3], scale);
      q.y = quant4(x[4], x[5], x[6], x[7], scale);
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(slot0 + i) * D + 8 * c) = q;
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

// Blocks [0, units * Hkv * 2) append; the blocks behind them (a step's
// prologue only) norm and rotate the queries of block_rows rows each.
// kMost: passes of a page's tokens, which wait in registers.
template <int D, int kMost, bool kStep>
__global__ void __launch_bounds__(kRowThreads, kMost <= 4 ? 4 : kMost <= 8 ? 3 : 2)
    k_append(AttnArgs a, AppendArgs p, int append_blocks, int block_rows) {
  extern __shared__ float2 s_table[];  // sines of a block's rows, of queries or of keys
  __shared__ float s_swap[kStep ? kRowThreads * 8 : 1];
  pdl_trigger();
  if ((int)blockIdx.x < append_blocks) {
    const int b = blockIdx.x;
    const int uh = b >> 1;
    append_unit<D, kMost, kStep>(a, p, uh / a.Hkv, uh % a.Hkv, b & 1, s_table, s_swap);
    return;
  }
  if constexpr (kStep) {
    __shared__ int s_start[kSmemSeqs + 1];
    const int row0 = (blockIdx.x - append_blocks) * block_rows;
    const int nr = min(block_rows, a.rows - row0);
    const int half = p.rope.rot >> 1;
    rope_items<D>(p.q, p.q_stride, a.Hq, row0, 0, nr * a.Hq, p.q_gamma, p.eps, p.q_out,
                  (int64_t)a.Hq * D, p.rope, s_table, s_swap, [&] {
                    // the rows' positions: their sequences by a search of the row starts
                    const bool in_smem = a.n_seqs <= kSmemSeqs;
                    if (in_smem) {
                      for (int i = threadIdx.x; i <= a.n_seqs; i += kRowThreads)
                        s_start[i] = a.row_start[i];
                      __syncthreads();
                    }
                    const int* start = in_smem ? s_start : a.row_start;
                    int last = -1, pos = 0;
#pragma unroll 1
                    for (int i = threadIdx.x; i < nr * half; i += kRowThreads) {
                      const int row = i / half;
                      if (row != last) {
                        int lo = 0, hi = a.n_seqs;  // largest s with start[s] <= row
                        while (hi - lo > 1) {
                          const int mid = (lo + hi) >> 1;
                          if (start[mid] <= row0 + row) lo = mid; else hi = mid;
                        }
                        const SeqView v = seq_view(a, lo);
                        pos = v.first + (row0 + row - v.row0);
                        last = row;
                      }
                      s_table[i] = rope_cs(p.rope, i - row * half, pos);
                    }
                    __syncthreads();
                  });
  }
}

// Rows whose heads a rope block takes: enough for every lane group to have
// kRopeUnroll head rows in flight.
template <int D>
int rope_block_rows(int heads) {
  return heads >= kRopeUnroll * Lanes<D>::kRows ? 1 : kRopeUnroll * Lanes<D>::kRows / heads;
}

template <int D>
cudaError_t rope_d(const bf16* x, int64_t x_stride, int heads, const int* positions,
                   const bf16* gamma, float eps, int rows, bf16* y, int64_t y_stride,
                   const RopeArgs& r, int sm_count, cudaStream_t s) {
  int br = rope_block_rows<D>(heads);
  // few rows: spread them over the SMs
  while (br > 1 && (rows + br - 1) / br < 2 * sm_count) br = (br + 1) / 2;
  const int blocks = (rows + br - 1) / br;
  const int per = Lanes<D>::kRows * (blocks < sm_count ? 1 : kRopeUnroll);
  const int shares = (br * heads + per - 1) / per;
  k_rope<D><<<dim3(blocks, shares), kRowThreads, (size_t)br * (r.rot / 2) * sizeof(float2), s>>>(
      x, x_stride, heads, positions, gamma, eps, rows, y, y_stride, r, br);
  return cudaGetLastError();
}

template <int D, int kMost>
cudaError_t append_dm(const AttnArgs& a, const AppendArgs& p, cudaStream_t s) {
  const int units = (a.rows >> a.page_shift) + 2 * a.n_seqs;
  const int blocks = units * a.Hkv * 2;
  if (!p.q) {
    k_append<D, kMost, false><<<blocks, kRowThreads, 0, s>>>(a, p, blocks, 0);
  } else {
    const int br = rope_block_rows<D>(a.Hq);
    const int q_blocks = (a.rows + br - 1) / br;
    const int table = std::max(br * (p.rope.rot / 2), Lanes<D>::kRows * (D / 2));
    k_append<D, kMost, true><<<blocks + q_blocks, kRowThreads, table * sizeof(float2), s>>>(
        a, p, blocks, br);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const AttnArgs& a, const AppendArgs& p, cudaStream_t s) {
  // passes of a page: a power of two from one to 128 tokens' worth
  const int passes = (1 << a.page_shift) / Lanes<D>::kRows;
  constexpr int kMax = 128 / Lanes<D>::kRows;
  if (passes <= 1) return append_dm<D, 1>(a, p, s);
  if (passes <= 2) return append_dm<D, 2>(a, p, s);
  if (passes <= 4) return append_dm<D, 4>(a, p, s);
  if (kMax == 8 || passes <= 8) return append_dm<D, (kMax < 8 ? kMax : 8)>(a, p, s);
  return append_dm<D, kMax>(a, p, s);
}

}  // namespace

cudaError_t launch_rope(int D, const bf16* x, int64_t x_stride, int heads, const int* positions,
                        const bf16* gamma, float eps, int rows, bf16* y, int64_t y_stride,
                        const RopeArgs& r, int sm_count, cudaStream_t s) {
  auto* f = D == 64 ? rope_d<64> : D == 128 ? rope_d<128> : rope_d<256>;
  return f(x, x_stride, heads, positions, gamma, eps, rows, y, y_stride, r, sm_count, s);
}

cudaError_t launch_append(int D, const AttnArgs& a, const AppendArgs& p, cudaStream_t s) {
  auto* f = D == 64 ? append_d<64> : D == 128 ? append_d<128> : append_d<256>;
  return f(a, p, s);
}

}  // namespace moe
