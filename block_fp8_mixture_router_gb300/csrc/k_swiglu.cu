// Element-wise kernels on rows: the gated activation and its gradient, and the rows'
// quantisation in front of a product.
//
//   h = silu(g) u,  dg = dh u s (1 + g (1 - s)),  du = dh silu(g),  s = 1 / (1 + e^-g)
//
// Every value is read and written once, so HBM bounds them, and the quotients behind codes
// nearly do: 131072 rows of 512 to codes 58 us (87 % of the copy's rate; the schedulers issue
// in 75 % of cycles), the gradient of 10493 rows of 1408 in bf16 23 us (96 %), of 131072 rows
// of 512 to codes 98 us (83 %; of 528, where groups straddle gates and ups and every operand
// is read twice, 158: 53 %), 131072 rows of 1024 quantised 68 us (88 %).  Eight lanes take a group of 128 columns, 16 values each: the
// group's largest is then three shuffles away and a lane's loads and stores are 16-byte
// vectors.  Blocks to an SM as measured: six for what has few values in flight (62 us with
// four for the first), four for the gradient (27 us with six).
#include "rows_device.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// Unit u = (row, group of 128 columns) of the eight lanes that a thread belongs to.
struct Unit {
  int row, c;
  bool on;
};

__device__ __forceinline__ Unit unit_of(unsigned u, int rows, int groups) {
  Unit r;
  r.row = (int)(u / (unsigned)groups);
  r.c = (int)(u - (unsigned)r.row * groups) * kGroup + 16 * (int)(threadIdx.x & 7);
  r.on = r.row < rows;
  return r;
}

// The sigmoid of z and that of -z, in fp32 at any z: 1 / (1 + e) with e = e^-|z|, which does
// not overflow, and e times it, which follows e^-|z| down to fp32's last subnormal and is 0
// behind it.  (An exponent held back instead leaves z s growing with z at far negative z, and
// 1 - s, times a far positive z, wants a quotient that is 1 to the last bit.)  e is the square
// of e^(-|z| / 2), a normal number for all z that matter: neither approximation meets a
// subnormal, and takes no steps for one.
struct Sigmoid {
  float s, other;
};

__device__ __forceinline__ Sigmoid sigmoid_any(float z) {
  float root, big;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(root) : "f"(fabsf(z) * -0.721347520444f));
  const float e = root * root;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(big) : "f"(1.0f + e));
  const float small = e * big;
  return z >= 0.0f ? Sigmoid{big, small} : Sigmoid{small, big};
}

template <bool kCodes>
__global__ void __launch_bounds__(kThreads, 6) k_swiglu(const bf16* gu, int64_t gu_stride, int rows,
                                                     int width, RowsOut out) {
  const Unit u = unit_of(blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3), rows, groups_of(width));
  const bf16* row = gu + (int64_t)u.row * gu_stride;
  const Vec16 rg = load16(row, u.c, width, u.on), ru = load16(row + width, u.c, width, u.on);
  float g[16], v[16];
  unpack16(rg, g);
  unpack16(ru, v);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= g[i] * sigmoid_any(g[i]).s;
  put16<kCodes, false>(out, u.row, u.c, width, u.on, v);
}

// Gradients of 16 gates and of 16 ups.
__device__ __forceinline__ void swiglu_back(const Vec16& rd, const Vec16& rg, const Vec16& ru,
                                            float (&dg)[16], float (&du)[16]) {
  float d[16], g[16], u[16];
  unpack16(rd, d);
  unpack16(rg, g);
  unpack16(ru, u);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const Sigmoid p = sigmoid_any(g[i]);
    const float z = g[i] * p.s;
    dg[i] = d[i] * u[i] * (p.s + z * p.other);
    du[i] = d[i] * z;
  }
}

// One group of the width at a time, both halves of the output.  In codes the width is a
// multiple of 128, so that groups of the output lie in one half.
template <bool kCodes>
__global__ void __launch_bounds__(kThreads, 4) k_swiglu_grad(const bf16* dh, int64_t dh_stride,
                                                          const bf16* gu, int64_t gu_stride,
                                                          int rows, int width, RowsOut out) {
  const Unit u = unit_of(blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3), rows, groups_of(width));
  const bf16* row = gu + (int64_t)u.row * gu_stride;
  const Vec16 rd = load16(dh + (int64_t)u.row * dh_stride, u.c, width, u.on);
  const Vec16 rg = load16(row, u.c, width, u.on), ru = load16(row + width, u.c, width, u.on);
  float dg[16], du[16];
  swiglu_back(rd, rg, ru, dg, du);
  if constexpr (kCodes) {
    put16<true, false>(out, u.row, u.c, 2 * width, u.on, dg);
    put16<true, false>(out, u.row, width + u.c, 2 * width, u.on, du);
  } else {
    RowsOut half = out;
    put16<false, false>(half, u.row, u.c, width, u.on, dg);
    half.v += width;
    put16<false, false>(half, u.row, u.c, width, u.on, du);
  }
}

// Columns a .. a + 7 and b .. b + 7 of a row.
__device__ __forceinline__ Vec16 load8_8(const bf16* row, int a, int b, bool on) {
  Vec16 v = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (on) {
    v.a = *reinterpret_cast<const uint4*>(row + a);
    v.b = *reinterpret_cast<const uint4*>(row + b);
  }
  return v;
}

// Codes at other widths (multiples of 8): one group of the output's 2 x width columns at a
// time; the group on the border holds gradients of gates and of ups, and so may a lane's two
// vectors of 8.
__global__ void __launch_bounds__(kThreads, 4) k_swiglu_grad_mixed(const bf16* dh, int64_t dh_stride,
                                                                const bf16* gu, int64_t gu_stride,
                                                                int rows, int width, RowsOut out) {
  const Unit u = unit_of(blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3), rows, groups_of(2 * width));
  const bool on = u.on && u.c < 2 * width, up0 = u.c >= width, up1 = u.c + 8 >= width;
  const int a = up0 ? u.c - width : u.c, b = up1 ? u.c + 8 - width : u.c + 8;
  const bf16* row = gu + (int64_t)u.row * gu_stride;
  const Vec16 rd = load8_8(dh + (int64_t)u.row * dh_stride, a, b, on);
  const Vec16 rg = load8_8(row, a, b, on), ru = load8_8(row + width, a, b, on);
  float dg[16], du[16];
  swiglu_back(rd, rg, ru, dg, du);
#pragma unroll
  for (int i = 0; i < 16; ++i) dg[i] = (i < 8 ? up0 : up1) ? du[i] : dg[i];
  put16<true, false>(out, u.row, u.c, 2 * width, u.on, dg);
}

__global__ void __launch_bounds__(kThreads, 6) k_quant_rows(const bf16* x, int64_t x_stride, int rows,
                                                         int width, RowsOut out) {
  const Unit u = unit_of(blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3), rows, groups_of(width));
  float v[16];
  unpack16(load16(x + (int64_t)u.row * x_stride, u.c, width, u.on), v);
  put16<true, true>(out, u.row, u.c, width, u.on, v);
  pdl_trigger();
}

unsigned grid_of(int rows, int width) {
  constexpr size_t per = kThreads / 8;
  return (unsigned)(((size_t)rows * groups_of(width) + per - 1) / per);
}

}  // namespace

cudaError_t launch_swiglu(const bf16* gu, int64_t gu_stride, int rows, int width,
                          const RowsOut& out, cudaStream_t s) {
  const unsigned grid = grid_of(rows, width);
  if (out.v)
    k_swiglu<false><<<grid, kThreads, 0, s>>>(gu, gu_stride, rows, width, out);
  else
    k_swiglu<true><<<grid, kThreads, 0, s>>>(gu, gu_stride, rows, width, out);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_grad(const bf16* dh, int64_t dh_stride, const bf16* gu,
                               int64_t gu_stride, int rows, int width, const RowsOut& out,
                               cudaStream_t s) {
  const unsigned grid = grid_of(rows, width);
  if (out.v)
    k_swiglu_grad<false><<<grid, kThreads, 0, s>>>(dh, dh_stride, gu, gu_stride, rows, width, out);
  else if (width % kGroup == 0)
    k_swiglu_grad<true><<<grid, kThreads, 0, s>>>(dh, dh_stride, gu, gu_stride, rows, width, out);
  else
    k_swiglu_grad_mixed<<<grid_of(rows, 2 * width), kThreads, 0, s>>>(dh, dh_stride, gu, gu_stride,
                                                                      rows, width, out);
  return cudaGetLastError();
}

cudaError_t launch_quant_rows(const bf16* x, int64_t x_stride, int rows, int width,
                              uint8_t* codes, float* scales, cudaStream_t s) {
  k_quant_rows<<<grid_of(rows, width), kThreads, 0, s>>>(x, x_stride, rows, width,
                                                         RowsOut{nullptr, 0, codes, scales});
  return cudaGetLastError();
}

}  // namespace moe
