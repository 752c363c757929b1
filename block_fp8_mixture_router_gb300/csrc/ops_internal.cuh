// Declarations shared by the kernels of the layer's parts (dispatch, combine, linear,
// swiglu) and their host code.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// Device status word bits.
constexpr int kOpsTimeout = 1;
constexpr int kOpsBadOrder = 2;
constexpr int kOpsBadBase = 4;  // shared memory that does not begin where the tiles need it

// Rows a kernel writes: bf16, or e4m3 codes with a scale for each 128 values.
struct RowsOut {
  bf16* v;            // nullptr: codes
  int64_t stride;     // of v, in values
  uint8_t* codes;     // [rows][width]
  float* scales;      // [rows][ceil(width / 128)]
};

inline __host__ __device__ int groups_of(int width) { return (width + kGroup - 1) / kGroup; }

// ---- dispatch and combine (k_dispatch.cu) -------------------------------------
struct OrderArgs {
  int T, k, E;
  int* starts;         // [E + 1]
  int* pair_of_slot;   // [T k]
  int* slot_of_pair;   // [T k]
};
constexpr int kSortPairs = 2048;  // pairs of a block of the sort's kernels

// idx [T][k] -> the order; x (unless nullptr) to its slots.  hist: kSortPairs-blocks x E ints.
cudaError_t launch_dispatch(const OrderArgs& o, const int* idx, const bf16* x, int64_t x_stride,
                            int width, const RowsOut& out, int* hist, int sm_count,
                            cudaStream_t s);
// y[t] = sum_j w[t][j] rows[slot(t, j)]; w nullptr: all ones.
cudaError_t launch_combine_rows(const OrderArgs& o, const bf16* rows, int64_t rows_stride,
                                const float* w, int width, bf16* y, int64_t y_stride, int* status,
                                cudaStream_t s);
cudaError_t launch_combine_grad(const OrderArgs& o, const bf16* dy, int64_t dy_stride,
                                const bf16* rows, int64_t rows_stride, const float* w, int width,
                                const RowsOut& out, float* dw, int* status, cudaStream_t s);

// ---- element-wise rows (k_swiglu.cu) -------------------------------------------
cudaError_t launch_swiglu(const bf16* gu, int64_t gu_stride, int rows, int width,
                          const RowsOut& out, cudaStream_t s);
cudaError_t launch_swiglu_grad(const bf16* dh, int64_t dh_stride, const bf16* gu,
                               int64_t gu_stride, int rows, int width, const RowsOut& out,
                               cudaStream_t s);
cudaError_t launch_quant_rows(const bf16* x, int64_t x_stride, int rows, int width,
                              uint8_t* codes, float* scales, cudaStream_t s);

// ---- the product (k_linear.cu) ---------------------------------------------------
struct LinArgs {
  CUtensorMap x;       // codes [rows][inner], boxes of 128 rows x 128 bytes
  CUtensorMap xs;      // the same in boxes of 32 rows
  CUtensorMap w;       // codes [groups][out][in], boxes of 128 x 128
  CUtensorMap out;     // y, boxes of 32 rows x 64 values
  const float* sx;     // [rows][ceil(inner / 128)]
  const float* sw;     // [groups][ceil(out / 128)][ceil(in / 128)]
  const int* starts;   // [groups + 1] on the device, or nullptr: one group of all rows
  int groups, rows;
  int inner, outer;    // contraction and output width
  bf16* y;
  int64_t y_stride;
  int* status;
};
// Few rows (k_linear_rows.cu): x bf16, or codes; the weights' codes.
cudaError_t launch_linear_rows(const LinArgs& a, const bf16* x, int64_t x_stride,
                               const uint8_t* codes, const uint8_t* w, cudaStream_t s);
cudaError_t setup_linear();
// trans: y = x W instead of x W^T.
cudaError_t launch_linear(const LinArgs& a, bool trans, int sm_count, bool pdl, cudaStream_t s);

}  // namespace moe
