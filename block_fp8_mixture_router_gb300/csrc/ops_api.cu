// C ABI of the layer's parts as operators: context, argument checks, launches.
//
// Conventions as in moe_api.cu: unsupported shapes are refused when the context is created,
// sizes are checked against the cap before anything is allocated, and every refusal is a
// status code.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "api_host.h"
#include "ops_internal.cuh"

using namespace moe;

struct moe_ops {
  moe_ops_config cfg;
  int device = 0;
  int sm_count = 0;
  cudaStream_t last_stream = nullptr;
  std::vector<void*> allocs;
  uint8_t* codes = nullptr;   // [max_rows top_k][max_width]: a product's rows
  float* scales = nullptr;    // [max_rows top_k][ceil(max_width / 128)]
  int* hist = nullptr;        // pairs of each expert in each block of the sort
  int* status = nullptr;
};

namespace {

constexpr int kMaxWidth = 65536;
constexpr size_t kMaxTop = kMaxTopK;

bool supported(const moe_ops_config* c) {
  return c->n_experts >= 1 && c->n_experts <= kMaxExperts && c->top_k >= 1 &&
         c->top_k <= (int)kMaxTop && c->max_rows >= 1 && c->max_rows <= 65536 &&
         c->max_width >= 0 && c->max_width <= kMaxWidth && c->max_width % 16 == 0;
}

// Byte sizes of everything a context allocates, in order.
struct Sizes {
  size_t codes, scales, hist, status;
  size_t total() const { return codes + scales + hist + status; }
};

Sizes sizes_of(const moe_ops_config* c) {
  const size_t pairs = (size_t)c->max_rows * c->top_k;
  Sizes s;
  s.codes = up256(std::max<size_t>(pairs * c->max_width, 1));
  s.scales = up256(std::max<size_t>(pairs * groups_of(c->max_width) * 4, 1));
  s.hist = up256((pairs + kSortPairs - 1) / kSortPairs * c->n_experts * 4);
  s.status = 256;
  return s;
}

void release(moe_ops* c) {
  for (void* p : c->allocs) cudaFree(p);
  c->allocs.clear();
}

// Widths of rows: whole 16-byte vectors of bf16; of codes too where they are codes.
bool width_ok(int width, bool codes) {
  return width >= 1 && width <= 2 * kMaxWidth && width % (codes ? 16 : 8) == 0;
}

// Rows to write or read: one of the two forms, well formed.
bool form_ok(const moe_rows* r, int width) {
  if (!r) return false;
  if (r->values) return !r->codes && !r->scales && rows_ok(r->values, r->stride, width);
  return r->codes && r->scales && aligned16(r->codes) &&
         (reinterpret_cast<uintptr_t>(r->scales) & 3) == 0;
}

bool bytes_overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an && bn && x < y + bn && y < x + an;
}

// Whether bf16 rows and rows of either form share a byte.
bool overlaps(const void* v, int64_t stride, int width, int rows, const moe_rows* r, int r_width,
              int r_rows) {
  if (rows < 1 || r_rows < 1) return false;
  const size_t bytes = 2 * ((size_t)(rows - 1) * stride + width);
  if (r->values) {
    // runs of as many rows of the longer array as the shorter one has
    const int run = std::min(rows, r_rows), all = std::max(rows, r_rows);
    for (int i = 0; i < all; i += run) {
      const bf16* a = static_cast<const bf16*>(v) + (rows > r_rows ? (int64_t)i * stride : 0);
      const bf16* b = static_cast<const bf16*>(r->values) +
                      (r_rows > rows ? (int64_t)i * r->stride : 0);
      if (overlap_rows(a, stride, width, b, r->stride, r_width, std::min(run, all - i)))
        return true;
    }
    return false;
  }
  return bytes_overlap(v, bytes, r->codes, (size_t)r_rows * r_width) ||
         bytes_overlap(v, bytes, r->scales, (size_t)r_rows * groups_of(r_width) * 4);
}

RowsOut out_of(const moe_rows* r) {
  return RowsOut{static_cast<bf16*>(r->values), r->stride, r->codes, r->scales};
}

int check_order(const moe_ops* c, const moe_order* o) {
  if (!o || o->tokens < 0) return MOE_ERR_INVALID_ARG;
  if (o->tokens > c->cfg.max_rows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (o->tokens == 0) return MOE_OK;
  return o->starts && o->pair_of_slot && o->slot_of_pair ? MOE_OK : MOE_ERR_INVALID_ARG;
}

OrderArgs order_args(const moe_ops* c, const moe_order* o) {
  return OrderArgs{o->tokens, c->cfg.top_k, c->cfg.n_experts, o->starts, o->pair_of_slot,
                   o->slot_of_pair};
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// y[t] = sum_j w rows: combine, and with w nullptr the gradient of dispatch.
int combine(moe_ops* c, const void* rows, int64_t rows_stride, const moe_order* order,
            const float* w, int width, void* y, int64_t y_stride, void* stream) {
  const int rc = check_order(c, order);
  if (rc != MOE_OK || order->tokens == 0) return rc;
  const int pairs = order->tokens * c->cfg.top_k;
  const moe_rows out = {y, y_stride, nullptr, nullptr};
  if (!width_ok(width, false) || !rows_ok(rows, rows_stride, width) || !form_ok(&out, width) ||
      overlaps(rows, rows_stride, width, pairs, &out, width, order->tokens))
    return MOE_ERR_INVALID_ARG;
  Device guard(c->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  c->last_stream = s;
  return status_of(launch_combine_rows(order_args(c, order), static_cast<const bf16*>(rows),
                                       rows_stride, w, width, static_cast<bf16*>(y), y_stride,
                                       c->status, s));
}

// Boxes of 128 bytes x box_rows rows under the 128-byte swizzle.
bool encode(CUtensorMap* m, const void* p, bool in_bf16, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
  if (!fn) return false;
  const cuuint32_t box[3] = {in_bf16 ? 64u : 128u, (cuuint32_t)box_rows, 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(m, in_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
            const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the kernel for few rows takes a product.  It costs the work of its row tiles (of
// eight rows of a group), each on all of the group's weights, about 3.5 M weights a
// microsecond; the tensor-core kernel's time is that of one tile's blocks, some 3 us and
// 0.0035 for each value of the contraction, as long as it has an SM for every tile.
// Measured, few / tensor-core kernel, in us, bf16 rows:
//   2560 x 2048: 1 row 3.9 / 11.6, 16 6.1 / 12.0, 48 12.4 / 12.1, 96 21 / 11.5
//   512 x 2048: 128 rows 8.0 / 11.8;  4096 x 4096: 8 7.0 / 17.6, 24 17.8 / 18.1, 48 31 / 18.0
//   256 experts of 1024 x 2048, rows of 1, 2, 4 tokens, eight each: 5.9 / 12.0, 9.6 / 12.0,
//   16.8 / 14.1; 64 experts, 4, 16, 32 tokens: 11.2 / 12.7, 26 / 27, 33 / 30.
bool few_rows(int rows, int groups, int inner, int outer) {
  const int64_t tiles = std::max((rows + 7) / 8, std::min(groups, rows));
  return tiles * inner * outer <= 9000000 + (int64_t)12300 * inner;
}

int linear(moe_ops* c, const moe_rows* x, const moe_block_weights* w, const int32_t* starts,
           int rows, void* y, int64_t y_stride, bool trans, void* stream) {
  if (!c || !w || rows < 0) return MOE_ERR_INVALID_ARG;
  if (w->groups < 1 || w->out < 1 || w->in < 1) return MOE_ERR_INVALID_ARG;
  if (w->groups > kMaxExperts || w->out > kMaxWidth || w->in > kMaxWidth || w->out % 16 ||
      w->in % 16 || rows > c->cfg.max_rows * c->cfg.top_k)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  const int inner = trans ? w->out : w->in, outer = trans ? w->in : w->out;
  if (x && x->values && inner > c->cfg.max_width) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!w->codes || !w->scales || !aligned16(w->codes) || (!starts && w->groups != 1) ||
      !form_ok(x, inner) || !rows_ok(y, y_stride, outer) ||
      overlaps(y, y_stride, outer, rows, x, inner, rows))
    return MOE_ERR_INVALID_ARG;
  Device guard(c->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  c->last_stream = s;
  LinArgs a = {};
  const uint8_t* codes = x->values ? c->codes : x->codes;
  a.sx = x->values ? c->scales : x->scales;
  a.sw = w->scales;
  a.starts = starts;
  a.groups = w->groups;
  a.rows = rows;
  a.inner = inner;
  a.outer = outer;
  a.y = static_cast<bf16*>(y);
  a.y_stride = y_stride;
  a.status = c->status;
  if (!trans && few_rows(rows, w->groups, inner, outer))
    return status_of(launch_linear_rows(a, static_cast<const bf16*>(x->values), x->stride,
                                        x->codes, w->codes, s));
  // (x as one group, so that one form of copy takes rows and weights)
  const cuuint64_t dx[3] = {(cuuint64_t)inner, (cuuint64_t)rows, 1};
  const cuuint64_t sx[2] = {(cuuint64_t)inner, (cuuint64_t)inner * rows};
  const cuuint64_t dw[3] = {(cuuint64_t)w->in, (cuuint64_t)w->out, (cuuint64_t)w->groups};
  const cuuint64_t sw[2] = {(cuuint64_t)w->in, (cuuint64_t)w->in * w->out};
  const cuuint64_t dy[2] = {(cuuint64_t)outer, (cuuint64_t)rows};
  const cuuint64_t sy[1] = {(cuuint64_t)(rows > 1 ? y_stride : outer) * 2};
  if (!encode(&a.x, codes, false, 3, dx, sx, 128) ||
      !encode(&a.xs, codes, false, 3, dx, sx, 32) ||
      !encode(&a.w, w->codes, false, 3, dw, sw, 128) ||
      !encode(&a.out, y, true, 2, dy, sy, 32))
    return MOE_ERR_CUDA;
  if (x->values &&
      launch_quant_rows(static_cast<const bf16*>(x->values), x->stride, rows, inner, c->codes,
                        c->scales, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  return status_of(launch_linear(a, trans, c->sm_count, x->values != nullptr, s));
}

}  // namespace

extern "C" {

int moe_ops_required_bytes(const moe_ops_config* cfg, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_INVALID_ARG;
  if (!supported(cfg)) return MOE_ERR_UNSUPPORTED_SHAPE;
  *bytes = sizes_of(cfg).total();
  return MOE_OK;
}

int moe_ops_create(const moe_ops_config* cfg, int device, moe_ops** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || device < 0) return MOE_ERR_INVALID_ARG;
  if (!supported(cfg)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const Sizes z = sizes_of(cfg);
  if (cfg->workspace_cap_bytes && z.total() > cfg->workspace_cap_bytes)
    return MOE_ERR_ALLOC_LIMIT;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device >= ndev) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  Device guard(device);
  if (!guard.ok) return MOE_ERR_CUDA;
  moe_ops* c = new (std::nothrow) moe_ops();
  if (!c) return MOE_ERR_CUDA;
  c->cfg = *cfg;
  c->device = device;
  bool ok = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, device) ==
            cudaSuccess;
  const size_t bytes[4] = {z.codes, z.scales, z.hist, z.status};
  void* p[4] = {};
  try {
    c->allocs.reserve(4);
    for (int i = 0; i < 4 && ok; ++i) {
      ok = cudaMalloc(&p[i], bytes[i]) == cudaSuccess;
      if (ok) c->allocs.push_back(p[i]);
    }
  } catch (const std::bad_alloc&) {
    ok = false;
  }
  if (ok) {
    c->codes = static_cast<uint8_t*>(p[0]);
    c->scales = static_cast<float*>(p[1]);
    c->hist = static_cast<int*>(p[2]);
    c->status = static_cast<int*>(p[3]);
    ok = cudaMemset(p[3], 0, z.status) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess &&
         setup_linear() == cudaSuccess;
  }
  if (!ok) {
    cudaGetLastError();
    release(c);
    delete c;
    return MOE_ERR_CUDA;
  }
  *out = c;
  return MOE_OK;
}

void moe_ops_destroy(moe_ops* ctx) {
  if (!ctx) return;
  Device guard(ctx->device);
  release(ctx);
  delete ctx;
}

int moe_ops_last_device_status(moe_ops* ctx) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  int v = 0;
  if (cudaStreamSynchronize(ctx->last_stream) != cudaSuccess ||
      cudaMemcpy(&v, ctx->status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess ||
      (v && cudaMemset(ctx->status, 0, sizeof(v)) != cudaSuccess)) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  if (v & kOpsBadBase) return MOE_ERR_CUDA;
  if (v & kOpsTimeout) return MOE_ERR_DEVICE_TIMEOUT;
  return v & kOpsBadOrder ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int moe_dispatch(moe_ops* ctx, const int32_t* idx, const void* x, int64_t x_stride, int width,
                 const moe_order* order, const moe_rows* rows, void* stream) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int rc = check_order(ctx, order);
  if (rc != MOE_OK || order->tokens == 0) return rc;
  if (!idx) return MOE_ERR_INVALID_ARG;
  RowsOut out = {};
  if (x) {
    if (!form_ok(rows, width) || !width_ok(width, rows->codes != nullptr) ||
        !rows_ok(x, x_stride, width) ||
        overlaps(x, x_stride, width, order->tokens, rows, width,
                 order->tokens * ctx->cfg.top_k))
      return MOE_ERR_INVALID_ARG;
    out = out_of(rows);
  }
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  return status_of(launch_dispatch(order_args(ctx, order), idx, static_cast<const bf16*>(x),
                                   x_stride, width, out, ctx->hist, ctx->sm_count, s));
}

int moe_dispatch_grad(moe_ops* ctx, const void* drows, int64_t drows_stride,
                      const moe_order* order, int width, void* dx, int64_t dx_stride,
                      void* stream) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  return combine(ctx, drows, drows_stride, order, nullptr, width, dx, dx_stride, stream);
}

int moe_combine(moe_ops* ctx, const void* rows, int64_t rows_stride, const moe_order* order,
                const float* weights, int width, void* y, int64_t y_stride, void* stream) {
  if (!ctx || (!weights && order && order->tokens > 0)) return MOE_ERR_INVALID_ARG;
  return combine(ctx, rows, rows_stride, order, weights, width, y, y_stride, stream);
}

int moe_combine_grad(moe_ops* ctx, const void* dy, int64_t dy_stride, const void* rows,
                     int64_t rows_stride, const moe_order* order, const float* weights, int width,
                     const moe_rows* drows, float* dweights, void* stream) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int rc = check_order(ctx, order);
  if (rc != MOE_OK || order->tokens == 0) return rc;
  const int pairs = order->tokens * ctx->cfg.top_k;
  if (!weights || !dweights || !form_ok(drows, width) ||
      !width_ok(width, drows->codes != nullptr) || !rows_ok(dy, dy_stride, width) ||
      !rows_ok(rows, rows_stride, width) ||
      overlaps(dy, dy_stride, width, order->tokens, drows, width, pairs) ||
      overlaps(rows, rows_stride, width, pairs, drows, width, pairs) ||
      bytes_overlap(weights, (size_t)pairs * 4, dweights, (size_t)pairs * 4))
    return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  return status_of(launch_combine_grad(
      order_args(ctx, order), static_cast<const bf16*>(dy), dy_stride,
      static_cast<const bf16*>(rows), rows_stride, weights, width, out_of(drows), dweights,
      ctx->status, s));
}

int moe_linear(moe_ops* ctx, const moe_rows* x, const moe_block_weights* w, const int32_t* starts,
               int rows, void* y, int64_t y_stride, void* stream) {
  return linear(ctx, x, w, starts, rows, y, y_stride, false, stream);
}

int moe_linear_grad(moe_ops* ctx, const moe_rows* dy, const moe_block_weights* w,
                    const int32_t* starts, int rows, void* dx, int64_t dx_stride, void* stream) {
  return linear(ctx, dy, w, starts, rows, dx, dx_stride, true, stream);
}

int moe_swiglu(moe_ops* ctx, const void* gate_up, int64_t gate_up_stride, int rows, int width,
               const moe_rows* h, void* stream) {
  if (!ctx || rows < 0) return MOE_ERR_INVALID_ARG;
  if (rows > ctx->cfg.max_rows * ctx->cfg.top_k) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!form_ok(h, width) || !width_ok(width, h->codes != nullptr) || width > kMaxWidth ||
      !rows_ok(gate_up, gate_up_stride, 2 * (int64_t)width) ||
      overlaps(gate_up, gate_up_stride, 2 * width, rows, h, width, rows))
    return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  return status_of(launch_swiglu(static_cast<const bf16*>(gate_up), gate_up_stride, rows, width,
                                 out_of(h), s));
}

int moe_swiglu_grad(moe_ops* ctx, const void* dh, int64_t dh_stride, const void* gate_up,
                    int64_t gate_up_stride, int rows, int width, const moe_rows* dgate_up,
                    void* stream) {
  if (!ctx || rows < 0) return MOE_ERR_INVALID_ARG;
  if (rows > ctx->cfg.max_rows * ctx->cfg.top_k) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  // (2 width is a multiple of 16, as codes want it, where width is one of 8)
  if (width < 1 || width > kMaxWidth || !form_ok(dgate_up, 2 * width) ||
      !width_ok(width, false) || !rows_ok(dh, dh_stride, width) ||
      !rows_ok(gate_up, gate_up_stride, 2 * (int64_t)width) ||
      overlaps(gate_up, gate_up_stride, 2 * width, rows, dgate_up, 2 * width, rows) ||
      overlaps(dh, dh_stride, width, rows, dgate_up, 2 * width, rows))
    return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  return status_of(launch_swiglu_grad(static_cast<const bf16*>(dh), dh_stride,
                                      static_cast<const bf16*>(gate_up), gate_up_stride, rows,
                                      width, out_of(dgate_up), s));
}

}  // extern "C"
