// C ABI of the attention operators: context, argument checks, launches.
//
// Conventions as in moe_api.cu: unsupported shapes are refused when the context
// is created, sizes are checked against the cap before anything is allocated,
// and every refusal is a status code.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "api_host.h"
#include "attn_internal.cuh"
#include "rope_turns.h"

using namespace moe;

static_assert(MOE_ROPE_PLAIN == 0 && MOE_ROPE_LINEAR == 1 && MOE_ROPE_BY_PARTS == 2,
              "RopeSpec's scalings");

struct moe_attn {
  moe_attn_config cfg;
  int device = 0;
  int sm_count = 0;
  int page_shift = 0;
  int dec_slots = 0;       // CTAs of a full decode grid
  cudaStream_t last_stream = nullptr;
  std::vector<void*> allocs;
  unsigned long long* turns = nullptr;  // [rotary_dim / 2]
  bf16* q = nullptr;                    // [max_rows][q_heads][head_dim]: a step's queries
  AttnSplit split{};
  int* status = nullptr;
};

namespace {

constexpr int kDecTileRows = kAttnSlotRows;

// The decode kernel takes a sequence whose rows (tokens x query heads of a key head) fit
// one of its tiles, or few tiles in all: it reads the keys once for every tile.  The
// prompt kernel takes the others, with 128 rows to a tile.  Tiles = sequences x key heads
// x tiles of a sequence; measured over 300 to 200000 keys, 1 to 8 query heads to a key
// head, prompt kernel's time over decode kernel's, geometric means:
//   head_dim   2 tiles     3      4      6      8     12     16     24     32
//         64      1.01   0.92   0.89   0.80   0.80   0.70   0.69   0.57   0.55
//        128      1.08   1.00   0.94   0.87   0.86   0.75   0.72   0.62   0.60
//        256      1.13   1.07   1.01   0.90   0.91   0.75   0.76   0.66   0.63
// hence from 3, 4 and 6 tiles on.
constexpr bool prompt_tiles(int head_dim, long long tiles) { return tiles > 1 + head_dim / 64; }

bool supported(const moe_attn_config* c) {
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->kv_heads < 1 || c->kv_heads > 64) return false;
  if (c->q_heads < c->kv_heads || c->q_heads % c->kv_heads) return false;
  if (c->q_heads / c->kv_heads > kAttnMaxGroup) return false;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 &&
      c->page_tokens != 128)
    return false;
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 2) return false;
  if (c->rope_layout != MOE_ROPE_HALF && c->rope_layout != MOE_ROPE_INTERLEAVED) return false;
  if (c->rope_scaling < MOE_ROPE_PLAIN || c->rope_scaling > MOE_ROPE_BY_PARTS) return false;
  if (!isfinite(c->softmax_scale) || c->softmax_scale < 0) return false;
  if (c->rotary_dim > 0) {
    if (!isfinite(c->rope_base) || c->rope_base <= 1) return false;
    if (!isfinite(c->rope_amplitude) || c->rope_amplitude <= 0) return false;
    if (c->rope_scaling != MOE_ROPE_PLAIN && (!isfinite(c->rope_factor) || c->rope_factor <= 0))
      return false;
    if (c->rope_scaling == MOE_ROPE_BY_PARTS &&
        (c->rope_trained_positions < 1 || !isfinite(c->rope_turns_low) ||
         !isfinite(c->rope_turns_high) || c->rope_turns_low < 0 ||
         c->rope_turns_high <= c->rope_turns_low))
      return false;
  }
  if (c->window < 0) return false;
  if (c->max_rows < 1 || c->max_rows > 65536) return false;
  if (c->max_seqs < 1 || c->max_seqs > kAttnMaxSeqs) return false;
  return true;
}

// Byte sizes of everything a context allocates, in order.
struct Sizes {
  size_t turns, q, part_o, part_sums, shared, status;
  size_t total() const { return turns + q + part_o + part_sums + shared + status; }
};

Sizes sizes_of(const moe_attn_config* c) {
  Sizes s;
  const size_t slots = 2 * (size_t)kAttnMaxCtas;
  s.turns = up256((size_t)std::max(c->rotary_dim / 2, 1) * 8);
  s.q = up256((size_t)c->max_rows * c->q_heads * c->head_dim * 2);
  // the larger of the decode kernel's and the prompt kernel's partial results
  const size_t rows =
      std::max(slots * kAttnSlotRows, (size_t)kAttnPromptCtas * kAttnPromptRows);
  s.part_o = up256(rows * c->head_dim * 4);
  s.part_sums = up256(rows * 16);
  s.shared = up256((size_t)kAttnMaxCtas * 16);
  s.status = 256;
  return s;
}

void release(moe_attn* c) {
  for (void* p : c->allocs) cudaFree(p);
  c->allocs.clear();
}

// Turns per position of every pair as 64-bit fractions of a turn.
std::vector<unsigned long long> turn_table(const moe_attn_config& c) {
  const RopeSpec spec{c.rotary_dim, c.rope_scaling, c.rope_base, c.rope_factor,
                      c.rope_trained_positions, c.rope_turns_low, c.rope_turns_high};
  std::vector<unsigned long long> t(std::max(c.rotary_dim / 2, 1), 0);
  for (int i = 0; i < c.rotary_dim / 2; ++i) t[i] = rope_turns(spec, i);
  return t;
}

RopeArgs rope_args(const moe_attn* c) {
  return RopeArgs{c->turns, c->cfg.rotary_dim, c->cfg.rope_layout == MOE_ROPE_INTERLEAVED,
                  (float)c->cfg.rope_amplitude};
}

int check_batch(const moe_attn* c, const moe_kv_cache* k, const moe_attn_batch* b) {
  if (!k || !b) return MOE_ERR_INVALID_ARG;
  if (b->rows < 0 || b->n_seqs < 0 || b->max_seq_rows < 0 || b->max_kv_len < 0)
    return MOE_ERR_INVALID_ARG;
  if (b->rows > c->cfg.max_rows || b->n_seqs > c->cfg.max_seqs) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (b->rows == 0) return MOE_OK;
  if (b->n_seqs < 1 || b->pages_stride < 1 || !b->row_start || !b->kv_len || !b->pages)
    return MOE_ERR_INVALID_ARG;
  if (k->n_pages < 1 || !k->k_codes || !k->v_codes || !k->k_scales || !k->v_scales ||
      !aligned16(k->k_codes) || !aligned16(k->v_codes))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

AttnArgs attn_args(const moe_attn* c, const moe_kv_cache* k, const moe_attn_batch* b) {
  AttnArgs a = {};
  a.Hq = c->cfg.q_heads;
  a.Hkv = c->cfg.kv_heads;
  a.g = a.Hq / a.Hkv;
  a.page_shift = c->page_shift;
  a.window = std::min(c->cfg.window, kAttnMaxTokens);
  const double scale =
      c->cfg.softmax_scale > 0 ? c->cfg.softmax_scale : 1.0 / sqrt((double)c->cfg.head_dim);
  a.scale = (float)(scale * 1.4426950408889634);  // the softmax runs in powers of two
  a.kc = k->k_codes;
  a.vc = k->v_codes;
  a.ks = k->k_scales;
  a.vs = k->v_scales;
  a.n_pages = k->n_pages;
  a.row_start = b->row_start;
  a.kv_len = b->kv_len;
  a.pages = b->pages;
  a.n_seqs = b->n_seqs;
  a.pages_stride = b->pages_stride;
  a.rows = b->rows;
  a.status = c->status;
  return a;
}

bool encode_pool(CUtensorMap* m, const void* pool, const AttnArgs& a, int D, int most) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (!encode) return false;
  const cuuint64_t tokens = (cuuint64_t)a.Hkv << a.page_shift;
  const cuuint64_t dims[3] = {(cuuint64_t)D, tokens, (cuuint64_t)a.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)D, tokens * D};
  const cuuint32_t box[3] = {(cuuint32_t)std::min(D, 128),
                             (cuuint32_t)std::min(1 << a.page_shift, most), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box,
                unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int run_attention(moe_attn* c, const AttnArgs& a, const moe_attn_batch* b, const bf16* q,
                  int64_t q_stride, bf16* out, int64_t out_stride, bool pdl, cudaStream_t s) {
  const int D = c->cfg.head_dim;
  const long long cap = (long long)b->pages_stride << c->page_shift;
  const long long keys = b->max_kv_len > 0 ? std::min<long long>(b->max_kv_len, cap) : cap;
  const int seq_rows = b->max_seq_rows > 0 ? std::min(b->max_seq_rows, b->rows) : b->rows;
  // Rows of a tile of the decode kernel: one row over 262143 keys with four query heads
  // to a key head takes 50 us with eight rows to a tile and 72 with 16.
  const int tile_rows = (long long)seq_rows * a.g <= 8 ? 8 : kDecTileRows;
  const int tq = tile_rows / a.g;
  const long long seq_tiles = (seq_rows + tq - 1) / tq;
  const long long units = (long long)b->rows / tq + b->n_seqs;  // per key head, at most
  const long long row_tiles = std::min(units, seq_tiles * b->n_seqs) * a.Hkv;
  const bool prompt =
      (long long)seq_rows * a.g > kDecTileRows && prompt_tiles(D, row_tiles);
  AttnMaps maps;
  if (!make_attn_maps(&maps, a, D, prompt)) return MOE_ERR_CUDA;
  if (prompt) {
    // Row blocks fewer than the SMs share their keys out, at least two tiles to a CTA.  How
    // many there are follows from the most rows of a sequence; the grid has room for more.
    // (Three sequences of 64 rows over 20000 keys, 16 heads of 128 to 4: 67 us with shares
    // after the grid's count, 47 after this one.)
    const int per = attn_prompt_tokens(D, a.g);
    const long long units = b->rows / per + (long long)b->n_seqs;
    const long long heads = std::min(units, ((long long)seq_rows + per - 1) / per * b->n_seqs) *
                            a.Hkv;
    const long long splits = std::max<long long>(
        1, std::min({std::min(c->sm_count, kAttnPromptParts) / heads,
                     kAttnPromptCtas / (units * a.Hkv), (keys + 127) / 128 / 2}));
    return launch_attn_prompt(D, a, maps, q, q_stride, out, out_stride, c->split, (int)units,
                              (int)splits, pdl, s) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  // The key tiles of all row tiles in equal runs, at least two (256 keys) to a CTA (one row
  // over 4096 keys: 9.0 us, with one tile to a CTA 9.5): balanced whatever the lengths, but
  // the CTAs find their runs and parts are joined.  So a CTA to a row tile where that fills
  // the GPU about as well: short sequences, and no more than two for each place.
  // Measured, sequences of one row x key heads of 128, in us, runs / a CTA each:
  //   32 x 1 over 100 keys 8.9 / 7.4, 1000 keys 12.1 / 13.4;
  //   32 x 4 over 100 12.8 / 7.9, 1000 15.7 / 15.7, ragged 14.9 / 13.4;
  //   128 x 4 over 100 14.8 / 15.7, 1000 37.6 / 34.6, ragged 38.0 / 29.4;
  //   1024 x 1 over 100 31 / 44, 1000 69 / 74; 4000 x 4 over 1000 678 / 1256.
  // Over some 150 such sizes each (1 to 4000 sequences, 100 to 1000 keys, equal and ragged) the
  // rule's choice takes 1.0 % longer than the better one at head_dim 64, 1.2 % at 128 and
  // 3.0 % at 256 (geometric means); the worst are ragged batches of 128 to 256 sequences.
  long long span = keys;
  if (a.window) span = std::min<long long>(span, (long long)a.window + tq + kAttnKeys);
  const long long unit_tiles = (span + kAttnKeys - 1) / kAttnKeys, places = c->dec_slots;
  const bool each = unit_tiles <= 8 && (row_tiles <= places
                                            ? unit_tiles * (places - row_tiles) <= 5 * places
                                            : unit_tiles > 1 && row_tiles <= 2 * places);
  long long grid = units * a.Hkv;
  if (!each) grid = std::max<long long>(1, std::min((grid * unit_tiles + 1) / 2, places));
  return launch_attn_decode(D, tile_rows, a, maps, q, q_stride, out, out_stride, c->split,
                            (int)grid, !each, pdl, s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

namespace moe {
bool make_attn_maps(AttnMaps* m, const AttnArgs& a, int D, bool prompt) {
  return encode_pool(&m->k, a.kc, a, D, 128) &&
         (prompt ? encode_pool(&m->v64, a.vc, a, D, 64) : encode_pool(&m->v, a.vc, a, D, 128));
}
}  // namespace moe

extern "C" {

int moe_attn_required_bytes(const moe_attn_config* cfg, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_INVALID_ARG;
  if (!supported(cfg)) return MOE_ERR_UNSUPPORTED_SHAPE;
  *bytes = sizes_of(cfg).total();
  return MOE_OK;
}

int moe_attn_create(const moe_attn_config* cfg, int device, moe_attn** out) {
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
  moe_attn* c = new (std::nothrow) moe_attn();
  if (!c) return MOE_ERR_CUDA;
  c->cfg = *cfg;
  c->device = device;
  while ((1 << c->page_shift) < cfg->page_tokens) ++c->page_shift;
  bool ok = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, device) ==
            cudaSuccess;
  const size_t bytes[6] = {z.turns, z.q, z.part_o, z.part_sums, z.shared, z.status};
  void* p[6] = {};
  try {
    c->allocs.reserve(6);
    for (int i = 0; i < 6 && ok; ++i) {
      ok = cudaMalloc(&p[i], bytes[i]) == cudaSuccess;
      if (ok) c->allocs.push_back(p[i]);
    }
    if (ok) {
      c->turns = static_cast<unsigned long long*>(p[0]);
      c->q = static_cast<bf16*>(p[1]);
      c->split.o = static_cast<float*>(p[2]);
      c->split.sums = static_cast<float4*>(p[3]);
      c->split.shared = static_cast<int4*>(p[4]);
      c->status = static_cast<int*>(p[5]);
      const std::vector<unsigned long long> t = turn_table(*cfg);
      ok = cudaMemcpy(p[0], t.data(), t.size() * 8, cudaMemcpyHostToDevice) == cudaSuccess &&
           cudaMemset(p[5], 0, z.status) == cudaSuccess &&
           cudaDeviceSynchronize() == cudaSuccess &&
           setup_attn_decode(cfg->head_dim) == cudaSuccess &&
           setup_attn_prompt(cfg->head_dim) == cudaSuccess;
    }
    if (ok) c->dec_slots = std::min(attn_decode_slots(cfg->head_dim, c->sm_count), kAttnMaxCtas);
  } catch (const std::bad_alloc&) {
    ok = false;
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

void moe_attn_destroy(moe_attn* ctx) {
  if (!ctx) return;
  Device guard(ctx->device);
  release(ctx);
  delete ctx;
}

int moe_attn_last_device_status(moe_attn* ctx) {
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
  if (v & kAttnTimeout) return MOE_ERR_DEVICE_TIMEOUT;
  return v & kAttnBadBatch ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int moe_rope(moe_attn* ctx, const void* x, int64_t x_stride, int heads, const int32_t* positions,
             const void* gamma, float eps, int rows, void* y, int64_t y_stride, void* stream) {
  if (!ctx || rows < 0 || heads < 1 || !isfinite(eps) || eps < 0) return MOE_ERR_INVALID_ARG;
  if (heads > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  const int64_t width = (int64_t)heads * ctx->cfg.head_dim;
  if (!rows_ok(x, x_stride, width) || !rows_ok(y, y_stride, width) || !positions ||
      (gamma && !aligned16(gamma)))
    return MOE_ERR_INVALID_ARG;
  const bool in_place = x == y && x_stride == y_stride;
  if (!in_place && overlap_rows(x, x_stride, width, y, y_stride, width, rows))
    return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  return launch_rope(ctx->cfg.head_dim, static_cast<const bf16*>(x), x_stride, heads, positions,
                     static_cast<const bf16*>(gamma), eps, rows, static_cast<bf16*>(y), y_stride,
                     rope_args(ctx), ctx->sm_count, s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_kv_append(moe_attn* ctx, const moe_kv_cache* cache, const void* k, int64_t k_stride,
                  const void* v, int64_t v_stride, const moe_attn_batch* batch, void* stream) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int rc = check_batch(ctx, cache, batch);
  if (rc != MOE_OK || batch->rows == 0) return rc;
  const int64_t width = (int64_t)ctx->cfg.kv_heads * ctx->cfg.head_dim;
  if (!rows_ok(k, k_stride, width) || !rows_ok(v, v_stride, width)) return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  AppendArgs p = {};
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return launch_append(ctx->cfg.head_dim, attn_args(ctx, cache, batch), p, s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_attn_forward(moe_attn* ctx, const moe_kv_cache* cache, const void* q, int64_t q_stride,
                     const moe_attn_batch* batch, void* out, int64_t out_stride, void* stream) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int rc = check_batch(ctx, cache, batch);
  if (rc != MOE_OK || batch->rows == 0) return rc;
  const int64_t width = (int64_t)ctx->cfg.q_heads * ctx->cfg.head_dim;
  if (!rows_ok(q, q_stride, width) || !rows_ok(out, out_stride, width) ||
      overlap_rows(q, q_stride, width, out, out_stride, width, batch->rows))
    return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  return run_attention(ctx, attn_args(ctx, cache, batch), batch, static_cast<const bf16*>(q),
                       q_stride, static_cast<bf16*>(out), out_stride, false, s);
}

int moe_attn_step(moe_attn* ctx, const moe_kv_cache* cache, const void* qkv, int64_t qkv_stride,
                  const void* q_gamma, const void* k_gamma, float eps,
                  const moe_attn_batch* batch, void* out, int64_t out_stride, void* stream) {
  if (!ctx || !isfinite(eps) || eps < 0) return MOE_ERR_INVALID_ARG;
  const int rc = check_batch(ctx, cache, batch);
  if (rc != MOE_OK || batch->rows == 0) return rc;
  const int64_t D = ctx->cfg.head_dim, Hq = ctx->cfg.q_heads, Hkv = ctx->cfg.kv_heads;
  const int64_t width = (Hq + 2 * Hkv) * D;
  if (!rows_ok(qkv, qkv_stride, width) || !rows_ok(out, out_stride, Hq * D) ||
      (q_gamma && !aligned16(q_gamma)) || (k_gamma && !aligned16(k_gamma)) ||
      overlap_rows(qkv, qkv_stride, width, out, out_stride, Hq * D, batch->rows))
    return MOE_ERR_INVALID_ARG;
  Device guard(ctx->device);
  if (!guard.ok) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ctx->last_stream = s;
  const AttnArgs a = attn_args(ctx, cache, batch);
  AppendArgs p = {};
  p.q = static_cast<const bf16*>(qkv);
  p.k = p.q + Hq * D;
  p.v = p.k + Hkv * D;
  p.q_stride = p.k_stride = p.v_stride = qkv_stride;
  p.q_out = ctx->q;
  p.q_gamma = static_cast<const bf16*>(q_gamma);
  p.k_gamma = static_cast<const bf16*>(k_gamma);
  p.eps = eps;
  p.rope = rope_args(ctx);
  if (launch_append((int)D, a, p, s) != cudaSuccess) return MOE_ERR_CUDA;
  return run_attention(ctx, a, batch, ctx->q, Hq * D, static_cast<bf16*>(out), out_stride, true,
                       s);
}

}  // extern "C"
