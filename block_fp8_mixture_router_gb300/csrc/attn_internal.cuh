// Declarations shared by the attention kernels and their host code.
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kAttnMaxGroup = 16;     // query heads of one key head
constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxTokens = 0x7FFF0000;  // positions and a tile behind them fit an int
constexpr int kAttnKeys = 128;        // keys of a tile of the decode kernel
constexpr int kScaleMinExp = -100;    // the smallest block scale is 2^-100, and 448 x the
constexpr int kScaleMaxExp = 120;     // largest, 2^120, holds every bf16 value

// Device status word bits.
constexpr int kAttnTimeout = 1;
constexpr int kAttnBadBatch = 2;

// What every attention kernel knows of the layer, the cache and the batch.
struct AttnArgs {
  int Hq, Hkv, g;        // query heads, key heads, query heads of a key head
  int page_shift;        // page_tokens = 1 << page_shift
  int window;            // 0 = none
  float scale;           // softmax scale x log2(e)
  // cache
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int n_pages;
  // batch
  const int* row_start;
  const int* kv_len;
  const int* pages;
  int n_seqs, pages_stride, rows;
  int* status;
};

// The rotation of a head: turns per position of each pair as 64-bit fractions of a turn,
// good to 0.51 units (rope_turns.h), so that position x entry, taken modulo 2^64, is the
// angle modulo one turn to 2^-65 of a turn per position: 2^-34 at the farthest.
struct RopeArgs {
  const unsigned long long* turns;  // [rot / 2]
  int rot;
  int interleaved;
  float amp;
};

// Partial results of key ranges that CTAs of one launch worked through: CTA c has
// slots 2c and 2c + 1 of kAttnSlotRows rows.
struct AttnSplit {
  float* o;        // [slots][kAttnSlotRows][D]: weighted sums of the values (the prompt
                   // kernel's: [CTAs][row tiles][D / 4][128 rows][4])
  float4* sums;    // [slots][kAttnSlotRows]: the rows' references (log2) for score + log2(value
                   // scale) and for the score, and the sum of 2^(score - the latter)
  int4* shared;    // [CTAs]: the unit that begins in this CTA and goes on in others:
                   // its parts (0: none), rows, first row, key head
};
constexpr int kAttnSlotRows = 16;
constexpr int kAttnPromptRows = 256;  // rows of a slot of the prompt kernel
constexpr int kAttnPromptCtas = 320;  // most CTAs of a launch of it that splits keys, with
                                      // those that find no rows
constexpr int kAttnPromptParts = 160; // most parts of a row block's keys
constexpr int kAttnMaxCtas = 512;  // CTAs of a launch that splits units

cudaError_t launch_rope(int D, const bf16* x, int64_t x_stride, int heads, const int* positions,
                        const bf16* gamma, float eps, int rows, bf16* y, int64_t y_stride,
                        const RopeArgs& r, int sm_count, cudaStream_t s);

// Append of k and v rows; with `q` the prologue of a step: queries and keys
// normed and rotated at the batch's positions, the queries written to q_out.
struct AppendArgs {
  const bf16* k;
  const bf16* v;
  int64_t k_stride, v_stride;
  const bf16* q;          // nullptr: append only, keys as they are
  int64_t q_stride;
  bf16* q_out;            // [rows][Hq][D]
  const bf16* q_gamma;
  const bf16* k_gamma;
  float eps;
  RopeArgs rope;
};
cudaError_t launch_append(int D, const AttnArgs& a, const AppendArgs& p, cudaStream_t s);

// The cache's codes as the TMA sees them: [page][kv_heads x page_tokens][head_dim],
// a box of a page's tokens of a head (v64: at most 64 of them), 128 bytes of each (64
// at head_dim 64), stored with the swizzle of that width.
struct AttnMaps {
  CUtensorMap k, v, v64;
};
// Encodes k and v, or, for the prompt kernel, k and v64.
bool make_attn_maps(AttnMaps* m, const AttnArgs& a, int D, bool prompt);

cudaError_t setup_attn_decode(int D);
int attn_decode_slots(int D, int sm_count);  // CTAs of a full grid
// tile_rows: 8 (at most eight query heads of a key head) or 16.
cudaError_t launch_attn_decode(int D, int tile_rows, const AttnArgs& a, const AttnMaps& m,
                               const bf16* q, int64_t q_stride, bf16* out, int64_t out_stride,
                               const AttnSplit& sp, int grid, bool split, bool pdl,
                               cudaStream_t s);

// The prompt kernel: `units` row blocks of attn_prompt_tokens tokens (at most, over
// all sequences) and `splits` shares of the keys for each.
int attn_prompt_tokens(int D, int g);
cudaError_t setup_attn_prompt(int D);
cudaError_t launch_attn_prompt(int D, const AttnArgs& a, const AttnMaps& m, const bf16* q,
                               int64_t q_stride, bf16* out, int64_t out_stride,
                               const AttnSplit& sp, int units, int splits, bool pdl,
                               cudaStream_t s);

}  // namespace moe
