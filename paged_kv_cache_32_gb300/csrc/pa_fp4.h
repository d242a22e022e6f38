// pa_fp4.h - caches held in 4 bits: layout and launchers (not part of the public ABI).
#pragma once

#include "pa_rope.h"
#include "pa_window.h"

namespace pa {

// Of each (block, kv head), every 16 tokens are one tile: [16][64] bytes of codes, then [16][8] scales.
constexpr int kFp4D = 128;
constexpr int kFp4Tokens = 16;
constexpr int kFp4RowBytes = kFp4D / 2;
constexpr int kFp4RowScales = kFp4D / 16;
constexpr int kFp4CodeBytes = kFp4Tokens * kFp4RowBytes;
constexpr int kFp4TileBytes = kFp4CodeBytes + kFp4Tokens * kFp4RowScales;

struct Fp4Rows {
  uint8_t* k_cache;
  uint8_t* v_cache;
  void* key;    // [T][Hkv][D], 16 bits; written by the read, else only read
  void* value;
  int64_t key_stride, value_stride;  // elements between tokens
  const int64_t* slot_mapping;       // [T]
  int32_t num_tokens, num_kv_heads, num_blocks, block_size;
  float k_scale, v_scale;
  int32_t* err_flag;                 // nullable
};
cudaError_t launch_fp4_write(int row_dtype, const Fp4Rows& p, cudaStream_t stream);
cudaError_t launch_fp4_read(int row_dtype, const Fp4Rows& p, cudaStream_t stream);
// rotary positions with the write, where the halves of the turned elements are no multiple of a group
cudaError_t launch_fp4_rope_cut(int row_dtype, const RopeAxesParams& p, cudaStream_t stream);

// rows attention (see pa_window.h); row_dtype: of q, out and the appended rows
cudaError_t launch_fp4_rows(int row_dtype, const WindowParams& p, bool slots, cudaStream_t stream);

// a decode step whose slabs are dealt out evenly to a grid of kFp4EvenGrid CTAs, in a workspace of fp4_even_workspace() bytes
constexpr int kFp4EvenGrid = 152 * 4;
size_t fp4_even_workspace();
cudaError_t launch_fp4_even(int row_dtype, const WindowParams& p, float* workspace, cudaStream_t stream);
// does a decode step use such a workspace?
bool fp4_deals_evenly(const pa_cache_desc* cache, const WindowParams& p);
// a decode step, with its kernel and split chosen (workspace: nullable); a chunk, with its kernel chosen too (a PA_* status)
int fp4_decode(const pa_cache_desc* cache, int32_t row_dtype, WindowParams& p, float* workspace, cudaStream_t stream);
int fp4_chunk(const pa_cache_desc* cache, int32_t row_dtype, WindowParams& p, cudaStream_t stream);

namespace host {
int check_cache_fp4(const pa_cache_desc* c);
// A cache's unit: such that six times it, its product with any scale and the inverse of that are ordinary fp32 numbers.
bool fp4_unit_ok(float x);
}

}  // namespace pa
