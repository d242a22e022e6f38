// pa_rope.h - launch parameters of the rotary cache write (not part of the public ABI).
#pragma once

#include "pa_internal.h"

namespace pa {

struct RopeParams {
  void* q_out;                  // [T][Hq][D], rows q_out_stride elements apart (may be q itself)
  const void* q;                // [T][Hq][D]
  const void* key;              // [T][Hkv][D]
  const void* value;            // [T][Hkv][D]
  void* k_cache;
  void* v_cache;
  int64_t q_out_stride, q_stride, key_stride, value_stride;  // elements between tokens
  const int32_t* positions;     // [T]
  const int64_t* slot_mapping;  // [T]
  const double* inv_freq;       // [rotary_dim / 2] radians per position
  int32_t num_tokens, num_q_heads, num_kv_heads, head_size, rotary_dim;
  int32_t num_blocks, block_size;
  float magnitude;
  float k_scale, v_scale;       // FP8 caches
  int32_t* err_flag;            // nullable
};

// dtype: the cache's (fp16 queries, keys and values for an FP8 cache)
cudaError_t launch_rope(int dtype, bool interleaved, const RopeParams& p, cudaStream_t stream);

}  // namespace pa
