// pa_window.h - launch parameters of the windowed attention kernels (not part of the public ABI).
#pragma once

#include "pa_launch.h"

namespace pa {

// Parameters of one windowed attention launch.  A query at position p of its sequence sees the
// positions i <= p with i > p - window or i < sinks.
struct WindowParams {
  void* out;                    // [queries][Hq][D]
  const void* q;                // [queries][Hq][D]
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;  // [N][M]
  const int32_t* seq_lens;      // [N]
  const int32_t* query_start;   // [N + 1]: the queries of a chunk; nullptr: query s is sequence s's last token
  int32_t* err_flag;            // nullable
  int32_t num_seqs, num_q_heads, num_kv_heads;
  int32_t max_blocks, block_size, num_blocks;
  int32_t num_query_tokens;     // rows of q and out
  int32_t max_query_len;        // bound on a sequence's queries (1 without query_start)
  int32_t window, sinks;        // >= 1, >= 0
  int32_t tiles;                // row groups (8 rows) or query tiles of a sequence's kv head in the grid
  int32_t cluster;              // rows kernels: CTAs that share one item's keys,
  int32_t warps;                // and warps of a CTA (3, 4 or 6; fp32: 4)
  float scale_log2;             // scale * log2(e)
  const float* alibi;           // nullable [Hq]: score_i += slope_h * (i - p)
  float k_scale, v_scale;       // FP8 caches
  int32_t test_expire_first_wait;  // test hook: each ring's first slab is never requested (0 in normal use)
  // the step's append (nullable): each sequence's new token, [N][Hkv][D], stored at position L - 1
  const void* new_k;
  const void* new_v;
  void* k_cache_out;
  void* v_cache_out;
};

// What a rows kernel needs before its launch: its shared memory, and clusters beyond the portable eight CTAs.
template <typename Kernel>
cudaError_t prepare_rows(Kernel kernel, size_t smem, int cluster) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

// items of a rows launch: eight query rows of one kv head each
inline long long window_items(const WindowParams& p) { return (long long)p.num_seqs * p.num_kv_heads * p.tiles; }

cudaError_t launch_window_rows_tc(int dtype, int head_size, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const WindowParams& p, cudaStream_t stream);
cudaError_t launch_window_rows_fp8(const CUtensorMap& tk, const CUtensorMap& tk32, const WindowParams& p,
                                   cudaStream_t stream);
cudaError_t launch_window_rows_f32(int head_size, const WindowParams& p, cudaStream_t stream);
}  // namespace pa
