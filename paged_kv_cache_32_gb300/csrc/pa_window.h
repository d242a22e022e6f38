// pa_window.h - launch parameters of the windowed attention kernels (not part of the public ABI).
#pragma once

#include "pa_internal.h"

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

// items of a rows launch: eight query rows of one kv head each
inline long long window_items(const WindowParams& p) { return (long long)p.num_seqs * p.num_kv_heads * p.tiles; }

cudaError_t launch_window_rows_tc(int dtype, int head_size, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const WindowParams& p, cudaStream_t stream);
cudaError_t launch_window_rows_fp8(const CUtensorMap& tk, const CUtensorMap& tk32, const WindowParams& p,
                                   cudaStream_t stream);
cudaError_t launch_window_rows_f32(int head_size, const WindowParams& p, cudaStream_t stream);
// Launch in clusters of `cluster` CTAs (1: none) as a programmatic dependent of the kernel before it (see
// launch_dependent).
template <typename... Params, typename... Args>
inline cudaError_t launch_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster,
                                  cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
