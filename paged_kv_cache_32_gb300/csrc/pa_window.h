// pa_window.h - launch parameters of the windowed attention kernels (not part of the public ABI).
#pragma once

#include <atomic>

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
  int32_t tiles;                // row groups (8 rows) of a kv head in the grid: each sequence's, or (slots) all of theirs
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

// Whether devices have room for a cluster of a kernel's beyond the portable eight CTAs, one of these per kernel.
struct ClusterRoom {
  static constexpr int kDevices = 64;
  std::atomic<signed char> known[kDevices] = {};  // 0: not asked yet, 1: yes, -1: no
};
constexpr int kPortableCluster = 8;

// What a rows kernel needs before its launch: its shared memory, and a cluster size that the current device places: a
// larger one than eight may fit none of its GPCs (a partition of a GPU may hold few SMs of each), and its launch would
// be an error, so *cluster becomes eight there.  The device is asked once.
template <typename Kernel>
cudaError_t prepare_rows(Kernel kernel, ClusterRoom& room, int threads, size_t smem, int32_t* cluster) {
  const void* f = reinterpret_cast<const void*>(kernel);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess || *cluster <= kPortableCluster) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const bool kept = dev < ClusterRoom::kDevices;
  int fits = kept ? room.known[dev].load(std::memory_order_relaxed) : 0;
  if (fits == 0) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)*cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)*cluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, f, &cfg) != cudaSuccess) {
      clusters = 0;
      (void)cudaGetLastError();  // the answer is no: the call goes on
    }
    fits = clusters > 0 ? 1 : -1;
    if (kept) room.known[dev].store((signed char)fits, std::memory_order_relaxed);
  }
  if (fits < 0) *cluster = kPortableCluster;
  return cudaSuccess;
}

// items of a rows launch: eight query rows of one kv head each
inline long long window_items(const WindowParams& p, bool slots) {
  return (long long)(slots ? 1 : p.num_seqs) * p.num_kv_heads * p.tiles;
}

// slots: the sequences' row groups lie one after the other in p.tiles slots (see rows_find)
cudaError_t launch_window_rows_tc(int dtype, int head_size, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const WindowParams& p, bool slots, cudaStream_t stream);
cudaError_t launch_window_rows_fp8(const CUtensorMap& tk, const CUtensorMap& tk32, const WindowParams& p, bool slots,
                                   cudaStream_t stream);
cudaError_t launch_window_rows_f32(int head_size, const WindowParams& p, bool slots, cudaStream_t stream);
}  // namespace pa
