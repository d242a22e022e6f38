// pa_prefill.h - launch parameters of the tensor-core chunked prefill (not part
// of the public ABI).
#pragma once

#include "pa_internal.h"

namespace pa {

// Parameters of one chunked-prefill launch.
struct PrefillParams {
  void* out;                    // [total_q][Hq][D]
  const void* q;                // [total_q][Hq][D]
  const void* k_cache;          // [num_blocks][Hkv][B][D]
  const void* v_cache;
  const int32_t* block_tables;  // [N][M]
  const int32_t* seq_lens;      // [N] cached tokens including the chunk
  const int32_t* query_start;   // [N + 1]
  int32_t* err_flag;            // nullable
  int32_t num_seqs, num_q_heads, num_kv_heads;
  int32_t max_blocks, block_size, num_blocks;
  int32_t head_size;            // 128; windowed form over 16-bit caches: 64 too
  int32_t q_tiles;              // query tiles of the longest chunk: ceil(max_query_len / 128) in the plain form
  int32_t num_query_tokens;     // rows of q and out
  float scale_log2;
  // windowed form (pa_prefill_window; window 0: the plain one): a query at position p sees the positions i <= p
  // with i > p - window or i < sinks; a query tile is 128 >> pack_log2 queries of 2^pack_log2 query heads of one
  // kv head
  int32_t window, sinks, pack_log2;
  int32_t max_query_len;        // windowed form: bound on a chunk's queries
  int32_t split;                // windowed form: CTAs of a cluster that share one item's key tiles
  // windowed form over an FP8 or a 4-bit cache: a value code's scale (the key codes' is part of scale_log2)
  float v_scale;
};

namespace host {
bool encode_query_map(CUtensorMap* map, const void* base, const pa_cache_desc* c, int32_t num_q_heads,
                      int32_t num_query_tokens, int heads);
}

// tk, tv: the caches as rows of D elements (box 64 columns x block_size rows, 128-byte swizzle);
// tq: q as [tokens][heads][D] (box 64 columns x 1 head x 128 tokens, windowed 2^pack_log2 heads x the tile's
// tokens, 128-byte swizzle); to: out, the same
// dtype: the cache's (FP8: windowed form only, tk and tv not used)
// mixed: windowed form, most sequences' chunks are far shorter than max_query_len (no field of the parameters: one
// more there, wherever it stood, moved the kernels' spills about and cost FP8 chunks 3 to 20 %)
cudaError_t launch_prefill_tc(int dtype, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                              const CUtensorMap& to, const PrefillParams& p, bool mixed,
                              cudaStream_t stream);
// sequences that the tile kernel over a 4-bit cache deals out with the longest first
constexpr int kDealMaxSeqs = 96;
// over a 4-bit cache, windowed form; row_dtype: of q and out
cudaError_t launch_prefill_fp4(int row_dtype, const CUtensorMap& tq, const CUtensorMap& to, const PrefillParams& p,
                               bool mixed, cudaStream_t stream);

}  // namespace pa
