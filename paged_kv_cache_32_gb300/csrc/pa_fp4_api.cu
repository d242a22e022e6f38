// pa_fp4_api.cu - the C-ABI entry points of caches held in 4 bits.  Every host-side check runs before any CUDA call, so an
// argument error launches nothing.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "pa.h"
#include "pa_fp4.h"

using namespace pa::host;

namespace pa {
namespace host {

int check_cache_fp4(const pa_cache_desc* c) {
  if (c == nullptr) return PA_ERR_NULL_POINTER;
  if (c->dtype != PA_FP4_E2M1) return PA_ERR_UNSUPPORTED;
  if (c->num_blocks < 0 || c->block_size <= 0 || c->num_kv_heads <= 0 || c->head_size <= 0) return PA_ERR_INVALID_ARG;
  if (c->head_size != pa::kFp4D || c->block_size % pa::kFp4Tokens != 0 || c->block_size > 256) return PA_ERR_UNSUPPORTED;
  if ((int64_t)c->num_blocks * c->num_kv_heads * c->block_size > kInt32Max) return PA_ERR_TOO_LARGE;
  return PA_OK;
}

bool fp4_unit_ok(float x) { return x >= 7.888609e-31f && x <= 1.2676506e30f; }  // 2^-100 .. 2^100

}  // namespace host
}  // namespace pa

namespace {

int check_row_dtype(int32_t row_dtype) { return row_dtype == PA_F16 || row_dtype == PA_BF16 ? PA_OK : PA_ERR_UNSUPPORTED; }

// The checks that the write and the read share, and their parameters.
int rows_params(pa::Fp4Rows& p, void* k_cache, void* v_cache, void* key, void* value, int64_t key_stride,
                int64_t value_stride, const int64_t* slot_mapping, int32_t num_tokens, const pa_cache_desc* cache,
                int32_t row_dtype, float k_scale, float v_scale, int32_t* err_flag) {
  int rc = check_cache_fp4(cache);
  if (rc == PA_OK) rc = check_row_dtype(row_dtype);
  if (rc != PA_OK) return rc;
  if (num_tokens < 0 || !fp4_unit_ok(k_scale) || !fp4_unit_ok(v_scale)) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (k_cache == nullptr || v_cache == nullptr || key == nullptr || value == nullptr || slot_mapping == nullptr)
    return PA_ERR_NULL_POINTER;
  const int64_t row = (int64_t)cache->num_kv_heads * cache->head_size;
  if (key_stride < row || value_stride < row) return PA_ERR_INVALID_ARG;
  const int64_t max_stride = ((int64_t)1 << 44) / num_tokens;
  if (key_stride > max_stride || value_stride > max_stride) return PA_ERR_TOO_LARGE;
  if ((int64_t)num_tokens * cache->num_kv_heads > kInt32Max) return PA_ERR_TOO_LARGE;
  if (key_stride % 8 != 0 || value_stride % 8 != 0 || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(key, 16) || !aligned(value, 16) || !aligned(slot_mapping, 8))
    return PA_ERR_MISALIGNED;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.key = key;
  p.value = value;
  p.key_stride = key_stride;
  p.value_stride = value_stride;
  p.slot_mapping = slot_mapping;
  p.num_tokens = num_tokens;
  p.num_kv_heads = cache->num_kv_heads;
  p.num_blocks = cache->num_blocks;
  p.block_size = cache->block_size;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err_flag = err_flag;
  return PA_OK;
}

// Checks that both attention calls share.
int check_attention(const pa_cache_desc* cache, int32_t row_dtype, int32_t num_seqs, int32_t num_q_heads,
                    int32_t max_blocks_per_seq, float scale, int32_t window, int32_t num_sinks, float k_scale,
                    float v_scale) {
  int rc = check_cache_fp4(cache);
  if (rc == PA_OK) rc = check_row_dtype(row_dtype);
  if (rc != PA_OK) return rc;
  if (num_seqs < 0 || num_q_heads <= 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
  if (num_q_heads % cache->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (!(scale == scale) || isinf(scale)) return PA_ERR_INVALID_ARG;
  if (window < 1 || num_sinks < 0 || !fp4_unit_ok(k_scale) || !fp4_unit_ok(v_scale)) return PA_ERR_INVALID_ARG;
  // positions are int32, with room for a key tile past the last one
  if ((int64_t)max_blocks_per_seq * cache->block_size > kInt32Max - 4096) return PA_ERR_TOO_LARGE;
  return PA_OK;
}

pa::WindowParams base_params(const pa_cache_desc* cache, void* out, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* block_tables, const int32_t* seq_lens,
                             int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks, float scale, int32_t window,
                             int32_t num_sinks, float k_scale, float v_scale, int32_t* err_flag) {
  pa::WindowParams p = {};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.err_flag = err_flag;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.max_blocks = max_blocks;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.num_query_tokens = num_seqs;
  p.max_query_len = 1;
  p.window = window;
  p.sinks = num_sinks;
  p.cluster = 1;
  p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  return p;
}

}  // namespace

extern "C" {

int pa_reshape_and_cache_fp4(void* k_cache, void* v_cache, const void* key, const void* value, int64_t key_stride,
                             int64_t value_stride, const int64_t* slot_mapping, int32_t num_tokens,
                             const pa_cache_desc* cache, int32_t row_dtype, float k_scale, float v_scale,
                             int32_t* err_flag, void* stream) {
  pa::Fp4Rows p = {};
  const int rc = rows_params(p, k_cache, v_cache, const_cast<void*>(key), const_cast<void*>(value), key_stride, value_stride,
                             slot_mapping, num_tokens, cache, row_dtype, k_scale, v_scale, err_flag);
  if (rc != PA_OK || num_tokens == 0) return rc;
  return pa::launch_fp4_write(row_dtype, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_read_cache_fp4(void* key, void* value, const void* k_cache, const void* v_cache, int64_t key_stride,
                      int64_t value_stride, const int64_t* slot_mapping, int32_t num_tokens, const pa_cache_desc* cache,
                      int32_t row_dtype, float k_scale, float v_scale, int32_t* err_flag, void* stream) {
  pa::Fp4Rows p = {};
  const int rc = rows_params(p, const_cast<void*>(k_cache), const_cast<void*>(v_cache), key, value, key_stride, value_stride,
                             slot_mapping, num_tokens, cache, row_dtype, k_scale, v_scale, err_flag);
  if (rc != PA_OK || num_tokens == 0) return rc;
  return pa::launch_fp4_read(row_dtype, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_decode_fp4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                    const pa_cache_desc* cache, int32_t window, int32_t num_sinks) {
  if (check_attention(cache, PA_F16, num_seqs, num_q_heads, max_blocks_per_seq, 1.f, window, num_sinks, 1.f, 1.f) != PA_OK)
    return 0;
  pa::WindowParams p = {};
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.window = window;
  p.sinks = num_sinks;
  return pa::fp4_deals_evenly(cache, p) ? pa::fp4_even_workspace() : 0;
}

int pa_decode_fp4(void* out, const void* q, void* k_cache, void* v_cache, const void* key, const void* value,
                  const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                  int32_t max_blocks_per_seq, const pa_cache_desc* cache, int32_t row_dtype, float scale, int32_t window,
                  int32_t num_sinks, float k_scale, float v_scale, const float* alibi_slopes, uint32_t test_flags,
                  void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const int rc = check_attention(cache, row_dtype, num_seqs, num_q_heads, max_blocks_per_seq, scale, window, num_sinks,
                                 k_scale, v_scale);
  if (rc != PA_OK) return rc;
  if ((key == nullptr) != (value == nullptr)) return PA_ERR_NULL_POINTER;
  if (num_seqs == 0) return PA_OK;
  if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr || seq_lens == nullptr)
    return PA_ERR_NULL_POINTER;
  if (block_tables == nullptr && max_blocks_per_seq > 0) return PA_ERR_NULL_POINTER;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(key, 16) ||
      !aligned(value, 16) || !aligned(seq_lens, 4) || !aligned(block_tables, 4) || !aligned(alibi_slopes, 4))
    return PA_ERR_MISALIGNED;
  if ((int64_t)num_seqs * num_q_heads > kInt32Max) return PA_ERR_TOO_LARGE;
  if (!aligned(workspace, 256)) return PA_ERR_MISALIGNED;
  pa::WindowParams p = base_params(cache, out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_q_heads,
                                   max_blocks_per_seq, scale, window, num_sinks, k_scale, v_scale, err_flag);
  p.alibi = alibi_slopes;
  p.test_expire_first_wait = (test_flags & PA_DECODE_TEST_EXPIRE_FIRST_WAIT) != 0u ? 1 : 0;
  p.new_k = key;
  p.new_v = value;
  p.k_cache_out = k_cache;
  p.v_cache_out = v_cache;
  if (workspace != nullptr && pa::fp4_deals_evenly(cache, p) && workspace_bytes < pa::fp4_even_workspace())
    return PA_ERR_WORKSPACE;
  return pa::fp4_decode(cache, row_dtype, p, static_cast<float*>(workspace), static_cast<cudaStream_t>(stream));
}

int pa_prefill_fp4(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   const int32_t* seq_lens, const int32_t* query_start, int32_t num_seqs, int32_t num_query_tokens,
                   int32_t num_q_heads, int32_t max_blocks_per_seq, int32_t max_query_len, const pa_cache_desc* cache,
                   int32_t row_dtype, float scale, int32_t window, int32_t num_sinks, float k_scale, float v_scale,
                   int32_t* err_flag, void* stream) {
  const int rc = check_attention(cache, row_dtype, num_seqs, num_q_heads, max_blocks_per_seq, scale, window, num_sinks,
                                 k_scale, v_scale);
  if (rc != PA_OK) return rc;
  if (num_query_tokens < 0 || max_query_len < 0 || !(scale > 0.f)) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PA_OK;
  if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr || seq_lens == nullptr ||
      query_start == nullptr || block_tables == nullptr)
    return PA_ERR_NULL_POINTER;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) ||
      !aligned(query_start, 4) || !aligned(block_tables, 4))
    return PA_ERR_MISALIGNED;
  if ((int64_t)num_query_tokens * num_q_heads * 128 > ((int64_t)1 << 40)) return PA_ERR_TOO_LARGE;
  pa::WindowParams p = base_params(cache, out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_q_heads,
                                   max_blocks_per_seq, scale, window, num_sinks, k_scale, v_scale, err_flag);
  p.query_start = query_start;
  p.num_query_tokens = num_query_tokens;
  p.max_query_len = std::min(max_query_len, num_query_tokens);  // no valid chunk is longer
  return pa::fp4_chunk(cache, row_dtype, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
