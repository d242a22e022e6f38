// pa_window_api.cu - the C-ABI entry points of windowed attention: argument
// validation, tensor maps, the choice of kernel and split.  Every host-side
// check runs before any CUDA call, so an argument error launches nothing.
#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "pa.h"
#include "pa_fp4.h"
#include "pa_prefill.h"
#include "pa_window.h"

using namespace pa::host;

namespace {

constexpr int kSms = 152;          // of a GB300, which the choices below were measured on: elsewhere slower, not wrong
constexpr int kMaxCluster = pa::kPortableCluster;  // (rows kernels also take the largest, twice that, where it fits)
constexpr int kMinCtaTokens = 64;  // tokens of a CTA below which a split no longer pays
constexpr int kFewItems = 4096;    // work items whose empty ones cost a few microseconds at most
constexpr int kLongShare = 600;    // fp32: tokens of a CTA that is split though every SM has its CTAs

// How the rows kernels spread over the SMs.  A warp holds 16 KB of slabs, so an SM takes 4 CTAs of 3 warps, 3 of 4
// or 2 of 6.
//  * Few items (at most half the SMs): CTAs of 6 warps, an item's keys split over a cluster until the CTAs fill the
//    SMs twice.  One sequence, 8 kv heads, 4096 keys: 10.8 us (clusters of 4: 15.4; 4 warps: 12.4); 64 items of
//    4096 keys: 27.1 us (4 warps: 29.4; clusters of 2: 29.2).  Clusters of 16 where each CTA has an SM of its own
//    and 256 keys: those 4096 keys 10.2 us, 16384 keys 25.2 -> 17.7 (1024 keys 7.0 -> 7.7; 16 such items, whose
//    clusters do not all find room at once, 12.2 -> 18.4).
//  * More: no split (a cluster waits for as many free places at once: two of 4 warps cost 94 -> 109 us on 1024
//    items of 1024 keys), and the CTA size whose last round is fullest, the smallest among equals.  1024 keys:
//    256 items 26.6 / 27.9 / 28.7 us with 6 / 4 / 3 warps, 384 items 42.8 / 37.4 / 38.7, 512 items 48.6 / 58.0 /
//    48.3, 768 items 69.9 / 67.8 / 74.5, 1024 items 92.2 / 93.4 / 87.9.  Six warps hold few slabs each of short items
//    (2048 FP8 items of 512 / 1024 keys: 71.5 / 109 us, with four 66 / 103), so not for many of those; of long ones,
//    whose lengths are seldom equal, they also win ties (96 sequences, 8 kv heads, W = 8192, contexts of up to 20000
//    tokens: bf16 351 -> 326 us, FP8 220 -> 204; equal lengths within 1%, but for 512 FP8 items of 4096, 89 -> 94).
//    (Splitting long items in two all the same evens out a last round of unequal contexts, 96 FP8 sequences of
//    2500 to 40000 tokens with a window of 8192: 240 -> 226 us, and costs as much when they are equal, 246 -> 264.)
//  * fp32 (CUDA cores): four warps a CTA, three CTAs an SM, split while that many are not there, in clusters of 16
//    up to two an SM (8 kv heads, 1024 / 4096 keys: 13.3 -> 11.7 and 28.0 -> 20.7 us; 16 items 15.1 -> 13.6 and
//    34.6 -> 26.9).  A warp walks its keys slowly there, so that the longest item sets the time: long ones are split
//    on as long as a CTA keeps kLongShare keys (392 items of head size 64, up to 1285 keys 77 -> 56 us, W = 3538 263
//    -> 187; 128 items, W = 4096, 137 -> 96; equal items of 1024 keys would lose, 80 -> 90).
void spread(int32_t dtype, long long items, long long max_keys, pa::WindowParams& p) {
  p.cluster = 1;
  if (dtype == PA_F32) {
    p.warps = 4;
    while (p.cluster < kMaxCluster && items * p.cluster * 2 <= 3 * kSms && max_keys / (2 * p.cluster) >= kMinCtaTokens)
      p.cluster *= 2;
    if (items * 2 * kMaxCluster <= 2 * kSms && max_keys / (2 * kMaxCluster) >= kMinCtaTokens) p.cluster = 2 * kMaxCluster;
    while (p.cluster < kMaxCluster && items * p.cluster * 2 <= 12 * kSms && max_keys / (2 * p.cluster) >= kLongShare)
      p.cluster *= 2;
    return;
  }
  if (items <= kSms / 2) {
    p.warps = 6;
    while (p.cluster < kMaxCluster && items * p.cluster * 2 <= 2 * kSms &&
           max_keys / (2 * p.cluster) >= kMinCtaTokens)
      p.cluster *= 2;
    if (items * 2 * kMaxCluster <= kSms && max_keys / (2 * kMaxCluster) >= 4 * kMinCtaTokens)
      p.cluster = 2 * kMaxCluster;
    return;
  }
  double best = 0.0;
  for (int warps : {3, 4, 6}) {
    const double rounds = (double)items / (kSms * (12 / warps));
    const double full = rounds / ceil(rounds);
    if (warps == 6 && max_keys < 1536 && items > 4 * kSms) break;
    if (full > best + (warps == 6 && max_keys >= 4096 ? -1e-9 : 1e-9)) {
      best = full;
      p.warps = warps;
    }
  }
}

// Checks that both entry points share.
int check_window(const pa_cache_desc* cache, int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
                 float scale, int32_t window, int32_t num_sinks) {
  const int rc = check_cache(cache);
  if (rc != PA_OK) return rc;
  if (num_seqs < 0 || num_q_heads <= 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
  if (num_q_heads % cache->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (!(scale == scale) || isinf(scale)) return PA_ERR_INVALID_ARG;
  if (window < 1 || num_sinks < 0) return PA_ERR_INVALID_ARG;
  // positions are int32, with room for a key tile past the last one
  if ((int64_t)max_blocks_per_seq * cache->block_size > kInt32Max - 4096) return PA_ERR_TOO_LARGE;
  return PA_OK;
}

// The scales of an FP8 cache; those of any other are 1, whatever the caller passes (the kernels multiply by them).
int check_scales(const pa_cache_desc* cache, float* k_scale, float* v_scale) {
  const bool fp8 = cache->dtype == PA_FP8_E4M3;
  if (!fp8 || *k_scale == 0.f) *k_scale = 1.f;
  if (!fp8 || *v_scale == 0.f) *v_scale = 1.f;
  return *k_scale > 0.f && !isinf(*k_scale) && *v_scale > 0.f && !isinf(*v_scale) ? PA_OK : PA_ERR_INVALID_ARG;
}

// A cache as (64 columns, rows, D / 64): a box of `rows` rows brings their 64-column parts one after the other
bool encode_slab_map(CUtensorMap* map, const void* base, const pa_cache_desc* c, int rows) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint32_t parts = (cuuint32_t)(c->head_size / 64);
  cuuint64_t dims[3] = {64, (cuuint64_t)c->num_blocks * c->num_kv_heads * c->block_size, parts};
  cuuint64_t strides[2] = {(cuuint64_t)c->head_size * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)rows, parts};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt =
      c->dtype == PA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(map, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Does a batch mix long chunks with many short ones, so that most items of a grid of `items` (the longest chunk's for
// every sequence) have no queries, when at most `real` have?  The forms for such batches pay for their search: a rows
// CTA about what two or three empty ones do.  A prompt of P among N - 1 single tokens, 64 / 8 heads, W = 1024, us with
// these forms and with the others: tiles, bf16, N = 32, P = 512 86 / 87, N = 128, P = 2048 285 / 624, N = 1024, P = 4096
// 1620 / 7890; fp32 rows 602 / 718, 2845 / 5120, 7080 / 46200.
bool mixes(long long items, long long real) { return items > kFewItems && items > 4 * real; }

// Launches the rows kernel of the cache's type (row_dtype: of queries and outputs over a 4-bit cache); p.tiles (row
// groups), p.cluster and p.warps are set here.
int launch_rows(const pa_cache_desc* cache, pa::WindowParams& p, cudaStream_t stream, int32_t row_dtype = PA_F16) {
  const long long rows = (long long)p.max_query_len * (p.num_q_heads / p.num_kv_heads);
  if (rows > kInt32Max - 8) return PA_ERR_TOO_LARGE;
  p.tiles = (int32_t)((rows + 7) / 8);
  bool slots = false;
  if (p.query_start != nullptr) {
    const long long real = (long long)p.num_query_tokens * (p.num_q_heads / p.num_kv_heads) / 8 + p.num_seqs;
    slots = real <= kInt32Max && mixes(pa::window_items(p, false), real * p.num_kv_heads);
    if (slots) p.tiles = (int32_t)real;
  }
  // keys that an item may see: its rows' windows, the first tokens, all within the table
  const long long cap = (long long)p.max_blocks * p.block_size;
  const long long reach = (long long)p.window + p.sinks + 8;
  const long long items = pa::window_items(p, slots);
  spread(cache->dtype, items, reach < cap ? reach : cap, p);
  if (items * p.cluster > kInt32Max) return PA_ERR_TOO_LARGE;
  cudaError_t e;
  if (cache->dtype == PA_F32) {
    e = pa::launch_window_rows_f32(cache->head_size, p, slots, stream);
  } else if (cache->dtype == PA_FP4_E2M1) {
    e = pa::launch_fp4_rows(row_dtype, p, slots, stream);
  } else if (cache->dtype == PA_FP8_E4M3) {
    CUtensorMap tk, tk32;
    if (!encode_fp8_key_map(&tk, p.k_cache, cache, pa::kTcSlabTokens) ||
        !encode_fp8_key_map(&tk32, p.k_cache, cache, 2 * pa::kTcSlabTokens))
      return PA_ERR_CUDA;
    e = pa::launch_window_rows_fp8(tk, tk32, p, slots, stream);
  } else {
    CUtensorMap tk, tv;
    // a slab is one 16-row box, or (8-token blocks) two 8-row boxes from two blocks
    const int box_rows = cache->block_size < pa::kTcSlabTokens ? cache->block_size : pa::kTcSlabTokens;
    if (!encode_slab_map(&tk, p.k_cache, cache, box_rows) || !encode_slab_map(&tv, p.v_cache, cache, box_rows))
      return PA_ERR_CUDA;
    e = pa::launch_window_rows_tc(cache->dtype, cache->head_size, tk, tv, p, slots, stream);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The tile kernel's query heads of a tile: the largest power of two that divides the group (at most 128).
int pack_log2(int G) {
  int k = 0;
  while (k < 7 && G % (2 << k) == 0) ++k;
  return k;
}

// 16-bit and FP8 caches whose blocks fit the 128-key tiles run on the tensor-core tile kernel, and every 4-bit cache
bool tile_kernel_takes(const pa_cache_desc* c) {
  return c->dtype == PA_FP4_E2M1 || (c->dtype != PA_F32 && 128 % c->block_size == 0);
}

// CTAs that share an item's key tiles: as many as leave each SM at most one, with four tiles or more each.  Over a 4-bit
// cache up to two an SM, with eight tiles or more: its tiles take longer to convert, so that the longest of unequal items
// is what a call waits for (they start with the longest, too).  With more items than that, two an item if that takes less
// time with all at the longest, by 6 us and 1.32 a key tile for every item of an SM and 12 us and 0.66 a tile for every
// half: by 7 % or more where whole items are dealt out with the longest first, or, with more sequences, by -15 %, since
// whole ones then come in any order.  (Every CTA ranks the sequences: not past 512.)  5 queries each, 64 / 8 heads, 20 /
// 40 / 64 / 100 sequences of unequal lengths up to 20000, in halves: 155 / 255 / 375 / 581 us, dealt out 211 / 284 / 342
// / -, in order 290 / 368 / 539 / 762; one chunk of 700 over 30000, 32 / 8 heads: 451 in halves, 560 dealt out.
int tile_split(long long items, long long max_keys, bool fp4, int seqs) {
  int c = 1;
  while (c < kMaxCluster && items * c * 2 <= kSms && max_keys / (128 * 2 * c) >= 4) c *= 2;
  while (fp4 && c < kMaxCluster && items * c * 2 <= 2 * kSms && max_keys / (128 * 2 * c) >= 8) c *= 2;
  if (fp4 && c == 1 && items > kSms && items <= 6 * kSms && seqs <= 512) {
    const double tiles = ceil(max_keys / 128.0);
    const double whole = ceil(items / (double)kSms) * (6.0 + 1.32 * tiles);
    const double halves = ceil(2 * items / (double)kSms) * (12.0 + 0.66 * tiles);
    if (halves <= (seqs <= pa::kDealMaxSeqs ? 0.93 : 1.15) * whole) c = 2;
  }
  return c;
}

// Is a chunk faster on the tile kernel than on the rows kernel?  By an estimate of both whose constants were fitted to
// 432 chunks of 1 to 17 queries (1 to 32 sequences, 7 to 64 query heads on 1 to 32 kv heads, 300 and 4096 keys, bf16 of
// head size 128 and 64, FP8), on which it loses at most 12% to the faster one:
//  * rows: 6 us and the longer of 1 us for `rate` keys of an eight-row group over all, and 0.85 us for each slab of 16
//    keys (FP8: 1.3 us for 32) of the warp with most;
//  * tiles: 5 us and, for each item that an SM gets, 1 us and `per_tile` a key tile.
// Over a 4-bit cache fitted apart, to 250 chunks of 1 to 64 queries (1 to 64 sequences, 300 to 20000 keys): 1 % lost on
// average, and up to a half (12 us for 18) for five queries over 300 keys.
// E.g. 32 sequences, 64 / 8 heads, 4096 keys, bf16: 2 queries each 95 us on rows and 104 on tiles, 5 queries 204 and
// 104; 8 sequences of 5 queries: 70 and 35; one of 3 with 300 keys: 7 and 10.5.
bool tiles_faster(const pa_cache_desc* cache, pa::WindowParams p, int pack) {
  const bool fp8 = cache->dtype == PA_FP8_E4M3, fp4 = cache->dtype == PA_FP4_E2M1;
  const int G = p.num_q_heads / p.num_kv_heads, queries = 128 >> pack;
  const double kv = (double)p.num_seqs * p.num_kv_heads;
  const double keys = std::min((double)p.max_blocks * p.block_size, (double)p.window + p.sinks + queries);
  const double groups = kv * ceil((double)p.max_query_len * G / 8);
  spread(cache->dtype, (long long)std::min(groups, 1e9), (long long)keys, p);
  const double slabs = ceil(keys / (fp8 || fp4 ? 32.0 : 16.0) / (p.warps * p.cluster));
  const bool narrow = cache->head_size == 64;
  const double rate = fp4 ? 32500.0 : fp8 ? 35000.0 : narrow ? 26000.0 : 30000.0;
  const double per_tile = fp4 ? 1.4 : narrow ? 1.6 : 1.3;
  const double rows_us = (fp4 ? 6.5 : 6.0) + std::max(groups * keys / rate, slabs * (fp4 ? 1.2 : fp8 ? 1.3 : 0.85));
  const double items = kv * ceil((double)p.max_query_len / queries) * (G >> pack);
  const int split = tile_split((long long)std::min(items, 1e9), (long long)keys, fp4, p.num_seqs);
  const double share = items * split / kSms, tiles = ceil(keys / 128.0) / split;
  const double tile_us =
      (fp4 ? 6.0 : 5.0) + std::max(1.0, 0.5 * (share + ceil(share))) * ((fp4 ? 4.0 : 1.0) + per_tile * tiles);
  return tile_us < rows_us;
}

// the tile kernel's work items: the longest chunk's tiles for every sequence and head group
long long tile_items(const pa::WindowParams& w, int pack) {
  const long long q_tiles = ((long long)w.max_query_len + (128 >> pack) - 1) / (128 >> pack);
  return w.num_seqs * q_tiles * (w.num_q_heads >> pack);
}

int launch_tiles(const pa_cache_desc* cache, const pa::WindowParams& w, int pack, cudaStream_t stream,
                 int32_t row_dtype = PA_F16) {
  const long long items = tile_items(w, pack);
  CUtensorMap tk, tv, tq, to;
  const bool fp8 = cache->dtype == PA_FP8_E4M3, fp4 = cache->dtype == PA_FP4_E2M1;  // read by plain loads
  pa_cache_desc rows = *cache;
  if (fp4) rows.dtype = row_dtype;
  if ((!fp8 && !fp4 && (!encode_cache_map(&tk, w.k_cache, cache, cache->block_size) ||
                !encode_cache_map(&tv, w.v_cache, cache, cache->block_size))) ||
      !encode_query_map(&tq, w.q, &rows, w.num_q_heads, w.num_query_tokens, 1 << pack) ||
      !encode_query_map(&to, w.out, &rows, w.num_q_heads, w.num_query_tokens, 1 << pack))
    return PA_ERR_CUDA;
  pa::PrefillParams p = {};
  p.out = w.out;
  p.q = w.q;
  p.k_cache = w.k_cache;
  p.v_cache = w.v_cache;
  p.block_tables = w.block_tables;
  p.seq_lens = w.seq_lens;
  p.query_start = w.query_start;
  p.err_flag = w.err_flag;
  p.num_seqs = w.num_seqs;
  p.num_q_heads = w.num_q_heads;
  p.num_kv_heads = w.num_kv_heads;
  p.max_blocks = w.max_blocks;
  p.block_size = w.block_size;
  p.num_blocks = w.num_blocks;
  p.head_size = cache->head_size;
  p.q_tiles = (int32_t)(items / w.num_seqs / (w.num_q_heads >> pack));
  p.num_query_tokens = w.num_query_tokens;
  p.scale_log2 = w.scale_log2 * w.k_scale;
  p.v_scale = w.v_scale;
  p.window = w.window;
  p.sinks = w.sinks;
  p.pack_log2 = pack;
  p.max_query_len = w.max_query_len;
  const bool mixed =
      mixes(items, ((long long)w.num_query_tokens / (128 >> pack) + w.num_seqs) * (w.num_q_heads >> pack));
  // (a split item of a sequence that lacks it still takes a cluster: not where many do)
  p.split = tile_split(mixed && items > kSms ? kInt32Max : items,
                       std::min((long long)w.max_blocks * w.block_size, (long long)w.window + w.sinks + 128), fp4,
                       w.num_seqs);
  if (fp4) {
    // (a masked score is -inf times the scale, which must not vanish; bf16 queries: times their row's, in the kernel)
    if (row_dtype == PA_F16) p.scale_log2 = std::max(p.scale_log2, 1.17549435e-38f);
    return pa::launch_prefill_fp4(row_dtype, tq, to, p, mixed, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  if (fp8) tk = tv = tq;
  return pa::launch_prefill_tc(cache->dtype, tk, tv, tq, to, p, mixed, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int launch_chunk(const pa_cache_desc* cache, pa::WindowParams& p, cudaStream_t stream, int32_t row_dtype = PA_F16) {
  const int pack = pack_log2(p.num_q_heads / p.num_kv_heads);
  // (the tile kernel counts its items in int32, with room for one grid stride past the end; the rows kernels' slots fit)
  if (tile_kernel_takes(cache) && tile_items(p, pack) <= kInt32Max - 4096 && tiles_faster(cache, p, pack))
    return launch_tiles(cache, p, pack, stream, row_dtype);
  return launch_rows(cache, p, stream, row_dtype);
}

pa::WindowParams base_params(const pa_cache_desc* cache, void* out, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* block_tables, const int32_t* seq_lens,
                             int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks, float scale, int32_t window,
                             int32_t num_sinks, int32_t* err_flag) {
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
  p.k_scale = p.v_scale = 1.f;
  return p;
}

}  // namespace

namespace pa {

// With a workspace, are the slabs dealt out evenly?  Where an item is long and there are many of them: 128 items of 4096
// tokens 31 us in clusters and 27 dealt out, of 20000 134 and 76 (contexts of 1250 to 20000: 116 and 45); 32 of 4096 10.8
// and 14.4, of 20000 27 both; one of 80000 38 and 18; 1024 of 1000 45 and 49.  Not where a window shorter than half of what
// the table holds makes items nearly equal and lets many start far from their sequence's: those run as well in one
// launch.  (The lengths themselves are on the device: short ones in a wide table cost a dealt out call 9 to 20 us for 6 to
// 14.)  ALiBi: only the clusters' kernel.
bool fp4_deals_evenly(const pa_cache_desc* cache, const WindowParams& p) {
  const long long cap = (long long)p.max_blocks * cache->block_size, reach = (long long)p.window + p.sinks;
  const long long keys = std::min(cap, reach), group = p.num_q_heads / p.num_kv_heads;
  const long long items = (long long)p.num_seqs * p.num_kv_heads * ((group + 7) / 8);
  return p.alibi == nullptr && 2 * reach >= cap && (keys >= 32768 || (keys >= 2048 && items * keys >= 300000));
}

int fp4_decode(const pa_cache_desc* cache, int32_t row_dtype, WindowParams& p, float* workspace, cudaStream_t stream) {
  if (workspace == nullptr || !fp4_deals_evenly(cache, p)) return launch_rows(cache, p, stream, row_dtype);
  return launch_fp4_even(row_dtype, p, workspace, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int fp4_chunk(const pa_cache_desc* cache, int32_t row_dtype, WindowParams& p, cudaStream_t stream) {
  return launch_chunk(cache, p, stream, row_dtype);
}

}  // namespace pa

extern "C" {

int pa_decode_window(void* out, const void* q, void* k_cache, void* v_cache, const void* key, const void* value,
                     const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                     int32_t max_blocks_per_seq, const pa_cache_desc* cache, float scale, int32_t window,
                     int32_t num_sinks, int32_t* err_flag, void* stream, const pa_decode_options* options) {
  int rc = check_window(cache, num_seqs, num_q_heads, max_blocks_per_seq, scale, window, num_sinks);
  if (rc != PA_OK) return rc;
  if ((key == nullptr) != (value == nullptr)) return PA_ERR_NULL_POINTER;
  if (key != nullptr && cache->dtype == PA_F32) return PA_ERR_UNSUPPORTED;  // the 16-bit and FP8 kernels append
  float k_scale = options != nullptr ? options->k_scale : 0.f, v_scale = options != nullptr ? options->v_scale : 0.f;
  rc = check_scales(cache, &k_scale, &v_scale);
  if (rc != PA_OK) return rc;
  if (num_seqs == 0) return PA_OK;
  if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr || seq_lens == nullptr)
    return PA_ERR_NULL_POINTER;
  if (block_tables == nullptr && max_blocks_per_seq > 0) return PA_ERR_NULL_POINTER;
  const uintptr_t qalign = cache->dtype == PA_F32 ? 4 : 16;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, qalign) || !aligned(out, 4) ||
      !aligned(key, 16) || !aligned(value, 16) || !aligned(seq_lens, 4) || !aligned(block_tables, 4))
    return PA_ERR_MISALIGNED;
  const float* alibi = options != nullptr ? options->alibi_slopes : nullptr;
  if (!aligned(alibi, 4)) return PA_ERR_MISALIGNED;
  if ((int64_t)num_seqs * num_q_heads > kInt32Max) return PA_ERR_TOO_LARGE;

  pa::WindowParams p = base_params(cache, out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_q_heads,
                                   max_blocks_per_seq, scale, window, num_sinks, err_flag);
  p.alibi = alibi;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.test_expire_first_wait =
      (options != nullptr && (options->test_flags & PA_DECODE_TEST_EXPIRE_FIRST_WAIT) != 0u) ? 1 : 0;
  p.new_k = key;
  p.new_v = value;
  p.k_cache_out = k_cache;
  p.v_cache_out = v_cache;
  return launch_rows(cache, p, static_cast<cudaStream_t>(stream));
}

int pa_prefill_window(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* query_start, int32_t num_seqs,
                      int32_t num_query_tokens, int32_t num_q_heads, int32_t max_blocks_per_seq,
                      int32_t max_query_len, const pa_cache_desc* cache, float scale, int32_t window,
                      int32_t num_sinks, float k_scale, float v_scale, int32_t* err_flag, void* stream) {
  int rc = check_window(cache, num_seqs, num_q_heads, max_blocks_per_seq, scale, window, num_sinks);
  if (rc != PA_OK) return rc;
  if (num_query_tokens < 0 || max_query_len < 0 || !(scale > 0.f)) return PA_ERR_INVALID_ARG;
  rc = check_scales(cache, &k_scale, &v_scale);
  if (rc != PA_OK) return rc;
  if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return PA_OK;
  if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr || seq_lens == nullptr ||
      query_start == nullptr || block_tables == nullptr)
    return PA_ERR_NULL_POINTER;
  const uintptr_t qalign = cache->dtype == PA_F32 ? 4 : 16;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, qalign) || !aligned(out, qalign) ||
      !aligned(seq_lens, 4) || !aligned(query_start, 4) || !aligned(block_tables, 4))
    return PA_ERR_MISALIGNED;
  if ((int64_t)num_query_tokens * num_q_heads * 128 > ((int64_t)1 << 40)) return PA_ERR_TOO_LARGE;

  pa::WindowParams p = base_params(cache, out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_q_heads,
                                   max_blocks_per_seq, scale, window, num_sinks, err_flag);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.query_start = query_start;
  p.num_query_tokens = num_query_tokens;
  p.max_query_len = std::min(max_query_len, num_query_tokens);  // no valid chunk is longer
  return launch_chunk(cache, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
