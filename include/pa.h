/*
 * pa.h - C ABI of the paged decode-attention library (libpa.so) for GB300 (sm_103a).
 *
 * The library implements the decode hot path of PagedAttention: single-query
 * attention over a KV cache held in fixed-size physical blocks reached through
 * per-sequence block tables, the slot-mapping append that writes new K/V into
 * the cache, and the whole-block copy used by copy-on-write.
 *
 * Sources (page title, section):
 *  [P1] "PagedAttention 详解：缓存的存储结构" - "Block Table", "软件地址翻译"
 *       (software address translation), "写入新 K/V" (writing new K/V).
 *  [P2] "PagedAttention 笔记" - "写时复制是正确性的边界" (copy-on-write).
 *  [P3] "vLLM 核心工程深度剖析" - "3.1 Kernel 签名与分块策略" (kernel signature),
 *       "4.1 Beam Search 中的 CoW" (block-level copy).
 *  [P4] "PagedAttention是什麼？" - "PagedAttention Kernel在做什麼？" (grid over
 *       sequence, head and partition; partition reduction for long contexts).
 *
 * Conventions shared by every call
 *  - All data pointers are DEVICE-ACCESSIBLE addresses owned by the caller.  No
 *    call allocates memory.  Between calls the library keeps only a lazily
 *    resolved driver entry point, per-kernel launch attributes and, for
 *    pa_decode_noalloc alone, one fixed scratch array per device (see there).
 *  - The K/V caches, the workspace and err_flag must be device memory (the
 *    caches are read by tensor-map copies).  For the decode calls, the appends
 *    and pa_copy_blocks, the small per-step arrays (q, out, block_tables,
 *    seq_lens, slot_mapping, new key/value, block_pairs, ALiBi slopes) may
 *    instead be pinned host memory mapped into the device's address space, as
 *    every cudaHostAlloc / cudaMallocHost allocation is under unified
 *    addressing: the kernels then read and write them in place over the host
 *    link (NVLink-C2C on GB300), with no copy in between, and the results are
 *    the same bytes as with device buffers.  pa_prefill and pa_prefill_window move q and out by
 *    tensor-map copies: those two must be device memory there.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Every call is asynchronous on that stream.
 *  - Cache layout (both K and V): [num_blocks][num_kv_heads][block_size][head_size],
 *    dense, element type `dtype`.  One (block, kv head) is one contiguous run of
 *    block_size * head_size elements.
 *  - Return value: PA_OK, or a PA_ERR_* code for an argument error detected on
 *    the host, in which case NOTHING is launched; PA_ERR_CUDA if a launch failed.
 *  - Data errors (a bad block ID or slot inside device arrays) are detected on
 *    the device, always: there is no switch that turns the checks off (each is
 *    one integer compare per block or slot, next to a memory access).  The
 *    offending item is skipped (never read or written out of bounds); if
 *    `err_flag` is non-NULL the first error code (PA_DEVERR_*) is stored there
 *    with an atomic compare-and-swap from 0.  `err_flag` is a device int32 the
 *    caller zeroes.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PA_F32 = 0, PA_F16 = 1, PA_BF16 = 2, PA_FP8_E4M3 = 3, PA_FP4_E2M1 = 4 } pa_dtype;

/* Shape of one layer's KV cache pair. */
typedef struct {
  int32_t num_blocks;   /* physical blocks in the pool */
  int32_t block_size;   /* tokens per block B: f16/bf16 8 or a multiple of 16 (<= 256); fp8, fp4 a multiple of 16
                           (<= 256); f32 any B >= 1 */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_size;    /* D: 64 or 128 (fp8, fp4: 128) */
  int32_t dtype;        /* pa_dtype of the cache, and of q/out and new key/value except for fp8, fp4 (see below) */
} pa_cache_desc;

/*
 * FP8 caches (dtype PA_FP8_E4M3).  ["PagedAttention 详解：缓存的存储结构"
 * "软件地址翻译": cache_t may be FP8, x = 16 / sizeof(cache_t) = 16 elements per
 * 16-byte access.]  The pages define nothing further; the reading implemented:
 *   - elements are OCP E4M3 codes (1 sign, 4 exponent bits with bias 7, 3
 *     mantissa bits; S.1111.111 is NaN; no infinities);
 *   - one fp32 scale per cache: a key code c stands for k_scale * e4m3(c), a
 *     value code for v_scale * e4m3(c) (scales > 0, passed per call);
 *   - keys   [num_blocks][num_kv_heads][block_size][head_size] bytes,
 *     values [num_blocks][num_kv_heads][block_size/16][head_size][16] bytes:
 *     the pages' value layout ([head_size][block_size], a dimension's tokens
 *     contiguous) tiled in 16-token groups, identical to it for block_size 16,
 *     so that the values of every 16 tokens of one head are contiguous;
 *   - q, out and the key/value rows written by pa_reshape_and_cache_fp8 are fp16;
 *   - written codes are the E4M3 code nearest to x / scale (fp32 division,
 *     ties to even; magnitudes past 448, infinities included, saturate to 448).
 */

/*
 * FP4 caches (dtype PA_FP4_E2M1): 4 bits an element and a scale for every 16, 72 bytes a row of 128.
 *   - a group is 16 neighbouring elements x of a row.  Its scale is s = e4m3(max |x| / (6 u)), u the cache's unit
 *     (k_scale or v_scale, one fp32 number per cache, passed per call, 2^-100 .. 2^100), ties to even, at most 448;
 *   - an element is held as the OCP E2M1 code (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6)
 *     nearest to x * (1 / (s u)), ties to even, magnitudes past 6 as 6; it stands for e2m1 * s * u.  6 u, the quotient,
 *     s u, its inverse and the product are single fp32 operations.  A group whose scale is 0 holds zeros.  Rows should be
 *     finite: an infinity becomes the largest number that the cache holds, a NaN some finite one;
 *   - keys and values alike are [num_blocks][num_kv_heads][block_size / 16][1152] bytes: of 16 tokens [16][64] bytes of
 *     codes (dimension 2 i in the low half of byte i, 2 i + 1 in the high one), then [16][8] bytes of scales;
 *   - q, out and new key/value rows are fp16 or bf16, as the calls' row_dtype says.
 * They are taken by pa_reshape_and_cache_fp4, pa_read_cache_fp4, pa_decode_fp4, pa_prefill_fp4, pa_rope_axes_and_cache
 * and pa_copy_blocks; the other calls return PA_ERR_UNSUPPORTED.
 */

/* Host-side status codes. */
enum {
  PA_OK = 0,
  PA_ERR_NULL_POINTER = 1, /* a required pointer is NULL */
  PA_ERR_UNSUPPORTED = 2,  /* dtype / head_size / block_size combination not built */
  PA_ERR_INVALID_ARG = 3,  /* negative size, Hq % Hkv != 0, bad partition size, ... */
  PA_ERR_WORKSPACE = 4,    /* workspace NULL or smaller than pa_decode_workspace_size() */
  PA_ERR_MISALIGNED = 5,   /* a pointer is not aligned as documented */
  PA_ERR_CUDA = 6,         /* a CUDA runtime call or kernel launch failed */
  PA_ERR_TOO_LARGE = 7     /* sizes exceed the index ranges the kernels use */
};

/* Device-side data error codes written to *err_flag. */
enum {
  PA_DEVERR_NONE = 0,
  PA_DEVERR_BLOCK_ID = 1, /* a block_tables entry outside [0, num_blocks) */
  PA_DEVERR_SLOT = 2,     /* a slot_mapping entry >= num_blocks * block_size */
  PA_DEVERR_PAIR = 3,     /* a copy pair with an ID outside [0, num_blocks) */
  PA_DEVERR_TIMEOUT = 4,  /* a bounded wait on an asynchronous copy expired */
  PA_DEVERR_QUERY = 5,    /* pa_prefill: a chunk outside [0, num_query_tokens), longer than
                             max_query_len or than its sequence, or a sequence past its table */
  PA_DEVERR_TABLES = 6,   /* pa_tables_*: lengths, blocks held or tokens wanted that do not fit together */
  PA_DEVERR_NO_BLOCKS = 7 /* pa_tables_extend: more blocks needed than are free */
};

/*
 * pa_decode - one decode step of paged attention for one layer.
 *   [P3 "3.1"] signature: out/q [num_seqs, num_heads, head_size], block_tables
 *   [num_seqs, max_blocks_per_seq], context lengths, scale.
 *   [P1 "软件地址翻译"] token i of sequence s lives at offset i % B of block
 *   block_tables[s][i / B].
 *
 *   out[s][h][:] = sum_i softmax_i(scale * q[s][h] . k_i) * v_i over the
 *   seq_lens[s] tokens of sequence s, where k_i, v_i are the K/V rows of kv head
 *   h / (num_q_heads / num_kv_heads) (consecutive query heads share a kv head).
 *   Accumulation is in fp32; out is rounded to `dtype` round-to-nearest-even.
 *   seq_lens[s] == 0 writes a zero row.  Table entries at or beyond
 *   ceil(seq_lens[s] / B) are never read.
 *
 *   out          [num_seqs][num_q_heads][head_size] of dtype (written)
 *   q            [num_seqs][num_q_heads][head_size] of dtype, 16-byte aligned (f32: 4)
 *   k_cache, v_cache  cache pair (layout above), 16-byte aligned
 *   block_tables int32 [num_seqs][max_blocks_per_seq], row-major
 *   seq_lens     int32 [num_seqs]; each <= max_blocks_per_seq * block_size (not checked
 *                on the device beyond the table width: longer values are clamped)
 *   scale        softmax scale (usually 1/sqrt(head_size))
 *   partition_size  0 = library default (1024 tokens); else tokens per partition, a
 *                multiple of block_size and, for f16/bf16/fp8 caches, of 16 (the
 *                kernels' 16-token slabs never straddle a partition).  Sequences longer
 *                than one partition are split across CTAs and merged with a
 *                log-sum-exp reduction [P4 "PagedAttention Kernel在做什麼？"].
 *   workspace    device scratch of at least pa_decode_workspace_size(...) bytes,
 *                256-byte aligned; may be NULL when that size is 0.  Its
 *                contents on entry do not matter.
 *   err_flag     nullable device int32 (see above).
 *   Launches: the decode kernel, then (when a sequence spans two partitions) the
 *   merge kernel, both with programmatic stream serialization.  Their CTAs may be
 *   scheduled while the kernel before them on `stream` finishes.  They read
 *   seq_lens and block_tables at once, and execute griddepcontrol.wait before
 *   they read anything else (q, the caches, key/value, the workspace) or write
 *   anything, so stream order holds as for a plain launch provided that those
 *   two inputs are not written by a kernel that lets its dependents start
 *   early (of this library only pa_tables_extend and pa_tables_trim write them, and
 *   let none start early; copies, and kernels that do
 *   not execute griddepcontrol.launch_dependents, complete first).  Stream
 *   capture records the dependencies as programmatic edges.
 */
int pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
              const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
              const pa_cache_desc* cache, float scale, int32_t partition_size, void* workspace,
              size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * pa_decode_ex - pa_decode with optional extensions (options may be NULL, which
 * is exactly pa_decode).
 *   alibi_slopes  nullable device fp32 [num_q_heads], 4-byte aligned.  The kernel
 *                 signature of [P3 "3.1"] carries per-head ALiBi slopes without
 *                 defining them; the reading implemented is the standard linear
 *                 bias towards the query's own position: score_i of head h gains
 *                 alibi_slopes[h] * (i - (seq_lens[s] - 1)).
 *   k_scale, v_scale  the dequantisation scales of an FP8 cache (pa_decode uses 1).
 *   test_flags    0 in normal use.  PA_DECODE_TEST_EXPIRE_FIRST_WAIT exists for
 *                 tests of the kernels' hang protection (every wait on an
 *                 asynchronous copy is bounded, and an expired wait ends the
 *                 work item with PA_DEVERR_TIMEOUT once the copies already in
 *                 flight have landed): the f16/bf16/fp8 kernels then never
 *                 request the first slab of each warp's ring and bound the wait
 *                 for it at 20000 cycles, so it expires.  The call reports
 *                 PA_DEVERR_TIMEOUT in *err_flag and its output is undefined;
 *                 later calls are unaffected.  Ignored for fp32 caches, which
 *                 do not wait.
 */
#define PA_DECODE_TEST_EXPIRE_FIRST_WAIT 1u
typedef struct {
  const float* alibi_slopes;
  float k_scale; /* FP8 caches only (> 0); 0 means 1.  Ignored for other dtypes. */
  float v_scale; /* FP8 caches only (> 0); 0 means 1.  Ignored for other dtypes. */
  uint32_t test_flags; /* 0, or PA_DECODE_TEST_EXPIRE_FIRST_WAIT (tests only) */
} pa_decode_options;

int pa_decode_ex(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                 const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
                 const pa_cache_desc* cache, float scale, int32_t partition_size, void* workspace,
                 size_t workspace_bytes, int32_t* err_flag, void* stream, const pa_decode_options* options);

/*
 * pa_decode_append - one decode step with its append fused in: for every
 *   sequence s with seq_lens[s] = L > 0, the new token's key[s][h][:] and
 *   value[s][h][:] are stored at position L - 1 of both caches, i.e. at
 *   offset (L - 1) % B of block block_tables[s][(L - 1) / B]
 *   [P1 "写入新 K/V": slot = block * B + offset], and out is pa_decode's over
 *   positions 0 .. L - 1, the new token included.  The result and the cache
 *   contents equal pa_reshape_and_cache with those slots followed by pa_decode,
 *   in one launch (plus the merge when a sequence spans two partitions): the
 *   CTA that streams the new token's slab takes the token's rows from key and
 *   value, and the first query-head group of each kv head stores them.
 *
 *   key, value   [num_seqs][num_kv_heads][head_size] of dtype (fp16 for an FP8 cache),
 *                16-byte aligned
 *   options      nullable, as for pa_decode_ex (ALiBi slopes, FP8 scales)
 *   other arguments as for pa_decode; f16, bf16 and FP8 caches (fp32: use
 *   pa_reshape_and_cache and pa_decode).  Over an FP8 cache the rows are
 *   quantised as pa_reshape_and_cache_fp8 does (code of x / scale, fp32
 *   division, ties to even, saturating at +-448), bit for bit.  The slot at
 *   position L - 1 must belong to this sequence alone (the block manager copies
 *   a shared partial block on write first); a sequence's other slots are not
 *   written.
 */
int pa_decode_append(void* out, const void* q, void* k_cache, void* v_cache, const void* key, const void* value,
                     const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                     int32_t max_blocks_per_seq, const pa_cache_desc* cache, float scale, int32_t partition_size,
                     void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream,
                     const pa_decode_options* options);

/* Partition size pa_decode uses for these arguments (resolves 0 to the default);
 * returns a value >= max_blocks_per_seq * block_size when no split happens, or a
 * negative PA_ERR_* code for invalid arguments. */
int32_t pa_decode_partition_size(int32_t max_blocks_per_seq, const pa_cache_desc* cache, int32_t partition_size);

/* Bytes of workspace pa_decode needs: (head_size + 2) * 4 bytes (fp32 partial output,
 * maximum and sum) per row (sequence, query head) and partition slot, each part padded
 * to 256 bytes.  A row has P_max = ceil(max_blocks_per_seq * block_size / partition)
 * slots; on the fp16/bf16/FP8 kernels, when 2 <= P_max <= 8, the last num_seqs / 12
 * (fp16/bf16) or num_seqs / 24 (FP8) sequences (the grid's last items) are split into
 * partitions of half the size, if that half is a multiple of block_size and of 32,
 * and their rows have 2 P_max slots.  0 when no sequence can span two partitions.  Returns
 * 0 for invalid arguments as well (pa_decode then reports the argument error). */
size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                const pa_cache_desc* cache, int32_t partition_size);

/*
 * pa_prefill - chunked prefill attention over the paged cache.
 *   ["PagedAttention 详解：缓存的存储结构" "使用流程": prompt blocks that hit the
 *   prefix cache take part in attention directly, only missed blocks are
 *   computed and written through slot_mapping; "vLLM 核心工程深度剖析" "6.1":
 *   long prompts are prefilled in chunks.]
 *   Sequence s holds seq_lens[s] = L tokens in the cache (the chunk's own K/V
 *   already written, e.g. by pa_reshape_and_cache), the last
 *   n = query_start[s+1] - query_start[s] of which are this chunk's queries.
 *   Query j of head h (position L - n + j) attends causally to cache positions
 *   0 .. L - n + j: out = softmax_i(scale * q . k_i) v_i, fp32 accumulation,
 *   out rounded to dtype.
 *
 *   out, q           [num_query_tokens][num_q_heads][head_size], 16-byte aligned;
 *                    out rows outside every chunk are not written
 *   query_start      int32 [num_seqs + 1] on the device: chunk s is rows
 *                    query_start[s] .. query_start[s+1] - 1
 *   seq_lens         int32 [num_seqs], n <= L <= max_blocks_per_seq * block_size
 *   max_query_len    upper bound on n over the sequences (sizes the grid)
 *   scale            finite and > 0 (the softmax scale, e.g. 1/sqrt(head_size))
 *   A sequence whose chunk breaks these rules is skipped and PA_DEVERR_QUERY is
 *   reported; a bad block ID gives PA_DEVERR_BLOCK_ID and that sequence's
 *   output is undefined.
 *   Supported: dtype f16 / bf16, head_size 128, block_size 8, 16, 32, 64 or 128.
 *   Runs on the tcgen05 tensor cores: a persistent kernel, one CTA per SM,
 *   whose CTAs walk the work items (sequence, query head, tile of 128 queries).
 */
int pa_prefill(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
               const int32_t* seq_lens, const int32_t* query_start, int32_t num_seqs, int32_t num_query_tokens,
               int32_t num_q_heads, int32_t max_blocks_per_seq, int32_t max_query_len, const pa_cache_desc* cache,
               float scale, int32_t* err_flag, void* stream);

/*
 * pa_reshape_and_cache - append new tokens' K/V through slot_mapping.
 *   [P1 "写入新 K/V"] slot = block_id * B + offset; the kernel decodes
 *   block_id = slot / B, offset = slot % B and stores key[t][h][:] and
 *   value[t][h][:] at (block_id, h, offset) of k_cache / v_cache.
 *   A negative slot marks a padding token and is skipped.
 *
 *   key, value   [num_tokens][num_kv_heads][head_size] of dtype, dense, 16-byte aligned
 *   slot_mapping int64 [num_tokens]
 *   Slots must be distinct (two tokens with one slot race; either may win).
 */
int pa_reshape_and_cache(void* k_cache, void* v_cache, const void* key, const void* value,
                         const int64_t* slot_mapping, int32_t num_tokens, const pa_cache_desc* cache,
                         int32_t* err_flag, void* stream);

/*
 * pa_reshape_and_cache_fp8 - the append for an FP8 cache (dtype PA_FP8_E4M3):
 *   fp16 key/value [num_tokens][num_kv_heads][head_size] (16-byte aligned) are
 *   written as E4M3 codes of x / k_scale and x / v_scale (see "FP8 caches"
 *   above): key[t][h][d] at (block, h, offset, d), value[t][h][d] at (block, h,
 *   offset / 16, d, offset % 16).  Slots as for pa_reshape_and_cache.
 *   k_scale, v_scale > 0.
 */
int pa_reshape_and_cache_fp8(void* k_cache, void* v_cache, const void* key, const void* value,
                             const int64_t* slot_mapping, int32_t num_tokens, const pa_cache_desc* cache,
                             float k_scale, float v_scale, int32_t* err_flag, void* stream);

/*
 * pa_copy_blocks - the copy step of copy-on-write [P2 "写时复制是正确性的边界";
 *   P3 "4.1"]: for every pair, the whole physical block dst of both caches
 *   (all kv heads, all slots) becomes a copy of block src.
 *
 *   block_pairs  int32 [num_pairs][2] = (src, dst)
 *   Precondition: no dst appears twice and no dst is also a src (the pairs are
 *   copied concurrently).  A pair with src == dst is a no-op.
 */
int pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* block_pairs, int32_t num_pairs,
                   const pa_cache_desc* cache, int32_t* err_flag, void* stream);

/*
 * pa_decode_noalloc - pa_decode for callers that cannot allocate device memory
 *   while they decode (for example a serving plugin whose host engine owns all
 *   device memory, or a decode loop that must stay out of the CUDA allocator).
 *   The pages have no counterpart: this is a deployment convenience.
 *
 *   Same arguments and results as pa_decode, without workspace: the split-KV
 *   scratch is a library-owned device array of PA_NOALLOC_MAX_WORKSPACE_BYTES
 *   bytes.  Sizes whose pa_decode_workspace_size() exceeds that limit return
 *   PA_ERR_WORKSPACE and launch nothing.  The call itself allocates nothing.
 *   - Which sizes fit: the workspace is about num_seqs * num_q_heads * P_max *
 *     (head_size + 2) * 4 bytes (pa_decode_workspace_size gives it exactly).
 *     At the default 1024-token partition, 64 sequences x 32 heads of up to
 *     2048 tokens need 2.3 MB and 128 x 32 heads of up to 1280 tokens 4.6 MB;
 *     8 sequences x 32 heads of 32768 tokens in 512-token partitions need
 *     8.5 MB.  128 sequences x 64 query heads of up to 4096 tokens need 18.4 MB,
 *     over the limit: pass partition_size 2048 (9.2 MB) for them.  Sequences
 *     that fit one partition need none.
 *   - The first call on a device, whatever its sizes, looks up the array's
 *     device address with that device current and caches it.  Under CUDA's lazy
 *     module loading (the default) that lookup is also when the array is
 *     committed on the device, where it then stays until the process exits.
 *     Make that first call before any stream capture and outside any
 *     latency-critical loop.  It returns PA_ERR_CUDA if the lookup fails.
 *   - All calls share the one array and it keeps the previous call's contents;
 *     nothing in it needs clearing, but calls that overlap on the GPU (other
 *     streams, other host threads) race on it: order them on one stream.
 */
#define PA_NOALLOC_MAX_WORKSPACE_BYTES ((size_t)16 << 20)
int pa_decode_noalloc(void* out, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                      int32_t max_blocks_per_seq, const pa_cache_desc* cache, float scale, int32_t partition_size,
                      int32_t* err_flag, void* stream);

/*
 * pa_rope_frequencies - the angle per position of each rotary pair (host; no CUDA call).
 *   Pair j < rotary_dim / 2 of a head turns by position * inv_freq[j] radians, inv_freq[j] =
 *   base^(-2 j / rotary_dim), stretched for contexts longer than the trained one by `scaling`:
 *     PA_ROPE_PLAIN   as is (scaling NULL is the same)
 *     PA_ROPE_LINEAR  inv_freq / factor (positions interpolated)
 *     PA_ROPE_NTK     base * factor^(r / (r - 2)), r = rotary_dim >= 4
 *     PA_ROPE_YARN    inv_freq / factor * ramp_j + inv_freq * (1 - ramp_j), ramp_j = clamp((j - lo) / (hi - lo), 0, 1),
 *                     lo = max(0, floor(d(beta_fast))), hi = min(r - 1, ceil(d(beta_slow))),
 *                     d(n) = r ln(original_max_position / (2 pi n)) / (2 ln base), hi - lo at least 1e-3;
 *                     *magnitude = attention_factor, or if that is 0: 0.1 ln(factor) + 1 (1 for factor <= 1)
 *     PA_ROPE_BANDS   by the turns n_j = original_max_position * inv_freq / (2 pi) of the trained length:
 *                     inv_freq / factor * (1 - keep_j) + inv_freq * keep_j,
 *                     keep_j = clamp((n_j - low_freq_factor) / (high_freq_factor - low_freq_factor), 0, 1)
 *   *magnitude is 1 except for PA_ROPE_YARN.  rotary_dim even, 2 .. 128; base, and the fields that the
 *   method names, finite and > 0 (attention_factor >= 0, high_freq_factor > low_freq_factor), such that the
 *   frequencies and the magnitude are finite; otherwise PA_ERR_INVALID_ARG, and inv_freq holds nothing of use.
 */
enum { PA_ROPE_PLAIN = 0, PA_ROPE_LINEAR = 1, PA_ROPE_NTK = 2, PA_ROPE_YARN = 3, PA_ROPE_BANDS = 4 };
typedef struct {
  int32_t method;               /* PA_ROPE_* */
  double factor;
  double original_max_position; /* YARN, BANDS */
  double beta_fast, beta_slow;  /* YARN (usually 32, 1) */
  double attention_factor;      /* YARN; 0: from factor */
  double low_freq_factor, high_freq_factor; /* BANDS (usually 1, 4) */
} pa_rope_scaling;

int pa_rope_frequencies(double* inv_freq, float* magnitude, int32_t rotary_dim, double base,
                        const pa_rope_scaling* scaling);

/*
 * pa_rope_and_cache - rotary positions applied to a step's new tokens, with their cache write, in one pass:
 *   the first rotary_dim elements of every head of q and key are turned,
 *     y_a = c x_a - s x_b,  y_b = c x_b + s x_a,  c = magnitude cos(a_j), s = magnitude sin(a_j),
 *     a_j = positions[t] * inv_freq[j],
 *   pairs (a, b) = (j, j + rotary_dim / 2), or (2j, 2j + 1) when `interleaved`; the other elements are copied.
 *   Turned queries go to q_out; turned keys, and values as they are, go to the token's slot of the caches as
 *   pa_reshape_and_cache / pa_reshape_and_cache_fp8 place them.  The angle is reduced to a fraction of a turn
 *   exactly (any int32 position), the rest is fp32, and each element is rounded once: to dtype, or over an FP8
 *   cache to the E4M3 code nearest to y / k_scale (x / v_scale), ties to even, saturating at +-448.
 *
 *   q, q_out     [num_tokens][num_q_heads][head_size] of dtype (fp16 for an FP8 cache); num_q_heads 0: no queries
 *   key, value   [num_tokens][num_kv_heads][head_size] of the same type
 *   *_stride     elements from one token to the next: at least the row of its heads, a multiple of 16 bytes
 *                (views of a fused projection); all four pointers 16-byte aligned
 *   q_out        q itself (same stride: in place), or apart from q, key and value
 *   positions    int32 [num_tokens];  inv_freq  double [rotary_dim / 2] on the device, finite
 *   slot_mapping int64 [num_tokens], distinct.  A negative slot marks a padding token: nothing of it is written,
 *                its row of q_out included.  A slot outside the pool gives PA_DEVERR_SLOT, and that token is
 *                skipped in the same way.
 *   k_scale, v_scale  FP8 caches (> 0; 0 means 1).  magnitude finite.
 *   The inputs may be pinned host memory mapped into the device's address space, as for the other appends.
 */
int pa_rope_and_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* key, const void* value,
                      int64_t q_out_stride, int64_t q_stride, int64_t key_stride, int64_t value_stride,
                      const int32_t* positions, const int64_t* slot_mapping, const double* inv_freq,
                      int32_t num_tokens, int32_t num_q_heads, int32_t rotary_dim, int32_t interleaved,
                      float magnitude, const pa_cache_desc* cache, float k_scale, float v_scale, int32_t* err_flag,
                      void* stream);

/*
 * pa_decode_window - one decode step with a sliding window and first tokens that stay visible: pa_decode
 *   where the query of sequence s, at position p = seq_lens[s] - 1, sees only the positions
 *     i <= p  with  i > p - window  or  i < num_sinks.
 *   A window no shorter than the sequence sees all of it.  Table entries of blocks that hold no visible
 *   position are never read and their blocks never touched: they may have been released.  Other positions of
 *   a block that holds a visible one are loaded and have no effect, whatever they contain.  A NaN in a query or
 *   in a key that it sees makes the whole row NaN (pa_decode: zeros), one in a value that element of it.
 *
 *   key, value   both NULL, or the step's append as in pa_decode_append (f16, bf16, FP8 caches): each
 *                sequence's new token is stored at position seq_lens[s] - 1 and attended in the same launch
 *   seq_lens     0 writes a zero row (and appends nothing).  A length past the table, or a negative one, gives
 *                PA_DEVERR_QUERY and nothing of that sequence is written.
 *   window >= 1, num_sinks >= 0.  Types, head sizes, block sizes, alignments and options as for pa_decode_ex
 *   (ALiBi slopes, FP8 scales, test_flags); caches, tables and lengths of any block size it takes.
 *   One launch, no workspace: a window bounds an item's keys, which the CTAs of one cluster share.  Two calls
 *   may overlap.  The kernel is a programmatic dependent of the one before it on `stream`; it reads nothing
 *   before that one has finished.
 */
int pa_decode_window(void* out, const void* q, void* k_cache, void* v_cache, const void* key, const void* value,
                     const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                     int32_t max_blocks_per_seq, const pa_cache_desc* cache, float scale, int32_t window,
                     int32_t num_sinks, int32_t* err_flag, void* stream, const pa_decode_options* options);

/*
 * pa_prefill_window - attention of a chunk of new tokens over the paged cache, with the window and first
 *   tokens of pa_decode_window: query j of sequence s, at position p = L - n + j, sees the positions i <= p
 *   with i > p - window or i < num_sinks.  The chunk's own K/V are in the cache already (pa_rope_and_cache,
 *   pa_reshape_and_cache).  Chunks of one token (a decode step) to whole prompts, and any mixture of them.
 *   (Many single tokens beside long chunks run faster as two calls, theirs to pa_decode_window: 1023 and a
 *   prompt of 4096, 64 / 8 heads, window 1024, bf16: 0.66 ms for 1.62.)
 *
 *   out, q, query_start, seq_lens, max_query_len  as for pa_prefill; query_start does not fall; out rows
 *                outside every chunk are not written.  A sequence whose chunk breaks the rules there is
 *                skipped (PA_DEVERR_QUERY).
 *   Table entries of blocks without a position that some query of the chunk sees are never read (they may
 *   have been released).  Value rows of positions that some queries of the chunk see and others do not must
 *   be finite.  NaN queries and keys as for pa_decode_window: only the rows that see them become NaN.
 *   scale        finite and > 0;  window >= 1;  num_sinks >= 0
 *   k_scale, v_scale  FP8 caches (> 0; 0 means 1): q and out are fp16.  Ignored for other caches.
 *   Every cache type, head size and block size of pa_decode.  No workspace.  Prompts are fast where the block
 *   size divides 128 (8 to 128; 16-bit and FP8 caches); others, and fp32, take the kernels for few queries,
 *   which read the keys again for every eight rows (a chunk of 4096, window 4096, 32 / 8 heads, fp16: blocks
 *   of 16 0.23 ms, of 48 or 256 2.5 ms).
 *   Softmax weights enter the value product as fp32 numbers over fp32 caches; as two bf16 terms (16 bits or
 *   more) over bf16; as one fp16 term, off by at most 2^-11 of a weight or 2^-25 of the row's largest, over FP8
 *   (pa_decode_window too) and for longer chunks over fp16, where few queries get two.
 */
int pa_prefill_window(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* query_start, int32_t num_seqs,
                      int32_t num_query_tokens, int32_t num_q_heads, int32_t max_blocks_per_seq,
                      int32_t max_query_len, const pa_cache_desc* cache, float scale, int32_t window,
                      int32_t num_sinks, float k_scale, float v_scale, int32_t* err_flag, void* stream);

/*
 * pa_reshape_and_cache_fp4 - the append for an FP4 cache (see "FP4 caches" above): key[t][h][:] and value[t][h][:] go to
 *   the slot of token t.  A slot's bytes are its own: no write touches another token's.
 *
 *   key, value   [num_tokens][num_kv_heads][128] of row_dtype (PA_F16, PA_BF16), *_stride elements from one token to
 *                the next (at least the row of its heads, a multiple of 8), 16-byte aligned
 *   slot_mapping int64 [num_tokens], as for pa_reshape_and_cache
 */
int pa_reshape_and_cache_fp4(void* k_cache, void* v_cache, const void* key, const void* value, int64_t key_stride,
                             int64_t value_stride, const int64_t* slot_mapping, int32_t num_tokens,
                             const pa_cache_desc* cache, int32_t row_dtype, float k_scale, float v_scale,
                             int32_t* err_flag, void* stream);

/*
 * pa_read_cache_fp4 - the rows that the slots of an FP4 cache hold, back in 16 bits (to move a prefix into another
 *   cache, to look at what was written): e2m1 * s * u, the fp32 product rounded once to row_dtype.  Arguments as for
 *   pa_reshape_and_cache_fp4; rows of negative slots, and of slots outside the pool (PA_DEVERR_SLOT), are not written.
 */
int pa_read_cache_fp4(void* key, void* value, const void* k_cache, const void* v_cache, int64_t key_stride,
                      int64_t value_stride, const int64_t* slot_mapping, int32_t num_tokens, const pa_cache_desc* cache,
                      int32_t row_dtype, float k_scale, float v_scale, int32_t* err_flag, void* stream);

/*
 * pa_decode_fp4, pa_prefill_fp4 - pa_decode_window and pa_prefill_window over an FP4 cache: the same rows, window, first
 *   tokens, append and errors.  window INT32_MAX (any number no smaller than the lengths) is attention over everything.
 *
 *   out, q       of row_dtype (PA_F16, PA_BF16), 16-byte aligned
 *   key, value   pa_decode_fp4: both NULL, or each sequence's new token of row_dtype, [num_seqs][num_kv_heads][128],
 *                stored at position seq_lens[s] - 1 in the bytes that pa_reshape_and_cache_fp4 writes, and attended
 *   alibi_slopes, test_flags  as in pa_decode_options (NULL, 0 in normal use)
 *   workspace    pa_decode_fp4: NULL, or device scratch of pa_decode_fp4_workspace_size(...) bytes, 256-byte aligned, with
 *                which long contexts of very different lengths keep every SM busy to the end (two launches then).  That
 *                size is a few MB, or 0 where these arguments use none (and for invalid ones).  Its contents on entry
 *                do not matter.  Calls that may overlap, and graphs that may be replayed at once, need one each.
 *   Softmax weights enter the value product as one fp16 term, off by at most 2^-11 of itself; weights below 2^-32 of the
 *   row's largest may count as 0.  A bf16 query row goes in as fp16 over a power of two:
 *   what lies more than 2^-14 below its largest element loses bits, by at most 2^-25 of the largest.
 */
int pa_decode_fp4(void* out, const void* q, void* k_cache, void* v_cache, const void* key, const void* value,
                  const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                  int32_t max_blocks_per_seq, const pa_cache_desc* cache, int32_t row_dtype, float scale, int32_t window,
                  int32_t num_sinks, float k_scale, float v_scale, const float* alibi_slopes, uint32_t test_flags,
                  void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);
size_t pa_decode_fp4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                    const pa_cache_desc* cache, int32_t window, int32_t num_sinks);
int pa_prefill_fp4(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   const int32_t* seq_lens, const int32_t* query_start, int32_t num_seqs, int32_t num_query_tokens,
                   int32_t num_q_heads, int32_t max_blocks_per_seq, int32_t max_query_len, const pa_cache_desc* cache,
                   int32_t row_dtype, float scale, int32_t window, int32_t num_sinks, float k_scale, float v_scale,
                   int32_t* err_flag, void* stream);

/*
 * pa_rope_axes_and_cache - pa_rope_and_cache with a position for each of several axes (time, height and width of images
 *   and video beside text): pair j of a token turns by a_j = positions[pair_axis[j]][t] * inv_freq[j].
 *
 *   positions    int32 [num_axes][num_tokens], num_axes 1 .. 4
 *   pair_axis    HOST array of rotary_dim / 2 axis numbers, read during the call (NULL: all axis 0, num_axes 1)
 *   row_dtype    FP4 caches: of q, q_out, key and value (PA_F16, PA_BF16), whose turned keys are rounded to it and then
 *                held as pa_reshape_and_cache_fp4 holds them (k_scale, v_scale the units).  Ignored for other caches.
 *   Everything else as for pa_rope_and_cache.
 */
int pa_rope_axes_and_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* key, const void* value,
                           int64_t q_out_stride, int64_t q_stride, int64_t key_stride, int64_t value_stride,
                           const int32_t* positions, int32_t num_axes, const uint8_t* pair_axis,
                           const int64_t* slot_mapping, const double* inv_freq, int32_t num_tokens, int32_t num_q_heads,
                           int32_t rotary_dim, int32_t interleaved, float magnitude, const pa_cache_desc* cache,
                           int32_t row_dtype, float k_scale, float v_scale, int32_t* err_flag, void* stream);

/*
 * pa_tables_extend, pa_tables_trim - block tables, lengths and slot maps kept on the GPU, for loops that learn a
 *   request's length there (captured steps, verified drafts).  The state, device memory that the caller makes once:
 *
 *   block_tables int32 [num_seqs][max_blocks_per_seq]: entries 0 .. held_blocks[s] - 1 are request s's blocks, its alone
 *   seq_lens     int32 [num_seqs], at most held_blocks[s] * block_size
 *   held_blocks  int32 [num_seqs]
 *   free_blocks  int32 [num_blocks]: entries 0 .. *num_free - 1 are a stack of the blocks that no request holds
 *   num_free     int32 [1]
 *
 *   pa_tables_extend gives request s new_tokens[s] >= 0 more tokens and the blocks that they need beyond those held
 *   (from the top of the stack; requests in order, a request's blocks in order), and writes, of the Q_s + j-th row, for
 *   its j-th new token (Q_s: the new tokens of the requests before):
 *     slot_mapping int64 [num_rows], its slot; positions int32 [num_rows], its position;
 *     query_start  int32 [num_seqs + 1], Q_s, and their sum at the end (without requests: one 0; with neither requests
 *     nor rows it may be NULL, or num_free, and the call does nothing).
 *   Rows past the sum get slot -1 (padding) and position 0.
 *   pa_tables_trim keeps the first keep_lens[s] <= seq_lens[s] tokens of request s: the blocks past them go back, their
 *   table entries become -1.  The first request's first such block comes out on top of the stack.  0 ends a request.
 *
 *   All or nothing: a request whose numbers do not fit (a negative one, more tokens than its table or than its blocks
 *   hold, more kept than there are, more rows than num_rows, a stack that does not fit) gives PA_DEVERR_TABLES, too few
 *   free blocks PA_DEVERR_NO_BLOCKS, and nothing of the state changes; extend then writes padding rows and zeros in
 *   query_start.  A block outside the pool gives PA_DEVERR_BLOCK_ID: extend's rows for it are padding,
 *   trim puts it back on the stack as it is.
 *   num_seqs <= 16384.  The arrays do not overlap.  Two calls on one state are ordered by the caller, on one stream.
 */
int pa_tables_extend(int32_t* block_tables, int32_t* seq_lens, int32_t* held_blocks, const int32_t* free_blocks,
                     int32_t* num_free, const int32_t* new_tokens, int64_t* slot_mapping, int32_t* positions,
                     int32_t* query_start, int32_t num_seqs, int32_t num_rows, int32_t max_blocks_per_seq,
                     int32_t block_size, int32_t num_blocks, int32_t* err_flag, void* stream);
int pa_tables_trim(int32_t* block_tables, int32_t* seq_lens, int32_t* held_blocks, int32_t* free_blocks,
                   int32_t* num_free, const int32_t* keep_lens, int32_t num_seqs, int32_t max_blocks_per_seq,
                   int32_t block_size, int32_t num_blocks, int32_t* err_flag, void* stream);

/* Static description of a status code (never NULL). */
const char* pa_status_string(int status);

/* Library ABI version: major * 10000 + minor * 100 + patch. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
