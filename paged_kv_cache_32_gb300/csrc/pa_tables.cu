// pa_tables.cu - block tables and slot maps kept on the GPU: requests grow by new tokens (extend) and fall back to fewer
// (trim), blocks come from and go back to a stack.
//
// With L_s tokens, h_s blocks held and n_s new tokens of request s, extend needs a_s = max(0, ceil((L_s + n_s) / B) - h_s)
// blocks.  Sums over the requests before s, Q_s of n and P_s of a, place everything: new token j of s is row Q_s + j of the
// slot map, its i-th fresh block is entry F - 1 - (P_s + i) of the stack of F blocks.  Trim to k_s tokens releases
// g_s = h_s - ceil(k_s / B) blocks; with sums R_s of g and R of all, its i-th one becomes entry F + R - 1 - (R_s + i), so
// that an extend by as much hands every request its own blocks again.
//
// Bound by latency: a step's requests are a few KB.  Every CTA adds up all requests (each thread a run of them) and keeps
// the sums in shared memory, so that none waits for another before it writes its rows, each of which finds its request
// by bisection.  The lengths, read by all, are written last: after a barrier of the cluster that a small call runs in,
// or by a second kernel.  Neither kernel lets a dependent launch start early: the decode kernels read lengths and tables
// before they wait for the kernel in front of them.
#include <algorithm>

#include "pa.h"
#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"

using namespace pa::host;

namespace pa {
namespace {

// Threads of a CTA: a step's few requests take one small CTA (64 requests of 5 tokens: 3.6 us a call, of 1024 threads 5).
constexpr int kSmall = 256, kLarge = 1024;
constexpr int kKept = 4;              // requests of a thread whose numbers it keeps between the two passes over them
constexpr int kAhead = 4;             // rows of a thread whose loads are in flight together
constexpr int kMaxSeqs = 16384;      // whose sums fit shared memory
constexpr int kMaxTablesCluster = 8;

struct TablesParams {
  int32_t* block_tables;     // [N][M]
  int32_t* seq_lens;         // [N]
  int32_t* held;             // [N]
  int32_t* free_blocks;      // [num_blocks], entries 0 .. num_free - 1 the stack
  int32_t* num_free;         // [1]
  const int32_t* wanted;     // [N]: new tokens (extend), tokens kept (trim)
  int64_t* slot_mapping;     // extend: [num_rows]
  int32_t* positions;        // extend: [num_rows]
  int32_t* query_start;      // extend: [N + 1]
  int32_t num_seqs, num_rows, max_blocks, block_size, num_blocks;
  int32_t* err_flag;         // nullable
};

struct Request {
  int len, held, wanted;
  int blocks;  // fresh ones, or released ones
  bool bad;
};

template <bool kTrim>
__device__ __forceinline__ Request request(const TablesParams& p, int s) {
  Request r = {p.seq_lens[s], p.held[s], p.wanted[s], 0, false};
  const int B = p.block_size;
  const long long room = (long long)p.max_blocks * B;
  const long long after = kTrim ? r.wanted : (long long)r.len + r.wanted;
  r.bad = r.len < 0 || r.held < 0 || r.held > p.max_blocks || (long long)r.held * B < r.len || r.wanted < 0 ||
          after > (kTrim ? (long long)r.len : room);
  if (!r.bad) {
    const int need = (int)((after + B - 1) / B);
    r.blocks = kTrim ? r.held - need : max(0, need - r.held);
  }
  return r;
}

// Sums of a call, the same in every CTA.
struct Sums {
  long long rows, blocks;  // of all requests
  int free;                // blocks on the stack before the call
  bool ok;
};

// Called by all threads.  rows_of, blocks_of (nullable): [N + 1], the sums over the requests before each one.
template <bool kTrim, int kThreads>
__device__ __forceinline__ Sums add_up(const TablesParams& p, long long* scratch, int* rows_of, int* blocks_of) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = (p.num_seqs + kThreads - 1) / kThreads;
  const int begin = min(p.num_seqs, run * (int)threadIdx.x), end = min(p.num_seqs, begin + run);
  long long rows = 0, blocks = 0;
  bool bad = false;
  int row[kKept] = {}, block[kKept] = {};
  if (run <= kKept) {
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      if (begin + i < end) {
        const Request r = request<kTrim>(p, begin + i);
        bad = bad || r.bad;
        row[i] = r.bad ? 0 : r.wanted;
        block[i] = r.blocks;
      }
    }
#pragma unroll
    for (int i = 0; i < kKept; ++i) rows += row[i], blocks += block[i];
  } else {
    for (int s = begin; s < end; ++s) {
      const Request r = request<kTrim>(p, s);
      bad = bad || r.bad;
      rows += r.bad ? 0 : r.wanted;
      blocks += r.blocks;
    }
  }
  long long rows_to = rows, blocks_to = blocks;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, rows_to, off), y = __shfl_up_sync(0xffffffffu, blocks_to, off);
    if (lane >= off) rows_to += x, blocks_to += y;
  }
  if (lane == 31) scratch[2 * warp] = rows_to, scratch[2 * warp + 1] = blocks_to;
  Sums sums = {0, 0, *p.num_free, false};
  bad = __syncthreads_or(bad);
  // the warps' sums, added up by the first one: scratch[2 w] becomes what lies before warp w, the last two the totals
  constexpr int kWarps = kThreads / 32;
  if (warp == 0) {
    const long long r = lane < kWarps ? scratch[2 * lane] : 0, b = lane < kWarps ? scratch[2 * lane + 1] : 0;
    long long x = r, y = b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) x += u, y += v;
    }
    if (lane < kWarps) scratch[2 * lane] = x - r, scratch[2 * lane + 1] = y - b;
    if (lane == 31) scratch[2 * kWarps] = x, scratch[2 * kWarps + 1] = y;
  }
  __syncthreads();
  rows_to += scratch[2 * warp], blocks_to += scratch[2 * warp + 1];
  sums.rows = scratch[2 * kWarps], sums.blocks = scratch[2 * kWarps + 1];
  const bool state = !bad && sums.free >= 0 && sums.free <= p.num_blocks;
  sums.ok = state && (kTrim ? sums.free + sums.blocks <= p.num_blocks
                            : sums.blocks <= sums.free && sums.rows <= p.num_rows);
  if (sums.ok && blocks_of != nullptr) {
    int q = (int)(rows_to - rows), b = (int)(blocks_to - blocks);
    auto put = [&](int s, int r, int n) {
      if (rows_of != nullptr) rows_of[s] = q;
      blocks_of[s] = b;
      q += r;
      b += n;
    };
    if (run <= kKept) {
#pragma unroll
      for (int i = 0; i < kKept; ++i)
        if (begin + i < end) put(begin + i, row[i], block[i]);
    } else {
      for (int s = begin; s < end; ++s) {
        const Request r = request<kTrim>(p, s);
        put(s, r.wanted, r.blocks);
      }
    }
    if (threadIdx.x == 0) {
      if (rows_of != nullptr) rows_of[p.num_seqs] = (int)sums.rows;
      blocks_of[p.num_seqs] = (int)sums.blocks;
    }
  }
  __syncthreads();
  return sums;
}

// the last request whose sum is at most x (x below the total: the one that x belongs to)
__device__ __forceinline__ int owner(const int* of, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (of[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One CTA: the new lengths, or the error.
template <bool kTrim, int kThreads>
__device__ __forceinline__ void commit(const TablesParams& p, const Sums& sums) {
  if (!sums.ok) {
    if (threadIdx.x == 0) {
      const bool short_of_blocks = !kTrim && sums.free >= 0 && sums.free <= p.num_blocks && sums.blocks > sums.free;
      report_error(p.err_flag, short_of_blocks ? PA_DEVERR_NO_BLOCKS : PA_DEVERR_TABLES);
    }
    return;
  }
  for (int s = threadIdx.x; s < p.num_seqs; s += kThreads) {
    const Request r = request<kTrim>(p, s);
    p.seq_lens[s] = kTrim ? r.wanted : r.len + r.wanted;
    p.held[s] = kTrim ? r.held - r.blocks : r.held + r.blocks;
  }
  if (threadIdx.x == 0) p.num_free[0] = kTrim ? sums.free + (int)sums.blocks : sums.free - (int)sums.blocks;
}

// every CTA of the one cluster has read the lengths
__device__ __forceinline__ void all_read() {
  if (gridDim.x > 1) cluster_sync_all();
  else __syncthreads();
}

// kAlone: the grid is one cluster, which writes the lengths too (else commit_kernel does).
template <bool kAlone, int kThreads>
__global__ void __launch_bounds__(kThreads) extend_kernel(const TablesParams p) {
  extern __shared__ int sums_of[];  // rows before each request, then blocks
  __shared__ long long scratch[2 * kThreads / 32 + 2];
  int* rows_of = sums_of;
  int* blocks_of = sums_of + p.num_seqs + 1;
  griddep_wait();
  const Sums sums = add_up<false, kThreads>(p, scratch, rows_of, blocks_of);
  const int B = p.block_size, total = sums.ok ? (int)sums.rows : 0;
  for (int s = blockIdx.x * kThreads + threadIdx.x; s <= p.num_seqs; s += gridDim.x * kThreads)
    p.query_start[s] = sums.ok ? rows_of[s] : 0;
  const long long step = (long long)gridDim.x * kThreads;
  for (long long t0 = (long long)blockIdx.x * kThreads + threadIdx.x; t0 < p.num_rows; t0 += kAhead * step) {
    int s[kAhead], held[kAhead], pos[kAhead], block[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const long long t = t0 + i * step;
      s[i] = t < total ? owner(rows_of, p.num_seqs, (int)t) : -1;
      held[i] = s[i] >= 0 ? p.held[s[i]] : 0;
      pos[i] = s[i] >= 0 ? p.seq_lens[s[i]] + (int)t - rows_of[s[i]] : 0;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      block[i] = -1;
      if (s[i] >= 0) {
        const int b = pos[i] / B;
        block[i] = b < held[i] ? p.block_tables[(long long)s[i] * p.max_blocks + b]
                               : p.free_blocks[sums.free - 1 - (blocks_of[s[i]] + b - held[i])];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const long long t = t0 + i * step;
      if (t >= p.num_rows) break;
      long long slot = -1;
      if (s[i] >= 0) {
        const int b = pos[i] / B, off = pos[i] - b * B;
        // (a fresh block's first token is new: the blocks held hold the others)
        if (b >= held[i] && off == 0) p.block_tables[(long long)s[i] * p.max_blocks + b] = block[i];
        if (block[i] >= 0 && block[i] < p.num_blocks) slot = (long long)block[i] * B + off;
        else report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
      }
      p.slot_mapping[t] = slot;
      p.positions[t] = pos[i];
    }
  }
  if constexpr (kAlone) {
    all_read();
    if (blockIdx.x == 0) commit<false, kThreads>(p, sums);
  }
  __threadfence();  // see the file comment
}

template <bool kAlone, int kThreads>
__global__ void __launch_bounds__(kThreads) trim_kernel(const TablesParams p) {
  extern __shared__ int blocks_of[];
  __shared__ long long scratch[2 * kThreads / 32 + 2];
  griddep_wait();
  const Sums sums = add_up<true, kThreads>(p, scratch, nullptr, blocks_of);
  const int B = p.block_size, total = sums.ok ? (int)sums.blocks : 0;
  const long long step = (long long)gridDim.x * kThreads;
  for (long long i0 = (long long)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += kAhead * step) {
    int32_t* entry[kAhead];
    int block[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long i = i0 + j * step;
      entry[j] = nullptr;
      if (i < total) {
        const int s = owner(blocks_of, p.num_seqs, (int)i);
        const int kept = (int)(((long long)p.wanted[s] + B - 1) / B);
        entry[j] = p.block_tables + (long long)s * p.max_blocks + kept + (i - blocks_of[s]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) block[j] = entry[j] != nullptr ? *entry[j] : 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (entry[j] == nullptr) break;
      if (block[j] < 0 || block[j] >= p.num_blocks) report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
      p.free_blocks[sums.free + total - 1 - (i0 + j * step)] = block[j];
      *entry[j] = -1;
    }
  }
  if constexpr (kAlone) {
    all_read();
    if (blockIdx.x == 0) commit<true, kThreads>(p, sums);
  }
  __threadfence();
}

template <bool kTrim>
__global__ void __launch_bounds__(kLarge) commit_kernel(const TablesParams p) {
  constexpr int kThreads = kLarge;
  __shared__ long long scratch[2 * kThreads / 32 + 2];
  griddep_wait();
  const Sums sums = add_up<kTrim, kThreads>(p, scratch, nullptr, nullptr);
  commit<kTrim, kThreads>(p, sums);
  __threadfence();
}

template <bool kTrim>
cudaError_t launch(const TablesParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)(p.num_seqs + 1) * sizeof(int) * (kTrim ? 1 : 2);
  const long long ctas = std::max(1ll, ((long long)p.num_rows + kAhead * kLarge - 1) / (kAhead * kLarge));
  auto run = [&](void (*kernel)(TablesParams), int grid, int threads, int cluster, size_t bytes) {
    cudaError_t e = cudaSuccess;
    if (bytes > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    return e != cudaSuccess ? e : launch_cluster(kernel, dim3((unsigned)grid), dim3(threads), bytes, cluster, true, stream, p);
  };
  // (few requests release few blocks, as a rule: one CTA, 11 us for one request that ends with 2500 blocks.  Its threads
  // walk what is released: 64 requests of 2500 blocks each take 0.36 ms there, 256 of them 1.6 ms, and 257, which eight
  // CTAs of 1024 threads take, 76 us.)
  if (p.num_seqs <= kSmall && ctas == 1)
    return run(kTrim ? trim_kernel<true, kSmall> : extend_kernel<true, kSmall>, 1, kSmall, 1, smem);
  if (kTrim || ctas <= kMaxTablesCluster) {
    int cluster = kTrim ? kMaxTablesCluster : 1;
    while (cluster < ctas) cluster *= 2;
    return run(kTrim ? trim_kernel<true, kLarge> : extend_kernel<true, kLarge>, cluster, kLarge, cluster, smem);
  }
  if constexpr (!kTrim) {
    const cudaError_t e = run(extend_kernel<false, kLarge>, (int)std::min(ctas, 152ll), kLarge, 1, smem);
    return e != cudaSuccess ? e : run(commit_kernel<false>, 1, kLarge, 1, 0);
  }
}

// Checks that both calls share.
int check_tables(const TablesParams& p) {
  if (p.num_seqs < 0 || p.max_blocks < 0 || p.block_size <= 0 || p.num_blocks < 0 || p.num_rows < 0)
    return PA_ERR_INVALID_ARG;
  if (p.num_seqs > kMaxSeqs || (int64_t)p.max_blocks * p.block_size > kInt32Max) return PA_ERR_TOO_LARGE;
  if (p.num_seqs == 0 && p.num_rows == 0) return PA_OK;
  if ((p.num_seqs > 0 && (p.seq_lens == nullptr || p.held == nullptr || p.wanted == nullptr ||
                          (p.block_tables == nullptr && p.max_blocks > 0))) ||
      p.num_free == nullptr || (p.free_blocks == nullptr && p.num_blocks > 0))
    return PA_ERR_NULL_POINTER;
  if (!aligned(p.block_tables, 4) || !aligned(p.seq_lens, 4) || !aligned(p.held, 4) || !aligned(p.free_blocks, 4) ||
      !aligned(p.num_free, 4) || !aligned(p.wanted, 4))
    return PA_ERR_MISALIGNED;
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_tables_extend(int32_t* block_tables, int32_t* seq_lens, int32_t* held_blocks, const int32_t* free_blocks,
                     int32_t* num_free, const int32_t* new_tokens, int64_t* slot_mapping, int32_t* positions,
                     int32_t* query_start, int32_t num_seqs, int32_t num_rows, int32_t max_blocks_per_seq,
                     int32_t block_size, int32_t num_blocks, int32_t* err_flag, void* stream) {
  const pa::TablesParams p = {block_tables, seq_lens,     held_blocks, const_cast<int32_t*>(free_blocks),
                              num_free,     new_tokens,   slot_mapping, positions,
                              query_start,  num_seqs,     num_rows,    max_blocks_per_seq,
                              block_size,   num_blocks,   err_flag};
  const int rc = pa::check_tables(p);
  // (no requests and no rows: only query_start[0] is to be written, if there is a state at all)
  if (rc != PA_OK || (num_seqs == 0 && num_rows == 0 && (query_start == nullptr || num_free == nullptr))) return rc;
  if (query_start == nullptr || (num_rows > 0 && (slot_mapping == nullptr || positions == nullptr)))
    return PA_ERR_NULL_POINTER;
  if (!aligned(num_free, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(query_start, 4))
    return PA_ERR_MISALIGNED;
  return pa::launch<false>(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_tables_trim(int32_t* block_tables, int32_t* seq_lens, int32_t* held_blocks, int32_t* free_blocks,
                   int32_t* num_free, const int32_t* keep_lens, int32_t num_seqs, int32_t max_blocks_per_seq,
                   int32_t block_size, int32_t num_blocks, int32_t* err_flag, void* stream) {
  pa::TablesParams p = {};
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.held = held_blocks;
  p.free_blocks = free_blocks;
  p.num_free = num_free;
  p.wanted = keep_lens;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.err_flag = err_flag;
  const int rc = pa::check_tables(p);
  if (rc != PA_OK || num_seqs == 0) return rc;
  return pa::launch<true>(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
