// pa_window_rows.cuh - what the rows kernels of windowed attention share: the
// work item, the visible slabs of its keys, bounded waits, and the merge of its
// warps and CTAs.
//
// Query rows.  The n queries of a sequence and the G query heads of a kv head
// give n * G rows that read the same K/V; row R is query R / G, head R % G of
// the group.  An item is eight consecutive rows of one kv head (the N of the
// mma.m16n8k16 tiles; a decode step has n = 1).  A row at position p sees the
// positions i <= p with i > p - W or i < S, so the rows of an item see
//   [0, S') and [lo, p_last],  lo = max(0, p_first - W + 1), S' = min(S, p_last + 1),
// which is walked as one list of slabs of SB tokens: the slabs of the first
// range, then those of the second that are not among them.  Table entries and
// tokens outside are never touched: their blocks may have been released.
//
// Split.  The slabs are divided evenly among the CTAs of a cluster, and the
// CTAs' results are merged through distributed shared memory in the same
// launch.  A window bounds the keys of an item, so that one cluster covers it:
// no partition workspace, no second kernel.
#pragma once

#include <math.h>

#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_window.h"

namespace pa {

constexpr int kRowsGroup = 8;  // rows of an item

// The start of a kernel launched as a programmatic dependent: everything it reads (lengths and tables among
// it) is read, and anything written, after the kernels before it have finished and their writes are visible,
// whatever they are; the kernel after it may be scheduled from here on.  What comes before is set-up that
// reads no memory.
__device__ __forceinline__ void griddep_begin() {
  griddep_wait();
  griddep_launch_dependents();
}

struct RowsItem {
  int s, hkv;
  int row0, gcount;     // first row (query * G + head) and number of rows
  int q0, base;         // q row of query 0, position of query 0
  int G;
  int L;                // tokens of the sequence
  int p_first, p_last;  // positions of the first and last row
  int lo_first, lo_last;  // lowest position of the window of the first and last row
  int sinks;            // S' (0 when the window reaches position 0 anyway, or none are visible)
  int n_sink, j_win;    // slabs of [0, S'), first slab of the rest
  int v0, v1;           // this CTA's slabs of the list
  bool empty;           // a decode row of an empty sequence: zeros
};

// The queries of sequence s: q rows q0 .. q0 + n - 1, the last of L tokens.  bad: a chunk outside q / out, longer than
// the caller's bound or than its sequence, or a sequence past its table.
struct RowsChunk {
  int q0, n, L;
  bool bad;
};
__device__ __forceinline__ RowsChunk rows_chunk(const WindowParams& p, int s) {
  RowsChunk c = {s, 1, __ldg(p.seq_lens + s), false};
  c.bad = c.L < 0 || (long long)c.L > (long long)p.max_blocks * p.block_size;
  if (p.query_start != nullptr) {
    c.q0 = __ldg(p.query_start + s);
    const long long len = (long long)__ldg(p.query_start + s + 1) - c.q0;
    c.bad = c.bad || c.q0 < 0 || len < 0 || c.q0 + len > p.num_query_tokens || len > p.max_query_len || c.L < len;
    c.n = (int)len;
  }
  return c;
}

// Slots (batches that mix long chunks with many short ones): the row groups of all sequences lie one after the other,
// so the grid holds no more than the rows of q fill and one a sequence, where the longest chunk's groups for every
// sequence would be mostly empty (1024 sequences, a chunk of 4096 among single tokens: 33.5 million items of which 41
// thousand exist, and past 2^31 no grid at all).  The CTA's threads add up the sequences' groups, each over a run of
// them, and find the one whose group lies in `slot`.  False: none does.  Called by all threads; sums: 8 + 1 numbers of
// shared memory, free again after the next barrier.  Chunks that overlap may need more slots than there are: reported.
__device__ __forceinline__ bool rows_find(const WindowParams& p, int slot, long long* sums, bool report, int& s,
                                          int& rg) {
  const int G = p.num_q_heads / p.num_kv_heads, threads = (int)blockDim.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long run = (p.num_seqs + threads - 1) / threads;
  const int begin = (int)min((long long)p.num_seqs, run * threadIdx.x);
  const int end = (int)min((long long)p.num_seqs, run * (threadIdx.x + 1));
  auto groups = [&](const RowsChunk& c) {
    return c.bad ? 0 : (int)(((long long)c.n * G + kRowsGroup - 1) / kRowsGroup);
  };
  long long mine = 0;
  for (int i = begin; i < end; ++i) {
    const RowsChunk c = rows_chunk(p, i);
    if (c.bad && report) report_error(p.err_flag, PA_DEVERR_QUERY);
    mine += groups(c);
  }
  long long upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  int* found = reinterpret_cast<int*>(sums + 8);
  if (lane == 31) sums[warp] = upto;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sums[w];
  if (report && threadIdx.x == threads - 1 && upto > p.tiles) report_error(p.err_flag, PA_DEVERR_QUERY);
  long long at = upto - mine;
  if (slot >= at && slot < upto) {
    int i = begin;
    for (int n; (n = groups(rows_chunk(p, i))) <= slot - at; ++i) at += n;
    found[0] = i;
    found[1] = (int)(slot - at);
  }
  __syncthreads();
  s = found[0];
  rg = found[1];
  return s >= 0;
}

// The item of this CTA's cluster and the CTA's share of its slabs (SB tokens each).  False: nothing to do (the
// same for every CTA of the cluster).  A bad chunk is reported once, and nothing of it is done.  Called by all
// threads.  SLOTS: the row groups lie in p.tiles slots, sums as for rows_find (a form of its own: with the choice at run
// time the fp32 kernel kept 130 registers for 157 and lost 5 %).
template <int SB, bool SLOTS>
__device__ __forceinline__ bool rows_item(const WindowParams& p, RowsItem& it, long long* sums) {
  const int C = p.cluster;
  const int rank = (int)(blockIdx.x % (unsigned)C);
  int id = (int)(blockIdx.x / (unsigned)C), rg;
  if constexpr (SLOTS) {
    it.hkv = id % p.num_kv_heads;
    id /= p.num_kv_heads;
    if (!rows_find(p, id, sums, id == 0 && it.hkv == 0 && rank == 0, it.s, rg)) return false;
  } else {
    rg = id % p.tiles;
    id /= p.tiles;
    it.hkv = id % p.num_kv_heads;
    it.s = id / p.num_kv_heads;
  }
  it.G = p.num_q_heads / p.num_kv_heads;
  it.row0 = rg * kRowsGroup;
  it.empty = false;
  const RowsChunk chunk = rows_chunk(p, it.s);
  if (chunk.bad) {
    if (rg == 0 && it.hkv == 0 && rank == 0 && threadIdx.x == 0) report_error(p.err_flag, PA_DEVERR_QUERY);
    return false;
  }
  const int L = chunk.L, n = chunk.n;
  it.q0 = chunk.q0;
  it.L = L;
  it.gcount = min((long long)kRowsGroup, (long long)n * it.G - it.row0);
  if (it.gcount <= 0) return false;
  if (L == 0) {  // a decode row of an empty sequence (a chunk's L >= n > 0)
    it.empty = true;
    return rank == 0;
  }
  it.base = L - n;
  it.p_first = it.base + it.row0 / it.G;
  it.p_last = it.base + (it.row0 + it.gcount - 1) / it.G;
  it.lo_first = max(0, it.p_first - p.window + 1);
  it.lo_last = max(0, it.p_last - p.window + 1);
  it.sinks = min(p.sinks, it.p_last + 1);
  it.n_sink = (it.sinks + SB - 1) / SB;
  it.j_win = max(it.lo_first / SB, it.n_sink);
  const int total = it.n_sink + max(0, it.p_last / SB + 1 - it.j_win);
  it.v0 = (int)((long long)total * rank / C);
  it.v1 = (int)((long long)total * (rank + 1) / C);
  return true;
}

// slab v of the item's list
__device__ __forceinline__ int rows_slab(const RowsItem& it, int v) {
  return v < it.n_sink ? v : v - it.n_sink + it.j_win;
}
// does some row of the item see one of the tokens t .. t + w - 1?
__device__ __forceinline__ bool rows_touch(const RowsItem& it, int t, int w) {
  return t <= it.p_last && (t < it.sinks || t + w > it.lo_first);
}
// does every row of the item see all of the tokens t .. t + w - 1?
__device__ __forceinline__ bool rows_full(const RowsItem& it, int t, int w) {
  return t + w - 1 <= it.p_first && (t >= it.lo_last || t + w <= it.sinks);
}
// does some row see token t?
__device__ __forceinline__ bool rows_any(const RowsItem& it, int t) {
  return t <= it.p_last && (t >= it.lo_first || t < it.sinks);
}

// row r's offset, in rows of D elements, in q and out
__device__ __forceinline__ size_t rows_offset(const WindowParams& p, const RowsItem& it, int r) {
  const int R = it.row0 + r;
  return ((size_t)it.q0 + R / it.G) * p.num_q_heads + (size_t)it.hkv * it.G + R % it.G;
}

template <typename T, int D>
__device__ __forceinline__ void rows_zero(const WindowParams& p, const RowsItem& it) {
  for (int i = threadIdx.x; i < it.gcount * D; i += blockDim.x)
    reinterpret_cast<T*>(p.out)[rows_offset(p, it, i / D) * D + i % D] = from_float<T>(0.f);
}

// The item's end.  Each of the NW warps left, at parts + w * STRIDE floats, its unnormalised O[8 rows][OROW]
// and then (m, l)[8 rows] (max score in log2 units, sum of 2^(s - m)).  With m* = max m and weights
// 2^(m - m*), O = sum weight O and l = sum weight l over the warps, then in the same way over the CTAs of the
// cluster, whose results sit in each CTA's `mine` (8 x D floats, then 8 pairs); each CTA writes its share of
// the output elements: O / l, zeros where l is 0 (no weight), NaN where a score was NaN (l is).  Called by every
// thread after the barrier that follows the warps' stores; wt: 8 * NW + 16 floats apart from the parts.
template <typename TOut, int D, int NW, int OROW, int STRIDE>
__device__ __forceinline__ void rows_finish(const WindowParams& p, const RowsItem& it, const float* parts, float* wt,
                                            float* mine) {
  float* mst = wt + 8 * NW;
  float* lsum = mst + 8;
  if (threadIdx.x < 8) {
    const int r = threadIdx.x;
    float mw[NW];
    float ms = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      mw[w] = parts[w * STRIDE + 8 * OROW + r * 2];
      ms = fmaxf(ms, mw[w]);
    }
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float x = mw[w] == -INFINITY ? 0.f : fast_exp2(mw[w] - ms);
      l += x * parts[w * STRIDE + 8 * OROW + r * 2 + 1];
      wt[r * NW + w] = x;
    }
    mst[r] = ms;
    lsum[r] = l;
    mine[8 * D + 2 * r] = ms;
    mine[8 * D + 2 * r + 1] = l;
  }
  __syncthreads();
  const int total = it.gcount * D;
  const int C = p.cluster;
#pragma unroll 4
  for (int i = threadIdx.x; i < total; i += NW * 32) {
    const int r = i / D, d = i % D;
    float acc = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) acc += wt[r * NW + w] * parts[w * STRIDE + r * OROW + d];
    if (C == 1) {
      const float l = lsum[r];
      reinterpret_cast<TOut*>(p.out)[rows_offset(p, it, r) * D + d] = from_float<TOut>(l == 0.f ? 0.f : acc / l);
    } else {
      mine[i] = acc;
    }
  }
  if (C == 1) return;
  cluster_sync_all();
  const int rank = (int)cluster_rank();
  for (int i = total * rank / C + threadIdx.x; i < total * (rank + 1) / C; i += NW * 32) {
    const int r = i / D, d = i % D;
    float mx = -INFINITY;
    for (int c = 0; c < C; ++c) mx = fmaxf(mx, ld_cluster(mine + 8 * D + 2 * r, c));
    float acc = 0.f, l = 0.f;
#pragma unroll 4
    for (int c = 0; c < C; ++c) {
      const float m = ld_cluster(mine + 8 * D + 2 * r, c);
      const float x = m == -INFINITY ? 0.f : fast_exp2(m - mx);
      l = fmaf(x, ld_cluster(mine + 8 * D + 2 * r + 1, c), l);
      acc = fmaf(x, ld_cluster(mine + i, c), acc);
    }
    reinterpret_cast<TOut*>(p.out)[rows_offset(p, it, r) * D + d] = from_float<TOut>(l == 0.f ? 0.f : acc / l);
  }
  cluster_sync_all();  // no CTA leaves while another reads its results
}

constexpr long long kRowsWaitCycles = 500ll * 1000 * 1000;  // bound on one wait: ~0.25 s at 2 GHz
constexpr long long kRowsTestWaitCycles = 20000;            // the test hook's bound on a ring's first wait

// Wait for a barrier phase; gives up (returning false) when the CTA's abort flag is set or after `limit` SM
// cycles, in which case it raises the flag.
__device__ __forceinline__ bool rows_wait(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag,
                                          long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if ((i & 15u) == 15u && clock64() - start > limit) {
      *abort_flag = 1;
      return false;
    }
  }
}

// Online softmax of one lane's scores for rows a and b (s0, s2 of a, s1, s3 of b, ...): moves the running
// maxima when a score exceeds one by more than kSlabSlack (log2 units), rescaling l and o, and returns the
// maxima to subtract: 0 for a row that has seen no token yet, so that masked scores (-inf) give weight 0.
template <int NSC, int KSTEPS>
__device__ __forceinline__ void rows_softmax_max(const float (&s)[NSC], float (&o)[KSTEPS][4], float& m_a, float& m_b,
                                                 float& l_a, float& l_b, float& sub_a, float& sub_b) {
  bool over = false;
#pragma unroll
  for (int i = 0; i < NSC; i += 2) over = over || s[i] - m_a > kSlabSlack || s[i + 1] - m_b > kSlabSlack;
  if (__any_sync(0xffffffffu, over)) {
    float mx_a = s[0], mx_b = s[1];
#pragma unroll
    for (int i = 2; i < NSC; i += 2) {
      mx_a = fmaxf(mx_a, s[i]);
      mx_b = fmaxf(mx_b, s[i + 1]);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
    }
    const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
    // (a row without a token yet has l = o = 0: any finite factor will do)
    const float al_a = mn_a == -INFINITY ? 1.f : fast_exp2(m_a - mn_a);
    const float al_b = mn_b == -INFINITY ? 1.f : fast_exp2(m_b - mn_b);
    m_a = mn_a;
    m_b = mn_b;
    l_a *= al_a;
    l_b *= al_b;
#pragma unroll
    for (int i = 0; i < KSTEPS; ++i) {
      o[i][0] *= al_a;
      o[i][1] *= al_b;
      o[i][2] *= al_a;
      o[i][3] *= al_b;
    }
  }
  sub_a = m_a == -INFINITY ? 0.f : m_a;
  sub_b = m_b == -INFINITY ? 0.f : m_b;
}

}  // namespace pa
