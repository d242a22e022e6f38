// pa_window_rows_tc.cu - attention of a few query rows over a window of an
// fp16 / bf16 cache: the decode step, and chunks that the tile kernel does not
// take (see pa_window_rows.cuh for the rows, the visible slabs and the split).
//
// Bound by HBM bandwidth: each visible token costs 2 D elements and 4 D flops a
// row.  A CTA of three, four or six warps streams 16-token slabs of K and V; every
// warp fills its own ring of NS slab buffers with tensor-map copies and drains it
// in order, so that an SM's twelve warps have up to 24 slabs (192 KB) in flight.
// 128 sequences, 64 / 8 heads of 128, bf16, the last 1024 of up to 16384 tokens:
// 88 us, 6.2 TB/s.
// A slab takes two mma.m16n8k16 contractions, S^T[16 tokens x 8 rows] = K Q^T
// and O^T[D x 8 rows] += V^T P^T, fp32 accumulation and an online softmax.  The
// weights enter the second one as two 16-bit terms (rounded part and residual:
// a single fp16 term would add an error of the size of the output's own
// rounding), which costs tensor work that the copies hide.
//
// A copy takes its issuing lane some 200 cycles, so a slab is two copies, one of
// K and one of V: the tensor maps see a cache as (64 columns, rows, D / 64), and
// a box brings a slab's rows of every 64-column part, one part after the other.
// Blocks of 8 tokens (SPLIT) make a slab of two such boxes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "pa.h"
#include "pa_window_rows.cuh"

namespace pa {
namespace {

template <int D, int NW, int NS>
struct RowsShape {
  static constexpr int SB = kTcSlabTokens;
  static constexpr int KSTEPS = D / 16;                    // k-steps of Q K^T = m-tiles of V^T P^T
  static constexpr int NBOX = D / 64;                      // 128-byte (64-element) boxes per row
  static constexpr int BOX_BYTES = SB * 128;
  static constexpr int TILE_BYTES = NBOX * BOX_BYTES;      // the slab's rows of K, or of V
  static constexpr int SLAB_BYTES = 2 * TILE_BYTES;        // K, then V
  static constexpr int RING_BYTES = NS * SLAB_BYTES;       // per warp
  static constexpr int OROW = D + 4;                       // merge row stride (floats): conflict-free stores
  static constexpr int BAR_OFF = NW * RING_BYTES;
  static constexpr int FLAG_OFF = BAR_OFF + NW * NS * 8;   // the CTA's abort flag
  static constexpr int STAGE_OFF = FLAG_OFF + 16;          // the appended token's K and V rows
  static constexpr int MINE_OFF = STAGE_OFF + 4 * D;       // the CTA's result: 8 x D floats, 8 (m, l)
  static constexpr int WT_OFF = MINE_OFF + (8 * D + 16) * 4;
  static constexpr int SMEM_BYTES = WT_OFF + (8 * NW + 16) * 4 + 1024;  // + alignment slack
  static constexpr int THREADS = NW * 32;
  static_assert(RING_BYTES >= (8 * OROW + 16) * 4, "a warp's ring holds its partial result at the end");
};

// Byte offset of 16-byte chunk c (8 columns) of row r in a slab's K or V tile: the 64-column parts one after the
// other, in SPLIT slabs for rows 0..7 first and then for rows 8..15; 128-byte swizzle.
template <int D, bool SPLIT>
__device__ __forceinline__ uint32_t tile_chunk(uint32_t r, uint32_t c) {
  constexpr uint32_t UP = SPLIT ? D / 64 * 1024 : 1024, PART = SPLIT ? 1024 : 2048;
  return (r >> 3) * UP + (c >> 3) * PART + swz128(r & 7, c & 7);
}

// One slab: S^T = K Q^T, online softmax update, O^T += V^T P^T.  bias: slopes of the lane's two rows in log2
// units; tok0: the slab's first token.
template <typename T, int D, bool SPLIT>
__device__ __forceinline__ void window_slab(const uint8_t* kst, const uint8_t* vst, int tok0, const RowsItem& it,
                                            const uint32_t (&qf)[D / 16][2], float (&o)[D / 16][4], float& m_a,
                                            float& m_b, float& l_a, float& l_b, int lane, float sl2, float bias_a,
                                            float bias_b, int pos_a, int pos_b, int window) {
  constexpr int KSTEPS = D / 16;
  const int g = lane >> 2, q4 = lane & 3;
  float sc[4] = {0.f, 0.f, 0.f, 0.f};  // two accumulators: shorter dependency chain
  float sd[4] = {0.f, 0.f, 0.f, 0.f};
  {
    const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
    const int khalf = lane >> 4;
#pragma unroll
    for (int j0 = 0; j0 < KSTEPS; j0 += 4) {  // four loads on their way before the first is used
      uint32_t f[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ldmatrix_x4(smem_u32(kst) + tile_chunk<D, SPLIT>(row, (j0 + j) * 2 + khalf), f[j][0], f[j][1], f[j][2], f[j][3]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        Mma<T>::run(j & 1 ? sd : sc, f[j][0], f[j][1], f[j][2], f[j][3], qf[j0 + j][0], qf[j0 + j][1]);
    }
  }
  // scores: (token g, row a = 2q4), (token g, row b = 2q4 + 1), (token g + 8, row a), (token g + 8, row b)
  const int t_lo = tok0 + g, t_hi = t_lo + 8;
  float s[4];
  s[0] = fmaf(bias_a, (float)(t_lo - pos_a), (sc[0] + sd[0]) * sl2);
  s[1] = fmaf(bias_b, (float)(t_lo - pos_b), (sc[1] + sd[1]) * sl2);
  s[2] = fmaf(bias_a, (float)(t_hi - pos_a), (sc[2] + sd[2]) * sl2);
  s[3] = fmaf(bias_b, (float)(t_hi - pos_b), (sc[3] + sd[3]) * sl2);
  const bool full = rows_full(it, tok0, kTcSlabTokens);
  if (!full) {
    auto sees = [&](int t, int pos) { return t <= pos && (t > pos - window || t < it.sinks); };
    if (!sees(t_lo, pos_a)) s[0] = -INFINITY;
    if (!sees(t_lo, pos_b)) s[1] = -INFINITY;
    if (!sees(t_hi, pos_a)) s[2] = -INFINITY;
    if (!sees(t_hi, pos_b)) s[3] = -INFINITY;
  }
  float sub_a, sub_b;
  rows_softmax_max(s, o, m_a, m_b, l_a, l_b, sub_a, sub_b);
  const float p0 = fast_exp2(s[0] - sub_a), p1 = fast_exp2(s[1] - sub_b);
  const float p2 = fast_exp2(s[2] - sub_a), p3 = fast_exp2(s[3] - sub_b);
  const uint32_t x0 = Mma<T>::pack(p0, p1), x1 = Mma<T>::pack(p2, p3);
  const uint32_t y0 = Mma<T>::pack(p0 - Mma<T>::lo(x0), p1 - Mma<T>::hi(x0));
  const uint32_t y1 = Mma<T>::pack(p2 - Mma<T>::lo(x1), p3 - Mma<T>::hi(x1));
  l_a += p0 + p2;
  l_b += p1 + p3;
  // P^T fragments: (tokens 2q4, 2q4 + 1 | + 8, + 9; row g)
  const uint32_t pb0 = movmatrix_trans(x0), pb1 = movmatrix_trans(x1);
  const uint32_t pc0 = movmatrix_trans(y0), pc1 = movmatrix_trans(y1);
  uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
  if (!full) {  // values of tokens that no row sees may hold NaN: zero them
    const int t0 = tok0 + 2 * q4;
    mlo = (rows_any(it, t0) ? 0x0000ffffu : 0u) | (rows_any(it, t0 + 1) ? 0xffff0000u : 0u);
    mhi = (rows_any(it, t0 + 8) ? 0x0000ffffu : 0u) | (rows_any(it, t0 + 9) ? 0xffff0000u : 0u);
  }
  const int row = (lane & 7) + (lane >> 4) * 8;
  const int dhalf = (lane >> 3) & 1;
#pragma unroll
  for (int i0 = 0; i0 < KSTEPS; i0 += 4) {
    uint32_t f[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ldmatrix_x4_trans(smem_u32(vst) + tile_chunk<D, SPLIT>(row, (i0 + i) * 2 + dhalf), f[i][0], f[i][1], f[i][2],
                        f[i][3]);
    if (!full) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i][0] &= mlo, f[i][1] &= mlo, f[i][2] &= mhi, f[i][3] &= mhi;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) Mma<T>::run(o[i0 + i], f[i][0], f[i][1], f[i][2], f[i][3], pb0, pb1);
#pragma unroll
    for (int i = 0; i < 4; ++i) Mma<T>::run(o[i0 + i], f[i][0], f[i][1], f[i][2], f[i][3], pc0, pc1);
  }
}

template <typename T, int D, int NW, int NS, bool SPLIT, bool SLOTS>
__global__ void __launch_bounds__(RowsShape<D, NW, NS>::THREADS)
    window_rows_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const WindowParams p) {
  using S = RowsShape<D, NW, NS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q4 = lane & 3;
  uint8_t* ring = smem + warp * S::RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF) + warp * NS;
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + S::FLAG_OFF);
  if (threadIdx.x == 0) {
    abort_flag[0] = 0;
    tma_prefetch_descriptor(&tmap_k);
    tma_prefetch_descriptor(&tmap_v);
  }
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  griddep_begin();
  RowsItem it;
  if (!rows_item<S::SB, SLOTS>(p, it, reinterpret_cast<long long*>(smem + S::WT_OFF))) return;
  if (it.empty) {
    rows_zero<T, D>(p, it);
    return;
  }
  // ---- this warp's slabs: v0 + warp + k * NW, k < n_my
  const int mine = it.v1 - it.v0;
  const int n_my = mine > warp ? (mine - warp + NW - 1) / NW : 0;
  const int B = p.block_size;
  const int32_t* table = p.block_tables + (size_t)it.s * p.max_blocks;
  auto slab_tok = [&](int k) { return rows_slab(it, it.v0 + warp + k * NW) * S::SB; };
  // lane l holds the table entries of this warp's slab 32 b + l: its block, or with 8-token blocks those of its
  // two halves (-1 for a half that no row sees)
  auto fetch = [&](int k, int& e0, int& e1) {
    e0 = e1 = -1;
    if (k < n_my) {
      const int tok0 = slab_tok(k);
      if (!SPLIT || rows_touch(it, tok0, B)) e0 = __ldg(table + tok0 / B);
      if (SPLIT && rows_touch(it, tok0 + B, B)) e1 = __ldg(table + tok0 / B + 1);
    }
  };
  int pb_batch = 0, pb_reg, pb_reg2;
  fetch(lane, pb_reg, pb_reg2);

  uint32_t valid_mask = 0;  // bit `stage`: the slab in that buffer was loaded
  auto issue = [&](int k) {  // called by the whole warp, k increasing
    if ((k >> 5) != pb_batch) {
      pb_batch = k >> 5;
      fetch(k + lane, pb_reg, pb_reg2);
    }
    const int pb = __shfl_sync(0xffffffffu, pb_reg, k & 31);
    const int pb2 = __shfl_sync(0xffffffffu, pb_reg2, k & 31);
    const int tok0 = slab_tok(k);
    const bool has1 = !SPLIT || rows_touch(it, tok0, B), has2 = SPLIT && rows_touch(it, tok0 + B, B);
    const bool valid = (!has1 || (pb >= 0 && pb < p.num_blocks)) && (!has2 || (pb2 >= 0 && pb2 < p.num_blocks));
    const int stage = k % NS;
    valid_mask = valid ? (valid_mask | (1u << stage)) : (valid_mask & ~(1u << stage));
    if (lane == 0) {
      uint64_t* bar = &bars[stage];
      uint8_t* dst = ring + stage * S::SLAB_BYTES;
      if (valid && !SPLIT) {
        const int y = (pb * p.num_kv_heads + it.hkv) * B + tok0 % B;  // first row
        mbar_arrive_expect_tx(bar, S::SLAB_BYTES);
        tma_load_3d(dst, &tmap_k, 0, y, 0, bar);
        tma_load_3d(dst + S::TILE_BYTES, &tmap_v, 0, y, 0, bar);
      } else if (valid) {
        // rows 8u .. 8u + 7 come from block u; those of a half that no row sees keep what they held: masked
        mbar_arrive_expect_tx(bar, (has1 ? S::SLAB_BYTES / 2 : 0) + (has2 ? S::SLAB_BYTES / 2 : 0));
        for (int u = has1 ? 0 : 1; u < (has2 ? 2 : 1); ++u) {
          const int y = ((u ? pb2 : pb) * p.num_kv_heads + it.hkv) * B;
          tma_load_3d(dst + u * (S::TILE_BYTES / 2), &tmap_k, 0, y, 0, bar);
          tma_load_3d(dst + S::TILE_BYTES + u * (S::TILE_BYTES / 2), &tmap_v, 0, y, 0, bar);
        }
      } else {
        report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
        mbar_arrive(bar);  // complete the phase without data; the slab is skipped
      }
    }
  };
  // test hook (pa_decode_options.test_flags): slab 0 of each ring is never requested and the first wait has a
  // short bound, so that wait expires and the abort path below runs
  const int first_issued = p.test_expire_first_wait ? 1 : 0;
  for (int k = first_issued; k < min(n_my, NS); ++k) issue(k);

  // ---- query fragments (B operand of S^T = K Q^T): row g, dims 16j + 2q4 (+ 8)
  uint32_t qf[S::KSTEPS][2];
  {
    const bool real = g < it.gcount;
    const uint32_t* qrow =
        reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + rows_offset(p, it, real ? g : 0) * D);
#pragma unroll
    for (int j = 0; j < S::KSTEPS; ++j) {
      qf[j][0] = real ? __ldg(qrow + (16 * j + 2 * q4) / 2) : 0u;
      qf[j][1] = real ? __ldg(qrow + (16 * j + 2 * q4 + 8) / 2) : 0u;
    }
  }
  // this lane's two rows: positions and ALiBi slopes in log2 units (0: no bias); rows past the item are
  // computed with the last row's position and not written
  const int ra = min(2 * q4, it.gcount - 1), rb = min(2 * q4 + 1, it.gcount - 1);
  const int pos_a = it.base + (it.row0 + ra) / it.G, pos_b = it.base + (it.row0 + rb) / it.G;
  float bias_a = 0.f, bias_b = 0.f;
  if (p.alibi != nullptr) {
    constexpr float kLog2e = 1.4426950408889634f;
    bias_a = __ldg(p.alibi + it.hkv * it.G + (it.row0 + ra) % it.G) * kLog2e;
    bias_b = __ldg(p.alibi + it.hkv * it.G + (it.row0 + rb) % it.G) * kLog2e;
  }

  // The step's append (one query row per sequence): the new token sits at position L - 1, in the list's last
  // slab.  The warp that takes it starts copying the token's rows into the stage.
  uint8_t* stage_rows = smem + S::STAGE_OFF;
  constexpr int CH = D * (int)sizeof(T) / 16;  // 16-byte chunks per row
  const int app_tok = p.new_k != nullptr ? it.L - 1 : -1;
  if (p.new_k != nullptr && n_my > 0 && slab_tok(n_my - 1) == app_tok / S::SB * S::SB && lane < 2 * CH) {
    const size_t row = (size_t)it.s * p.num_kv_heads + it.hkv;
    const void* src = static_cast<const uint4*>(lane >= CH ? p.new_v : p.new_k) + row * CH + lane % CH;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.commit_group;" ::"r"(
                     smem_u32(stage_rows + 16 * lane)),
                 "l"(src)
                 : "memory");
  }

  float o[S::KSTEPS][4];
#pragma unroll
  for (int i = 0; i < S::KSTEPS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m_a = -INFINITY, m_b = -INFINITY;  // running max (log2 units) of rows 2q4, 2q4 + 1
  float l_a = 0.f, l_b = 0.f;              // this lane's share of the running sums
  int k = 0;
  for (; k < n_my; ++k) {
    const int stage = k % NS;
    const long long limit = (k == 0 && p.test_expire_first_wait) ? kRowsTestWaitCycles : kRowsWaitCycles;
    if (!__all_sync(0xffffffffu, rows_wait(&bars[stage], (k / NS) & 1, abort_flag, limit))) break;
    if ((valid_mask >> stage) & 1u) {
      const int tok0 = slab_tok(k);
      uint8_t* kst = ring + stage * S::SLAB_BYTES;
      if (app_tok >= tok0 && app_tok < tok0 + S::SB) {
        // the token's rows replace those of its slot in the tiles; the CTA of the kv head's first rows also
        // stores them into the caches (lane l moves chunk l % CH of the key or the value)
        if (lane < 2 * CH) {
          const bool is_v = lane >= CH;
          const int c = lane % CH, r = app_tok - tok0;
          asm volatile("cp.async.wait_all;" ::: "memory");
          const uint4 x = *reinterpret_cast<const uint4*>(stage_rows + 16 * lane);
          *reinterpret_cast<uint4*>(kst + (is_v ? S::TILE_BYTES : 0) + tile_chunk<D, SPLIT>(r, c)) = x;
          if (it.row0 == 0) {
            const int pb = __ldg(table + app_tok / B);  // in the pool: the slab is valid
            const size_t dst = (((size_t)pb * p.num_kv_heads + it.hkv) * B + app_tok % B) * CH + c;
            static_cast<uint4*>(is_v ? p.v_cache_out : p.k_cache_out)[dst] = x;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the async proxy refills the buffer
        }
        __syncwarp();
      }
      window_slab<T, D, SPLIT>(kst, kst + S::TILE_BYTES, tok0, it, qf, o, m_a, m_b, l_a, l_b, lane, p.scale_log2,
                               bias_a, bias_b, pos_a, pos_b, p.window);
    }
    __syncwarp();
    if (k + NS < n_my) issue(k + NS);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // the staged rows' copy, if its slab was skipped
  if (k < n_my) {  // timed out: let this warp's copies already in flight land first
    if (lane == 0) {
      report_error(p.err_flag, PA_DEVERR_TIMEOUT);
      for (int kk = max(k, first_issued); kk < min(n_my, k + NS); ++kk) drain_phase(&bars[kk % NS], (kk / NS) & 1);
    }
    __syncwarp();
  }

  // ---- per-warp totals into the warp's (now idle) ring, then merge the warps and the cluster
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l_a += __shfl_xor_sync(0xffffffffu, l_a, off);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, off);
  }
  float* wo = reinterpret_cast<float*>(ring);  // [8 rows][OROW], then [8 rows][2]
  float* wml = wo + 8 * S::OROW;
#pragma unroll
  for (int i = 0; i < S::KSTEPS; ++i) {
    wo[(2 * q4) * S::OROW + 16 * i + g] = o[i][0];
    wo[(2 * q4 + 1) * S::OROW + 16 * i + g] = o[i][1];
    wo[(2 * q4) * S::OROW + 16 * i + g + 8] = o[i][2];
    wo[(2 * q4 + 1) * S::OROW + 16 * i + g + 8] = o[i][3];
  }
  if (g == 0) {
    wml[(2 * q4) * 2] = m_a;
    wml[(2 * q4) * 2 + 1] = l_a;
    wml[(2 * q4 + 1) * 2] = m_b;
    wml[(2 * q4 + 1) * 2 + 1] = l_b;
  }
  __syncthreads();
  rows_finish<T, D, NW, S::OROW, S::RING_BYTES / 4>(p, it, reinterpret_cast<const float*>(smem),
                                                    reinterpret_cast<float*>(smem + S::WT_OFF),
                                                    reinterpret_cast<float*>(smem + S::MINE_OFF));
}

template <typename T, int D, int NW, int NS, bool SPLIT, bool SLOTS>
cudaError_t launch_form(const CUtensorMap& tk, const CUtensorMap& tv, WindowParams p, cudaStream_t stream) {
  using S = RowsShape<D, NW, NS>;
  auto kernel = window_rows_tc_kernel<T, D, NW, NS, SPLIT, SLOTS>;
  static ClusterRoom room;
  cudaError_t e = prepare_rows(kernel, room, S::THREADS, S::SMEM_BYTES, &p.cluster);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, dim3((unsigned)(window_items(p, SLOTS) * p.cluster)), dim3(S::THREADS), S::SMEM_BYTES,
                        p.cluster, true, stream, tk, tv, p);
}

template <typename T, int D, int NW, int NS, bool SPLIT>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, const WindowParams& p, bool slots,
                        cudaStream_t stream) {
  return slots ? launch_form<T, D, NW, NS, SPLIT, true>(tk, tv, p, stream)
               : launch_form<T, D, NW, NS, SPLIT, false>(tk, tv, p, stream);
}

template <typename T, int D, int NS, bool SPLIT>
cudaError_t launch_warps(const CUtensorMap& tk, const CUtensorMap& tv, const WindowParams& p, bool slots,
                         cudaStream_t stream) {
  if (p.warps == 3) return launch_rows<T, D, 3, NS, SPLIT>(tk, tv, p, slots, stream);
  if (p.warps == 4) return launch_rows<T, D, 4, NS, SPLIT>(tk, tv, p, slots, stream);
  if (p.warps == 6) return launch_rows<T, D, 6, NS, SPLIT>(tk, tv, p, slots, stream);
  return cudaErrorInvalidValue;
}

// two slabs a warp (four of head size 64): a deeper ring leaves fewer warps an SM and gained nothing
template <typename T>
cudaError_t launch_type(int head_size, const CUtensorMap& tk, const CUtensorMap& tv, const WindowParams& p,
                        bool slots, cudaStream_t stream) {
  const bool split = p.block_size < kTcSlabTokens;
  if (head_size == 128)
    return split ? launch_warps<T, 128, 2, true>(tk, tv, p, slots, stream)
                 : launch_warps<T, 128, 2, false>(tk, tv, p, slots, stream);
  if (head_size == 64)
    return split ? launch_warps<T, 64, 4, true>(tk, tv, p, slots, stream)
                 : launch_warps<T, 64, 4, false>(tk, tv, p, slots, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_window_rows_tc(int dtype, int head_size, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const WindowParams& p, bool slots, cudaStream_t stream) {
  if (dtype == PA_F16) return launch_type<__half>(head_size, tk, tv, p, slots, stream);
  if (dtype == PA_BF16) return launch_type<__nv_bfloat16>(head_size, tk, tv, p, slots, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
