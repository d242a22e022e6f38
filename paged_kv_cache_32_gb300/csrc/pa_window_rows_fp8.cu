// pa_window_rows_fp8.cu - attention of a few query rows over a window of an FP8
// (E4M3) cache: the decode step and chunks of new tokens (see pa_window_rows.cuh
// for the rows, the visible slabs and the split).
//
// Key code c stands for k_scale * e4m3(c) and value code c for v_scale * e4m3(c);
// queries and outputs are fp16.  k_scale is folded into the softmax scale,
// v_scale into the output.  The structure is that of the 16-bit kernel with
// slabs of 32 tokens (two sub-slabs of 16, each inside one block: one 2 KB key
// box and one 2 KB run of values).  The codes convert exactly to fp16, so both
// contractions run on mma.m16n8k16 in fp16.  A 32-bit ldmatrix element holds
// four codes, which fixes the k order inside an MMA (slots 2c, 2c + 1, 2c + 8,
// 2c + 9 <- elements 4c .. 4c + 3): the query fragments are loaded in that order,
// and the key rows are read in the order tau so that after the transpose of P
// every weight lands in the slot of its token.  Bound by the conversions and
// MMAs as much as by HBM (one byte an element): the weights stay one fp16 term.
// 96 sequences, 32 / 8 heads, the last 8192 of up to 40000 tokens: 238 us, 5.9 TB/s.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "pa.h"
#include "pa_fp8.cuh"
#include "pa_window_rows.cuh"

namespace pa {
namespace {

template <int D, int NW, int NS>
struct RowsFp8Shape {
  static constexpr int SUB = kTcSlabTokens;               // tokens of a sub-slab (inside one block)
  static constexpr int SB = 2 * SUB;                      // tokens of a slab
  static constexpr int KBOX = SUB * D;                    // key box: 16 rows x D bytes
  static constexpr int VBOX = D * SUB;                    // values: D rows x 16 bytes, contiguous
  static constexpr int SLAB_BYTES = 2 * (KBOX + VBOX);    // keys of both sub-slabs, then their values
  static constexpr int RING_BYTES = NS * SLAB_BYTES;      // per warp
  static constexpr int OROW = D + 4;
  static constexpr int BAR_OFF = NW * RING_BYTES;
  static constexpr int FLAG_OFF = BAR_OFF + NW * NS * 8;
  static constexpr int STAGE_OFF = FLAG_OFF + 16;         // the appended token's fp16 K and V rows
  static constexpr int MINE_OFF = STAGE_OFF + 4 * D;
  static constexpr int WT_OFF = MINE_OFF + (8 * D + 16) * 4;
  static constexpr int SMEM_BYTES = WT_OFF + (8 * NW + 16) * 4 + 1024;
  static constexpr int THREADS = NW * 32;
  static_assert(D == 128, "a key is one 128-byte swizzle row");
  static_assert(RING_BYTES >= (8 * OROW + 16) * 4, "a warp's ring holds its partial result at the end");
};

// key row of the S MMA's A row r (see the file comment)
__device__ __forceinline__ int key_row(int r) {
  return r < 8 ? 4 * (r >> 1) + (r & 1) : 4 * ((r - 8) >> 1) + 2 + (r & 1);
}

template <int D>
__device__ __forceinline__ void window_slab_fp8(const uint8_t* kst, const uint8_t* vst, int tok0, const RowsItem& it,
                                                const uint32_t (&qf)[D / 16][2], float (&o)[D / 16][4], float& m_a,
                                                float& m_b, float& l_a, float& l_b, int lane, float sl2, float bias_a,
                                                float bias_b, int pos_a, int pos_b, int window) {
  constexpr int KBOX = 16 * D, VBOX = D * 16;
  const int g = lane >> 2, c = lane & 3;
  float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  float sd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  {
    const int mi = lane >> 3;
    const int krow = key_row((lane & 7) + 8 * (mi & 1));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {  // 32 dimensions = two k-steps per ldmatrix.x4
        uint32_t r0, r1, r2, r3;
        ldmatrix_x4(smem_u32(kst + u * KBOX) + swz128(krow, 2 * j + (mi >> 1)), r0, r1, r2, r3);
        uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
        codes_to_half(r0, a0, a2);
        codes_to_half(r1, a1, a3);
        codes_to_half(r2, b0, b2);
        codes_to_half(r3, b1, b3);
        Mma<__half>::run(sc[u], a0, a1, a2, a3, qf[2 * j][0], qf[2 * j][1]);
        Mma<__half>::run(sd[u], b0, b1, b2, b3, qf[2 * j + 1][0], qf[2 * j + 1][1]);
      }
    }
  }
  // scores 4u .. 4u + 3: (token 16u + tau(g), rows a, b), (token 16u + tau(g + 8), rows a, b)
  const bool full = rows_full(it, tok0, 32);
  float s[8];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t_lo = tok0 + 16 * u + key_row(g), t_hi = tok0 + 16 * u + key_row(g + 8);
    s[4 * u] = fmaf(bias_a, (float)(t_lo - pos_a), (sc[u][0] + sd[u][0]) * sl2);
    s[4 * u + 1] = fmaf(bias_b, (float)(t_lo - pos_b), (sc[u][1] + sd[u][1]) * sl2);
    s[4 * u + 2] = fmaf(bias_a, (float)(t_hi - pos_a), (sc[u][2] + sd[u][2]) * sl2);
    s[4 * u + 3] = fmaf(bias_b, (float)(t_hi - pos_b), (sc[u][3] + sd[u][3]) * sl2);
    if (!full) {
      auto sees = [&](int t, int pos) { return t <= pos && (t > pos - window || t < it.sinks); };
      if (!sees(t_lo, pos_a)) s[4 * u] = -INFINITY;
      if (!sees(t_lo, pos_b)) s[4 * u + 1] = -INFINITY;
      if (!sees(t_hi, pos_a)) s[4 * u + 2] = -INFINITY;
      if (!sees(t_hi, pos_b)) s[4 * u + 3] = -INFINITY;
    }
  }
  float sub_a, sub_b;
  rows_softmax_max(s, o, m_a, m_b, l_a, l_b, sub_a, sub_b);
  uint32_t pb[2][2];
  uint32_t m_lo[2] = {0xffffffffu, 0xffffffffu}, m_hi[2] = {0xffffffffu, 0xffffffffu};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t x0 = Mma<__half>::pack(fast_exp2(s[4 * u] - sub_a), fast_exp2(s[4 * u + 1] - sub_b));
    const uint32_t x1 = Mma<__half>::pack(fast_exp2(s[4 * u + 2] - sub_a), fast_exp2(s[4 * u + 3] - sub_b));
    // the sums use the rounded weights that the value MMA multiplies with
    l_a += Mma<__half>::lo(x0) + Mma<__half>::lo(x1);
    l_b += Mma<__half>::hi(x0) + Mma<__half>::hi(x1);
    pb[u][0] = movmatrix_trans(x0);
    pb[u][1] = movmatrix_trans(x1);
    if (!full) {  // values of tokens that no row sees may be NaN codes: zero them
      const int t0 = tok0 + 16 * u + 4 * c;
      m_lo[u] = (rows_any(it, t0) ? 0x0000ffffu : 0u) | (rows_any(it, t0 + 1) ? 0xffff0000u : 0u);
      m_hi[u] = (rows_any(it, t0 + 2) ? 0x0000ffffu : 0u) | (rows_any(it, t0 + 3) ? 0xffff0000u : 0u);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t r0, r1, r2, r3;
      ldmatrix_x4(smem_u32(vst + u * VBOX) + (32 * i + lane) * 16, r0, r1, r2, r3);
      // m-tile 2i: dimensions 32i + g (r0) and 32i + 8 + g (r1); m-tile 2i + 1: r2, r3
      uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
      codes_to_half(r0, a0, a2);
      codes_to_half(r1, a1, a3);
      codes_to_half(r2, b0, b2);
      codes_to_half(r3, b1, b3);
      if (!full) {
        a0 &= m_lo[u], a1 &= m_lo[u], b0 &= m_lo[u], b1 &= m_lo[u];
        a2 &= m_hi[u], a3 &= m_hi[u], b2 &= m_hi[u], b3 &= m_hi[u];
      }
      Mma<__half>::run(o[2 * i], a0, a1, a2, a3, pb[u][0], pb[u][1]);
      Mma<__half>::run(o[2 * i + 1], b0, b1, b2, b3, pb[u][0], pb[u][1]);
    }
  }
}

// E4M3 codes of four fp16 values over `scale` (fp32 division, ties to even, saturating), as the quantising append
__device__ __forceinline__ uint32_t quantise4(uint2 h, float scale) {
  const __half2 a = *reinterpret_cast<const __half2*>(&h.x), b = *reinterpret_cast<const __half2*>(&h.y);
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(__low2float(a), scale), __fdiv_rn(__high2float(a), scale)), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(__low2float(b), scale), __fdiv_rn(__high2float(b), scale)), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int D, int NW, int NS, bool SLOTS>
__global__ void __launch_bounds__(RowsFp8Shape<D, NW, NS>::THREADS)
    window_rows_fp8_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_k32,
                           const WindowParams p) {
  using S = RowsFp8Shape<D, NW, NS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * S::RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF) + warp * NS;
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + S::FLAG_OFF);
  const int B = p.block_size;
  // B a multiple of 32: a slab lies in one block, so one 32-row key box and one 4 KB run of values fetch it
  const bool whole = B % S::SB == 0;
  if (threadIdx.x == 0) {
    abort_flag[0] = 0;
    tma_prefetch_descriptor(whole ? &tmap_k32 : &tmap_k);
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
    rows_zero<__half, D>(p, it);
    return;
  }
  const int mine = it.v1 - it.v0;
  const int n_my = mine > warp ? (mine - warp + NW - 1) / NW : 0;
  const uint8_t* v_cache = static_cast<const uint8_t*>(p.v_cache);
  const int32_t* table = p.block_tables + (size_t)it.s * p.max_blocks;
  auto slab_tok = [&](int k) { return rows_slab(it, it.v0 + warp + k * NW) * S::SB; };
  // does sub-slab u of the slab at tok0 have to be loaded (a whole slab: with the other)?
  auto wanted = [&](int tok0, int u) { return rows_touch(it, tok0 + u * S::SUB, S::SUB); };
  // lane l holds the table entries of both sub-slabs of slab 32 b + l (-1: not wanted)
  auto fetch = [&](int k, int& e0, int& e1) {
    e0 = e1 = -1;
    if (k < n_my) {
      const int tok0 = slab_tok(k);
      if (whole || wanted(tok0, 0)) e0 = __ldg(table + tok0 / B);
      if (!whole && wanted(tok0, 1)) e1 = __ldg(table + (tok0 + S::SUB) / B);
    }
  };
  int pb_batch = 0, pb_reg0, pb_reg1;
  fetch(lane, pb_reg0, pb_reg1);

  uint32_t valid_mask = 0;
  auto issue = [&](int k) {  // the whole warp, k increasing
    if ((k >> 5) != pb_batch) {
      pb_batch = k >> 5;
      fetch(k + lane, pb_reg0, pb_reg1);
    }
    const int pb0 = __shfl_sync(0xffffffffu, pb_reg0, k & 31), pb1 = __shfl_sync(0xffffffffu, pb_reg1, k & 31);
    const int tok0 = slab_tok(k);
    const bool has0 = whole || wanted(tok0, 0), has1 = !whole && wanted(tok0, 1);
    const bool valid = (!has0 || (pb0 >= 0 && pb0 < p.num_blocks)) && (!has1 || (pb1 >= 0 && pb1 < p.num_blocks));
    const int stage = k % NS;
    valid_mask = valid ? (valid_mask | (1u << stage)) : (valid_mask & ~(1u << stage));
    if (lane == 0) {
      uint64_t* bar = &bars[stage];
      uint8_t* dst = ring + stage * S::SLAB_BYTES;
      if (valid && whole) {
        const size_t row = (size_t)(pb0 * p.num_kv_heads + it.hkv) * B + tok0 % B;
        mbar_arrive_expect_tx(bar, S::SLAB_BYTES);
        tma_load_2d(dst, &tmap_k32, 0, (int)row, bar);
        bulk_load_1d(dst + 2 * S::KBOX, v_cache + row * D, 2 * S::VBOX, bar);
      } else if (valid) {
        // (a sub-slab that no row sees keeps what its tiles held: masked)
        mbar_arrive_expect_tx(bar, ((has0 ? 1 : 0) + (has1 ? 1 : 0)) * (S::KBOX + S::VBOX));
        for (int u = has0 ? 0 : 1; u < (has1 ? 2 : 1); ++u) {
          const size_t row =
              (size_t)((u ? pb1 : pb0) * p.num_kv_heads + it.hkv) * B + (tok0 + u * S::SUB) % B;
          tma_load_2d(dst + u * S::KBOX, &tmap_k, 0, (int)row, bar);
          bulk_load_1d(dst + 2 * S::KBOX + u * S::VBOX, v_cache + row * D, S::VBOX, bar);
        }
      } else {
        report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
        mbar_arrive(bar);
      }
    }
  };
  const int first_issued = p.test_expire_first_wait ? 1 : 0;  // test hook: see pa_decode_options.test_flags
  for (int k = first_issued; k < min(n_my, NS); ++k) issue(k);

  // ---- query fragments in the k order of the file comment: slots (2c, 2c + 1 | 2c + 8, 2c + 9) <- 4c .. 4c + 3
  uint32_t qf[D / 16][2];
  {
    const bool real = g < it.gcount;
    const uint32_t* qrow =
        reinterpret_cast<const uint32_t*>(static_cast<const __half*>(p.q) + rows_offset(p, it, real ? g : 0) * D);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      qf[j][0] = real ? __ldg(qrow + (16 * j + 4 * c) / 2) : 0u;
      qf[j][1] = real ? __ldg(qrow + (16 * j + 4 * c + 2) / 2) : 0u;
    }
  }
  // rows past the item are computed with the last row's position and not written
  const int ra = min(2 * c, it.gcount - 1), rb = min(2 * c + 1, it.gcount - 1);
  const int pos_a = it.base + (it.row0 + ra) / it.G, pos_b = it.base + (it.row0 + rb) / it.G;
  float bias_a = 0.f, bias_b = 0.f;
  if (p.alibi != nullptr) {
    constexpr float kLog2e = 1.4426950408889634f;
    bias_a = __ldg(p.alibi + it.hkv * it.G + (it.row0 + ra) % it.G) * kLog2e;
    bias_b = __ldg(p.alibi + it.hkv * it.G + (it.row0 + rb) % it.G) * kLog2e;
  }
  const float sl2 = p.scale_log2 * p.k_scale;  // scores of the stored codes, in log2 units

  // the step's append: the warp of the list's last slab starts copying the new token's fp16 rows (lanes 0..15
  // the key, 16..31 the value, 16 bytes each)
  uint8_t* stage_rows = smem + S::STAGE_OFF;
  const int app_tok = p.new_k != nullptr ? it.L - 1 : -1;
  if (p.new_k != nullptr && n_my > 0 && slab_tok(n_my - 1) == app_tok / S::SB * S::SB) {
    constexpr int CH = D * 2 / 16;
    const size_t row = (size_t)it.s * p.num_kv_heads + it.hkv;
    const void* src = static_cast<const uint4*>(lane >= CH ? p.new_v : p.new_k) + row * CH + lane % CH;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.commit_group;" ::"r"(
                     smem_u32(stage_rows + 16 * lane)),
                 "l"(src)
                 : "memory");
  }

  float o[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m_a = -INFINITY, m_b = -INFINITY;
  float l_a = 0.f, l_b = 0.f;
  int k = 0;
  for (; k < n_my; ++k) {
    const int stage = k % NS;
    const long long limit = (k == 0 && p.test_expire_first_wait) ? kRowsTestWaitCycles : kRowsWaitCycles;
    if (!__all_sync(0xffffffffu, rows_wait(&bars[stage], (k / NS) & 1, abort_flag, limit))) break;
    if ((valid_mask >> stage) & 1u) {
      const int tok0 = slab_tok(k);
      uint8_t* kst = ring + stage * S::SLAB_BYTES;
      if (app_tok >= tok0 && app_tok < tok0 + S::SB) {
        // the token's codes replace those of its slot in the tiles; the CTA of the kv head's first rows also
        // stores them into the caches.  Lane l: dimensions 4l .. 4l + 3
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        const uint32_t kc = quantise4(*reinterpret_cast<const uint2*>(stage_rows + 8 * lane), p.k_scale);
        const uint32_t vc = quantise4(*reinterpret_cast<const uint2*>(stage_rows + 2 * D + 8 * lane), p.v_scale);
        const int u = (app_tok - tok0) >> 4, rr = (app_tok - tok0) & 15;
        *reinterpret_cast<uint32_t*>(kst + u * S::KBOX + swz128(rr, lane >> 2) + 4 * (lane & 3)) = kc;
        uint8_t* vt = kst + 2 * S::KBOX + u * S::VBOX + rr;
#pragma unroll
        for (int i = 0; i < 4; ++i) vt[(4 * lane + i) * 16] = (uint8_t)(vc >> (8 * i));
        if (it.row0 == 0) {
          const int off = app_tok % B;  // the block is in the pool: the slab is valid
          const size_t head = ((size_t)__ldg(table + app_tok / B) * p.num_kv_heads + it.hkv) * (size_t)B * D;
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.k_cache_out) + head + (size_t)off * D + 4 * lane) = kc;
          uint8_t* vg = static_cast<uint8_t*>(p.v_cache_out) + head + (size_t)(off / 16) * D * 16 + off % 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) vg[(4 * lane + i) * 16] = (uint8_t)(vc >> (8 * i));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the async proxy refills the buffer
        __syncwarp();
      }
      window_slab_fp8<D>(kst, kst + 2 * S::KBOX, tok0, it, qf, o, m_a, m_b, l_a, l_b, lane, sl2, bias_a, bias_b, pos_a,
                         pos_b, p.window);
    }
    __syncwarp();
    if (k + NS < n_my) issue(k + NS);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (k < n_my) {  // timed out: let this warp's copies already in flight land first
    if (lane == 0) {
      report_error(p.err_flag, PA_DEVERR_TIMEOUT);
      for (int kk = max(k, first_issued); kk < min(n_my, k + NS); ++kk) drain_phase(&bars[kk % NS], (kk / NS) & 1);
    }
    __syncwarp();
  }

#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l_a += __shfl_xor_sync(0xffffffffu, l_a, off);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, off);
  }
  float* wo = reinterpret_cast<float*>(ring);
  float* wml = wo + 8 * S::OROW;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    wo[(2 * c) * S::OROW + 16 * i + g] = o[i][0] * p.v_scale;
    wo[(2 * c + 1) * S::OROW + 16 * i + g] = o[i][1] * p.v_scale;
    wo[(2 * c) * S::OROW + 16 * i + g + 8] = o[i][2] * p.v_scale;
    wo[(2 * c + 1) * S::OROW + 16 * i + g + 8] = o[i][3] * p.v_scale;
  }
  if (g == 0) {
    wml[(2 * c) * 2] = m_a;
    wml[(2 * c) * 2 + 1] = l_a;
    wml[(2 * c + 1) * 2] = m_b;
    wml[(2 * c + 1) * 2 + 1] = l_b;
  }
  __syncthreads();
  rows_finish<__half, D, NW, S::OROW, S::RING_BYTES / 4>(p, it, reinterpret_cast<const float*>(smem),
                                                         reinterpret_cast<float*>(smem + S::WT_OFF),
                                                         reinterpret_cast<float*>(smem + S::MINE_OFF));
}

}  // namespace

template <int NW, bool SLOTS>
static cudaError_t launch_form(const CUtensorMap& tk, const CUtensorMap& tk32, WindowParams p, cudaStream_t stream) {
  using S = RowsFp8Shape<128, NW, 2>;
  auto kernel = window_rows_fp8_kernel<128, NW, 2, SLOTS>;
  static ClusterRoom room;
  cudaError_t e = prepare_rows(kernel, room, S::THREADS, S::SMEM_BYTES, &p.cluster);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, dim3((unsigned)(window_items(p, SLOTS) * p.cluster)), dim3(S::THREADS), S::SMEM_BYTES,
                        p.cluster, true, stream, tk, tk32, p);
}

template <int NW>
static cudaError_t launch_warps(const CUtensorMap& tk, const CUtensorMap& tk32, const WindowParams& p, bool slots,
                                cudaStream_t stream) {
  return slots ? launch_form<NW, true>(tk, tk32, p, stream) : launch_form<NW, false>(tk, tk32, p, stream);
}

cudaError_t launch_window_rows_fp8(const CUtensorMap& tk, const CUtensorMap& tk32, const WindowParams& p, bool slots,
                                   cudaStream_t stream) {
  if (p.warps == 3) return launch_warps<3>(tk, tk32, p, slots, stream);
  if (p.warps == 4) return launch_warps<4>(tk, tk32, p, slots, stream);
  if (p.warps == 6) return launch_warps<6>(tk, tk32, p, slots, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
