// pa_fp4_rows.cu - attention of a few query rows over a cache held in 4 bits: the decode step and short chunks (see
// pa_window_rows.cuh for the rows, the visible slabs and the split).
//
// A code times its group's scale is exact in fp16, so both contractions run on mma.m16n8k16 in fp16 with fp32
// accumulation; the cache's unit is folded into the softmax scale (keys) and the output (values).  Queries in bf16 go in
// as fp16 after each row has been scaled by a power of two that brings its largest element into [1, 2): what lies
// more than 2^-14 below that loses bits, by at most 2^-25 of the largest element.
//
// Fragments.  A row's order of dimensions inside the S contraction is free, so thread (g, c) = (lane / 4, lane % 4)
// takes the 16 bytes with dimensions 32 c .. 32 c + 31 of its key row, two whole groups, with one load, and the query
// fragments follow.  For P V the thread takes group g, dimensions 16 g .. 16 g + 15, of four tokens: rows g and g + 8 of
// m-tile i are dimensions 16 g + 2 i and + 1.  An A fragment wants the same dimension of two tokens side by side: the two
// tokens' bytes (two dimensions each) exchange nibbles before they are converted, 4 operations for 16 elements.
// Row r of the S tile is token pi(r), so that the transposed P finds thread c's tokens c, (c ^ 1) + 4 and those + 8:
// rows that are neighbours in the tile lie in different halves of the banks for both products.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "pa.h"
#include "pa_fp4.cuh"
#include "pa_window_rows.cuh"

namespace pa {
namespace {

template <int NW, int NS>
struct RowsFp4Shape {
  static constexpr int D = kFp4D;
  static constexpr int SUBS = 2;                           // tiles of a slab, each inside one block
  static constexpr int SB = SUBS * kFp4Tokens;             // tokens of a slab
  static constexpr int HALF = SUBS * kFp4TileBytes;        // the slab's keys; its values follow
  static constexpr int SLAB_BYTES = 2 * HALF;
  static constexpr int RING_BYTES = NS * SLAB_BYTES;       // per warp
  static constexpr int OROW = D + 4;
  static constexpr int BAR_OFF = NW * RING_BYTES;
  static constexpr int FLAG_OFF = BAR_OFF + NW * NS * 8;
  static constexpr int STAGE_OFF = (FLAG_OFF + 4 + 15) / 16 * 16;  // the appended token's 16-bit K and V rows
  static constexpr int MINE_OFF = STAGE_OFF + 4 * D;
  static constexpr int WT_OFF = MINE_OFF + (8 * D + 16) * 4;
  static constexpr int SMEM_BYTES = WT_OFF + (8 * NW + 16) * 4 + 128;
  static constexpr int THREADS = NW * 32;
  static_assert(RING_BYTES >= (8 * OROW + 16) * 4, "a warp's ring holds its partial result at the end");
  static_assert(RING_BYTES % 16 == 0 && NS <= 32, "copies are 16-byte aligned; a bit a stage");
};

// token of the S MMA's A row r (see the file comment)
__device__ __forceinline__ int token_of(int r) {
  const int x = r & 7;
  return (r & 8) + ((x & 1) ? ((x >> 1) ^ 1) + 4 : x >> 1);
}

// One slab: kst the key tiles, vst the value tiles.  sl2a, sl2b: score scale of rows 2c and 2c + 1 (log2 units).
template <int SUBS>
__device__ __forceinline__ void fp4_slab(const uint8_t* kst, const uint8_t* vst, int tok0, const RowsItem& it,
                                         const uint32_t (&qf)[8][2], float (&o)[8][4], float& m_a, float& m_b, float& l_a,
                                         float& l_b, int lane, float sl2a, float sl2b, float bias_a, float bias_b,
                                         int pos_a, int pos_b, int window) {
  const int g = lane >> 2, c = lane & 3, row = token_of(g);
  float sc[SUBS][4];
#pragma unroll
  for (int u = 0; u < SUBS; ++u) {
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
    const uint8_t* t = kst + u * kFp4TileBytes;
    const uint4 lo = *reinterpret_cast<const uint4*>(t + row * kFp4RowBytes + 16 * c);
    const uint4 hi = *reinterpret_cast<const uint4*>(t + (row + 8) * kFp4RowBytes + 16 * c);
    const uint8_t* s = t + kFp4CodeBytes + 2 * c;
    const uint32_t slo = fp4_scales_to_half(*reinterpret_cast<const uint16_t*>(s + row * kFp4RowScales));
    const uint32_t shi = fp4_scales_to_half(*reinterpret_cast<const uint16_t*>(s + (row + 8) * kFp4RowScales));
    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // 8 dimensions: two k-steps
      const uint32_t sa = w < 2 ? half_dup_lo(slo) : half_dup_hi(slo), sb = w < 2 ? half_dup_lo(shi) : half_dup_hi(shi);
      uint32_t a[4], b[4];
      fp4_to_half(lw[w], a[0], a[1], a[2], a[3]);
      fp4_to_half(hw[w], b[0], b[1], b[2], b[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = half_mul(a[i], sa), b[i] = half_mul(b[i], sb);
      Mma<__half>::run(x, a[0], b[0], a[1], b[1], qf[2 * w][0], qf[2 * w][1]);
      Mma<__half>::run(y, a[2], b[2], a[3], b[3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[u][i] = x[i] + y[i];
  }
  // scores 4u .. 4u + 3: (token 16u + pi(g), rows a, b), (token 16u + pi(g) + 8, rows a, b)
  const bool full = rows_full(it, tok0, 16 * SUBS);
  float s[4 * SUBS];
#pragma unroll
  for (int u = 0; u < SUBS; ++u) {
    const int t_lo = tok0 + 16 * u + row, t_hi = t_lo + 8;
    s[4 * u] = fmaf(bias_a, (float)(t_lo - pos_a), sc[u][0] * sl2a);
    s[4 * u + 1] = fmaf(bias_b, (float)(t_lo - pos_b), sc[u][1] * sl2b);
    s[4 * u + 2] = fmaf(bias_a, (float)(t_hi - pos_a), sc[u][2] * sl2a);
    s[4 * u + 3] = fmaf(bias_b, (float)(t_hi - pos_b), sc[u][3] * sl2b);
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
#pragma unroll
  for (int u = 0; u < SUBS; ++u) {
    const uint32_t x0 = Mma<__half>::pack(fast_exp2(s[4 * u] - sub_a), fast_exp2(s[4 * u + 1] - sub_b));
    const uint32_t x1 = Mma<__half>::pack(fast_exp2(s[4 * u + 2] - sub_a), fast_exp2(s[4 * u + 3] - sub_b));
    // the sums use the rounded weights that the value MMA multiplies with
    l_a += Mma<__half>::lo(x0) + Mma<__half>::lo(x1);
    l_b += Mma<__half>::hi(x0) + Mma<__half>::hi(x1);
    const uint32_t p0 = movmatrix_trans(x0), p1 = movmatrix_trans(x1);
    const uint8_t* t = vst + u * kFp4TileBytes;
    // this thread's tokens t0, t1 and those + 8
    const int t0 = c, t1 = (c ^ 1) + 4;
    const uint8_t* sp = t + kFp4CodeBytes + g;
    uint32_t s01 = fp4_scales_to_half(sp[t0 * kFp4RowScales] | (uint32_t)sp[t1 * kFp4RowScales] << 8);
    uint32_t s89 = fp4_scales_to_half(sp[(t0 + 8) * kFp4RowScales] | (uint32_t)sp[(t1 + 8) * kFp4RowScales] << 8);
    if (!full) {  // scales of tokens that no row sees may be NaN: their values are zeros (every code is finite)
      const int at = tok0 + 16 * u;
      s01 &= (rows_any(it, at + t0) ? 0x0000ffffu : 0u) | (rows_any(it, at + t1) ? 0xffff0000u : 0u);
      s89 &= (rows_any(it, at + t0 + 8) ? 0x0000ffffu : 0u) | (rows_any(it, at + t1 + 8) ? 0xffff0000u : 0u);
    }
    const uint8_t* vp = t + 8 * g;
    const uint2 va = *reinterpret_cast<const uint2*>(vp + t0 * kFp4RowBytes);
    const uint2 vb = *reinterpret_cast<const uint2*>(vp + t1 * kFp4RowBytes);
    const uint2 vc = *reinterpret_cast<const uint2*>(vp + (t0 + 8) * kFp4RowBytes);
    const uint2 vd = *reinterpret_cast<const uint2*>(vp + (t1 + 8) * kFp4RowBytes);
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // 8 dimensions: four m-tiles
      const uint32_t a = w ? va.y : va.x, b = w ? vb.y : vb.x, cc = w ? vc.y : vc.x, d = w ? vd.y : vd.x;
      uint32_t e0[4], o0[4], e1[4], o1[4];  // even and odd dimensions of the tokens (t0, t1), and of those + 8
      fp4_to_half((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), e0[0], e0[1], e0[2], e0[3]);
      fp4_to_half(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), o0[0], o0[1], o0[2], o0[3]);
      fp4_to_half((cc & 0x0f0f0f0fu) | ((d << 4) & 0xf0f0f0f0u), e1[0], e1[1], e1[2], e1[3]);
      fp4_to_half(((cc >> 4) & 0x0f0f0f0fu) | (d & 0xf0f0f0f0u), o1[0], o1[1], o1[2], o1[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        Mma<__half>::run(o[4 * w + i], half_mul(e0[i], s01), half_mul(o0[i], s01), half_mul(e1[i], s89),
                         half_mul(o1[i], s89), p0, p1);
    }
  }
}

// Lane l: elements 4l .. 4l + 3 of an appended row as codes (2 bytes), and the scale of their group: the bytes that the
// append call writes.
template <typename T>
__device__ __forceinline__ void quantise_row(uint2 h, float unit, uint32_t& codes, uint32_t& scale) {
  const float x[8] = {Mma<T>::lo(h.x), Mma<T>::hi(h.x), Mma<T>::lo(h.y), Mma<T>::hi(h.y), 0.f, 0.f, 0.f, 0.f};
  float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  scale = fp4_scale_code(amax, __fmul_rn(6.f, unit));
  codes = fp4_codes8(x, fp4_inverse(scale, unit)) & 0xffffu;
}
__device__ __forceinline__ void store_quantised(uint8_t* tile, int r, int lane, uint32_t codes, uint32_t scale) {
  *reinterpret_cast<uint16_t*>(tile + r * kFp4RowBytes + 2 * lane) = (uint16_t)codes;
  if (lane % 4 == 0) tile[kFp4CodeBytes + r * kFp4RowScales + lane / 4] = (uint8_t)scale;
}

template <typename T, int NW, int NS, bool SLOTS>
__global__ void __launch_bounds__(RowsFp4Shape<NW, NS>::THREADS) fp4_rows_kernel(const WindowParams p) {
  using S = RowsFp4Shape<NW, NS>;
  constexpr int D = S::D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * S::RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF) + warp * NS;
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + S::FLAG_OFF);
  const int B = p.block_size;
  const bool whole = B % S::SB == 0;  // a slab lies in one block: its tiles are one run
  if (threadIdx.x == 0) abort_flag[0] = 0;
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
  const int mine = it.v1 - it.v0;
  const int n_my = mine > warp ? (mine - warp + NW - 1) / NW : 0;
  const uint8_t* k_cache = static_cast<const uint8_t*>(p.k_cache);
  const uint8_t* v_cache = static_cast<const uint8_t*>(p.v_cache);
  const int32_t* table = p.block_tables + (size_t)it.s * p.max_blocks;
  auto slab_tok = [&](int k) { return rows_slab(it, it.v0 + warp + k * NW) * S::SB; };
  // does tile u of the slab at tok0 have to be loaded (a whole slab: with the others)?
  auto wanted = [&](int tok0, int u) { return rows_touch(it, tok0 + u * kFp4Tokens, kFp4Tokens); };
  // lane l holds the table entries of the tiles of slab 32 b + l (-1: not wanted)
  auto fetch = [&](int k, int (&e)[S::SUBS]) {
#pragma unroll
    for (int u = 0; u < S::SUBS; ++u) e[u] = -1;
    if (k < n_my) {
      const int tok0 = slab_tok(k);
#pragma unroll
      for (int u = 0; u < S::SUBS; ++u)
        if (whole ? u == 0 : wanted(tok0, u)) e[u] = __ldg(table + (tok0 + u * kFp4Tokens) / B);
    }
  };
  int pb_batch = 0, pb_reg[S::SUBS];
  fetch(lane, pb_reg);

  uint32_t valid_mask = 0;
  auto issue = [&](int k) {  // the whole warp, k increasing
    if ((k >> 5) != pb_batch) {
      pb_batch = k >> 5;
      fetch(k + lane, pb_reg);
    }
    const int tok0 = slab_tok(k), stage = k % NS;
    int pb[S::SUBS];
    bool has[S::SUBS], valid = true;
    uint32_t tiles = 0;
#pragma unroll
    for (int u = 0; u < S::SUBS; ++u) {
      pb[u] = __shfl_sync(0xffffffffu, pb_reg[u], k & 31);
      has[u] = whole ? u == 0 : wanted(tok0, u);
      valid = valid && (!has[u] || (pb[u] >= 0 && pb[u] < p.num_blocks));
      tiles += has[u] ? 1 : 0;
    }
    valid_mask = valid ? (valid_mask | (1u << stage)) : (valid_mask & ~(1u << stage));
    if (lane == 0) {
      uint64_t* bar = &bars[stage];
      uint8_t* dst = ring + stage * S::SLAB_BYTES;
      if (valid) {
        const uint32_t bytes = whole ? (uint32_t)S::HALF : (uint32_t)kFp4TileBytes;
        mbar_arrive_expect_tx(bar, 2 * tiles * bytes);
        // (a tile that no row sees keeps what its place held: masked)
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) {
          if (has[u]) {
            const size_t at = fp4_tile(pb[u], p.num_kv_heads, it.hkv, B, (tok0 + u * kFp4Tokens) % B);
            bulk_load_1d(dst + u * kFp4TileBytes, k_cache + at, bytes, bar);
            bulk_load_1d(dst + S::HALF + u * kFp4TileBytes, v_cache + at, bytes, bar);
          }
        }
      } else {
        report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
        mbar_arrive(bar);
      }
    }
  };
  const int first_issued = p.test_expire_first_wait ? 1 : 0;  // test hook: see pa_decode_options.test_flags
  for (int k = first_issued; k < min(n_my, NS); ++k) issue(k);

  // ---- query fragments: k-step w, slots (2c, 2c + 1 | 2c + 8, 2c + 9) <- dimensions 32c + 4w .. + 3
  uint32_t qf[8][2];
  float q_unit = 1.f;  // row g's fragments times this are the query
  {
    const bool real = g < it.gcount;
    const uint4* qrow = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + rows_offset(p, it, real ? g : 0) * D + 32 * c);
    uint32_t x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = real ? __ldg(qrow + i) : make_uint4(0, 0, 0, 0);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
    if constexpr (!std::is_same<T, __half>::value) {
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fmaxf(fabsf(Mma<T>::lo(x[i])), fabsf(Mma<T>::hi(x[i]))));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      float inv;
      row_power(mx, q_unit, inv);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = Mma<__half>::pack(Mma<T>::lo(x[i]) * inv, Mma<T>::hi(x[i]) * inv);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) qf[i][0] = x[2 * i], qf[i][1] = x[2 * i + 1];
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
  const float sl2 = p.scale_log2 * p.k_scale;  // scores of the stored numbers, in log2 units
  const float sl2a = sl2 * __shfl_sync(0xffffffffu, q_unit, 8 * c), sl2b = sl2 * __shfl_sync(0xffffffffu, q_unit, 8 * c + 4);

  // the step's append: the warp of the list's last slab starts copying the new token's rows (lanes 0..15 the key,
  // 16..31 the value, 16 bytes each)
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

  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
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
        // the token's bytes replace those of its slot in the tiles; the CTA of the kv head's first rows also stores
        // them into the caches
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        uint32_t kc, ks, vc, vs;
        quantise_row<T>(*reinterpret_cast<const uint2*>(stage_rows + 8 * lane), p.k_scale, kc, ks);
        quantise_row<T>(*reinterpret_cast<const uint2*>(stage_rows + 2 * D + 8 * lane), p.v_scale, vc, vs);
        const int u = (app_tok - tok0) / kFp4Tokens, r = app_tok % kFp4Tokens;
        store_quantised(kst + u * kFp4TileBytes, r, lane, kc, ks);
        store_quantised(kst + S::HALF + u * kFp4TileBytes, r, lane, vc, vs);
        if (it.row0 == 0) {  // the block is in the pool: the slab is valid
          const size_t at = fp4_tile(__ldg(table + app_tok / B), p.num_kv_heads, it.hkv, B, app_tok % B);
          store_quantised(static_cast<uint8_t*>(p.k_cache_out) + at, r, lane, kc, ks);
          store_quantised(static_cast<uint8_t*>(p.v_cache_out) + at, r, lane, vc, vs);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the async proxy refills the buffer
        __syncwarp();
      }
      fp4_slab<S::SUBS>(kst, kst + S::HALF, tok0, it, qf, o, m_a, m_b, l_a, l_b, lane, sl2a, sl2b, bias_a, bias_b, pos_a,
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
  for (int i = 0; i < 8; ++i) {
    float* at = wo + 16 * g + 2 * i;
    *reinterpret_cast<float2*>(at + (2 * c) * S::OROW) = make_float2(o[i][0] * p.v_scale, o[i][2] * p.v_scale);
    *reinterpret_cast<float2*>(at + (2 * c + 1) * S::OROW) = make_float2(o[i][1] * p.v_scale, o[i][3] * p.v_scale);
  }
  if (g == 0) {
    wml[(2 * c) * 2] = m_a;
    wml[(2 * c) * 2 + 1] = l_a;
    wml[(2 * c + 1) * 2] = m_b;
    wml[(2 * c + 1) * 2 + 1] = l_b;
  }
  __syncthreads();
  rows_finish<T, D, NW, S::OROW, S::RING_BYTES / 4>(p, it, reinterpret_cast<const float*>(smem),
                                                    reinterpret_cast<float*>(smem + S::WT_OFF),
                                                    reinterpret_cast<float*>(smem + S::MINE_OFF));
}

constexpr int kStages = 3;

template <typename T, int NW, bool SLOTS>
cudaError_t launch_form(WindowParams p, cudaStream_t stream) {
  using S = RowsFp4Shape<NW, kStages>;
  auto kernel = fp4_rows_kernel<T, NW, kStages, SLOTS>;
  static ClusterRoom room;
  cudaError_t e = prepare_rows(kernel, room, S::THREADS, S::SMEM_BYTES, &p.cluster);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, dim3((unsigned)(window_items(p, SLOTS) * p.cluster)), dim3(S::THREADS), S::SMEM_BYTES,
                        p.cluster, true, stream, p);
}

template <typename T>
cudaError_t launch_type(const WindowParams& p, bool slots, cudaStream_t stream) {
  if (p.warps == 3) return slots ? launch_form<T, 3, true>(p, stream) : launch_form<T, 3, false>(p, stream);
  if (p.warps == 4) return slots ? launch_form<T, 4, true>(p, stream) : launch_form<T, 4, false>(p, stream);
  if (p.warps == 6) return slots ? launch_form<T, 6, true>(p, stream) : launch_form<T, 6, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_fp4_rows(int row_dtype, const WindowParams& p, bool slots, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_type<__half>(p, slots, stream) : launch_type<__nv_bfloat16>(p, slots, stream);
}

}  // namespace pa
