// pa_fp4_rows.cu - attention of a few query rows over a cache held in 4 bits: the decode step and short chunks (see
// pa_window_rows.cuh for the rows, the visible slabs and the split).
//
// A code times its group's scale is exact in fp16, so both contractions run on mma.m16n8k16 in fp16 with fp32
// accumulation; the cache's unit is folded into the softmax scale (keys) and the normalised output (values).  Queries in bf16 go in
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
//
// Bound by latencies: of 16 tokens (2304 bytes) an SM's share of HBM takes 96 cycles, and some 290 instructions, 64
// conversions and 64 products with scales at half rate among them, take its four schedulers at least 73; sixteen warps
// take about 135, stalled on fixed latencies, the half-rate pipes and one another.  (The copies alone run at 0.87 of the
// copy peak.)
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

constexpr int kFp4Subs = 2;

template <int NW, int NS>
struct RowsFp4Shape {
  static constexpr int D = kFp4D;
  static constexpr int SUBS = kFp4Subs;                    // tiles of a slab, each inside one block
  static constexpr int SB = SUBS * kFp4Tokens;             // tokens of a slab
  static constexpr int HALF = SUBS * kFp4TileBytes;        // the slab's keys; its values follow
  static constexpr int SLAB_BYTES = 2 * HALF;
  static constexpr int RING_BYTES = NS * SLAB_BYTES;       // per warp
  static constexpr int OROW = D + 4;
  static constexpr int BAR_OFF = NW * RING_BYTES;
  static constexpr int FLAG_OFF = BAR_OFF + NW * NS * 8;
  static constexpr int STAGE_OFF = (FLAG_OFF + 4 + 15) / 16 * 16;  // the appended token's 16-bit K and V rows
  static constexpr int WT_OFF = STAGE_OFF + 4 * D;         // weights of the merge; sums of the search for an item
  static constexpr int WT_BYTES = (8 * NW + 16) * 4 < 16 * 16 ? 16 * 16 : (8 * NW + 16) * 4;
  static constexpr int MINE_OFF = WT_OFF + WT_BYTES;       // clusters: this CTA's result
  static constexpr int WALK_OFF = MINE_OFF;                // even deal: where the CTA is
  static constexpr int EVEN_BYTES = WALK_OFF + 64 + 128;
  static constexpr int SMEM_BYTES = MINE_OFF + (8 * D + 16) * 4 + 128;
  static constexpr int THREADS = NW * 32;
  static_assert(RING_BYTES >= (8 * OROW + 16) * 4, "a warp's ring holds its partial result at the end");
  static_assert(RING_BYTES % 16 == 0 && NS <= 32, "copies are 16-byte aligned; a bit a stage");
};

__device__ __forceinline__ __half2 scales_of(uint32_t x) {
  const uint32_t h = fp4_scales_to_half(x);
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ uint32_t times(uint32_t a, __half2 b) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// token of the S MMA's A row r (see the file comment)
__device__ __forceinline__ int token_of(int r) {
  const int x = r & 7;
  return (r & 8) + ((x & 1) ? ((x >> 1) ^ 1) + 4 : x >> 1);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// |x|, or 1 for one too small to divide by
__device__ __forceinline__ float score_scale(float x) { return fabsf(x) >= 7.888609e-31f ? fabsf(x) : 1.f; }  // 2^-100

// One slab: kst the key tiles, vst the value tiles.  sl2a, sl2b > 0: score scale of rows 2c and 2c + 1 (log2 units);
// bias_a, bias_b: their ALiBi slopes in units of raw scores.  o: the
// unnormalised outputs, and in the last entry the rows' sums of weights (one more MMA, by ones).
// kFull: every row sees every token of the slab.  kDecode: the rows are one token's, without ALiBi.
template <int SUBS, bool kFull, bool kDecode>
__device__ __forceinline__ void fp4_slab(const uint8_t* kst, const uint8_t* vst, int tok0, const RowsItem& it,
                                         const uint32_t (&qf)[8][2], float (&o)[9][4], float& m_a, float& m_b, int lane,
                                         float sl2a, float sl2b, bool alibi, float bias_a, float bias_b, int pos_a,
                                         int pos_b, int window) {
  const int g = lane >> 2, c = lane & 3, row = token_of(g);
  float s[4 * SUBS];  // raw scores 4u .. 4u + 3: (token 16u + pi(g), rows a, b), (token 16u + pi(g) + 8, rows a, b)
  const uint8_t* kp = kst + row * kFp4RowBytes + 16 * c;
  const uint8_t* ks = kst + kFp4CodeBytes + row * kFp4RowScales + 2 * c;
#pragma unroll
  for (int u = 0; u < SUBS; ++u) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    const uint4 lo = *reinterpret_cast<const uint4*>(kp + u * kFp4TileBytes);
    const uint4 hi = *reinterpret_cast<const uint4*>(kp + u * kFp4TileBytes + 8 * kFp4RowBytes);
    const __half2 slo = scales_of(*reinterpret_cast<const uint16_t*>(ks + u * kFp4TileBytes));
    const __half2 shi = scales_of(*reinterpret_cast<const uint16_t*>(ks + u * kFp4TileBytes + 8 * kFp4RowScales));
    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // 8 dimensions: two k-steps
      const __half2 sa = w < 2 ? __low2half2(slo) : __high2half2(slo), sb = w < 2 ? __low2half2(shi) : __high2half2(shi);
      uint32_t a[4], b[4];
      fp4_to_half(lw[w], a[0], a[1], a[2], a[3]);
      fp4_to_half(hw[w], b[0], b[1], b[2], b[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = times(a[i], sa), b[i] = times(b[i], sb);
      Mma<__half>::run(x, a[0], b[0], a[1], b[1], qf[2 * w][0], qf[2 * w][1]);
      Mma<__half>::run(x, a[2], b[2], a[3], b[3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[4 * u + i] = x[i];
  }
  if (!kDecode && alibi) {
#pragma unroll
    for (int i = 0; i < 4 * SUBS; ++i) {
      const int t = tok0 + 16 * (i / 4) + row + 8 * ((i >> 1) & 1);
      s[i] = i & 1 ? fmaf(bias_b, (float)(t - pos_b), s[i]) : fmaf(bias_a, (float)(t - pos_a), s[i]);
    }
  }
  if constexpr (!kFull) {
#pragma unroll
    for (int i = 0; i < 4 * SUBS; ++i) {
      const int t = tok0 + 16 * (i / 4) + row + 8 * ((i >> 1) & 1), pos = kDecode ? it.p_last : i & 1 ? pos_b : pos_a;
      if (!(t <= pos && (t > pos - window || t < it.sinks))) s[i] = -INFINITY;
    }
  }
  // a running maximum moves only when a score exceeds it by more than kSlabSlack (log2 units); a NaN score moves none and
  // makes its row's weights NaN
  float mx_a, mx_b;
  if constexpr (SUBS == 1) {
    mx_a = fmaxf(s[0], s[2]), mx_b = fmaxf(s[1], s[3]);
  } else {
    mx_a = max3(s[0], s[2], s[4]), mx_b = max3(s[1], s[3], s[5]);
#pragma unroll
    for (int i = 6; i + 2 < 4 * SUBS; i += 4) mx_a = max3(mx_a, s[i], s[i + 2]), mx_b = max3(mx_b, s[i + 1], s[i + 3]);
    mx_a = fmaxf(mx_a, s[4 * SUBS - 2]), mx_b = fmaxf(mx_b, s[4 * SUBS - 1]);
  }
  if (__any_sync(0xffffffffu, fmaf(mx_a, sl2a, -m_a) > kSlabSlack || fmaf(mx_b, sl2b, -m_b) > kSlabSlack)) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
    }
    const float mn_a = fmaxf(m_a, mx_a * sl2a), mn_b = fmaxf(m_b, mx_b * sl2b);
    // (a row without a token yet has o = 0: any finite factor will do)
    const float al_a = mn_a == -INFINITY ? 1.f : fast_exp2(m_a - mn_a);
    const float al_b = mn_b == -INFINITY ? 1.f : fast_exp2(m_b - mn_b);
    m_a = mn_a;
    m_b = mn_b;
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      o[i][0] *= al_a;
      o[i][1] *= al_b;
      o[i][2] *= al_a;
      o[i][3] *= al_b;
    }
  }
  // weights 2^(shift + s - m); of a row that has seen no token yet scores are masked (-inf) and weigh nothing
  const float sub_a = !kFull && m_a == -INFINITY ? 0.f : kFp4WeightShift - m_a;
  const float sub_b = !kFull && m_b == -INFINITY ? 0.f : kFp4WeightShift - m_b;
  // this thread's tokens t0, t1 and those + 8
  const int t0 = c, t1 = (c ^ 1) + 4;
  const uint8_t* vp = vst + 8 * g;
  const uint8_t* vs = vst + kFp4CodeBytes + g;
  constexpr uint32_t kOnes = 0x3c003c00u;
#pragma unroll
  for (int u = 0; u < SUBS; ++u) {
    const uint32_t x0 = Mma<__half>::pack(fast_exp2(fmaf(s[4 * u], sl2a, sub_a)), fast_exp2(fmaf(s[4 * u + 1], sl2b, sub_b)));
    const uint32_t x1 = Mma<__half>::pack(fast_exp2(fmaf(s[4 * u + 2], sl2a, sub_a)), fast_exp2(fmaf(s[4 * u + 3], sl2b, sub_b)));
    const uint32_t p0 = movmatrix_trans(x0), p1 = movmatrix_trans(x1);
    const uint8_t* sp = vs + u * kFp4TileBytes;
    uint32_t c01 = sp[t0 * kFp4RowScales] | (uint32_t)sp[t1 * kFp4RowScales] << 8;
    uint32_t c89 = sp[(t0 + 8) * kFp4RowScales] | (uint32_t)sp[(t1 + 8) * kFp4RowScales] << 8;
    if constexpr (!kFull) {  // scales of tokens that no row sees may be NaN: their values are zeros (every code is finite)
      const int at = tok0 + 16 * u;
      c01 &= (rows_any(it, at + t0) ? 0x00ffu : 0u) | (rows_any(it, at + t1) ? 0xff00u : 0u);
      c89 &= (rows_any(it, at + t0 + 8) ? 0x00ffu : 0u) | (rows_any(it, at + t1 + 8) ? 0xff00u : 0u);
    }
    const __half2 s01 = scales_of(c01), s89 = scales_of(c89);
    const uint8_t* vt = vp + u * kFp4TileBytes;
    const uint2 va = *reinterpret_cast<const uint2*>(vt + t0 * kFp4RowBytes);
    const uint2 vb = *reinterpret_cast<const uint2*>(vt + t1 * kFp4RowBytes);
    const uint2 vc = *reinterpret_cast<const uint2*>(vt + (t0 + 8) * kFp4RowBytes);
    const uint2 vd = *reinterpret_cast<const uint2*>(vt + (t1 + 8) * kFp4RowBytes);
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
        Mma<__half>::run(o[4 * w + i], times(e0[i], s01), times(o0[i], s01), times(e1[i], s89), times(o1[i], s89), p0, p1);
    }
    Mma<__half>::run(o[8], kOnes, kOnes, kOnes, kOnes, p0, p1);
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

// One warp of a CTA at an item: slabs it.v0 + warp, + NW, ... below it.v1 of the item's list go through its ring.
// kDecode: the rows are one token's, without ALiBi.
template <typename T, int NW, int NS, bool kDecode>
struct Fp4Warp {
  using S = RowsFp4Shape<NW, NS>;
  static constexpr int D = kFp4D;
  // Lane l holds, of slab 32 b + l, the caches' tiles that its tiles are (whole: the first one): kNone, one that no row
  // sees; kBad, of a block outside the pool.
  static constexpr int kNone = -1, kBad = -2;

  const WindowParams& p;
  uint8_t* smem;
  uint8_t* ring;
  uint64_t* bars;
  volatile int32_t* abort_flag;
  const int warp, lane;
  int n_my = 0;             // slabs of this warp
  int held[S::SUBS];
  uint32_t bad = 0;         // of the 32 slabs, those with a block outside the pool
  uint32_t bad_stages = 0;
  uint32_t done = 0;        // slabs that the ring has taken before this item
  uint32_t qf[8][2];        // query fragments: k-step w, slots (2c, 2c + 1 | 2c + 8, 2c + 9) <- dimensions 32c + 4w .. + 3
  float sl2a, sl2b;
  float o[9][4], m_a, m_b;

  __device__ __forceinline__ Fp4Warp(const WindowParams& params, uint8_t* shared)
      : p(params), smem(shared), ring(shared + (threadIdx.x >> 5) * S::RING_BYTES),
        bars(reinterpret_cast<uint64_t*>(shared + S::BAR_OFF) + (threadIdx.x >> 5) * NS),
        abort_flag(reinterpret_cast<volatile int32_t*>(shared + S::FLAG_OFF)), warp(threadIdx.x >> 5),
        lane(threadIdx.x & 31) {}

  __device__ __forceinline__ bool whole() const { return p.block_size % S::SB == 0; }  // a slab's tiles are one run
  __device__ __forceinline__ int slab_tok(const RowsItem& it, int k) const {
    return rows_slab(it, it.v0 + warp + k * NW) * S::SB;
  }
  __device__ __forceinline__ int first_issued() const { return p.test_expire_first_wait ? 1 : 0; }

  __device__ __forceinline__ void next_batch(const RowsItem& it, int k0) {
    const int B = p.block_size, k = k0 + lane;
#pragma unroll
    for (int u = 0; u < S::SUBS; ++u) held[u] = kNone;
    bool mine_bad = false;
    if (k < n_my) {
      const int tok0 = slab_tok(it, k);
#pragma unroll
      for (int u = 0; u < S::SUBS; ++u) {
        const int t = tok0 + u * kFp4Tokens;
        if (whole() ? u == 0 : rows_touch(it, t, kFp4Tokens)) {
          const int b = t / B, block = __ldg(p.block_tables + (size_t)it.s * p.max_blocks + b);
          held[u] = block >= 0 && block < p.num_blocks
                        ? (block * p.num_kv_heads + it.hkv) * (B / kFp4Tokens) + (t - b * B) / kFp4Tokens
                        : kBad;
          mine_bad = mine_bad || held[u] == kBad;
        }
      }
    }
    bad = __ballot_sync(0xffffffffu, mine_bad);
  }

  // the whole warp, k increasing; a slab's copies by the lane that has its tiles
  __device__ __forceinline__ void issue(const RowsItem& it, int k) {
    if (k % 32 == 0 && k > 0) next_batch(it, k);
    const uint32_t stage = (done + k) % NS;
    bool valid = true;
    if ((bad | bad_stages) != 0) {
      valid = !((bad >> (k & 31)) & 1u);
      bad_stages = (bad_stages & ~(1u << stage)) | (valid ? 0u : 1u << stage);
    }
    if (lane == (k & 31)) {
      uint64_t* bar = &bars[stage];
      uint8_t* dst = ring + stage * S::SLAB_BYTES;
      const uint8_t* k_cache = static_cast<const uint8_t*>(p.k_cache);
      const uint8_t* v_cache = static_cast<const uint8_t*>(p.v_cache);
      if (!valid) {
        report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
        mbar_arrive(bar);
      } else if (whole()) {
        const size_t at = (size_t)held[0] * kFp4TileBytes;
        mbar_arrive_expect_tx(bar, 2 * S::HALF);
        bulk_load_1d(dst, k_cache + at, S::HALF, bar);
        bulk_load_1d(dst + S::HALF, v_cache + at, S::HALF, bar);
      } else {
        uint32_t tiles = 0;
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) tiles += held[u] >= 0 ? 1 : 0;
        mbar_arrive_expect_tx(bar, 2 * tiles * kFp4TileBytes);
        // (a tile that no row sees keeps what its place held: masked)
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) {
          if (held[u] >= 0) {
            const size_t at = (size_t)held[u] * kFp4TileBytes;
            bulk_load_1d(dst + u * kFp4TileBytes, k_cache + at, kFp4TileBytes, bar);
            bulk_load_1d(dst + S::HALF + u * kFp4TileBytes, v_cache + at, kFp4TileBytes, bar);
          }
        }
      }
    }
  }

  // the first copies of an item
  __device__ __forceinline__ void begin(const RowsItem& it) {
    const int mine = it.v1 - it.v0;
    n_my = mine > warp ? (mine - warp + NW - 1) / NW : 0;
    next_batch(it, 0);
    for (int k = first_issued(); k < min(n_my, NS); ++k) issue(it, k);
  }
  // lane 0: the copies of stages k0 .. that are in flight, when the CTA gives up
  __device__ __forceinline__ void drain(int k0) {
    for (int kk = max(k0, first_issued()); kk < min(n_my, k0 + NS); ++kk)
      drain_phase(&bars[(done + kk) % NS], ((done + kk) / NS) & 1);
  }

  __device__ __forceinline__ void load_query(const RowsItem& it) {
    const int g = lane >> 2, c = lane & 3;
    // Scores of the stored numbers are positive multiples of the raw ones, in log2 units: a negative scale turns the query
    // round, and one too small for that makes it zeros.
    float sl2 = p.scale_log2 * p.k_scale;
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
      float unit, inv;
      row_power(mx, unit, inv);
      sl2 *= unit;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = Mma<__half>::pack(Mma<T>::lo(x[i]) * inv, Mma<T>::hi(x[i]) * inv);
    }
    const uint32_t flip = sl2 < 0.f ? 0x80008000u : 0u, keep = score_scale(sl2) == fabsf(sl2) ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) qf[i][0] = (x[2 * i] ^ flip) & keep, qf[i][1] = (x[2 * i + 1] ^ flip) & keep;
    sl2a = score_scale(__shfl_sync(0xffffffffu, sl2, 8 * c));
    sl2b = score_scale(__shfl_sync(0xffffffffu, sl2, 8 * c + 4));
  }

  // The item's slabs, whose first copies and query are there.  False: a wait has run out; what was in flight has landed.
  __device__ __forceinline__ bool run(const RowsItem& it) {
    const int B = p.block_size, c = lane & 3;
    // rows past the item are computed with the last row's position and not written
    const int ra = min(2 * c, it.gcount - 1), rb = min(2 * c + 1, it.gcount - 1);
    int pos_a = it.p_last, pos_b = it.p_last;
    float bias_a = 0.f, bias_b = 0.f;
    if constexpr (!kDecode) {
      pos_a = it.base + (it.row0 + ra) / it.G, pos_b = it.base + (it.row0 + rb) / it.G;
      if (p.alibi != nullptr) {
        constexpr float kLog2e = 1.4426950408889634f;
        bias_a = __ldg(p.alibi + it.hkv * it.G + (it.row0 + ra) % it.G) * kLog2e / sl2a;
        bias_b = __ldg(p.alibi + it.hkv * it.G + (it.row0 + rb) % it.G) * kLog2e / sl2b;
      }
    }
    // the step's append: the warp of the list's last slab starts copying the new token's rows (lanes 0..15 the key,
    // 16..31 the value, 16 bytes each)
    uint8_t* stage_rows = smem + S::STAGE_OFF;
    const int app_tok = p.new_k != nullptr ? it.L - 1 : -1;
    if (p.new_k != nullptr && n_my > 0 && slab_tok(it, n_my - 1) == app_tok / S::SB * S::SB) {
      constexpr int CH = D * 2 / 16;
      const size_t row = (size_t)it.s * p.num_kv_heads + it.hkv;
      const void* src = static_cast<const uint4*>(lane >= CH ? p.new_v : p.new_k) + row * CH + lane % CH;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.commit_group;" ::"r"(
                       smem_u32(stage_rows + 16 * lane)),
                   "l"(src)
                   : "memory");
    }
#pragma unroll
    for (int i = 0; i < 9; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m_a = m_b = -INFINITY;
    int k = 0;
    long long limit = p.test_expire_first_wait ? kRowsTestWaitCycles : kRowsWaitCycles;
    for (; k < n_my; ++k) {
      const uint32_t at = done + k, stage = at % NS;
      if (!__all_sync(0xffffffffu, rows_wait(&bars[stage], (at / NS) & 1, abort_flag, limit))) break;
      limit = kRowsWaitCycles;
      if (bad_stages == 0 || !((bad_stages >> stage) & 1u)) {
        const int tok0 = slab_tok(it, k);
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
            const int block = __ldg(p.block_tables + (size_t)it.s * p.max_blocks + app_tok / B);
            const size_t to = fp4_tile(block, p.num_kv_heads, it.hkv, B, app_tok % B);
            store_quantised(static_cast<uint8_t*>(p.k_cache_out) + to, r, lane, kc, ks);
            store_quantised(static_cast<uint8_t*>(p.v_cache_out) + to, r, lane, vc, vs);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the async proxy refills the buffer
          __syncwarp();
        }
        auto slab = [&](auto full) {
          fp4_slab<S::SUBS, decltype(full)::value, kDecode>(kst, kst + S::HALF, tok0, it, qf, o, m_a, m_b, lane, sl2a, sl2b,
                                                            !kDecode && p.alibi != nullptr, bias_a, bias_b, pos_a, pos_b,
                                                            p.window);
        };
        if (rows_full(it, tok0, S::SB)) slab(std::true_type());
        else slab(std::false_type());
      }
      __syncwarp();
      if (k + NS < n_my) issue(it, k + NS);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    const bool ok = k >= n_my;
    if (!ok) {
      if (lane == 0) {
        report_error(p.err_flag, PA_DEVERR_TIMEOUT);
        drain(k);
      }
      __syncwarp();
    }
    done += n_my;
    return ok;
  }

  // unnormalised O[8 rows][OROW] of the stored numbers, then (max score in log2 units, sum)[8 rows].  The values' unit
  // comes after the division by the sum: a unit near the largest (2^100) times what a row has added up would be infinite.
  __device__ __forceinline__ void store(float* wo) const {
    const int g = lane >> 2, c = lane & 3;
    float* wml = wo + 8 * S::OROW;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float* at = wo + 16 * g + 2 * i;
      *reinterpret_cast<float2*>(at + (2 * c) * S::OROW) = make_float2(o[i][0], o[i][2]);
      *reinterpret_cast<float2*>(at + (2 * c + 1) * S::OROW) = make_float2(o[i][1], o[i][3]);
    }
    if (g == 0) {
      wml[(2 * c) * 2] = m_a;
      wml[(2 * c) * 2 + 1] = o[8][0];
      wml[(2 * c + 1) * 2] = m_b;
      wml[(2 * c + 1) * 2 + 1] = o[8][1];
    }
  }
};

template <int NW, int NS>
__device__ __forceinline__ uint8_t* set_up(uint8_t* raw) {
  using S = RowsFp4Shape<NW, NS>;
  // (by an offset: a pointer made from a number would be read with generic loads)
  uint8_t* smem = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
  if (threadIdx.x == 0) *reinterpret_cast<volatile int32_t*>(smem + S::FLAG_OFF) = 0;
  if ((threadIdx.x & 31) == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF) + (threadIdx.x >> 5) * NS;
    for (int i = 0; i < NS; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  return smem;
}

template <typename T, int NW, int NS, bool SLOTS>
__global__ void __launch_bounds__(RowsFp4Shape<NW, NS>::THREADS) fp4_rows_kernel(const WindowParams p) {
  using S = RowsFp4Shape<NW, NS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = set_up<NW, NS>(smem_raw);
  griddep_begin();
  RowsItem it;
  if (!rows_item<S::SB, SLOTS>(p, it, reinterpret_cast<long long*>(smem + S::WT_OFF))) return;
  if (it.empty) {
    rows_zero<T, S::D>(p, it);
    return;
  }
  Fp4Warp<T, NW, NS, false> w(p, smem);
  w.begin(it);
  w.load_query(it);
  w.run(it);
  w.store(reinterpret_cast<float*>(w.ring));
  __syncthreads();
  rows_finish<T, S::D, NW, S::OROW, S::RING_BYTES / 4>(p, it, reinterpret_cast<const float*>(smem),
                                                       reinterpret_cast<float*>(smem + S::WT_OFF),
                                                       reinterpret_cast<float*>(smem + S::MINE_OFF), p.v_scale);
}

// ---------------------------------------------------------------- decode, slabs dealt out evenly
// The slabs of all items, sequence by sequence, lie one after the other; each of G CTAs takes an equal share, which may
// start and end inside an item.  An item that one CTA holds whole is written by it; of any other, every CTA leaves its part
// (unnormalised rows, their maxima and sums) in the workspace, and the CTA that holds the item's first slab a record of
// where they lie, from which the kernel behind puts them together.  So contexts of any lengths keep every SM busy to the
// end, and one of 20000 tokens is spread over all.  A CTA has at most two parts: of an item that started before it
// (slot 0), and of one that goes on after it (slot 1).
struct EvenRecord {
  int32_t s, hkv, row0;  // s < 0: no item that goes on starts in this CTA
  int32_t last;          // the CTA that holds the item's last slab
};
constexpr int kPartFloats = 8 * kFp4D + 16;  // [8][D], then (m, l)[8]
__host__ __device__ inline size_t even_records(int grid) { return ((size_t)grid * 2 * kPartFloats * 4 + 255) / 256 * 256; }

// Where a CTA is: the item, its first slab of it, the slabs left of its share; and what it will record.
struct EvenWalk {
  long long total;
  int32_t left, s, item, off, ctas;
  EvenRecord record;
};
static_assert(sizeof(EvenWalk) <= 64, "its place in shared memory");

// slabs that the item of sequence s's last token sees; -1: a length that is not one
template <int SB>
__device__ __forceinline__ int decode_slabs(const WindowParams& p, int L) {
  if (L < 0 || (long long)L > (long long)p.max_blocks * p.block_size) return -1;
  if (L == 0) return 0;
  const int n_sink = (min(p.sinks, L) + SB - 1) / SB;
  return n_sink + max(0, (L - 1) / SB + 1 - max(max(0, L - p.window) / SB, n_sink));
}

// What the CTA's warps left, put together: the item's rows of `out`, or (part not null) their maxima and sums and the
// unnormalised rows, all relative to them, for the join.
template <typename T, int NW, int STRIDE>
__device__ __forceinline__ void write_rows(const WindowParams& p, const RowsItem& it, const float* parts, float* wt,
                                           float* part) {
  constexpr int D = kFp4D, OROW = D + 4;
  float* lsum = wt + 8 * NW;
  if (threadIdx.x < 8) {
    const int r = threadIdx.x;
    float ms = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) ms = fmaxf(ms, parts[w * STRIDE + 8 * OROW + r * 2]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float m = parts[w * STRIDE + 8 * OROW + r * 2], x = m == -INFINITY ? 0.f : fast_exp2(m - ms);
      l += x * parts[w * STRIDE + 8 * OROW + r * 2 + 1];  // (0 times a NaN stays one)
      wt[r * NW + w] = x;
    }
    lsum[r] = l;
    if (part != nullptr) *reinterpret_cast<float2*>(part + 8 * D + 2 * r) = make_float2(ms, l);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < it.gcount * (D / 4); i += NW * 32) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float x = wt[r * NW + w];
      const float4 v = *reinterpret_cast<const float4*>(parts + w * STRIDE + r * OROW + d);
      acc.x = fmaf(x, v.x, acc.x), acc.y = fmaf(x, v.y, acc.y), acc.z = fmaf(x, v.z, acc.z), acc.w = fmaf(x, v.w, acc.w);
    }
    if (part != nullptr) {
      *reinterpret_cast<float4*>(part + r * D + d) = acc;
    } else {
      const float inv = lsum[r] == 0.f ? 0.f : 1.f / lsum[r];
      uint2 y;
      y.x = Mma<T>::pack(acc.x * inv * p.v_scale, acc.y * inv * p.v_scale);
      y.y = Mma<T>::pack(acc.z * inv * p.v_scale, acc.w * inv * p.v_scale);
      *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + rows_offset(p, it, r) * D + d) = y;
    }
  }
}

// Warps of a CTA, slabs of a ring, CTAs of an SM: 16 warps of 118 registers.  96 sequences of up to 16384 tokens, 64 / 8
// heads: 138 us, with three CTAs 150, five (96 registers, spills) 151, two of eight warps 157, slabs of 64 tokens 159.
constexpr int kEvenWarps = 4, kEvenStages = 2, kEvenResident = 4;
constexpr int kEvenMinSlabs = kEvenWarps;  // of a CTA: fewer CTAs take part in small calls

template <typename T>
__global__ void __launch_bounds__(kEvenWarps * 32, kEvenResident) fp4_even_kernel(const WindowParams p, float* workspace) {
  constexpr int NW = kEvenWarps, NS = kEvenStages;
  using S = RowsFp4Shape<NW, NS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = set_up<NW, NS>(smem_raw);
  griddep_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = blockIdx.x;
  const int per = p.num_kv_heads * p.tiles;  // items of a sequence
  EvenRecord* record = reinterpret_cast<EvenRecord*>(reinterpret_cast<uint8_t*>(workspace) + even_records(gridDim.x)) + me;

  // ---- the sum of all slabs, and the item in which this CTA's share starts
  long long* sums = reinterpret_cast<long long*>(smem + S::WT_OFF);
  int* start = reinterpret_cast<int*>(sums + 8);
  long long total = 0;
  int ctas;
  {
    const int run = (p.num_seqs + NW * 32 - 1) / (NW * 32);
    const int begin = min(p.num_seqs, run * (int)threadIdx.x), end = min(p.num_seqs, begin + run);
    long long own = 0;
    for (int s = begin; s < end; ++s) {
      const int n = decode_slabs<S::SB>(p, __ldg(p.seq_lens + s));
      if (n < 0 && me == 0) report_error(p.err_flag, PA_DEVERR_QUERY);
      own += max(n, 0);
    }
    long long upto = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    for (int w = 0; w < NW; ++w) {
      if (w < warp) upto += sums[w];
      total += sums[w];
    }
    total *= per;
    ctas = (int)max(1ll, min((long long)gridDim.x, total / kEvenMinSlabs));
    const long long x = total * me / ctas;
    long long at = (upto - own) * per;
    if (me < ctas && x >= at && x < upto * per) {  // the thread in whose run of sequences x lies
      int s = begin, n;
      for (;; ++s) {
        n = max(0, decode_slabs<S::SB>(p, __ldg(p.seq_lens + s)));
        if (x < at + (long long)n * per) break;
        at += (long long)n * per;
      }
      start[0] = s;
      start[1] = (int)((x - at) / n);
      start[2] = (int)((x - at) % n);
    }
  }
  // ---- rows of empty sequences
  for (int e = me; e < p.num_seqs; e += gridDim.x) {
    if (__ldg(p.seq_lens + e) == 0) {
      T* out = static_cast<T*>(p.out) + (size_t)e * p.num_q_heads * S::D;
      for (int i = threadIdx.x; i < p.num_q_heads * S::D; i += NW * 32) out[i] = from_float<T>(0.f);
    }
  }
  __syncthreads();
  // Where the CTA is, in shared memory and read again after an item's slabs, whose loop needs the registers (128 a thread
  // for four CTAs an SM; kept in registers, 52 bytes were spilled and 96 sequences took 146 us for 140).
  volatile EvenWalk* walk = reinterpret_cast<volatile EvenWalk*>(smem + S::WALK_OFF);
  if (threadIdx.x == 0) {
    // (a share is counted in 32 bits: one that long would take hours)
    walk->left = me < ctas ? (int)(total * (me + 1) / ctas - total * me / ctas) : 0;
    walk->s = start[0];
    walk->item = start[1];
    walk->off = start[2];
    walk->total = total;
    walk->ctas = ctas;
    walk->record.s = -1;
  }
  __syncthreads();
  auto rows_of = [&](RowsItem& it, int& n) {
    const int s = walk->s, item = walk->item, L = __ldg(p.seq_lens + s);
    n = decode_slabs<S::SB>(p, L);
    it.s = it.q0 = s;
    it.hkv = item / p.tiles;
    it.G = p.num_q_heads / p.num_kv_heads;
    it.row0 = item % p.tiles * kRowsGroup;
    it.gcount = min(kRowsGroup, it.G - it.row0);
    it.L = L;
    it.base = it.p_first = it.p_last = L - 1;
    it.lo_first = it.lo_last = max(0, L - p.window);
    it.sinks = min(p.sinks, L);
    it.n_sink = (it.sinks + S::SB - 1) / S::SB;
    it.j_win = max(it.lo_first / S::SB, it.n_sink);
    it.v0 = walk->off;
    it.v1 = min(n, it.v0 + walk->left);
    it.empty = false;
  };
  Fp4Warp<T, NW, NS, true> w(p, smem);
  while (walk->left > 0) {
    int n;
    {
      RowsItem it;
      rows_of(it, n);
      w.begin(it);
      w.load_query(it);
      w.run(it);
    }
    w.store(reinterpret_cast<float*>(w.ring));
    __syncthreads();
    if (*w.abort_flag) break;  // a wait has run out, and nothing is in flight
    RowsItem it;
    rows_of(it, n);
    const bool head = it.v0 == 0, tail = it.v1 == n;
    write_rows<T, NW, S::RING_BYTES / 4>(p, it, reinterpret_cast<const float*>(smem),
                                         reinterpret_cast<float*>(smem + S::WT_OFF),
                                         head && tail ? nullptr : workspace + (size_t)(2 * me + (head ? 1 : 0)) * kPartFloats);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the parts have been read: copies may take their place
    __syncthreads();
    if (threadIdx.x == 0) {
      const int left = walk->left - (it.v1 - it.v0);
      if (head && !tail) {  // (the CTA's share ends here)
        const long long all = walk->total;
        const int g = walk->ctas;
        const long long end = all * (me + 1) / g + (n - it.v1);  // behind the item's last slab
        long long last = (end - 1) * g / all;
        while (all * (last + 1) / g < end) ++last;
        while (all * last / g >= end) --last;
        walk->record.s = it.s;
        walk->record.hkv = it.hkv;
        walk->record.row0 = it.row0;
        walk->record.last = (int)last;
      }
      if (left > 0) {  // the next item with slabs
        int s = it.s, item = walk->item + 1;
        if (item == per) {
          item = 0;
          do ++s;
          while (decode_slabs<S::SB>(p, __ldg(p.seq_lens + s)) <= 0);
        }
        walk->s = s;
        walk->item = item;
        walk->off = 0;
      }
      walk->left = left;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    EvenRecord r;
    r.s = walk->record.s, r.hkv = walk->record.hkv, r.row0 = walk->record.row0, r.last = walk->record.last;
    *record = r;
  }
}

// One CTA for each of the kernel's in front: puts the parts of the item together whose first slab lay in it.  Eight rows
// and kJoinGroups groups of warps, each with every kJoinGroups-th part.
constexpr int kJoinGroups = 4, kJoinThreads = 8 * kJoinGroups * 32;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) fp4_join_kernel(const WindowParams p, const float* workspace) {
  __shared__ float4 acc_of[kJoinGroups][8][32];
  __shared__ float2 ml_of[kJoinGroups][8];
  griddep_begin();
  const int me = blockIdx.x, group = threadIdx.x >> 8, r = (threadIdx.x >> 5) & 7, lane = threadIdx.x & 31;
  const EvenRecord rec =
      reinterpret_cast<const EvenRecord*>(reinterpret_cast<const uint8_t*>(workspace) + even_records(gridDim.x))[me];
  const int G = p.num_q_heads / p.num_kv_heads;
  if (rec.s < 0) return;
  const int parts = rec.last - me + 1;
  // part i: slot 1 of this CTA, then slot 0 of those behind
  auto part = [&](int i) { return workspace + (size_t)(2 * (me + i) + (i == 0 ? 1 : 0)) * kPartFloats; };
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float mx = -INFINITY, l = 0.f;
#pragma unroll 2
  for (int first = group; first < parts; first += 4 * kJoinGroups) {
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(first + j * kJoinGroups, parts - 1);
      ml[j] = *reinterpret_cast<const float2*>(part(i) + 8 * kFp4D + 2 * r);
      v[j] = *reinterpret_cast<const float4*>(part(i) + r * kFp4D + 4 * lane);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (first + j * kJoinGroups >= parts) ml[j] = make_float2(-INFINITY, 0.f), v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float up = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), mx);
    const float old = mx == -INFINITY ? 0.f : fast_exp2(mx - up);
    acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
    l *= old;  // (0 times a NaN stays one)
    mx = up;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w = ml[j].x == -INFINITY ? 0.f : fast_exp2(ml[j].x - mx);
      l = fmaf(w, ml[j].y, l);
      acc.x = fmaf(w, v[j].x, acc.x), acc.y = fmaf(w, v[j].y, acc.y), acc.z = fmaf(w, v[j].z, acc.z), acc.w = fmaf(w, v[j].w, acc.w);
    }
  }
  acc_of[group][r][lane] = acc;
  if (lane == 0) ml_of[group][r] = make_float2(mx, l);
  __syncthreads();
  if (group > 0 || rec.row0 + r >= G) return;
  for (int g = 1; g < kJoinGroups; ++g) mx = fmaxf(mx, ml_of[g][r].x);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
  for (int g = 0; g < kJoinGroups; ++g) {
    const float2 ml = ml_of[g][r];
    const float4 v = acc_of[g][r][lane];
    const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - mx);
    l = fmaf(w, ml.y, l);
    acc.x = fmaf(w, v.x, acc.x), acc.y = fmaf(w, v.y, acc.y), acc.z = fmaf(w, v.z, acc.z), acc.w = fmaf(w, v.w, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 y;
  y.x = Mma<T>::pack(acc.x * inv * p.v_scale, acc.y * inv * p.v_scale);
  y.y = Mma<T>::pack(acc.z * inv * p.v_scale, acc.w * inv * p.v_scale);
  T* out = static_cast<T*>(p.out) + ((size_t)rec.s * p.num_q_heads + (size_t)rec.hkv * G + rec.row0 + r) * kFp4D;
  *reinterpret_cast<uint2*>(out + 4 * lane) = y;
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

template <typename T>
cudaError_t launch_even(WindowParams p, float* workspace, cudaStream_t stream) {
  using S = RowsFp4Shape<kEvenWarps, kEvenStages>;
  static_assert(kEvenResident * (S::EVEN_BYTES + 1024) <= 228 * 1024, "shared memory of the resident CTAs");
  auto kernel = fp4_even_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::EVEN_BYTES);
  if (e != cudaSuccess) return e;
  p.tiles = (p.num_q_heads / p.num_kv_heads + kRowsGroup - 1) / kRowsGroup;
  p.cluster = 1;
  e = launch_cluster(kernel, dim3(kFp4EvenGrid), dim3(S::THREADS), S::EVEN_BYTES, 1, true, stream, p, workspace);
  if (e != cudaSuccess) return e;
  return launch_cluster(fp4_join_kernel<T>, dim3(kFp4EvenGrid), dim3(kJoinThreads), 0, 1, true, stream, p,
                        (const float*)workspace);
}

}  // namespace

static_assert(kFp4EvenGrid == 152 * kEvenResident, "the grid fills a GB300");

size_t fp4_even_workspace() { return even_records(kFp4EvenGrid) + kFp4EvenGrid * sizeof(EvenRecord); }

cudaError_t launch_fp4_even(int row_dtype, const WindowParams& p, float* workspace, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_even<__half>(p, workspace, stream) : launch_even<__nv_bfloat16>(p, workspace, stream);
}

cudaError_t launch_fp4_rows(int row_dtype, const WindowParams& p, bool slots, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_type<__half>(p, slots, stream) : launch_type<__nv_bfloat16>(p, slots, stream);
}

}  // namespace pa
