// pa_window_rows_f32.cu - attention of a few query rows over a window of an
// fp32 cache (see pa_window_rows.cuh for the rows, the visible slabs and the
// split).
//
// fp32 keeps full products, so it runs on the CUDA cores.  A warp takes slabs of
// 16 tokens, four tokens (a step) at a time: every lane holds D / 32 elements of
// the four K and V rows, the 8 rows x 4 tokens = 32 partial dot products are
// reduced together (a halving exchange: 31 shuffles leave score j in lane j,
// where a sum of each alone would take 160), the online softmax works on one
// score a lane, and the 32 weights are passed round for O += P V.  Bound by
// instruction issue as much as by HBM: the products go as packed pairs of rows, and
// a lane works out its token's cache row once a slab (single products and a row for
// every copy: 304 us where it now takes 191).  No load is waited for either:
// each lane copies its own elements kRing - 1 steps ahead into shared memory
// (cp.async: no registers, and no barrier, since it alone reads them back).
// 128 sequences, 64 / 8 heads of 128, 1024 keys: 191 us, 5.7 TB/s.
#include <cuda.h>
#include <math.h>

#include "pa.h"
#include "pa_window_rows.cuh"

namespace pa {
namespace {

constexpr int kF32Slab = 16;
constexpr int kF32Warps = 4;

constexpr int kRing = 4;  // steps in flight per warp, the one in use included

// this lane's elements of a row into its slot, zeros unless `take`
template <int VEC>
__device__ __forceinline__ void copy_row(float* slot, const float* src, bool take) {
  const uint32_t bytes = take ? VEC * 4 : 0;
  if constexpr (VEC == 4)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(slot)), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(slot)), "l"(src), "r"(bytes) : "memory");
}

// a * b + c of two pairs, one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

template <int D, bool SLOTS>
__global__ void __launch_bounds__(kF32Warps * 32) window_rows_f32_kernel(const WindowParams p) {
  constexpr int VEC = D / 32, OROW = D, STRIDE = 8 * D + 16;
  constexpr int STEP = 8 * D;  // floats of a step: four rows of K, then of V
  // [warp][step of the ring][K: token 0..3, V: token 0..3][D]; at the end a warp's partial result
  extern __shared__ __align__(16) float ring_all[];
  __shared__ __align__(16) float wt[8 * kF32Warps + 16];
  __shared__ float mine[8 * D + 16];
  static_assert(kRing * STEP >= STRIDE, "a warp's ring holds its partial result");
  griddep_begin();
  RowsItem it;
  if (!rows_item<kF32Slab, SLOTS>(p, it, reinterpret_cast<long long*>(wt))) return;
  if (it.empty) {
    rows_zero<float, D>(p, it);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* kc = static_cast<const float*>(p.k_cache) + lane * VEC;
  const float* vc = static_cast<const float*>(p.v_cache) + lane * VEC;
  const int32_t* table = p.block_tables + (size_t)it.s * p.max_blocks;
  const int B = p.block_size;

  float2 q[4][VEC], o[4][VEC];  // rows 2r and 2r + 1
  auto q_at = [&](int r, int e) {  // (q is 4-byte aligned only)
    return r < it.gcount ? __ldg(static_cast<const float*>(p.q) + rows_offset(p, it, r) * D + lane * VEC + e) : 0.f;
  };
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      q[r][e] = make_float2(q_at(2 * r, e), q_at(2 * r + 1, e));
      o[r][e] = make_float2(0.f, 0.f);
    }
  }
  // this lane's row and its token of four (lane = 8 * token + row); rows past the item: the last row's position
  const int my_row = min(lane & 7, it.gcount - 1), my_tok = lane >> 3;
  const int pos = it.base + (it.row0 + my_row) / it.G;
  const float bias =
      p.alibi != nullptr ? __ldg(p.alibi + it.hkv * it.G + (it.row0 + my_row) % it.G) * 1.4426950408889634f : 0.f;
  float m = -INFINITY, l = 0.f;  // of the lane's row (l: of its token of each four)

  float* ring = ring_all + warp * (kRing * STEP) + lane * VEC;
  const int mine_n = it.v1 - it.v0, n_my = mine_n > warp ? (mine_n - warp + kF32Warps - 1) / kF32Warps : 0;
  auto slab_tok = [&](int k) { return rows_slab(it, it.v0 + warp + k * kF32Warps) * kF32Slab; };
  // lane t < 16: the cache row of token t of slab k (-1: seen by no row, or not in the pool)
  auto fetch = [&](int k) {
    int e = -1;
    if (k < n_my && lane < kF32Slab) {
      const int t = slab_tok(k) + lane;
      if (rows_any(it, t)) {
        e = __ldg(table + t / B);
        if (e < 0 || e >= p.num_blocks) {
          report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
          e = -1;
        } else {
          e = (e * p.num_kv_heads + it.hkv) * B + t % B;  // (every row's number fits int32)
        }
      }
    }
    return e;
  };
  int entry = fetch(0), entry_next = fetch(1);   // of the slab being copied and the one after it
  unsigned live = 0, live_prev = 0;              // its tokens that take part, and those of the slab before
  const int steps = 4 * n_my;
  auto issue = [&](int i) {  // the copies of step i: tokens 4 (i % 4) .. of slab i / 4
    if (i < steps) {
      if (i % 4 == 0) {
        if (i > 0) {
          entry = entry_next;
          entry_next = fetch(i / 4 + 1);
        }
        live_prev = live;
        live = __ballot_sync(0xffffffffu, entry >= 0);
      }
      const int t0 = 4 * (i % 4);
      float* st = ring + (i % kRing) * STEP;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int e = __shfl_sync(0xffffffffu, entry, t0 + t);
        const size_t row = (size_t)max(e, 0) * D;
        copy_row<VEC>(st + t * D, kc + row, e >= 0);
        copy_row<VEC>(st + (4 + t) * D, vc + row, e >= 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");  // (empty past the end: the count of groups stays that of steps)
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(i);

  for (int i = 0; i < steps; ++i) {
    issue(i + kRing - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");  // step i has landed
    {
      // the slab being copied is this step's, or the one after it
      const unsigned in = (i + kRing - 1 < steps ? (i + kRing - 1) / 4 : n_my - 1) == i / 4 ? live : live_prev;
      const int t0 = 4 * (i % 4), tok0 = slab_tok(i / 4);
      const bool mine_in = (in >> (t0 + my_tok)) & 1u;  // the lane's token takes part
      const float* st = ring + (i % kRing) * STEP;
      float k[4][VEC], x[4][VEC];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) k[t][e] = st[t * D + e];
      float dot[32];  // value 8 * token + row
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float2 d = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) d = fma2(q[r][i], make_float2(k[t][i], k[t][i]), d);
          dot[8 * t + 2 * r] = d.x;
          dot[8 * t + 2 * r + 1] = d.y;
        }
      // halving exchange: after the step with offset w, a lane keeps the values whose bit w equals its own
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
          const float give = up ? dot[i] : dot[i + w], keep = up ? dot[i + w] : dot[i];
          dot[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
      }
      const int t_me = tok0 + t0 + my_tok;
      float s = fmaf(bias, (float)(t_me - pos), dot[0] * p.scale_log2);
      if (!(mine_in && t_me <= pos && (t_me > pos - p.window || t_me < it.sinks))) s = -INFINITY;
      float mx = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float mn = fmaxf(m, mx);
      if (__any_sync(0xffffffffu, mn > m)) {
        const float al = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
        m = mn;
        l *= al;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float a0 = __shfl_sync(0xffffffffu, al, 2 * r), a1 = __shfl_sync(0xffffffffu, al, 2 * r + 1);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[r][i].x *= a0, o[r][i].y *= a1;
        }
      }
      const float pe = fast_exp2(s - (m == -INFINITY ? 0.f : m));
      l += pe;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[t][e] = st[(4 + t) * D + e];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float2 w = make_float2(__shfl_sync(0xffffffffu, pe, 8 * t + 2 * r),
                                       __shfl_sync(0xffffffffu, pe, 8 * t + 2 * r + 1));
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[r][i] = fma2(w, make_float2(x[t][i], x[t][i]), o[r][i]);
        }
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  asm volatile("cp.async.wait_all;" ::: "memory");
  float* wo = ring_all + warp * (kRing * STEP);
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int i = 0; i < VEC; ++i) wo[r * OROW + lane * VEC + i] = r % 2 ? o[r / 2][i].y : o[r / 2][i].x;
  if (lane < 8) {
    wo[8 * OROW + 2 * lane] = m;
    wo[8 * OROW + 2 * lane + 1] = l;
  }
  __syncthreads();
  rows_finish<float, D, kF32Warps, OROW, kRing * STEP>(p, it, ring_all, wt, mine);
}

template <int D, bool SLOTS>
cudaError_t launch_form(WindowParams p, cudaStream_t stream) {
  auto kernel = window_rows_f32_kernel<D, SLOTS>;
  constexpr size_t kSmem = (size_t)kF32Warps * kRing * 8 * D * sizeof(float);
  static ClusterRoom room;
  cudaError_t e = prepare_rows(kernel, room, kF32Warps * 32, kSmem, &p.cluster);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, dim3((unsigned)(window_items(p, SLOTS) * p.cluster)), dim3(kF32Warps * 32), kSmem, p.cluster,
                        true, stream, p);
}

}  // namespace

cudaError_t launch_window_rows_f32(int head_size, const WindowParams& p, bool slots, cudaStream_t stream) {
  if (head_size == 64) return slots ? launch_form<64, true>(p, stream) : launch_form<64, false>(p, stream);
  if (head_size == 128) return slots ? launch_form<128, true>(p, stream) : launch_form<128, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
