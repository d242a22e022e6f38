// pa_window_rows_f32.cu - attention of a few query rows over a window of an
// fp32 cache (see pa_window_rows.cuh for the rows, the visible slabs and the
// split).
//
// fp32 keeps full products, so it runs on the CUDA cores.  A warp takes slabs of
// 16 tokens, four tokens at a time: every lane holds D / 32 elements of the four
// K and V rows (coalesced loads, eight in flight), the 8 rows x 4 tokens = 32
// partial dot products are reduced together (a halving exchange: 31 shuffles
// leave score j in lane j, where a sum of each alone would take 160), the online
// softmax works on one score a lane, and the 32 weights are passed round for
// O += P V.  About 350 instructions per 4 KB of K/V at D = 128: at four
// instructions a clock an SM could take in 47 bytes a clock, twice its share of
// HBM, so the copies bound it.
#include <cuda.h>
#include <math.h>

#include "pa.h"
#include "pa_window_rows.cuh"

namespace pa {
namespace {

constexpr int kF32Slab = 16;
constexpr int kF32Warps = 4;

template <int VEC>
__device__ __forceinline__ void load_row(const float* src, float (&x)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(src));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = __ldg(reinterpret_cast<const float2*>(src));
    x[0] = v.x, x[1] = v.y;
  }
}

template <int D>
__global__ void __launch_bounds__(kF32Warps * 32) window_rows_f32_kernel(const WindowParams p) {
  constexpr int VEC = D / 32, OROW = D, STRIDE = 8 * D + 16;
  __shared__ float parts[kF32Warps * STRIDE];
  __shared__ float wt[8 * kF32Warps + 16];
  __shared__ float mine[8 * D + 16];
  griddep_begin();
  RowsItem it;
  if (!rows_item<kF32Slab>(p, it)) return;
  if (it.empty) {
    rows_zero<float, D>(p, it);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* kc = static_cast<const float*>(p.k_cache) + lane * VEC;
  const float* vc = static_cast<const float*>(p.v_cache) + lane * VEC;
  const int32_t* table = p.block_tables + (size_t)it.s * p.max_blocks;
  const int B = p.block_size;

  float q[8][VEC], o[8][VEC];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      // (q is 4-byte aligned only)
      q[r][e] = r < it.gcount ? __ldg(static_cast<const float*>(p.q) + rows_offset(p, it, r) * D + lane * VEC + e) : 0.f;
      o[r][e] = 0.f;
    }
  }
  // this lane's row and its token of four (lane = 8 * token + row); rows past the item: the last row's position
  const int my_row = min(lane & 7, it.gcount - 1), my_tok = lane >> 3;
  const int pos = it.base + (it.row0 + my_row) / it.G;
  const float bias =
      p.alibi != nullptr ? __ldg(p.alibi + it.hkv * it.G + (it.row0 + my_row) % it.G) * 1.4426950408889634f : 0.f;
  float m = -INFINITY, l = 0.f;  // of the lane's row (l: of its token of each four)

  for (int v = it.v0 + warp; v < it.v1; v += kF32Warps) {
    const int tok0 = rows_slab(it, v) * kF32Slab;
    // lane t < 16: the block of the slab's token t (-1: seen by no row, or not in the pool)
    int entry = -1;
    if (lane < kF32Slab && rows_any(it, tok0 + lane)) {
      entry = __ldg(table + (tok0 + lane) / B);
      if (entry < 0 || entry >= p.num_blocks) {
        report_error(p.err_flag, PA_DEVERR_BLOCK_ID);
        entry = -1;
      }
    }
#pragma unroll 1
    for (int t0 = 0; t0 < kF32Slab; t0 += 4) {
      float k[4][VEC], x[4][VEC];
      bool mine_in = false;  // the lane's token takes part
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int e = __shfl_sync(0xffffffffu, entry, t0 + t);
        if (t == my_tok) mine_in = e >= 0;
        if (e >= 0) {
          const size_t row = (((size_t)e * p.num_kv_heads + it.hkv) * B + (tok0 + t0 + t) % B) * D;
          load_row<VEC>(kc + row, k[t]);
          load_row<VEC>(vc + row, x[t]);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) k[t][i] = x[t][i] = 0.f;
        }
      }
      float dot[32];  // value 8 * token + row
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          float d = q[r][0] * k[t][0];
#pragma unroll
          for (int i = 1; i < VEC; ++i) d = fmaf(q[r][i], k[t][i], d);
          dot[8 * t + r] = d;
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
        for (int r = 0; r < 8; ++r) {
          const float a = __shfl_sync(0xffffffffu, al, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[r][i] *= a;
        }
      }
      const float pe = fast_exp2(s - (m == -INFINITY ? 0.f : m));
      l += pe;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float w = __shfl_sync(0xffffffffu, pe, 8 * t + r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[r][i] = fmaf(w, x[t][i], o[r][i]);
        }
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  float* wo = parts + warp * STRIDE;
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int i = 0; i < VEC; ++i) wo[r * OROW + lane * VEC + i] = o[r][i];
  if (lane < 8) {
    wo[8 * OROW + 2 * lane] = m;
    wo[8 * OROW + 2 * lane + 1] = l;
  }
  __syncthreads();
  rows_finish<float, D, kF32Warps, OROW, STRIDE>(p, it, parts, wt, mine);
}

template <int D>
cudaError_t launch_f32(const WindowParams& p, cudaStream_t stream) {
  return launch_cluster(window_rows_f32_kernel<D>, dim3((unsigned)(window_items(p) * p.cluster)), dim3(kF32Warps * 32), 0,
                        p.cluster, true, stream, p);
}

}  // namespace

cudaError_t launch_window_rows_f32(int head_size, const WindowParams& p, cudaStream_t stream) {
  if (head_size == 64) return launch_f32<64>(p, stream);
  if (head_size == 128) return launch_f32<128>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
