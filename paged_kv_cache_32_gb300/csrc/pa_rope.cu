// pa_rope.cu - rotary positions with the cache write: the first r elements of
// every query and key head turn by position * f_j, keys and values go to their
// cache slots, in one pass over them.
//
// For pair j of a token at position t, with c = m cos(t f_j), s = m sin(t f_j):
//   y_a = c x_a - s x_b,  y_b = c x_b + s x_a,  (a, b) = (j, j + r / 2) or (2j, 2j + 1).
//
// Angles.  t f_j reaches millions of radians, where an fp32 product is off by
// whole fractions of a turn.  f_j / 2 pi is therefore held as a 64-bit fixed-point
// fraction of a turn: the 64-bit product with the integer t drops whole turns
// exactly and leaves the fraction to 2^-64 t turns; sincospif takes it from there.
// One angle per (token, pair) and CTA, kept in shared memory for all heads.
//
// Bound by HBM bandwidth: 4 + (cache / element) bytes moved an element against
// about 75 instructions per 64 bytes.  Work is cut into units of two vectors of
// V elements (the two halves' elements V u .. of a pair range, or 2 V neighbouring
// elements), D / 2 V units a head whatever r is; the units of all tokens and
// heads are one flat range, of which a CTA takes kIter x 256 side by side, all
// loads of a thread's units issued before the first is used.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_rope.h"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;

// Vectors of V elements of T, moved with one access each.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};
template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// f / 2 pi as a fraction of a turn in units of 2^-64 (whole turns per position drop out)
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  const double t = f * 0.15915494309189533577;  // 1 / 2 pi
  const double frac = t - floor(t);             // [0, 1]
  const unsigned long long hi = (unsigned long long)(frac * 4294967296.0);  // < 2^33: wraps below
  const double rest = frac * 4294967296.0 - (double)hi;
  return (hi << 32) + (unsigned long long)(rest * 4294967296.0);
}

// E4M3 code of x / scale (fp32 division, ties to even, saturating)
__device__ __forceinline__ uint8_t code_of(float x, float scale) {
  return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
}

struct RopeToken {
  long long row;  // cache row (block * Hkv * B + offset) of kv head 0; < 0: the token is skipped
  int pos, off;
};

// T: queries, keys, values; FP8: the cache holds E4M3 codes (else T); V: elements of a vector; ITER: units of a
// thread.
template <typename T, bool FP8, bool INTERLEAVED, int V, int ITER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int tokens_per_cta) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* cs = reinterpret_cast<float2*>(smem);  // [token][r / 2]: (c, s)
  const int half = p.rotary_dim / 2, D = p.head_size;
  RopeToken* tok = reinterpret_cast<RopeToken*>(cs + (size_t)tokens_per_cta * half);
  const int per_head = D / (2 * V);
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int per_token = heads * per_head;
  const long long total = (long long)p.num_tokens * per_token;
  const long long u0 = (long long)blockIdx.x * (kRopeThreads * ITER);
  const int t0 = (int)(u0 / per_token);
  const int rem0 = (int)(u0 - (long long)t0 * per_token);  // unit of token t0 that this CTA starts with
  const long long last = min(total, u0 + kRopeThreads * ITER) - 1;
  const int nt = (int)(last / per_token) - t0 + 1;
  griddep_wait();
  griddep_launch_dependents();

  for (int i = threadIdx.x; i < nt; i += kRopeThreads) {
    const long long slot = p.slot_mapping[t0 + i];
    RopeToken x;
    x.pos = p.positions[t0 + i];
    x.row = -1;
    x.off = 0;
    if (slot >= 0) {
      const long long block = slot / p.block_size;
      x.off = (int)(slot - block * p.block_size);
      if (block < p.num_blocks)
        x.row = block * p.num_kv_heads * p.block_size + x.off;
      else
        report_error(p.err_flag, PA_DEVERR_SLOT);
    }
    tok[i] = x;
  }
  // ---- the loads of this thread's units
  Vec<T, V> a[ITER], b[ITER];
  int token[ITER], head[ITER], unit[ITER];
#pragma unroll
  for (int k = 0; k < ITER; ++k) {
    const int i = rem0 + k * kRopeThreads + threadIdx.x;
    token[k] = i / per_token;
    const int r = i - token[k] * per_token;
    head[k] = r / per_head;
    unit[k] = r - head[k] * per_head;
    if (token[k] >= nt || t0 + token[k] >= p.num_tokens) {
      token[k] = -1;
      continue;
    }
    const long long t = t0 + token[k];
    const T* src;
    if (head[k] < p.num_q_heads) {
      src = static_cast<const T*>(p.q) + t * p.q_stride + (size_t)head[k] * D;
    } else if (head[k] < p.num_q_heads + p.num_kv_heads) {
      src = static_cast<const T*>(p.key) + t * p.key_stride + (size_t)(head[k] - p.num_q_heads) * D;
    } else {
      src = static_cast<const T*>(p.value) + t * p.value_stride +
            (size_t)(head[k] - p.num_q_heads - p.num_kv_heads) * D;
    }
    // the unit's vectors: e0, e1 (a pair range of the halves layout: r / 2 apart, else side by side)
    const bool apart = !INTERLEAVED && unit[k] * V < half;
    const int e0 = apart ? unit[k] * V : INTERLEAVED ? unit[k] * 2 * V : p.rotary_dim + (unit[k] * V - half) * 2;
    const int e1 = apart ? e0 + half : e0 + V;
    a[k] = *reinterpret_cast<const Vec<T, V>*>(src + e0);
    b[k] = *reinterpret_cast<const Vec<T, V>*>(src + e1);
  }
  // ---- angles of the CTA's tokens
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    const unsigned long long f = turn_fraction(p.inv_freq[j]);
    const long long turns = (long long)(f * (unsigned long long)(long long)p.positions[t0 + t]);
    float s, c;
    sincospif(__ll2float_rn(turns) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns in [-1, 1]
    cs[i] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < ITER; ++k) {
    if (token[k] < 0) continue;
    const RopeToken x = tok[token[k]];
    if (x.row < 0) continue;  // padding, or a slot outside the pool
    const int h = head[k];
    const bool is_q = h < p.num_q_heads, is_v = h >= p.num_q_heads + p.num_kv_heads;
    const bool apart = !INTERLEAVED && unit[k] * V < half;
    const int e0 = apart ? unit[k] * V : INTERLEAVED ? unit[k] * 2 * V : p.rotary_dim + (unit[k] * V - half) * 2;
    const int e1 = apart ? e0 + half : e0 + V;
    float u[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = to_float<T>(a[k].x[i]), w[i] = to_float<T>(b[k].x[i]);
    if (!is_v) {
      const float2* ct = cs + (size_t)token[k] * half + unit[k] * V;
      if constexpr (INTERLEAVED) {
        // pairs V unit .. V unit + V - 1: neighbours within u, then within w
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (unit[k] * V + i < half) {
            const float2 c = ct[i];
            float& x0 = 2 * i < V ? u[(2 * i) % V] : w[(2 * i) % V];
            float& x1 = 2 * i + 1 < V ? u[(2 * i + 1) % V] : w[(2 * i + 1) % V];
            const float y0 = c.x * x0 - c.y * x1, y1 = c.x * x1 + c.y * x0;
            x0 = y0, x1 = y1;
          }
        }
      } else if (apart) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 c = ct[i];
          const float y0 = c.x * u[i] - c.y * w[i], y1 = c.x * w[i] + c.y * u[i];
          u[i] = y0, w[i] = y1;
        }
      }
    }
    if (is_q || !FP8) {
      T* dst;
      if (is_q) {
        dst = static_cast<T*>(p.q_out) + (t0 + token[k]) * p.q_out_stride + (size_t)h * D;
      } else {
        const int hk = h - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
        dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) + (x.row + (long long)hk * p.block_size) * D;
      }
      Vec<T, V> y, z;
#pragma unroll
      for (int i = 0; i < V; ++i) y.x[i] = from_float<T>(u[i]), z.x[i] = from_float<T>(w[i]);
      *reinterpret_cast<Vec<T, V>*>(dst + e0) = y;
      *reinterpret_cast<Vec<T, V>*>(dst + e1) = z;
    } else if (!is_v) {
      uint8_t* dst = static_cast<uint8_t*>(p.k_cache) + (x.row + (long long)(h - p.num_q_heads) * p.block_size) * D;
      Vec<uint8_t, V> y, z;
#pragma unroll
      for (int i = 0; i < V; ++i) y.x[i] = code_of(u[i], p.k_scale), z.x[i] = code_of(w[i], p.k_scale);
      *reinterpret_cast<Vec<uint8_t, V>*>(dst + e0) = y;
      *reinterpret_cast<Vec<uint8_t, V>*>(dst + e1) = z;
    } else {
      // values [block][head][off / 16][d][off % 16]
      const int hk = h - p.num_q_heads - p.num_kv_heads;
      uint8_t* dst = static_cast<uint8_t*>(p.v_cache) +
                     (x.row - x.off + (long long)hk * p.block_size + x.off / 16 * 16) * D + x.off % 16;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dst[(size_t)(e0 + i) * 16] = code_of(u[i], p.v_scale);
        dst[(size_t)(e1 + i) * 16] = code_of(w[i], p.v_scale);
      }
    }
  }
}

template <typename T, bool FP8, bool INTERLEAVED, int V, int ITER>
cudaError_t launch_iter(const RopeParams& p, cudaStream_t stream) {
  const int per_token = (p.num_q_heads + 2 * p.num_kv_heads) * (p.head_size / (2 * V));
  const long long total = (long long)p.num_tokens * per_token;
  const long long ctas = (total + kRopeThreads * ITER - 1) / (kRopeThreads * ITER);
  const int tokens = (kRopeThreads * ITER - 1) / per_token + 2;  // that a CTA's units may touch
  const size_t smem = (size_t)tokens * (p.rotary_dim / 2 * sizeof(float2) + sizeof(RopeToken)) + 16;
  return launch_dependent(rope_kernel<T, FP8, INTERLEAVED, V, ITER>, dim3((unsigned)ctas), dim3(kRopeThreads), smem,
                          stream, p, tokens);
}

template <typename T, bool FP8, bool INTERLEAVED, int V>
cudaError_t launch_vec(const RopeParams& p, cudaStream_t stream) {
  // one unit a thread while that leaves the grid small (a decode step), else four
  const long long units = (long long)p.num_tokens * (p.num_q_heads + 2 * p.num_kv_heads) * (p.head_size / (2 * V));
  return units < 4ll * 152 * 2 * kRopeThreads ? launch_iter<T, FP8, INTERLEAVED, V, 1>(p, stream)
                                              : launch_iter<T, FP8, INTERLEAVED, V, 4>(p, stream);
}

template <typename T, bool FP8, int VMAX>
cudaError_t launch_type(bool interleaved, const RopeParams& p, cudaStream_t stream) {
  if (interleaved) return launch_vec<T, FP8, true, VMAX>(p, stream);
  // halves: vectors that neither half of the pairs cuts
  const int half = p.rotary_dim / 2;
  if (half % VMAX == 0) return launch_vec<T, FP8, false, VMAX>(p, stream);
  if (half % 2 == 0) return launch_vec<T, FP8, false, 2>(p, stream);
  return launch_vec<T, FP8, false, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope(int dtype, bool interleaved, const RopeParams& p, cudaStream_t stream) {
  if (dtype == PA_F32) return launch_type<float, false, 4>(interleaved, p, stream);
  if (dtype == PA_F16) return launch_type<__half, false, 8>(interleaved, p, stream);
  if (dtype == PA_BF16) return launch_type<__nv_bfloat16, false, 8>(interleaved, p, stream);
  if (dtype == PA_FP8_E4M3) return launch_type<__half, true, 8>(interleaved, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
