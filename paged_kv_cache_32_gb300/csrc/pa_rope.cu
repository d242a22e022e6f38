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
// exactly.  What is left of rounding is that of 1 / 2 pi and of its product with f_j to 53
// bits, together at most 2^-52 t f_j / 2 pi turns (f_j <= 1 and any int32 t: 2^-23.6), and of
// the fraction to fp32 for sincospif.
// One angle per (token, pair) and CTA, kept in shared memory for all heads.
//
// Bound by HBM bandwidth: 4 + (cache / element) bytes moved an element.  Work is
// cut into units of two vectors of V elements (elements V u .. of both halves of
// the pairs, or 2 V neighbouring elements), D / 2 V units a head whatever r is.
// A CTA walks groups of tokens, or a part of each (where a token has more units
// than its threads hold, or several tokens cut into parts fill them better); a
// thread has the same units of every group, so their heads, elements and offsets
// are worked out once, and the next group's loads are issued as soon as the
// present one is stored.  Two more warps, a thread
// per pair, work out the next group's slots and angles meanwhile (their chain of
// a load, a 64-bit division and a sine is longer than a group's stores).  (c, s)
// lie in shared memory so that the units of a head read neighbouring banks: by
// pairs of elements, then units.  The fixed-point frequencies, which take fp64
// operations (two a clock and SM here), are made once per CTA.
//
// Values of an FP8 cache lie with a dimension's 16 tokens side by side: warps of
// their own (the grid's first CTAs) take up to 16 tokens of one head, quantise
// them into shared memory and write each run of slots that follow one another
// inside a 16-token group with as few stores as its length allows, 16 bytes for
// a whole group (9001 tokens, 64 / 8 heads: single bytes from the units 118 us, these 74).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_rope.h"

namespace pa {
namespace {

// Threads with units (two warps more for the angles), CTAs of an SM, units of a thread.  Measured on a prompt of
// 9001 tokens, 64 / 8 heads of 128, bf16 (halves), and of 24576, 32 / 32 heads, fp16 (neighbours): 60 and 183 us
// (6.1 and 6.6 TB/s; 57 and 182 with groups in parts); 256 x 2 x 4: 85 and 318, 256 x 3 x 2: 78 and 248, 256 x 4 x 2: 101 and 329, 384 x 3 x 2: 95
// and 311, 768 x 1 x 1: 72 and 217 us.  More rows at once than these 304 tokens lose more in DRAM than the
// loads in flight gain; issuing a unit's next load right after its stores, between its neighbours', made a
// warp's waits cover loads just issued (71 and 216 us).
constexpr int kRopeThreads = 384;
constexpr int kRopeResident = 2;
// narrow vectors, for halves that no 16 bytes divide: more units a thread (the 9001 tokens with 36 and 34 turned
// elements: 85 and 150 us; before a token's parts were evened out 95 and 167, then with two units 136 and 208, with
// eight, which spill, 145 and 332)
template <typename T, int V>
constexpr int kUnits = sizeof(T) * V >= 16 ? 2 : 4;

// Vectors of V elements of T, moved with one access; 16-bit pairs are handled as 32-bit words.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
  __device__ __forceinline__ void get(float (&f)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = x[i];
    } else if constexpr (V == 1) {
      f[0] = Mma<T>::lo(reinterpret_cast<const unsigned short&>(x[0]));
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[2 * i] = Mma<T>::lo(w[i]), f[2 * i + 1] = Mma<T>::hi(w[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = from_float<T>(f[i]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = Mma<T>::pack(f[2 * i], f[2 * i + 1]);
    }
  }
};

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

// E4M3 codes of V values over `scale`, packed in order
template <int V>
__device__ __forceinline__ Vec<uint8_t, V> codes_of(const float (&f)[V], float scale) {
  Vec<uint8_t, V> y;
  if constexpr (V == 1) {
    y.x[0] = code_of(f[0], scale);
  } else {
    unsigned short* h = reinterpret_cast<unsigned short*>(y.x);
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      h[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale)),
                                      __NV_SATFINITE, __NV_E4M3);
  }
  return y;
}

constexpr int kMaxHalf = 64;  // pairs of the largest head
constexpr int kRopeWarps = (kRopeThreads + kMaxHalf) / 32;
constexpr int kMaxGroup = 16; // tokens of a group

// How the units are dealt out: groups of `tokens` tokens, each cut into `parts` parts of `part_units` units (a
// multiple of the units of a head).  The CTAs of a part walk its groups.
struct RopePlan {
  int tokens, parts, part_units, groups;
  int log2_per_head;  // units of a head
  int value_ctas;     // FP8: the grid's first CTAs, whose warps take the values of value_tokens tokens of one kv head
  int value_tokens;
};

// One warp: values of kv head `head` into an FP8 cache, through `codes` (kValueTokens rows of kCodeRow bytes): the runs
// of slots, inside one 16-token group each, that start with one of the tokens t0 .. t0 + n - 1 (n <= 16; a run that
// started earlier belongs to the warp of its start, one that goes on past them to this one).  So every group that a
// prompt fills is written with 16-byte stores, wherever it starts in the batch.
constexpr int kValueTokens = 16;
constexpr int kCodeRow = 128 + 8;  // a token's codes, padded
__device__ __forceinline__ void fp8_values(const RopeParams& p, int t0, int n, int head, uint8_t* codes) {
  constexpr int D = 128;  // of every FP8 cache
  const int lane = threadIdx.x & 31;
  const bool real = t0 + lane < p.num_tokens;
  // the tokens' rows (256 bytes each) are on their way while the slots are looked at
  if (lane < 2 * n)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __half*>(p.value) +
                                                  (long long)(t0 + lane / 2) * p.value_stride + (size_t)head * D + lane % 2 * 64));
  long long slot = real ? p.slot_mapping[t0 + lane] : -1;
  long long before = lane == 0 && t0 > 0 ? p.slot_mapping[t0 - 1] : -1;
  // the tokens outside the pool end a run like padding
  if (slot >= (long long)p.num_blocks * p.block_size) {
    if (head == 0 && lane < n) report_error(p.err_flag, PA_DEVERR_SLOT);
    slot = -1;
  }
  const long long left = __shfl_up_sync(0xffffffffu, slot, 1);
  if (lane > 0) before = left;
  // where a lane's token goes, and whether it starts a run
  long long at = 0;
  int off = 0;
  if (slot >= 0) {
    const long long block = slot / p.block_size;
    off = (int)(slot - block * p.block_size);
    at = ((block * p.num_kv_heads + head) * p.block_size + off / 16 * 16) * D + off % 16;
  }
  const unsigned all_starts =
      __ballot_sync(0xffffffffu, !real || slot < 0 || slot != before + 1 || off % 16 == 0);
  const unsigned live = __ballot_sync(0xffffffffu, slot >= 0);
  const unsigned mine = all_starts & live & (0xffffffffu >> (32 - n));
  if (mine == 0) return;
  // (a run has at most 16 tokens, so the next start after the n tokens is among the 32)
  const int first = __ffs(mine) - 1, last = __ffs(all_starts & (0xffffffffu << n)) - 1;
  for (int base = first; base < last; base += kValueTokens) {
    const int end = min(last, base + kValueTokens);
    Vec<__half, 8> x[kValueTokens / 2];  // lane: dimensions 8 (lane % 16) .. of the tokens base + lane / 16 + 2 i
    const __half* src =
        static_cast<const __half*>(p.value) + (long long)(t0 + base) * p.value_stride + (size_t)head * D + 8 * (lane & 15);
#pragma unroll
    for (int i = 0; i < kValueTokens / 2; ++i) {
      const int t = (lane >> 4) + 2 * i;
      if (base + t < end) x[i] = *reinterpret_cast<const Vec<__half, 8>*>(src + (long long)t * p.value_stride);
    }
    __syncwarp();  // the codes of the tokens before have been read
#pragma unroll
    for (int i = 0; i < kValueTokens / 2; ++i) {
      const int t = (lane >> 4) + 2 * i;
      if (base + t < end) {
        float f[8];
        x[i].get(f);
        *reinterpret_cast<Vec<uint8_t, 8>*>(codes + t * kCodeRow + 8 * (lane & 15)) = codes_of(f, p.v_scale);
      }
    }
    __syncwarp();
    for (int a = base; a < end;) {
      const unsigned later = a < 31 ? all_starts & (0xffffffffu << (a + 1)) : 0u;
      const int next = later ? min(end, __ffs(later) - 1) : end, len = next - a;
      const long long to = __shfl_sync(0xffffffffu, at, a);
      const int o = __shfl_sync(0xffffffffu, off, a) % 16;
      if ((live >> a) & 1u) {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const int d = 32 * j + lane;
          const uint8_t* from = codes + (a - base) * kCodeRow + d;
          uint8_t* dst = static_cast<uint8_t*>(p.v_cache) + to + d * 16;
          auto word = [&](int i) {
            return from[i * kCodeRow] | from[(i + 1) * kCodeRow] << 8 | from[(i + 2) * kCodeRow] << 16 |
                   (uint32_t)from[(i + 3) * kCodeRow] << 24;
          };
          if (len == 16) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(word(0), word(4), word(8), word(12));
          } else {
            for (int i = 0; i < len;) {
              if ((o + i) % 4 == 0 && len - i >= 4) {
                *reinterpret_cast<uint32_t*>(dst + i) = word(i);
                i += 4;
              } else {
                dst[i] = from[i * kCodeRow];
                ++i;
              }
            }
          }
        }
      }
      a = next;
    }
  }
}

// T: queries, keys, values; FP8: the cache holds E4M3 codes (else T); V: elements of a vector
template <typename T, bool FP8, bool INTERLEAVED, int V>
__global__ void __launch_bounds__(kRopeThreads + kMaxHalf, kRopeResident) rope_kernel(const RopeParams p, const RopePlan plan) {
  // (c, s) of token, pair; two groups in turn (FP8: or the values' codes)
  constexpr int kBatch = kUnits<T, V>;
  constexpr int kCs = kMaxGroup * kMaxHalf, kCodes = FP8 ? kRopeWarps * kValueTokens * kCodeRow / 16 : 0;
  __shared__ __align__(16) float2 cs_all[2][kCs > kCodes ? kCs : kCodes];
  // cache row (block * Hkv * B + offset) of the token's kv head 0; < 0: the token is skipped
  __shared__ long long tok_all[2][kMaxGroup];
  const int half = p.rotary_dim / 2, D = p.head_size, per_head = 1 << plan.log2_per_head;
  const int heads = p.num_q_heads + (FP8 ? 1 : 2) * p.num_kv_heads;  // (FP8: values apart)
  const int per_token = heads << plan.log2_per_head;
  // pair V u + i of a token at [i / 2][u][i % 2] (V = 1: [u])
  auto cs_at = [&](int u, int i) { return V == 1 ? u : ((i / 2) * per_head + u) * 2 + i % 2; };
  griddep_wait();
  griddep_launch_dependents();
  int cta = blockIdx.x;
  if constexpr (FP8) {
    if (cta < plan.value_ctas) {
      const int w = threadIdx.x >> 5, unit = cta * kRopeWarps + w, t0 = unit / p.num_kv_heads * plan.value_tokens;
      if (t0 < p.num_tokens)
        fp8_values(p, t0, min(plan.value_tokens, p.num_tokens - t0), unit % p.num_kv_heads,
                   reinterpret_cast<uint8_t*>(cs_all) + w * (kValueTokens * kCodeRow));
      return;
    }
    cta -= plan.value_ctas;
  }
  const int part = cta % plan.parts;
  const int first = cta / plan.parts, step = (gridDim.x - plan.value_ctas) / plan.parts;
  // this part's units of a group and the tokens they belong to
  const int begin = part * plan.part_units, end = min(plan.tokens * per_token, begin + plan.part_units);
  const int tok_lo = begin / per_token, tok_hi = (end + per_token - 1) / per_token;

  if (threadIdx.x >= kRopeThreads) {
    // ---- slots and angles, one group ahead of the units
    const int j = threadIdx.x - kRopeThreads;
    const unsigned long long f = j < half ? turn_fraction(p.inv_freq[j]) : 0ull;
    // lane t: slot and position of token t of a group, loaded a group ahead
    const int lane = threadIdx.x & 31;
    auto fetch = [&](int group, long long& slot, int& position) {
      const long long t = (long long)group * plan.tokens + lane;
      const bool real = lane < plan.tokens && t < p.num_tokens;
      slot = real ? p.slot_mapping[t] : -1;
      position = real ? p.positions[t] : 0;
    };
    long long slot;
    int position, buf = 0;
    fetch(first, slot, position);
    for (int group = first; group < plan.groups; group += step, buf ^= 1) {
      const int nt = min(plan.tokens, p.num_tokens - group * plan.tokens);
      if (j < nt) {
        long long row = -1;
        if (slot >= 0) {
          const long long block = slot / p.block_size;
          if (block < p.num_blocks)
            row = block * p.num_kv_heads * p.block_size + (slot - block * p.block_size);
          else
            report_error(p.err_flag, PA_DEVERR_SLOT);
        }
        tok_all[buf][j] = row;
      }
      for (int t = tok_lo; t < min(nt, tok_hi); ++t) {
        const long long at = __shfl_sync(0xffffffffu, position, t);
        if (j < half) {
          const long long turns = (long long)(f * (unsigned long long)at);
          float s, c;
          sincospif(__ll2float_rn(turns) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns in [-1, 1]
          cs_all[buf][t * kMaxHalf + cs_at(j / V, j % V)] = make_float2(c * p.magnitude, s * p.magnitude);
        }
      }
      fetch(group + step, slot, position);
      __syncthreads();
    }
    return;
  }
  // ---- this thread's units: the same heads and elements of every group
  enum { kNone = -1, kQ = 0, kK = 1, kV = 2 };
  int kind[kBatch], tl[kBatch], unit[kBatch], apart[kBatch];
  const T* src[kBatch];     // in token 0's row of the group's first token's array
  long long dst[kBatch];    // elements from the row of q_out, or of kv head 0 in the cache
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int i = begin + k * kRopeThreads + threadIdx.x;
    kind[k] = kNone;
    tl[k] = unit[k] = apart[k] = 0;
    src[k] = nullptr;
    dst[k] = 0;
    if (i >= end) continue;
    tl[k] = i / per_token;
    const int r = i - tl[k] * per_token, h = r >> plan.log2_per_head;
    unit[k] = r & (per_head - 1);
    const bool cut = !INTERLEAVED && unit[k] * V < half;  // a vector of each half, else two side by side
    const int e0 = cut ? unit[k] * V : unit[k] * 2 * V;
    apart[k] = cut ? half : V;
    const int hk = (h - p.num_q_heads) % p.num_kv_heads;
    kind[k] = h < p.num_q_heads ? kQ : h < p.num_q_heads + p.num_kv_heads ? kK : kV;
    if (kind[k] == kQ) {
      src[k] = static_cast<const T*>(p.q) + tl[k] * p.q_stride + (size_t)h * D + e0;
      dst[k] = tl[k] * p.q_out_stride + (long long)h * D + e0;
    } else {
      src[k] = kind[k] == kK ? static_cast<const T*>(p.key) + tl[k] * p.key_stride + (size_t)hk * D + e0
                             : static_cast<const T*>(p.value) + tl[k] * p.value_stride + (size_t)hk * D + e0;
      dst[k] = (long long)hk * p.block_size * D + e0;
    }
  }
  Vec<T, V> a[kBatch], b[kBatch];
  auto load = [&](int t0, int k) {
    if (kind[k] == kNone || t0 + tl[k] >= p.num_tokens) return;
    const long long stride = kind[k] == kQ ? p.q_stride : kind[k] == kK ? p.key_stride : p.value_stride;
    const T* x = src[k] + t0 * stride;
    a[k] = *reinterpret_cast<const Vec<T, V>*>(x);
    b[k] = *reinterpret_cast<const Vec<T, V>*>(x + apart[k]);
  };
#pragma unroll
  for (int k = 0; k < kBatch; ++k) load(first * plan.tokens, k);

  int buf = 0;
  for (int group = first; group < plan.groups; group += step, buf ^= 1) {
    const int t0 = group * plan.tokens, nt = min(plan.tokens, p.num_tokens - t0);
    const float2* cs = cs_all[buf];
    const long long* tok = tok_all[buf];
    __syncthreads();  // this group's are written, and the ones before, whose buffers come next, have been read
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const long long row = tok[tl[k]];
      // (a row < 0: padding, or a slot outside the pool)
      if (kind[k] != kNone && tl[k] < nt && row >= 0) {
        float u[V], w[V];
        a[k].get(u);
        b[k].get(w);
        if (kind[k] != kV && unit[k] * V < half) {
          const float2* ct = cs + tl[k] * kMaxHalf;
          float2 c[V];
          if constexpr (V == 1) {
            c[0] = ct[cs_at(unit[k], 0)];
          } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
              const float4 x4 = *reinterpret_cast<const float4*>(ct + cs_at(unit[k], i));
              c[i] = make_float2(x4.x, x4.y), c[i + 1] = make_float2(x4.z, x4.w);
            }
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            // pair V unit + i: elements i of both vectors, or neighbours (2i, 2i + 1) of the two in a row
            if (!INTERLEAVED || unit[k] * V + i < half) {
              float& x0 = !INTERLEAVED ? u[i] : 2 * i < V ? u[(2 * i) % V] : w[(2 * i) % V];
              float& x1 = !INTERLEAVED ? w[i] : 2 * i + 1 < V ? u[(2 * i + 1) % V] : w[(2 * i + 1) % V];
              const float y0 = c[i].x * x0 - c[i].y * x1, y1 = c[i].x * x1 + c[i].y * x0;
              x0 = y0, x1 = y1;
            }
          }
        }
        if (kind[k] == kQ || !FP8) {
          T* d = kind[k] == kQ ? static_cast<T*>(p.q_out) + t0 * p.q_out_stride
                               : static_cast<T*>(kind[k] == kK ? p.k_cache : p.v_cache) + row * D;
          Vec<T, V> y, z;
          y.set(u);
          z.set(w);
          *reinterpret_cast<Vec<T, V>*>(d + dst[k]) = y;
          *reinterpret_cast<Vec<T, V>*>(d + dst[k] + apart[k]) = z;
        } else {
          uint8_t* d = static_cast<uint8_t*>(p.k_cache) + row * D + dst[k];
          *reinterpret_cast<Vec<uint8_t, V>*>(d) = codes_of(u, p.k_scale);
          *reinterpret_cast<Vec<uint8_t, V>*>(d + apart[k]) = codes_of(w, p.k_scale);
        }
      }
    }
    if (group + step < plan.groups) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) load((group + step) * plan.tokens, k);
    }
  }
}

template <typename T, bool FP8, bool INTERLEAVED, int V>
cudaError_t launch_vec(const RopeParams& p, cudaStream_t stream) {
  RopePlan plan;
  const int per_head = p.head_size / (2 * V);
  plan.log2_per_head = 0;
  while ((1 << plan.log2_per_head) < per_head) ++plan.log2_per_head;
  const long long per_token = (long long)(p.num_q_heads + (FP8 ? 1 : 2) * p.num_kv_heads) * per_head;
  constexpr int kCtas = 152 * kRopeResident;  // of a GB300 (elsewhere slower, not wrong: no CTA waits for another)
  // units of a CTA and group: as many as its threads hold, or, while that leaves SMs idle (a decode step), fewer
  long long most = (long long)kUnits<T, V> * kRopeThreads;
  while (most > kRopeThreads && per_token * p.num_tokens < kCtas * most) most /= 2;
  plan.tokens = (int)(most / per_token);
  plan.tokens = plan.tokens < 1 ? 1 : plan.tokens > kMaxGroup ? kMaxGroup : plan.tokens;
  plan.parts = plan.tokens > 1 ? 1 : (int)((per_token + most - 1) / most);
  auto groups = [&](int tokens) { return ((long long)p.num_tokens + tokens - 1) / tokens; };
  auto walkers = [&](int parts) { return (long long)(kCtas / parts > 0 ? kCtas / parts : 1); };  // CTAs of a part
  auto rounds = [&](int tokens, int parts) { return (groups(tokens) + walkers(parts) - 1) / walkers(parts); };
  // a prompt's groups are of the size that takes the fewest rounds, by at least a twentieth, since then the threads
  // hold most units: 512 units a token and room for 768: three tokens in two parts, not one in one (9001 tokens, 64 / 8
  // heads, bf16: 60.2 -> 57.3 us; 13619 tokens, 40 / 8 heads, fp32: 138 -> 119; an FP8 cache of 40 heads a token, whose
  // pace its conversions set, 85 -> 90)
  long long best = rounds(plan.tokens, plan.parts);
  for (int tokens = 1; best > 4 && tokens <= kMaxGroup; ++tokens) {
    const int parts = (int)((per_token * tokens + most - 1) / most);
    if (rounds(tokens, parts) * 20 <= best * 19) {
      best = rounds(tokens, parts);
      plan.tokens = tokens;
      plan.parts = parts;
    }
  }
  const long long group_units = per_token * plan.tokens;
  plan.part_units = (int)((group_units + plan.parts - 1) / plan.parts + per_head - 1) / per_head * per_head;
  plan.groups = (int)groups(plan.tokens);
  // (a step's tokens lie in groups of their own: fewer a warp, more warps)
  plan.value_tokens = p.num_tokens <= 256 ? 1 : p.num_tokens <= 2048 ? 4 : kValueTokens;
  const long long value_warps =
      ((long long)p.num_tokens + plan.value_tokens - 1) / plan.value_tokens * p.num_kv_heads;
  plan.value_ctas = FP8 ? (int)((value_warps + kRopeWarps - 1) / kRopeWarps) : 0;
  const int grid = plan.value_ctas + (int)std::min(groups(plan.tokens), walkers(plan.parts)) * plan.parts;
  return launch_dependent(rope_kernel<T, FP8, INTERLEAVED, V>, dim3((unsigned)grid), dim3(kRopeThreads + kMaxHalf), 0, stream, p,
                          plan);
}

template <typename T, bool FP8, int VMAX>
cudaError_t launch_type(bool interleaved, const RopeParams& p, cudaStream_t stream) {
  if (interleaved) return launch_vec<T, FP8, true, VMAX>(p, stream);
  // halves: vectors that neither half of the pairs cuts
  const int half = p.rotary_dim / 2;
  if (half % VMAX == 0) return launch_vec<T, FP8, false, VMAX>(p, stream);
  if (VMAX > 4 && half % 4 == 0) return launch_vec<T, FP8, false, 4>(p, stream);
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
