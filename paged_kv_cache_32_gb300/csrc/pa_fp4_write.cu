// pa_fp4_write.cu - rows into and out of a cache held in 4 bits: the quantising append, the same with rotary positions,
// and the read of rows back.
//
// A group is 16 neighbouring elements x of a row: s = e4m3(max |x| / (6 unit)), codes e2m1(x * (1 / (s unit))), every
// step one fp32 operation, so that the bytes are the same whoever writes them (the append inside a decode step, too).
// A group, 32 bytes of a row, is one thread's, a row 8 threads'.
// Bound by HBM: 256 bytes read and 72 written a row (the read back: the other way round).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_rope_angle.cuh"

namespace pa {
namespace {

constexpr int kRowThreads = kFp4D / 16;  // threads of a row
constexpr int kThreads = 256;
constexpr int kRows = kThreads / kRowThreads;  // rows that a CTA takes at a time

struct Group16 {  // 16 elements in 16 bits
  uint4 a, b;
};
template <typename T>
__device__ __forceinline__ void unpack(const Group16& v, float (&f)[16]) {
  const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[2 * i] = Mma<T>::lo(w[i]), f[2 * i + 1] = Mma<T>::hi(w[i]);
}
template <typename T>
__device__ __forceinline__ Group16 pack(const float (&f)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = Mma<T>::pack(f[2 * i], f[2 * i + 1]);
  return {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}
__device__ __forceinline__ Group16 load_group(const void* src) {
  const uint4* x = static_cast<const uint4*>(src);
  return {__ldg(x), __ldg(x + 1)};
}
__device__ __forceinline__ void store_group(void* dst, const Group16& v) {
  static_cast<uint4*>(dst)[0] = v.a;
  static_cast<uint4*>(dst)[1] = v.b;
}

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Thread j (0 .. 7) of a row, all 32 lanes of the warp together: group j to its place in the tile at `tile` (nullptr: the
// row is not written), row r of it.
__device__ __forceinline__ void store_row(uint8_t* tile, int r, int j, const float (&f)[16], float unit) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
  const uint32_t scale = fp4_scale_code(amax, __fmul_rn(6.f, unit));
  const float inv = fp4_inverse(scale, unit);
  const float lo[8] = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
  const float hi[8] = {f[8], f[9], f[10], f[11], f[12], f[13], f[14], f[15]};
  const uint2 codes = make_uint2(fp4_codes8(lo, inv), fp4_codes8(hi, inv));
  // the scales of four groups into one word
  uint32_t s = scale | __shfl_down_sync(0xffffffffu, scale, 1) << 8;
  s |= __shfl_down_sync(0xffffffffu, s, 2) << 16;
  if (tile == nullptr) return;
  *reinterpret_cast<uint2*>(tile + r * kFp4RowBytes + 8 * j) = codes;
  if (j % 4 == 0) *reinterpret_cast<uint32_t*>(tile + kFp4CodeBytes + r * kFp4RowScales + j) = s;
}

// the block and offset of a token's slot; false: padding, or outside the pool (reported if `report`)
template <typename P>
__device__ __forceinline__ bool find_slot(const P& p, long long slot, bool report, int& block, int& off) {
  if (slot < 0) return false;
  if (slot < (long long)p.num_blocks * p.block_size) {  // (a pool's rows are counted in int32)
    block = (int)slot / p.block_size;
    off = (int)slot - block * p.block_size;
    return true;
  }
  if (report) report_error(p.err_flag, PA_DEVERR_SLOT);
  return false;
}

// Rows of a thread, kRows of the CTA apart: their loads are in flight together.  A prompt's 320016 rows written and read
// back: 44 us (24 + 20, 4.3 and 5.2 TB/s), with four 47; one 16-byte vector a thread, four rows 64 (36 + 28), one row 83.
// A decode step's few rows go to as many CTAs as there are (64 tokens, 8 heads: 1.7 us each).
constexpr int kBatch = 2;

// Row `row` of the tokens' keys and values: token, head, which.  (At most 2^32 - 2 rows.)
struct RowAt {
  unsigned t;
  int h;
  bool is_v;
};
__device__ __forceinline__ RowAt row_at(const Fp4Rows& p, unsigned row) {
  const unsigned per_token = 2u * (unsigned)p.num_kv_heads, t = row / per_token, h2 = row - t * per_token;
  const bool is_v = h2 >= (unsigned)p.num_kv_heads;
  return {t, (int)(is_v ? h2 - p.num_kv_heads : h2), is_v};
}
template <typename T>
__device__ __forceinline__ T* row_ptr(const Fp4Rows& p, const RowAt& r, int j) {
  return static_cast<T*>(r.is_v ? p.value : p.key) + (long long)r.t * (r.is_v ? p.value_stride : p.key_stride) +
         (size_t)r.h * kFp4D + 16 * j;
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) fp4_write_kernel(const Fp4Rows p) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned rows = 2u * (unsigned)p.num_kv_heads * (unsigned)p.num_tokens;
  const unsigned first = blockIdx.x * (unsigned)(kRows * R) + threadIdx.x / kRowThreads;
  const int j = threadIdx.x % kRowThreads;
  RowAt at[R];
  Group16 x[R];
  long long slot[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const unsigned row = first + i * kRows;
    x[i] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    slot[i] = -1;
    at[i] = {0, 0, false};
    if (row < rows) {
      at[i] = row_at(p, row);
      slot[i] = __ldg(p.slot_mapping + at[i].t);
      x[i] = load_group(row_ptr<T>(p, at[i], j));
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    uint8_t* tile = nullptr;
    int block, off = 0;
    if (find_slot(p, slot[i], !at[i].is_v && at[i].h == 0 && j == 0, block, off))
      tile = (at[i].is_v ? p.v_cache : p.k_cache) + fp4_tile(block, p.num_kv_heads, at[i].h, p.block_size, off);
    float f[16];
    unpack<T>(x[i], f);
    store_row(tile, off % kFp4Tokens, j, f, at[i].is_v ? p.v_scale : p.k_scale);
  }
}

// Rows back in 16 bits: each is the fp32 product e2m1 * scale * unit, rounded once.
template <typename T, int R>
__global__ void __launch_bounds__(kThreads) fp4_read_kernel(const Fp4Rows p) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned rows = 2u * (unsigned)p.num_kv_heads * (unsigned)p.num_tokens;
  const unsigned first = blockIdx.x * (unsigned)(kRows * R) + threadIdx.x / kRowThreads;
  const int j = threadIdx.x % kRowThreads;
  RowAt at[R];
  long long slot[R];
  uint2 codes[R];
  uint32_t scale[R];
  bool real[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const unsigned row = first + i * kRows;
    at[i] = {0, 0, false};
    slot[i] = -1;
    if (row < rows) {
      at[i] = row_at(p, row);
      slot[i] = __ldg(p.slot_mapping + at[i].t);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    int block, off;
    codes[i] = make_uint2(0, 0);
    scale[i] = 0;
    real[i] = find_slot(p, slot[i], !at[i].is_v && at[i].h == 0 && j == 0, block, off);
    if (real[i]) {
      const uint8_t* tile = (at[i].is_v ? p.v_cache : p.k_cache) + fp4_tile(block, p.num_kv_heads, at[i].h, p.block_size, off);
      const int r = off % kFp4Tokens;
      codes[i] = *reinterpret_cast<const uint2*>(tile + r * kFp4RowBytes + 8 * j);
      scale[i] = tile[kFp4CodeBytes + r * kFp4RowScales + j];
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!real[i]) continue;
    const uint32_t s2 = half_dup_lo(fp4_scales_to_half(scale[i]));
    uint32_t x[8];
    fp4_to_half(codes[i].x, x[0], x[1], x[2], x[3]);
    fp4_to_half(codes[i].y, x[4], x[5], x[6], x[7]);
    const float unit = at[i].is_v ? p.v_scale : p.k_scale;
    float f[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t y = half_mul(x[k], s2);
      f[2 * k] = Mma<__half>::lo(y) * unit;
      f[2 * k + 1] = Mma<__half>::hi(y) * unit;
    }
    store_group(row_ptr<T>(p, at[i], j), pack<T>(f));
  }
}

// Rotary positions with the write where the halves of the turned elements cut groups of 16 (other rotary sizes:
// pa_rope.cu).  A CTA walks tokens; its first threads work out the pairs' angles, then its rows (query heads, keys,
// values) go by 32 at a time through shared memory, where a warp turns four rows, a lane a pair, before each thread
// takes its group.  A turned row is rounded to T first, then held in 4 bits, so that the cache is what the append makes
// of the rows that the call over a 16-bit cache turns, bit for bit.  (9001 tokens, 64 / 8 heads, 34 turned elements: 83
// us, where 50 would move the bytes; 64 tokens: 4.3 us.  Bound by latencies: a CTA has one token's rows in flight, half of
// the warps fit, and they wait for those loads, for the two barriers a token and for shared memory; HBM 0.46 of its rate,
// issue slots 0.48.)
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) fp4_rope_cut_kernel(const RopeAxesParams p) {
  __shared__ float2 cs[kFp4D / 2];
  __shared__ __align__(16) T rows[kRows][kFp4D];
  const int half = p.rotary_dim / 2, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const bool has_pair = threadIdx.x < half;
  const unsigned long long f = has_pair ? turn_fraction(p.inv_freq[threadIdx.x]) : 0ull;
  const int* positions = p.positions + (has_pair ? (long long)p.axis[threadIdx.x] * p.num_tokens : 0);
  const int w = threadIdx.x / kRowThreads, j = threadIdx.x % kRowThreads;
  const int per_token = p.num_q_heads + 2 * p.num_kv_heads;
  for (long long t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    int block, off;
    if (!find_slot(p, p.slot_mapping[t], threadIdx.x == 0, block, off)) continue;
    __syncthreads();  // the angles of the token before have been used
    if (has_pair) cs[threadIdx.x] = turn_of(f, positions[t], p.magnitude);
    __syncthreads();
    for (int first = 0; first < per_token; first += kRows) {
      const int row = first + w;
      const bool real = row < per_token, is_q = row < p.num_q_heads, is_v = row >= p.num_q_heads + p.num_kv_heads;
      const int h = is_q ? row : (row - p.num_q_heads) % p.num_kv_heads;
      Group16 x = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (real) {
        const T* src = is_q ? static_cast<const T*>(p.q) + t * p.q_stride
                            : is_v ? static_cast<const T*>(p.value) + t * p.value_stride
                                   : static_cast<const T*>(p.key) + t * p.key_stride;
        const uint4* at = reinterpret_cast<const uint4*>(src + (size_t)h * kFp4D + 16 * j);
        x = {at[0], at[1]};  // (not through the read-only path: q_out may be q)
        if (!is_v) store_group(&rows[w][16 * j], x);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 32 / kRowThreads; ++i) {  // the warp's rows
        const int wi = threadIdx.x / 32 * (32 / kRowThreads) + i;
        if (first + wi < p.num_q_heads + p.num_kv_heads) {
          for (int pair = lane; pair < half; pair += 32) {
            float x0 = to_f32(rows[wi][pair]), x1 = to_f32(rows[wi][pair + half]);
            turn_pair(cs[pair], x0, x1);
            rows[wi][pair] = from_float<T>(x0);
            rows[wi][pair + half] = from_float<T>(x1);
          }
        }
      }
      __syncwarp();
      if (real && !is_v) {
        const uint4* at = reinterpret_cast<const uint4*>(&rows[w][16 * j]);
        x = {at[0], at[1]};
      }
      if (real && is_q) store_group(static_cast<T*>(p.q_out) + t * p.q_out_stride + (size_t)h * kFp4D + 16 * j, x);
      if (first + kRows > p.num_q_heads) {  // (rows of keys or values among them)
        float g[16];
        unpack<T>(x, g);
        uint8_t* tile = real && !is_q ? static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                                            fp4_tile(block, p.num_kv_heads, h, p.block_size, off)
                                      : nullptr;
        store_row(tile, off % kFp4Tokens, j, g, is_v ? p.v_scale : p.k_scale);
      }
      __syncwarp();  // the rows have been read before the next ones take their place
    }
  }
}

template <typename T, int R>
cudaError_t launch_batch(bool read, const Fp4Rows& p, long long rows, cudaStream_t stream) {
  const dim3 grid((unsigned)((rows + kRows * R - 1) / (kRows * R)));
  return read ? launch_dependent(fp4_read_kernel<T, R>, grid, dim3(kThreads), 0, stream, p)
              : launch_dependent(fp4_write_kernel<T, R>, grid, dim3(kThreads), 0, stream, p);
}

template <typename T>
cudaError_t launch_rows_of(bool read, const Fp4Rows& p, cudaStream_t stream) {
  const long long rows = 2ll * p.num_kv_heads * p.num_tokens;
  return rows < 152ll * 8 * kRows * kBatch ? launch_batch<T, 1>(read, p, rows, stream)
                                           : launch_batch<T, kBatch>(read, p, rows, stream);
}

}  // namespace

cudaError_t launch_fp4_write(int row_dtype, const Fp4Rows& p, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_rows_of<__half>(false, p, stream) : launch_rows_of<__nv_bfloat16>(false, p, stream);
}
cudaError_t launch_fp4_read(int row_dtype, const Fp4Rows& p, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_rows_of<__half>(true, p, stream) : launch_rows_of<__nv_bfloat16>(true, p, stream);
}
cudaError_t launch_fp4_rope_cut(int row_dtype, const RopeAxesParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)(p.num_tokens < 152 * 4 ? p.num_tokens : 152 * 4)), block(kThreads);
  return row_dtype == PA_F16 ? launch_dependent(fp4_rope_cut_kernel<__half>, grid, block, 0, stream, p)
                             : launch_dependent(fp4_rope_cut_kernel<__nv_bfloat16>, grid, block, 0, stream, p);
}

}  // namespace pa
