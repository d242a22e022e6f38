// pa_fp4_write.cu - rows into and out of a cache held in 4 bits: the quantising append, the same with rotary positions,
// and the read of rows back.
//
// A group is 16 neighbouring elements x of a row: s = e4m3(max |x| / (6 unit)), codes e2m1(x * (1 / (s unit))), every
// step one fp32 operation, so that the bytes are the same whoever writes them (the append inside a decode step, too).
// Eight elements, 16 bytes of a row, are one thread's: a group's maximum takes one shuffle, a row 16 threads.
// Bound by HBM: 256 bytes read and 72 written a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_rope_angle.cuh"

namespace pa {
namespace {

constexpr int kRowThreads = kFp4D / 8;  // threads of a row
constexpr int kThreads = 256;
constexpr int kRows = kThreads / kRowThreads;  // rows that a CTA takes at a time

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = Mma<T>::lo(v.x), f[1] = Mma<T>::hi(v.x), f[2] = Mma<T>::lo(v.y), f[3] = Mma<T>::hi(v.y);
  f[4] = Mma<T>::lo(v.z), f[5] = Mma<T>::hi(v.z), f[6] = Mma<T>::lo(v.w), f[7] = Mma<T>::hi(v.w);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(Mma<T>::pack(f[0], f[1]), Mma<T>::pack(f[2], f[3]), Mma<T>::pack(f[4], f[5]),
                    Mma<T>::pack(f[6], f[7]));
}

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Thread j (0 .. 15) of a row, all 32 lanes of the warp together: elements 8 j .. to their place in the tile at `tile`
// (nullptr: the row is not written), row r of it.
__device__ __forceinline__ void store_row(uint8_t* tile, int r, int j, const float (&f)[8], float unit, float unit6) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const uint32_t scale = fp4_scale_code(amax, unit6);
  const uint32_t codes = fp4_codes8(f, fp4_inverse(scale, unit));
  // the scales of four groups (eight threads) into one word
  uint32_t s = scale | __shfl_down_sync(0xffffffffu, scale, 2) << 8;
  s |= __shfl_down_sync(0xffffffffu, s, 4) << 16;
  if (tile == nullptr) return;
  *reinterpret_cast<uint32_t*>(tile + r * kFp4RowBytes + 4 * j) = codes;
  if (j % 8 == 0) *reinterpret_cast<uint32_t*>(tile + kFp4CodeBytes + r * kFp4RowScales + j / 2) = s;
}

// the block and offset of a token's slot; false: padding, or outside the pool (reported if `report`)
template <typename P>
__device__ __forceinline__ bool find_slot(const P& p, long long slot, bool report, long long& block, int& off) {
  if (slot < 0) return false;
  block = slot / p.block_size;
  off = (int)(slot - block * p.block_size);
  if (block < p.num_blocks) return true;
  if (report) report_error(p.err_flag, PA_DEVERR_SLOT);
  return false;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) fp4_write_kernel(const Fp4Rows p) {
  griddep_wait();
  griddep_launch_dependents();
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kRowThreads;
  const int j = threadIdx.x % kRowThreads, per_token = 2 * p.num_kv_heads;
  const long long t = row / per_token;
  const int h2 = (int)(row - t * per_token), h = h2 % p.num_kv_heads;
  const bool is_v = h2 >= p.num_kv_heads;
  uint8_t* tile = nullptr;
  int off = 0;
  float f[8] = {};
  if (t < p.num_tokens) {
    long long block;
    if (find_slot(p, p.slot_mapping[t], h2 == 0 && j == 0, block, off)) {
      const T* src = static_cast<const T*>(is_v ? p.value : p.key) + t * (is_v ? p.value_stride : p.key_stride) +
                     (size_t)h * kFp4D + 8 * j;
      unpack8<T>(*reinterpret_cast<const uint4*>(src), f);
      tile = (is_v ? p.v_cache : p.k_cache) + fp4_tile(block, p.num_kv_heads, h, p.block_size, off);
    }
  }
  const float unit = is_v ? p.v_scale : p.k_scale;
  store_row(tile, off % kFp4Tokens, j, f, unit, __fmul_rn(6.f, unit));
}

// Rows back in 16 bits: each is the fp32 product e2m1 * scale * unit, rounded once.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp4_read_kernel(const Fp4Rows p) {
  griddep_wait();
  griddep_launch_dependents();
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kRowThreads;
  const int j = threadIdx.x % kRowThreads, per_token = 2 * p.num_kv_heads;
  const long long t = row / per_token;
  if (t >= p.num_tokens) return;
  const int h2 = (int)(row - t * per_token), h = h2 % p.num_kv_heads;
  const bool is_v = h2 >= p.num_kv_heads;
  long long block;
  int off;
  if (!find_slot(p, p.slot_mapping[t], h2 == 0 && j == 0, block, off)) return;
  const uint8_t* tile =
      (is_v ? p.v_cache : p.k_cache) + fp4_tile(block, p.num_kv_heads, h, p.block_size, off);
  const int r = off % kFp4Tokens;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(tile + r * kFp4RowBytes + 4 * j);
  const uint32_t s2 = fp4_scales_to_half(tile[kFp4CodeBytes + r * kFp4RowScales + j / 2]);
  uint32_t x[4];
  fp4_to_half(codes, x[0], x[1], x[2], x[3]);
  const float unit = is_v ? p.v_scale : p.k_scale;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t y = half_mul(x[i], half_dup_lo(s2));
    f[2 * i] = Mma<__half>::lo(y) * unit;
    f[2 * i + 1] = Mma<__half>::hi(y) * unit;
  }
  T* dst = static_cast<T*>(is_v ? p.value : p.key) + t * (is_v ? p.value_stride : p.key_stride) + (size_t)h * kFp4D + 8 * j;
  *reinterpret_cast<uint4*>(dst) = pack8<T>(f);
}

// Rotary positions with the write.  A CTA takes one token: its first threads work out the pairs' angles, then its rows
// (query heads, keys, values) go by 16 at a time.  A turned row is rounded to T first, then held in 4 bits, so that the
// cache is what the append makes of the same rows in T.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) fp4_rope_kernel(const RopeAxesParams p) {
  __shared__ float2 cs[kFp4D / 2];
  __shared__ __align__(16) T rows[kRows][kFp4D];
  const int t = blockIdx.x, half = p.rotary_dim / 2;
  griddep_wait();
  griddep_launch_dependents();
  long long block;
  int off;
  if (!find_slot(p, p.slot_mapping[t], threadIdx.x == 0, block, off)) return;
  if (threadIdx.x < half)
    cs[threadIdx.x] = turn_of(turn_fraction(p.inv_freq[threadIdx.x]),
                              p.positions[(long long)p.axis[threadIdx.x] * p.num_tokens + t], p.magnitude);
  __syncthreads();
  const int w = threadIdx.x / kRowThreads, j = threadIdx.x % kRowThreads;
  const int per_token = p.num_q_heads + 2 * p.num_kv_heads;
  for (int first = 0; first < per_token; first += kRows) {
    const int row = first + w;
    const bool real = row < per_token, is_q = row < p.num_q_heads, is_v = row >= p.num_q_heads + p.num_kv_heads;
    const int h = is_q ? row : (row - p.num_q_heads) % p.num_kv_heads;
    float f[8] = {};
    if (real) {
      const T* src = is_q ? static_cast<const T*>(p.q) + t * p.q_stride
                          : is_v ? static_cast<const T*>(p.value) + t * p.value_stride
                                 : static_cast<const T*>(p.key) + t * p.key_stride;
      const uint4 x = *reinterpret_cast<const uint4*>(src + (size_t)h * kFp4D + 8 * j);
      unpack8<T>(x, f);
      *reinterpret_cast<uint4*>(&rows[w][8 * j]) = x;
    }
    __syncwarp();  // a row belongs to one warp
    if (real && !is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = 8 * j + i;
        if (e < p.rotary_dim) {
          const bool second = INTERLEAVED ? e & 1 : e >= half;
          const int pair = INTERLEAVED ? e / 2 : second ? e - half : e;
          const float other =
              to_f32(rows[w][INTERLEAVED ? e ^ 1 : second ? e - half : e + half]);
          const float2 c = cs[pair];
          f[i] = second ? c.x * f[i] + c.y * other : c.x * f[i] - c.y * other;
        }
      }
    }
    const uint4 y = pack8<T>(f);
    if (real && is_q)
      *reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + t * p.q_out_stride + (size_t)h * kFp4D + 8 * j) = y;
    unpack8<T>(y, f);
    uint8_t* tile = real && !is_q ? static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                                        fp4_tile(block, p.num_kv_heads, h, p.block_size, off)
                                  : nullptr;
    const float unit = is_v ? p.v_scale : p.k_scale;
    store_row(tile, off % kFp4Tokens, j, f, unit, __fmul_rn(6.f, unit));
    __syncwarp();  // the row has been read before the next one takes its place
  }
}

template <typename T>
cudaError_t launch_rows_of(bool read, const Fp4Rows& p, cudaStream_t stream) {
  const long long rows = 2ll * p.num_kv_heads * p.num_tokens;
  const dim3 grid((unsigned)((rows + kRows - 1) / kRows));
  return read ? launch_dependent(fp4_read_kernel<T>, grid, dim3(kThreads), 0, stream, p)
              : launch_dependent(fp4_write_kernel<T>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_fp4_write(int row_dtype, const Fp4Rows& p, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_rows_of<__half>(false, p, stream) : launch_rows_of<__nv_bfloat16>(false, p, stream);
}
cudaError_t launch_fp4_read(int row_dtype, const Fp4Rows& p, cudaStream_t stream) {
  return row_dtype == PA_F16 ? launch_rows_of<__half>(true, p, stream) : launch_rows_of<__nv_bfloat16>(true, p, stream);
}
cudaError_t launch_fp4_rope(int row_dtype, bool interleaved, const RopeAxesParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.num_tokens), block(kThreads);
  if (row_dtype == PA_F16)
    return interleaved ? launch_dependent(fp4_rope_kernel<__half, true>, grid, block, 0, stream, p)
                       : launch_dependent(fp4_rope_kernel<__half, false>, grid, block, 0, stream, p);
  return interleaved ? launch_dependent(fp4_rope_kernel<__nv_bfloat16, true>, grid, block, 0, stream, p)
                     : launch_dependent(fp4_rope_kernel<__nv_bfloat16, false>, grid, block, 0, stream, p);
}

}  // namespace pa
