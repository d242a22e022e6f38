// pa_rope_api.cu - the C-ABI entry points of rotary positions: the frequencies
// (host) and the rotary cache write.  Every host-side check runs before any
// CUDA call, so an argument error launches nothing.
#include <cuda_runtime.h>

#include <math.h>

#include "pa.h"
#include "pa_fp4.h"
#include "pa_rope.h"

using namespace pa::host;

namespace {

constexpr double kTwoPi = 6.283185307179586477;

bool positive(double x) { return x > 0.0 && !isinf(x); }

// The checks that both calls share (of a cache that one of them takes) and their parameters.  *done: there is nothing to
// launch, or the call is refused.
int rope_params(pa::RopeParams& p, bool* done, void* q_out, void* k_cache, void* v_cache, const void* q, const void* key,
                const void* value, int64_t q_out_stride, int64_t q_stride, int64_t key_stride, int64_t value_stride,
                const int32_t* positions, const int64_t* slot_mapping, const double* inv_freq, int32_t num_tokens,
                int32_t num_q_heads, int32_t rotary_dim, int32_t interleaved, float magnitude, const pa_cache_desc* cache,
                float k_scale, float v_scale, int32_t* err_flag) {
  *done = true;
  const int64_t D = cache->head_size;
  if (num_tokens < 0 || num_q_heads < 0) return PA_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > D) return PA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return PA_ERR_INVALID_ARG;
  if (!(magnitude == magnitude) || isinf(magnitude)) return PA_ERR_INVALID_ARG;
  if (k_scale == 0.f) k_scale = 1.f;
  if (v_scale == 0.f) v_scale = 1.f;
  if (cache->dtype == PA_FP8_E4M3 && (!(k_scale > 0.f) || isinf(k_scale) || !(v_scale > 0.f) || isinf(v_scale)))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (k_cache == nullptr || v_cache == nullptr || key == nullptr || value == nullptr || positions == nullptr ||
      slot_mapping == nullptr || inv_freq == nullptr || (num_q_heads > 0 && (q == nullptr || q_out == nullptr)))
    return PA_ERR_NULL_POINTER;
  // rows of one token are dense; tokens may be further apart (views of a fused projection), 16-byte steps
  const int64_t vec = 16 / (cache->dtype == PA_F32 ? 4 : 2);
  const int64_t q_row = num_q_heads * D, kv_row = cache->num_kv_heads * D;
  if (key_stride < kv_row || value_stride < kv_row) return PA_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return PA_ERR_INVALID_ARG;
  const int64_t max_stride = ((int64_t)1 << 44) / num_tokens;
  if (key_stride > max_stride || value_stride > max_stride ||
      (num_q_heads > 0 && (q_stride > max_stride || q_out_stride > max_stride)))
    return PA_ERR_TOO_LARGE;
  if (key_stride % vec != 0 || value_stride % vec != 0 ||
      (num_q_heads > 0 && (q_stride % vec != 0 || q_out_stride % vec != 0)))
    return PA_ERR_MISALIGNED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(key, 16) || !aligned(value, 16) ||
      !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(inv_freq, 8) ||
      (num_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
    return PA_ERR_MISALIGNED;
  // q_out is q itself, or apart from the inputs
  const int64_t e = vec == 4 ? 4 : 2;
  auto overlap = [&](const void* x, int64_t xs, int64_t x_row) {
    const uintptr_t a = (uintptr_t)q_out, b = (uintptr_t)x;
    const uintptr_t a_end = a + ((num_tokens - 1) * q_out_stride + q_row) * e;
    const uintptr_t b_end = b + ((num_tokens - 1) * xs + x_row) * e;
    if (a >= b_end || b >= a_end) return false;
    if (xs != q_out_stride || num_tokens == 1) return true;
    // rows of one buffer, the same distance apart: apart if the columns are
    const int64_t step = xs * e;
    const int64_t d = (int64_t)((a > b ? a - b : b - a) % (uintptr_t)step);
    return a > b ? !(d >= x_row * e && d + q_row * e <= step) : !(d >= q_row * e && d + x_row * e <= step);
  };
  if (num_q_heads > 0 && (((q_out != q || q_out_stride != q_stride) && overlap(q, q_stride, q_row)) ||
                          overlap(key, key_stride, kv_row) || overlap(value, value_stride, kv_row)))
    return PA_ERR_INVALID_ARG;
  // a token's elements are counted in int32
  if (((int64_t)num_q_heads + 2 * (int64_t)cache->num_kv_heads) * D > kInt32Max / 32) return PA_ERR_TOO_LARGE;

  p.q_out = q_out;
  p.q = q;
  p.key = key;
  p.value = value;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.q_out_stride = q_out_stride;
  p.q_stride = q_stride;
  p.key_stride = key_stride;
  p.value_stride = value_stride;
  p.positions = positions;
  p.slot_mapping = slot_mapping;
  p.inv_freq = inv_freq;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.head_size = cache->head_size;
  p.rotary_dim = rotary_dim;
  p.num_blocks = cache->num_blocks;
  p.block_size = cache->block_size;
  p.magnitude = magnitude;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err_flag = err_flag;
  *done = false;
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_rope_frequencies(double* inv_freq, float* magnitude, int32_t rotary_dim, double base,
                        const pa_rope_scaling* scaling) {
  if (inv_freq == nullptr || magnitude == nullptr) return PA_ERR_NULL_POINTER;
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 128 || !positive(base)) return PA_ERR_INVALID_ARG;
  const int r = rotary_dim, method = scaling != nullptr ? scaling->method : PA_ROPE_PLAIN;
  const double factor = scaling != nullptr ? scaling->factor : 1.0;
  if (method < PA_ROPE_PLAIN || method > PA_ROPE_BANDS) return PA_ERR_INVALID_ARG;
  if (method != PA_ROPE_PLAIN && !positive(factor)) return PA_ERR_INVALID_ARG;
  if (method == PA_ROPE_NTK) {
    if (r < 4) return PA_ERR_INVALID_ARG;  // the base's exponent r / (r - 2)
    base *= pow(factor, (double)r / (r - 2));
    if (!positive(base)) return PA_ERR_INVALID_ARG;
  }
  double lo = 0.0, hi = 0.0, mag = 1.0;
  if (method == PA_ROPE_YARN) {
    if (!positive(scaling->original_max_position) || !positive(scaling->beta_fast) ||
        !positive(scaling->beta_slow) || base == 1.0 ||
        !(scaling->attention_factor == 0.0 || positive(scaling->attention_factor)))
      return PA_ERR_INVALID_ARG;
    // the pair whose wavelength makes n turns over the trained length
    auto pair_of = [&](double n) {
      return r * log(scaling->original_max_position / (n * kTwoPi)) / (2.0 * log(base));
    };
    lo = fmax(0.0, floor(pair_of(scaling->beta_fast)));
    hi = fmin(r - 1.0, ceil(pair_of(scaling->beta_slow)));
    mag = scaling->attention_factor > 0.0 ? scaling->attention_factor : factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
    if (isinf((float)mag)) return PA_ERR_INVALID_ARG;
  }
  if (method == PA_ROPE_BANDS &&
      (!positive(scaling->original_max_position) || !positive(scaling->low_freq_factor) ||
       !positive(scaling->high_freq_factor) || !(scaling->high_freq_factor > scaling->low_freq_factor)))
    return PA_ERR_INVALID_ARG;
  for (int j = 0; j < r / 2; ++j) {
    double f = pow(base, -2.0 * j / r);
    if (method == PA_ROPE_LINEAR) f /= factor;
    if (method == PA_ROPE_YARN) {
      const double ramp = fmin(1.0, fmax(0.0, (j - lo) / fmax(hi - lo, 1e-3)));
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    if (method == PA_ROPE_BANDS) {
      const double turns = scaling->original_max_position * f / kTwoPi;  // over the trained length
      const double keep = fmin(1.0, fmax(0.0, (turns - scaling->low_freq_factor) /
                                                  (scaling->high_freq_factor - scaling->low_freq_factor)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    if (!isfinite(f)) return PA_ERR_INVALID_ARG;  // a factor so small that 1 / factor is none
    inv_freq[j] = f;
  }
  *magnitude = (float)mag;
  return PA_OK;
}

int pa_rope_and_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* key, const void* value,
                      int64_t q_out_stride, int64_t q_stride, int64_t key_stride, int64_t value_stride,
                      const int32_t* positions, const int64_t* slot_mapping, const double* inv_freq,
                      int32_t num_tokens, int32_t num_q_heads, int32_t rotary_dim, int32_t interleaved,
                      float magnitude, const pa_cache_desc* cache, float k_scale, float v_scale, int32_t* err_flag,
                      void* stream) {
  int rc = check_cache(cache);
  if (rc != PA_OK) return rc;
  pa::RopeParams p = {};
  bool done;
  rc = rope_params(p, &done, q_out, k_cache, v_cache, q, key, value, q_out_stride, q_stride, key_stride, value_stride,
                   positions, slot_mapping, inv_freq, num_tokens, num_q_heads, rotary_dim, interleaved, magnitude, cache,
                   k_scale, v_scale, err_flag);
  if (done) return rc;
  cudaError_t err = pa::launch_rope(cache->dtype, interleaved != 0, p, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_rope_axes_and_cache(void* q_out, void* k_cache, void* v_cache, const void* q, const void* key, const void* value,
                           int64_t q_out_stride, int64_t q_stride, int64_t key_stride, int64_t value_stride,
                           const int32_t* positions, int32_t num_axes, const uint8_t* pair_axis,
                           const int64_t* slot_mapping, const double* inv_freq, int32_t num_tokens, int32_t num_q_heads,
                           int32_t rotary_dim, int32_t interleaved, float magnitude, const pa_cache_desc* cache,
                           int32_t row_dtype, float k_scale, float v_scale, int32_t* err_flag, void* stream) {
  const bool fp4 = cache != nullptr && cache->dtype == PA_FP4_E2M1;
  int rc = fp4 ? check_cache_fp4(cache) : check_cache(cache);
  if (rc != PA_OK) return rc;
  if (fp4 && row_dtype != PA_F16 && row_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (fp4 && (!fp4_unit_ok(k_scale) || !fp4_unit_ok(v_scale))) return PA_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > pa::kMaxAxes) return PA_ERR_INVALID_ARG;
  pa::RopeAxesParams p = {};
  bool done;
  rc = rope_params(p, &done, q_out, k_cache, v_cache, q, key, value, q_out_stride, q_stride, key_stride, value_stride,
                   positions, slot_mapping, inv_freq, num_tokens, num_q_heads, rotary_dim, interleaved, magnitude, cache,
                   k_scale, v_scale, err_flag);
  if (rc == PA_OK && pair_axis == nullptr && num_axes > 1) rc = PA_ERR_NULL_POINTER;
  for (int j = 0; rc == PA_OK && pair_axis != nullptr && j < rotary_dim / 2; ++j) {
    if (pair_axis[j] >= num_axes) rc = PA_ERR_INVALID_ARG;
    p.axis[j] = pair_axis[j];
  }
  if (done || rc != PA_OK) return rc;
  p.num_axes = num_axes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t err = fp4 ? pa::launch_rope_fp4(row_dtype, interleaved != 0, p, st)
                              : pa::launch_rope_axes(cache->dtype, interleaved != 0, p, st);
  return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
