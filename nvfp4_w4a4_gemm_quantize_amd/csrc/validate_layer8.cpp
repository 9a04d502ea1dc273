// Host-side argument validation of the attention layer in 8 bits (no HIP dependency).
#include "validate_layer8.h"

#include <math.h>

#include "../../include/nvfp4.h"
#include "validate_serving.h"

namespace nvfp4 {

static bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

static int validate_rotary_dim(int rotary_dim) {
  if (rotary_dim <= 0) return NVFP4_ESHAPE;
  return rotary_dim % 16 || rotary_dim > 1024 ? NVFP4_EUNSUPPORTED : NVFP4_OK;
}

int make_rotary_steps(int rotary_dim, double base, int scaling, double factor, double original_length,
                      double slow_turns, double fast_turns, const double* pair_factors, uint64_t* steps,
                      double* amplitude) {
  const int rc = validate_rotary_dim(rotary_dim);
  if (rc) return rc;
  const bool ramp = scaling == NVFP4_ROPE_YARN || scaling == NVFP4_ROPE_WAVELENGTH;
  if (!steps || !amplitude || scaling < NVFP4_ROPE_NONE || scaling > NVFP4_ROPE_WAVELENGTH) return NVFP4_EINVAL;
  if (!(base > 1) || !isfinite(base)) return NVFP4_EINVAL;
  if (scaling != NVFP4_ROPE_NONE && (!(factor >= 1) || !isfinite(factor))) return NVFP4_EINVAL;
  if (ramp && (!(original_length > 0) || !isfinite(original_length) || !(slow_turns > 0) || !(fast_turns > slow_turns) ||
               !isfinite(fast_turns)))
    return NVFP4_EINVAL;
  const int n = rotary_dim / 2;
  if (pair_factors)
    for (int i = 0; i < n; ++i)
      if (!(pair_factors[i] > 0) || !isfinite(pair_factors[i])) return NVFP4_EINVAL;

  const long double two_pi = 6.283185307179586476925286766559005768L;
  long double b = base;
  if (scaling == NVFP4_ROPE_NTK) b *= powl((long double)factor, (long double)rotary_dim / (rotary_dim - 2));
  // YaRN: the pairs between the one that makes fast_turns over the original length and the one that makes slow_turns
  long double first = 0, last = 0;
  if (scaling == NVFP4_ROPE_YARN) {
    auto pair_of = [&](double turns) { return rotary_dim * logl(original_length / (turns * two_pi)) / (2 * logl(b)); };
    first = fmaxl(floorl(pair_of(fast_turns)), 0);
    last = fminl(ceill(pair_of(slow_turns)), rotary_dim - 1);
  }
  for (int i = 0; i < n; ++i) {
    const long double own = powl(b, -2.0L * i / rotary_dim) / two_pi;   // turns a position
    long double w = own;
    if (scaling == NVFP4_ROPE_LINEAR) w = own / factor;
    if (scaling == NVFP4_ROPE_YARN) {
      const long double r = fminl(fmaxl((i - first) / fmaxl(last - first, 0.001L), 0), 1);
      w = own / factor * r + own * (1 - r);
    }
    if (scaling == NVFP4_ROPE_WAVELENGTH) {
      const long double keep = fminl(fmaxl((original_length * own - slow_turns) / ((long double)fast_turns - slow_turns), 0), 1);
      w = own * keep + own / factor * (1 - keep);
    }
    if (pair_factors) w /= pair_factors[i];
    w -= floorl(w);                                                     // whole turns are none
    const long double units = rintl(ldexpl(w, 64));
    steps[i] = units >= ldexpl(1, 64) ? 0 : (uint64_t)units;
  }
  *amplitude = scaling == NVFP4_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
  return NVFP4_OK;
}

int validate_rotation(const void* positions, const void* steps, int rotary_dim, int layout, double amplitude,
                      int head_dim, int64_t tokens) {
  const int rc = validate_rotary_dim(rotary_dim);
  if (rc) return rc;
  if (rotary_dim > head_dim) return NVFP4_ESHAPE;
  if ((layout != NVFP4_ROTARY_HALF && layout != NVFP4_ROTARY_INTERLEAVED) || !isfinite(amplitude)) return NVFP4_EINVAL;
  if (tokens == 0) return NVFP4_OK;
  if (!positions || !steps) return NVFP4_EINVAL;
  return !aligned(positions, 4) || !aligned(steps, 8) ? NVFP4_EALIGN : NVFP4_OK;
}

int validate_rotary_rows(const void* x, int64_t ld_x, int64_t tokens, int num_heads, int head_dim, const void* out,
                         int64_t ld_out) {
  if (tokens < 0 || num_heads <= 0 || head_dim <= 0) return NVFP4_ESHAPE;
  if (head_dim % 16 || head_dim > 1024 || num_heads > 65536 || tokens > INT32_MAX) return NVFP4_EUNSUPPORTED;
  if (tokens * head_dim >= (int64_t)1 << 36) return NVFP4_EUNSUPPORTED;   // a thread 16 columns of a token: one launch
  const int64_t cols = (int64_t)num_heads * head_dim;
  if (ld_x < cols || ld_out < cols) return NVFP4_ESHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!x || !out) return NVFP4_EINVAL;
  if (x == out && ld_x != ld_out && tokens > 1) return NVFP4_EINVAL;
  if (!aligned(x, 16) || !aligned(out, 16) || ld_x % 8 || ld_out % 8) return NVFP4_EALIGN;
  return NVFP4_OK;
}

int validate_block_cache(const void* k_cache, const void* v_cache, int cache_dtype, int64_t num_pages, int page_size,
                         int num_kv_heads, int head_dim, int64_t page_stride, int64_t head_stride,
                         int64_t token_stride, const void* k_blocks, const void* v_blocks) {
  if (cache_dtype != NVFP4_CACHE_E4M3_BLOCKS && cache_dtype != NVFP4_CACHE_INT8_BLOCKS) return NVFP4_EINVAL;
  // elements of one byte, as an E4M3 cache has them
  const int rc = validate_cache(k_cache, v_cache, NVFP4_CACHE_E4M3, num_pages, page_size, num_kv_heads, head_dim, page_stride,
                                head_stride, token_stride, nullptr, nullptr);
  if (rc) return rc;
  return !k_blocks || !v_blocks ? NVFP4_EINVAL : NVFP4_OK;
}

// Columns of int8 rows: whole 16-byte pieces, and few enough that a sum of products of
// two codes (2^14 at most) fits 32 bits.
static int validate_int8_cols(int64_t cols) {
  if (cols <= 0) return NVFP4_ESHAPE;
  return cols % 16 || cols >= 1 << 17 ? NVFP4_EUNSUPPORTED : NVFP4_OK;
}

int validate_int8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, const void* codes, const void* scales) {
  if (rows < 0) return NVFP4_ESHAPE;
  const int rc = validate_int8_cols(cols);
  if (rc) return rc;
  if (ld_x < cols) return NVFP4_ESHAPE;
  if (rows == 0) return NVFP4_OK;
  if (rows > INT32_MAX) return NVFP4_EUNSUPPORTED;
  if (!x || !codes || !scales) return NVFP4_EINVAL;
  return !aligned(x, 16) || ld_x % 8 || !aligned(codes, 16) || !aligned(scales, 4) ? NVFP4_EALIGN : NVFP4_OK;
}

int validate_w8a8_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n <= 0) return NVFP4_ESHAPE;
  const int rc = validate_int8_cols(k);
  if (rc) return rc;
  // tiles are counted in 32 bits
  return m > INT32_MAX || n > INT32_MAX || ((m + 63) / 64) * ((n + 63) / 64) > INT32_MAX / 64 ? NVFP4_EUNSUPPORTED : NVFP4_OK;
}

int validate_gemm_w8a8(const void* a, const void* a_scale, int64_t m, const void* w, const void* w_scale, int64_t n, int64_t k,
                       const void* out, int out_dtype, int64_t ld_out, const void* workspace, size_t workspace_bytes,
                       size_t needed) {
  const int rc = validate_w8a8_sizes(m, n, k);
  if (rc) return rc;
  if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_EINVAL;
  if (ld_out < n) return NVFP4_ESHAPE;
  if (m == 0) return NVFP4_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return NVFP4_EINVAL;
  const unsigned element = out_dtype == NVFP4_OUT_BF16 ? 2 : 4;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(out, element) ||
      !aligned(workspace, 16))
    return NVFP4_EALIGN;
  return workspace && workspace_bytes < needed ? NVFP4_ESIZE : NVFP4_OK;
}

}  // namespace nvfp4
