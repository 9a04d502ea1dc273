// C ABI entry points of the attention layer in 8 bits: validate, describe, launch.
// Declared and documented in include/nvfp4.h.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/nvfp4.h"
#include "kernels.h"
#include "layer8.h"
#include "validate_layer8.h"
#include "validate_serving.h"

using namespace nvfp4;

static CacheView cache_view(void* k, void* v, int dtype, int64_t num_pages, int page_size, int heads, int dim,
                            int64_t page_stride, int64_t head_stride, int64_t token_stride, const float* k_scale,
                            const float* v_scale, uint8_t* k_blocks, uint8_t* v_blocks) {
  CacheView c{};
  c.k = k;
  c.v = v;
  c.num_pages = num_pages;
  c.page_stride = page_stride;
  c.head_stride = head_stride;
  c.token_stride = token_stride;
  c.fp8 = dtype == NVFP4_CACHE_E4M3;
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  c.blocks = dtype == NVFP4_CACHE_E4M3_BLOCKS ? kBlocksE4m3 : dtype == NVFP4_CACHE_INT8_BLOCKS ? kBlocksInt8 : kBlocksNone;
  c.k_blocks = k_blocks;
  c.v_blocks = v_blocks;
  c.page_shift = page_shift_of(page_size);
  c.heads = heads;
  c.dim = dim;
  return c;
}

static RotaryArgs rotation(const int32_t* positions, const uint64_t* steps, int rotary_dim, int layout, double amplitude) {
  RotaryArgs r{};
  r.steps = steps;
  r.positions = positions;
  r.dim = rotary_dim;
  r.interleaved = layout == NVFP4_ROTARY_INTERLEAVED;
  r.amplitude = amplitude;
  return r;
}

static RotaryRows rotary_rows(const uint16_t* x, int64_t ld_x, int64_t tokens, int heads, int dim, uint16_t* out, int64_t ld_out) {
  RotaryRows r{};
  r.x = x;
  r.out = out;
  r.ld_x = ld_x;
  r.ld_out = ld_out;
  r.tokens = tokens;
  r.heads = heads;
  r.dim = dim;
  return r;
}

extern "C" {

int rotary_steps(int rotary_dim, double base, int scaling, double factor, double original_length, double slow_turns,
                 double fast_turns, const double* pair_factors, uint64_t* steps, double* amplitude) {
  return make_rotary_steps(rotary_dim, base, scaling, factor, original_length, slow_turns, fast_turns, pair_factors, steps,
                           amplitude);
}

int rotary(const uint16_t* x, int64_t ld_x, int64_t tokens, int num_heads, int head_dim, const int32_t* positions,
           const uint64_t* steps, int rotary_dim, int layout, double amplitude, uint16_t* out, int64_t ld_out,
           nvfp4_stream_t stream) {
  int rc = validate_rotary_rows(x, ld_x, tokens, num_heads, head_dim, out, ld_out);
  if (rc) return rc;
  rc = validate_rotation(positions, steps, rotary_dim, layout, amplitude, head_dim, tokens);
  if (rc || tokens == 0) return rc;
  return hip_status(launch_rotary(rotary_rows(x, ld_x, tokens, num_heads, head_dim, out, ld_out),
                                  rotation(positions, steps, rotary_dim, layout, amplitude), (hipStream_t)stream));
}

int paged_kv_append(const uint16_t* q, int64_t ld_q, int num_heads, uint16_t* q_out, int64_t ld_q_out, const uint16_t* k,
                    int64_t ld_k, const uint16_t* v, int64_t ld_v, const int32_t* positions, const int64_t* slots,
                    int64_t tokens, const uint64_t* steps, int rotary_dim, int layout, double amplitude, void* k_cache,
                    void* v_cache, int cache_dtype, int64_t num_pages, int page_size, int num_kv_heads, int head_dim,
                    int64_t page_stride, int64_t head_stride, int64_t token_stride, const float* k_scale,
                    const float* v_scale, uint8_t* k_blocks, uint8_t* v_blocks, nvfp4_stream_t stream) {
  const bool blocks = cache_dtype == NVFP4_CACHE_E4M3_BLOCKS || cache_dtype == NVFP4_CACHE_INT8_BLOCKS;
  if (blocks ? (k_scale || v_scale) : (k_blocks || v_blocks)) return NVFP4_EINVAL;
  int rc = blocks ? validate_block_cache(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride,
                                         head_stride, token_stride, k_blocks, v_blocks)
                  : validate_cache(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride,
                                   head_stride, token_stride, k_scale, v_scale);
  if (rc) return rc;
  rc = validate_paged_kv_write(k, ld_k, v, ld_v, slots, tokens, num_kv_heads, head_dim);
  if (rc) return rc;
  // 2 head_dim threads for 16 tokens, and q's beside them: one launch
  if (tokens * head_dim >= (int64_t)1 << 34) return NVFP4_EUNSUPPORTED;
  if (num_heads < 0) return NVFP4_ESHAPE;
  if (num_heads > 0) {
    rc = validate_rotary_rows(q, ld_q, tokens, num_heads, head_dim, q_out, ld_q_out);
    if (rc) return rc;
  } else if (q || q_out) {
    return NVFP4_EINVAL;
  }
  if (rotary_dim == 0) {
    if (steps) return NVFP4_EINVAL;
  } else {
    rc = validate_rotation(positions, steps, rotary_dim, layout, amplitude, head_dim, tokens);
    if (rc) return rc;
  }
  if (tokens == 0) return NVFP4_OK;
  AppendArgs a{};
  a.q = rotary_rows(q, ld_q, tokens, num_heads, head_dim, q_out, ld_q_out);
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.tokens = tokens;
  a.rot = rotation(positions, steps, rotary_dim, layout, amplitude);
  a.cache = cache_view(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride, head_stride,
                       token_stride, k_scale, v_scale, k_blocks, v_blocks);
  return hip_status(launch_paged_kv_append(a, (hipStream_t)stream));
}

int paged_attention_blocks(const uint16_t* q, int64_t ld_q, int64_t tokens, const int32_t* q_start, const int32_t* seq_lens,
                           int64_t num_requests, int64_t max_new, int64_t max_seq, int num_heads, const void* k_cache,
                           const void* v_cache, int cache_dtype, int64_t num_pages, int page_size, int num_kv_heads,
                           int head_dim, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                           const uint8_t* k_blocks, const uint8_t* v_blocks, const int32_t* block_table, int64_t max_pages,
                           int64_t ld_table, float scale, int64_t window, void* out, int out_dtype, int64_t ld_out, float* lse,
                           void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  int rc = validate_attention_sizes(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new, max_seq);
  if (rc) return rc;
  rc = validate_block_cache(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride, head_stride,
                            token_stride, k_blocks, v_blocks);
  if (rc) return rc;
  if (num_requests == 0) {
    if (!(out_dtype & NVFP4_OUT_CLEAR_PADDING)) return NVFP4_OK;
    rc = validate_attention_padding(tokens, num_heads, head_dim, out, out_dtype, ld_out, lse);
  } else {
    rc = validate_paged_attention(q, ld_q, tokens, q_start, seq_lens, num_heads, head_dim, block_table, max_pages, ld_table, scale,
                                  window, out, out_dtype, ld_out, lse, workspace, workspace_bytes,
                                  attention_workspace_bytes(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new,
                                                            max_seq));
  }
  if (rc || tokens == 0) return rc;
  AttentionArgs a{};
  a.q = q;
  a.q_start = q_start;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.cache = cache_view(const_cast<void*>(k_cache), const_cast<void*>(v_cache), cache_dtype, num_pages, page_size, num_kv_heads,
                       head_dim, page_stride, head_stride, token_stride, nullptr, nullptr, const_cast<uint8_t*>(k_blocks),
                       const_cast<uint8_t*>(v_blocks));
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.ld_q = ld_q;
  a.ld_table = ld_table;
  a.ld_out = ld_out;
  a.requests = num_requests;
  a.tokens = tokens;
  a.max_new = max_new;
  a.max_seq = max_seq;
  a.max_pages = max_pages;
  a.window = window > INT32_MAX ? 0 : (int)window;   // no sequence is that long
  a.scale = scale;
  a.hq = num_heads;
  a.group = num_heads / num_kv_heads;
  a.out_bf16 = (out_dtype & ~NVFP4_OUT_CLEAR_PADDING) == NVFP4_OUT_BF16;
  a.clear_padding = (out_dtype & NVFP4_OUT_CLEAR_PADDING) != 0;
  return hip_status(launch_paged_attention(a, (hipStream_t)stream));
}

int int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int8_t* codes, float* scales,
                  nvfp4_stream_t stream) {
  const int rc = validate_int8_quantize(x, rows, cols, ld_x, codes, scales);
  if (rc || rows == 0) return rc;
  return hip_status(launch_int8_quantize(x, rows, cols, ld_x, codes, scales, (hipStream_t)stream));
}

static Int8Args int8_args(const int8_t* a, const float* a_scale, int64_t m, const int8_t* w, const float* w_scale, int64_t n,
                          int64_t k, void* out, int out_dtype, int64_t ld_out, void* workspace) {
  Int8Args g{};
  g.a = a;
  g.a_scale = a_scale;
  g.w = w;
  g.w_scale = w_scale;
  g.out = out;
  g.workspace = workspace;
  g.m = m;
  g.n = n;
  g.k = k;
  g.ld_out = ld_out;
  g.out_bf16 = out_dtype == NVFP4_OUT_BF16;
  return g;
}

size_t gemm_w8a8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (validate_w8a8_sizes(m, n, k)) return 0;
  // the largest of any product of up to m tokens
  size_t bytes = int8_workspace_bytes(m < kInt8FewTokens ? m : kInt8FewTokens, n, k);
  const int64_t most = m < int8_split_tokens(n) ? m : int8_split_tokens(n);
  for (int64_t t = kInt8FewTokens + 1; t <= most; t = t / kInt8TokenStep * kInt8TokenStep + kInt8TokenStep + 1) {
    const size_t own = int8_workspace_bytes(t, n, k);
    if (own > bytes) bytes = own;
  }
  return bytes;
}

// What a call with a workspace reads and writes of it: at most gemm_w8a8_workspace_bytes.
static size_t needed_bytes(const void* workspace, int64_t m, int64_t n, int64_t k) {
  return !workspace || validate_w8a8_sizes(m, n, k) ? 0 : int8_workspace_bytes(m, n, k);
}

int gemm_w8a8(const int8_t* a, const float* a_scale, int64_t m, const int8_t* w, const float* w_scale, int64_t n, int64_t k,
              void* out, int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  const int rc = validate_gemm_w8a8(a, a_scale, m, w, w_scale, n, k, out, out_dtype, ld_out, workspace, workspace_bytes,
                                    needed_bytes(workspace, m, n, k));
  if (rc || m == 0) return rc;
  return hip_status(launch_gemm_w8a8(int8_args(a, a_scale, m, w, w_scale, n, k, out, out_dtype, ld_out, workspace),
                                     (hipStream_t)stream));
}

int int8_linear(const uint16_t* x, int64_t m, int64_t k, int64_t ld_x, int8_t* a, float* a_scale, const int8_t* w,
                const float* w_scale, int64_t n, void* out, int out_dtype, int64_t ld_out, void* workspace,
                size_t workspace_bytes, nvfp4_stream_t stream) {
  int rc = validate_int8_quantize(x, m, k, ld_x, a, a_scale);
  if (rc) return rc;
  rc = validate_gemm_w8a8(a, a_scale, m, w, w_scale, n, k, out, out_dtype, ld_out, workspace, workspace_bytes,
                          needed_bytes(workspace, m, n, k));
  if (rc || m == 0) return rc;
  return hip_status(launch_int8_linear(x, ld_x, a, a_scale,
                                       int8_args(a, a_scale, m, w, w_scale, n, k, out, out_dtype, ld_out, workspace),
                                       (hipStream_t)stream));
}

}  // extern "C"
