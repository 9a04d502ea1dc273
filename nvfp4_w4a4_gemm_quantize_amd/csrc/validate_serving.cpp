// Host-side argument validation of the paged serving step (no HIP dependency).
#include "validate_serving.h"

#include <math.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

static bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int page_shift_of(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

static int validate_head_dim(int head_dim) {
  if (head_dim <= 0) return NVFP4_ESHAPE;
  return head_dim == 64 || head_dim == 128 || head_dim == 256 ? NVFP4_OK : NVFP4_EUNSUPPORTED;
}

int validate_paged_plan(const void* ctx_lens, const void* new_lens, int64_t num_requests, int page_size,
                        const void* free_pages, int64_t num_free, const void* free_cursor, const void* block_table,
                        int64_t max_pages, int64_t ld_table, const void* q_start, const void* seq_lens,
                        const void* positions, const void* slots, int64_t max_tokens, const void* counts) {
  if (num_requests < 0 || num_free < 0 || max_pages < 0 || max_tokens < 0 || ld_table < max_pages || page_size <= 0)
    return NVFP4_ESHAPE;
  if (page_shift_of(page_size) < 0 || num_requests > INT32_MAX || num_free > INT32_MAX || max_pages > INT32_MAX ||
      max_tokens > INT32_MAX)
    return NVFP4_EUNSUPPORTED;
  if (!q_start || !counts || (num_requests > 0 && (!ctx_lens || !new_lens || !seq_lens)) ||
      (num_requests > 0 && max_pages > 0 && !block_table) || (num_free > 0 && !free_pages) ||
      (max_tokens > 0 && (!positions || !slots)))
    return NVFP4_EINVAL;
  if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(free_cursor, 4) ||
      !aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) ||
      !aligned(slots, 8) || !aligned(counts, 4))
    return NVFP4_EALIGN;
  return NVFP4_OK;
}

int validate_cache(const void* k_cache, const void* v_cache, int cache_dtype, int64_t num_pages, int page_size,
                   int num_kv_heads, int head_dim, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                   const void* k_scale, const void* v_scale) {
  if (cache_dtype != NVFP4_CACHE_BF16 && cache_dtype != NVFP4_CACHE_E4M3) return NVFP4_EINVAL;
  if (num_kv_heads <= 0 || num_pages <= 0 || page_size <= 0) return NVFP4_ESHAPE;
  int rc = validate_head_dim(head_dim);
  if (rc) return rc;
  if (page_shift_of(page_size) < 0 || num_kv_heads > 65536 || num_pages > INT32_MAX) return NVFP4_EUNSUPPORTED;
  if (page_stride < 0 || head_stride < 0 || token_stride < head_dim) return NVFP4_ESHAPE;
  if (!k_cache || !v_cache || (cache_dtype == NVFP4_CACHE_BF16 && (k_scale || v_scale))) return NVFP4_EINVAL;
  const int64_t bytes = cache_dtype == NVFP4_CACHE_BF16 ? 2 : 1;
  // 32-bit offsets inside a page, page strides in 32 bits of 16-byte units
  if (token_stride > INT32_MAX / (page_size * bytes) || page_stride / (16 / bytes) > UINT32_MAX) return NVFP4_EUNSUPPORTED;
  const int64_t unit = 16 / bytes;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || page_stride % unit || head_stride % unit ||
      token_stride % unit || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return NVFP4_EALIGN;
  return NVFP4_OK;
}

int validate_paged_kv_write(const void* k, int64_t ld_k, const void* v, int64_t ld_v, const void* slots,
                            int64_t tokens, int num_kv_heads, int head_dim) {
  if (tokens < 0 || num_kv_heads <= 0) return NVFP4_ESHAPE;
  int rc = validate_head_dim(head_dim);
  if (rc) return rc;
  const int64_t cols = (int64_t)num_kv_heads * head_dim;
  if (ld_k < cols || ld_v < cols) return NVFP4_ESHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (tokens > INT32_MAX) return NVFP4_EUNSUPPORTED;
  if (!k || !v || !slots) return NVFP4_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || ld_k % 8 || ld_v % 8 || !aligned(slots, 8)) return NVFP4_EALIGN;
  return NVFP4_OK;
}

int validate_attention_sizes(int64_t tokens, int64_t num_requests, int num_heads, int num_kv_heads, int head_dim,
                             int64_t max_new, int64_t max_seq) {
  if (tokens < 0 || num_requests < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      max_new < 0 || max_seq < 0)
    return NVFP4_ESHAPE;
  int rc = validate_head_dim(head_dim);
  if (rc) return rc;
  // rows and workgroups are counted in 32 bits
  if (num_heads > 65536 || tokens > INT32_MAX / num_heads || num_requests > INT32_MAX / 64 / num_kv_heads ||
      max_new > INT32_MAX || max_seq > INT32_MAX)
    return NVFP4_EUNSUPPORTED;
  return NVFP4_OK;
}

int validate_paged_attention(const void* q, int64_t ld_q, int64_t tokens, const void* q_start, const void* seq_lens,
                             int num_heads, int head_dim, const void* block_table, int64_t max_pages,
                             int64_t ld_table, float scale, int64_t window, const void* out, int out_dtype,
                             int64_t ld_out, const void* lse, const void* workspace, size_t workspace_bytes,
                             size_t needed) {
  const int64_t cols = (int64_t)num_heads * head_dim;
  const int out_kind = out_dtype & ~NVFP4_OUT_CLEAR_PADDING;
  if (out_kind != NVFP4_OUT_F32 && out_kind != NVFP4_OUT_BF16) return NVFP4_EINVAL;
  if (!isfinite(scale) || window < 0) return NVFP4_EINVAL;
  if (ld_q < cols || ld_out < cols || max_pages <= 0 || ld_table < max_pages) return NVFP4_ESHAPE;
  if (max_pages > INT32_MAX) return NVFP4_EUNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  if (!q || !q_start || !seq_lens || !block_table || !out || !workspace) return NVFP4_EINVAL;
  if (!aligned(q, 16) || ld_q % 8 || !aligned(out, 16) || ld_out % 4 || !aligned(q_start, 4) ||
      !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
    return NVFP4_EALIGN;
  return workspace_bytes < needed ? NVFP4_ESIZE : NVFP4_OK;
}

int validate_verify_sizes(int64_t num_requests, int64_t max_drafts, int64_t vocab) {
  if (num_requests < 0 || max_drafts < 0 || vocab <= 0) return NVFP4_ESHAPE;
  return num_requests > 65535 || max_drafts > 255 || vocab > INT32_MAX - 4096 ? NVFP4_EUNSUPPORTED : NVFP4_OK;
}

int validate_verify_drafts(const void* logits, int logits_dtype, int64_t ld_logits, int64_t rows, int64_t vocab,
                           const void* row_start, const void* num_drafts, int64_t max_drafts,
                           const void* draft_tokens, const void* draft_probs, int64_t ld_probs,
                           const void* temperature, const void* uniform, const void* noise, int64_t ld_noise,
                           const void* out_tokens, const void* num_accepted, const void* logprobs,
                           const void* workspace, size_t workspace_bytes, size_t needed) {
  if (logits_dtype != NVFP4_LOGITS_F32 && logits_dtype != NVFP4_LOGITS_BF16) return NVFP4_EINVAL;
  if (rows < 0 || ld_logits < vocab || ld_noise < vocab || (draft_probs && ld_probs < vocab)) return NVFP4_ESHAPE;
  if (!logits || !row_start || !num_drafts || !noise || !out_tokens || !num_accepted || !logprobs || !workspace ||
      (max_drafts > 0 && (!draft_tokens || !uniform)))
    return NVFP4_EINVAL;
  if (!aligned(logits, 16) || !aligned(noise, 16) || !aligned(draft_probs, 16) || !aligned(workspace, 16) ||
      !aligned(row_start, 4) || !aligned(num_drafts, 4) || !aligned(draft_tokens, 4) || !aligned(temperature, 4) ||
      !aligned(uniform, 4) || !aligned(out_tokens, 4) || !aligned(num_accepted, 4) || !aligned(logprobs, 4))
    return NVFP4_EALIGN;
  return workspace_bytes < needed ? NVFP4_ESIZE : NVFP4_OK;
}

}  // namespace nvfp4
