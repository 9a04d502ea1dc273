// C ABI entry points of the paged serving step: validate, describe, launch.
// Declared and documented in include/nvfp4.h.
#include <hip/hip_runtime.h>

#include "../../include/nvfp4.h"
#include "kernels.h"
#include "serving.h"
#include "validate_serving.h"

using namespace nvfp4;

static CacheView cache_view(void* k, void* v, int dtype, int64_t num_pages, int page_size, int heads, int dim,
                            int64_t page_stride, int64_t head_stride, int64_t token_stride, const float* k_scale,
                            const float* v_scale) {
  CacheView c{};
  c.k = k;
  c.v = v;
  c.num_pages = num_pages;
  c.page_stride = page_stride;
  c.head_stride = head_stride;
  c.token_stride = token_stride;
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  c.fp8 = dtype == NVFP4_CACHE_E4M3;
  c.page_shift = page_shift_of(page_size);
  c.heads = heads;
  c.dim = dim;
  return c;
}

extern "C" {

int paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int64_t num_requests, int page_size,
               const int32_t* free_pages, int64_t num_free, const int32_t* free_cursor, int32_t* block_table,
               int64_t max_pages, int64_t ld_table, int32_t* q_start, int32_t* seq_lens, int32_t* positions,
               int64_t* slots, int64_t max_tokens, int32_t* counts, nvfp4_stream_t stream) {
  int rc = validate_paged_plan(ctx_lens, new_lens, num_requests, page_size, free_pages, num_free, free_cursor,
                               block_table, max_pages, ld_table, q_start, seq_lens, positions, slots, max_tokens,
                               counts);
  if (rc) return rc;
  PlanArgs a{};
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_cursor = free_cursor;
  a.block_table = block_table;
  a.q_start = q_start;
  a.seq_lens = seq_lens;
  a.positions = positions;
  a.slots = slots;
  a.counts = counts;
  a.requests = num_requests;
  a.num_free = num_free;
  a.max_pages = max_pages;
  a.ld_table = ld_table;
  a.max_tokens = max_tokens;
  a.page_shift = page_shift_of(page_size);
  a.in_place = (num_requests > 0 && ctx_lens == seq_lens) || (free_cursor >= counts && free_cursor < counts + 4);
  return hip_status(launch_paged_plan(a, (hipStream_t)stream));
}

int paged_kv_write(const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, const int64_t* slots,
                   int64_t tokens, void* k_cache, void* v_cache, int cache_dtype, int64_t num_pages, int page_size,
                   int num_kv_heads, int head_dim, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                   const float* k_scale, const float* v_scale, nvfp4_stream_t stream) {
  int rc = validate_cache(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride,
                          head_stride, token_stride, k_scale, v_scale);
  if (rc) return rc;
  rc = validate_paged_kv_write(k, ld_k, v, ld_v, slots, tokens, num_kv_heads, head_dim);
  if (rc || tokens == 0) return rc;
  KvWriteArgs a{};
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.tokens = tokens;
  a.cache = cache_view(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride,
                       head_stride, token_stride, k_scale, v_scale);
  return hip_status(launch_paged_kv_write(a, (hipStream_t)stream));
}

size_t paged_attention_workspace_bytes(int64_t tokens, int64_t num_requests, int num_heads, int num_kv_heads,
                                       int head_dim, int64_t max_new, int64_t max_seq) {
  if (validate_attention_sizes(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new, max_seq)) return 0;
  return attention_workspace_bytes(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new, max_seq);
}

int paged_attention(const uint16_t* q, int64_t ld_q, int64_t tokens, const int32_t* q_start, const int32_t* seq_lens,
                    int64_t num_requests, int64_t max_new, int64_t max_seq, int num_heads, const void* k_cache,
                    const void* v_cache, int cache_dtype, int64_t num_pages, int page_size, int num_kv_heads,
                    int head_dim, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                    const int32_t* block_table, int64_t max_pages, int64_t ld_table, float scale, int64_t window,
                    const float* k_scale, const float* v_scale, void* out, int out_dtype, int64_t ld_out, float* lse,
                    void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  int rc = validate_attention_sizes(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new, max_seq);
  if (rc) return rc;
  rc = validate_cache(k_cache, v_cache, cache_dtype, num_pages, page_size, num_kv_heads, head_dim, page_stride,
                      head_stride, token_stride, k_scale, v_scale);
  if (rc) return rc;
  if (num_requests == 0) {
    if (!(out_dtype & NVFP4_OUT_CLEAR_PADDING)) return NVFP4_OK;
    rc = validate_attention_padding(tokens, num_heads, head_dim, out, out_dtype, ld_out, lse);
  } else {
    rc = validate_paged_attention(q, ld_q, tokens, q_start, seq_lens, num_heads, head_dim, block_table, max_pages,
                                  ld_table, scale, window, out, out_dtype, ld_out, lse, workspace, workspace_bytes,
                                  attention_workspace_bytes(tokens, num_requests, num_heads, num_kv_heads, head_dim,
                                                            max_new, max_seq));
  }
  if (rc || tokens == 0) return rc;
  AttentionArgs a{};
  a.q = q;
  a.q_start = q_start;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.cache = cache_view(const_cast<void*>(k_cache), const_cast<void*>(v_cache), cache_dtype, num_pages, page_size,
                       num_kv_heads, head_dim, page_stride, head_stride, token_stride, k_scale, v_scale);
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

size_t verify_drafts_workspace_bytes(int64_t num_requests, int64_t max_drafts, int64_t vocab) {
  return validate_verify_sizes(num_requests, max_drafts, vocab) ? 0 : verify_workspace_bytes(num_requests, max_drafts, vocab);
}

int verify_drafts(const void* logits, int logits_dtype, int64_t ld_logits, int64_t rows, int64_t vocab,
                  const int32_t* row_start, const int32_t* num_drafts, int64_t num_requests, int64_t max_drafts,
                  const int32_t* draft_tokens, const float* draft_probs, int64_t ld_probs, const float* temperature,
                  const float* uniform, const float* noise, int64_t ld_noise, int32_t* out_tokens,
                  int32_t* num_accepted, float* logprobs, void* workspace, size_t workspace_bytes,
                  nvfp4_stream_t stream) {
  int rc = validate_verify_sizes(num_requests, max_drafts, vocab);
  if (rc || num_requests == 0) return rc;
  rc = validate_verify_drafts(logits, logits_dtype, ld_logits, rows, vocab, row_start, num_drafts, max_drafts,
                              draft_tokens, draft_probs, ld_probs, temperature, uniform, noise, ld_noise, out_tokens,
                              num_accepted, logprobs, workspace, workspace_bytes,
                              verify_workspace_bytes(num_requests, max_drafts, vocab));
  if (rc) return rc;
  VerifyArgs a{};
  a.logits = logits;
  a.row_start = row_start;
  a.num_drafts = num_drafts;
  a.draft_tokens = draft_tokens;
  a.draft_probs = draft_probs;
  a.temperature = temperature;
  a.uniform = uniform;
  a.noise = noise;
  a.out_tokens = out_tokens;
  a.num_accepted = num_accepted;
  a.logprobs = logprobs;
  a.workspace = workspace;
  a.ld_logits = ld_logits;
  a.rows = rows;
  a.requests = num_requests;
  a.max_drafts = max_drafts;
  a.vocab = vocab;
  a.ld_probs = ld_probs;
  a.ld_noise = ld_noise;
  a.logits_f32 = logits_dtype == NVFP4_LOGITS_F32;
  return hip_status(launch_verify_drafts(a, (hipStream_t)stream));
}

}  // extern "C"
