// Host-side argument validation of the paged serving step's entry points.  Pure
// C++ (no HIP headers), so it can be compiled and exercised without a GPU.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// log2 of a page size, -1 if it is none.
int page_shift_of(int page_size);

int validate_paged_plan(const void* ctx_lens, const void* new_lens, int64_t num_requests, int page_size,
                        const void* free_pages, int64_t num_free, const void* free_cursor, const void* block_table,
                        int64_t max_pages, int64_t ld_table, const void* q_start, const void* seq_lens,
                        const void* positions, const void* slots, int64_t max_tokens, const void* counts);
int validate_cache(const void* k_cache, const void* v_cache, int cache_dtype, int64_t num_pages, int page_size,
                   int num_kv_heads, int head_dim, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                   const void* k_scale, const void* v_scale);
int validate_paged_kv_write(const void* k, int64_t ld_k, const void* v, int64_t ld_v, const void* slots,
                            int64_t tokens, int num_kv_heads, int head_dim);
int validate_attention_sizes(int64_t tokens, int64_t num_requests, int num_heads, int num_kv_heads, int head_dim,
                             int64_t max_new, int64_t max_seq);
int validate_paged_attention(const void* q, int64_t ld_q, int64_t tokens, const void* q_start, const void* seq_lens,
                             int num_heads, int head_dim, const void* block_table, int64_t max_pages,
                             int64_t ld_table, float scale, int64_t window, const void* out, int out_dtype,
                             int64_t ld_out, const void* lse, const void* workspace, size_t workspace_bytes,
                             size_t needed);
// A batch without requests, whose rows are to be cleared.
int validate_attention_padding(int64_t tokens, int num_heads, int head_dim, const void* out, int out_dtype,
                               int64_t ld_out, const void* lse);
int validate_verify_sizes(int64_t num_requests, int64_t max_drafts, int64_t vocab);
int validate_verify_drafts(const void* logits, int logits_dtype, int64_t ld_logits, int64_t rows, int64_t vocab,
                           const void* row_start, const void* num_drafts, int64_t max_drafts,
                           const void* draft_tokens, const void* draft_probs, int64_t ld_probs,
                           const void* temperature, const void* uniform, const void* noise, int64_t ld_noise,
                           const void* out_tokens, const void* num_accepted, const void* logprobs,
                           const void* workspace, size_t workspace_bytes, size_t needed);

}  // namespace nvfp4
