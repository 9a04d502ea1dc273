// Internal launcher interface of the paged serving step (plan, K/V write,
// attention, draft verification) between the C ABI layer and the HIP kernels.
// Launchers enqueue on the given stream and return the launch status; all
// argument validation happens before they are called.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

struct PlanArgs {
  const int32_t* ctx_lens;     // [requests]
  const int32_t* new_lens;     // [requests]
  const int32_t* free_pages;   // [num_free]
  const int32_t* free_cursor;  // [1] or null (0)
  int32_t* block_table;        // [requests, max_pages], row stride ld_table
  int32_t* q_start;            // [requests + 1]
  int32_t* seq_lens;           // [requests]
  int32_t* positions;          // [max_tokens]
  int64_t* slots;              // [max_tokens]
  int32_t* counts;             // [4]
  int64_t requests, num_free, max_pages, ld_table, max_tokens;
  int page_shift;
  bool in_place;               // seq_lens is ctx_lens, or counts hold free_cursor
};
hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t st);

// A paged K/V cache: element (page, head, token in page, d) of either cache
// lies at page * page_stride + head * head_stride + token * token_stride + d
// elements.
struct CacheView {
  void* k;
  void* v;
  int64_t num_pages, page_stride, head_stride, token_stride;
  const float* k_scale;        // [kv heads] or null (1)
  const float* v_scale;
  int fp8;                     // E4M3 elements, else bf16
  int page_shift;              // log2(page size)
  int heads, dim;
  // Caches with a scale for each 16 tokens and head (kBlocks*): E8M0 bytes
  // [pages, heads, page size / 16], contiguous; fp8 is 0 and k_scale, v_scale null.
  int blocks;
  uint8_t* k_blocks;
  uint8_t* v_blocks;
};
enum { kBlocksNone, kBlocksE4m3, kBlocksInt8 };
constexpr int kBlockTokens = 16;
// The largest scale bytes: with them the largest code is below 2^128, and INT8 scales
// times weights up to 2^8 are.
constexpr int kMostE4m3 = 246, kMostInt8 = 240;

struct KvWriteArgs {
  const uint16_t* k;
  const uint16_t* v;
  const int64_t* slots;
  int64_t ld_k, ld_v, tokens;
  CacheView cache;
};
hipError_t launch_paged_kv_write(const KvWriteArgs& a, hipStream_t st);

struct AttentionArgs {
  const uint16_t* q;           // [tokens, hq * dim], row stride ld_q
  const int32_t* q_start;      // [requests + 1]
  const int32_t* seq_lens;     // [requests]
  const int32_t* block_table;  // [requests, max_pages], row stride ld_table
  CacheView cache;
  void* out;                   // [tokens, hq * dim], row stride ld_out
  float* lse;                  // [tokens, hq] or null
  void* workspace;
  int64_t ld_q, ld_table, ld_out, requests, tokens, max_new, max_seq, max_pages;
  int window;                  // 0: none
  float scale;
  int hq, group, out_bf16;
  bool clear_padding;          // rows of no request get 0 and lse = -inf
  // n / group = mulhi(n, group_mul) >> group_shift for n < 2^31, group > 1; set by the launcher
  uint32_t group_mul;
  int group_shift;
  int stream_rows;             // requests with at most so many rows a KV head are the streaming kernel's; likewise
};
size_t attention_workspace_bytes(int64_t tokens, int64_t requests, int hq, int hkv, int dim, int64_t max_new,
                                 int64_t max_seq);
hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t st);

struct VerifyArgs {
  const void* logits;          // [rows, vocab], row stride ld_logits
  const int32_t* row_start;    // [requests]
  const int32_t* num_drafts;   // [requests]
  const int32_t* draft_tokens; // [requests, max_drafts]
  const float* draft_probs;    // [requests, max_drafts, vocab] (row stride ld_probs) or null
  const float* temperature;    // [requests] or null (1)
  const float* uniform;        // [requests, max_drafts]
  const float* noise;          // [requests, vocab], row stride ld_noise
  int32_t* out_tokens;         // [requests, max_drafts + 1]
  int32_t* num_accepted;       // [requests]
  float* logprobs;             // [requests, max_drafts + 1]
  void* workspace;
  int64_t ld_logits, rows, requests, max_drafts, vocab, ld_probs, ld_noise;
  int logits_f32;
};
size_t verify_workspace_bytes(int64_t requests, int64_t max_drafts, int64_t vocab);
hipError_t launch_verify_drafts(const VerifyArgs& a, hipStream_t st);

}  // namespace nvfp4
