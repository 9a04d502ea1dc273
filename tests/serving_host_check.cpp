// Host-only check of the paged serving step's C ABI layer (abi_serving.cpp +
// validate_serving.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer
// and no GPU code: the launchers are stubs that keep their arguments.  Checks that
// a rejected call reaches no launcher and that an accepted one reaches the right
// one with the arguments the header documents.
#include <stdio.h>
#include <stdlib.h>

#include "../include/nvfp4.h"
#include "../nvfp4_w4a4_gemm_quantize_amd/csrc/kernels.h"
#include "../nvfp4_w4a4_gemm_quantize_amd/csrc/serving.h"

static int g_calls, g_cases;
static nvfp4::PlanArgs g_plan;
static nvfp4::KvWriteArgs g_write;
static nvfp4::AttentionArgs g_attention;
static nvfp4::VerifyArgs g_verify;
static hipError_t g_result = hipSuccess;

namespace nvfp4 {
int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }
hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t) {
  ++g_calls;
  g_plan = a;
  return g_result;
}
hipError_t launch_paged_kv_write(const KvWriteArgs& a, hipStream_t) {
  ++g_calls;
  g_write = a;
  return g_result;
}
size_t attention_workspace_bytes(int64_t, int64_t, int, int, int, int64_t, int64_t) { return 1000; }
hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t) {
  ++g_calls;
  g_attention = a;
  return g_result;
}
size_t verify_workspace_bytes(int64_t, int64_t, int64_t) { return 500; }
hipError_t launch_verify_drafts(const VerifyArgs& a, hipStream_t) {
  ++g_calls;
  g_verify = a;
  return g_result;
}
}  // namespace nvfp4

#define CHECK(c)                                                       \
  do {                                                                 \
    ++g_cases;                                                         \
    if (!(c)) {                                                        \
      fprintf(stderr, "FAILED at line %d: %s\n", __LINE__, #c);        \
      exit(1);                                                         \
    }                                                                  \
  } while (0)

template <class T>
static T* dev(uintptr_t at = 0x10000) { return reinterpret_cast<T*>(at); }

static int plan(int64_t requests, int page_size) {
  g_calls = 0;
  return paged_plan(dev<int32_t>(), dev<int32_t>(0x20000), requests, page_size, dev<int32_t>(), 5, nullptr, dev<int32_t>(), 7, 9,
                    dev<int32_t>(), dev<int32_t>(), dev<int32_t>(), dev<int64_t>(), 11, dev<int32_t>(), nullptr);
}
static int kv_write(int64_t tokens, int dtype, int page_size, const float* scale) {
  g_calls = 0;
  return paged_kv_write(dev<uint16_t>(), 264, dev<uint16_t>(), 272, dev<int64_t>(), tokens, dev<void>(), dev<void>(0x20000), dtype, 6,
                        page_size, 2, 128, 8192, 2048, 128, scale, nullptr, nullptr);
}
static int attention(int64_t tokens, int heads, size_t bytes, float scale) {
  g_calls = 0;
  return paged_attention(dev<uint16_t>(), 1024, tokens, dev<int32_t>(), dev<int32_t>(), 3, 4, 500, heads, dev<void>(), dev<void>(),
                         NVFP4_CACHE_E4M3, 6, 32, 2, 128, 8192, 4096, 128, dev<int32_t>(), 17, 20, scale, 33, dev<float>(),
                         dev<float>(), dev<void>(), NVFP4_OUT_BF16, 1028, nullptr, dev<void>(), bytes, nullptr);
}
static int verify(int64_t requests, int64_t drafts, size_t bytes) {
  g_calls = 0;
  return verify_drafts(dev<void>(), NVFP4_LOGITS_F32, 101, 12, 100, dev<int32_t>(), dev<int32_t>(), requests, drafts, dev<int32_t>(),
                       dev<float>(), 104, nullptr, dev<float>(), dev<float>(), 108, dev<int32_t>(), dev<int32_t>(), dev<float>(),
                       dev<void>(), bytes, nullptr);
}

int main() {
  CHECK(plan(3, 64) == NVFP4_OK && g_calls == 1);
  CHECK(g_plan.page_shift == 6 && g_plan.requests == 3 && g_plan.num_free == 5 && g_plan.max_pages == 7 && g_plan.ld_table == 9 &&
        g_plan.max_tokens == 11 && g_plan.new_lens == dev<int32_t>(0x20000) && g_plan.free_cursor == nullptr);
  CHECK(plan(0, 16) == NVFP4_OK && g_calls == 1);   // the counts are written all the same
  CHECK(plan(3, 48) == NVFP4_EUNSUPPORTED && g_calls == 0);
  CHECK(plan(-3, 16) == NVFP4_ESHAPE && g_calls == 0);

  CHECK(kv_write(9, NVFP4_CACHE_E4M3, 1024, dev<float>()) == NVFP4_OK && g_calls == 1);
  CHECK(g_write.tokens == 9 && g_write.ld_k == 264 && g_write.ld_v == 272 && g_write.cache.fp8 && g_write.cache.page_shift == 10 &&
        g_write.cache.num_pages == 6 && g_write.cache.page_stride == 8192 && g_write.cache.head_stride == 2048 &&
        g_write.cache.token_stride == 128 && g_write.cache.heads == 2 && g_write.cache.dim == 128 &&
        g_write.cache.v == dev<void>(0x20000) && g_write.cache.k_scale == dev<float>() && g_write.cache.v_scale == nullptr);
  CHECK(kv_write(9, NVFP4_CACHE_BF16, 16, nullptr) == NVFP4_OK && g_calls == 1 && !g_write.cache.fp8);
  CHECK(kv_write(9, NVFP4_CACHE_BF16, 16, dev<float>()) == NVFP4_EINVAL && g_calls == 0);
  CHECK(kv_write(0, NVFP4_CACHE_BF16, 16, nullptr) == NVFP4_OK && g_calls == 0);
  CHECK(kv_write(1, NVFP4_CACHE_BF16, 12, nullptr) == NVFP4_EUNSUPPORTED && g_calls == 0);

  CHECK(attention(10, 8, 1000, 0.5f) == NVFP4_OK && g_calls == 1);
  CHECK(g_attention.hq == 8 && g_attention.group == 4 && g_attention.out_bf16 == 1 && g_attention.window == 33 &&
        g_attention.scale == 0.5f && g_attention.tokens == 10 && g_attention.requests == 3 && g_attention.max_new == 4 &&
        g_attention.max_seq == 500 && g_attention.max_pages == 17 && g_attention.ld_table == 20 && g_attention.ld_q == 1024 &&
        g_attention.ld_out == 1028 && g_attention.cache.fp8 && g_attention.lse == nullptr);
  CHECK(attention(10, 8, 999, 0.5f) == NVFP4_ESIZE && g_calls == 0);
  CHECK(attention(10, 7, 1000, 0.5f) == NVFP4_ESHAPE && g_calls == 0);
  CHECK(attention(0, 8, 1000, 0.5f) == NVFP4_OK && g_calls == 0);
  CHECK(attention(10, 8, 1000, 0.f / 0.f * 1.f) == NVFP4_EINVAL && g_calls == 0);

  CHECK(verify(4, 2, 500) == NVFP4_OK && g_calls == 1);
  CHECK(g_verify.logits_f32 == 1 && g_verify.rows == 12 && g_verify.vocab == 100 && g_verify.ld_logits == 101 && g_verify.ld_probs == 104 &&
        g_verify.ld_noise == 108 && g_verify.requests == 4 && g_verify.max_drafts == 2 && g_verify.temperature == nullptr);
  CHECK(verify(4, 2, 499) == NVFP4_ESIZE && g_calls == 0);
  CHECK(verify(0, 2, 0) == NVFP4_OK && g_calls == 0);
  CHECK(verify(4, 256, 500) == NVFP4_EUNSUPPORTED && g_calls == 0);

  g_result = hipErrorInvalidValue;   // a launch that fails is reported
  CHECK(plan(3, 64) == NVFP4_EHIP && kv_write(9, NVFP4_CACHE_BF16, 16, nullptr) == NVFP4_EHIP &&
        attention(10, 8, 1000, 0.5f) == NVFP4_EHIP && verify(4, 2, 500) == NVFP4_EHIP);
  printf("serving host check: %d cases ok\n", g_cases);
  return 0;
}
