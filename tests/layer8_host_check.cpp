// Host-only check of the C ABI layer of the attention layer in 8 bits (abi_layer8.cpp,
// validate_layer8.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer and no
// GPU code: the launchers are stubs that keep their arguments.  Checks that a rejected
// call reaches no launcher and that an accepted one reaches the right one with the
// arguments the header documents.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../include/nvfp4.h"
#include "../nvfp4_w4a4_gemm_quantize_amd/csrc/kernels.h"
#include "../nvfp4_w4a4_gemm_quantize_amd/csrc/layer8.h"

static int g_calls, g_cases;
static nvfp4::RotaryRows g_rows;
static nvfp4::RotaryArgs g_rot;
static nvfp4::AppendArgs g_append;
static nvfp4::AttentionArgs g_attention;
static nvfp4::Int8Args g_int8;
static int64_t g_quantize[3];
static hipError_t g_result = hipSuccess;

namespace nvfp4 {
int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }
hipError_t launch_rotary(const RotaryRows& a, const RotaryArgs& rot, hipStream_t) {
  ++g_calls;
  g_rows = a;
  g_rot = rot;
  return g_result;
}
hipError_t launch_paged_kv_append(const AppendArgs& a, hipStream_t) {
  ++g_calls;
  g_append = a;
  return g_result;
}
size_t attention_workspace_bytes(int64_t, int64_t, int, int, int, int64_t, int64_t) { return 1000; }
hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t) {
  ++g_calls;
  g_attention = a;
  return g_result;
}
hipError_t launch_int8_quantize(const uint16_t*, int64_t rows, int64_t cols, int64_t ld, int8_t*, float*, hipStream_t) {
  ++g_calls;
  g_quantize[0] = rows;
  g_quantize[1] = cols;
  g_quantize[2] = ld;
  return g_result;
}
size_t int8_workspace_bytes(int64_t, int64_t, int64_t) { return 700; }
hipError_t launch_gemm_w8a8(const Int8Args& a, hipStream_t) {
  ++g_calls;
  g_int8 = a;
  return g_result;
}
hipError_t launch_int8_linear(const uint16_t*, int64_t ld_x, int8_t* codes, float* scales, const Int8Args& a, hipStream_t) {
  ++g_calls;
  g_int8 = a;
  g_quantize[2] = ld_x;
  if (codes != a.a || scales != a.a_scale) exit(1);
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

static int rot(int64_t tokens, int dim, int rotary_dim, double amplitude) {
  g_calls = 0;
  return rotary(dev<uint16_t>(), 1032, tokens, 4, dim, dev<int32_t>(), dev<uint64_t>(0x20000), rotary_dim, NVFP4_ROTARY_INTERLEAVED,
                amplitude, dev<uint16_t>(0x30000), 1040, nullptr);
}
static int append(int64_t tokens, int dtype, int heads, int rotary_dim) {
  const bool blocks = dtype >= NVFP4_CACHE_E4M3_BLOCKS;
  g_calls = 0;
  return paged_kv_append(heads ? dev<uint16_t>() : nullptr, 1024, heads, heads ? dev<uint16_t>(0x50000) : nullptr, 1032, dev<uint16_t>(), 264,
                         dev<uint16_t>(0x20000), 272, dev<int32_t>(), dev<int64_t>(), tokens, rotary_dim ? dev<uint64_t>() : nullptr,
                         rotary_dim, NVFP4_ROTARY_HALF, 1.5f, dev<void>(), dev<void>(0x20000), dtype, 6, 32, 2, 128, 8192, 4096, 128,
                         dtype == NVFP4_CACHE_E4M3 ? dev<float>() : nullptr, nullptr, blocks ? dev<uint8_t>(0x30000) : nullptr,
                         blocks ? dev<uint8_t>(0x40000) : nullptr, nullptr);
}
static int attention(int64_t tokens, int dtype, int heads, size_t bytes) {
  g_calls = 0;
  return paged_attention_blocks(dev<uint16_t>(), 1024, tokens, dev<int32_t>(), dev<int32_t>(), 3, 4, 500, heads, dev<void>(), dev<void>(),
                                dtype, 6, 32, 2, 128, 8192, 4096, 128, dev<uint8_t>(0x30000), dev<uint8_t>(0x40000), dev<int32_t>(), 17, 20,
                                0.5f, 33, dev<void>(), NVFP4_OUT_BF16 | NVFP4_OUT_CLEAR_PADDING, 1028, nullptr, dev<void>(), bytes, nullptr);
}
static int linear(int64_t m, int64_t k, int dtype, size_t bytes = 700) {
  g_calls = 0;
  return int8_linear(dev<uint16_t>(), m, k, 2056, dev<int8_t>(), dev<float>(), dev<int8_t>(0x20000), dev<float>(0x30004), 99, dev<void>(), dtype,
                     101, dev<void>(0x70000), bytes, nullptr);
}

int main() {
  // every scaling at every size writes its table and no more
  for (int dim = 16; dim <= 1024; dim += 16)
    for (int scaling = NVFP4_ROPE_NONE; scaling <= NVFP4_ROPE_WAVELENGTH; ++scaling) {
      std::vector<uint64_t> steps(dim / 2);
      std::vector<double> factors(dim / 2, 1.5);
      double amplitude = 0;
      CHECK(rotary_steps(dim, 1e4, scaling, 8.0, 4096.0, 1.0, 32.0, factors.data(), steps.data(), &amplitude) == NVFP4_OK);
      CHECK(amplitude >= 1 && steps[0] != 0);
    }

  CHECK(rot(9, 256, 64, 2.f) == NVFP4_OK && g_calls == 1);
  CHECK(g_rows.tokens == 9 && g_rows.heads == 4 && g_rows.dim == 256 && g_rows.ld_x == 1032 && g_rows.ld_out == 1040 &&
        g_rows.out == dev<uint16_t>(0x30000) && g_rot.dim == 64 && g_rot.interleaved == 1 && g_rot.amplitude == 2.f &&
        g_rot.steps == dev<uint64_t>(0x20000));
  CHECK(rot(0, 256, 64, 2.f) == NVFP4_OK && g_calls == 0);
  CHECK(rot(9, 256, 272, 2.f) == NVFP4_ESHAPE && g_calls == 0);
  CHECK(rot(9, 200, 64, 2.f) == NVFP4_EUNSUPPORTED && g_calls == 0);

  CHECK(append(7, NVFP4_CACHE_INT8_BLOCKS, 8, 64) == NVFP4_OK && g_calls == 1);
  CHECK(g_append.cache.blocks == nvfp4::kBlocksInt8 && g_append.cache.fp8 == 0 && g_append.cache.k_blocks == dev<uint8_t>(0x30000) &&
        g_append.cache.v_blocks == dev<uint8_t>(0x40000) && g_append.cache.page_shift == 5 && g_append.cache.k_scale == nullptr &&
        g_append.q.heads == 8 && g_append.q.dim == 128 && g_append.q.ld_out == 1032 && g_append.q.tokens == 7 && g_append.ld_k == 264 &&
        g_append.ld_v == 272 && g_append.tokens == 7 && g_append.rot.dim == 64 && g_append.rot.interleaved == 0 &&
        g_append.rot.amplitude == 1.5f);
  CHECK(append(7, NVFP4_CACHE_E4M3_BLOCKS, 0, 0) == NVFP4_OK && g_calls == 1 && g_append.cache.blocks == nvfp4::kBlocksE4m3 &&
        g_append.q.heads == 0 && g_append.rot.dim == 0);
  CHECK(append(7, NVFP4_CACHE_E4M3, 8, 128) == NVFP4_OK && g_calls == 1 && g_append.cache.fp8 == 1 &&
        g_append.cache.blocks == nvfp4::kBlocksNone && g_append.cache.k_scale == dev<float>());
  CHECK(append(7, NVFP4_CACHE_BF16, 8, 16) == NVFP4_OK && g_calls == 1 && g_append.cache.fp8 == 0);
  CHECK(append(0, NVFP4_CACHE_INT8_BLOCKS, 8, 64) == NVFP4_OK && g_calls == 0);
  CHECK(append(7, 4, 8, 64) == NVFP4_EINVAL && g_calls == 0);
  CHECK(append(7, NVFP4_CACHE_BF16, 8, 144) == NVFP4_ESHAPE && g_calls == 0);

  CHECK(attention(10, NVFP4_CACHE_E4M3_BLOCKS, 8, 1000) == NVFP4_OK && g_calls == 1);
  CHECK(g_attention.cache.blocks == nvfp4::kBlocksE4m3 && g_attention.cache.k_blocks == dev<uint8_t>(0x30000) && g_attention.group == 4 &&
        g_attention.window == 33 && g_attention.max_pages == 17 && g_attention.ld_table == 20 && g_attention.out_bf16 == 1 &&
        g_attention.clear_padding && g_attention.ld_out == 1028 && g_attention.requests == 3 && g_attention.max_new == 4);
  CHECK(attention(10, NVFP4_CACHE_E4M3, 8, 1000) == NVFP4_EINVAL && g_calls == 0);
  CHECK(attention(10, NVFP4_CACHE_INT8_BLOCKS, 7, 1000) == NVFP4_ESHAPE && g_calls == 0);
  CHECK(attention(10, NVFP4_CACHE_INT8_BLOCKS, 8, 999) == NVFP4_ESIZE && g_calls == 0);
  CHECK(attention(0, NVFP4_CACHE_INT8_BLOCKS, 8, 1000) == NVFP4_OK && g_calls == 0);

  CHECK(linear(5, 2048, NVFP4_OUT_F32) == NVFP4_OK && g_calls == 1 && g_quantize[2] == 2056 && g_int8.m == 5 && g_int8.k == 2048 &&
        g_int8.n == 99 && g_int8.ld_out == 101 && g_int8.out_bf16 == 0 && g_int8.workspace == dev<void>(0x70000));
  CHECK(linear(5, 2048, NVFP4_OUT_F32, 699) == NVFP4_ESIZE && g_calls == 0);
  CHECK(linear(0, 2048, NVFP4_OUT_F32) == NVFP4_OK && g_calls == 0);
  CHECK(linear(5, 2056, NVFP4_OUT_F32) == NVFP4_EUNSUPPORTED && g_calls == 0);
  CHECK(linear(5, 4096, NVFP4_OUT_F32) == NVFP4_ESHAPE && g_calls == 0);
  CHECK(linear(5, 2048, 7) == NVFP4_EINVAL && g_calls == 0);
  g_calls = 0;
  CHECK(int8_quantize(dev<uint16_t>(), 6, 64, 72, dev<int8_t>(), dev<float>(), nullptr) == NVFP4_OK && g_calls == 1 && g_quantize[0] == 6 &&
        g_quantize[1] == 64 && g_quantize[2] == 72);
  g_calls = 0;
  CHECK(gemm_w8a8(dev<int8_t>(), dev<float>(0x40000), 6, dev<int8_t>(0x20000), dev<float>(0x30000), 10, 96, dev<void>(), NVFP4_OUT_BF16, 12,
                  nullptr, 0, nullptr) == NVFP4_OK && g_calls == 1 && g_int8.m == 6 && g_int8.n == 10 && g_int8.k == 96 && g_int8.ld_out == 12 &&
        g_int8.out_bf16 == 1 && g_int8.workspace == nullptr && g_int8.w == dev<int8_t>(0x20000) && g_int8.a_scale == dev<float>(0x40000));

  g_result = hipErrorInvalidValue;   // a launch that fails is reported
  CHECK(rot(9, 256, 64, 2.f) == NVFP4_EHIP && append(7, NVFP4_CACHE_BF16, 8, 16) == NVFP4_EHIP &&
        attention(10, NVFP4_CACHE_E4M3_BLOCKS, 8, 1000) == NVFP4_EHIP && linear(5, 2048, NVFP4_OUT_F32) == NVFP4_EHIP);
  printf("layer8 host check: %d cases ok\n", g_cases);
  return 0;
}
