// Internal launcher interface of the attention layer in 8 bits (rotary positions,
// rotated append to the paged cache, int8 linear layers) between the C ABI layer
// and the HIP kernels; its attention is serving.h's with a block-scaled CacheView.
// Launchers enqueue on the given stream and return the launch status; all
// argument validation happens before they are called.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "serving.h"

namespace nvfp4 {

// A launch counts its threads in 32 bits: of more, some are not started, without an error.
inline bool one_launch(int64_t blocks, int threads) { return blocks * threads <= (int64_t)UINT32_MAX; }

// A rotation: pair i of a head turns by steps[i] * position 2^-64ths of a turn.
struct RotaryArgs {
  const uint64_t* steps;       // [dim / 2]
  const int32_t* positions;    // [tokens]; negative: not turned
  int dim;                     // leading columns of a head that are rotated; 0: none
  int interleaved;             // pairs (2 i, 2 i + 1), else (i, i + dim / 2)
  double amplitude;            // on cosine and sine
};

// Rows of `heads` heads of `dim` columns, rotated from x to out.
struct RotaryRows {
  const uint16_t* x;
  uint16_t* out;
  int64_t ld_x, ld_out, tokens;
  int heads, dim;
};
hipError_t launch_rotary(const RotaryRows& a, const RotaryArgs& rot, hipStream_t st);

struct AppendArgs {
  RotaryRows q;                // heads 0: no q
  const uint16_t* k;
  const uint16_t* v;
  const int64_t* slots;
  int64_t ld_k, ld_v, tokens;
  RotaryArgs rot;
  CacheView cache;
};
hipError_t launch_paged_kv_append(const AppendArgs& a, hipStream_t st);

hipError_t launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, float* scales,
                                hipStream_t st);

struct Int8Args {
  const int8_t* a;             // [m, k]
  const float* a_scale;        // [m]
  const int8_t* w;             // [n, k]
  const float* w_scale;        // [n]
  void* out;                   // [m, n], row stride ld_out
  void* workspace;             // int8_workspace_bytes(m, n, k), or null: k is not split
  int64_t m, n, k, ld_out;
  int out_bf16;
  // set by the launcher: parts of k, and where the workgroups of a tile count themselves and leave their sums
  int splits;
  uint32_t* arrived;
  int* parts;
};
// Of a product of exactly these sizes.  It is the same for tokens 1 - 32 (but for those of the
// streaming kernel, which needs none) and for those of one multiple of 64.
size_t int8_workspace_bytes(int64_t m, int64_t n, int64_t k);
constexpr int64_t kInt8FewTokens = 32, kInt8TokenStep = 64;
// Tokens beyond which no product of n channels is split along k: more than 128 tiles of
// 128 x 128, or of smaller ones, fill the chip by themselves.
inline int64_t int8_split_tokens(int64_t n) { return 128 / ((n + 127) / 128) * 128; }
hipError_t launch_gemm_w8a8(const Int8Args& a, hipStream_t st);
// x [g.m, g.k] quantised into codes and scales (g.a and g.a_scale), and the product.
hipError_t launch_int8_linear(const uint16_t* x, int64_t ld_x, int8_t* codes, float* scales, const Int8Args& g, hipStream_t st);

}  // namespace nvfp4
