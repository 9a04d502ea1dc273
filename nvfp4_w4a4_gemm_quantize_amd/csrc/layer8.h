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

// A rotation: pair i of a head turns by steps[i] * position 2^-64ths of a turn.
struct RotaryArgs {
  const uint64_t* steps;       // [dim / 2]
  const int32_t* positions;    // [tokens]; negative: not turned
  int dim;                     // leading columns of a head that are rotated; 0: none
  int interleaved;             // pairs (2 i, 2 i + 1), else (i, i + dim / 2)
  float amplitude;             // on cosine and sine
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

}  // namespace nvfp4
