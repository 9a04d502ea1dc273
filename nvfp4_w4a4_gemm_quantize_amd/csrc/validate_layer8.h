// Host-side argument validation of the attention layer in 8 bits, and the host
// function that makes a rotation's table.  Pure C++ (no HIP headers), so it can be
// compiled and exercised without a GPU.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// What rotary_steps writes (include/nvfp4.h); a status code.
int make_rotary_steps(int rotary_dim, double base, int scaling, double factor, double original_length,
                      double slow_turns, double fast_turns, const double* pair_factors, uint64_t* steps,
                      float* amplitude);
int validate_rotation(const void* positions, const void* steps, int rotary_dim, int layout, float amplitude,
                      int head_dim, int64_t tokens);
int validate_rotary_rows(const void* x, int64_t ld_x, int64_t tokens, int num_heads, int head_dim, const void* out,
                         int64_t ld_out);
// A cache with a scale for each block: kinds NVFP4_CACHE_E4M3_BLOCKS and NVFP4_CACHE_INT8_BLOCKS.
int validate_block_cache(const void* k_cache, const void* v_cache, int cache_dtype, int64_t num_pages, int page_size,
                         int num_kv_heads, int head_dim, int64_t page_stride, int64_t head_stride,
                         int64_t token_stride, const void* k_blocks, const void* v_blocks);

}  // namespace nvfp4
