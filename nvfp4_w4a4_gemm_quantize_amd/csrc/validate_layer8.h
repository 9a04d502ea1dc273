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
                      double* amplitude);
int validate_rotation(const void* positions, const void* steps, int rotary_dim, int layout, double amplitude,
                      int head_dim, int64_t tokens);
int validate_rotary_rows(const void* x, int64_t ld_x, int64_t tokens, int num_heads, int head_dim, const void* out,
                         int64_t ld_out);
// A cache with a scale for each block: kinds NVFP4_CACHE_E4M3_BLOCKS and NVFP4_CACHE_INT8_BLOCKS.
int validate_block_cache(const void* k_cache, const void* v_cache, int cache_dtype, int64_t num_pages, int page_size,
                         int num_kv_heads, int head_dim, int64_t page_stride, int64_t head_stride,
                         int64_t token_stride, const void* k_blocks, const void* v_blocks);
int validate_int8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, const void* codes, const void* scales);
int validate_w8a8_sizes(int64_t m, int64_t n, int64_t k);
int validate_gemm_w8a8(const void* a, const void* a_scale, int64_t m, const void* w, const void* w_scale, int64_t n, int64_t k,
                       const void* out, int out_dtype, int64_t ld_out, const void* workspace, size_t workspace_bytes,
                       size_t needed);

}  // namespace nvfp4
