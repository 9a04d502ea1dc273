// What the attention kernels of the paged serving step share: the split of
// the work over requests, the cache's addresses and the softmax's pieces.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>

#include "serving.h"

namespace nvfp4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Rows (new tokens x heads of a KV head's group) up to which a request goes to
// the streaming kernel (attention_decode.hip); more go to the tiled kernel
// (attention_chunk.hip).
constexpr int kDecodeRows = 32;
// The streaming kernel's workgroups: a fixed grid that shares all key tiles.
constexpr int kDecodeWaves = 4, kDecodeGrid = 512, kDecodeTile = 32;
// Rows and waves of a workgroup of the tiled kernel.
constexpr int kChunkRows = 256, kChunkWaves = 8;

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2 p;
  p[0] = (__bf16)lo;
  p[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, p);
}

// Two E4M3 bytes (the low or high half of w) as bf16: exact, three significand
// bits into eight.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI));
}

// A request's new tokens and keys.
struct RequestLens {
  int64_t start;    // first row of q
  int64_t tokens;   // new tokens
  int64_t keys;     // keys, the new ones among them
};
__device__ __forceinline__ RequestLens request_lens(const AttentionArgs& a, int64_t r) {
  RequestLens l;
  const int64_t s0 = min(max((int64_t)a.q_start[r], (int64_t)0), a.tokens);
  const int64_t s1 = min((int64_t)a.q_start[r + 1], a.tokens);
  l.start = s0;
  l.tokens = max(s1 - s0, (int64_t)0);
  l.keys = min(max((int64_t)a.seq_lens[r], (int64_t)0), a.max_pages << a.cache.page_shift);
  return l;
}
// The position of new token i; keys past the table are cut off, positions are not.
__device__ __forceinline__ int64_t token_pos(const AttentionArgs& a, int64_t r, const RequestLens& l, int64_t i) {
  return (int64_t)a.seq_lens[r] - l.tokens + i;
}

// Launches of the two kernels and of their joins (attention_*.hip).
hipError_t launch_attention_decode(const AttentionArgs& a, hipStream_t st);
hipError_t launch_attention_chunk(const AttentionArgs& a, void* workspace, hipStream_t st);
size_t attention_decode_workspace(int64_t requests, int dim);
size_t attention_chunk_workspace(int64_t tokens, int64_t requests, int hq, int hkv, int dim, int64_t max_seq);

}  // namespace nvfp4
