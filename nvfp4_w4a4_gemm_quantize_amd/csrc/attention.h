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
// Rows and waves of a workgroup of the tiled kernel, and its grid: one workgroup a CU.
constexpr int kChunkRows = 256, kChunkWaves = 8, kChunkGrid = 256;

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

// Element types of the cache as the kernels are built for them.
enum CacheKind { kCacheBf16, kCacheE4m3, kCacheE4m3Blocks, kCacheInt8Blocks };
constexpr bool has_blocks(int kind) { return kind >= kCacheE4m3Blocks; }
inline CacheKind cache_kind(const CacheView& c) {
  return c.blocks == kBlocksInt8 ? kCacheInt8Blocks : c.blocks == kBlocksE4m3 ? kCacheE4m3Blocks : c.fp8 ? kCacheE4m3 : kCacheBf16;
}

// Two 8-bit elements (the low or high half of w) times a power of two as bf16: exact,
// E4M3's four significand bits and INT8's eight into eight.  The E4M3 conversion has
// the scale as its operand, for nothing.
template <int KIND, bool HI>
__device__ __forceinline__ uint32_t to_bf16(uint32_t w, float scale) {
  if constexpr (KIND == kCacheInt8Blocks) {
    const int x = (int)w;
    const float lo = (float)(HI ? x << 8 >> 24 : x << 24 >> 24), hi = (float)(HI ? x >> 24 : x << 16 >> 24);
    return pack_bf16(lo * scale, hi * scale);
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, KIND == kCacheE4m3 ? 1.0f : scale, HI));
  }
}

// The scale byte of 16 tokens of a head, of K in bits 0-7 and of V in bits 8-15, as its
// place (page, token in page) has it; within the bytes that stand for finite values.
__device__ __forceinline__ int block_scales(const CacheView& c, int head, uint32_t page, int token) {
  const int64_t at = ((int64_t)page * c.heads + head) << (c.page_shift - 4) | token >> 4;
  const int most = c.blocks == kBlocksInt8 ? kMostInt8 : kMostE4m3;
  return min(max((int)c.k_blocks[at], 1), most) | min(max((int)c.v_blocks[at], 1), most) << 8;
}
__device__ __forceinline__ float scale_of(int scales, bool values) {
  return __uint_as_float((uint32_t)(values ? scales >> 8 : scales & 0xff) << 23);
}

// A request's new tokens and keys.  Lengths fit 32 bits; none is negative but
// pos0 where the request is shorter than its chunk.
struct RequestLens {
  int start;    // first row of q
  int tokens;   // new tokens
  int keys;     // keys that the table has room for, the new ones among them
  int pos0;     // position of the first new token
};
__device__ __forceinline__ RequestLens request_lens(const AttentionArgs& a, int r) {
  RequestLens l;
  const int rows = (int)a.tokens, seq = max(a.seq_lens[r], 0);
  l.start = min(max(a.q_start[r], 0), rows);
  l.tokens = max(min(a.q_start[r + 1], rows) - l.start, 0);
  l.keys = (int)min((int64_t)seq, a.max_pages << a.cache.page_shift);
  l.pos0 = seq - l.tokens;
  return l;
}
// First key that a row at this position may see (it sees none at a negative one).
__device__ __forceinline__ int low_of(const AttentionArgs& a, int pos) {
  return a.window && pos >= a.window ? pos - a.window + 1 : 0;
}
// n / group for 0 <= n < 2^31.
__device__ __forceinline__ int div_group(const AttentionArgs& a, int n) {
  return a.group == 1 ? n : (int)(__umulhi((uint32_t)n, a.group_mul) >> a.group_shift);
}
// floor(n / d) through the fp64 reciprocal, 0 <= n < 2^43, 0 < d.
__device__ __forceinline__ int64_t div_f64(int64_t n, int64_t d) { return (int64_t)((double)n / (double)d); }

// Infinities and NaN among the values.  0 * inf is not 0, so in a tile of which some
// row does not see every key they are taken out of the product, and a row that sees
// them gets them added at the end: its sum is infinite or NaN whatever the weight is.
// A word of the cache without them:
template <int KIND>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if (KIND == kCacheInt8Blocks) return w;
  if (KIND != kCacheBf16) {
    const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return w & ~((nan >> 7) * 0xffu);
  }
  const uint32_t bad = ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  return w & ~((bad >> 15) * 0xffffu);
}
// x + what four columns at p hold of infinities and NaN, times by.
template <int KIND>
__device__ __forceinline__ f32x4 add_not_finite(f32x4 x, const uint8_t* p, float by) {
  if (KIND == kCacheInt8Blocks) return x;
  float v[4];
  if constexpr (KIND != kCacheBf16) {
    const uint32_t w = *(const uint32_t*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (w >> 8 * i & 0x7f) == 0x7f ? NAN : 0.f;
  } else {
    const u32x2 w = *(const u32x2*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i >> 1] >> 16 * (i & 1) << 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(fabsf(v[i]) < INFINITY)) x[i] = fmaf(v[i], by, x[i]);
  return x;
}

// Two neighbouring floats as one device-scope atomic: past the XCD's own L2.
__device__ __forceinline__ void store_shared(float* p, float x, float y) {
  const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
  __hip_atomic_store((uint64_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_shared(const float* p) {
  const uint64_t v = __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
// This wave's stores have been acknowledged, and none is moved behind this.
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Parts of workgroups g0 .. g1 joined in their order, four columns at d: their
// common maximum (log2 units), the sum and the unnormalised output.  Eight parts'
// loads are in flight together.
// SHARED: parts that workgroups of the same launch have left (load_shared).
template <int D, bool SHARED, class Slot>
__device__ __forceinline__ float join_parts(const float2* ml, const float* o, Slot slot_of, int g0, int g1, int d, float* den,
                                            f32x4* num) {
  constexpr int kAtOnce = 8;
  float top = -INFINITY;
  *den = 0.f;
  *num = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int g = g0; g <= g1; g += kAtOnce) {
    float2 m[kAtOnce];
    f32x4 x[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int64_t slot = slot_of(min(g + i, g1));
      if constexpr (SHARED) {
        m[i] = load_shared((const float*)(ml + slot));
        const float2 lo = load_shared(o + slot * D + d), hi = load_shared(o + slot * D + d + 2);
        x[i] = f32x4{lo.x, lo.y, hi.x, hi.y};
      } else {
        m[i] = ml[slot];
        x[i] = *(const f32x4*)(o + slot * D + d);
      }
    }
    float to = top;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) to = fmaxf(to, m[i].x);
    const float by = top == to ? 1.f : exp2_fast(top - to);   // -inf before the first part: 0
    *den *= by;
    *num *= by;
    top = to;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (g + i > g1) break;
      const float w = m[i].x == -INFINITY ? 0.f : exp2_fast(m[i].x - top);
      *den = fmaf(w, m[i].y, *den);
#pragma unroll
      for (int k = 0; k < 4; ++k) (*num)[k] = fmaf(w, x[i][k], (*num)[k]);
    }
  }
  return top;
}

// Four columns of row `at` of a head's rows that begin at token `start`, and its
// log-sum-exp: num / den * vs and log(den) + top.
template <int D>
__device__ __forceinline__ void write_row(const AttentionArgs& a, int start, int head, int at, int d, float top, float den,
                                          f32x4 num, float vs) {
  const int token = div_group(a, at), hq = head * a.group + at - token * a.group;
  const int64_t trow = start + token;
  const float inv = den == 0.f ? 0.f : vs / den;
  if (a.out_bf16)
    *(u32x2*)((uint16_t*)a.out + trow * a.ld_out + hq * D + d) = u32x2{pack_bf16(num[0] * inv, num[1] * inv), pack_bf16(num[2] * inv, num[3] * inv)};
  else
    *(f32x4*)((float*)a.out + trow * a.ld_out + hq * D + d) = num * inv;
  if (a.lse && d == 0) a.lse[trow * a.hq + hq] = den == 0.f ? -INFINITY : kLn2 * (top + __log2f(den));
}

// Rows of no request, from `row` on: 0 and lse = -inf, a row a workgroup.
__device__ __forceinline__ void clear_padding(const AttentionArgs& a, int row) {
  const int pieces = a.hq * a.cache.dim / 4;
  for (int64_t t = max(row, 0) + (int64_t)blockIdx.x; t < a.tokens; t += gridDim.x) {
    for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
      if (a.out_bf16)
        *(u32x2*)((uint16_t*)a.out + t * a.ld_out + 4 * i) = u32x2{0u, 0u};
      else
        *(f32x4*)((float*)a.out + t * a.ld_out + 4 * i) = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (a.lse)
      for (int i = threadIdx.x; i < a.hq; i += blockDim.x) a.lse[t * a.hq + i] = -INFINITY;
  }
}

// Launches of the two kernels and of their joins (attention_*.hip).
hipError_t launch_attention_decode(const AttentionArgs& a, hipStream_t st);
hipError_t launch_attention_chunk(const AttentionArgs& a, void* workspace, hipStream_t st);
constexpr size_t kArrivedBytes = kDecodeGrid * sizeof(uint32_t);
size_t attention_decode_workspace(int dim);   // beside the counters
size_t attention_chunk_workspace(int64_t requests, int dim);

}  // namespace nvfp4
