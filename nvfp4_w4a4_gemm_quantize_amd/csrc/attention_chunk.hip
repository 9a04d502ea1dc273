// Attention of a chunk of new tokens over the paged cache on gfx950: the tiled
// kernel (requests with more than 32 rows a KV head).
//
// Mathematics as in attention_decode.hip: one pass over the keys with the
// running maximum and sum; S^T = K Q^T and O^T = V^T P^T in 32x32x16 bf16
// MFMAs, so that a softmax row lies in two lanes and P^T feeds the second
// product without leaving its registers (the k index of that product stands
// for the keys in the order in which the first product leaves them).
//
// Tile: 256 rows (new tokens x heads of the group) of one KV head for eight
// waves of 32 rows; K and V pass through LDS a tile of 64 keys at a time (32
// for heads of 256).  An E4M3 cache becomes bf16 on its way into LDS, once for
// all eight waves.
#include "attention.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 64 * kChunkWaves;

// LDS layout of a tile: [keys][D] bf16, the 16-byte pieces of a row permuted so
// that the lanes of one read instruction meet different banks: keys are read as
// 16 bytes of 32 rows, values as 32 bytes of 4 rows (the transposing read).
template <int D>
__device__ __forceinline__ int key_swizzle(int row) {
  return D == 64 ? (row >> 1) & 7 : row & 15;
}
template <int D>
__device__ __forceinline__ int value_swizzle(int row) {
  return (D == 64 ? (row >> 1) & 3 : row & 3) << 1;
}

// 4 keys x 16 columns a group of 16 lanes; a lane gets the keys of its column.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  typedef __attribute__((address_space(3))) bf16x4* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_ptr)(uintptr_t)p));
}

struct ChunkWorkspace {
  float2* ml;   // [splits][tokens * hq]
  float* o;     // [splits][tokens * hq][dim]
};
__host__ __device__ inline ChunkWorkspace chunk_workspace(void* ws, int64_t rows, int splits) {
  ChunkWorkspace w;
  w.ml = (float2*)ws;
  w.o = (float*)((uint8_t*)ws + (rows * splits * 8 + 255) / 256 * 256);
  return w;
}

int64_t row_tiles(int64_t tokens, int64_t requests, int group) { return tokens * group / kChunkRows + requests; }

// Parts of the keys: enough for two workgroups a CU, of at least 512 keys.
int chunk_splits(int64_t tokens, int64_t requests, int group, int hkv, int64_t max_seq) {
  const int64_t wgs = row_tiles(tokens, requests, group) * hkv;
  if (wgs >= 256) return 1;
  return (int)max(min(min(512 / wgs, (max_seq + 511) / 512), (int64_t)64), (int64_t)1);
}

}  // namespace

template <int D, bool FP8>
__global__ __launch_bounds__(kThreads, 2) void attention_chunk_kernel(AttentionArgs a, ChunkWorkspace ws, int splits) {
  constexpr int KT = D == 256 ? 32 : 64;
  constexpr int NK = KT / 32;                 // key fragments of a tile
  constexpr int KS = D / 16;                  // k steps of the first product
  constexpr int DF = D / 32;                  // fragments of O
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int ROW = D * 2;                  // bytes of an LDS row
  constexpr int EP = 16 / EB;                 // elements of a 16-byte piece in the cache
  constexpr int PIECES = KT * D / EP / kThreads;   // 16-byte pieces a thread brings of K (and of V)
  constexpr int PPR = D / EP;                 // pieces a row
  static_assert(KT * D / EP % kThreads == 0 || KT * D / EP < kThreads, "");
  constexpr int NP = PIECES > 0 ? PIECES : 1;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_k[2][KT * ROW], lds_v[2][KT * ROW];
  __shared__ int32_t lds_held[2][KT / 16];

  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hkv = a.cache.heads, group = a.group;
  const int head = blockIdx.x % hkv;
  const int split = blockIdx.x / hkv % splits;
  const int64_t tiles = gridDim.x / hkv / splits;
  const int64_t vt = tiles - 1 - blockIdx.x / hkv / splits;   // long tiles of a prompt first

  // Row tiles are numbered without a prefix sum: request r's start at
  // floor(q_start[r] G / 256) + r, which leaves room for all of them and
  // sometimes a number that stands for none.
  int64_t lo = 0, hi = a.requests - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if ((int64_t)a.q_start[mid] * group / kChunkRows + mid <= vt) lo = mid; else hi = mid - 1;
  }
  const int64_t r = lo;
  const RequestLens l = request_lens(a, r);
  const int64_t nrows = l.tokens * group, b = vt - ((int64_t)a.q_start[r] * group / kChunkRows + r);
  if (nrows <= kDecodeRows || b < 0 || b * kChunkRows >= nrows) return;

  const int64_t row0 = b * kChunkRows, row_end = min(row0 + kChunkRows, nrows);
  const int64_t pos_first = token_pos(a, r, l, row0 / group), pos_last = token_pos(a, r, l, (row_end - 1) / group);
  const int64_t keys = min(l.keys, pos_last + 1);
  const int64_t low = a.window ? max(pos_first - a.window + 1, (int64_t)0) : 0;
  const int64_t begin = low / KT * KT;
  const int64_t all = max((keys - begin + KT - 1) / KT, (int64_t)0);
  const int64_t share = (all + splits - 1) / splits;
  const int64_t t_begin = min(split * share, all), t_end = min(t_begin + share, all);

  float c = a.scale * kLog2e;
  if (a.cache.k_scale) c *= a.cache.k_scale[head];
  const uint32_t flip = c < 0.f ? 0x80008000u : 0u;
  c = fabsf(c);

  // this lane's row of q, the B operand: column c32, k = 8 columns of q
  const int64_t my_row = row0 + wave * 32 + c32;
  const bool live = my_row < nrows;
  const int64_t my_token = live ? my_row / group : 0;
  const int my_head = head * group + (live ? (int)(my_row % group) : 0);
  const int64_t my_pos = live ? token_pos(a, r, l, my_token) : -1;
  const int64_t wave_row = row0 + wave * 32;
  const bool wave_live = wave_row < nrows;
  const int64_t wave_pos0 = token_pos(a, r, l, wave_row / group);
  const int64_t wave_pos1 = token_pos(a, r, l, min(wave_row + 31, nrows - 1) / group);
  bf16x8 q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    u32x4 w = *(const u32x4*)(a.q + (l.start + my_token) * a.ld_q + (int64_t)my_head * D + s * 16 + h * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = live ? w[i] ^ flip : 0u;
    q[s] = __builtin_bit_cast(bf16x8, w);
  }

  const int32_t* table = a.block_table + r * a.ld_table;
  const int64_t page_mask = ((int64_t)1 << a.cache.page_shift) - 1;
  const int64_t head_off = head * a.cache.head_stride;
  u32x4 kr[NP], vr[NP];
  int32_t held_r[NP];
  const bool loads = PIECES > 0 || tid < KT * D / EP;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int piece = i * kThreads + tid, row = piece / PPR, col = piece % PPR;
      const int64_t key = begin + t * KT + row;
      int32_t page = -1;
      if (loads && key < keys) page = table[key >> a.cache.page_shift];
      held_r[i] = page >= 0 && page < a.cache.num_pages;
      kr[i] = vr[i] = u32x4{0u, 0u, 0u, 0u};   // what lies in unwritten or foreign places may be NaN
      if (held_r[i] && key >= low) {
        const int64_t at = (page * a.cache.page_stride + head_off + (key & page_mask) * a.cache.token_stride + col * EP) * EB;
        kr[i] = *(const u32x4*)((const uint8_t*)a.cache.k + at);
        vr[i] = *(const u32x4*)((const uint8_t*)a.cache.v + at);
      }
    }
  };
  auto store = [&](int stage) {
    if (!loads) return;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int piece = i * kThreads + tid, row = piece / PPR, col = piece % PPR;
      uint8_t* kp = lds_k[stage] + row * ROW;
      uint8_t* vp = lds_v[stage] + row * ROW;
      const int ks = key_swizzle<D>(row), vs = value_swizzle<D>(row);
      if constexpr (FP8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          *(u32x4*)(kp + ((2 * col + j) ^ ks) * 16) = u32x4{e4m3_bf16<false>(kr[i][2 * j]), e4m3_bf16<true>(kr[i][2 * j]), e4m3_bf16<false>(kr[i][2 * j + 1]), e4m3_bf16<true>(kr[i][2 * j + 1])};
          *(u32x4*)(vp + ((2 * col + j) ^ vs) * 16) = u32x4{e4m3_bf16<false>(vr[i][2 * j]), e4m3_bf16<true>(vr[i][2 * j]), e4m3_bf16<false>(vr[i][2 * j + 1]), e4m3_bf16<true>(vr[i][2 * j + 1])};
        }
      } else {
        *(u32x4*)(kp + (col ^ ks) * 16) = kr[i];
        *(u32x4*)(vp + (col ^ vs) * 16) = vr[i];
      }
      // a page holds 16 keys or a multiple: one key of 16 tells whether there is one
      if (col == 0 && row % 16 == 0) lds_held[stage][row / 16] = held_r[i];
    }
  };

  float m = -INFINITY, sum = 0.f;
  f32x16 o[DF];
#pragma unroll
  for (int i = 0; i < DF; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;

  // lane parts of the LDS addresses
  const int k_row = c32 * ROW, k_x = (h ^ key_swizzle<D>(c32)) * 16;
  const int v_r = 4 * h + ((lane & 15) >> 2);
  const int v_row = v_r * ROW + (lane & 1) * 8, v_x = ((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swizzle<D>(v_r)) * 16;

  if (t_begin < t_end) {
    load(t_begin);
    store(0);
  }
  __syncthreads();
  for (int64_t t = t_begin; t < t_end; ++t) {
    const int stage = (int)(t - t_begin) & 1;
    const bool more = t + 1 < t_end;
    if (more) load(t + 1);
    const int64_t key0 = begin + t * KT;
    if (wave_live && key0 <= wave_pos1 && !(a.window && key0 + KT <= wave_pos0 - a.window + 1)) {
      f32x16 s[NK];
#pragma unroll
      for (int f = 0; f < NK; ++f) {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[f][j] = 0.f;
#pragma unroll
        for (int st = 0; st < KS; ++st) {
          const bf16x8 kf = *(const bf16x8*)(lds_k[stage] + f * 32 * ROW + k_row + ((st * 32) ^ k_x));
          s[f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[st], s[f], 0, 0, 0);
        }
      }
      int32_t held = 1;
#pragma unroll
      for (int i = 0; i < KT / 16; ++i) held &= lds_held[stage][i];
      const bool full = __builtin_amdgcn_readfirstlane(held) && key0 + KT - 1 <= wave_pos0 && key0 + KT <= keys &&
                        (a.window == 0 || key0 > wave_pos1 - a.window);
      if (!full) {
#pragma unroll
        for (int f = 0; f < NK; ++f)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int in = f * 32 + 8 * (j >> 2) + 4 * h + (j & 3);
            const int64_t key = key0 + in;
            if (key > my_pos || key >= keys || !lds_held[stage][in / 16] || (a.window && key <= my_pos - a.window)) s[f][j] = -INFINITY;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int f = 0; f < NK; ++f)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, s[f][j]);
      if (__any(top > m)) {
        top = fmaxf(top, __shfl_xor(top, 32));
        const float to = fmaxf(m, top);
        const float by = m == to ? 1.f : m == -INFINITY ? 0.f : exp2_fast(c * (m - to));
        m = to;
        sum *= by;
#pragma unroll
        for (int i = 0; i < DF; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[i][j] *= by;
      }
      const float ref = m == -INFINITY ? 0.f : c * m;
#pragma unroll
      for (int f = 0; f < NK; ++f)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            e[j] = exp2_fast(fmaf(s[f][8 * u + j], c, -ref));
            if (!full && s[f][8 * u + j] == -INFINITY) e[j] = 0.f;
          }
          sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
          // P in bf16, the matrix instruction's type with V: 2^-8 relative a term at most, averaged over the keys
          const bf16x8 p = __builtin_bit_cast(bf16x8, u32x4{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7])});
#pragma unroll
          for (int i = 0; i < DF; ++i) {
            const uint8_t* vp = lds_v[stage] + (f * 32 + u * 16) * ROW + v_row + ((i * 64) ^ v_x);
            const u32x2 v0 = read_transposed(vp), v1 = read_transposed(vp + 8 * ROW);
            o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, u32x4{v0[0], v0[1], v1[0], v1[1]}), p, o[i], 0, 0, 0);
          }
        }
    }
    if (more) store(stage ^ 1);
    __syncthreads();
  }

  sum += __shfl_xor(sum, 32);
  if (!live) return;
  const int64_t trow = l.start + my_token;
  const float top = m == -INFINITY ? -INFINITY : c * m;
  if (splits == 1) {
    const float vs = a.cache.v_scale ? a.cache.v_scale[head] : 1.f;
    const float inv = sum == 0.f ? 0.f : vs / sum;
#pragma unroll
    for (int i = 0; i < DF; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = trow * a.ld_out + (int64_t)my_head * D + 32 * i + 8 * j + 4 * h;
        const f32x4 x = f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]} * inv;
        if (a.out_bf16)
          *(u32x2*)((uint16_t*)a.out + at) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        else
          *(f32x4*)((float*)a.out + at) = x;
      }
    if (a.lse && h == 0) a.lse[trow * a.hq + my_head] = sum == 0.f ? -INFINITY : kLn2 * (top + __log2f(sum));
  } else {
    const int64_t slot = (split * a.tokens + trow) * a.hq + my_head;
    if (h == 0) ws.ml[slot] = make_float2(top, sum);
    if (t_begin < t_end)
#pragma unroll
      for (int i = 0; i < DF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *(f32x4*)(ws.o + slot * D + 32 * i + 8 * j + 4 * h) = f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
  }
}

// Joins the parts of a token's rows in the order of their keys; a part without keys has sum 0.
template <int D>
__global__ __launch_bounds__(256) void attention_chunk_join_kernel(AttentionArgs a, ChunkWorkspace ws, int splits) {
  const int64_t trow = blockIdx.x;
  int64_t lo = 0, hi = a.requests - 1;   // the request of the token: the last that starts at or before it
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (a.q_start[mid] <= trow) lo = mid; else hi = mid - 1;
  }
  const RequestLens l = request_lens(a, lo);
  if (trow >= l.start + l.tokens || l.tokens * a.group <= kDecodeRows) return;
  for (int e = threadIdx.x; e < a.hq * (D / 4); e += 256) {
    const int hq = e / (D / 4), d = (e % (D / 4)) * 4;
    float top = -INFINITY, den = 0.f;
    f32x4 num = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) top = fmaxf(top, ws.ml[(s * a.tokens + trow) * a.hq + hq].x);
    for (int s = 0; s < splits; ++s) {
      const int64_t slot = (s * a.tokens + trow) * a.hq + hq;
      const float2 ml = ws.ml[slot];
      if (ml.y == 0.f) continue;
      const float by = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
      den = fmaf(by, ml.y, den);
      const f32x4 ow = *(const f32x4*)(ws.o + slot * D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) num[i] = fmaf(by, ow[i], num[i]);
    }
    const float vs = a.cache.v_scale ? a.cache.v_scale[hq / a.group] : 1.f;
    const float inv = den == 0.f ? 0.f : vs / den;
    if (a.out_bf16)
      *(u32x2*)((uint16_t*)a.out + trow * a.ld_out + (int64_t)hq * D + d) = u32x2{pack_bf16(num[0] * inv, num[1] * inv), pack_bf16(num[2] * inv, num[3] * inv)};
    else
      *(f32x4*)((float*)a.out + trow * a.ld_out + (int64_t)hq * D + d) = num * inv;
    if (a.lse && d == 0) a.lse[trow * a.hq + hq] = den == 0.f ? -INFINITY : kLn2 * (top + __log2f(den));
  }
}

size_t attention_chunk_workspace(int64_t tokens, int64_t requests, int hq, int hkv, int dim, int64_t max_seq) {
  const int splits = chunk_splits(tokens, requests, hq / hkv, hkv, max_seq);
  if (splits == 1) return 0;
  return (size_t)(uintptr_t)chunk_workspace(nullptr, tokens * hq, splits).o + (size_t)splits * tokens * hq * dim * sizeof(float);
}

namespace {

template <int D, bool FP8>
hipError_t launch(const AttentionArgs& a, void* workspace, hipStream_t st) {
  const int splits = chunk_splits(a.tokens, a.requests, a.group, a.cache.heads, a.max_seq);
  const ChunkWorkspace ws = chunk_workspace(workspace, a.tokens * a.hq, splits);
  const unsigned grid = (unsigned)(row_tiles(a.tokens, a.requests, a.group) * a.cache.heads * splits);
  attention_chunk_kernel<D, FP8><<<grid, kThreads, 0, st>>>(a, ws, splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  attention_chunk_join_kernel<D><<<(unsigned)a.tokens, 256, 0, st>>>(a, ws, splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_chunk(const AttentionArgs& a, void* workspace, hipStream_t st) {
  switch (a.cache.dim) {
    case 64: return a.cache.fp8 ? launch<64, true>(a, workspace, st) : launch<64, false>(a, workspace, st);
    case 128: return a.cache.fp8 ? launch<128, true>(a, workspace, st) : launch<128, false>(a, workspace, st);
    default: return a.cache.fp8 ? launch<256, true>(a, workspace, st) : launch<256, false>(a, workspace, st);
  }
}

// ------------------------------------------------------------- dispatch ----

// A request with at most 32 rows a KV head goes to the streaming kernel, any
// other to the tiled one; both are launched where the batch may hold both.
static bool may_stream(int64_t max_new, int group) { return max_new > 0 && group <= kDecodeRows; }
static bool may_tile(int64_t max_new, int group) { return max_new * group > kDecodeRows; }

size_t attention_workspace_bytes(int64_t tokens, int64_t requests, int hq, int hkv, int dim, int64_t max_new,
                                 int64_t max_seq) {
  const int group = hq / hkv;
  size_t n = 16;
  if (may_stream(max_new, group)) n += (attention_decode_workspace(requests, dim) + 255) / 256 * 256;
  if (may_tile(max_new, group)) n += attention_chunk_workspace(tokens, requests, hq, hkv, dim, max_seq);
  return n;
}

hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t st) {
  uint8_t* ws = (uint8_t*)a.workspace;
  if (may_stream(a.max_new, a.group)) {
    hipError_t e = launch_attention_decode(a, st);
    if (e != hipSuccess) return e;
    ws += (attention_decode_workspace(a.requests, a.cache.dim) + 255) / 256 * 256;
  }
  return may_tile(a.max_new, a.group) ? launch_attention_chunk(a, ws, st) : hipSuccess;
}

}  // namespace nvfp4
