// Rotary positions on gfx950, on their own (rotary) and on the way into the paged
// cache (paged_kv_append).  Declared and documented in include/nvfp4.h.
//
// Pair (a, b) of a head at position p becomes (a cos t - b sin t, b cos t + a sin t)
// times the amplitude, with t = 2 pi p step / 2^64.  step * p modulo 2^64 is the
// fraction of a turn whatever p is: whole turns fall off by themselves, and an angle
// is as exact at position 10^6 as at 1 (in fp32 radians it would be off by 0.03).
//
// A thread owns 16 columns of a head (a unit: 8 pairs) of one token, finds their
// cosines and sines once and uses them for several heads, so that the angles' some
// 400 instructions stay beside the loads.
#include <hip/hip_runtime.h>

#include "attention.h"
#include "layer8.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// cos and sin of x / 2^32 turns times amplitude, rounded once.  The nearest quarter is
// taken off, which leaves at most an eighth of a turn, where the Taylor series up to x^11
// and x^10 are off by less than 10^-10.  In fp64, whose FMA takes no longer here: fp32's
// last digit would move a hundred times as many 8-bit codes of rotated keys to the other
// side of a tie.
__device__ __forceinline__ float2 cos_sin(uint32_t x, double amplitude) {
  const uint32_t quarter = (x + 0x20000000u) >> 30;
  const double t = (double)(int32_t)(x - (quarter << 30)) * 1.46291807926715968e-9;   // 2 pi / 2^32
  const double u = t * t;
  const double s = fma(t * u, fma(u, fma(u, fma(u, fma(u, -1. / 39916800, 1. / 362880), -1. / 5040), 1. / 120), -1. / 6), t);
  const double c = fma(u, fma(u, fma(u, fma(u, fma(u, -1. / 3628800, 1. / 40320), -1. / 720), 1. / 24), -0.5), 1.);
  const float cc = (float)((quarter & 1 ? s : c) * amplitude), ss = (float)((quarter & 1 ? c : s) * amplitude);
  return make_float2((quarter + 1) & 2 ? -cc : cc, quarter & 2 ? -ss : ss);
}

// The turns of unit u's eight pairs at a position.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void find_turn(Turn& t, const RotaryArgs& rot, int unit, int position) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t phase = rot.steps[unit * 8 + i] * (uint64_t)(uint32_t)position;
    const float2 cs = cos_sin((uint32_t)(phase >> 32), rot.amplitude);
    t.c[i] = position < 0 ? 1.f : cs.x;
    t.s[i] = position < 0 ? 0.f : cs.y;
  }
}

// Columns of a unit: two runs of eight, at lo and hi.
struct UnitAt {
  int lo, hi;
  bool turns;
};
__device__ __forceinline__ UnitAt unit_at(const RotaryArgs& rot, int unit) {
  UnitAt at;
  at.turns = unit * 16 < rot.dim;
  const bool split = at.turns && !rot.interleaved;
  at.lo = split ? unit * 8 : unit * 16;
  at.hi = split ? unit * 8 + rot.dim / 2 : unit * 16 + 8;
  return at;
}

__device__ __forceinline__ void unpack(const u32x4& w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 pack(const float* f) {
  return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// x[0 .. 7] and x[8 .. 15]: the unit's two runs.
__device__ __forceinline__ void turn_unit(float* x, const Turn& t, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = interleaved ? x[2 * i] : x[i], b = interleaved ? x[2 * i + 1] : x[8 + i];
    const float ra = fmaf(a, t.c[i], -(b * t.s[i])), rb = fmaf(b, t.c[i], a * t.s[i]);
    // (the other layout's registers: both are known at compile time but for the choice)
    if (interleaved) {
      x[2 * i] = ra;
      x[2 * i + 1] = rb;
    } else {
      x[i] = ra;
      x[8 + i] = rb;
    }
  }
}

}  // namespace

// --------------------------------------------------------------- rotary ----
//
// Bound by HBM: 4 bytes an element.  Thread (token, unit) takes `per` heads from
// `per * blockIdx.y` on, four heads' loads in flight.
template <bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryRows a, RotaryArgs rot, int per) {
  const int units = a.dim / 16;
  const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = item / units;
  if (t >= a.tokens) return;
  const int unit = (int)(item - t * units), h0 = blockIdx.y * per, h1 = min(h0 + per, a.heads);
  const UnitAt at = unit_at(rot, unit);
  if (!at.turns && a.x == a.out) return;   // in place
  Turn turn;
  if (at.turns) find_turn(turn, rot, unit, rot.positions[t]);
  const uint16_t* x = a.x + t * a.ld_x;
  uint16_t* out = a.out + t * a.ld_out;
  constexpr int kAtOnce = 4;
  for (int h = h0; h < h1; h += kAtOnce) {
    u32x4 lo[kAtOnce], hi[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int64_t head = (int64_t)min(h + i, h1 - 1) * a.dim;
      lo[i] = *(const u32x4*)(x + head + at.lo);
      hi[i] = *(const u32x4*)(x + head + at.hi);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (h + i >= h1) break;
      const int64_t head = (int64_t)(h + i) * a.dim;
      if (at.turns) {
        float f[16];
        unpack(lo[i], f);
        unpack(hi[i], f + 8);
        turn_unit(f, turn, INTERLEAVED);
        lo[i] = pack(f);
        hi[i] = pack(f + 8);
      }
      *(u32x4*)(out + head + at.lo) = lo[i];
      *(u32x4*)(out + head + at.hi) = hi[i];
    }
  }
}

namespace {

// Heads a thread takes: as many as leave the chip 2^17 threads (eight waves a SIMD's
// worth), four at least, which are in flight together.
int heads_per_thread(int64_t items, int heads) {
  const int64_t per = items * heads >> 17;
  return (int)max((int64_t)1, min(per, (int64_t)heads));
}

}  // namespace

hipError_t launch_rotary(const RotaryRows& a, const RotaryArgs& rot, hipStream_t st) {
  const int64_t items = a.tokens * (a.dim / 16);
  const int per = heads_per_thread(items, a.heads);
  const dim3 grid((unsigned)((items + kThreads - 1) / kThreads), (unsigned)((a.heads + per - 1) / per));
  if (rot.interleaved)
    rotary_kernel<true><<<grid, kThreads, 0, st>>>(a, rot, per);
  else
    rotary_kernel<false><<<grid, kThreads, 0, st>>>(a, rot, per);
  return hipGetLastError();
}

// --------------------------------------------------------------- append ----
//
// q and k are rotated in fp32, and q is rounded to bf16, k to the cache's type alone;
// v goes there as it is.  Caches with one scale a head (or none) have nothing that
// joins tokens: heads q, k, v are one list, of which a thread (token, unit) takes a part.
//
// Block-scaled caches: a wave takes one run (the neighbouring rows of the call that lie
// in one block of 16 tokens) of one head of K or V, so that the block's largest value
// is a reduction over the wave and its codes are written once.  Scale 2^(e - 127) with
//     e = max(e_old, smallest e with max |x| <= M 2^(e - 127)), M = 448 or 127;
// a run that holds the block's first token begins the block (no e_old, the places that
// are not the run's become 0), any other leaves the rest as it is, divided by
// 2^(e - e_old) where the scale rises.  A power of two, because an E4M3 code then keeps
// its digits whenever it is rescaled, and the attention's conversion to bf16 is exact
// with the scale in it.
namespace {

__device__ __forceinline__ uint32_t codes4(const float* f, bool int8) {
  if (int8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r = fminf(fmaxf(rintf(f[i]), -127.f), 127.f);
      w |= ((uint32_t)(int)(f[i] != f[i] ? 0.f : r) & 0xffu) << (8 * i);
    }
    return w;
  }
  float g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = f[i] != f[i] ? f[i] : fminf(fmaxf(f[i], -448.f), 448.f);   // a NaN stays one
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(g[0], g[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(g[2], g[3], w, true);
}
__device__ __forceinline__ u32x2 codes8(const float* f, bool int8) { return u32x2{codes4(f, int8), codes4(f + 4, int8)}; }

// Four codes times 2^by (by <= 0), rounded to nearest even again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, int by, bool int8) {
  float f[4];
  if (int8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = ldexpf((float)(int8_t)(w >> (8 * i)), by);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __builtin_amdgcn_cvt_f32_fp8((int)(w >> (8 * i)), 0);
      f[i] = ldexpf(lo, by);
    }
  }
  return codes4(f, int8);
}

// E8M0 byte of the smallest power of two s with top <= M s, within 1 .. the largest.
__device__ __forceinline__ int needed_scale(float top, bool int8) {
  const uint32_t b = __float_as_uint(top), m = b & 0x7fffffu;
  const int e = (int)(b >> 23);
  // 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8
  return int8 ? min(max(e - 6 + (m > 0x7e0000u), 1), kMostInt8) : min(max(e - 8 + (m > 0x600000u), 1), kMostE4m3);
}

// Byte (= element) offset of a slot's first column.
__device__ __forceinline__ int64_t place_at(const CacheView& c, int64_t slot, int head) {
  return (slot >> c.page_shift) * c.page_stride + head * c.head_stride + (slot & (((int64_t)1 << c.page_shift) - 1)) * c.token_stride;
}

}  // namespace

template <bool INTERLEAVED, bool FP8>
__global__ __launch_bounds__(kThreads) void append_rows_kernel(AppendArgs a, int per) {
  const CacheView& c = a.cache;
  const int units = c.dim / 16, heads = a.q.heads + 2 * c.heads;
  const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = item / units;
  if (t >= a.tokens) return;
  const int unit = (int)(item - t * units), h0 = blockIdx.y * per, h1 = min(h0 + per, heads);
  const UnitAt at = unit_at(a.rot, unit);
  Turn turn;
  if (at.turns && h0 < a.q.heads + c.heads) find_turn(turn, a.rot, unit, a.rot.positions[t]);
  const int64_t slot = a.slots[t];
  const bool held = slot >= 0 && slot >> c.page_shift < c.num_pages;
  constexpr int kAtOnce = 4;
  for (int h = h0; h < h1; h += kAtOnce) {
    u32x4 lo[kAtOnce], hi[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int head = min(h + i, h1 - 1), kv = head - a.q.heads;
      const uint16_t* x = kv < 0           ? a.q.x + t * a.q.ld_x + (int64_t)head * c.dim
                          : kv < c.heads ? a.k + t * a.ld_k + (int64_t)kv * c.dim
                                         : a.v + t * a.ld_v + (int64_t)(kv - c.heads) * c.dim;
      lo[i] = *(const u32x4*)(x + at.lo);
      hi[i] = *(const u32x4*)(x + at.hi);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int head = h + i, kv = head - a.q.heads;
      if (head >= h1) break;
      if (kv >= 0 && !held) continue;
      float f[16];
      unpack(lo[i], f);
      unpack(hi[i], f + 8);
      if (at.turns && kv < c.heads) turn_unit(f, turn, INTERLEAVED);
      if (kv < 0) {
        uint16_t* out = a.q.out + t * a.q.ld_out + (int64_t)head * c.dim;
        *(u32x4*)(out + at.lo) = pack(f);
        *(u32x4*)(out + at.hi) = pack(f + 8);
        continue;
      }
      const bool is_v = kv >= c.heads;
      const int hk = is_v ? kv - c.heads : kv;
      const int64_t to = place_at(c, slot, hk);
      if constexpr (FP8) {
        const float* scales = is_v ? c.v_scale : c.k_scale;
        const float scale = scales ? scales[hk] : 1.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] /= scale;
        uint8_t* p = (uint8_t*)(is_v ? c.v : c.k) + to;
        *(u32x2*)(p + at.lo) = codes8(f, false);
        *(u32x2*)(p + at.hi) = codes8(f + 8, false);
      } else {
        uint16_t* p = (uint16_t*)(is_v ? c.v : c.k) + to;
        *(u32x4*)(p + at.lo) = pack(f);
        *(u32x4*)(p + at.hi) = pack(f + 8);
      }
    }
  }
}

// Rows 16 w .. 16 w + 15 of the call are window w; waves (window, share, head, K or V)
// take every `shares`-th of the runs that begin in it.
template <bool INTERLEAVED, bool INT8, int D>
__global__ __launch_bounds__(kThreads) void append_blocks_kernel(AppendArgs a, int shares, int64_t waves) {
  constexpr int U = D / 16;                 // units, so lanes, of a row
  constexpr int ROWS = 64 / U;              // places of the block that a pass covers
  constexpr int PASSES = kBlockTokens / ROWS;
  const CacheView& c = a.cache;
  const int lane = threadIdx.x & 63, unit = lane % U, lane_row = lane / U;
  int64_t id = (int64_t)blockIdx.x * (kThreads / 64) + uniform((int)(threadIdx.x >> 6));
  if (id >= waves) return;
  const bool is_v = id & 1;
  id >>= 1;
  const int head = (int)(id % c.heads);
  id /= c.heads;
  const int share = (int)(id % shares);
  const int64_t t0 = id / shares * kBlockTokens;
  const uint16_t* x = is_v ? a.v + (int64_t)head * D : a.k + (int64_t)head * D;
  const int64_t ld = is_v ? a.ld_v : a.ld_k;
  uint8_t* cache = (uint8_t*)(is_v ? c.v : c.k);
  uint8_t* scales = is_v ? c.v_blocks : c.k_blocks;
  UnitAt at = unit_at(a.rot, unit);
  if (is_v) at = UnitAt{unit * 16, unit * 16 + 8, false};

  // the window's rows that begin a run
  auto slot_of = [&](int64_t t) {
    if (t < 0 || t >= a.tokens) return (int64_t)-1;
    const int64_t s = a.slots[t];
    return s >= 0 && s >> c.page_shift < c.num_pages ? s : (int64_t)-1;
  };
  const int64_t mine = lane < kBlockTokens ? slot_of(t0 + lane) : -1;
  const int64_t prev = lane < kBlockTokens ? slot_of(t0 + lane - 1) : -1;
  uint64_t begins = __ballot(mine >= 0 && (prev < 0 || prev != mine - 1 || mine % kBlockTokens == 0));
  for (int skip = share; begins; skip = shares - 1) {
    for (; skip > 0 && begins; --skip) begins &= begins - 1;
    if (!begins) break;
    const int64_t t = t0 + __builtin_ctzll(begins);
    begins &= begins - 1;
    const int64_t s0 = uniform(slot_of(t));
    const int place0 = (int)(s0 % kBlockTokens);
    const bool next = lane < kBlockTokens - place0 && slot_of(t + lane) == s0 + lane;
    const int place1 = place0 + __builtin_ctzll(~__ballot(next));   // the run: places [place0, place1)
    const bool fresh = place0 == 0;
    const int64_t block = ((s0 >> c.page_shift) * c.heads + head) << (c.page_shift - 4) | (s0 & (((int64_t)1 << c.page_shift) - 1)) >> 4;
    const int64_t first = place_at(c, s0 - place0, head);
    const int old = fresh ? 1 : min(max((int)scales[block], 1), INT8 ? kMostInt8 : kMostE4m3);

    u32x4 lo[PASSES], hi[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int place = p * ROWS + lane_row;
      const bool in = place >= place0 && place < place1;
      const uint16_t* row = x + (in ? t + place - place0 : t) * ld;
      lo[p] = *(const u32x4*)(row + at.lo);
      hi[p] = *(const u32x4*)(row + at.hi);
    }
    float f[PASSES][16];
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int place = p * ROWS + lane_row;
      const bool in = place >= place0 && place < place1;
      unpack(lo[p], f[p]);
      unpack(hi[p], f[p] + 8);
      if (in && at.turns) {
        Turn turn;
        find_turn(turn, a.rot, unit, a.rot.positions[t + place - place0]);
        turn_unit(f[p], turn, INTERLEAVED);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float m = fabsf(f[p][i]);
        top = in && m < INFINITY ? fmaxf(top, m) : top;
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const int e = max(needed_scale(top, INT8), old);
    const bool rises = !fresh && e > old;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int place = p * ROWS + lane_row;
      uint8_t* to = cache + first + place * c.token_stride;
      if (place >= place0 && place < place1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[p][i] = ldexpf(f[p][i], 127 - e);
        *(u32x2*)(to + at.lo) = codes8(f[p], INT8);
        *(u32x2*)(to + at.hi) = codes8(f[p] + 8, INT8);
      } else if (fresh) {
        *(u32x4*)(to + unit * 16) = u32x4{0u, 0u, 0u, 0u};
      } else if (rises) {
        u32x4 w = *(const u32x4*)(to + unit * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = rescale4(w[i], old - e, INT8);
        *(u32x4*)(to + unit * 16) = w;
      }
    }
    if (lane == 0) scales[block] = (uint8_t)e;
  }
}

namespace {

template <bool INTERLEAVED, bool INT8>
hipError_t launch_blocks(const AppendArgs& a, hipStream_t st) {
  const CacheView& c = a.cache;
  const int64_t windows = (a.tokens + kBlockTokens - 1) / kBlockTokens;
  // every row may be a run of its own (single tokens): a wave for each of them while
  // that leaves the chip room, else one a window, as prompts have
  const int64_t each = windows * c.heads * 2;
  const int shares = each * 16 <= 8192 ? 16 : each * 4 <= 8192 ? 4 : 1;
  const int64_t waves = each * shares;
  const unsigned grid = (unsigned)((waves + kThreads / 64 - 1) / (kThreads / 64));
  switch (c.dim) {
    case 64: append_blocks_kernel<INTERLEAVED, INT8, 64><<<grid, kThreads, 0, st>>>(a, shares, waves); break;
    case 128: append_blocks_kernel<INTERLEAVED, INT8, 128><<<grid, kThreads, 0, st>>>(a, shares, waves); break;
    default: append_blocks_kernel<INTERLEAVED, INT8, 256><<<grid, kThreads, 0, st>>>(a, shares, waves);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_kv_append(const AppendArgs& a, hipStream_t st) {
  const CacheView& c = a.cache;
  const bool inter = a.rot.interleaved;
  if (c.blocks != kBlocksNone) {
    if (a.q.heads > 0) {
      const hipError_t e = launch_rotary(a.q, a.rot, st);
      if (e != hipSuccess) return e;
    }
    if (c.blocks == kBlocksInt8) return inter ? launch_blocks<true, true>(a, st) : launch_blocks<false, true>(a, st);
    return inter ? launch_blocks<true, false>(a, st) : launch_blocks<false, false>(a, st);
  }
  const int heads = a.q.heads + 2 * c.heads;
  const int64_t items = a.tokens * (c.dim / 16);
  const int per = heads_per_thread(items, heads);
  const dim3 grid((unsigned)((items + kThreads - 1) / kThreads), (unsigned)((heads + per - 1) / per));
  if (inter) {
    if (c.fp8) append_rows_kernel<true, true><<<grid, kThreads, 0, st>>>(a, per);
    else append_rows_kernel<true, false><<<grid, kThreads, 0, st>>>(a, per);
  } else {
    if (c.fp8) append_rows_kernel<false, true><<<grid, kThreads, 0, st>>>(a, per);
    else append_rows_kernel<false, false><<<grid, kThreads, 0, st>>>(a, per);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
