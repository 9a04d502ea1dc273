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

#include <algorithm>

#include "attention.h"
#include "layer8.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// cos and sin of x / 2^32 turns times amplitude, rounded by who uses them.  The nearest quarter is
// taken off, which leaves at most an eighth of a turn, where the Taylor series up to x^11
// and x^10 are off by 7 10^-12 and 1.2 10^-10 at most (what x's last place weighs, 1.5 10^-9
// radians, is more).  In fp64, whose FMA takes no longer here; block-scaled keys are turned
// in it too.
__device__ __forceinline__ double2 cos_sin(uint32_t x, double amplitude) {
  const uint32_t quarter = (x + 0x20000000u) >> 30;
  const double t = (double)(int32_t)(x - (quarter << 30)) * 1.46291807926715968e-9;   // 2 pi / 2^32
  const double u = t * t;
  const double s = fma(t * u, fma(u, fma(u, fma(u, fma(u, -1. / 39916800, 1. / 362880), -1. / 5040), 1. / 120), -1. / 6), t);
  const double c = fma(u, fma(u, fma(u, fma(u, fma(u, -1. / 3628800, 1. / 40320), -1. / 720), 1. / 24), -0.5), 1.);
  const double cc = (quarter & 1 ? s : c) * amplitude, ss = (quarter & 1 ? c : s) * amplitude;
  return make_double2((quarter + 1) & 2 ? -cc : cc, quarter & 2 ? -ss : ss);
}

// Columns of a unit: two runs of eight, at lo and hi, half of the rotated part (or of the
// rest) apart in either layout, so that neighbouring lanes read neighbouring 16 bytes.
// Halves: pairs unit * 8 on.  Interleaved: four pairs in each run.
struct UnitAt {
  int lo, hi;
  bool turns;
};
__device__ __forceinline__ UnitAt unit_at(int rotated, int dim, int unit) {
  UnitAt at;
  at.turns = unit * 16 < rotated;
  const int from = at.turns ? 0 : rotated, half = (at.turns ? rotated : dim - rotated) / 2;
  at.lo = from + (unit - from / 16) * 8;
  at.hi = at.lo + half;
  return at;
}

// The turns of a unit's eight pairs at a position; false for a negative one, whose row is not
// turned.  It is left out and not turned by 0: 0 * inf is NaN, and -0 + 0 is 0.
template <typename T>
struct Turn {
  T c[8], s[8];
};
template <bool INTERLEAVED, typename T>
__device__ __forceinline__ bool find_turn(Turn<T>& t, const RotaryArgs& rot, int unit, int position) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = INTERLEAVED ? unit * 4 + (i < 4 ? i : rot.dim / 4 + i - 4) : unit * 8 + i;
    const uint64_t phase = rot.steps[pair] * (uint64_t)(uint32_t)position;
    const double2 cs = cos_sin((uint32_t)(phase >> 32), rot.amplitude);
    t.c[i] = (T)cs.x;
    t.s[i] = (T)cs.y;
  }
  return position >= 0;
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
template <bool INTERLEAVED, typename T>
__device__ __forceinline__ void turn_unit(float* x, const Turn<T>& t) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = x[INTERLEAVED ? 2 * i : i];
    float& b = x[INTERLEAVED ? 2 * i + 1 : 8 + i];
    const T ra = fma((T)a, t.c[i], -((T)b * t.s[i])), rb = fma((T)b, t.c[i], (T)a * t.s[i]);
    a = (float)ra;
    b = (float)rb;
  }
}

}  // namespace

// --------------------------------------------------------------- rotary ----
//
// Bound by HBM: 4 bytes an element (16384 tokens, 48 heads of 128: 77 us, 5.2 TB/s; 8
// tokens: 4.4 us, latency).  Thread (token, unit) takes `per` heads of its block's group,
// four heads' loads in flight.
namespace {

template <bool INTERLEAVED, int THREADS>
__device__ __forceinline__ void rotary_rows(const RotaryRows& a, const RotaryArgs& rot, int units, int64_t block, int groups, int per) {
  const int group = (int)(block % groups);
  const int64_t item = block / groups * THREADS + threadIdx.x;
  const int64_t t = item / units;
  if (t >= a.tokens) return;
  const int unit = (int)(item - t * units), h0 = group * per, h1 = min(h0 + per, a.heads);
  const UnitAt at = unit_at(rot.dim, a.dim, unit);
  if (!at.turns && a.x == a.out) return;   // in place
  const uint16_t* x = a.x + t * a.ld_x;
  uint16_t* out = a.out + t * a.ld_out;
  constexpr int kAtOnce = 4;
  u32x4 lo[kAtOnce], hi[kAtOnce];
  auto load = [&](int i, int h) {
    lo[i] = *(const u32x4*)(x + (int64_t)h * a.dim + at.lo);
    hi[i] = *(const u32x4*)(x + (int64_t)h * a.dim + at.hi);
  };
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) load(i, min(h0 + i, h1 - 1));
  Turn<float> turn;
  const bool turns = at.turns && find_turn<INTERLEAVED>(turn, rot, unit, rot.positions[t]);
  for (int h = h0; h < h1; h += kAtOnce) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (h + i >= h1) break;
      const int64_t head = (int64_t)(h + i) * a.dim;
      if (turns) {
        float f[16];
        unpack(lo[i], f);
        unpack(hi[i], f + 8);
        turn_unit<INTERLEAVED>(f, turn);
        lo[i] = pack(f);
        hi[i] = pack(f + 8);
      }
      *(u32x4*)(out + head + at.lo) = lo[i];
      *(u32x4*)(out + head + at.hi) = hi[i];
      if (h + kAtOnce + i < h1) load(i, h + kAtOnce + i);
    }
  }
}

}  // namespace

template <bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryRows a, RotaryArgs rot, int groups, int per) {
  rotary_rows<INTERLEAVED, kThreads>(a, rot, a.dim / 16, blockIdx.x, groups, per);
}

namespace {

// Heads a thread takes, and the grid of blocks x groups of heads.  Four are in flight
// together; more pay only where the chip is filled many times over (16384 tokens, 48
// heads of 128: 6 heads a thread 77 us, 48 heads 92; 2000 tokens, 40 heads: 4 a thread 9.6
// us, 1 12.4), and few tokens want all the threads there can be.
struct RotaryGrid {
  int groups, per;
  int64_t blocks;
};
RotaryGrid rotary_grid(int64_t tokens, int heads, int dim, int threads) {
  const int64_t items = tokens * (dim / 16);
  RotaryGrid g;
  const int64_t all = items * heads, per = std::max(std::min<int64_t>(all >> 16, 4), all >> 20);
  g.per = (int)std::max<int64_t>(1, std::min<int64_t>(per, heads));
  g.groups = (heads + g.per - 1) / g.per;
  g.blocks = (items + threads - 1) / threads * g.groups;
  return g;
}

}  // namespace

hipError_t launch_rotary(const RotaryRows& a, const RotaryArgs& rot, hipStream_t st) {
  const RotaryGrid g = rotary_grid(a.tokens, a.heads, a.dim, kThreads);
  if (rot.interleaved)
    rotary_kernel<true><<<(unsigned)g.blocks, kThreads, 0, st>>>(a, rot, g.groups, g.per);
  else
    rotary_kernel<false><<<(unsigned)g.blocks, kThreads, 0, st>>>(a, rot, g.groups, g.per);
  return hipGetLastError();
}

// --------------------------------------------------------------- append ----
//
// q and k are rotated in fp32, k of block-scaled caches in fp64 rounded to fp32 (its codes are
// the formula's but for ties), and q is rounded to bf16, k to the cache's type alone; v
// goes there as it is.  Caches with one scale a head (or none) have nothing that
// joins tokens: heads q, k, v are one list, of which a thread (token, unit) takes a part.
//
// Block-scaled caches: a workgroup takes one run (the neighbouring rows of the call that
// lie in one block of 16 tokens) of one head of K or V, so that the block's largest value
// is a reduction over its lanes and its codes are written once.  Scale 2^(e - 127) with
//     e = max(e_old, smallest e with max |x| <= M 2^(e - 127)), M = 448 or 127;
// a run that holds the block's first token begins the block (no e_old, the places that
// are not the run's become 0), any other leaves the rest as it is, divided by
// 2^(e - e_old) where the scale rises.  A power of two, because an E4M3 code then keeps
// its digits whenever it is rescaled, and the attention's conversion to bf16 is exact
// with the scale in it.
//
// Bound by HBM: 16384 tokens of 40 heads of q and 8 of k and v, 128 each, into E4M3 blocks
// 84 us, 5.2 TB/s; 64 single tokens 6.2 us, latency: slots, then rows and scales, then
// stores.  8 chunks of up to 777 tokens, 16 heads of 64, bf16: 11 us, 3.9 TB/s.
namespace {

// Four values in steps of their scale as codes, rounded to nearest even.  CLAMP: they may
// lie beyond the largest code (infinities), or be NaN for INT8.
template <bool INT8, bool CLAMP>
__device__ __forceinline__ uint32_t codes4(const float* f) {
  if constexpr (INT8) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = f[i];
      if (CLAMP) x = x != x ? 0.f : fminf(fmaxf(x, -127.f), 127.f);
      b[i] = __float_as_uint(x + 12582912.f);   // 1.5 * 2^23: the sum's last bits are the whole number
    }
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    return lo | hi;
  } else {
    float g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = !CLAMP || f[i] != f[i] ? f[i] : fminf(fmaxf(f[i], -448.f), 448.f);   // a NaN stays one
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(g[0], g[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(g[2], g[3], w, true);
  }
}
template <bool INT8, bool CLAMP>
__device__ __forceinline__ u32x2 codes8(const float* f) {
  return u32x2{codes4<INT8, CLAMP>(f), codes4<INT8, CLAMP>(f + 4)};
}

// Four codes times a power of two up to 1, rounded to nearest even again.
template <bool INT8>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float by) {
  float f[4];
  if (INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i)) * by;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __builtin_amdgcn_cvt_f32_fp8((int)(w >> (8 * i)), 0) * by;
  }
  return codes4<INT8, false>(f);
}

// E8M0 byte of the smallest power of two s with top <= M s, within 1 .. the largest; top
// by its bits.
__device__ __forceinline__ int needed_scale(uint32_t top, bool int8) {
  const uint32_t b = top, m = b & 0x7fffffu;
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
__global__ __launch_bounds__(kThreads) void append_rows_kernel(AppendArgs a, int groups, int per) {
  const CacheView& c = a.cache;
  const int units = c.dim / 16, heads = a.q.heads + 2 * c.heads, group = blockIdx.x % groups;
  const int64_t item = (int64_t)(blockIdx.x / groups) * kThreads + threadIdx.x;
  const int64_t t = item / units;
  if (t >= a.tokens) return;
  const int unit = (int)(item - t * units), h0 = group * per, h1 = min(h0 + per, heads);
  const UnitAt at = unit_at(a.rot.dim, c.dim, unit);
  constexpr int kAtOnce = 4;
  u32x4 lo[kAtOnce], hi[kAtOnce];
  auto load = [&](int i, int head) {
    const int kv = head - a.q.heads;
    const uint16_t* x = kv < 0           ? a.q.x + t * a.q.ld_x + (int64_t)head * c.dim
                        : kv < c.heads ? a.k + t * a.ld_k + (int64_t)kv * c.dim
                                       : a.v + t * a.ld_v + (int64_t)(kv - c.heads) * c.dim;
    lo[i] = *(const u32x4*)(x + at.lo);
    hi[i] = *(const u32x4*)(x + at.hi);
  };
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) load(i, min(h0 + i, h1 - 1));
  Turn<float> turn;
  const bool turns = at.turns && h0 < a.q.heads + c.heads && find_turn<INTERLEAVED>(turn, a.rot, unit, a.rot.positions[t]);
  const int64_t slot = a.slots[t];
  const bool held = slot >= 0 && slot >> c.page_shift < c.num_pages;
  for (int h = h0; h < h1; h += kAtOnce) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int head = h + i, kv = head - a.q.heads;
      if (head >= h1) break;
      u32x4 w[2] = {lo[i], hi[i]};
      if (head + kAtOnce < h1) load(i, head + kAtOnce);
      if (kv >= 0 && !held) continue;
      float f[16];
      unpack(w[0], f);
      unpack(w[1], f + 8);
      if (turns && kv < c.heads) {
        turn_unit<INTERLEAVED>(f, turn);
        if (!FP8 || kv < 0) w[0] = pack(f), w[1] = pack(f + 8);   // else w stays as it is, a NaN's bits too
      }
      if (kv < 0) {
        uint16_t* out = a.q.out + t * a.q.ld_out + (int64_t)head * c.dim;
        *(u32x4*)(out + at.lo) = w[0];
        *(u32x4*)(out + at.hi) = w[1];
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
        *(u32x2*)(p + at.lo) = codes8<false, true>(f);
        *(u32x2*)(p + at.hi) = codes8<false, true>(f + 8);
      } else {
        uint16_t* p = (uint16_t*)(is_v ? c.v : c.k) + to;
        *(u32x4*)(p + at.lo) = w[0];
        *(u32x4*)(p + at.hi) = w[1];
      }
    }
  }
}

namespace {

// Lanes of a run: all 16 places of its block, 16 columns a lane.  One, two or four waves
// are a workgroup, so that a lane's values are few whatever the head (8192 tokens of q, k
// and v, 24/4 heads of 256: one wave in four passes 74 us, here 43; 1000 tokens 58, 17).
constexpr int run_threads(int dim) { return kBlockTokens * dim / 16; }

// Largest of a workgroup's values.  Two turns of `joint`, one barrier: whoever writes a
// turn again has passed the other's barrier, after which no one reads this one.
template <int THREADS>
__device__ __forceinline__ uint32_t max_of(uint32_t x, uint32_t (*joint)[4], int& turn) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d));
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) joint[turn][threadIdx.x >> 6] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) x = max(x, joint[turn][w]);
    turn ^= 1;
  }
  return uniform((int)x);
}

// Rows 16 w .. 16 w + 15 of the call are window w.  This workgroup takes heads [h0, h1) of K
// or V, and of the runs that begin in its window every `shares`-th from `share` on.
template <bool INTERLEAVED, bool INT8, int D>
__device__ __forceinline__ void append_runs(const AppendArgs& a, int64_t window, int share, int shares, int h0, int h1, bool is_v) {
  constexpr int U = D / 16;                 // units, so lanes, of a row
  __shared__ uint32_t joint[2][4];
  int joint_turn = 0;
  const CacheView& c = a.cache;
  const int lane = threadIdx.x & 63, unit = threadIdx.x % U, place = threadIdx.x / U;
  const int64_t t0 = window * kBlockTokens;
  const uint16_t* x = is_v ? a.v : a.k;
  const int64_t ld = is_v ? a.ld_v : a.ld_k;
  uint8_t* cache = (uint8_t*)(is_v ? c.v : c.k);
  uint8_t* scales = is_v ? c.v_blocks : c.k_blocks;
  const UnitAt at = unit_at(is_v ? 0 : a.rot.dim, D, unit);

  // the window's rows that begin a run, and the window after it, where its last may end;
  // every wave finds them for itself
  auto slot_of = [&](int64_t t) {
    if (t < 0 || t >= a.tokens) return (int64_t)-1;
    const int64_t s = a.slots[t];
    return s >= 0 && s >> c.page_shift < c.num_pages ? s : (int64_t)-1;
  };
  const int64_t mine = lane < 2 * kBlockTokens ? slot_of(t0 + lane) : -1;
  const int64_t before = slot_of(t0 - 1), left = __shfl_up(mine, 1), prev = lane ? left : before;
  uint64_t begins = __ballot(lane < kBlockTokens && mine >= 0 && (prev < 0 || prev != mine - 1 || mine % kBlockTokens == 0));
  for (int skip = share; begins; skip = shares - 1) {
    for (; skip > 0 && begins; --skip) begins &= begins - 1;
    if (!begins) break;
    const int first = __builtin_ctzll(begins);
    const int64_t t = t0 + first;
    begins &= begins - 1;
    const int64_t s0 = uniform(__shfl(mine, first)), behind = __shfl(mine, first + lane);
    const int place0 = (int)(s0 % kBlockTokens);
    const bool next = lane < kBlockTokens - place0 && behind == s0 + lane;
    const int place1 = place0 + __builtin_ctzll(~__ballot(next));   // the run: places [place0, place1)
    const bool fresh = place0 == 0, in = place >= place0 && place < place1;
    int64_t block = ((s0 >> c.page_shift) * c.heads + h0) << (c.page_shift - 4) | (s0 & (((int64_t)1 << c.page_shift) - 1)) >> 4;
    uint8_t* to = cache + place_at(c, s0 - place0, h0) + place * c.token_stride;

    // a lane's row: of a place outside the run the run's first, which is not used
    const int64_t from = in ? t + place - place0 : t;
    const uint16_t* row = x + from * ld;
    u32x4 lo = *(const u32x4*)(row + (int64_t)h0 * D + at.lo), hi = *(const u32x4*)(row + (int64_t)h0 * D + at.hi);
    // in fp64: of 16 million codes of rotated keys 0 to 3 are beside the formula's, with fp32's products 14 to 18
    int old = scales[block];
    Turn<double> turn;
    const bool turns = in && at.turns && find_turn<INTERLEAVED>(turn, a.rot, unit, a.rot.positions[from]);
    for (int h = h0; h < h1; ++h, block += (int64_t)1 << (c.page_shift - 4), to += c.head_stride) {
      constexpr int kMost = INT8 ? kMostInt8 : kMostE4m3;
      old = fresh ? 1 : min(max(old, 1), kMost);
      float f[16];
      unpack(lo, f);
      unpack(hi, f + 8);
      if (h + 1 < h1) {
        lo = *(const u32x4*)(row + (int64_t)(h + 1) * D + at.lo);
        hi = *(const u32x4*)(row + (int64_t)(h + 1) * D + at.hi);
      }
      if (turns) turn_unit<INTERLEAVED>(f, turn);
      uint32_t top = 0;                     // largest magnitude's bits: infinities and NaN come last
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
      top = max_of<run_threads(D)>(in ? top : 0, joint, joint_turn);
      const bool odd = top >= 0x7f800000u;   // rare: the largest finite value, and clamped codes
      if (odd) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t m = __float_as_uint(f[i]) & 0x7fffffffu;
          if (m < 0x7f800000u) top = max(top, m);
        }
        top = max_of<run_threads(D)>(in ? top : 0, joint, joint_turn);
      }
      const int e = max(needed_scale(top, INT8), old);
      const bool clamp = odd || e == kMost;   // at the largest scale a value may lie beyond its codes
      const bool rises = !fresh && e > old;
      const float by = __uint_as_float((uint32_t)(254 - e) << 23), shrink = e - old > 126 ? 0.f : __uint_as_float((uint32_t)(127 + old - e) << 23);
      if (in) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] *= by;
        if (clamp) {
          *(u32x2*)(to + at.lo) = codes8<INT8, true>(f);
          *(u32x2*)(to + at.hi) = codes8<INT8, true>(f + 8);
        } else {
          *(u32x2*)(to + at.lo) = codes8<INT8, false>(f);
          *(u32x2*)(to + at.hi) = codes8<INT8, false>(f + 8);
        }
      } else if (fresh) {
        *(u32x4*)(to + unit * 16) = u32x4{0u, 0u, 0u, 0u};
      } else if (rises) {
        u32x4 w = *(const u32x4*)(to + unit * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = rescale4<INT8>(w[i], shrink);
        *(u32x4*)(to + unit * 16) = w;
      }
      if (threadIdx.x == 0) scales[block] = (uint8_t)e;
      if (h + 1 < h1) old = scales[block + ((int64_t)1 << (c.page_shift - 4))];
    }
  }
}

}  // namespace

// The first `kv` workgroups write K and V, the others rotate q.
template <bool INTERLEAVED, bool INT8, int D>
__global__ __launch_bounds__(run_threads(D)) void append_blocks_kernel(AppendArgs a, int shares, int head_groups, int heads, int kv, int q_groups,
                                                                       int q_per) {
  if ((int)blockIdx.x >= kv) {
    rotary_rows<INTERLEAVED, run_threads(D)>(a.q, a.rot, D / 16, blockIdx.x - kv, q_groups, q_per);
    return;
  }
  int id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  const int h0 = id % head_groups * heads;
  id /= head_groups;
  append_runs<INTERLEAVED, INT8, D>(a, id / shares, id % shares, shares, h0, min(h0 + heads, a.cache.heads), is_v);
}

namespace {

template <bool INTERLEAVED, bool INT8, int D>
hipError_t launch_blocks(const AppendArgs& a, hipStream_t st) {
  const CacheView& c = a.cache;
  const int64_t windows = (a.tokens + kBlockTokens - 1) / kBlockTokens;
  // Every row may be a run of its own (single tokens): a workgroup for each of them and
  // for every head while that leaves the chip room; prompts, with one run a window, share
  // a run's angles between heads.
  const int64_t each = windows * c.heads * 2, waves = each * (run_threads(D) / 64);
  const int shares = waves * 16 <= 16384 ? 16 : waves * 4 <= 16384 ? 4 : 1;
  const int heads = (int)std::max<int64_t>(1, std::min<int64_t>(waves / 4096, c.heads)), groups = (c.heads + heads - 1) / heads;
  const int64_t kv = windows * 2 * groups * shares;
  RotaryGrid q{1, 1, 0};
  if (a.q.heads > 0) q = rotary_grid(a.tokens, a.q.heads, D, run_threads(D));
  append_blocks_kernel<INTERLEAVED, INT8, D>
      <<<(unsigned)(kv + q.blocks), run_threads(D), 0, st>>>(a, shares, groups, heads, (int)kv, q.groups, q.per);
  return hipGetLastError();
}
template <bool INTERLEAVED, bool INT8>
hipError_t launch_blocks(const AppendArgs& a, hipStream_t st) {
  return a.cache.dim == 64    ? launch_blocks<INTERLEAVED, INT8, 64>(a, st)
         : a.cache.dim == 128 ? launch_blocks<INTERLEAVED, INT8, 128>(a, st)
                              : launch_blocks<INTERLEAVED, INT8, 256>(a, st);
}

}  // namespace

hipError_t launch_paged_kv_append(const AppendArgs& a, hipStream_t st) {
  const CacheView& c = a.cache;
  const bool inter = a.rot.interleaved;
  if (c.blocks == kBlocksInt8) return inter ? launch_blocks<true, true>(a, st) : launch_blocks<false, true>(a, st);
  if (c.blocks == kBlocksE4m3) return inter ? launch_blocks<true, false>(a, st) : launch_blocks<false, false>(a, st);
  const RotaryGrid g = rotary_grid(a.tokens, a.q.heads + 2 * c.heads, c.dim, kThreads);
  const unsigned grid = (unsigned)g.blocks;
  if (inter) {
    if (c.fp8) append_rows_kernel<true, true><<<grid, kThreads, 0, st>>>(a, g.groups, g.per);
    else append_rows_kernel<true, false><<<grid, kThreads, 0, st>>>(a, g.groups, g.per);
  } else {
    if (c.fp8) append_rows_kernel<false, true><<<grid, kThreads, 0, st>>>(a, g.groups, g.per);
    else append_rows_kernel<false, false><<<grid, kThreads, 0, st>>>(a, g.groups, g.per);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
