// Linear layers in 8-bit integers on gfx950: y = s_m t_n sum_k a_mk w_nk, with a scale for
// each token (s) and each output channel (t).  Declared and documented in include/nvfp4.h.
//
// The products are v_mfma_i32_*_i8: the sums are exact in 32 bits (|a w| <= 2^14 and
// k < 2^17), so no split of k and no order of its parts can change a result.
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "layer8.h"

namespace nvfp4 {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));   // at any address of a float
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2 p;
  p[0] = (__bf16)lo;
  p[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, p);
}

// Largest 15-bit magnitude pattern of eight bf16 values: it rises with |x|, infinities
// and NaN last.
__device__ __forceinline__ uint32_t magnitude(const u32x4& w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, w[i] >> 16 & 0x7fffu));
  return m;
}

// Scale of a row and what its values are multiplied by, from its largest magnitude.
// Rows below 2^-120, whose 127 / amax would leave fp32, count as 0; a row with an
// infinity or NaN has the scale NaN and so a result of NaN.
struct RowScale {
  float scale, by;
};
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  const float top = __uint_as_float(bits << 16);
  if (bits >= 0x7f80u) return RowScale{__uint_as_float(0x7fc00000u), 0.f};
  if (top < 0x1p-120f) return RowScale{0.f, 0.f};
  return RowScale{top / 127.f, 127.f / top};
}

// Eight bf16 values as codes: nearest, ties to even.  |x * by| <= 127 (1 + 2^-23), so
// none needs a clamp.
__device__ __forceinline__ u32x2 codes8(const u32x4& w, float by) {
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t two = w[2 * i + (j >> 1)];
      const float x = __uint_as_float(j & 1 ? two & 0xffff0000u : two << 16);
      // by is 0 for rows of scale 0 or NaN: 0 * inf is no code
      const int q = by == 0.f ? 0 : (int)rintf(x * by);
      word |= ((uint32_t)q & 0xffu) << (8 * j);
    }
    c[i] = word;
  }
  return c;
}

}  // namespace

// ------------------------------------------------------------- quantise ----
//
// A wave or a workgroup a row: its largest magnitude, then its codes.  Bound by HBM: 3
// bytes an element; the row's first HELD x THREADS x 8 values stay in registers between
// the two, the rest is read again from the caches.  4096 rows of 5120: 17.4 - 20 us, 3.1 -
// 3.6 TB/s (14.4 where the rows lie in the last-level cache): 4096 waves are one round of four
// a SIMD, which all read and then all write; they wait 74% of their cycles.
template <int THREADS, int HELD>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void int8_quantize_kernel(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                                            int8_t* codes, float* scales, uint32_t* clear, int clears) {
  // for the product behind
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < clears; i += gridDim.x * blockDim.x) clear[i] = 0;
  constexpr int BLOCK = THREADS < 256 ? 256 : THREADS, ROWS = BLOCK / THREADS;
  __shared__ uint32_t tops[BLOCK / 64];
  const int tid = threadIdx.x % THREADS;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
  if (THREADS < 256 && row >= rows) return;
  const uint16_t* p = x + row * ld;
  const int64_t pieces = cols / 8;
  u32x4 held[HELD];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int64_t at = tid + i * THREADS;
    held[i] = at < pieces ? *(const u32x4*)(p + at * 8) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int i = 0; i < HELD; ++i) top = max(top, magnitude(held[i]));
  for (int64_t at = tid + HELD * THREADS; at < pieces; at += THREADS) top = max(top, magnitude(*(const u32x4*)(p + at * 8)));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if (THREADS > 64) {
    if (tid % 64 == 0) tops[tid / 64] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) top = max(top, tops[w]);
  }
  const RowScale s = row_scale(top);
  int8_t* c = codes + row * cols;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int64_t at = tid + i * THREADS;
    if (at < pieces) *(u32x2*)(c + at * 8) = codes8(held[i], s.by);
  }
  for (int64_t at = tid + HELD * THREADS; at < pieces; at += THREADS)
    *(u32x2*)(c + at * 8) = codes8(*(const u32x4*)(p + at * 8), s.by);
  if (tid == 0) scales[row] = s.scale;
}

namespace {

constexpr int64_t kQuantiseRows = 1 << 23;   // of a launch: with 256 threads a row half of what it counts

hipError_t quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, float* scales, uint32_t* clear,
                    int clears, hipStream_t st) {
  for (; rows > kQuantiseRows; rows -= kQuantiseRows, x += kQuantiseRows * ld, codes += kQuantiseRows * cols, scales += kQuantiseRows, clears = 0) {
    const hipError_t e = quantize(x, kQuantiseRows, cols, ld, codes, scales, clear, clears, st);
    if (e != hipSuccess) return e;
  }
  const unsigned four = (unsigned)((rows + 3) / 4);
  if (rows >= 256 && cols <= 4096)
    int8_quantize_kernel<64, 8><<<four, 256, 0, st>>>(x, rows, cols, ld, codes, scales, clear, clears);
  else if (rows >= 1024 && cols <= 8192)
    int8_quantize_kernel<64, 16><<<four, 256, 0, st>>>(x, rows, cols, ld, codes, scales, clear, clears);
  else if (rows >= 256 || cols <= 2048)
    int8_quantize_kernel<256, 8><<<(unsigned)rows, 256, 0, st>>>(x, rows, cols, ld, codes, scales, clear, clears);
  else
    int8_quantize_kernel<1024, 4><<<(unsigned)rows, 1024, 0, st>>>(x, rows, cols, ld, codes, scales, clear, clears);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, float* scales,
                                hipStream_t st) {
  return quantize(x, rows, cols, ld, codes, scales, nullptr, 0, st);
}

// ---------------------------------------------------------------- tiles ----
//
// Output tile BM tokens x BN channels; k in stages of 128 bytes of every row, which pass
// through LDS several stages deep by direct loads (global_load_lds: no registers, no
// VALU).  Whole lines: with stages of 64 bytes such a load took twice as long (27 bytes a
// clock and CU against 44), and they bounded the kernel.  The waves split the tile into
// MF x NF fragments of 32 x 32 each; a stage is four products of 32 k, and the next
// stages' loads are spread among them.  v_mfma_i32_32x32x32_i8 takes W's rows as its rows
// and the tokens as its columns, so that a lane ends with one token and runs of four
// channels.
//
// 4096 tokens, 17408 x 5120, take 297 - 320 us, 2.3 - 2.45 POP/s, the matrix unit busy for 61 -
// 63% of the cycles at 1.82 GHz.  Bound by how the products are fed: the waves wait 39% of
// their cycles, with two places in LDS and one workgroup a CU, whose start and epilogue
// nothing covers; and less by the power that sets the clock (with codes that are all zero it
// took 306 us where random ones took 337; loads of the next tile before the epilogue changed
// nothing).  777 tokens, 4104 x 2064: 16 - 17 us, 0.8 PFLOP/s, of which
// 7 are the launch, the first stages and the epilogue: 231 tiles of 128 x 128 are one round
// (at other sizes of it a stage is 0.35 us, its loads alone 0.25, its products alone 0.2).
//
// LDS layout of a stage: [rows][128] bytes, the 16-byte pieces of row r permuted by
// (r >> 1) & 7: sixteen lanes that read one piece of sixteen rows meet all banks once.
// The permutation is made by the loads' source addresses.
//
// Rows past m and n repeat the last one (their products are not stored).  A last stage
// that is not full goes through registers, zero-filled, after the others.
namespace {

constexpr int kStageBytes = 128;   // of a row

template <int MF, int NF, int WM, int WN, int STAGES>
struct TileShape {
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int BM = 32 * MF * WM, BN = 32 * NF * WN;
  static constexpr int ROWS = BM + BN;                  // tokens, then channels
  static constexpr int STAGE = ROWS * kStageBytes;
  static constexpr int LOADS = ROWS / 8 / WAVES;        // direct loads of a wave a stage, 8 rows each
  static constexpr int TURN = WAVES * 32 * (32 * NF + 4) * 4;   // the epilogue's bytes
  static constexpr int LDS = STAGES * STAGE > TURN ? STAGES * STAGE : TURN;
  static_assert(ROWS % (8 * WAVES) == 0 && WAVES % 2 == 0 && STAGES >= 2, "");
};

// Global -> LDS copy of 16 bytes a lane: lane l's bytes land at dst + 16 l, read from
// base + voff.  Inline asm, so that the compiler adds no waits of its own before later
// LDS reads; it has no register results.  The s_nop covers the wait states between a
// VALU write of the base and its use.
__device__ __forceinline__ void dma16(const int8_t* base, uint32_t voff, uint8_t* dst) {
  const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)dst;
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(at) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_arrived() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// This wave's LDS reads have arrived.
__device__ __forceinline__ void wait_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Which tile workgroup b of `count` takes.  The hardware deals workgroups to the eight
// XCDs in turn; each gets a contiguous run of the order, which goes through groups of
// eight tile columns row by row, so that the tiles which an XCD holds at once read few
// rows of a and of w through its L2.
constexpr int kXcds = 8, kGroupCols = 8;
__device__ __forceinline__ int xcd_order(int b, int count) {
  const int x = b % kXcds, each = count / kXcds, rest = count % kXcds;
  return x * each + min(x, rest) + b / kXcds;
}
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int t, int tiles_m, int tiles_n) {
  const int group = t / (kGroupCols * tiles_m), in = t - group * kGroupCols * tiles_m;
  const int width = min(kGroupCols, tiles_n - group * kGroupCols);
  return TileAt{in / width, group * kGroupCols + in % width};
}

// Parts of a sum that other workgroups add to: as device-scope atomics, which pass the
// L2 that an XCD keeps for itself.
__device__ __forceinline__ void store_shared(int* p, int x, int y) {
  __hip_atomic_store((uint64_t*)p, (uint64_t)(uint32_t)y << 32 | (uint32_t)x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t load_shared(const int* p) {
  return __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Channels [n0, n0 + BN) of tokens [m0, m0 + BM), stages [begin, end) of k.  With parts
// of k in several workgroups (splits > 1) all of a tile's leave their sums at `part`
// and the one that counts itself last at `arrived` adds them up: whole numbers, whose
// order does not matter.
//
// LINES (k no multiple of 128, so that a stage's part of a row lies in two lines): the
// loads take whole lines all the same.  Line l of a row holds its bytes from 128 l - o on, o
// the row's offset in its first line, and stage s is read from lines s and s + 1, which has
// to be there one stage earlier.  k is a multiple of 16, so rows 32 apart have the same o,
// and a lane's fragments all lie alike.
template <int MF, int NF, int WM, int WN, int STAGES, bool LINES>
__device__ __forceinline__ void int8_tile(const Int8Args& a, int64_t m0, int64_t n0, int begin, int end, int split, int splits,
                                          int* part, uint32_t* arrived, uint8_t* lds) {
  using S = TileShape<MF, NF, WM, WN, STAGES>;
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wave_m = wave / WN, wave_n = wave % WN;
  const int64_t k = a.k;
  const int full = min(end, (int)(k / kStageBytes)) - begin, lines = full + LINES;

  // this wave's loads: 8 rows of the stage each, lane = row * 8 + place of a piece (rows
  // 8 i of waves of one parity have the same permutation)
  const int8_t* base[S::LOADS];
  uint32_t voff[S::LOADS], most[S::LOADS];   // most: of the last line, what lies behind the matrix is its last piece
  const int lane_row = lane >> 3, piece = (lane & 7) ^ ((wave * 4 + (lane_row >> 1)) & 7);
  // the part of a row that a lane of load i begins at
  auto rows_of = [&](int i, int64_t& from, int64_t& last) {
    const int row = (i * S::WAVES + wave) * 8;
    const bool tokens = row < S::BM;
    last = (tokens ? a.m : a.n) - 1;
    from = min(tokens ? m0 + row : n0 + row - S::BM, last);
    return (tokens ? a.a : a.w) + from * k + (int64_t)begin * kStageBytes;
  };
#pragma unroll
  for (int i = 0; i < S::LOADS; ++i) {
    int64_t from, last;
    base[i] = rows_of(i, from, last);
    voff[i] = (uint32_t)(min((int64_t)lane_row, last - from) * k) + piece * 16;
    if constexpr (LINES) {
      const uint32_t offset = (uint32_t)(uintptr_t)(base[i] + voff[i] - piece * 16) % kStageBytes;
      base[i] -= kStageBytes;
      voff[i] += kStageBytes - offset;
      most[i] = (uint32_t)min((last + 1 - from) * k - 16 - (int64_t)(begin + full - 1) * kStageBytes, (int64_t)UINT32_MAX);
    }
  }
  auto slot = [&](int s) { return lds + (uint32_t)s % STAGES * S::STAGE; };
  auto issue_one = [&](int s, int i) {
    const uint32_t at = LINES ? min(voff[i], s == full ? most[i] : UINT32_MAX) : voff[i];
    dma16(base[i] + (int64_t)s * kStageBytes, at, slot(s) + (i * S::WAVES + wave) * 1024);
  };
  auto issue = [&](int s) {
#pragma unroll
    for (int i = 0; i < S::LOADS; ++i) issue_one(s, i);
  };

  // The epilogue's scales, asked for now: behind the products they would be waited for
  // (0.2 - 0.4 us of a tile).
  // A row leaves in wide stores, COLS / 8 lanes each, or a lane a channel.
  constexpr int COLS = 32 * NF, LANES = COLS / 8;
  const int64_t col0 = n0 + wave_n * COLS;
  const bool wide = ((uintptr_t)a.out & 15) == 0 && a.ld_out % (a.out_bf16 ? 8 : 4) == 0 && col0 + COLS <= a.n;
  float a_scale[MF], w_scale = 0.f;
  f32x4 w_scales[2] = {};
#pragma unroll
  for (int i = 0; i < MF; ++i) a_scale[i] = a.a_scale[min(m0 + (wave_m * MF + i) * 32 + c32, a.m - 1)];
  if (wide) {
    w_scales[0] = *(const f32x4_any*)(a.w_scale + col0 + lane % LANES * 8);
    w_scales[1] = *(const f32x4_any*)(a.w_scale + col0 + lane % LANES * 8 + 4);
  } else {
    w_scale = a.w_scale[min(col0 + lane % COLS, a.n - 1)];
  }

  i32x16 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const int lane_at = c32 * kStageBytes + ((h ^ ((c32 >> 1) & 7)) * 16);
  const int a_skew = LINES ? (int)((uintptr_t)a.a / 16 + c32 * (uint32_t)(k / 16)) & 7 : 0;   // o / 16
  const int w_skew = LINES ? (int)((uintptr_t)a.w / 16 + c32 * (uint32_t)(k / 16)) & 7 : 0;
  struct Fragments {
    i32x4 a[MF], w[NF];
  };
  // quarter of the stage whose rows lie in place `stage`, and on from there in place `behind`
  auto read = [&](Fragments& f, const uint8_t* stage, const uint8_t* behind, int quarter) {
    auto lane_of = [&](int skew) {
      if constexpr (!LINES) return stage + (lane_at ^ (quarter * 32));
      const int at = quarter * 2 + h + skew;
      return (at & 8 ? behind : stage) + c32 * kStageBytes + (((at & 7) ^ ((c32 >> 1) & 7)) * 16);
    };
    const uint8_t *pa = lane_of(a_skew), *pw = lane_of(w_skew);
#pragma unroll
    for (int i = 0; i < MF; ++i) f.a[i] = *(const i32x4*)(pa + (wave_m * MF + i) * 32 * kStageBytes);
#pragma unroll
    for (int j = 0; j < NF; ++j) f.w[j] = *(const i32x4*)(pw + (S::BM + (wave_n * NF + j) * 32) * kStageBytes);
  };
  auto multiply = [&](const Fragments& f) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[j], f.a[i], acc[i][j], 0, 0, 0);
  };

  // A quarter of a stage is read while the one before is multiplied.  Before the last of
  // them all have read the whole stage: behind that barrier its place is filled anew, and
  // the next stage, waited for before it, is there for all.
  Fragments f0, f1;
  constexpr int kAhead = STAGES - 2 - LINES;   // places of which nothing has to be there
  if (full > 0) {
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
      if (s < lines) issue(s);
    if (lines >= STAGES) {
#pragma unroll
      for (int i = 0; i < S::LOADS / 2; ++i) issue_one(STAGES - 1, i);
      wait_arrived<kAhead * S::LOADS + S::LOADS / 2>();
    } else {
      wait_arrived<0>();
    }
    stage_barrier();
    read(f0, slot(0), slot(1), 0);
    // products of a quarter with loads `first` .. `last` - 1 of stage `of` spread among them
    auto multiply_and_issue = [&](const Fragments& f, int of, auto first, auto last) {
      constexpr int FIRST = decltype(first)::value, COUNT = decltype(last)::value - FIRST, ALL = MF * NF;
#pragma unroll
      for (int e = 0; e < ALL; ++e) {
        acc[e / NF][e % NF] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[e % NF], f.a[e / NF], acc[e / NF][e % NF], 0, 0, 0);
#pragma unroll
        for (int i = e * COUNT / ALL; i < (e + 1) * COUNT / ALL; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          issue_one(of, FIRST + i);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    constexpr std::integral_constant<int, 0> kNone{};
    constexpr std::integral_constant<int, S::LOADS / 2> kHalf{};
    constexpr std::integral_constant<int, S::LOADS> kAll{};
    int s = 0;
#pragma unroll 1
    for (; s + STAGES < lines; ++s) {
      read(f1, slot(s), slot(s + 1), 1);
      multiply_and_issue(f0, s + STAGES - 1, kHalf, kAll);
      read(f0, slot(s), slot(s + 1), 2);
      multiply(f1);
      read(f1, slot(s), slot(s + 1), 3);
      multiply(f0);
      wait_arrived<kAhead * S::LOADS>();
      wait_read();
      stage_barrier();
      read(f0, slot(s + 1), slot(s + 2), 0);
      multiply_and_issue(f1, s + STAGES, kNone, kHalf);
    }
    if (lines >= STAGES) {
#pragma unroll
      for (int i = S::LOADS / 2; i < S::LOADS; ++i) issue_one(s + STAGES - 1, i);
    }
#pragma unroll 1
    for (; s < full; ++s) {
      read(f1, slot(s), slot(s + 1), 1);
      multiply(f0);
      read(f0, slot(s), slot(s + 1), 2);
      multiply(f1);
      read(f1, slot(s), slot(s + 1), 3);
      multiply(f0);
      wait_arrived<0>();
      stage_barrier();
      if (s + 1 < full) read(f0, slot(s + 1), slot(s + 2), 0);
      multiply(f1);
    }
  }
  if (end > begin + full) {   // the last pieces of the rows, the others 0
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::LOADS; ++i) {
      const bool in = (int64_t)(begin + full) * kStageBytes + piece * 16 < k;
      int64_t from, last;
      const int8_t* row = rows_of(i, from, last) + min((int64_t)lane_row, last - from) * k;
      *(u32x4*)(lds + (i * S::WAVES + wave) * 1024 + lane * 16) =
          in ? *(const u32x4*)(row + (int64_t)full * kStageBytes + piece * 16) : u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();
#pragma unroll
    for (int quarter = 0; quarter < 4; ++quarter) {
      const uint8_t* p = lds + (lane_at ^ (quarter * 32));
#pragma unroll
      for (int i = 0; i < MF; ++i) f0.a[i] = *(const i32x4*)(p + (wave_m * MF + i) * 32 * kStageBytes);
#pragma unroll
      for (int j = 0; j < NF; ++j) f0.w[j] = *(const i32x4*)(p + (S::BM + (wave_n * NF + j) * 32) * kStageBytes);
      multiply(f0);
    }
  }

  if (splits > 1) {
    constexpr int kEach = MF * NF * 16 * 64;   // numbers of a wave
    int* mine = part + ((int64_t)split * S::WAVES + wave) * kEach + 2 * lane;
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int e = 0; e < 16; e += 2) store_shared(mine + ((i * NF + j) * 16 + e) * 64, acc[i][j][e], acc[i][j][e + 1]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the parts have been acknowledged
    __syncthreads();
    uint32_t* last = (uint32_t*)lds;
    if (tid == 0) *last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const bool join = *last == (uint32_t)(splits - 1);
    __syncthreads();
    if (!join) return;
    for (int other = 0; other < splits; ++other) {
      if (other == split) continue;
      const int* theirs = part + ((int64_t)other * S::WAVES + wave) * kEach + 2 * lane;
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const uint64_t v = load_shared(theirs + ((i * NF + j) * 16 + e) * 64);
            acc[i][j][e] += (int)(uint32_t)v;
            acc[i][j][e + 1] += (int)(uint32_t)(v >> 32);
          }
    }
  }

  // Epilogue: a wave turns 32 tokens x 32 NF channels at a time through its own part of
  // LDS (the stages are done with), so that rows leave in whole runs.
  constexpr int LD = COLS + 4;
  float* turn = (float*)lds + wave * 32 * LD;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t row0 = m0 + (wave_m * MF + i) * 32;
    if (row0 >= a.m || col0 >= a.n) break;
    const float s = a_scale[i];
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(turn + c32 * LD + 32 * j + 8 * q + 4 * h) =
            f32x4{(float)acc[i][j][4 * q] * s, (float)acc[i][j][4 * q + 1] * s, (float)acc[i][j][4 * q + 2] * s,
                  (float)acc[i][j][4 * q + 3] * s};
    __builtin_amdgcn_wave_barrier();
    if (wide) {
      const int c = lane % LANES * 8;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 64 / LANES) {
        const int r = r0 + lane / LANES;
        const f32x4 x0 = *(const f32x4*)(turn + r * LD + c) * w_scales[0], x1 = *(const f32x4*)(turn + r * LD + c + 4) * w_scales[1];
        if (row0 + r < a.m) {
          const int64_t at = (row0 + r) * a.ld_out + col0 + c;
          if (a.out_bf16) {
            *(u32x4*)((uint16_t*)a.out + at) =
                u32x4{pack_bf16(x0[0], x0[1]), pack_bf16(x0[2], x0[3]), pack_bf16(x1[0], x1[1]), pack_bf16(x1[2], x1[3])};
          } else {
            *(f32x4*)((float*)a.out + at) = x0;
            *(f32x4*)((float*)a.out + at + 4) = x1;
          }
        }
      }
    } else {
      const int c = lane % COLS;
      const int64_t col = min(col0 + c, a.n - 1);
#pragma unroll 8
      for (int r0 = 0; r0 < 32; r0 += 64 / COLS) {
        const int r = r0 + lane / COLS;
        const float y = turn[r * LD + c] * w_scale;
        if (row0 + r < a.m && col0 + c < a.n) {
          const int64_t at = (row0 + r) * a.ld_out + col;
          if (a.out_bf16)
            ((uint16_t*)a.out)[at] = (uint16_t)pack_bf16(y, 0.f);
          else
            ((float*)a.out)[at] = y;
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

template <int MF, int NF, int WM, int WN, int STAGES, bool LINES>
__global__ __launch_bounds__(64 * WM * WN, 2) void int8_tile_kernel(Int8Args a, int tiles_m, int tiles_n) {
  using S = TileShape<MF, NF, WM, WN, STAGES>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  // the parts of a tile's k lie an XCD's run of tiles apart, so that parts of neighbouring
  // tiles, which read the same rows, meet in one L2
  const int tiles = tiles_m * tiles_n, order = xcd_order(blockIdx.x, tiles * a.splits);
  const int split = order / tiles, tile = order - split * tiles;
  const TileAt at = tile_at(tile, tiles_m, tiles_n);
  const int stages = (int)((a.k + kStageBytes - 1) / kStageBytes);
  const int begin = (int)((int64_t)stages * split / a.splits), end = (int)((int64_t)stages * (split + 1) / a.splits);
  int8_tile<MF, NF, WM, WN, STAGES, LINES>(a, (int64_t)at.m * S::BM, (int64_t)at.n * S::BN, begin, end, split, a.splits,
                                    a.parts + (int64_t)tile * a.splits * S::BM * S::BN, a.arrived + tile, lds);
}

// 256 x 256 tiles, one a CU, and the last ones, which would not fill the chip once more,
// as four of 128 x 128 each.
__global__ __launch_bounds__(512, 2) void int8_large_kernel(Int8Args a, int tiles_m, int tiles_n, int whole) {
  using L = TileShape<4, 2, 2, 4, 2>;
  using Q = TileShape<2, 1, 2, 4, 4>;
  static_assert(L::BM == 2 * Q::BM && L::BN == 2 * Q::BN && L::LDS >= Q::LDS, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[L::LDS];
  const int stages = (int)((a.k + kStageBytes - 1) / kStageBytes);
  const int b = blockIdx.x;
  if (b < whole) {
    const int order = xcd_order(b, whole);
    const TileAt at = tile_at(order, tiles_m, tiles_n);
    int8_tile<4, 2, 2, 4, 2, false>(a, (int64_t)at.m * L::BM, (int64_t)at.n * L::BN, 0, stages, 0, 1, nullptr, nullptr, lds);
  } else {
    const int order = xcd_order(b - whole, (tiles_m * tiles_n - whole) * 4);
    const TileAt at = tile_at(whole + order / 4, tiles_m, tiles_n);
    const int64_t m0 = (int64_t)at.m * L::BM + (order & 1) * Q::BM, n0 = (int64_t)at.n * L::BN + (order >> 1 & 1) * Q::BN;
    if (m0 >= a.m || n0 >= a.n) return;
    int8_tile<2, 1, 2, 4, 4, false>(a, m0, n0, 0, stages, 0, 1, nullptr, nullptr, lds);
  }
}

// --------------------------------------------------------------- stream ----
//
// A few tokens: bound by the weights' bytes, so these go from HBM straight into registers
// as operands of v_mfma_i32_16x16x64_i8, whose rows are 16 channels and whose columns 16
// tokens; the tokens' codes lie in LDS.  A workgroup owns 16 channels, its waves take k in
// parts (stages of 64 bytes of every row, eight of them in flight and eight more asked for)
// and add their sums in LDS.  One token, 17408 x 5120: 19.2 us, 4.7 TB/s.
//
// QUANTISE: every workgroup finds the scales and codes itself while its first weights are
// on their way, which spares a launch; the first one writes them out.
namespace {

constexpr int kStreamCodes = 40960;   // bytes of codes in LDS: with the sums beside them three workgroups a CU
constexpr int kStreamTokens = 16;
constexpr int kQuantiseHeld = 8;      // pieces of eight values a thread holds: up to 16384 values in all

// Bytes from a token's codes to the next one's: sixteen more than k, which moves the tokens
// that a read takes together to different banks.
__host__ __device__ inline int stream_row(int64_t k) { return (int)k + 16; }

}  // namespace

template <int WAVES, bool QUANTISE>
__global__ __launch_bounds__(64 * WAVES) void int8_stream_kernel(Int8Args a, const uint16_t* x, int64_t ld_x, int8_t* codes_out,
                                                                 float* scales_out) {
  constexpr int N = 8, THREADS = 64 * WAVES;
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];   // [m][stream_row(k)]
  __shared__ int part[WAVES][16][17];
  __shared__ float scales[kStreamTokens];
  __shared__ uint32_t tops[kStreamTokens];
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = (int)a.m, k = (int)a.k, row = stream_row(k);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int stages = (k + 63) / 64;
  const int s0 = stages * wave / WAVES, count = stages * (wave + 1) / WAVES - s0, groups = (count + N - 1) / N;
  const int8_t* w = a.w + min(n0 + c16, a.n - 1) * (int64_t)k;
  // stage s0 + u of the rows, clamped to their last pieces: what is no stage of this wave,
  // or lies behind the row's end, is multiplied by 0
  auto at = [&](int u) { return min((s0 + u) * 64 + g * 16, k - 16); };
  auto load = [&](i32x4 (&f)[N], int group) {
#pragma unroll
    for (int u = 0; u < N; ++u) f[u] = *(const i32x4*)(w + at(group * N + u));
  };
  i32x4 even[N], odd[N];
  if (groups > 0) load(even, 0);
  if (groups > 1) load(odd, 1);

  if (QUANTISE) {
    const int pieces = m * k / 8, each = k / 8;
    u32x4 held[kQuantiseHeld];
    uint32_t top = 0;
    if (tid < kStreamTokens) tops[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantiseHeld; ++i) {
      const int p = tid + i * THREADS;
      held[i] = u32x4{0u, 0u, 0u, 0u};
      if (p < pieces) {
        const int t = m == 1 ? 0 : p / each;
        held[i] = *(const u32x4*)(x + t * ld_x + (p - t * each) * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < kQuantiseHeld; ++i) {
      const int p = tid + i * THREADS;
      if (m == 1)
        top = max(top, magnitude(held[i]));
      else if (p < pieces)
        atomicMax(&tops[p / each], magnitude(held[i]));
    }
    if (m == 1) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
      if (lane == 0) atomicMax(&tops[0], top);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantiseHeld; ++i) {
      const int p = tid + i * THREADS;
      if (p >= pieces) break;
      const int t = m == 1 ? 0 : p / each, c = (p - t * each) * 8;
      const u32x2 q = codes8(held[i], row_scale(tops[t]).by);
      *(u32x2*)(codes + t * row + c) = q;
      if (blockIdx.x == 0) *(u32x2*)(codes_out + (int64_t)t * k + c) = q;
    }
    if (tid < m) {
      scales[tid] = row_scale(tops[tid]).scale;
      if (blockIdx.x == 0) scales_out[tid] = scales[tid];
    }
  } else {
    const int each = k / 16;
    for (int p = tid; p < m * each; p += THREADS) {
      const int t = p / each, c = (p - t * each) * 16;
      *(u32x4*)(codes + t * row + c) = *(const u32x4*)(a.a + (int64_t)t * k + c);
    }
    if (tid < m) scales[tid] = a.a_scale[tid];
  }
  __syncthreads();

  const uint8_t* mine = codes + min(c16, m - 1) * row;
  i32x4 acc = {0, 0, 0, 0};
  auto multiply = [&](i32x4 (&f)[N], int group) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int s = group * N + u;
      i32x4 c = *(const i32x4*)(mine + at(s));
      if (s >= count || (s0 + s) * 64 + g * 16 >= k) c = i32x4{0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[u], c, acc, 0, 0, 0);
    }
  };
#pragma unroll 1
  for (int i = 0; i < groups; i += 2) {
    multiply(even, i);
    if (i + 2 < groups) load(even, i + 2);
    if (i + 1 < groups) multiply(odd, i + 1);
    if (i + 3 < groups) load(odd, i + 3);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) part[wave][c16][4 * g + r] = acc[r];
  __syncthreads();
  for (int e = tid; e < m * 16; e += THREADS) {
    const int token = e / 16, c = e % 16;
    if (n0 + c >= a.n) continue;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) sum += part[v][token][c];
    const float y = (float)sum * scales[token] * a.w_scale[n0 + c];
    const int64_t to = token * a.ld_out + n0 + c;
    if (a.out_bf16)
      ((uint16_t*)a.out)[to] = (uint16_t)pack_bf16(y, 0.f);
    else
      ((float*)a.out)[to] = y;
  }
}

namespace {

template <bool QUANTISE>
hipError_t launch_stream(const Int8Args& a, const uint16_t* x, int64_t ld_x, int8_t* codes, float* scales, hipStream_t st) {
  const unsigned grid = (unsigned)((a.n + 15) / 16);
  const size_t lds = (size_t)a.m * stream_row(a.k);
  if (grid >= 1024)
    int8_stream_kernel<4, QUANTISE><<<grid, 256, lds, st>>>(a, x, ld_x, codes, scales);
  else
    int8_stream_kernel<8, QUANTISE><<<grid, 512, lds, st>>>(a, x, ld_x, codes, scales);
  return hipGetLastError();
}

// How a product is computed: by the streaming kernel, or in tiles of which kind and in how
// many parts of k.
enum Int8Kind { kStream, kTiles32, kTiles64, kTiles128, kTiles256, kTilesMany, kTiles64Square };
struct Int8Plan {
  Int8Kind kind;
  int64_t bm, bn, tiles_m, tiles_n;
  int splits;
};
void set_tiles(Int8Plan& p, int64_t m, int64_t n) {
  p.bm = p.kind == kTiles32 ? 32 : p.kind == kTiles64 || p.kind == kTiles64Square ? 64 : p.kind == kTiles256 ? 256 : 128;
  p.bn = p.kind == kTiles32 || p.kind == kTiles64Square ? 64 : p.kind == kTiles256 ? 256 : 128;
  p.tiles_m = (m + p.bm - 1) / p.bm;
  p.tiles_n = (n + p.bn - 1) / p.bn;
}
// The streaming kernel finds the codes too where their values fit its registers (one
// token, 17408 x 5120: 19.2 us, in two launches 21.7).
bool stream_quantises(int64_t m, int64_t k) { return m * k <= 8 * 256 * kQuantiseHeld; }
// It reads no weight twice and has nothing to fill, but every workgroup copies or finds
// all codes (8 tokens, 1024 x 5120: 5.9 us, tiles 10.0; 8 tokens, 17408 x 5120: 24.6, tiles
// 22.6; 2 tokens, 13605 x 12992: 48.9, tiles 41.7).
bool streams(int64_t m, int64_t n, int64_t k) {
  if (n > 1 << 27) return false;   // 16 threads a channel: a launch has no more
  if (n * k > 40000000) return m <= 4 && stream_quantises(m, k);
  return m * k <= kStreamCodes && m <= kStreamTokens;
}

// Tiles: by what their rounds over the chip take, in one unit, as measured with k = 5120: a
// round of 64 x 128 (one a CU) 14, of 128 x 128 21 (two a CU: 40 for both), of 256 x 256 60, of
// which a last round in quarters takes a third.  Of 120 drawn sizes the choice was 1.3% off
// the best on average, 10% at most.
// 200 tokens, 5120 x 5120: 64 x 128 17.9 us, 128 x 128 21.3; 512 tokens: 32.6, 22.5; 1024 tokens:
// 128 x 128 43.2, two a CU 38.5, 256 x 256 42.1; 2048 tokens: two a CU 71.6, 256 x 256 55.8; 713
// tokens, 10312 x 4608: 48.6, 61.8.  Few tiles are split along k (37 tokens, 5120 x 17408, 80
// tiles of 64 x 64: three parts 23.2 us, one 41).
//
// A last round of up to 128 tiles of 256 x 256 goes as quarters: 2048 tokens, k = 5120, beyond a
// full round 16 tiles 103 us (whole 128), 64 106 (126), 128 133 (138), but 144 148 (146) and
// 160 151 (139).
// Fewer than 110 tiles of 64 x 128 go as 64 x 64 ones: 64 of them (256 tokens, 2048 x 5120, two
// parts) 12.9 us, as 64 x 128 in four parts 15.8; 80 (128 tokens, 5120 x 5120) 13.9, in three
// parts 14.5; beyond a CU's tile each 160 (256 tokens, 5120 x 5120) 20.6, 18.2.  Between 110
// and 128 the smaller ones would still be ahead (512 tokens, 2048 x 5120: 14.1, 16.6), and
// over a long k the larger ones, with more parts, are already below 110 (k = 17408: 256 tokens,
// 2048 channels 27.9, 25.6; 128 tokens, 5120 channels 47, 34; but 192 tokens, 4096 channels
// 35.5, 40.3).
Int8Plan plan_int8(int64_t m, int64_t n, int64_t k) {
  Int8Plan p{kStream, 0, 0, 0, 0, 1};
  if (streams(m, n, k)) return p;
  const int64_t cus = 256;
  auto tiles_of = [&](Int8Kind kind) {
    p.kind = kind;
    set_tiles(p, m, n);
    return p.tiles_m * p.tiles_n;
  };
  auto rounds = [](int64_t tiles, int64_t at_once) { return (double)((tiles + at_once - 1) / at_once); };
  if (m <= 32) {
    tiles_of(kTiles32);
  } else if (tiles_of(kTiles64) < 110) {
    tiles_of(kTiles64Square);
  } else {
    const int64_t t64 = tiles_of(kTiles64), t128 = tiles_of(kTiles128), t256 = tiles_of(kTiles256), rest = t256 % cus;
    const double large = t256 > cus && rest <= 128 ? (double)(t256 / cus) + (rest ? 0.35 : 0.) : rounds(t256, cus);
    double cost[4] = {14. * rounds(t64, cus), 21. * rounds(t128, cus), 40. * rounds(t128, 2 * cus), 60. * large};
    const Int8Kind kinds[4] = {kTiles64, kTiles128, kTilesMany, kTiles256};
    if (!one_launch(t64, 512)) cost[0] = HUGE_VAL;
    if (!one_launch(t128, 512)) cost[1] = HUGE_VAL;
    tiles_of(kinds[std::min_element(cost, cost + 4) - cost]);
  }
  if (p.kind == kTiles256) return p;
  const int64_t stages = (k + kStageBytes - 1) / kStageBytes, tiles = p.tiles_m * p.tiles_n;
  int64_t splits = std::min(cus / tiles, stages / 10);
  // Two of these are in a CU, so that a part more pays where the tiles are well below two
  // a CU and k is long: one part and two, 607 tokens, 1069 x 15744 (170 tiles) 33.7 us, 30.6;
  // 300 tokens, 2048 x 16384 (160) 35.8, 29.1; but x 8192 (607 tokens, 1069 channels) 19.9 both,
  // and with 256 tiles (512 tokens, 2048 x 16384) 37.2, 39.5.
  if (p.kind == kTiles64Square && tiles * splits < 200 && splits * 40 < stages) ++splits;
  p.splits = (int)std::max<int64_t>(1, splits);
  return p;
}

size_t arrived_bytes(const Int8Plan& p) { return (size_t)(p.tiles_m * p.tiles_n * 4 + 255) / 256 * 256; }

// Whether to load by lines where a tile kernel can; the first row's line must not begin
// before the matrix.  Tiles of 128 channels gain (200 tokens, 5120 x 5136: 20.2 us, by stages
// 24.2; 777 tokens, 4104 x 4112: 24.9, 27.0; k = 5120 and 4096 17.8 and 22.2), those of 64, whose
// few loads a stage want all the places in flight, do not (20 tokens, 9000 x 4112: 15.6,
// 13.8), and two places are too few for it.
bool whole_lines(const Int8Args& a) { return a.k % kStageBytes && ((uintptr_t)a.a | (uintptr_t)a.w) % kStageBytes == 0; }

template <int MF, int NF, int WM, int WN, int STAGES, bool LINES>
hipError_t launch_tiles(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
  using S = TileShape<MF, NF, WM, WN, STAGES>;
  const unsigned grid = (unsigned)(p.tiles_m * p.tiles_n * a.splits);
  if (!one_launch(p.tiles_m * p.tiles_n * a.splits, S::THREADS)) return hipErrorInvalidConfiguration;
  if (LINES && whole_lines(a))
    int8_tile_kernel<MF, NF, WM, WN, STAGES, LINES><<<grid, S::THREADS, 0, st>>>(a, (int)p.tiles_m, (int)p.tiles_n);
  else
    int8_tile_kernel<MF, NF, WM, WN, STAGES, false><<<grid, S::THREADS, 0, st>>>(a, (int)p.tiles_m, (int)p.tiles_n);
  return hipGetLastError();
}

}  // namespace

size_t int8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m == 0) return 0;
  const Int8Plan p = plan_int8(m, n, k);
  return p.splits == 1 ? 0 : arrived_bytes(p) + (size_t)(p.tiles_m * p.tiles_n * p.splits * p.bm * p.bn) * 4;
}

namespace {

__global__ __launch_bounds__(256) void int8_clear_kernel(uint32_t* p, int count) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < count) p[i] = 0;
}

// The plan with its workspace; `clears` counters have to be 0 before it runs.
Int8Args with_plan(const Int8Args& args, const Int8Plan& p, int* clears) {
  Int8Args a = args;
  a.splits = a.workspace ? p.splits : 1;
  a.arrived = (uint32_t*)a.workspace;
  a.parts = (int*)((uint8_t*)a.workspace + arrived_bytes(p));
  *clears = a.splits > 1 ? (int)(p.tiles_m * p.tiles_n) : 0;
  return a;
}

hipError_t product(const Int8Args& a, const Int8Plan& p, hipStream_t st) {
  switch (p.kind) {
    case kStream: return launch_stream<false>(a, nullptr, 0, nullptr, nullptr, st);
    case kTiles32: return launch_tiles<1, 1, 1, 2, 4, false>(a, p, st);
    case kTiles64: return launch_tiles<1, 1, 2, 4, 4, true>(a, p, st);
    case kTiles64Square: return launch_tiles<1, 1, 2, 2, 4, false>(a, p, st);
    case kTiles128: return launch_tiles<1, 2, 4, 2, 4, true>(a, p, st);
    case kTilesMany: return launch_tiles<2, 2, 2, 2, 2, false>(a, p, st);
    default: {
      // rounds of one tile a CU; the last one in quarters where that is shorter
      const int tiles = (int)(p.tiles_m * p.tiles_n), rest = tiles % 256, whole = rest > 128 || tiles < 256 ? tiles : tiles - rest;
      int8_large_kernel<<<(unsigned)(whole + 4 * (tiles - whole)), 512, 0, st>>>(a, (int)p.tiles_m, (int)p.tiles_n, whole);
      return hipGetLastError();
    }
  }
}

}  // namespace

hipError_t launch_gemm_w8a8(const Int8Args& args, hipStream_t st) {
  const Int8Plan p = plan_int8(args.m, args.n, args.k);
  int clears;
  const Int8Args a = with_plan(args, p, &clears);
  if (clears) {
    int8_clear_kernel<<<(unsigned)((clears + 255) / 256), 256, 0, st>>>(a.arrived, clears);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return product(a, p, st);
}

hipError_t launch_int8_linear(const uint16_t* x, int64_t ld_x, int8_t* codes, float* scales, const Int8Args& args, hipStream_t st) {
  const Int8Plan p = plan_int8(args.m, args.n, args.k);
  if (p.kind == kStream && stream_quantises(args.m, args.k)) return launch_stream<true>(args, x, ld_x, codes, scales, st);
  int clears;
  const Int8Args a = with_plan(args, p, &clears);
  const hipError_t e = quantize(x, a.m, a.k, ld_x, codes, scales, a.arrived, clears, st);
  return e != hipSuccess ? e : product(a, p, st);
}

}  // namespace nvfp4
