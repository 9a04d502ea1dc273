// Linear layers in 8-bit integers on gfx950: y = s_m t_n sum_k a_mk w_nk, with a scale for
// each token (s) and each output channel (t).  Declared and documented in include/nvfp4.h.
//
// The products are v_mfma_i32_*_i8: the sums are exact in 32 bits (|a w| <= 2^14 and
// k < 2^17), so no split of k and no order of its parts can change a result.
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>

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
// bytes an element; the row's first kHeld x THREADS x 8 values stay in registers between
// the two, the rest (rows beyond 16384) is read again from the caches.
template <int THREADS>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                                            int8_t* codes, float* scales) {
  constexpr int kHeld = 8, ROWS = 256 / THREADS;
  __shared__ uint32_t tops[4];
  const int tid = threadIdx.x % THREADS;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
  if (THREADS < 256 && row >= rows) return;
  const uint16_t* p = x + row * ld;
  const int64_t pieces = cols / 8;
  u32x4 held[kHeld];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t at = tid + i * THREADS;
    held[i] = at < pieces ? *(const u32x4*)(p + at * 8) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) top = max(top, magnitude(held[i]));
  for (int64_t at = tid + kHeld * THREADS; at < pieces; at += THREADS) top = max(top, magnitude(*(const u32x4*)(p + at * 8)));
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
  for (int i = 0; i < kHeld; ++i) {
    const int64_t at = tid + i * THREADS;
    if (at < pieces) *(u32x2*)(c + at * 8) = codes8(held[i], s.by);
  }
  for (int64_t at = tid + kHeld * THREADS; at < pieces; at += THREADS)
    *(u32x2*)(c + at * 8) = codes8(*(const u32x4*)(p + at * 8), s.by);
  if (tid == 0) scales[row] = s.scale;
}

hipError_t launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, float* scales,
                                hipStream_t st) {
  if (cols <= 4096 && rows >= 1024)
    int8_quantize_kernel<64><<<(unsigned)((rows + 3) / 4), 256, 0, st>>>(x, rows, cols, ld, codes, scales);
  else
    int8_quantize_kernel<256><<<(unsigned)rows, 256, 0, st>>>(x, rows, cols, ld, codes, scales);
  return hipGetLastError();
}

// ---------------------------------------------------------------- tiles ----
//
// Output tile BM tokens x BN channels; k in stages of 64 bytes of every row, which pass
// through LDS four stages deep by direct loads (global_load_lds: no registers, no VALU).
// The waves split the tile into MF x NF fragments of 32 x 32 each; a stage is two
// products of 32 k.  v_mfma_i32_32x32x32_i8 takes W's rows as its rows and the tokens as
// its columns, so that a lane ends with one token and runs of four channels.
//
// LDS layout of a stage: [rows][64] bytes, the 16-byte pieces of row r permuted by
// (r >> 2) & 3: sixteen lanes that read one piece of sixteen rows meet all banks once.
// The permutation is made by the loads' source addresses.
//
// Rows past m and n repeat the last one (their products are not stored).  A last stage
// that is not full goes through registers, zero-filled, after the others.
namespace {

constexpr int kStageBytes = 64;   // of a row
constexpr int kStages = 4;

template <int MF, int NF, int WM, int WN>
struct TileShape {
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int BM = 32 * MF * WM, BN = 32 * NF * WN;
  static constexpr int ROWS = BM + BN;                  // tokens, then channels
  static constexpr int STAGE = ROWS * kStageBytes;
  static constexpr int LOADS = ROWS / 16 / WAVES;       // direct loads of a wave a stage, 16 rows each
  static_assert(ROWS % (16 * WAVES) == 0, "");
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
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace

template <int MF, int NF, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void int8_tile_kernel(Int8Args a, int tiles_m, int tiles_n) {
  using S = TileShape<MF, NF, WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages][S::STAGE];
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wave_m = wave / WN, wave_n = wave % WN;
  const int tile = blockIdx.x;
  const int bm = tile % tiles_m, bn = tile / tiles_m;
  const int64_t m0 = (int64_t)bm * S::BM, n0 = (int64_t)bn * S::BN;
  const int64_t k = a.k;
  const int full = (int)(k / kStageBytes);

  // this wave's loads: 16 rows of the stage each, lane = row * 4 + place of a piece
  const int8_t* base[S::LOADS];
  uint32_t voff[S::LOADS];
  const int lane_row = lane >> 2, piece = (lane & 3) ^ ((lane_row >> 2) & 3);
#pragma unroll
  for (int i = 0; i < S::LOADS; ++i) {
    const int row = (i * S::WAVES + wave) * 16;
    const bool tokens = row < S::BM;
    const int64_t first = tokens ? m0 + row : n0 + row - S::BM, last = (tokens ? a.m : a.n) - 1;
    const int64_t from = min(first, last);
    base[i] = (tokens ? a.a : a.w) + from * k;
    voff[i] = (uint32_t)(min((int64_t)lane_row, last - from) * k) + piece * 16;
  }
  auto issue = [&](int stage) {
#pragma unroll
    for (int i = 0; i < S::LOADS; ++i)
      dma16(base[i] + (int64_t)stage * kStageBytes, voff[i], lds[stage % kStages] + (i * S::WAVES + wave) * 1024);
  };

  i32x16 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const int lane_at = c32 * kStageBytes + ((h ^ ((c32 >> 2) & 3)) * 16);
  struct Fragments {
    i32x4 a[MF], w[NF];
  };
  auto read = [&](Fragments& f, const uint8_t* stage, int half) {
    const uint8_t* p = stage + (lane_at ^ (half * 32));
#pragma unroll
    for (int i = 0; i < MF; ++i) f.a[i] = *(const i32x4*)(p + (wave_m * MF + i) * 32 * kStageBytes);
#pragma unroll
    for (int j = 0; j < NF; ++j) f.w[j] = *(const i32x4*)(p + (S::BM + (wave_n * NF + j) * 32) * kStageBytes);
  };
  auto multiply = [&](const Fragments& f) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[j], f.a[i], acc[i][j], 0, 0, 0);
  };

  // Half 0 of a stage is read while half 1 of the stage before is multiplied, and half 1
  // while half 0 is; the stage that three stages on will be needed is asked for behind the
  // barrier, when all have read the one whose place it takes.
  Fragments f0, f1;
  if (full > 0) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
      if (s < full) issue(s);
    if (full >= kStages - 1) wait_arrived<(kStages - 2) * S::LOADS>(); else wait_arrived<0>();
    stage_barrier();
    read(f0, lds[0], 0);
#pragma unroll 1
    for (int s = 0; s < full; ++s) {
      read(f1, lds[s % kStages], 1);
      multiply(f0);
      if (s + kStages - 1 < full) {
        wait_arrived<(kStages - 3) * S::LOADS>();
      } else {
        wait_arrived<0>();
      }
      stage_barrier();
      if (s + kStages - 1 < full) issue(s + kStages - 1);
      if (s + 1 < full) read(f0, lds[(s + 1) % kStages], 0);
      multiply(f1);
    }
  }
  if (k % kStageBytes) {   // the last pieces of the rows, the others 0
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::LOADS; ++i) {
      const bool in = (int64_t)full * kStageBytes + piece * 16 < k;
      *(u32x4*)(lds[0] + (i * S::WAVES + wave) * 1024 + lane * 16) =
          in ? *(const u32x4*)(base[i] + (int64_t)full * kStageBytes + voff[i]) : u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      read(f0, lds[0], half);
      multiply(f0);
    }
  }

  // Epilogue: a wave turns 32 tokens x 32 NF channels at a time through its own part of
  // LDS (the stages are done with), so that rows leave in whole runs.
  constexpr int COLS = 32 * NF, LD = COLS + 4;
  static_assert(S::WAVES * 32 * LD * 4 <= kStages * S::STAGE, "");
  float* turn = (float*)&lds[0][0] + wave * 32 * LD;
  __syncthreads();
  const int64_t col0 = n0 + wave_n * COLS;
  const bool wide = a.out_bf16 ? a.ld_out % 8 == 0 && ((uintptr_t)a.out & 15) == 0 : a.ld_out % 4 == 0 && ((uintptr_t)a.out & 15) == 0;
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t row0 = m0 + (wave_m * MF + i) * 32;
    const float s = row0 + c32 < a.m ? a.a_scale[row0 + c32] : 0.f;
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(turn + c32 * LD + 32 * j + 8 * q + 4 * h) =
            f32x4{(float)acc[i][j][4 * q] * s, (float)acc[i][j][4 * q + 1] * s, (float)acc[i][j][4 * q + 2] * s,
                  (float)acc[i][j][4 * q + 3] * s};
    __builtin_amdgcn_wave_barrier();
    if (wide && col0 + COLS <= a.n) {
      constexpr int LANES = COLS / 8;          // lanes of a row, eight channels each
      const int c = lane % LANES * 8;
      const f32x4 t0 = *(const f32x4_any*)(a.w_scale + col0 + c), t1 = *(const f32x4_any*)(a.w_scale + col0 + c + 4);
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 64 / LANES) {
        const int r = r0 + lane / LANES;
        const f32x4 x0 = *(const f32x4*)(turn + r * LD + c) * t0, x1 = *(const f32x4*)(turn + r * LD + c + 4) * t1;
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
      for (int e = lane; e < 32 * COLS; e += 64) {
        const int r = e / COLS, c = e % COLS;
        if (row0 + r >= a.m || col0 + c >= a.n) continue;
        const float y = turn[r * LD + c] * a.w_scale[col0 + c];
        const int64_t at = (row0 + r) * a.ld_out + col0 + c;
        if (a.out_bf16)
          ((uint16_t*)a.out)[at] = (uint16_t)pack_bf16(y, 0.f);
        else
          ((float*)a.out)[at] = y;
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

namespace {

template <int MF, int NF, int WM, int WN>
hipError_t launch_tiles(const Int8Args& a, hipStream_t st) {
  using S = TileShape<MF, NF, WM, WN>;
  const int64_t tm = (a.m + S::BM - 1) / S::BM, tn = (a.n + S::BN - 1) / S::BN;
  int8_tile_kernel<MF, NF, WM, WN><<<(unsigned)(tm * tn), S::THREADS, 0, st>>>(a, (int)tm, (int)tn);
  return hipGetLastError();
}

}  // namespace

// --------------------------------------------------------------- stream ----
//
// Few tokens (up to 64): bound by the weights' bytes, so these go from HBM straight into
// registers as operands of v_mfma_i32_16x16x64_i8, whose rows are 16 channels and whose
// columns 16 tokens.  A workgroup owns 16 channels, its waves take k in parts (stages of 64
// bytes of every row) and add their sums in LDS.
namespace {

constexpr int kStreamTokens = 64;

}  // namespace

template <int MF, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void int8_stream_kernel(Int8Args a) {
  constexpr int kAtOnce = MF == 1 ? 8 : 4;   // stages in flight
  __shared__ int part[WAVES][MF][16][17];
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16, k = a.k;
  const int stages = (int)((k + 63) / 64);
  const int s0 = stages * wave / WAVES, s1 = stages * (wave + 1) / WAVES;
  const int8_t* w = a.w + min(n0 + c16, a.n - 1) * k + g * 16;
  const int8_t* x[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) x[i] = a.a + min((int64_t)(i * 16 + c16), a.m - 1) * k + g * 16;
  i32x4 acc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) acc[i] = i32x4{0, 0, 0, 0};
  const int whole = k % 64 ? min(s1, stages - 1) : s1;   // stages of all 64 bytes
  int s = s0;
  auto step = [&](auto count) {
    constexpr int N = decltype(count)::value;
    i32x4 wf[N], xf[MF][N];
#pragma unroll
    for (int u = 0; u < N; ++u) wf[u] = *(const i32x4*)(w + (int64_t)(s + u) * 64);
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i) xf[i][u] = *(const i32x4*)(x[i] + (int64_t)(s + u) * 64);
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[u], xf[i][u], acc[i], 0, 0, 0);
    s += N;
  };
  while (s + kAtOnce <= whole) step(std::integral_constant<int, kAtOnce>{});
  while (s < whole) step(std::integral_constant<int, 1>{});
  if (s < s1) {   // the last stage of rows that end inside one
    const bool in = (int64_t)s * 64 + g * 16 < k;
    const i32x4 zero = {0, 0, 0, 0}, wf = in ? *(const i32x4*)(w + (int64_t)s * 64) : zero;
#pragma unroll
    for (int i = 0; i < MF; ++i)
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, in ? *(const i32x4*)(x[i] + (int64_t)s * 64) : zero, acc[i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][i][c16][4 * g + r] = acc[i][r];
  __syncthreads();
  for (int e = tid; e < MF * 256; e += 64 * WAVES) {
    const int token = e / 16, c = e % 16;
    if (token >= a.m || n0 + c >= a.n) continue;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) sum += part[v][token / 16][token % 16][c];
    const float y = (float)sum * a.a_scale[token] * a.w_scale[n0 + c];
    const int64_t at = token * a.ld_out + n0 + c;
    if (a.out_bf16)
      ((uint16_t*)a.out)[at] = (uint16_t)pack_bf16(y, 0.f);
    else
      ((float*)a.out)[at] = y;
  }
}

namespace {

template <int MF>
hipError_t launch_stream(const Int8Args& a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.n + 15) / 16);
  if (grid >= 1024)
    int8_stream_kernel<MF, 4><<<grid, 256, 0, st>>>(a);
  else
    int8_stream_kernel<MF, 8><<<grid, 512, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w8a8(const Int8Args& a, hipStream_t st) {
  if (a.m <= kStreamTokens) {
    switch ((a.m + 15) / 16) {
      case 1: return launch_stream<1>(a, st);
      case 2: return launch_stream<2>(a, st);
      case 3: return launch_stream<3>(a, st);
      default: return launch_stream<4>(a, st);
    }
  }
  // a tile of 256 x 256 reads half of what four of 128 x 128 read, where there are enough
  const int64_t large = ((a.m + 255) / 256) * ((a.n + 255) / 256);
  return large >= 256 ? launch_tiles<4, 2, 2, 4>(a, st) : launch_tiles<2, 2, 2, 2>(a, st);
}

}  // namespace nvfp4
