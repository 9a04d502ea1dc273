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
// for heads of 256), four tiles of each, brought by direct loads that are two
// tiles ahead.  A wave reads every key of a tile from LDS once for its 32 rows: 128
// bytes a clock of the LDS' 256, which is why waves have 32 rows and not 16.
// An E4M3 cache becomes bf16 on its way into LDS, once for all eight waves.
//
// Bound by the matrix unit and the power it may draw: a long prompt holds 1.8 -
// 2.05 GHz, and the MFMAs take 60% of the cycles; the rest is the softmax, whose
// exponentials share the issue slots.  8192 tokens after 8192, 40 heads of 128 over
// 8: 1690 - 1830 us on different cards, 1.13 - 1.22 PFLOP/s (a large bf16 product
// reaches 1.61); heads of 64 (64 over 16) 1770 - 1840 us, 900 - 930 TFLOP/s: half the
// product for each exponential; 4096 after 4096, 24 heads of 256 over 4: 595 - 620 us,
// 1.0 PFLOP/s.  Over E4M3, on a card where these took 1765, 1797 and 605: 1885, 1807
// and 669; a third of the LDS' cycles go into the converted tiles' stores, whose bank
// conflicts take a sixth of all, and the matrix unit is busy for 48% of the cycles in
// place of 60% (heads of 256: 39%, 49%).  8 windowed chunks of up to 777, heads of 64,
// take 82 us, over E4M3 85: 1.4 us a tile of keys, shares between 57 and 80 us long, and
// a part's 8 us beside its keys (its queries, page numbers and first keys; its output).
#include <float.h>
#include <math.h>

#include "attention.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 64 * kChunkWaves;
constexpr int kExtraKeys = 512;
constexpr int kSlots = 4;    // tiles in LDS: tile j lies in slot j % 4

// LDS layout of a tile: [keys][D] bf16, the 16-byte pieces of a row permuted so
// that the lanes of one read instruction meet different banks: keys are read as
// 16 bytes of 32 rows, values as 64 bytes of 4 rows (the transposing read).
template <int D>
__device__ __forceinline__ int key_swizzle(int row) {
  return D == 64 ? (row >> 1) & 7 : row & 15;
}
template <int D>
__device__ __forceinline__ int value_swizzle(int row) {
  return (D == 64 ? (row >> 1) & 1 : row & 3) << 2;
}

// 4 keys x 16 columns a group of 16 lanes; a lane gets the keys of its column.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  typedef __attribute__((address_space(3))) bf16x4* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_ptr)(uintptr_t)p));
}

// Global -> LDS copy of 16 bytes a lane: lane l's bytes land at dst + 16 l, read
// from base + voff (a uniform base and 32-bit lane offsets).  In inline asm, so
// that the compiler adds no waits of its own before later LDS reads; arrival is
// waited for with wait_arrived and published with the barrier.  It has no register
// results.  The s_nop covers five wait states between a VALU write of the base
// (or of M0) and its use.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t voff, uint8_t* dst) {
  const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)dst;
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(at) : "memory");
}
// All but the last N vector memory instructions have arrived.
template <int N>
__device__ __forceinline__ void wait_arrived() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// A barrier that nothing is moved across; WRITES: after this wave's LDS writes.
template <bool WRITES>
__device__ __forceinline__ void phase_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  if (WRITES)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else
    asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The work of all row tiles and KV heads forms one line that a fixed grid shares
// evenly.  A row tile's length on it is the keys that its last row may see, in
// units of 1 / group keys, and `extra`, what a tile costs beside and what a cut is
// worth (512 keys; 256 to 1536 measured the same within 5%, 1 up to 60% slower);
// it grows by 256 from a request's tile to the next until the window ends it, so a
// request's length has a closed form.  A cut between two shares that falls less
// than `extra` from a tile's end or start is moved there.
struct ChunkLine {
  int tiles, rising;
  int64_t context, cap, extra;
};
__device__ __forceinline__ ChunkLine chunk_line(const AttentionArgs& a, const RequestLens& l) {
  ChunkLine c;
  const int rows = l.tokens * a.group;
  c.tiles = rows > a.stream_rows ? (rows + kChunkRows - 1) / kChunkRows : 0;
  c.context = (int64_t)max(l.pos0, 0) * a.group;
  c.cap = a.window ? (int64_t)a.window * a.group + kChunkRows : INT64_MAX / 4;
  c.extra = (int64_t)kExtraKeys * a.group;
  c.rising = (int)min(max((c.cap - c.context) >> 8, (int64_t)0), (int64_t)c.tiles);
  return c;
}
static_assert(kChunkRows == 256, "");
__device__ __forceinline__ int64_t line_length(const ChunkLine& c, int b) {
  return min(c.context + (int64_t)(b + 1) * kChunkRows, c.cap) + c.extra;
}
__device__ __forceinline__ int64_t line_before(const ChunkLine& c, int b) {   // the tiles before tile b
  const int k = min(b, c.rising);
  return k * (c.context + c.extra) + (int64_t)(kChunkRows / 2) * k * (k + 1) + (b > k ? (b - k) * (c.cap + c.extra) : 0);
}

struct ChunkWorkspace {
  int64_t* prefix;   // [requests + 1]: length before a request (of one head); then a workgroup's share
  float2* ml;        // [2 * grid][kChunkRows]: a workgroup's part that begins inside a tile, and that begins with one
  float* o;          // [2 * grid][kChunkRows][dim]
};
__host__ __device__ inline ChunkWorkspace chunk_workspace(void* ws, int64_t requests) {
  ChunkWorkspace w;
  w.prefix = (int64_t*)ws;
  uint8_t* p = (uint8_t*)ws + ((requests + 2) * 8 + 255) / 256 * 256;
  w.ml = (float2*)p;
  w.o = (float*)(p + (size_t)2 * kChunkGrid * kChunkRows * sizeof(float2));
  return w;
}

// Row tiles can also be numbered without a prefix sum: request r's start at
// floor(q_start[r] G / 256) + r, which leaves room for all of them and
// sometimes a number that stands for none.
int64_t row_tiles(int64_t tokens, int64_t requests, int group) { return tokens * group / kChunkRows + requests; }
struct RowTile {
  int r, b;   // request and its row tile
};
__device__ __forceinline__ RowTile row_tile(const AttentionArgs& a, int number) {
  int lo = 0, hi = (int)a.requests - 1;
  auto start = [&](int r) { return (int)((int64_t)a.q_start[r] * a.group >> 8) + r; };
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start(mid) <= number) lo = mid; else hi = mid - 1;
  }
  return RowTile{lo, number - start(lo)};
}

}  // namespace

template <int D, bool FP8>
__global__ __launch_bounds__(kThreads, 2) void attention_chunk_kernel(AttentionArgs a, ChunkWorkspace ws, int numbers) {
  constexpr int KT = D == 256 ? 32 : 64;      // keys of a tile
  constexpr int NK = KT / 32;                 // key fragments of a tile
  constexpr int NG = KT / 16;                 // 16-key groups: a page holds whole ones
  constexpr int KS = D / 16;                  // k steps of the first product
  constexpr int DF = D / 32;                  // fragments of O
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int ROW = D * 2;                  // bytes of an LDS row
  constexpr int PPR = D * EB / 16;            // 16-byte pieces of a row in the cache
  constexpr int RPI = 64 / PPR;               // rows that one load instruction of a wave brings
  constexpr int LOADS = KT / RPI / kChunkWaves;   // such instructions a wave issues for K (and for V)
  constexpr bool SPARE = LOADS == 0;          // heads of 64 in FP8: half of the waves bring a tile
  constexpr int NL = SPARE ? 1 : LOADS;
  // Softmax beside the matrix unit.  Heads of 64 and 128: the two waves of a SIMD take
  // turns, one multiplies while the other computes weights (a prompt of 8192 over 8192
  // keys, 40 heads of 128: 1840 us; mixed 1930 - 2080).  Heads of 256, whose O leaves a
  // wave no registers for operands of two products at once: every wave weighs between
  // the matrix instructions (4096 over 4096, 24 heads: 605 us, E4M3 669; turns 1336 and
  // 1585, with 65 registers spilled).
  constexpr bool MIXED = D == 256;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_k[kSlots][KT * ROW], lds_v[kSlots][KT * ROW];

  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hkv = a.cache.heads, group = a.group;

  if (a.clear_padding) clear_padding(a, a.q_start[a.requests]);

  // prefix of the line over runs of requests
  __shared__ int64_t before[kThreads + 1];
  __shared__ int64_t wave_sum[kChunkWaves];
  const int requests = (int)a.requests, run = (requests + kThreads - 1) / kThreads;
  const int place = blockIdx.x % 8 * (kChunkGrid / 8) + blockIdx.x / 8;
  int64_t x_begin = 0, x_end = 1, per_head = 0;
  if (numbers == 0) {
    const int r0 = min(tid * run, requests), r1 = min(r0 + run, requests);
    int64_t own = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      const ChunkLine cl = chunk_line(a, request_lens(a, r));
      own += line_before(cl, cl.tiles);
    }
    int64_t inc = own;
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t u = __shfl_up(inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < wave; ++w) inc += wave_sum[w];
    if (tid == 0) before[0] = 0;
    before[tid + 1] = inc;
    __syncthreads();
    per_head = uniform(before[kThreads]);
    // Workgroups take their shares XCD by XCD, so that those of an XCD, which have one
    // L2, read the same heads' keys.
    const int64_t share = uniform(max((per_head * hkv + kChunkGrid - 1) / kChunkGrid, (int64_t)kExtraKeys * group));
    if (place == 0) {
      int64_t t = inc - own;
#pragma unroll 1
      for (int r = r0; r < r1; ++r) {
        ws.prefix[r] = t;
        const ChunkLine cl = chunk_line(a, request_lens(a, r));
        t += line_before(cl, cl.tiles);
      }
      if (tid == 0) {
        ws.prefix[requests] = per_head;
        ws.prefix[requests + 1] = share;
      }
    }
    x_begin = place * share;
    x_end = uniform(min(x_begin + share, per_head * hkv));
  }

  __shared__ int not_finite[kChunkWaves];   // the wave took infinities or NaN out of values of the row tile

  for (int64_t x = x_begin; x < x_end;) {
  // the head, request and row tile, and the part of its keys
  int head, r, b, part = 0;
  bool whole = true;
  double share_from = 0., share_to = 1.;
  RequestLens l;
  if (numbers) {              // a row tile a workgroup, long tiles of a prompt first
    head = blockIdx.x % hkv;
    const RowTile t = row_tile(a, numbers - 1 - (int)blockIdx.x / hkv);
    r = uniform(t.r), b = uniform(t.b);
    l = request_lens(a, r);
    if (l.tokens * group <= a.stream_rows || b < 0 || b * kChunkRows >= l.tokens * group) return;
    x = x_end;
  } else {                    // a share of the line
    head = 0;
#pragma unroll 1
    for (int step = 1 << (31 - __builtin_clz(hkv)); step > 0; step >>= 1)
      if (head + step < hkv && (head + step) * per_head <= x) head += step;
    const int64_t y = uniform(x - head * per_head);
    int at = 0;
#pragma unroll 1
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (before[at + step] <= y) at += step;
    r = uniform(at * run);
    int64_t base = before[at];
    l = request_lens(a, r);
    ChunkLine line = chunk_line(a, l);
#pragma unroll 1
    while (y >= base + line_before(line, line.tiles)) {   // ends: y < before[at + 1]
      base += line_before(line, line.tiles);
      l = request_lens(a, ++r);
      line = chunk_line(a, l);
    }
    r = uniform(r);
    b = 0;                                                // the last tile that begins at or before y
    int b_end = line.tiles;
#pragma unroll 1
    while (b_end - b > 1) {
      const int mid = (b + b_end) >> 1;
      if (base + line_before(line, mid) <= y) b = mid; else b_end = mid;
    }
    b = uniform(b);
    const int64_t length = line_length(line, b), offset = y - base - line_before(line, b);
    int64_t from = offset, to = min(from + (x_end - x), length);
    if (x == x_begin) from = from < line.extra ? 0 : length - from < line.extra ? length : from;
    to = to < line.extra ? 0 : length - to < line.extra ? length : to;
    x = uniform(x + length - offset);                     // the next tile begins there
    if (from >= to) continue;
    whole = uniform((int)(to - from == length));
    part = from == 0;                                     // at most one part begins with its tile, and one inside
    share_from = (double)from / (double)length;           // the same on both sides of a cut
    share_to = to == length ? 1. : (double)to / (double)length;
  }
  __syncthreads();   // what the row tile before left in LDS has been read
  if (lane == 0) not_finite[wave] = 0;
  l.start = uniform(l.start), l.tokens = uniform(l.tokens), l.keys = uniform(l.keys), l.pos0 = uniform(l.pos0);

  const int nrows = l.tokens * group;
  const int row0 = b * kChunkRows, row_end = min(row0 + kChunkRows, nrows);
  const int pos_first = l.pos0 + div_group(a, row0), pos_last = l.pos0 + div_group(a, row_end - 1);
  const int keys = min(l.keys, max(pos_last, -1) + 1), low = low_of(a, pos_first);
  const int begin = low & ~(KT - 1), all = max(keys - begin + KT - 1, 0) / KT;
  const int t_begin = uniform((int)(all * share_from)), n = uniform((int)(all * share_to) - t_begin);

  float c = a.scale * kLog2e;
  if (a.cache.k_scale) c *= a.cache.k_scale[head];
  const uint32_t flip = c < 0.f ? 0x80008000u : 0u, spoil = c == c ? 0u : 0x7fff7fffu;   // a NaN scale goes into q
  c = fmaxf(fabsf(c), FLT_MIN);   // never 0: a hidden score's -inf stays one

  // this lane's row of q, the B operand: column c32, k = 8 columns of q
  const int my_row = row0 + wave * 32 + c32;
  const bool live = my_row < nrows;
  const int my_token = live ? div_group(a, my_row) : 0;
  const int my_head = head * group + (live ? my_row - my_token * group : 0);
  bf16x8 q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    u32x4 w = *(const u32x4*)(a.q + (int64_t)(l.start + my_token) * a.ld_q + my_head * D + s * 16 + h * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = live ? (w[i] ^ flip) | spoil : 0u;
    q[s] = __builtin_bit_cast(bf16x8, w);
  }
  // positions relative to the first key of the part
  const int origin = uniform(begin + t_begin * KT);
  const int my_pos = live ? max(l.pos0 + my_token, -1) - origin : INT32_MIN / 2, my_low = low_of(a, l.pos0 + my_token) - origin;
  const int wave_row = min(row0 + wave * 32, nrows - 1);
  const int wave_pos = uniform(max(l.pos0 + div_group(a, wave_row), -1) - origin);   // keys up to it are seen by all rows
  const int wave_low = uniform(low_of(a, l.pos0 + div_group(a, min(wave_row + 31, nrows - 1))) - origin);
  const int keys_rel = uniform(keys - origin), low_rel = uniform(low - origin);

  // Where the keys lie.  A missing page is looked for once in the part's whole
  // table: only if there is one do tiles look again.
  const int page_shift = a.cache.page_shift, page_mask = (1 << page_shift) - 1;
  const uint32_t num_pages = (uint32_t)a.cache.num_pages;
  const int32_t* table = a.block_table + (int64_t)r * a.ld_table;
  auto page_at = [&](int key) { return (uint32_t)table[(uint32_t)(origin + min(key, keys_rel - 1)) >> page_shift]; };
  bool missing = false;
  if (n > 0) {
    const int last = (origin + min(n * KT, keys_rel) - 1) >> page_shift;
#pragma unroll 1
    for (int i = (origin >> page_shift) + lane; i <= last; i += 64) missing |= (uint32_t)table[i] >= num_pages;
    missing = __any(missing);
  }
  // A bit for every key of tile j that the request holds.
  constexpr uint64_t kAll = ~(uint64_t)0 >> (64 - KT);
  auto held_keys = [&](int j) {
    uint64_t held = kAll;
    const int top = keys_rel - j * KT, bottom = low_rel - j * KT;   // keys of the tile in [bottom, top)
    if (top < KT) held &= top > 0 ? ((uint64_t)1 << top) - 1 : 0;
    if (bottom > 0) held &= bottom < 64 ? ~(((uint64_t)1 << bottom) - 1) : 0;
    if (missing)
#pragma unroll 1
      for (int g = 0; g < NG; ++g)
        if (page_at(min(j, n - 1) * KT + 16 * g) >= num_pages) held &= ~((uint64_t)0xffff << (16 * g));
    return (uint64_t)uniform((int64_t)held);
  };
  // Tiles [held_from, held_to) are held in full, tiles [seen_from, seen_to) also
  // seen in full by every row of this wave.
  const int held_from = missing ? 0 : max(low_rel + KT - 1, 0) / KT, held_to = missing ? 0 : max(keys_rel, 0) / KT;
  const int seen_from = max(held_from, (max(wave_low, 0) + KT - 1) / KT);
  const int seen_to = min(held_to, (max(wave_pos, -1) + 1) / KT);
  // ... and tiles [all_from, all_to) by every row of the workgroup.
  const int all_from = max(held_from, (max(low_of(a, pos_last) - origin, 0) + KT - 1) / KT);
  const int all_to = min(held_to, (max(pos_first, -1) + 1 > origin ? max(pos_first, -1) + 1 - origin : 0) / KT);
  auto partly = [&](int j) { return j < all_from || j >= all_to; };

  // A load instruction i of this wave brings rows (i * 8 + wave) * RPI on; a
  // lane's 16 bytes go to consecutive LDS addresses, so the bank permutation is
  // made on the source side.  Without a page any page serves: its scores are
  // hidden and its values cleared.
  const uint32_t page_units = (uint32_t)(a.cache.page_stride * EB / 16), row_bytes = (uint32_t)a.cache.token_stride * EB;
  const int lane_row = lane / PPR, lane_col = lane % PPR;
  const int wave_rows = wave * RPI % 16;      // the permutations depend on the row modulo 16
  const uint32_t k_voff = (uint32_t)lane_row * row_bytes + (FP8 ? lane_col : lane_col ^ key_swizzle<D>(wave_rows + lane_row)) * 16;
  const uint32_t v_voff = (uint32_t)lane_row * row_bytes + (FP8 ? lane_col : lane_col ^ value_swizzle<D>(wave_rows + lane_row)) * 16;
  const bool brings = !SPARE || wave < KT / RPI;
  const uint8_t* k_base = (const uint8_t*)a.cache.k + head * a.cache.head_stride * EB;
  const uint8_t* v_base = (const uint8_t*)a.cache.v + head * a.cache.head_stride * EB;
  auto row_of = [&](int i) { return (i * kChunkWaves + wave) * RPI; };
  // Byte offsets of this wave's load instructions for 64 tiles at a time, a tile a lane.
  int64_t lane_at[NL];
  auto locate = [&](int j0) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int key = min(j0 + lane, n - 1) * KT + row_of(i);
      const uint32_t page = page_at(key);
      lane_at[i] = (int64_t)((uint64_t)(page < num_pages ? page : 0) * page_units << 4) +
                   (uint32_t)((origin + key) & page_mask) * row_bytes;
    }
  };
  typedef int64_t Offsets __attribute__((ext_vector_type(2)));
  auto offsets_of = [&](int j) {
    Offsets at = {0, 0};
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint32_t lo = __builtin_amdgcn_readlane((int)lane_at[i], j & 63), hi = __builtin_amdgcn_readlane((int)(lane_at[i] >> 32), j & 63);
      at[i] = (int64_t)((uint64_t)hi << 32 | lo);
    }
    return at;
  };
  // bf16: straight into LDS.  E4M3: into registers, a step later converted into LDS.
  u32x4 kr[FP8 ? NL : 1], vr[FP8 ? NL : 1];
  auto bring = [&](const uint8_t* base, const Offsets& at, int i, uint8_t* lds, uint32_t voff, u32x4* regs) {
    if constexpr (FP8) {
      if (brings) regs[i] = *(const u32x4*)(base + at[i] + voff);
    } else {
      dma16(base + at[i], voff, lds + (i * kChunkWaves + wave) * 1024);
    }
  };
  auto bring_all = [&](const uint8_t* base, const Offsets& at, uint8_t* lds, uint32_t voff, u32x4* regs) {
#pragma unroll
    for (int i = 0; i < NL; ++i) bring(base, at, i, lds, voff, regs);
  };
  // Values of keys that the request does not hold are cleared in LDS, by the lanes
  // that brought them: they may be NaN, and 0 * NaN is not 0.  Nor may infinities and
  // NaN of keys that not every row sees stay: they are added at the end.
  auto settle = [&](uint8_t* lds, u32x4* regs, bool values, int j) {
    if constexpr (FP8) {
      if (brings) {
        if (values && partly(j)) {
          const uint64_t held = held_keys(j);
          uint32_t odd = 0;
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            const uint32_t keep = held >> ((i * kChunkWaves + wave) * RPI + lane_row) & 1 ? 0xffffffffu : 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w = regs[i][k] & keep;
              regs[i][k] = finite_only<true>(w);
              odd |= w ^ regs[i][k];
            }
          }
          if (odd) not_finite[wave] = 1;
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int row = (i * kChunkWaves + wave) * RPI + lane_row;
          const int x = values ? value_swizzle<D>(row) : key_swizzle<D>(row);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w0 = regs[i][2 * k], w1 = regs[i][2 * k + 1];
            *(u32x4*)(lds + row * ROW + ((2 * lane_col + k) ^ x) * 16) =
                u32x4{e4m3_bf16<false>(w0), e4m3_bf16<true>(w0), e4m3_bf16<false>(w1), e4m3_bf16<true>(w1)};
          }
        }
      }
    }
  };
  auto clear_values = [&](uint8_t* lds, int j) {
    if constexpr (!FP8) {
      if (!partly(j)) return;
      const uint64_t held = held_keys(j);
      bool odd = false;
      constexpr int kUnroll = MIXED ? 1 : 2 * NL;   // heads of 256 have no registers to spare here
#pragma unroll kUnroll
      for (int i = 0; i < 2 * NL; ++i) {
        const int at = (i >> 1) * kChunkWaves + wave;
        const uint32_t keep = held >> (at * RPI + lane_row) & 1 ? 0xffffffffu : 0u;
        u32x2* p = (u32x2*)(lds + at * 1024 + lane * 16 + (i & 1) * 8);
        u32x2 w = *p;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = w[k] & keep;
          w[k] = finite_only<false>(x);
          odd |= w[k] != x;
        }
        *p = w;
      }
      if (odd) not_finite[wave] = 1;
    }
  };

  float m = -INFINITY, sum = 0.f;
  f32x16 o[DF], s[NK];
  bf16x8 p[2 * NK];
#pragma unroll
  for (int i = 0; i < DF; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;

  // lane parts of the LDS addresses
  const int k_row = c32 * ROW, k_x = (h ^ key_swizzle<D>(c32)) * 16;
  const int v_r = 4 * h + ((lane & 15) >> 2);
  const int v_row = v_r * ROW + (lane & 1) * 8, v_x = ((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swizzle<D>(v_r)) * 16;

  auto key_fragment = [&](const uint8_t* kt, int f, int st) {        // keys 32f on, columns 16st on
    return *(const bf16x8*)(kt + f * 32 * ROW + k_row + ((st * 32) ^ k_x));
  };
  auto value_fragment = [&](const uint8_t* vt, int u, int i) {       // keys 16u on, columns 32i on
    const uint8_t* vp = vt + u * 16 * ROW + v_row + ((i * 64) ^ v_x);
    const u32x2 v0 = read_transposed(vp), v1 = read_transposed(vp + 8 * ROW);
    return __builtin_bit_cast(bf16x8, u32x4{v0[0], v0[1], v1[0], v1[1]});
  };
  // Scores of tile j that the lane's row does not see.
  auto hide = [&](int j) {
    // a bit for every key of the tile that this lane's row sees
    const int bottom = my_low - j * KT, end = my_pos + 1 - j * KT;
    uint64_t see = held_keys(j);
    see = end <= 0 ? 0 : end < 64 ? see & (((uint64_t)1 << end) - 1) : see;
    see = bottom <= 0 ? see : bottom < 64 ? see & (~(uint64_t)0 << bottom) : 0;
#pragma unroll
    for (int f = 0; f < NK; ++f) {
      const uint32_t bits = (uint32_t)(see >> (32 * f)) >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[f][i] = bits >> (8 * (i >> 2) + (i & 3)) & 1 ? s[f][i] : -INFINITY;
    }
  };
  auto largest = [&] {
    float top = s[0][0];
#pragma unroll
    for (int f = 0; f < NK; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[f][i]);
    return top;
  };
  // The maximum, in log2 units, up to date; top is the tile's beyond what it is taken
  // for (0 before there is one).  It may lag behind by a factor of 2^8, which costs no
  // precision: O is scaled anew only when it does not suffice any more.
  auto reference = [&] { return m == -INFINITY ? 0.f : m; };
  // This path, and for heads of 256 that to `hide`, are marked as the rare ones: over E4M3
  // 45 registers are spilled and not 52, off the common path (4096 after 4096, heads of
  // 256: 670 us, unmarked 815; heads of 128, 8192 after 8192: 1883, 1922).
  auto raise = [&](float top) {
    if (__builtin_expect(__any(top > 8.f || (m == -INFINITY && top > m)), 0)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      // Heads of 256 have weights rounded to bf16 that are still to be multiplied: their
      // maximum is taken in whole steps, by which a rounded weight is scaled exactly.
      const float old = reference(), to = fmaxf(m, MIXED ? ceilf(old + top) : old + top);
      const float by = m == to ? 1.f : m == -INFINITY ? 0.f : MIXED ? ldexpf(1.f, (int)fmaxf(m - to, -200.f)) : exp2_fast(m - to);
      m = to;
      sum *= by;
#pragma unroll
      for (int i = 0; i < DF; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[i][k] *= by;
      if constexpr (MIXED) {
#pragma unroll
        for (int u = 0; u < 2 * NK; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) p[u][i] = (__bf16)((float)p[u][i] * by);
      } else {                               // the exponents, which are at hand already
        const float shift = old - reference();
#pragma unroll
        for (int f = 0; f < NK; ++f)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[f][i] += shift;
      }
    }
  };
  // Weights of 16 keys.  In bf16, the matrix instruction's type with V: 2^-8 relative a
  // term at most, averaged over the keys.
  auto weigh = [&](int u, float ref) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = s[u >> 1][8 * (u & 1) + i];
      e[i] = exp2_fast(MIXED ? fmaf(x, c, -ref) : x);
    }
    sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    u32x4 w = {pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7])};
    if constexpr (MIXED) asm volatile("" : "+v"(w), "+v"(sum));   // here, among the products, and not where the next turn needs them
    p[u] = __builtin_bit_cast(bf16x8, w);
  };

  if (n > 0) {
    if constexpr (!MIXED) {
      // The first product of the next tile, then the second of this one, four fragments
      // a step, their operands read kAhead steps before (an LDS read takes longer than
      // the four instructions of a step); those of the first steps are read before the
      // barrier that begins the phase.  The exponents' arguments and their maximum are
      // found beside the second product, where the vector unit would idle.
      constexpr int kAhead = 2;
      constexpr int QK = NK * KS / 4, STEPS = QK + NK * DF / 2;
      bf16x8 frag[kAhead + 1][4];
      auto read_operands = [&](const uint8_t* kt, const uint8_t* vt, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * t + i, v = e - 4 * QK;
          frag[t % (kAhead + 1)][i] = t < QK ? key_fragment(kt, e % NK, e / NK) : value_fragment(vt, v / DF, v % DF);
        }
      };
      float top0;
      auto products = [&](const uint8_t* kt, const uint8_t* vt, auto between) {
        const float ref = reference();
#pragma unroll
        for (int f = 0; f < NK; ++f)
#pragma unroll
          for (int j = 0; j < 16; ++j) s[f][j] = 0.f;
#pragma unroll
        for (int t = 0; t < STEPS; ++t) {
          if (t + kAhead < STEPS) {
            read_operands(kt, vt, t + kAhead);
            if (t + kAhead < QK) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);   // a step's LDS reads, then four products
            else __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * t + i, v = e - 4 * QK, at = t % (kAhead + 1);
            if (t < QK) s[e % NK] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag[at][i], q[e / NK], s[e % NK], 0, 0, 0);
            else o[v % DF] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag[at][i], p[v / DF], o[v % DF], 0, 0, 0);
          }
          if (t > QK) {                      // a step after the last of the scores
            constexpr int kEach = 16 / (STEPS - QK - 1) + 1;
#pragma unroll
            for (int i = (t - QK - 1) * kEach; i < (t - QK) * kEach && i < 16; ++i)
#pragma unroll
              for (int f = 0; f < NK; ++f) {
                s[f][i] = fmaf(s[f][i], c, -ref);
                top0 = i + f == 0 ? s[0][0] : fmaxf(top0, s[f][i]);
              }
          }
          __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
          between(t);
        }
      };
      // Before the loop: keys 0 - 2, values 0 and 1.  The loop begins at tile -1, whose
      // values and weights are 0, so that tile 0's scores need no code of their own.
      constexpr int kLead = FP8 ? 5 : 4;       // the tile whose keys are asked for while tile 0's values are multiplied
      locate(0);
      Offsets key_at, value_at;
#pragma unroll
      for (int i = 0; i < KT * ROW / 16 / kThreads; ++i) *(u32x4*)(lds_v[3] + (i * kThreads + tid) * 16) = u32x4{0u, 0u, 0u, 0u};
#pragma unroll 1
      for (int j = 0; j < 3; ++j) {
        key_at = offsets_of(j);
        bring_all(k_base, key_at, lds_k[j], k_voff, kr);
        settle(lds_k[j], kr, false, j);
        if (j == 2) break;
        bring_all(v_base, key_at, lds_v[j], v_voff, vr);
        settle(lds_v[j], vr, true, j);
      }
      value_at = key_at;
      if constexpr (FP8) {                     // in registers: keys 3, values 2
        bring_all(v_base, value_at, nullptr, v_voff, vr);
        value_at = offsets_of(3);
        bring_all(k_base, value_at, nullptr, k_voff, kr);
      }
      key_at = offsets_of(kLead - 1);
#pragma unroll
      for (int u = 0; u < 2 * NK; ++u) p[u] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
      wait_arrived<0>();
#pragma unroll 1
      for (int j = 0; j < 2; ++j)
        clear_values(lds_v[j], j);
      phase_barrier<true>();
      // The two waves of a SIMD take turns: while waves 0-3 multiply, waves 4-7,
      // one barrier behind, run their softmax, and the other way round.
      if (wave >= kChunkWaves / 2) phase_barrier<false>();
#pragma unroll
      for (int t = 0; t < kAhead; ++t) read_operands(lds_k[0], lds_v[3], t);
#pragma unroll 1
      for (int j = -1; j < n; ++j) {
        // Products: O += values j, S = keys j + 1.  Tile j + 4's keys take the place of
        // tile j's, tile j + 3's values that of tile j - 1's, which all have read; they
        // are waited for in the next products and read at the end of the softmax after.
        uint8_t* const free_k = lds_k[j & 3];
        uint8_t* const free_v = lds_v[(j + 3) & 3];
        settle(free_k, kr, false, j);
        settle(free_v, vr, true, j + 3);
        __builtin_amdgcn_s_setprio(1);
        products(lds_k[(j + 1) & 3], lds_v[j & 3], [&](int step) {
          if (step < NL) bring(k_base, key_at, step, free_k, k_voff, kr);
          else if (step < 2 * NL) bring(v_base, value_at, step - NL, free_v, v_voff, vr);
        });
        __builtin_amdgcn_s_setprio(0);
        if constexpr (!FP8) {                  // all but what this phase asked for has arrived: tile j + 2's values
          wait_arrived<2 * NL>();
          clear_values(lds_v[(j + 2) & 3], j + 2);
        }
        phase_barrier<true>();
        if (j + 1 < n) {
          if (j + 1 < seen_from || j + 1 >= seen_to) {
            hide(j + 1);
            top0 = largest();
          }
          raise(top0);
#pragma unroll
          for (int u = 0; u < 2 * NK; ++u) weigh(u, 0.f);
        }
        if (((j + 1 + kLead) & 63) == 0) locate(j + 1 + kLead);
        value_at = key_at;
        key_at = offsets_of(j + 1 + kLead);
#pragma unroll
        for (int t = 0; t < kAhead; ++t) read_operands(lds_k[(j + 2) & 3], lds_v[(j + 1) & 3], t);
        phase_barrier<false>();
      }
      if (wave < kChunkWaves / 2) phase_barrier<false>();
    } else {
      // Fragment e of the second product (O's fragment fastest), then of the first: the
      // matrix instructions of a tile in order, operands RING - 1 instructions ahead.
      constexpr int PV = 2 * DF, QK = KS, RING = 4;
      bf16x8 ring[RING];
      auto read_fragment = [&](const uint8_t* kt, const uint8_t* vt, int e) {
        ring[e % RING] = e < PV ? value_fragment(vt, e / DF, e % DF) : key_fragment(kt, 0, e - PV);
      };
      auto multiply = [&](int e) {
        if (e < PV) {
          o[e % DF] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[e % RING], p[e / DF], o[e % DF], 0, 0, 0);
        } else {
          f32x16 zero;
#pragma unroll
          for (int j = 0; j < 16; ++j) zero[j] = 0.f;
          s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[e % RING], q[e - PV], e == PV ? zero : s[0], 0, 0, 0);
        }
      };
      auto read_first = [&](const uint8_t* kt, const uint8_t* vt) {
#pragma unroll
        for (int e = 0; e < RING - 1; ++e) read_fragment(kt, vt, e);
      };
      // Before the loop: keys 0 - 3, values 0 and 1, and tile 0's scores.  Tile -1's
      // values and weights are 0.
      constexpr int kLead = FP8 ? 5 : 4;       // the tile whose keys are asked for in tile 0's turn
      locate(0);
      Offsets key_at, value_at, value_next;
#pragma unroll
      for (int i = 0; i < KT * ROW / 16 / kThreads; ++i) *(u32x4*)(lds_v[3] + (i * kThreads + tid) * 16) = u32x4{0u, 0u, 0u, 0u};
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        key_at = offsets_of(j);
        bring_all(k_base, key_at, lds_k[j], k_voff, kr);
        settle(lds_k[j], kr, false, j);
        if (j >= 2) continue;
        bring_all(v_base, key_at, lds_v[j], v_voff, vr);
        settle(lds_v[j], vr, true, j);
      }
      value_at = offsets_of(2);
      value_next = offsets_of(3);
      if constexpr (FP8) {                     // in registers: keys 4, values 2
        bring_all(v_base, value_at, nullptr, v_voff, vr);
        key_at = offsets_of(4);
        bring_all(k_base, key_at, nullptr, k_voff, kr);
        value_at = value_next;
        value_next = key_at;
      }
      key_at = offsets_of(kLead);
#pragma unroll
      for (int u = 0; u < 2 * NK; ++u) p[u] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
      wait_arrived<0>();
#pragma unroll 1
      for (int j = 0; j < 2; ++j)
        clear_values(lds_v[j], j);
      phase_barrier<true>();
#pragma unroll
      for (int e = PV; e < PV + QK; ++e) {
        read_fragment(lds_k[0], lds_v[3], e);
        multiply(e);
      }
      if constexpr (!FP8) read_first(lds_k[1], lds_v[3]);
      phase_barrier<true>();                   // tile 0's keys have been read by all
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        // Tile j's turn: O += values j - 1, weights j from scores j, scores j + 1 from
        // keys j + 1.  Tile j + 4's keys take the place of tile j's, tile j + 2's values
        // that of tile j - 2's, which all have read; they are waited for in the next turn
        // and read from the end of the one after.
        uint8_t* const free_k = lds_k[j & 3];
        uint8_t* const free_v = lds_v[(j + 2) & 3];
        const uint8_t* const kt = lds_k[(j + 1) & 3];
        const uint8_t* const vt = lds_v[(j + 3) & 3];
        settle(free_k, kr, false, j);
        settle(free_v, vr, true, j + 2);
        if constexpr (FP8) read_first(kt, vt);   // not across the conversions, whose registers they would take
        if (__builtin_expect(j < seen_from || j >= seen_to, 0)) hide(j);
        raise(fmaf(largest(), c, -reference()));
        const float ref = reference();
        auto turn = [&](int e) {               // fragment e's product, the read of the one RING - 1 on before it
          const int ahead = e + RING - 1;
          if (ahead < PV + QK) {
            read_fragment(kt, vt, ahead);
            if (ahead < PV) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
          multiply(e);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        };
#pragma unroll
        for (int e = 0; e < PV; ++e) {
          turn(e);
          const int u = e / DF;
          if (u > 0) {                         // the weights of the 16 keys whose old ones are done with
            if (e % DF == 0) weigh(0, ref);
            __builtin_amdgcn_sched_group_barrier(0x002, 28 / DF, 0);
          }
          if (e % (PV / 4) == 1) {
            const int i = e / (PV / 4);
            if (i < NL) bring(k_base, key_at, i, free_k, k_voff, kr);
            else if (i < 2 * NL) bring(v_base, value_at, i - NL, free_v, v_voff, vr);
          }
        }
        weigh(1, ref);
#pragma unroll
        for (int e = PV; e < PV + QK; ++e) turn(e);
        if (((j + 1 + kLead) & 63) == 0) locate(j + 1 + kLead);
        value_at = value_next;
        value_next = key_at;
        key_at = offsets_of(j + 1 + kLead);
        if constexpr (!FP8) {                  // all but what this turn asked for has arrived: tile j + 1's values
          wait_arrived<2 * NL>();
          clear_values(lds_v[(j + 1) & 3], j + 1);
        }
        if constexpr (!FP8) read_first(lds_k[(j + 2) & 3], lds_v[j & 3]);
        phase_barrier<true>();
      }
#pragma unroll
      for (int e = 0; e < PV; ++e) {           // the last tile's values
        if (FP8 || e >= RING - 1) read_fragment(lds_k[0], lds_v[(n - 1) & 3], e);
        multiply(e);
      }
    }
    wait_arrived<0>();                       // nothing may still be on its way into LDS when the workgroup ends
  }

  sum += __shfl_xor(sum, 32);
  const float top = m;
  if (live) {
    const int trow = l.start + my_token;
    const int64_t slot = ((int64_t)place * 2 + part) * kChunkRows + wave * 32 + c32;
    const float vs = a.cache.v_scale ? a.cache.v_scale[head] : 1.f;
    const float by = !whole ? 1.f : sum == 0.f ? 0.f : vs / sum;
    const int64_t at = (int64_t)trow * a.ld_out + my_head * D + 4 * h;
    if (whole && a.out_bf16) {
#pragma unroll
      for (int i = 0; i < DF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *(u32x2*)((uint16_t*)a.out + at + 32 * i + 8 * j) =
              u32x2{pack_bf16(o[i][4 * j] * by, o[i][4 * j + 1] * by), pack_bf16(o[i][4 * j + 2] * by, o[i][4 * j + 3] * by)};
    } else {
      float* to = whole ? (float*)a.out + at : ws.o + slot * D + 4 * h;
#pragma unroll
      for (int i = 0; i < DF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *(f32x4*)(to + 32 * i + 8 * j) = f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]} * by;
    }
    bool odd = false;
    if (n > 0)
#pragma unroll 1
      for (int w = 0; w < kChunkWaves; ++w) odd |= not_finite[w] != 0;
    if (odd) {   // rare, and slow: what the row sees of them, added to what has just been written
#pragma unroll 1
      for (int key = max(my_low, 0); key < min(min(keys_rel, my_pos + 1), n * KT); ++key) {
        if (!partly(key / KT)) {
          key = all_to * KT - 1;
          continue;
        }
        const uint32_t page = page_at(key);
        if (page >= num_pages) continue;
        const uint8_t* token = v_base + (int64_t)((uint64_t)page * page_units << 4) + (uint32_t)((origin + key) & page_mask) * row_bytes;
#pragma unroll 1
        for (int d = 4 * h; d < D; d += 8) {
          if (whole && a.out_bf16) {
            uint16_t* to = (uint16_t*)a.out + at - 4 * h + d;
            const u32x2 w = *(u32x2*)to;
            const f32x4 x = add_not_finite<FP8>(f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                                                      __uint_as_float(w[1] & 0xffff0000u)}, token + d * EB, by);
            *(u32x2*)to = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
          } else {
            f32x4* to = (f32x4*)(whole ? (float*)a.out + at - 4 * h + d : ws.o + slot * D + d);
            *to = add_not_finite<FP8>(*to, token + d * EB, by);
          }
        }
      }
    }
    if (h == 0) {
      if (!whole) ws.ml[slot] = make_float2(top, sum);
      else if (a.lse) a.lse[(int64_t)trow * a.hq + my_head] = sum == 0.f ? -INFINITY : kLn2 * (top + __log2f(sum));
    }
  }
  }
}

// Joins the parts of a row tile that several workgroups hold, in the order of
// their keys.  Grid (row tile numbers x KV heads, 8): 32 rows a workgroup.
template <int D>
__global__ __launch_bounds__(256) void attention_chunk_join_kernel(AttentionArgs a, ChunkWorkspace ws) {
  const int hkv = a.cache.heads, group = a.group;
  const int head = blockIdx.x % hkv;
  const RowTile t = row_tile(a, blockIdx.x / hkv);
  const RequestLens l = request_lens(a, t.r);
  const ChunkLine line = chunk_line(a, l);
  if (t.b < 0 || t.b >= line.tiles) return;
  const int64_t share = ws.prefix[a.requests + 1];
  const int64_t x0 = head * ws.prefix[a.requests] + ws.prefix[t.r] + line_before(line, t.b);
  // the first part is held by the workgroup of the last cut that was moved to the tile's start or before it
  const int g0 = (int)div_f64(x0 + line.extra - 1, share), g1 = (int)div_f64(x0 + line_length(line, t.b) - line.extra, share);
  if (g0 >= g1) return;
  const int nrows = min(l.tokens * group - t.b * kChunkRows, kChunkRows);
  const float vs = a.cache.v_scale ? a.cache.v_scale[head] : 1.f;
  for (int e = threadIdx.x; e < 32 * (D / 4); e += 256) {
    const int at = blockIdx.y * 32 + e / (D / 4), d = (e % (D / 4)) * 4;
    if (at >= nrows) return;
    auto slot_of = [&](int wg) { return (int64_t)(wg * 2 + (wg == g0 ? 1 : 0)) * kChunkRows + at; };
    float den;
    f32x4 num;
    const float top = join_parts<D, false>(ws.ml, ws.o, slot_of, g0, g1, d, &den, &num);
    write_row<D>(a, l.start, head, t.b * kChunkRows + at, d, top, den, num, vs);
  }
}

size_t attention_chunk_workspace(int64_t requests, int dim) {
  return (size_t)(uintptr_t)chunk_workspace(nullptr, requests).o + (size_t)2 * kChunkGrid * kChunkRows * dim * sizeof(float);
}

namespace {

// Whether row tiles are handed out whole, one a workgroup as they finish, with nothing
// to join, or cut into equal shares.  Shares cost what a workgroup takes for about 1500
// keys (parts of O written and read, the join's launch); whole tiles cost the longest
// one at least, and a last round that is not full, of which the shortest tile at most
// is lost where they come long ones first.  The host knows bounds alone: it takes the
// lengths of several requests as three quarters of the longest, and their last tiles
// as half full.  Three tiles a workgroup and more fill the chip whatever they are.
// Heads of 128, whole against shares: prompts of 1024, 2048, 4096, 5000, 8192 tokens 38
// against 46, 65 / 78, 155 / 183, 227 / 240, 507 / 559 us; 512 tokens after 8192 190 /
// 100, 128 after 65536 1353 / 175; 8 windowed chunks (heads of 64) 103 / 92; both
// kernels' times, 256 single tokens over 2000 keys beside 512 tokens after 8192 558 / 487.
bool tiles_alone(const AttentionArgs& a) {
  const double round = (double)kChunkGrid / a.cache.heads, all = (double)row_tiles(a.tokens, a.requests, a.group) / round;
  const bool one = a.requests == 1;
  // Where the other kernel takes the requests of few rows, those of many are taken for
  // as few as their tokens allow, and a workgroup finds nothing for each other one: a
  // round of these costs what 150 keys do.
  const double many = a.stream_rows ? fmin((double)a.requests, ceil((double)a.tokens / a.max_new)) : (double)a.requests;
  const double rows = (double)(a.stream_rows ? max(a.tokens - a.requests, (int64_t)1) : a.tokens) * a.group / kChunkRows;
  const double tiles = (one ? ceil(rows) : rows + 0.5 * many) / round, rounds = ceil((one ? ceil(rows) : rows + many) / round);
  double longest = (double)max(a.max_seq, a.max_new);
  if (a.window) longest = fmin(longest, (double)a.window + (double)kChunkRows / a.group);
  const double average = kExtraKeys + (one ? fmax(longest - 0.5 * a.tokens, 0.5 * longest) : 0.75 * longest);
  const double shortest = one ? kExtraKeys + fmax(longest - a.tokens, 0.) : average;
  const double whole = tiles >= 3. ? tiles * average : fmax(longest + kExtraKeys, fmin(rounds * average, tiles * average + shortest));
  return whole + fmax(all - rounds, 0.) * 150. < tiles * average + 1500.;
}

template <int D, bool FP8>
hipError_t launch(const AttentionArgs& a, void* workspace, hipStream_t st) {
  const ChunkWorkspace ws = chunk_workspace(workspace, a.requests);
  const int64_t numbers = row_tiles(a.tokens, a.requests, a.group);
  if (tiles_alone(a)) {
    attention_chunk_kernel<D, FP8><<<(unsigned)(numbers * a.cache.heads), kThreads, 0, st>>>(a, ws, (int)numbers);
    return hipGetLastError();
  }
  attention_chunk_kernel<D, FP8><<<kChunkGrid, kThreads, 0, st>>>(a, ws, 0);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attention_chunk_join_kernel<D><<<dim3((unsigned)(numbers * a.cache.heads), 8), 256, 0, st>>>(a, ws);
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
// other to the tiled one (64 decoded tokens over 8192 keys, heads of 128: streaming
// 362 us, tiled 496); both are launched where the batch may hold both.  Where it has
// no request of 33 rows the tiled kernel is not launched, and where requests bring 64
// rows and more on average, or a quarter of the largest request's, the tiled kernel
// takes all of them, which spares launches and the second pass over the chip (32
// requests of up to 32 tokens over 4096 keys: 92 us, both kernels 112; of up to 10
// 93 against 113).
// Clears the padding rows of a batch that has nothing else (it brings no new tokens).
__global__ __launch_bounds__(256) void attention_padding_kernel(AttentionArgs a) { clear_padding(a, a.q_start[a.requests]); }

static bool may_tile(int64_t max_new, int group) { return max_new * group > kDecodeRows; }
static bool may_stream(int64_t tokens, int64_t requests, int64_t max_new, int group) {
  return max_new > 0 && group <= kDecodeRows && 
         !(may_tile(max_new, group) && (tokens * group >= 64 * requests || 4 * tokens >= max_new * requests));
}

size_t attention_workspace_bytes(int64_t tokens, int64_t requests, int hq, int hkv, int dim, int64_t max_new,
                                 int64_t max_seq) {
  size_t n = 16 + kArrivedBytes;
  // what serves a step serves smaller ones: whatever the tokens, and with the streaming
  // kernel's parts for groups above its rows too, whose calls never use them
  if (max_new > 0) n += (attention_decode_workspace(dim) + 255) / 256 * 256;
  if (may_tile(max_new, hq / hkv)) n += attention_chunk_workspace(requests, dim);
  return n;
}

hipError_t launch_paged_attention(const AttentionArgs& args, hipStream_t st) {
  AttentionArgs a = args;
  if (a.group > 1) {
    int s = 31 - __builtin_clz(a.group);
    const bool power = (a.group & (a.group - 1)) == 0;
    a.group_mul = power ? 1u << 31 : (uint32_t)(((uint64_t)1 << (32 + s)) / a.group + 1);
    a.group_shift = power ? s - 1 : s;
  }
  // the counters that have to be 0 between calls lie first whichever kernels run
  uint8_t* ws = (uint8_t*)a.workspace + kArrivedBytes;
  a.stream_rows = 0;
  if (may_stream(a.tokens, a.requests, a.max_new, a.group)) {
    a.stream_rows = kDecodeRows;
    hipError_t e = launch_attention_decode(a, st);
    if (e != hipSuccess) return e;
    a.clear_padding = false;   // done
    ws += (attention_decode_workspace(a.cache.dim) + 255) / 256 * 256;
  }
  if (may_tile(a.max_new, a.group)) return launch_attention_chunk(a, ws, st);
  if (!a.clear_padding) return hipSuccess;
  attention_padding_kernel<<<(unsigned)min(a.tokens, (int64_t)1024), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
