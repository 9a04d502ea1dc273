// Attention of a few new tokens a request (a decoded token, a handful of
// drafts) over the paged cache on gfx950: the streaming kernel.
//
// Mathematics, per row (new token, query head) with c = scale * k_scale * log2 e
// and m the running maximum of q.k over the keys seen so far:
//     l <- l 2^(c (m_old - m)) + sum_j 2^(c (s_j - m)),
//     O <- O 2^(c (m_old - m)) + sum_j 2^(c (s_j - m)) v_j,
// so K and V are read once; O / l * v_scale is the output.  A negative c is
// folded into the sign of q, so that the largest s is always the largest score.
//
// Bound by the cache's bytes.  The rows of one KV head's group (tokens x heads
// of the group, up to 32) share each key tile, as the columns of 16x16x32
// bf16 MFMAs: S^T = K Q^T and O^T = V^T P^T.  Everything stays in registers:
//   - K: a lane loads 16 bytes of one key; lanes l & 15 are the tile's keys.
//   - S^T: column = row of q = l & 15, rows = keys 4 g + r (g = l >> 4), so a
//     softmax row lies in four lanes and P^T is already the B operand of the
//     second product if its k index (g, j) stands for key 4 g + j (j < 4) and
//     16 + 4 g + j - 4 (j >= 4): a sum does not mind the order of its terms.
//   - V: a lane loads, for those eight keys, D / 16 neighbouring columns; an
//     8 x (D / 16) transpose inside the lane (v_perm) makes the A operands,
//     whose row l & 15 of operand i stands for column (l & 15) D / 16 + i.
// So there is no LDS traffic and no barrier in the loop, every load is a
// whole cache line over a wave, and the next tile's loads are in flight while a
// tile is computed.  An E4M3 cache halves the bytes; its elements become bf16
// exactly after the load (scales go into c and the output).
//
// Split: the key tiles of all requests and KV heads form one line that a fixed
// grid shares evenly, so a long request among short ones, or one request alone,
// fills the chip.  A workgroup that holds all of a (request, head) writes its
// output; a part leaves (max, sum, O) in the workspace (at most two a workgroup),
// and the workgroup whose part arrives last joins all of them in the order of
// their keys, whatever the order in which they came (a second kernel for that
// cost 4 us of the GPU's time and as much of the host's, a third of one decoded
// token).  The line's prefix is recomputed by every workgroup (8 bytes a request).
//
// Measured: 64 requests of up to 16384 keys, 40 heads of 128 over 8: 388 us, 5.7 TB/s
// of the keys and values (a large copy moves 5.0).  E4M3: 32 requests of 8192 keys with
// five tokens each, 24 heads of 256 over 4: 129 - 138 us among other calls, 133 - 151
// alone, 3.9 - 4.2 TB/s; there the conversion and the transpose share the issue slots
// with two fragments of rows, and O takes the registers that more loads in flight would
// need (two tiles ahead spilled: 173 us).  With ragged lengths, and so fewer bytes, less:
// 32 requests of up to 8192 keys, 32 rows of 256, 2.8 TB/s over E4M3 and 3.4 over bf16;
// 64 requests, heads of 128, 20 rows, 3.6 over E4M3 and 5.1; one token, heads of 128,
// 4.1 and 5.2, heads of 64 3.6 and 5.3.  One token over 1000 keys: 10 us, latency.
#include <float.h>

#include "attention.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 64 * kDecodeWaves;

struct DecodeWorkspace {
  uint32_t* arrived;   // [grid] parts that have been left of the item that begins in a workgroup's share; 0 between calls
  float2* ml;          // [2 * grid][kDecodeRows] (max in log2 units, sum)
  float* o;            // [2 * grid][kDecodeRows][dim]
};
__host__ __device__ inline DecodeWorkspace decode_workspace(void* ws) {
  DecodeWorkspace w;
  w.arrived = (uint32_t*)ws;
  w.ml = (float2*)((uint8_t*)ws + kArrivedBytes);
  w.o = (float*)(w.ml + 2 * kDecodeGrid * kDecodeRows);
  return w;
}

// A request's part of the line: first key (a tile's start) and tiles of one
// head; 0 tiles if it has no rows here.  A request whose rows see nothing has one.
struct DecodeItem {
  RequestLens l;
  int begin, tiles;
};
__device__ __forceinline__ DecodeItem decode_item(const AttentionArgs& a, int r) {
  DecodeItem it;
  it.l = request_lens(a, r);
  it.begin = low_of(a, it.l.pos0) & ~(kDecodeTile - 1);
  it.tiles = max((it.l.keys - it.begin + kDecodeTile - 1) >> 5, 1);
  if (it.l.tokens == 0 || it.l.tokens > kDecodeRows || it.l.tokens * a.group > kDecodeRows) it.tiles = 0;
  return it;
}
static_assert(kDecodeTile == 32 && kDecodeWaves == 4, "");

// One key tile's K and V in registers.
template <int D, bool FP8>
struct DecodeTile {
  static constexpr int KW = FP8 ? D / 64 : D / 32;             // 16-byte words a lane holds of a key
  static constexpr int VW = D / 16 * (FP8 ? 1 : 2) / 4;        // 4-byte words a lane holds of a value row
  u32x4 k[2][KW];
  uint32_t v[8][VW];
};

template <int W>
__device__ __forceinline__ void load_words(uint32_t* out, const uint8_t* p) {
  if constexpr (W == 1) {
    out[0] = *(const uint32_t*)p;
  } else if constexpr (W == 2) {
    const u32x2 x = *(const u32x2*)p;
    out[0] = x[0], out[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4 x = *(const u32x4*)(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[4 * i + j] = x[j];
    }
  }
}

}  // namespace

// As many workgroups as the registers let be resident: two a CU, one for heads of 256
// (64 requests over up to 16384 keys, heads of 128: 388 us, with one 396; 32 x 8192 E4M3
// keys of 256: 132 us with one, 159 with two, of which one waits for the other).
constexpr int decode_grid(int dim) { return dim <= 128 ? kDecodeGrid : kDecodeGrid / 2; }

template <int D, bool FP8, int NF>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void attention_decode_kernel(AttentionArgs a) {
  using Tile = DecodeTile<D, FP8>;
  constexpr int KS = D / 32;      // k steps of the first product
  constexpr int DV = D / 16;      // value columns a lane holds = fragments of O
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int LD = D + 4;
  constexpr int GRID = decode_grid(D);
  __shared__ int64_t before[kThreads + 1];
  __shared__ int64_t wave_sum[kDecodeWaves];
  __shared__ __attribute__((aligned(16))) float o_part[kDecodeWaves][16][LD];
  __shared__ float2 ml_part[kDecodeWaves][16];
  __shared__ int not_finite[kDecodeWaves];
  __shared__ int last_part;

  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hkv = a.cache.heads, group = a.group;
  const DecodeWorkspace ws = decode_workspace(a.workspace);
  const int padding = a.clear_padding ? a.q_start[a.requests] : INT32_MAX;   // first row of no request

  // prefix of the tiles over runs of requests
  const int requests = (int)a.requests, run = (requests + kThreads - 1) / kThreads;
  const int r0 = min(tid * run, requests), r1 = min(r0 + run, requests);
  int64_t sum = 0;
  for (int r = r0; r < r1; ++r) sum += decode_item(a, r).tiles;
  int64_t inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 63) wave_sum[wave] = inc;
  __syncthreads();
  for (int w = 0; w < wave; ++w) inc += wave_sum[w];
  if (tid == 0) before[0] = 0;
  before[tid + 1] = inc;
  __syncthreads();
  const int64_t total = uniform(before[kThreads] * hkv);
  // at least one tile a wave: a smaller share would only add parts to join
  const int64_t per = max((total + GRID - 1) / GRID, (int64_t)kDecodeWaves);
  const int64_t x_begin = blockIdx.x * per, x_end = min(x_begin + per, total);
  const int page_mask = (1 << a.cache.page_shift) - 1;
  const uint32_t page_units = (uint32_t)(a.cache.page_stride * EB / 16), row_bytes = (uint32_t)a.cache.token_stride * EB;
  const uint32_t k_lane = (uint32_t)c16 * row_bytes + g * 16;
  uint32_t v_lane[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v_lane[j] = (uint32_t)(4 * g + j) * row_bytes + c16 * DV * EB;
  int row_token[NF], row_head[NF];
#pragma unroll
  for (int n = 0; n < NF; ++n) {
    row_token[n] = div_group(a, n * 16 + c16);
    row_head[n] = n * 16 + c16 - row_token[n] * group;
  }

  for (int64_t x = x_begin; x < x_end;) {
    // the request and head at x
    int lo = 0;
#pragma unroll
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (before[lo + step] * hkv <= x) lo += step;
    int r = lo * run;
    int64_t base = before[lo];
    DecodeItem it = decode_item(a, r);
    while (x >= (base + it.tiles) * hkv) {   // ends: x < before[lo + 1] * hkv
      base += it.tiles;
      it = decode_item(a, ++r);
    }
    r = uniform(r);
    it.l.start = uniform(it.l.start), it.l.tokens = uniform(it.l.tokens), it.l.pos0 = uniform(it.l.pos0);
    it.tiles = uniform(it.tiles);
    const int64_t in_request = x - base * hkv;
    const int head = uniform((int)div_f64(in_request, it.tiles));
    const int first = uniform((int)(in_request - (int64_t)head * it.tiles));
    const int n = uniform((int)min((int64_t)(it.tiles - first), x_end - x));   // tiles [first, first + n) of this head
    const bool whole = n == it.tiles;
    const int part = x == x_begin ? 0 : 1;
    x += n;

    const int nrows = it.l.tokens * group;
    // positions relative to the first key of the part
    const int origin = uniform(it.begin + first * kDecodeTile);
    const int pos0 = it.l.pos0, pos_last = pos0 + it.l.tokens - 1;
    const int keys = uniform(min(it.l.keys, max(pos_last, -1) + 1) - origin);
    const int low = uniform(low_of(a, pos0) - origin);   // first key that a row may see
    // tiles [seen_from, seen_to) are seen in full by every row
    const int seen_from = uniform((max(low_of(a, pos_last) - origin, 0) + kDecodeTile - 1) >> 5);
    const int seen_to = uniform(max(min(keys, max(pos0, -1) + 1 - origin), 0) >> 5);
    float c = a.scale * kLog2e;
    if (a.cache.k_scale) c *= a.cache.k_scale[head];
    const uint32_t flip = c < 0.f ? 0x80008000u : 0u, spoil = c == c ? 0u : 0x7fff7fffu;   // a NaN scale goes into q
    c = fmaxf(fabsf(c), FLT_MIN);   // never 0: a hidden score's -inf stays one

    // Q, the B operand: column c16 = row of q, k = 8 columns of q
    bf16x8 q[NF][KS];
    int row_pos[NF], row_low[NF];
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      const bool live = n * 16 + c16 < nrows;
      row_pos[n] = live ? max(pos0 + row_token[n], -1) - origin : INT32_MIN / 2;
      row_low[n] = low_of(a, pos0 + row_token[n]) - origin;
      const uint16_t* qr = a.q + (int64_t)(it.l.start + (live ? row_token[n] : 0)) * a.ld_q + (head * group + (live ? row_head[n] : 0)) * D;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // E4M3 keys are loaded 16 columns at a time: steps 2 i, 2 i + 1 take a lane's halves
        const int chunk = FP8 ? (s >> 1) * 8 + g * 2 + (s & 1) : s * 4 + g;
        u32x4 w = *(const u32x4*)(qr + chunk * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = live ? (w[i] ^ flip) | spoil : 0u;
        q[n][s] = __builtin_bit_cast(bf16x8, w);
      }
    }

    bool odd = false;   // infinities or NaN were taken out of values that not every row sees
    float m[NF], l[NF];
    f32x4 o[NF][DV];
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.f;
#pragma unroll
      for (int i = 0; i < DV; ++i) o[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // Byte offsets of the two 16-key groups of this wave's tiles, 64 tiles at a
    // time, a tile a lane: tile k of the wave is tile wave + 4 k of the part.
    // Without a page any page serves: its scores are hidden and its values cleared.
    const int32_t* table = a.block_table + (int64_t)r * a.ld_table;
    const uint32_t num_pages = (uint32_t)a.cache.num_pages;
    int64_t lane_at[2];
    uint64_t without[2];            // a bit for each of these tiles whose group has no page
    auto locate = [&](int k0) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int key = (wave + (k0 + lane) * kDecodeWaves) * kDecodeTile + 16 * f;
        const uint32_t page = key < keys ? (uint32_t)table[(uint32_t)(origin + key) >> a.cache.page_shift] : num_pages;
        without[f] = __ballot(page >= num_pages);
        lane_at[f] = (int64_t)((uint64_t)(page < num_pages ? page : 0) * page_units << 4) +
                     (uint32_t)((origin + key) & page_mask) * row_bytes;
      }
    };
    auto group_at = [&](int k, int f) {
      const uint32_t lo = __builtin_amdgcn_readlane((int)lane_at[f], k & 63), hi = __builtin_amdgcn_readlane((int)(lane_at[f] >> 32), k & 63);
      return (int64_t)((uint64_t)hi << 32 | lo);
    };
    const uint8_t* k_base = (const uint8_t*)a.cache.k + head * a.cache.head_stride * EB;
    const uint8_t* v_base = (const uint8_t*)a.cache.v + head * a.cache.head_stride * EB;
    auto load_keys = [&](Tile& tile, int k) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint8_t* kp = k_base + group_at(k, f);
#pragma unroll
        for (int st = 0; st < Tile::KW; ++st) tile.k[f][st] = *(const u32x4*)(kp + k_lane + st * 64);
      }
    };
    auto load_values = [&](Tile& tile, int k) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint8_t* vp = v_base + group_at(k, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_words<Tile::VW>(tile.v[4 * f + j], vp + v_lane[j]);
      }
    };
    auto scores = [&](Tile& tile, f32x4 (&s)[NF][2]) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int n = 0; n < NF; ++n) s[n][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < KS; ++st) {
          bf16x8 kf;
          if constexpr (FP8) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              w[2 * i] = e4m3_bf16<false>(tile.k[f][st >> 1][(st & 1) * 2 + i]);
              w[2 * i + 1] = e4m3_bf16<true>(tile.k[f][st >> 1][(st & 1) * 2 + i]);
            }
            kf = __builtin_bit_cast(bf16x8, w);
          } else {
            kf = __builtin_bit_cast(bf16x8, tile.k[f][st]);
          }
#pragma unroll
          for (int n = 0; n < NF; ++n) s[n][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[n][st], s[n][f], 0, 0, 0);
        }
      }
    };
    // softmax step and second product
    auto values = [&](Tile& tile, f32x4 (&s)[NF][2], int k, bool gap0, bool gap1) {
      const int at = wave + k * kDecodeWaves;
      const bool partly = at < seen_from || at >= seen_to;
      if (gap0 || gap1 || partly) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = at * kDecodeTile + 16 * f + 4 * g + j;
            const bool held = !(f ? gap1 : gap0) & (key < keys) & (key >= low);
#pragma unroll
            for (int n = 0; n < NF; ++n) {
              const bool seen = held & (key <= row_pos[n]) & (key >= row_low[n]);
              s[n][f][j] = seen ? s[n][f][j] : -INFINITY;
            }
            // what lies in unwritten or foreign places may be NaN, and 0 * NaN is not 0
#pragma unroll
            for (int w = 0; w < Tile::VW; ++w) {
              const uint32_t x = held ? tile.v[4 * f + j][w] : 0u, finite = finite_only<FP8>(x);
              odd |= partly && finite != x;
              tile.v[4 * f + j][w] = partly ? finite : x;
            }
          }
      }
      bf16x8 p[NF];
#pragma unroll
      for (int n = 0; n < NF; ++n) {
        float top = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                          fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
        // The maximum may lag behind by a factor of 2^8, which costs no precision: O
        // is scaled anew only when it does not suffice any more.
        if (__any(c * (top - m[n]) > 8.f || (m[n] == -INFINITY && top > m[n]))) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float to = fmaxf(m[n], top);
          const float by = m[n] == to ? 1.f : m[n] == -INFINITY ? 0.f : exp2_fast(c * (m[n] - to));
          m[n] = to;
          l[n] *= by;
#pragma unroll
          for (int i = 0; i < DV; ++i) o[n][i] *= by;
        }
        const float ref = m[n] == -INFINITY ? 0.f : c * m[n];
        u32x4 w;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = exp2_fast(fmaf(s[n][f][j], c, -ref));
          l[n] += (e[0] + e[1]) + (e[2] + e[3]);
          // P in bf16, the matrix instruction's type with V: 2^-8 relative a term at most, averaged over the keys
          w[2 * f] = pack_bf16(e[0], e[1]);
          w[2 * f + 1] = pack_bf16(e[2], e[3]);
        }
        p[n] = __builtin_bit_cast(bf16x8, w);
      }
#pragma unroll
      for (int i4 = 0; i4 < DV / 4; ++i4) {
        u32x4 vt[4];   // A operands of columns 4 i4 .. 4 i4 + 3
        if constexpr (FP8) {
          uint32_t b[2][4];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint32_t x0 = tile.v[4 * f][i4], x1 = tile.v[4 * f + 1][i4], x2 = tile.v[4 * f + 2][i4], x3 = tile.v[4 * f + 3][i4];
            const uint32_t a01 = __builtin_amdgcn_perm(x1, x0, 0x05010400u), b01 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
            const uint32_t a23 = __builtin_amdgcn_perm(x3, x2, 0x05010400u), b23 = __builtin_amdgcn_perm(x3, x2, 0x07030602u);
            b[f][0] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
            b[f][1] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
            b[f][2] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
            b[f][3] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vt[i] = u32x4{e4m3_bf16<false>(b[0][i]), e4m3_bf16<true>(b[0][i]), e4m3_bf16<false>(b[1][i]), e4m3_bf16<true>(b[1][i])};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              vt[i][j] = __builtin_amdgcn_perm(tile.v[2 * j + 1][2 * i4 + (i >> 1)], tile.v[2 * j][2 * i4 + (i >> 1)],
                                               (i & 1) ? 0x07060302u : 0x05040100u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < NF; ++n)
            o[n][4 * i4 + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vt[i]), p[n], o[n][4 * i4 + i], 0, 0, 0);
      }
    };

    // a tile's keys are loaded once the tile before has given its scores, its
    // values once the products with the values before are done
    Tile tile;
    const int mine = (n - wave + kDecodeWaves - 1) >> 2;   // tiles of this wave
    if (mine > 0) {
      locate(0);
      load_keys(tile, 0);
      load_values(tile, 0);
      for (int k = 0; k < mine; ++k) {
        const bool gap0 = without[0] >> (k & 63) & 1, gap1 = without[1] >> (k & 63) & 1;
        f32x4 s[NF][2];
        scores(tile, s);
        const bool more = k + 1 < mine;
        if (more) {
          if (((k + 1) & 63) == 0) locate(k + 1);
          load_keys(tile, k + 1);
        }
        values(tile, s, k, gap0, gap1);
        if (more) load_values(tile, k + 1);
      }
    }

    // what a row of the part sees of them, four columns at d (rare, and slow)
    auto add_odd = [&](int row, int d, f32x4 x) {
      const int pos = max(pos0 + div_group(a, row), -1), row_end = min(min(keys, pos + 1 - origin), n * kDecodeTile);
      for (int key = max(max(low_of(a, pos) - origin, low), 0); key < row_end; ++key) {
        if (key >> 5 >= seen_from && key >> 5 < seen_to) {   // seen by every row: nothing was taken out
          key = seen_to * kDecodeTile - 1;
          continue;
        }
        const uint32_t page = (uint32_t)table[(uint32_t)(origin + key) >> a.cache.page_shift];
        if (page >= num_pages) continue;
        const int64_t token = (int64_t)((uint64_t)page * page_units << 4) + (uint32_t)((origin + key) & page_mask) * row_bytes;
        x = add_not_finite<FP8>(x, v_base + token + d * EB, 1.f);
      }
      return x;
    };

    // join the waves in their order, 16 rows at a time
    const float vs = a.cache.v_scale ? a.cache.v_scale[head] : 1.f;
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      float ls = l[n];
      ls += __shfl_xor(ls, 16);
      ls += __shfl_xor(ls, 32);
      __syncthreads();   // the buffers of the fragment or item before have been read
      if (lane == 0) not_finite[wave] = 0;
      if (odd) not_finite[wave] = 1;
      if (g == 0) ml_part[wave][c16] = make_float2(m[n] == -INFINITY ? -INFINITY : c * m[n], ls);
#pragma unroll
      for (int rr = 0; rr < 4; ++rr)
#pragma unroll
        for (int i = 0; i < DV; i += 4)
          *(f32x4*)&o_part[wave][c16][(4 * g + rr) * DV + i] = f32x4{o[n][i][rr], o[n][i + 1][rr], o[n][i + 2][rr], o[n][i + 3][rr]};
      __syncthreads();
      for (int e = tid; e < 16 * D / 4; e += kThreads) {
        const int row = e / (D / 4), d = (e % (D / 4)) * 4, at = n * 16 + row;
        if (at >= nrows) continue;
        float top = -INFINITY, den = 0.f;
        f32x4 num = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) top = fmaxf(top, ml_part[w][row].x);
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) {
          const float2 ml = ml_part[w][row];
          const float by = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
          den = fmaf(by, ml.y, den);
          const f32x4 ow = *(const f32x4*)&o_part[w][row][d];
#pragma unroll
          for (int i = 0; i < 4; ++i) num[i] = fmaf(by, ow[i], num[i]);
        }
        if (not_finite[0] | not_finite[1] | not_finite[2] | not_finite[3]) num = add_odd(at, d, num);
        if (whole) {
          write_row<D>(a, it.l.start, head, at, d, top, den, num, vs);
        } else {
          const int64_t slot = ((int64_t)blockIdx.x * 2 + part) * kDecodeRows + at;
          store_shared(ws.o + slot * D + d, num[0], num[1]);
          store_shared(ws.o + slot * D + d + 2, num[2], num[3]);
          if (d == 0) store_shared((float*)&ws.ml[slot], top, den);
        }
      }
    }
    if (whole) continue;

    // the item's parts lie in workgroups g0 .. g1; every one counts itself at g0,
    // in whose share no other item can begin and go on
    const int64_t x0 = x - n - first;
    const int g0 = uniform((int)div_f64(x0, per)), g1 = uniform((int)div_f64(x0 + it.tiles - 1, per));
    // Parts are written and read as device-scope atomics, which pass the L2 that an XCD
    // keeps for itself, so that a part is where every XCD sees it once its stores are
    // acknowledged (the wait), and no cache has to be written back or invalidated: a
    // release and an acquire of the device cost 30 us of the drafts' 140.
    wait_stores();
    __syncthreads();
    if (tid == 0) last_part = __hip_atomic_fetch_add(&ws.arrived[g0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(g1 - g0);
    __syncthreads();
    if (!last_part) continue;
    for (int e = tid; e < nrows * (D / 4); e += kThreads) {
      const int at = e / (D / 4), d = (e % (D / 4)) * 4;
      // workgroup g's part is its first unless the item starts inside g's share
      auto slot_of = [&](int wg) { return (int64_t)(wg * 2 + (x0 > wg * per ? 1 : 0)) * kDecodeRows + at; };
      float den;
      f32x4 num;
      const float top = join_parts<D, true>(ws.ml, ws.o, slot_of, g0, g1, d, &den, &num);
      write_row<D>(a, it.l.start, head, at, d, top, den, num, vs);
    }
    if (tid == 0) ws.arrived[g0] = 0;   // for the next call
  }
  clear_padding(a, padding);
}

size_t attention_decode_workspace(int dim) {
  const DecodeWorkspace w = decode_workspace(nullptr);
  return (size_t)(uintptr_t)w.o - kArrivedBytes + (size_t)2 * kDecodeGrid * kDecodeRows * dim * sizeof(float);
}

namespace {

template <int D, bool FP8>
hipError_t launch(const AttentionArgs& a, hipStream_t st) {
  // rows a request may have here: one fragment of 16 or two
  const int64_t rows = min(a.max_new, (int64_t)(kDecodeRows / a.group)) * a.group;
  const unsigned grid = decode_grid(D);
  if (rows <= 16)
    attention_decode_kernel<D, FP8, 1><<<grid, kThreads, 0, st>>>(a);
  else
    attention_decode_kernel<D, FP8, 2><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_decode(const AttentionArgs& a, hipStream_t st) {
  switch (a.cache.dim) {
    case 64: return a.cache.fp8 ? launch<64, true>(a, st) : launch<64, false>(a, st);
    case 128: return a.cache.fp8 ? launch<128, true>(a, st) : launch<128, false>(a, st);
    default: return a.cache.fp8 ? launch<256, true>(a, st) : launch<256, false>(a, st);
  }
}

}  // namespace nvfp4
