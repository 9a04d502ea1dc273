// Verification of drafted tokens against the target's probabilities on gfx950.
//
// Per request, with target probabilities p_i = softmax(logits_i / T) and draft
// probabilities q_i (one at the draft where none are given): draft i is kept
// while u_i q_i(d_i) < p_i(d_i); after a kept drafts the next token is drawn
// from w = max(p_a - q_a, 0) (p_a if every draft was kept, or if w is zero
// everywhere) as argmax_v of w_v / E_v (-1 where w_v is 0).  With E_v standard
// exponential that argmax is v with probability w_v / sum w (a race of
// exponential clocks), it needs no running sum over the vocabulary, and so no
// order of summation can change the token: parts of the vocabulary are searched
// independently.
//
// Bound by HBM at batch sizes: every logit row is read once for its maximum,
// its argument and its sum of exponentials (verify_rows_kernel), then one row a
// request again, with the draft row and the noise (verify_draw_kernel, whose
// last workgroup of a request joins its slices).  A row is cut into slices so
// that a single request still fills the chip; the parts' order is fixed.  A
// thread takes 32 logits at a time: their loads are in flight together, and the
// running maximum and sum are touched once for all of them.  Exponentials are
// 2^((x - top) k), k = log2 e / T (not x k - top k: logits may be the type's
// lowest value, whose product overflows).  A score's relative error is p's, about
// 2^-22 + 2^-23 |x - top| k (the exponential, and three roundings of its argument), times
// p / w where a draft's probability is taken off, and the 2^-23 of the noise's hardware
// reciprocal: words are misjudged only against others whose scores lie that close.
//
// Measured: 64 requests of four drafts with their probabilities over 131072 words: 39 us.
// The rows take 19 of them, 3.4 TB/s: a workgroup has one batch of loads, then reduces
// with none in flight (waves wait for 52% of their cycles); the draw takes 18, 4.6 TB/s
// of what it reads (73 of its 84 MB from HBM: part of the drawn row is still in a cache);
// 7 requests of seven drafts over 100003 fp32 words 17.6 us, one request of three over
// 32768 15.1: two launches and the chain from rows to draw.
#include <float.h>
#include <hip/hip_runtime.h>

#include <type_traits>

#include "serving.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;              // vectors of 8 logits that a thread has in flight
constexpr int64_t kSlice = 8192;      // elements of a slice at least: one batch a thread
constexpr int kMaxSlices = 64;        // one a lane of the joins
constexpr int kMaxRequests = 65536;   // counters, at one place whatever a call's sizes
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct RowPart {
  float top, sum;      // largest logit and sum of exp((logit - top) / T)
  int32_t at, pad;     // its lowest index
};
struct DrawPart {
  float score;
  int32_t at, any, pad;   // any: a weight is positive
};
struct VerifyWorkspace {
  uint32_t* arrived;   // [kMaxRequests] slices that have been left of a request; 0 between calls
  RowPart* rows;       // [requests][max_drafts + 1][slices]
  DrawPart* draws;     // [requests][slices]
};
__host__ __device__ inline VerifyWorkspace verify_workspace(void* ws, int64_t requests, int64_t max_drafts, int slices) {
  VerifyWorkspace w;
  w.arrived = (uint32_t*)ws;
  w.rows = (RowPart*)(w.arrived + kMaxRequests);
  w.draws = (DrawPart*)(w.rows + requests * (max_drafts + 1) * slices);
  return w;
}

// Slices of a row: of one batch a thread while the rows alone do not give ten
// workgroups a CU, then fewer and longer ones.  Aiming at 2560 workgroups, against 640
// and 10240: 64 requests of four drafts over 131072 words 38 us, 51, 41; 256 of two 91,
// 109, 115; 7 of seven over 100003 17.5, 19.2, 17.2.  Slices of 2048 at least instead
// of 8192: 38, 90, 21.
int verify_slices(int64_t requests, int64_t max_drafts, int64_t vocab) {
  const int64_t most = (vocab + kSlice - 1) / kSlice, rows = requests * (max_drafts + 1);
  const int64_t n = min(most, max((2560 + rows - 1) / max(rows, (int64_t)1), (int64_t)1));
  return (int)min(n, (int64_t)kMaxSlices);
}
// Elements of a slice: whole vectors, so that aligned rows stay aligned.
__device__ __forceinline__ int64_t slice_length(int64_t vocab, int slices) { return ((vocab + slices - 1) / slices + 63) / 64 * 64; }

// Four or eight neighbouring elements; rows may start at any element.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32>
__device__ __forceinline__ void load8(float (&x)[8], const void* row, int64_t v) {
  if constexpr (F32) {
    const f32x4u a = *(const f32x4u*)((const float*)row + v), b = *(const f32x4u*)((const float*)row + v + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  } else {
    const u32x4u a = *(const u32x4u*)((const uint16_t*)row + v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(a[i] << 16), x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
template <bool F32>
__device__ __forceinline__ float load1(const void* row, int64_t v) {
  return F32 ? ((const float*)row)[v] : __uint_as_float((uint32_t)((const uint16_t*)row)[v] << 16);
}

// NaN counts as -inf.
__device__ __forceinline__ float clean(float logit) { return fmaxf(logit, -INFINITY); }
// exp((x - top) / T), k = log2 e / T; 0 if nothing has a probability
__device__ __forceinline__ float term(float x, float top, float k) {
  return top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((x - top) * k);
}

struct Best {
  float score;
  int32_t at;
};
// The larger score, the lower index among equals.
__device__ __forceinline__ Best better(Best a, Best b) {
  return b.score > a.score || (b.score == a.score && b.at < a.at) ? b : a;
}
__device__ __forceinline__ Best wave_best(Best b) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    Best o;
    o.score = __shfl_xor(b.score, d);
    o.at = __shfl_xor(b.at, d);
    b = better(b, o);
  }
  return b;
}

__device__ __forceinline__ float temperature_of(const VerifyArgs& a, int64_t r, bool* greedy) {
  const float t = a.temperature ? a.temperature[r] : 1.f;
  *greedy = t == 0.f;
  return t == 0.f ? 1.f : t;
}
// log2 e / T, finite: below T = 4e-39 every logit but the largest is out of reach anyway
__device__ __forceinline__ float scale_of(float t) {
  const float k = kLog2e / t;
  return k > FLT_MAX ? FLT_MAX : k;   // a NaN stays one: nothing is sampled
}
// Drafts of a request; -1: nothing to sample.  Its rows have to lie in the logits.
__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int64_t r) {
  const int64_t n = min((int64_t)a.num_drafts[r], a.max_drafts), first = a.row_start[r];
  return n < 0 || first < 0 || first + n >= a.rows ? -1 : (int)n;
}
template <bool F32>
__device__ __forceinline__ const void* logits_row(const VerifyArgs& a, int64_t r, int64_t i) {
  const int64_t at = (a.row_start[r] + i) * a.ld_logits;
  return F32 ? (const void*)((const float*)a.logits + at) : (const void*)((const uint16_t*)a.logits + at);
}

}  // namespace

// Grid (slices, max_drafts + 1, requests): a slice of one row.
template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_rows_kernel(VerifyArgs a, VerifyWorkspace ws) {
  const int slices = gridDim.x, slice = blockIdx.x, i = blockIdx.y, tid = threadIdx.x;
  const int64_t r = blockIdx.z;
  const int n = drafts_of(a, r);
  if (i > n) return;
  bool greedy;
  const float k = scale_of(temperature_of(a, r, &greedy));
  const void* row = logits_row<F32>(a, r, i);
  const int64_t each = slice_length(a.vocab, slices), v0 = min(slice * each, a.vocab), v1 = min(v0 + each, a.vocab);
  float top = -INFINITY, sum = 0.f;
  int32_t at = INT32_MAX;
  for (int64_t base = v0; base < v1; base += kBatch * kThreads * 8) {
    float x[kBatch][8];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t v = base + (b * kThreads + tid) * 8;
      if (v + 8 <= v1) {
        load8<F32>(x[b], row, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[b][j] = v + j < v1 ? load1<F32>(row, v + j) : -INFINITY;
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, x[b][j]);
    if (m > top) {
      sum *= term(top, m, k);   // 0 before the first
      top = m;
#pragma unroll
      for (int b = kBatch - 1; b >= 0; --b)   // a thread's elements rise with b and j
#pragma unroll
        for (int j = 7; j >= 0; --j)
          if (x[b][j] == m) at = (int32_t)(base + (b * kThreads + tid) * 8 + j);
    }
    if (top > -INFINITY) {
      float e[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        e[b] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) e[b] += __builtin_amdgcn_exp2f((clean(x[b][j]) - top) * k);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) sum += e[b];
    }
  }
  __shared__ RowPart part[kThreads / 64];
  float m = top;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  sum *= term(top, m, k);
  if (top != m) at = INT32_MAX;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    sum += __shfl_xor(sum, d);
    at = min(at, __shfl_xor(at, d));
  }
  if ((tid & 63) == 0) part[tid >> 6] = RowPart{m, sum, at, 0};
  __syncthreads();
  if (tid == 0) {
    RowPart p = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) {
      const RowPart o = part[w];
      const float to = fmaxf(p.top, o.top);
      p.sum = p.sum * term(p.top, to, k) + o.sum * term(o.top, to, k);
      p.at = p.top == o.top ? min(p.at, o.at) : p.top == to ? p.at : o.at;
      p.top = to;
    }
    ws.rows[(r * (a.max_drafts + 1) + i) * slices + slice] = p;
  }
}

namespace {

// Every row's statistics (into LDS, [256]) and the number of drafts kept, by the
// whole workgroup: a wave joins a row's slices, a slice a lane, in a fixed order.
template <bool F32>
__device__ int accept(const VerifyArgs& a, const VerifyWorkspace& ws, int64_t r, int n, int slices, float k, bool greedy,
                      RowPart* rows) {
  __shared__ int kept;
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid == 0) kept = n;
  for (int i = tid >> 6; i <= n; i += kThreads / 64) {
    RowPart p = {-INFINITY, 0.f, INT32_MAX, 0};
    if (lane < slices) p = ws.rows[(r * (a.max_drafts + 1) + i) * slices + lane];
    float m = p.top;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    p.sum *= term(p.top, m, k);
    if (p.top != m) p.at = INT32_MAX;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      p.sum += __shfl_xor(p.sum, d);
      p.at = min(p.at, __shfl_xor(p.at, d));
    }
    if (lane == 0) rows[i] = RowPart{m, p.sum, p.at, 0};
  }
  // thread i: draft i (its loads do not wait for the joins)
  int32_t d = -1;
  float x = 0.f, uq = 0.f;
  if (tid < n) {
    d = a.draft_tokens[r * a.max_drafts + tid];
    if (d >= 0 && d < a.vocab && !greedy) {
      x = clean(load1<F32>(logits_row<F32>(a, r, tid), d));
      uq = a.uniform[r * a.max_drafts + tid] * (a.draft_probs ? a.draft_probs[(r * a.max_drafts + tid) * a.ld_probs + d] : 1.f);
    }
  }
  __syncthreads();
  if (tid < n) {
    const RowPart p = rows[tid];
    const bool inside = d >= 0 && d < a.vocab;
    const bool ok = inside && (greedy ? d == p.at : p.sum > 0.f && uq < term(x, p.top, k) / p.sum);
    if (!ok) atomicMin(&kept, tid);   // a minimum: the order does not matter
  }
  __syncthreads();
  return kept;
}

// The race over words [v0, v1) of a row by the whole workgroup; q and refused: what
// is taken off (null, -1: nothing).  All threads have the result.
template <bool F32>
__device__ DrawPart race(const void* row, const RowPart& p, float k, const float* q, int32_t refused, const float* noise,
                         int64_t v0, int64_t v1) {
  __shared__ Best part[kThreads / 64];
  __shared__ int part_any[kThreads / 64];
  const int tid = threadIdx.x;
  const float inv = p.sum > 0.f ? 1.f / p.sum : 0.f, top = p.top == -INFINITY ? 0.f : p.top;
  Best best = {-INFINITY, INT32_MAX};
  bool any = false;
  auto take = [&](float x, float qv, float e, int32_t v) {   // v rises: the first of equals stays
    const float w = __builtin_amdgcn_exp2f((clean(x) - top) * k) * inv - qv;
    const float score = w > 0.f ? w * __builtin_amdgcn_rcpf(e) : -1.f;
    any |= w > 0.f;
    best.at = score > best.score ? v : best.at;
    best.score = fmaxf(best.score, score);
  };
  auto run = [&](auto taken) {   // 0: nothing, 1: q, 2: one word
    constexpr int kTaken = decltype(taken)::value;
    constexpr int B = kBatch / 2;
    const int vectors = (int)((v1 - v0) >> 3);
    for (int base = 0; base < vectors; base += B * kThreads) {
      float x[B][8], e[B][8], qv[B][8];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int64_t v = v0 + 8 * (int64_t)min(base + b * kThreads + tid, vectors - 1);   // beyond: the last again, not taken
        load8<F32>(x[b], row, v);
        load8<true>(e[b], noise, v);
        if (kTaken == 1) load8<true>(qv[b], q, v);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int i = base + b * kThreads + tid;
        if (i < vectors) {
          const int32_t v = (int32_t)(v0 + 8 * (int64_t)i);
#pragma unroll
          for (int j = 0; j < 8; ++j) take(x[b][j], kTaken == 1 ? qv[b][j] : kTaken == 2 && v + j == refused ? 1.f : 0.f, e[b][j], v + j);
        }
      }
    }
    const int64_t v = v0 + 8 * (int64_t)vectors + tid;   // what is left of a vector
    if (v < v1) take(load1<F32>(row, v), kTaken == 1 ? q[v] : kTaken == 2 && v == refused ? 1.f : 0.f, noise[v], (int32_t)v);
  };
  if (q) run(std::integral_constant<int, 1>{});
  else if (refused >= 0) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 0>{});
  best = wave_best(best);
  const int some = __any(any);
  if ((tid & 63) == 0) {
    part[tid >> 6] = best;
    part_any[tid >> 6] = some;
  }
  __syncthreads();
  best = part[0];
  int all = part_any[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) {
    best = better(best, part[w]);
    all |= part_any[w];
  }
  __syncthreads();
  return DrawPart{best.score, best.at, all, 0};
}

}  // namespace

// Grid (slices, requests): the race over a slice of the row after the kept drafts,
// and by the last slice to arrive (or the first, where there is nothing to draw) the
// tokens, their count and their log-probabilities.
template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, VerifyWorkspace ws) {
  __shared__ RowPart rows[kThreads];
  __shared__ int last_slice;
  const int slices = gridDim.x, slice = blockIdx.x, i = threadIdx.x;
  const int64_t r = blockIdx.y, out = r * (a.max_drafts + 1) + i;
  const int n = drafts_of(a, r);
  if (n < 0) {
    if (slice > 0) return;
    if (i <= a.max_drafts) {
      a.out_tokens[out] = -1;
      a.logprobs[out] = 0.f;
    }
    if (i == 0) a.num_accepted[r] = 0;
    return;
  }
  bool greedy;
  const float t = temperature_of(a, r, &greedy), k = scale_of(t);
  if (greedy && slice > 0) return;   // the argument of the maximum is known
  const int kept = accept<F32>(a, ws, r, n, slices, k, greedy, rows);
  DrawPart d = {-INFINITY, INT32_MAX, 0, 0};
  if (!greedy) {
    const bool rest = kept < n;      // a draft was refused: draw from what it leaves
    const void* row = logits_row<F32>(a, r, kept);
    const float* noise = a.noise + r * a.ld_noise;
    const int64_t each = slice_length(a.vocab, slices), v0 = min(slice * each, a.vocab), v1 = min(v0 + each, a.vocab);
    d = race<F32>(row, rows[kept], k, rest && a.draft_probs ? a.draft_probs + (r * a.max_drafts + kept) * a.ld_probs : nullptr,
                  rest && !a.draft_probs ? a.draft_tokens[r * a.max_drafts + kept] : -1, noise, v0, v1);
    if (slices > 1) {
      // Slices are left and read as device-scope atomics, which pass the L2 that an XCD
      // keeps for itself: a slice is where every XCD sees it once its stores are
      // acknowledged (the wait).
      if (i == 0) {
        uint64_t* to = (uint64_t*)(ws.draws + r * slices + slice);
        __hip_atomic_store(to, (uint64_t)(uint32_t)d.at << 32 | __float_as_uint(d.score), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(to + 1, (uint64_t)d.any, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        last_slice = __hip_atomic_fetch_add(&ws.arrived[r], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(slices - 1);
      }
      __syncthreads();
      if (!last_slice) return;
      if (i == 0) ws.arrived[r] = 0;   // for the next call
      d = DrawPart{-INFINITY, INT32_MAX, 0, 0};
      if ((i & 63) < slices) {         // every wave joins the slices, a slice a lane
        const uint64_t* from = (const uint64_t*)(ws.draws + r * slices + (i & 63));
        const uint64_t v = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        d.score = __uint_as_float((uint32_t)v);
        d.at = (int32_t)(v >> 32);
        d.any = (int32_t)__hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      const Best b = wave_best(Best{d.score, d.at});
      d = DrawPart{b.score, b.at, __any(d.any), 0};
    }
    // a refused draft that leaves nothing (p = q up to rounding): p in its place
    if (!d.any && rest) d = race<F32>(row, rows[kept], k, nullptr, -1, noise, 0, a.vocab);
  }
  if (i == 0) a.num_accepted[r] = kept;
  if (i > a.max_drafts) return;
  int32_t token = -1;
  if (i < kept) token = a.draft_tokens[r * a.max_drafts + i];
  if (i == kept) token = greedy ? (rows[i].at == INT32_MAX ? -1 : rows[i].at) : d.any ? d.at : -1;
  float lp = 0.f;
  if (token >= 0) {
    const float x = clean(load1<F32>(logits_row<F32>(a, r, i), token));
    lp = (x - rows[i].top) / t - kLn2 * __builtin_amdgcn_logf(rows[i].sum);
  }
  a.out_tokens[out] = token;
  a.logprobs[out] = lp;
}

// Enough for any smaller call too: rows times slices is below 2560 + rows while there
// are several slices, and the rows themselves after that.
size_t verify_workspace_bytes(int64_t requests, int64_t max_drafts, int64_t vocab) {
  const int64_t rows = requests * (max_drafts + 1), most = min((vocab + kSlice - 1) / kSlice, (int64_t)kMaxSlices);
  const int64_t parts = max(rows, min(rows * most, (int64_t)2 * 2560));
  return kMaxRequests * sizeof(uint32_t) + parts * (sizeof(RowPart) + sizeof(DrawPart)) + 16;
}

namespace {

template <bool F32>
hipError_t launch(const VerifyArgs& a, hipStream_t st) {
  const int slices = verify_slices(a.requests, a.max_drafts, a.vocab);
  const VerifyWorkspace ws = verify_workspace(a.workspace, a.requests, a.max_drafts, slices);
  verify_rows_kernel<F32><<<dim3(slices, (unsigned)a.max_drafts + 1, (unsigned)a.requests), kThreads, 0, st>>>(a, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_draw_kernel<F32><<<dim3(slices, (unsigned)a.requests), kThreads, 0, st>>>(a, ws);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_drafts(const VerifyArgs& a, hipStream_t st) {
  return a.logits_f32 ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace nvfp4
