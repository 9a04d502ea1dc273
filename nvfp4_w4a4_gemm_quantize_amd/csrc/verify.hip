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
// request again, with the draft row and the noise (verify_draw_kernel), then
// the parts are joined (verify_join_kernel).  A row is cut into slices so
// that a single request still fills the chip; the parts' order is fixed.
#include <hip/hip_runtime.h>

#include "serving.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kSlice = 8192;      // elements of a slice at least: 32 a thread

struct RowPart {
  float top, sum;      // largest x (x = logit / T) and sum of exp(x - top)
  int32_t at, pad;     // its lowest index
};
struct DrawPart {
  float score;
  int32_t at, any, pad;   // any: a weight is positive
};
struct VerifyWorkspace {
  RowPart* rows;       // [requests][max_drafts + 1][slices]
  DrawPart* draws;     // [requests][slices][2]: from w, and from p in its place
};
__host__ __device__ inline VerifyWorkspace verify_workspace(void* ws, int64_t requests, int64_t max_drafts, int slices) {
  VerifyWorkspace w;
  w.rows = (RowPart*)ws;
  w.draws = (DrawPart*)(w.rows + requests * (max_drafts + 1) * slices);
  return w;
}

int verify_slices(int64_t vocab) {
  const int64_t n = (vocab + kSlice - 1) / kSlice;
  return (int)(n < 1 ? 1 : n > 64 ? 64 : n);
}

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

// A logit as x = logit / T; NaN counts as -inf.
__device__ __forceinline__ float scaled(float logit, float t) { return fmaxf(logit, -INFINITY) / t; }

__device__ __forceinline__ float softmax_term(float x, float top) { return top == -INFINITY ? 0.f : __expf(x - top); }

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
  const float t = temperature_of(a, r, &greedy);
  const void* row = logits_row<F32>(a, r, i);
  const int64_t each = (a.vocab + slices - 1) / slices, v0 = slice * each, v1 = min(v0 + each, a.vocab);
  float top = -INFINITY, sum = 0.f;
  int32_t at = INT32_MAX;
  auto take = [&](const float (&x)[8], int64_t v, int count) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, x[j]);
    if (m > top) {
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (x[j] == m) at = (int32_t)(v + j);
      sum *= top == -INFINITY ? 0.f : __expf(top - m);
      top = m;
    }
    float e = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) e += softmax_term(x[j], top);
    sum += e;
  };
  for (int64_t v = v0 + tid * 8; v < v1; v += kThreads * 8) {
    float x[8];
    if (v + 8 <= v1) {
      load8<F32>(x, row, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = scaled(x[j], t);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = v + j < v1 ? scaled(load1<F32>(row, v + j), t) : -INFINITY;
    }
    take(x, v, 8);
  }
  __shared__ RowPart part[kThreads / 64];
  float m = top;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  sum *= softmax_term(top, m);
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
      p.sum = p.sum * softmax_term(p.top, to) + o.sum * softmax_term(o.top, to);
      p.at = p.top == o.top ? min(p.at, o.at) : p.top == to ? p.at : o.at;
      p.top = to;
    }
    ws.rows[(r * (a.max_drafts + 1) + i) * slices + slice] = p;
  }
}

namespace {

// A row's slices joined in their order.
__device__ __forceinline__ RowPart join_row(const RowPart* parts, int slices) {
  RowPart p = parts[0];
  for (int s = 1; s < slices; ++s) {
    const RowPart o = parts[s];
    const float to = fmaxf(p.top, o.top);
    p.sum = p.sum * softmax_term(p.top, to) + o.sum * softmax_term(o.top, to);
    p.at = p.top == o.top ? min(p.at, o.at) : p.top == to ? p.at : o.at;
    p.top = to;
  }
  return p;
}

// Every row's statistics and the number of drafts kept, by the whole workgroup
// (thread i: row i).  rows: LDS [256].
template <bool F32>
__device__ int accept(const VerifyArgs& a, const VerifyWorkspace& ws, int64_t r, int n, int slices, float t, bool greedy,
                      RowPart* rows) {
  __shared__ int kept;
  const int i = threadIdx.x;
  if (i == 0) kept = n;
  __syncthreads();
  if (i <= n) {
    const RowPart p = join_row(ws.rows + (r * (a.max_drafts + 1) + i) * slices, slices);
    rows[i] = p;
    if (i < n) {
      const int32_t d = a.draft_tokens[r * a.max_drafts + i];
      bool ok = d >= 0 && d < a.vocab;
      if (ok && greedy) {
        ok = d == p.at;
      } else if (ok) {
        const float x = scaled(load1<F32>(logits_row<F32>(a, r, i), d), t);
        const float pd = p.sum > 0.f ? softmax_term(x, p.top) / p.sum : 0.f;
        const float qd = a.draft_probs ? a.draft_probs[(r * a.max_drafts + i) * a.ld_probs + d] : 1.f;
        ok = a.uniform[r * a.max_drafts + i] * qd < pd;
      }
      if (!ok) atomicMin(&kept, i);   // a minimum: the order does not matter
    }
  }
  __syncthreads();
  return kept;
}

}  // namespace

// Grid (slices, requests): the race over a slice of the row after the kept drafts.
template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, VerifyWorkspace ws) {
  __shared__ RowPart rows[kThreads];
  __shared__ Best part[2][kThreads / 64];
  __shared__ int part_any[2][kThreads / 64];
  const int slices = gridDim.x, slice = blockIdx.x, tid = threadIdx.x;
  const int64_t r = blockIdx.y;
  const int n = drafts_of(a, r);
  if (n < 0) return;
  bool greedy;
  const float t = temperature_of(a, r, &greedy);
  if (greedy) return;   // the argument of the maximum is known
  const int kept = accept<F32>(a, ws, r, n, slices, t, greedy, rows);
  const RowPart p = rows[kept];
  const void* row = logits_row<F32>(a, r, kept);
  const bool rest = kept < n;   // a draft was refused: draw from what it leaves
  const float* q = rest && a.draft_probs ? a.draft_probs + (r * a.max_drafts + kept) * a.ld_probs : nullptr;
  const int32_t refused = rest && !a.draft_probs ? a.draft_tokens[r * a.max_drafts + kept] : -1;
  const float* noise = a.noise + r * a.ld_noise;
  const int64_t each = (a.vocab + slices - 1) / slices, v0 = slice * each, v1 = min(v0 + each, a.vocab);
  // [0]: from w; [1]: from p in its place.  The first word of weight 0 stands for all of them.
  Best best[2] = {{-INFINITY, INT32_MAX}, {-INFINITY, INT32_MAX}};
  int32_t none[2] = {INT32_MAX, INT32_MAX};
  int any[2] = {0, 0};
  auto take = [&](float x, float qv, float e, int64_t v) {
    const float pv = p.sum > 0.f ? softmax_term(x, p.top) / p.sum : 0.f;
    const float w[2] = {pv - qv, pv};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (w[k] > 0.f) {
        best[k] = better(best[k], Best{w[k] / e, (int32_t)v});
        any[k] = 1;
      } else {
        none[k] = min(none[k], (int32_t)v);
      }
    }
  };
  for (int64_t v = v0 + tid * 8; v < v1; v += kThreads * 8) {
    float x[8], e[8], qv[8];
    if (v + 8 <= v1) {
      load8<F32>(x, row, v);
      load8<true>(e, noise, v);
      if (q) load8<true>(qv, q, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = v + j < v1;
        x[j] = in ? load1<F32>(row, v + j) : -INFINITY;
        e[j] = in ? noise[v + j] : 1.f;
        if (q) qv[j] = in ? q[v + j] : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v + j < v1) take(scaled(x[j], t), q ? qv[j] : v + j == refused ? 1.f : 0.f, e[j], v + j);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Best b = wave_best(none[k] == INT32_MAX ? best[k] : better(best[k], Best{-1.f, none[k]}));
    const int some = __any(any[k]);
    if ((tid & 63) == 0) {
      part[k][tid >> 6] = b;
      part_any[k][tid >> 6] = some;
    }
  }
  __syncthreads();
  if (tid < 2) {
    Best b = part[tid][0];
    int some = part_any[tid][0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) {
      b = better(b, part[tid][w]);
      some |= part_any[tid][w];
    }
    ws.draws[(r * slices + slice) * 2 + tid] = DrawPart{b.score, b.at, some, 0};
  }
}

// Grid (requests): the tokens, their count and their log-probabilities.
template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_join_kernel(VerifyArgs a, VerifyWorkspace ws, int slices) {
  __shared__ RowPart rows[kThreads];
  const int64_t r = blockIdx.x;
  const int i = threadIdx.x, n = drafts_of(a, r);
  const int64_t out = r * (a.max_drafts + 1) + i;
  if (n < 0) {
    if (i <= a.max_drafts) {
      a.out_tokens[out] = -1;
      a.logprobs[out] = 0.f;
    }
    if (i == 0) a.num_accepted[r] = 0;
    return;
  }
  bool greedy;
  const float t = temperature_of(a, r, &greedy);
  const int kept = accept<F32>(a, ws, r, n, slices, t, greedy, rows);
  if (i == 0) a.num_accepted[r] = kept;
  if (i > a.max_drafts) return;
  int32_t token = -1;
  if (i < kept) {
    token = a.draft_tokens[r * a.max_drafts + i];
  } else if (i == kept) {
    if (greedy) {
      token = rows[i].at;
    } else {
      Best left = {-INFINITY, INT32_MAX}, whole = left;
      int left_any = 0, whole_any = 0;
      for (int s = 0; s < slices; ++s) {
        const DrawPart* d = ws.draws + (r * slices + s) * 2;
        left = better(left, Best{d[0].score, d[0].at});
        whole = better(whole, Best{d[1].score, d[1].at});
        left_any |= d[0].any;
        whole_any |= d[1].any;
      }
      token = left_any ? left.at : whole_any ? whole.at : -1;
    }
    if (token == INT32_MAX) token = -1;   // nothing has a probability
  }
  float lp = 0.f;
  if (token >= 0) {
    const float x = scaled(load1<F32>(logits_row<F32>(a, r, i), token), t);
    lp = x - rows[i].top - __logf(rows[i].sum);
  }
  a.out_tokens[out] = token;
  a.logprobs[out] = lp;
}

size_t verify_workspace_bytes(int64_t requests, int64_t max_drafts, int64_t vocab) {
  const int slices = verify_slices(vocab);
  return (size_t)(uintptr_t)(verify_workspace(nullptr, requests, max_drafts, slices).draws + requests * slices * 2) + 16;
}

namespace {

template <bool F32>
hipError_t launch(const VerifyArgs& a, hipStream_t st) {
  const int slices = verify_slices(a.vocab);
  const VerifyWorkspace ws = verify_workspace(a.workspace, a.requests, a.max_drafts, slices);
  verify_rows_kernel<F32><<<dim3(slices, (unsigned)a.max_drafts + 1, (unsigned)a.requests), kThreads, 0, st>>>(a, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_draw_kernel<F32><<<dim3(slices, (unsigned)a.requests), kThreads, 0, st>>>(a, ws);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_join_kernel<F32><<<(unsigned)a.requests, kThreads, 0, st>>>(a, ws, slices);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_drafts(const VerifyArgs& a, hipStream_t st) {
  return a.logits_f32 ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace nvfp4
