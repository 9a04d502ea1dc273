// The bookkeeping of a paged serving step on gfx950: the plan (block tables
// and slot maps from request lengths) and the write of new K/V rows into the
// paged cache.  Declared and documented in include/nvfp4.h.
#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>

#include "serving.h"

namespace nvfp4 {

// ---------------------------------------------------------------- plan ----
//
// Two prefix sums over the requests: of their new tokens (q_start) and of the
// pages that they need beyond those that their context holds,
//   before_r = min(ceil(ctx_r / P), max_pages),
//   after_r  = min(ceil((ctx_r + new_r) / P), max_pages),
//   need_r   = after_r - before_r.
// The j-th page needed over all requests is free_pages[cursor + j], so a page
// is found from its request's prefix alone and no workgroup waits for another.
//
// One launch, bound by latency: every workgroup repeats the scan (8 bytes a
// request, from L2), which costs less than a second launch to share it (a launch takes
// the host 3.6 us; 8 requests of one token 3.1 us on the GPU, 1024 requests with 5000
// tokens 6.1); then
// tokens, pages and requests are dealt out over the whole grid.  A thread owns
// a run of ceil(R / 256) requests in the scan; a token finds its run by binary
// search in LDS and its request by walking the run.
//
// Every workgroup reads the lengths and the cursor at its own time, and twice, so
// nothing of that launch may write them.  A step in place (seq_lens is ctx_lens, or
// the cursor lies in counts) writes these two last where it has one workgroup (8
// requests of one token, replayed in a graph: 2.8 us, with separate tensors 2.7);
// otherwise a second launch of one workgroup does (1024 requests with 5000 tokens 7.8
// us, 3.8).  Inputs that share memory with outputs in any other way give wrong plans, but
// every walk ends with the requests and every column is checked, so nothing is read or
// written out of range.
constexpr int kPlanThreads = 256;

namespace {

enum PlanPart {
  kPlanAll,      // nothing in place
  kPlanOne,      // in place, one workgroup
  kPlanTables,   // all but seq_lens and counts
  kPlanCarry,    // these two, one workgroup
};

struct PlanLens {
  int64_t ctx, tokens, before, need;
};

__device__ __forceinline__ PlanLens plan_lens(const PlanArgs& a, int64_t r) {
  PlanLens l;
  l.ctx = max(a.ctx_lens[r], 0);
  l.tokens = max(a.new_lens[r], 0);
  const int64_t up = ((int64_t)1 << a.page_shift) - 1;
  l.before = min((l.ctx + up) >> a.page_shift, a.max_pages);
  l.need = min((l.ctx + l.tokens + up) >> a.page_shift, a.max_pages) - l.before;
  return l;
}

// The last run whose prefix is <= x (prefix[0] == 0 <= x).
__device__ __forceinline__ int plan_run(const int64_t* prefix, int64_t x) {
  int lo = 0;
#pragma unroll
  for (int step = kPlanThreads / 2; step > 0; step >>= 1)
    if (prefix[lo + step] <= x) lo += step;
  return lo;
}

}  // namespace

template <PlanPart PART>
__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(PlanArgs a) {
  __shared__ int64_t tok[kPlanThreads + 1], pg[kPlanThreads + 1];
  __shared__ int64_t wave_tok[kPlanThreads / 64], wave_pg[kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t run = (a.requests + kPlanThreads - 1) / kPlanThreads;
  const int64_t r0 = min(tid * run, a.requests), r1 = min(r0 + run, a.requests);
  int64_t st = 0, sp = 0;
  for (int64_t r = r0; r < r1; ++r) {
    const PlanLens l = plan_lens(a, r);
    st += l.tokens;
    sp += l.need;
  }
  int64_t it = st, ip = sp;   // inclusive scans over the wave, then over the waves
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t ut = __shfl_up(it, d), up = __shfl_up(ip, d);
    if (lane >= d) {
      it += ut;
      ip += up;
    }
  }
  if (lane == 63) {
    wave_tok[wave] = it;
    wave_pg[wave] = ip;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    it += wave_tok[w];
    ip += wave_pg[w];
  }
  if (tid == 0) tok[0] = pg[0] = 0;
  tok[tid + 1] = it;
  pg[tid + 1] = ip;
  __syncthreads();
  const int64_t total = tok[kPlanThreads], pages = pg[kPlanThreads];
  const int64_t cursor = a.free_cursor ? max(*a.free_cursor, 0) : 0;
  const int64_t left = max(a.num_free - cursor, (int64_t)0);
  const int64_t stride = (int64_t)gridDim.x * kPlanThreads, first = (int64_t)blockIdx.x * kPlanThreads + tid;

  // per page needed
  for (int64_t p = first; PART != kPlanCarry && p < pages; p += stride) {
    const int w = plan_run(pg, p);
    int64_t r = w * run, base = pg[w];
    PlanLens l = plan_lens(a, r);
    while (p >= base + l.need && r + 1 < a.requests) {   // p < pg[w + 1]
      base += l.need;
      l = plan_lens(a, ++r);
    }
    if (p - base < l.need) a.block_table[r * a.ld_table + l.before + (p - base)] = p < left ? a.free_pages[cursor + p] : -1;
  }
  // per token; the tail of the buffers is padding
  for (int64_t t = first; PART != kPlanCarry && t < a.max_tokens; t += stride) {
    int64_t pos = -1, slot = -1;
    if (t < total) {
      const int w = plan_run(tok, t);
      int64_t r = w * run, base = tok[w], pbase = pg[w];
      PlanLens l = plan_lens(a, r);
      while (t >= base + l.tokens && r + 1 < a.requests) {   // t < tok[w + 1]
        base += l.tokens;
        pbase += l.need;
        l = plan_lens(a, ++r);
      }
      pos = l.ctx + (t - base);
      const int64_t c = pos >> a.page_shift;
      if (c < a.max_pages) {
        const int64_t p = pbase + (c - l.before);   // pages of this step come from the free list, not through the table
        const int32_t page = c < l.before ? a.block_table[r * a.ld_table + c] : p < left ? a.free_pages[cursor + p] : -1;
        if (page >= 0) slot = ((int64_t)page << a.page_shift) + (pos & (((int64_t)1 << a.page_shift) - 1));
      }
    }
    a.positions[t] = (int32_t)pos;
    a.slots[t] = slot;
  }
  if (PART == kPlanOne) __syncthreads();
  // per request (a thread's run goes to one workgroup of the grid)
  if (tid % gridDim.x == blockIdx.x) {
    int64_t t = tok[tid];
    for (int64_t r = r0; r < r1; ++r) {
      const PlanLens l = plan_lens(a, r);
      if (PART != kPlanCarry) a.q_start[r] = (int32_t)min(t, a.max_tokens);
      if (PART != kPlanTables) a.seq_lens[r] = (int32_t)min(l.ctx + l.tokens, (int64_t)INT32_MAX);
      t += l.tokens;
    }
  }
  if (first == 0) {
    const int64_t taken = min(pages, left);
    if (PART != kPlanCarry) a.q_start[a.requests] = (int32_t)min(total, a.max_tokens);
    if (PART != kPlanTables) {
      a.counts[0] = (int32_t)min(total, (int64_t)INT32_MAX);
      a.counts[1] = (int32_t)taken;
      a.counts[2] = (int32_t)min(pages - taken, (int64_t)INT32_MAX);
      a.counts[3] = (int32_t)(cursor + taken);
    }
  }
}

hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t st) {
  // one token a thread up to 1024 workgroups (four a CU), then several
  const int64_t want = (max(a.max_tokens, a.requests) + kPlanThreads - 1) / kPlanThreads;
  const unsigned grid = (unsigned)min(max(want, (int64_t)1), (int64_t)1024);
  if (!a.in_place) {
    paged_plan_kernel<kPlanAll><<<grid, kPlanThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  if (grid == 1) {
    paged_plan_kernel<kPlanOne><<<1, kPlanThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  paged_plan_kernel<kPlanTables><<<grid, kPlanThreads, 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  paged_plan_kernel<kPlanCarry><<<1, kPlanThreads, 0, st>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------------ K/V write ----
//
// cache[slot / P, h, slot % P, :] = row, rounded for an E4M3 cache to nearest
// even of clamp(x / scale[h], +-448) (the clamp: E4M3 has no infinity, and a
// calibrated scale may be exceeded).  Bound by HBM: every thread moves 16 bytes
// of K and of V, the two loads in flight together; a token's row is contiguous
// on the way in, and per head on the way out.  Measured: 16384 tokens, 8 heads of 128,
// into E4M3: 22 us, 4.5 TB/s (a large copy moves 5.0); 64 decoded tokens 2.7 us.
namespace {

__device__ __forceinline__ float bf16_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ uint2 to_e4m3(uint4 x, float scale) {
  uint32_t in[4] = {x.x, x.y, x.z, x.w}, out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int w = 0;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = in[j * 2 + (i >> 1)];
      const float y = bf16_f32((i & 1) ? word >> 16 : word & 0xffffu) / scale;
      f[i] = y != y ? y : fminf(fmaxf(y, -448.f), 448.f);   // a NaN stays one
    }
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
    out[j] = (uint32_t)w;
  }
  return make_uint2(out[0], out[1]);
}

}  // namespace

template <bool FP8>
__global__ __launch_bounds__(256) void paged_kv_write_kernel(KvWriteArgs a, int tokens_per_block) {
  const CacheView& c = a.cache;
  const int per_token = c.heads * c.dim / 8;   // 16-byte pieces of a row
  const int64_t t0 = (int64_t)blockIdx.x * tokens_per_block;
  const int dim_shift = 31 - __builtin_clz(c.dim);
  for (int i = threadIdx.x; i < tokens_per_block * per_token; i += 256) {
    const int dt = i / per_token, e = (i - dt * per_token) * 8;
    const int64_t t = t0 + dt;
    if (t >= a.tokens) return;
    const int64_t slot = a.slots[t], page = slot >> c.page_shift;
    if (slot < 0 || page >= c.num_pages) continue;
    const uint4 k = *(const uint4*)(a.k + t * a.ld_k + e), v = *(const uint4*)(a.v + t * a.ld_v + e);
    const int h = e >> dim_shift, d = e & (c.dim - 1);
    const int64_t at = page * c.page_stride + h * c.head_stride +
                       (slot & (((int64_t)1 << c.page_shift) - 1)) * c.token_stride + d;
    if (FP8) {
      *(uint2*)((uint8_t*)c.k + at) = to_e4m3(k, c.k_scale ? c.k_scale[h] : 1.f);
      *(uint2*)((uint8_t*)c.v + at) = to_e4m3(v, c.v_scale ? c.v_scale[h] : 1.f);
    } else {
      *(uint4*)((uint16_t*)c.k + at) = k;
      *(uint4*)((uint16_t*)c.v + at) = v;
    }
  }
}

hipError_t launch_paged_kv_write(const KvWriteArgs& a, hipStream_t st) {
  const int per_token = a.cache.heads * a.cache.dim / 8;
  const int tpb = per_token < 256 ? 256 / per_token : 1;
  const unsigned grid = (unsigned)((a.tokens + tpb - 1) / tpb);
  if (a.cache.fp8)
    paged_kv_write_kernel<true><<<grid, 256, 0, st>>>(a, tpb);
  else
    paged_kv_write_kernel<false><<<grid, 256, 0, st>>>(a, tpb);
  return hipGetLastError();
}

}  // namespace nvfp4
