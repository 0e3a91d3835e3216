// page_plan.cuh - the paged cache's bookkeeping of one step, on the GPU.
//
// From each request's cached length c_r and its new tokens n_r (page size P):
//     have_r = ceil(c_r / P), need_r = ceil((c_r + n_r) / P) - have_r
//     cu = exclusive sum of n, off = exclusive sum of need
//     table[r][have_r + k] = free[off_r + k]                    k < need_r
//     token cu_r + j: position c_r + j, slot table[r][pos / P] P + pos % P
// Everything but the two running sums is independent per token and per page,
// and the sums are over at most 16,384 requests, so every CTA forms them
// itself in shared memory (8 bytes a request) instead of waiting for another
// kernel: one launch, no workspace. A thread takes four consecutive tokens,
// finds the first one's request by bisection and walks on from there; the
// slots and positions leave in 16-byte stores.
#pragma once

#include "sm100.cuh"

namespace loza {

constexpr int kPlanThreads = 256;
constexpr int kPlanMaxBatch = 16384;

struct PlanParams {
  const int32_t *ctx, *add, *free_pages;
  int32_t* table;
  int64_t table_stride;
  int batch, max_pages, n_free, page_shift;
  int64_t capacity;
  int32_t *cu, *seqlens, *positions, *counts;
  int64_t* slots;
};

struct PlanRequest {
  int ctx, add, have, need;
  PlanRequest() = default;
  __device__ __forceinline__ PlanRequest(const PlanParams& p, int r) {
    // a length outside [0, 2^30) counts as zero (sums of two stay in 31 bits)
    const int c = p.ctx[r], n = p.add[r];
    ctx = (unsigned)c < (1u << 30) ? c : 0;
    add = (unsigned)n < (1u << 30) ? n : 0;
    const int up = (1 << p.page_shift) - 1;
    have = (ctx + up) >> p.page_shift;
    need = (int)(((unsigned)ctx + (unsigned)add + (unsigned)up) >> p.page_shift) - have;
  }
  // the table has no room for its pages, or the free list ends before them
  __device__ __forceinline__ bool is_short(const PlanParams& p, int off) const {
    return have + need > p.max_pages || (need > 0 && (int64_t)off + need > p.n_free);
  }
};

// Largest r in [0, n) with start[r] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int plan_find(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p) {
  extern __shared__ int plan_smem[];
  int* cu = plan_smem;                // [batch + 1]
  int* off = plan_smem + p.batch + 1; // [batch + 1]
  __shared__ int warp_tok[kPlanThreads / 32], warp_pg[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  int64_t tok0 = 0, pg0 = 0;  // sums before this chunk of requests
  int shorts = 0;
  PlanRequest ahead{};  // of the next chunk, on its way while this one is summed
  if (tid < p.batch) ahead = PlanRequest(p, tid);
  for (int base = 0; base < p.batch; base += kPlanThreads) {
    const int r = base + tid;
    const PlanRequest q = ahead;
    ahead = PlanRequest{};
    if (r + kPlanThreads < p.batch) ahead = PlanRequest(p, r + kPlanThreads);
    const int add = q.add, need = q.need, have = q.have, ctx = q.ctx;
    int64_t st = add, sp = need;  // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, st, o), b = __shfl_up_sync(0xffffffffu, sp, o);
      if (lane >= o) { st += a; sp += b; }
    }
    // a warp's sums are kept saturated: past 2^31 - 1 nothing can be addressed
    if (lane == 31) {
      warp_tok[warp] = (int)min(st, (int64_t)INT32_MAX);
      warp_pg[warp] = (int)min(sp, (int64_t)INT32_MAX);
    }
    __syncthreads();
    int64_t bt = tok0, bp = pg0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) { bt += warp_tok[w]; bp += warp_pg[w]; }
      tok0 += warp_tok[w];
      pg0 += warp_pg[w];
    }
    int mine = 0;
    if (r < p.batch) {
      const int c = (int)min(bt + st - add, (int64_t)INT32_MAX), o = (int)min(bp + sp - need, (int64_t)INT32_MAX);
      cu[r] = c;
      off[r] = o;
      const bool lacks = have + need > p.max_pages || (need > 0 && (int64_t)o + need > p.n_free);
      mine = lacks;
      if (blockIdx.x == 0) {
        p.cu[r] = c;
        p.seqlens[r] = lacks ? ctx : ctx + add;
      }
    }
    shorts += __syncthreads_count(mine);  // also: the warp sums are free again
  }
  const int tokens = (int)min(tok0, (int64_t)INT32_MAX), pages = (int)min(pg0, (int64_t)INT32_MAX);
  if (tid == 0) {
    cu[p.batch] = tokens;
    off[p.batch] = pages;
    if (blockIdx.x == 0) {
      p.cu[p.batch] = tokens;
      p.counts[0] = tokens;
      p.counts[1] = pages;
      p.counts[2] = shorts;
    }
  }
  __syncthreads();

  const int64_t stride = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t t4 = (int64_t)blockIdx.x * kPlanThreads + tid; t4 * 4 < p.capacity; t4 += stride) {
    const int64_t t0 = t4 * 4;
    int pos[4] = {0, 0, 0, 0};
    long long slot[4] = {-1, -1, -1, -1};
    if (t0 < tokens) {
      int r = plan_find(cu, p.batch, (int)t0);
      PlanRequest q(p, r);
      bool lacks = q.is_short(p, off[r]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t t = t0 + e;
        if (t >= tokens) break;
        if (t >= cu[r + 1]) {
          do ++r; while (t >= cu[r + 1]);
          q = PlanRequest(p, r);
          lacks = q.is_short(p, off[r]);
        }
        pos[e] = q.ctx + (int)(t - cu[r]);
        const int col = pos[e] >> p.page_shift;
        if (!lacks) {
          const int page = col < q.have ? p.table[r * p.table_stride + col] : p.free_pages[off[r] + (col - q.have)];
          if (page >= 0)
            slot[e] = ((long long)page << p.page_shift) + (pos[e] & ((1 << p.page_shift) - 1));
        }
      }
    }
    if (t0 + 4 <= p.capacity) {
      reinterpret_cast<int4*>(p.positions)[t4] = make_int4(pos[0], pos[1], pos[2], pos[3]);
      reinterpret_cast<longlong2*>(p.slots)[t4 * 2] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2*>(p.slots)[t4 * 2 + 1] = make_longlong2(slot[2], slot[3]);
    } else {
      for (int e = 0; e < 4 && t0 + e < p.capacity; ++e) {
        p.positions[t0 + e] = pos[e];
        p.slots[t0 + e] = slot[e];
      }
    }
  }
  for (int64_t g = (int64_t)blockIdx.x * kPlanThreads + tid; g < min(pages, p.n_free); g += stride) {
    const int r = plan_find(off, p.batch, (int)g);
    const PlanRequest q(p, r);
    if (!q.is_short(p, off[r])) p.table[r * p.table_stride + q.have + ((int)g - off[r])] = p.free_pages[g];
  }
}

}  // namespace loza
