// decode_paged_kv.cuh - attention of one new token over paged K and V pools
// (per-head or grouped heads), split over the cache's length and joined.
//
// For sequence n and query head h (key head h / g, g = n_heads / n_kv_heads),
// over the visible keys t of the window (see SsaWindow) at the last position:
//     z_t = scale q.k_t,  LSE = ln sum e^{z_t},  O = sum e^{z_t - LSE} v_t
// Every visible K and V row is asked for once per up to 16 query heads and used
// for 2 (d_qk + d_v) operations a head: at most 32 per byte, so up to 16 heads
// on a key head HBM bounds it and the matrix instructions only have to stay out
// of the way (16 heads on one, 64 sequences of 65,536: 317 us, 6.8 TB/s). Larger
// groups read every row once per 16 heads, from HBM too (71 on one: 2.66 GB for
// 0.54 GB of rows), and take as many times as long (32 on one 620-740 us, as the
// parts of a sequence find each other's rows in L2 or not; 71 1,825).
// Shapes: (d_qk, d_v) in {(64,64), (128,128), (192,128)}.
//
// Split. The work is cut into steps of 64 keys of one (sequence, key head,
// chunk of its query heads); all steps of the batch, in that order, are dealt
// to the CTAs (two per SM) in equal contiguous ranges, so ragged lengths
// balance without the host knowing them. A CTA walks its range item by item.
// An item that lies in one CTA is written out by it; the others leave
// (reference, sum, weighted values) per range in the workspace, at most two
// per CTA, and the CTA where such an item begins leaves its place, by which
// decode_paged_join_kernel adds the parts up in the order of the CTAs.
// Nothing is atomic and the order of every sum is fixed by the lengths.
//
// Inside a CTA each of four warps owns 16 keys of every step and runs alone:
// its own ring of tiles filled by 16-byte cp.async (masked rows and pages that
// are not there are filled with zeros and never read from memory), its own
// running maximum and sums; the four meet only at the end of an item, while
// the next item's queries and first tiles are on their way. Keys are
// the rows of the matrix products, so a group of up to 8 heads (NT = 1) needs
// no padding to 16: S^T (16 keys x 8 heads) = K Q^T, then O^T (d_v x 8 heads)
// += V^T P^T, with P^T turned in registers by movmatrix. P is fed as two
// 16-bit parts, high and remainder: rounded once to 16 bits it would cost as
// much accuracy as the output's own rounding, and the second product is free
// beside the loads. Each step's products are summed from zero by the matrix
// unit and added to the running sums by a rounded addition: the unit cuts its
// 32-bit sums off toward zero, and a chain of it over 2,048 steps drifts by
// 2.5e-5 (8e-6 over 450, 32 sequences of 16K-49K), which fp16 outputs show; with
// the additions below 1e-6, at the same times (575 and 574 us there).
#pragma once

#include <cuda_fp16.h>

#include "cp_async.cuh"
#include "prefill.cuh"
#include "sm100.cuh"

namespace loza {

constexpr int kPkvWarps = 4;
constexpr int kPkvThreads = kPkvWarps * 32;
constexpr int kPkvStep = 64;       // keys of one step: 16 per warp
constexpr int kPkvCtasPerSm = 2;
constexpr int kPkvHeads = 16;      // query heads of an item, at most

struct PagedKvParams {
  const void* q;                   // [batch, n_heads, d_qk], rows q_stride apart
  const void *k, *v;               // pools
  int64_t q_stride;
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;  // strides, elements
  const int32_t *table, *seqlens;
  int64_t table_stride;
  int batch, max_seqlen, num_pages, page_shift;
  int n_kv, group, chunks, chunk;  // items per (sequence): n_kv * chunks, of `chunk` heads (the last fewer)
  SsaWindow win;
  float scale_log2;
  void* out;                       // [batch, n_heads, d_v]
  float* lse;                      // [batch, n_heads]
  float *part_o, *part_ml;         // [ctas][2][16][d_v], [ctas][2][16][2]
  int4* split;                     // [ctas]: {sequence, item, last CTA} of the item that begins in a CTA and ends in
                                   // a later one; sequence -1: none
  int ctas;
};

// The steps of one sequence: sink steps first, then the local ones.
struct PagedKvSpan {
  int len, lo, sinks, first, steps;
  __device__ __forceinline__ PagedKvSpan(const PagedKvParams& p, int n) {
    len = min(max(p.seqlens[n], 0), p.max_seqlen);
    lo = len > 0 ? p.win.lo(len - 1) : 0;
    sinks = (min(p.win.sink_end, len) + kPkvStep - 1) / kPkvStep;
    first = max(lo / kPkvStep, sinks);
    const int end = (len + kPkvStep - 1) / kPkvStep;
    steps = sinks + max(end - first, 0);
  }
  __device__ __forceinline__ int key(int step) const {
    return (step < sinks ? step : first + (step - sinks)) * kPkvStep;
  }
  // bit j: key t0 + j is visible, j = 0 .. 15
  __device__ __forceinline__ uint32_t visible16(const PagedKvParams& p, int t0) const {
    auto below = [](int x) -> uint32_t { return x <= 0 ? 0u : (x >= 16 ? 0xFFFFu : (1u << x) - 1u); };
    return below(len - t0) & (below(p.win.sink_end - t0) | ~below(lo - t0));
  }
};

template <typename T> struct Mma16;
template <> struct Mma16<__nv_bfloat16> {
  static constexpr float kRef = 0.f;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
};
template <> struct Mma16<__half> {
  // P is kept at 2^14 times its value against the running maximum: fp16 loses
  // what is below 2^-25, which many small weights together would feel.
  static constexpr float kRef = 14.f;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <int DQK, int DV, int NT>
struct PagedKvLayout {
  static constexpr int kTileBytes = 16 * (DQK + DV) * 2;  // one warp's K and V rows of a step
  static constexpr int kStages = DQK + DV <= 128 ? 6 : (DQK + DV <= 256 ? 3 : 2);
  static constexpr int kRing = kPkvWarps * kStages * kTileBytes;
  static constexpr int kQBytes = 8 * NT * DQK * 2;                // each warp's copy of an item's queries
  static constexpr int kQ = kPkvWarps * kQBytes;
  static constexpr int kMl = kPkvWarps * kPkvHeads * 2 * 4;       // [warp][16 heads]{reference, sum}
  static constexpr int kMask = kPkvWarps * kStages * 4;
  static constexpr int kSmem = kRing + kQ + kMl + kMask;
  // a warp's weighted values of 8 heads go to its last stage, which a new item's first tiles leave free
  static_assert(8 * DV * 4 <= kTileBytes, "the join's staging fits a stage");
  static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
};

// A range of one item's steps: [step, s_end) of item `item` of sequence n.
struct PagedKvPiece {
  int n, item, step, s_end;
  PagedKvSpan span;
};

template <typename T, int DQK, int DV, int NT>
__global__ void __launch_bounds__(kPkvThreads, kPkvCtasPerSm) decode_paged_kv_kernel(const PagedKvParams p) {
  using L = PagedKvLayout<DQK, DV, NT>;
  constexpr int S = L::kStages;
  constexpr int KC = DQK / 8, VC = DV / 8;  // 16-byte chunks per row
  extern __shared__ __align__(128) uint8_t pkv_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, c2 = (lane & 3) * 2;  // fragment row and first column of this lane
  float* ml = reinterpret_cast<float*>(pkv_smem + L::kRing + L::kQ);
  volatile uint32_t* masks =
      reinterpret_cast<volatile uint32_t*>(pkv_smem + L::kRing + L::kQ + L::kMl) + warp * S;
  const uint32_t ring = smem_u32(pkv_smem) + (uint32_t)(warp * S * L::kTileBytes);
  const uint32_t qbuf = smem_u32(pkv_smem) + (uint32_t)(L::kRing + warp * L::kQBytes);
  // staging of warp w: in its last stage
  auto staging = [&](int w) {
    return reinterpret_cast<float*>(pkv_smem + (w * S + S - 1) * L::kTileBytes);
  };

  // ---- this CTA's range of steps: the steps of every 32 sequences (in the ring's memory, which nothing is on
  // its way to yet), then their running sum by every warp for itself
  const int items = p.n_kv * p.chunks, groups = (p.batch + 31) / 32;
  int64_t* sums = reinterpret_cast<int64_t*>(pkv_smem);
  static_assert(65535 / 32 * 8 + 8 <= L::kRing, "a batch's sums fit the ring");
#pragma unroll 4
  for (int g = warp; g < groups; g += kPkvWarps) {
    const int n0 = g * 32 + lane;
    int64_t s = n0 < p.batch ? PagedKvSpan(p, n0).steps : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[g] = s * items;
  }
  __syncthreads();
  int64_t total = 0;
  for (int g = lane; g < groups; g += 32) total += sums[g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int64_t ctas = min((int64_t)p.ctas, total);  // so that no range is empty
  griddep_launch_dependents();
  // sequences without keys: their rows are nobody's item
  for (int s = blockIdx.x; s < p.batch; s += gridDim.x) {
    if (PagedKvSpan(p, s).steps > 0) continue;
    const int64_t row = (int64_t)s * p.n_kv * p.group;
    for (int x = tid; x < p.n_kv * p.group * VC; x += kPkvThreads)
      reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * DV)[x] = make_uint4(0, 0, 0, 0);
    for (int x = tid; x < p.n_kv * p.group; x += kPkvThreads) p.lse[row + x] = -INFINITY;
  }
  if (blockIdx.x >= ctas) {
    if (tid == 0) p.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int64_t begin = total * blockIdx.x / ctas, end = total * (blockIdx.x + 1) / ctas;
  // the first of 32 values whose running sum (from `before`) passes `begin`; before: the sum of those ahead of it
  auto find = [&](int64_t own, int64_t& before) -> int {
    int64_t s = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += a;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + s > begin);
    const int l = hit ? __ffs(hit) - 1 : 31;
    before += __shfl_sync(0xffffffffu, hit ? s - own : s, l);
    return hit ? l : -1;
  };
  int64_t before = 0;
  int group = 0;
  for (int g0 = 0; g0 < groups; g0 += 32) {
    const int l = find(g0 + lane < groups ? sums[g0 + lane] : 0, before);
    if (l >= 0) {
      group = g0 + l;
      break;
    }
  }
  const int n0 = group * 32 + lane;
  const int n = group * 32 + find(n0 < p.batch ? (int64_t)PagedKvSpan(p, n0).steps * items : 0, before);
  __syncthreads();  // the ring is free
  PagedKvPiece cur{n, 0, 0, 0, PagedKvSpan(p, n)};
  cur.item = (int)((begin - before) / cur.span.steps);
  cur.step = (int)((begin - before) % cur.span.steps);
  int64_t left = end - begin;
  cur.s_end = (int)min((int64_t)cur.span.steps, cur.step + left);

  const T* kbase = static_cast<const T*>(p.k);
  const T* vbase = static_cast<const T*>(p.v);

  // Fill stage `st` with this warp's 16 keys of step `s` (of `s_end`) and
  // commit one group; past the end the group is empty.
  int page_next = -1;  // page of the next step to be issued, read one step ahead
  auto page_of = [&](const PagedKvSpan& sp, int seq, int s, int s_end) -> int {
    if (s >= s_end) return -1;
    const int t0 = sp.key(s) + warp * 16;
    if (t0 >= sp.len) return -1;
    return p.table[seq * p.table_stride + (t0 >> p.page_shift)];
  };
  auto issue = [&](const PagedKvSpan& sp, int seq, int kvh, int s, int s_end, int st) {
    const int page = page_next;
    page_next = page_of(sp, seq, s + 1, s_end);
    if (s < s_end) {
      const int t0 = sp.key(s) + warp * 16;
      const bool here = (unsigned)page < (unsigned)p.num_pages;
      const uint32_t vis = here ? sp.visible16(p, t0) : 0u;
      if (lane == 0) masks[st] = vis;
      if (vis) {
        const int64_t row = t0 & ((1 << p.page_shift) - 1);
        const T* ks = kbase + (int64_t)page * p.k_page + row * p.k_row + kvh * p.k_head;
        const T* vs = vbase + (int64_t)page * p.v_page + row * p.v_row + kvh * p.v_head;
        const uint32_t kd = ring + (uint32_t)(st * L::kTileBytes), vd = kd + 16 * DQK * 2;
#pragma unroll
        for (int i = 0; i < KC / 2; ++i) {
          const int x = i * 32 + lane, r = x / KC, c = x % KC;
          const uint32_t ok = (vis >> r) & 1u;
          cp_async<16>(kd + r * (DQK * 2) + ((c ^ (r & 7)) << 4), ks + (ok ? r : 0) * p.k_row + c * 8, ok * 16);
        }
#pragma unroll
        for (int i = 0; i < VC / 2; ++i) {
          const int x = i * 32 + lane, r = x / VC, c = x % VC;
          const uint32_t ok = (vis >> r) & 1u;
          cp_async<16>(vd + r * (DV * 2) + ((c ^ (r & 7)) << 4), vs + (ok ? r : 0) * p.v_row + c * 8, ok * 16);
        }
      }
    }
    cp_async_commit();
  };
  // An item's queries into this warp's buffer (rows past the item's heads are zeros), and its first tiles.
  auto prologue = [&](const PagedKvPiece& c, int first_page) {
    __syncwarp();  // every lane is past its reads of the ring
    const int kvh = c.item / p.chunks, h0 = (c.item % p.chunks) * p.chunk;
    const int heads = min(p.chunk, p.group - h0);
    const T* qrow = static_cast<const T*>(p.q) + (int64_t)c.n * p.q_stride + (int64_t)(kvh * p.group + h0) * DQK;
#pragma unroll
    for (int i = 0; i < NT * KC / 4; ++i) {
      const int x = i * 32 + lane, r = x / KC, ch = x % KC;
      const uint32_t ok = r < heads;
      cp_async<16>(qbuf + r * (DQK * 2) + ((ch ^ (r & 7)) << 4), qrow + (ok ? r * DQK : 0) + ch * 8, ok * 16);
    }
    page_next = first_page;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(c.span, c.n, kvh, c.step + i, c.s_end, i);
  };

  prologue(cur, page_of(cur.span, cur.n, cur.step, cur.s_end));

  while (true) {
    const int kvh = cur.item / p.chunks, h0 = (cur.item % p.chunks) * p.chunk;
    const int heads = min(p.chunk, p.group - h0);
    // ---- the next piece of the range, and its first page
    left -= cur.s_end - cur.step;
    const bool more = left > 0;
    PagedKvPiece next = cur;
    int next_page = -1;
    if (more) {
      if (++next.item == items) {
        next.item = 0;
        do {
          ++next.n;
          next.span = PagedKvSpan(p, next.n);
        } while (next.span.steps == 0);
      }
      next.step = 0;
      next.s_end = (int)min((int64_t)next.span.steps, left);
      next_page = page_of(next.span, next.n, 0, next.s_end);
    }
    // ---- Q^T fragments: B operand (16 d x 8 heads) per 16 columns of d
    uint32_t qf[NT][DQK / 16][2];
    cp_async_wait<S - 2>();  // the queries came with the first tile
    __syncwarp();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < DQK / 32; ++k) {
        uint32_t a[4];
        const int r = t * 8 + (lane & 7), ch = 4 * k + (lane >> 3);
        ldsm4(a, qbuf + r * (DQK * 2) + ((ch ^ (r & 7)) << 4));
        qf[t][2 * k][0] = a[0];
        qf[t][2 * k][1] = a[1];
        qf[t][2 * k + 1][0] = a[2];
        qf[t][2 * k + 1][1] = a[3];
      }
    float o[NT][DV / 16][4];
    float ref[NT][2], sum[NT][2];  // heads c2, c2 + 1 of each tile of 8
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      ref[t][0] = ref[t][1] = -INFINITY;
      sum[t][0] = sum[t][1] = 0.f;
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][k][e] = 0.f;
    }

    int st = 0;
    for (int s = cur.step; s < cur.s_end; ++s) {
      cp_async_wait<S - 2>();
      __syncwarp();
      issue(cur.span, cur.n, kvh, s + S - 1, cur.s_end, st == 0 ? S - 1 : st - 1);
      const uint32_t vis = masks[st];
      if (vis) {
        const uint32_t kd = ring + (uint32_t)(st * L::kTileBytes), vd = kd + 16 * DQK * 2;
        // S^T = K Q^T
        float z[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) z[t][0] = z[t][1] = z[t][2] = z[t][3] = 0.f;
        const int lr = lane & 15, lc = lane >> 4;  // ldmatrix: row, and which of two chunks
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k) {
          uint32_t a[4];
          ldsm4(a, kd + lr * (DQK * 2) + (((2 * k + lc) ^ (lr & 7)) << 4));
#pragma unroll
          for (int t = 0; t < NT; ++t) Mma16<T>::mma(z[t], a, qf[t][k][0], qf[t][k][1]);
        }
        const bool vlo = (vis >> gid) & 1u, vhi = (vis >> (gid + 8)) & 1u;
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float m0, m1;
          z[t][0] = vlo ? z[t][0] * p.scale_log2 : -INFINITY;
          z[t][1] = vlo ? z[t][1] * p.scale_log2 : -INFINITY;
          z[t][2] = vhi ? z[t][2] * p.scale_log2 : -INFINITY;
          z[t][3] = vhi ? z[t][3] * p.scale_log2 : -INFINITY;
          m0 = fmaxf(z[t][0], z[t][2]);
          m1 = fmaxf(z[t][1], z[t][3]);
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o2));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o2));
          }
          m0 = fmaxf(ref[t][0], m0 - Mma16<T>::kRef);
          m1 = fmaxf(ref[t][1], m1 - Mma16<T>::kRef);
          if (__any_sync(0xffffffffu, m0 != ref[t][0] || m1 != ref[t][1])) {
            // a head whose every score so far is -inf keeps zero sums (no inf - inf)
            const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(ref[t][0] - m0);
            const float a1 = m1 == -INFINITY ? 0.f : ex2_approx(ref[t][1] - m1);
            ref[t][0] = m0;
            ref[t][1] = m1;
            sum[t][0] *= a0;
            sum[t][1] *= a1;
#pragma unroll
            for (int k = 0; k < DV / 16; ++k) {
              o[t][k][0] *= a0;
              o[t][k][1] *= a1;
              o[t][k][2] *= a0;
              o[t][k][3] *= a1;
            }
          }
          const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
          const float p0 = ex2_approx(z[t][0] - r0), p1 = ex2_approx(z[t][1] - r1);
          const float p2 = ex2_approx(z[t][2] - r0), p3 = ex2_approx(z[t][3] - r1);
          sum[t][0] += p0 + p2;
          sum[t][1] += p1 + p3;
          const uint32_t h01 = Mma16<T>::pack(p0, p1), h23 = Mma16<T>::pack(p2, p3);
          const float2 u01 = Mma16<T>::unpack(h01), u23 = Mma16<T>::unpack(h23);
          ph[t][0] = movmatrix_trans(h01);
          ph[t][1] = movmatrix_trans(h23);
          pl[t][0] = movmatrix_trans(Mma16<T>::pack(p0 - u01.x, p1 - u01.y));
          pl[t][1] = movmatrix_trans(Mma16<T>::pack(p2 - u23.x, p3 - u23.y));
        }
        // O^T += V^T P^T
        const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;  // key row, which chunk of d_v
#pragma unroll
        for (int k = 0; k < DV / 16; ++k) {
          uint32_t a[4];
          ldsm4_trans(a, vd + vr * (DV * 2) + (((2 * k + vc) ^ (vr & 7)) << 4));
          float f[NT][4];  // of this step alone
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f[t][0] = f[t][1] = f[t][2] = f[t][3] = 0.f;
            Mma16<T>::mma(f[t], a, pl[t][0], pl[t][1]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) Mma16<T>::mma(f[t], a, ph[t][0], ph[t][1]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][k][e] += f[t][e];
        }
      }
      st = st + 1 == S ? 0 : st + 1;
    }

    const bool whole = cur.step == 0 && cur.s_end == cur.span.steps;
    const int slot = (int)blockIdx.x * 2 + (cur.step == 0 ? 1 : 0);
    if (!more && tid == 0) {
      // the batch's step that ends this item; its CTA is the last c with floor(total c / ctas) <= it:
      // c = ((it + 1) ctas - 1) / total
      const int64_t last = end - cur.s_end + cur.span.steps - 1;
      p.split[blockIdx.x] = make_int4(cur.step == 0 && !whole ? cur.n : -1, cur.item,
                                      (int)(((last + 1) * ctas - 1) / total), 0);
    }
    if (more) prologue(next, next_page);  // on its way while this item's results are joined

    // ---- join the four warps
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int o2 = 4; o2 < 32; o2 <<= 1) {
        sum[t][0] += __shfl_xor_sync(0xffffffffu, sum[t][0], o2);
        sum[t][1] += __shfl_xor_sync(0xffffffffu, sum[t][1], o2);
      }
      if (gid == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ml[(warp * kPkvHeads + t * 8 + c2 + e) * 2] = ref[t][e];
          ml[(warp * kPkvHeads + t * 8 + c2 + e) * 2 + 1] = sum[t][e];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t * 8 >= heads) break;  // the same for the whole CTA
      float wgt[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kPkvWarps; ++w) m = fmaxf(m, ml[(w * kPkvHeads + t * 8 + c2 + e) * 2]);
        wgt[e] = ref[t][e] == m ? 1.f : ex2_approx(ref[t][e] - m);
      }
      // [warp][head][d_v], the columns of head pair c turned by 8 c: no bank conflicts
      float* jo = staging(warp);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = (k * 16 + gid + (e >> 1) * 8) ^ ((lane & 3) * 8);
          jo[(c2 + (e & 1)) * DV + col] = o[t][k][e] * wgt[e & 1];
        }
      __syncthreads();
      const int nh = min(8, heads - t * 8);
      for (int x = tid; x < nh * (DV / 8); x += kPkvThreads) {
        const int h = x / (DV / 8), c8 = (x % (DV / 8)) * 8;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kPkvWarps; ++w) m = fmaxf(m, ml[(w * kPkvHeads + t * 8 + h) * 2]);
#pragma unroll
        for (int w = 0; w < kPkvWarps; ++w) {
          const float mw = ml[(w * kPkvHeads + t * 8 + h) * 2];
          l += (mw == m ? 1.f : ex2_approx(mw - m)) * ml[(w * kPkvHeads + t * 8 + h) * 2 + 1];
        }
        float acc[8] = {};
#pragma unroll
        for (int w = 0; w < kPkvWarps; ++w) {
          const float4* src = reinterpret_cast<const float4*>(staging(w) + h * DV + (c8 ^ ((h >> 1) * 8)));
          const float4 a = src[0], b = src[1];
          acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
          acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
        }
        if (whole) {
          const int64_t row = ((int64_t)cur.n * p.n_kv + kvh) * p.group + h0 + t * 8 + h;
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no keys: zeros; NaN stays NaN
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] *= inv;
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * DV + c8) =
              make_uint4(Mma16<T>::pack(acc[0], acc[1]), Mma16<T>::pack(acc[2], acc[3]),
                         Mma16<T>::pack(acc[4], acc[5]), Mma16<T>::pack(acc[6], acc[7]));
          if (c8 == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          const int64_t row = (int64_t)slot * kPkvHeads + t * 8 + h;
          float4* dst = reinterpret_cast<float4*>(p.part_o + row * DV + c8);
          dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
          dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
          if (c8 == 0) *reinterpret_cast<float2*>(p.part_ml + row * 2) = make_float2(m, l);
        }
      }
      __syncthreads();  // the staging area and the sums are free again
    }
    if (!more) break;
    cur = next;
  }
}

// One CTA per (CTA of the first kernel, query head of its items): adds up the
// parts of the item that begins in that CTA and ends in a later one. 16-byte
// pieces of the row by groups of threads; each group takes every 256 / (d_v / 8)th
// part, so a row of a few hundred parts is a few loads deep.
template <typename T, int DV>
__global__ void __launch_bounds__(256) decode_paged_join_kernel(const PagedKvParams p) {
  constexpr int G = 256 / (DV / 8);  // groups of threads
  __shared__ float red[G][DV + 4];
  __shared__ float red_l[G], red_m[8];
  const int tid = threadIdx.x, c8 = (tid % (DV / 8)) * 8, g = tid / (DV / 8), h = blockIdx.y;
  griddep_wait();
  const int4 s = p.split[blockIdx.x];
  if (s.x < 0) return;
  const int kvh = s.y / p.chunks, h0 = (s.y % p.chunks) * p.chunk;
  if (h >= min(p.chunk, p.group - h0)) return;
  const int c0 = blockIdx.x, parts = s.z - c0 + 1;
  // an item's first part is its CTA's slot 1 (it begins there); each later part begins its CTA's range: slot 0
  auto row_of = [&](int j) { return ((int64_t)(c0 + j) * 2 + (j == 0 ? 1 : 0)) * kPkvHeads + h; };
  float m = -INFINITY;
  for (int j = tid; j < parts; j += 256) m = fmaxf(m, p.part_ml[row_of(j) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) red_m[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, red_m[w]);
  float l = 0.f, acc[8] = {};
#pragma unroll 4
  for (int j = g; j < parts; j += G) {
    const int64_t row = row_of(j);
    const float2 v = *reinterpret_cast<const float2*>(p.part_ml + row * 2);
    const float4* src = reinterpret_cast<const float4*>(p.part_o + row * DV + c8);
    const float4 u = src[0], w = src[1];
    const float f = v.x == m ? 1.f : ex2_approx(v.x - m);
    l = fmaf(v.y, f, l);
    acc[0] = fmaf(u.x, f, acc[0]); acc[1] = fmaf(u.y, f, acc[1]);
    acc[2] = fmaf(u.z, f, acc[2]); acc[3] = fmaf(u.w, f, acc[3]);
    acc[4] = fmaf(w.x, f, acc[4]); acc[5] = fmaf(w.y, f, acc[5]);
    acc[6] = fmaf(w.z, f, acc[6]); acc[7] = fmaf(w.w, f, acc[7]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) red[g][c8 + e] = acc[e];
  if (c8 == 0) red_l[g] = l;
  __syncthreads();
  if (tid >= DV / 2) return;  // two columns a thread
  float x = 0.f, y = 0.f;
  l = 0.f;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    x += red[k][2 * tid];
    y += red[k][2 * tid + 1];
    l += red_l[k];
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no keys: zeros; NaN stays NaN
  const int64_t row = ((int64_t)s.x * p.n_kv + kvh) * p.group + h0 + h;
  reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * DV)[tid] = Mma16<T>::pack(x * inv, y * inv);
  if (tid == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Both kernels for a call (decode_paged_kv.cu); false if a launch failed.
template <typename T>
bool pkv_run(const PagedKvParams& p, int d_qk, cudaStream_t st);

}  // namespace loza
