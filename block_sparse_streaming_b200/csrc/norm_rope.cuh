// norm_rope.cuh - RMS norm of query and key heads and the position rotation in
// one pass, with the keys and values written straight into a paged cache, and
// the gradient of both.
//
// Each head row x (d columns) of token t becomes
//     n_c = w_c x_c / rms,  rms = sqrt(mean_{c < norm_dim} x_c^2 + eps)   c < norm_dim
//     n_c = x_c                                                      otherwise
//     (y_a, y_b) = scale (n_a cos - n_b sin, n_a sin + n_b cos)
// for the pairs (a, b) of the rotated columns [off, off + 2 half): b = a + half
// (half layout) or b = a + 1 (interleaved), pair i turning by position_t *
// inv_freq_i. The angle is formed in 64 bits and reduced to a fraction of a
// turn before it is rounded, so far positions lose nothing: a 32-bit product
// at position 10^6 is off by 0.03 rad. Everything else is 32-bit, rounded once
// when the row is stored.
//
// Gradient, with u = x / rms and R^T the transposed rotation (scale included):
//     dn = R^T dy,  g = w dn,  dx = (g - u mean(g u)) / rms,  dw = sum dn u
// (columns without norm: dx = dn). Weight gradients are summed in registers
// over a warp's rows, then over the CTA's warps, then over the CTAs by
// norm_rope_dw_kernel, each in a fixed order: no atomics, the same bits every
// run for one GPU.
//
// Both are bound by HBM: every row is read once and written once. A task is a
// pair of 16-byte vectors of one row (for rotated columns the two halves of
// the same pairs, or two neighbouring vectors when interleaved), so a rotation
// never leaves its lane; `lph` lanes (a power of two) share a row and
// 32 / lph rows share a warp. The angles of a token are formed once per warp
// in shared memory and then live in registers for all of its heads. Rows whose
// sizes, offsets or strides are no multiple of a vector run the same code with
// one element per vector.
#pragma once

#include <cuda_fp16.h>

#include "sm100.cuh"

namespace loza {

constexpr int kNrThreads = 128;  // four warps, each on its own (token, part of the heads)
constexpr int kNrWarps = kNrThreads / 32;

struct NrShape {
  int d, norm_dim, rope_off, half, interleaved, lph, nrope, npass, ntasks;
  float scale, sign, eps, inv_norm;  // sign -1: the transposed rotation
  const double* inv_freq;
  const int32_t* positions;
  int64_t tokens;
};

struct NrSide {
  const void *x, *dy, *w;
  void* out;          // may be null (the row then only goes to the pool)
  int64_t x_stride, dy_stride, out_stride;
  int heads;
  int skip_pass;      // out == x and nothing but the rotated columns changes
};

struct NrPool {  // one of the two pools of a paged cache
  void* base;
  int64_t page_stride, row_stride, head_stride;
};

struct NrFwdParams {
  NrShape s;
  NrSide q, k;
  NrPool k_pool, v_pool;
  const void* v;
  int64_t v_stride;
  const int64_t* slots;
  int64_t n_slots;  // num_pages * page_size
  int page_shift, d_v, parts;
};

struct NrBwdParams {
  NrShape s;
  NrSide q, k;
  float* partial;   // [gridDim.x][norm_dim]
  int q_ctas;       // CTAs [0, q_ctas) take the queries, the others the keys
  int parts_q, parts_k;
};

// Conversions between a 16-bit or 32-bit element type and float.
template <typename T> struct Elt;
template <> struct Elt<float> {
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};
template <> struct Elt<__half> {
  static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};
template <> struct Elt<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};

// VEC elements moved as one unit (16 bytes, or a single element).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T e[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack_zero() {
  Pack<T, VEC> r;
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.e[i] = Elt<T>::down(0.f);
  return r;
}

// The columns of one lane's task: vectors at a and b (b < 0: none, a < 0: no task).
template <int VEC>
struct NrTask {
  int a, b;
  bool rot;
  NrTask() = default;
  __device__ __forceinline__ NrTask(const NrShape& s, int t) {
    a = b = -1;
    rot = t < s.nrope;
    if (rot) {
      a = s.rope_off + (s.interleaved ? 2 * t * VEC : t * VEC);
      b = s.interleaved ? a + VEC : a + s.half;
    } else if (t < s.ntasks) {
      const int n = (s.npass + 1) >> 1, i = t - s.nrope;
      a = i * VEC;
      if (a >= s.rope_off) a += 2 * s.half;
      if (i + n < s.npass) {
        b = (i + n) * VEC;
        if (b >= s.rope_off) b += 2 * s.half;
      }
    }
  }
};

// cos and sin of one token's angles (times scale and sign), by the whole warp.
__device__ __forceinline__ void nr_angles(const NrShape& s, int64_t tok, float2* tab, int lane) {
  if (s.half == 0) return;
  const double pos = (double)s.positions[tok];
  __syncwarp();  // the previous token's angles have been read
  for (int i = lane; i < s.half; i += 32) {
    double turns = pos * (s.inv_freq[i] * 0.15915494309189533577);  // 1 / (2 pi)
    turns -= rint(turns);
    float sn, cs;
    sincospif(2.f * (float)turns, &sn, &cs);
    tab[i] = make_float2(cs * s.scale, sn * s.scale * s.sign);
  }
  __syncwarp();
}

template <int VEC, int NV>
__device__ __forceinline__ void nr_read_angles(const NrTask<VEC> (&task)[NV], int t0, int lph, const float2* tab,
                                               float2 (&cs)[NV][VEC]) {
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      cs[v][e] = task[v].rot ? tab[(t0 + v * lph) * VEC + e] : make_float2(1.f, 0.f);
}

// Rotates the VEC pairs of one task in place.
template <int VEC>
__device__ __forceinline__ void nr_rotate(float (&a)[VEC], float (&b)[VEC], const float2 (&cs)[VEC], bool inter) {
  if (VEC > 1 && inter) {
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 c0 = cs[e], c1 = cs[VEC / 2 + e];
      const float x0 = a[2 * e], y0 = a[2 * e + 1], x1 = b[2 * e], y1 = b[2 * e + 1];
      a[2 * e] = x0 * c0.x - y0 * c0.y;
      a[2 * e + 1] = x0 * c0.y + y0 * c0.x;
      b[2 * e] = x1 * c1.x - y1 * c1.y;
      b[2 * e + 1] = x1 * c1.y + y1 * c1.x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * cs[e].x - y * cs[e].y;
      b[e] = x * cs[e].y + y * cs[e].x;
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void nr_unpack(const Pack<T, VEC>& p, float (&f)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = Elt<T>::up(p.e[e]);
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> nr_pack(const float (&f)[VEC]) {
  Pack<T, VEC> p;
#pragma unroll
  for (int e = 0; e < VEC; ++e) p.e[e] = Elt<T>::down(f[e]);
  return p;
}

__device__ __forceinline__ float nr_row_sum(float v, int lph) {
  for (int o = lph >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The rows of one side of one token that belong to this warp: row groups
// g0, g0 + step, ... of 32 / lph heads each.
template <typename T, int VEC, int NV, int U>
__device__ __forceinline__ void nr_forward_rows(const NrShape& s, const NrSide& sd, int64_t tok, int g0, int step,
                                                const NrTask<VEC> (&task)[NV], const float2 (&cs)[NV][VEC], int lane,
                                                T* pool, int64_t pool_head) {
  using P = Pack<T, VEC>;
  const int rows = 32 / s.lph, sub = lane / s.lph;
  const T* xrow = static_cast<const T*>(sd.x) + tok * sd.x_stride;
  T* orow = sd.out ? static_cast<T*>(sd.out) + tok * sd.out_stride : nullptr;
  const T* w = static_cast<const T*>(sd.w);
  P wa[NV], wb[NV];
  if (w) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      wa[v] = wb[v] = pack_zero<T, VEC>();
      if (task[v].a >= 0 && task[v].a < s.norm_dim) wa[v] = *reinterpret_cast<const P*>(w + task[v].a);
      if (task[v].b >= 0 && task[v].b < s.norm_dim) wb[v] = *reinterpret_cast<const P*>(w + task[v].b);
    }
  }
  const int groups = (sd.heads + rows - 1) / rows;
  for (int g = g0; g < groups; g += step * U) {
    P xa[U][NV], xb[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (g + u * step) * rows + sub;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        xa[u][v] = xb[u][v] = pack_zero<T, VEC>();
        if (h >= sd.heads || (sd.skip_pass && !task[v].rot)) continue;
        if (task[v].a >= 0) xa[u][v] = *reinterpret_cast<const P*>(xrow + (int64_t)h * s.d + task[v].a);
        if (task[v].b >= 0) xb[u][v] = *reinterpret_cast<const P*>(xrow + (int64_t)h * s.d + task[v].b);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g + u * step >= groups) break;  // the same for the whole warp
      const int h = (g + u * step) * rows + sub;
      float fa[NV][VEC], fb[NV][VEC];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        nr_unpack<T, VEC>(xa[u][v], fa[v]);
        nr_unpack<T, VEC>(xb[u][v], fb[v]);
      }
      if (w) {
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (task[v].a >= 0 && task[v].a < s.norm_dim)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sq = fmaf(fa[v][e], fa[v][e], sq);
          if (task[v].b >= 0 && task[v].b < s.norm_dim)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sq = fmaf(fb[v][e], fb[v][e], sq);
        }
        const float r = rsqrtf(fmaf(nr_row_sum(sq, s.lph), s.inv_norm, s.eps));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (task[v].a >= 0 && task[v].a < s.norm_dim)
#pragma unroll
            for (int e = 0; e < VEC; ++e) fa[v][e] *= r * Elt<T>::up(wa[v].e[e]);
          if (task[v].b >= 0 && task[v].b < s.norm_dim)
#pragma unroll
            for (int e = 0; e < VEC; ++e) fb[v][e] *= r * Elt<T>::up(wb[v].e[e]);
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (task[v].rot) nr_rotate<VEC>(fa[v], fb[v], cs[v], s.interleaved);
        if (h >= sd.heads || (sd.skip_pass && !task[v].rot)) continue;
        const P ya = nr_pack<T, VEC>(fa[v]), yb = nr_pack<T, VEC>(fb[v]);
        if (orow) {
          if (task[v].a >= 0) *reinterpret_cast<P*>(orow + (int64_t)h * s.d + task[v].a) = ya;
          if (task[v].b >= 0) *reinterpret_cast<P*>(orow + (int64_t)h * s.d + task[v].b) = yb;
        }
        if (pool) {
          if (task[v].a >= 0) *reinterpret_cast<P*>(pool + h * pool_head + task[v].a) = ya;
          if (task[v].b >= 0) *reinterpret_cast<P*>(pool + h * pool_head + task[v].b) = yb;
        }
      }
    }
  }
}

// A warp takes one part of one token's row groups: the query groups, then the
// key groups, then the value vectors, dealt round robin over `parts` warps.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NrFwdParams p) {
  extern __shared__ float2 nr_smem[];
  constexpr int U = NV * VEC >= 16 ? 2 : 4;  // row groups in flight per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kNrWarps + warp;
  const int64_t tok = unit / p.parts;
  const int part = (int)(unit - tok * p.parts);
  if (tok >= p.s.tokens) return;  // no block-wide barrier below
  float2* tab = nr_smem + (size_t)warp * p.s.half;
  NrTask<VEC> task[NV];
  float2 cs[NV][VEC];
  const int t0 = lane & (p.s.lph - 1);
  nr_angles(p.s, tok, tab, lane);
#pragma unroll
  for (int v = 0; v < NV; ++v) task[v] = NrTask<VEC>(p.s, t0 + v * p.s.lph);
  nr_read_angles<VEC, NV>(task, t0, p.s.lph, tab, cs);

  const int rows = 32 / p.s.lph;
  const int gq = (p.q.heads + rows - 1) / rows, gk = (p.k.heads + rows - 1) / rows;
  nr_forward_rows<T, VEC, NV, U>(p.s, p.q, tok, part, p.parts, task, cs, lane, nullptr, 0);
  if (p.k.heads == 0) return;
  int64_t slot = -1;
  if (p.slots) {
    slot = p.slots[tok];
    if (slot < 0 || slot >= p.n_slots) slot = -1;  // a padded row, or a page that is not there
  }
  const int64_t page = slot >> p.page_shift, row = slot & ((1 << p.page_shift) - 1);
  T* kp = slot >= 0 && p.k_pool.base
              ? static_cast<T*>(p.k_pool.base) + page * p.k_pool.page_stride + row * p.k_pool.row_stride : nullptr;
  if (kp || p.k.out) {
    const int first = (part + p.parts - gq % p.parts) % p.parts;
    nr_forward_rows<T, VEC, NV, U>(p.s, p.k, tok, first, p.parts, task, cs, lane, kp, p.k_pool.head_stride);
  }
  if (slot >= 0 && p.v_pool.base) {
    using P = Pack<T, VEC>;
    const int first = (part + p.parts - (gq + gk) % p.parts) % p.parts;
    const int per = p.d_v / VEC, n = p.k.heads * per;
    const T* src = static_cast<const T*>(p.v) + tok * p.v_stride;
    T* dst = static_cast<T*>(p.v_pool.base) + page * p.v_pool.page_stride + row * p.v_pool.row_stride;
    for (int i = first * 32 + lane; i < n; i += p.parts * 32) {
      const int h = i / per;
      *reinterpret_cast<P*>(dst + h * p.v_pool.head_stride + (i - h * per) * VEC) =
          *reinterpret_cast<const P*>(src + (int64_t)i * VEC);
    }
  }
}

// CTAs [0, q_ctas) walk the query rows, the others the key rows, so that a
// warp has one set of weight gradients in registers.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kNrThreads) norm_rope_backward_kernel(const NrBwdParams p) {
  extern __shared__ float2 nr_smem[];  // kNrWarps tables of angles, then kNrWarps rows of norm_dim floats
  using P = Pack<T, VEC>;
  constexpr int U = NV * VEC >= 16 ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_q = (int)blockIdx.x < p.q_ctas;
  const NrSide& sd = is_q ? p.q : p.k;
  const NrShape& s = p.s;
  const int parts = is_q ? p.parts_q : p.parts_k;
  const int cta = is_q ? blockIdx.x : blockIdx.x - p.q_ctas;
  const int ctas = is_q ? p.q_ctas : gridDim.x - p.q_ctas;
  float2* tab = nr_smem + (size_t)warp * s.half;
  float* sums = reinterpret_cast<float*>(nr_smem + (size_t)kNrWarps * s.half);
  const int lph = s.lph, t0 = lane & (lph - 1), rows = 32 / lph, sub = lane / lph;
  const int groups = (sd.heads + rows - 1) / rows;
  const T* w = static_cast<const T*>(sd.w);
  NrTask<VEC> task[NV];
  P wa[NV], wb[NV];
  float dwa[NV][VEC], dwb[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    task[v] = NrTask<VEC>(s, t0 + v * lph);
    wa[v] = wb[v] = pack_zero<T, VEC>();
    if (w && task[v].a >= 0 && task[v].a < s.norm_dim) wa[v] = *reinterpret_cast<const P*>(w + task[v].a);
    if (w && task[v].b >= 0 && task[v].b < s.norm_dim) wb[v] = *reinterpret_cast<const P*>(w + task[v].b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dwa[v][e] = dwb[v][e] = 0.f;
  }
  const int64_t units = s.tokens * parts;
  for (int64_t unit = (int64_t)cta * kNrWarps + warp; unit < units; unit += (int64_t)ctas * kNrWarps) {
    const int64_t tok = unit / parts;
    const int part = (int)(unit - tok * parts);
    float2 cs[NV][VEC];
    nr_angles(s, tok, tab, lane);
    nr_read_angles<VEC, NV>(task, t0, lph, tab, cs);
    const T* xrow = static_cast<const T*>(sd.x) + tok * sd.x_stride;
    const T* yrow = static_cast<const T*>(sd.dy) + tok * sd.dy_stride;
    T* orow = static_cast<T*>(sd.out) + tok * sd.out_stride;
    for (int g = part; g < groups; g += parts * U) {
      P xa[U][NV], xb[U][NV], ya[U][NV], yb[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (g + u * parts) * rows + sub;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          xa[u][v] = xb[u][v] = ya[u][v] = yb[u][v] = pack_zero<T, VEC>();
          if (h >= sd.heads) continue;
          const int64_t at = (int64_t)h * s.d;
          if (task[v].a >= 0) {
            ya[u][v] = *reinterpret_cast<const P*>(yrow + at + task[v].a);
            if (w) xa[u][v] = *reinterpret_cast<const P*>(xrow + at + task[v].a);
          }
          if (task[v].b >= 0) {
            yb[u][v] = *reinterpret_cast<const P*>(yrow + at + task[v].b);
            if (w) xb[u][v] = *reinterpret_cast<const P*>(xrow + at + task[v].b);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g + u * parts >= groups) break;  // the same for the whole warp
        const int h = (g + u * parts) * rows + sub;
        float fa[NV][VEC], fb[NV][VEC];  // dn
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          nr_unpack<T, VEC>(ya[u][v], fa[v]);
          nr_unpack<T, VEC>(yb[u][v], fb[v]);
          if (task[v].rot) nr_rotate<VEC>(fa[v], fb[v], cs[v], s.interleaved);
        }
        if (w) {
          float sq = 0.f, dot = 0.f;  // sum x^2, sum g x
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float ga[VEC], gb[VEC];
            nr_unpack<T, VEC>(xa[u][v], ga);
            nr_unpack<T, VEC>(xb[u][v], gb);
            if (task[v].a >= 0 && task[v].a < s.norm_dim)
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                sq = fmaf(ga[e], ga[e], sq);
                dot = fmaf(fa[v][e] * Elt<T>::up(wa[v].e[e]), ga[e], dot);
              }
            if (task[v].b >= 0 && task[v].b < s.norm_dim)
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                sq = fmaf(gb[e], gb[e], sq);
                dot = fmaf(fb[v][e] * Elt<T>::up(wb[v].e[e]), gb[e], dot);
              }
          }
          sq = nr_row_sum(sq, lph);
          dot = nr_row_sum(dot, lph);
          const float r = rsqrtf(fmaf(sq, s.inv_norm, s.eps));
          const float c = dot * r * s.inv_norm;  // mean(g u)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float ga[VEC], gb[VEC];
            nr_unpack<T, VEC>(xa[u][v], ga);
            nr_unpack<T, VEC>(xb[u][v], gb);
            if (task[v].a >= 0 && task[v].a < s.norm_dim)
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float ux = ga[e] * r;
                dwa[v][e] = fmaf(fa[v][e], ux, dwa[v][e]);
                fa[v][e] = r * (fa[v][e] * Elt<T>::up(wa[v].e[e]) - ux * c);
              }
            if (task[v].b >= 0 && task[v].b < s.norm_dim)
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float ux = gb[e] * r;
                dwb[v][e] = fmaf(fb[v][e], ux, dwb[v][e]);
                fb[v][e] = r * (fb[v][e] * Elt<T>::up(wb[v].e[e]) - ux * c);
              }
          }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (h >= sd.heads) continue;
          const int64_t at = (int64_t)h * s.d;
          if (task[v].a >= 0) *reinterpret_cast<P*>(orow + at + task[v].a) = nr_pack<T, VEC>(fa[v]);
          if (task[v].b >= 0) *reinterpret_cast<P*>(orow + at + task[v].b) = nr_pack<T, VEC>(fb[v]);
        }
      }
    }
  }
  griddep_launch_dependents();
  if (!w) return;  // the same for the whole CTA
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float a = dwa[v][e], b = dwb[v][e];
      for (int o = lph; o < 32; o <<= 1) {  // rows of the warp that share these columns
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      if (sub == 0) {
        if (task[v].a >= 0 && task[v].a < s.norm_dim) sums[warp * s.norm_dim + task[v].a + e] = a;
        if (task[v].b >= 0 && task[v].b < s.norm_dim) sums[warp * s.norm_dim + task[v].b + e] = b;
      }
    }
  __syncthreads();
  for (int c = threadIdx.x; c < s.norm_dim; c += kNrThreads) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kNrWarps; ++k) t += sums[k * s.norm_dim + c];
    p.partial[(size_t)blockIdx.x * s.norm_dim + c] = t;
  }
}

// dw[side][c] = sum over the side's CTAs of partial[cta][c], in a fixed order:
// 32 columns per block, 8 threads per column each over every 8th CTA.
struct NrDwParams {
  const float* partial;
  float *dqw, *dkw;
  int norm_dim, q_ctas, ctas;
};
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const NrDwParams p) {
  __shared__ float part[8][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), j = threadIdx.x >> 5;
  const bool is_q = blockIdx.y == 0;
  float* out = is_q ? p.dqw : p.dkw;
  griddep_wait();
  if (!out) return;
  const int c0 = is_q ? 0 : p.q_ctas, c1 = is_q ? p.q_ctas : p.ctas;
  float t = 0.f;
  if (col < p.norm_dim)
    for (int c = c0 + j; c < c1; c += 8) t += p.partial[(size_t)c * p.norm_dim + col];
  part[j][threadIdx.x & 31] = t;
  __syncthreads();
  if (j == 0 && col < p.norm_dim) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += part[k][threadIdx.x & 31];
    out[col] = sum;
  }
}

}  // namespace loza
