// norm_rope.cuh - RMS norm of query and key heads and the position rotation in
// one pass, with the keys and values written straight into a paged cache, and
// the gradient of both.
//
// Each head row x (d columns) of token t becomes
//     n_c = w_c x_c / rms,  rms = sqrt(mean_{c < norm_dim} x_c^2 + eps)   c < norm_dim
//     n_c = x_c                                                      otherwise
//     (y_a, y_b) = scale (n_a cos - n_b sin, n_a sin + n_b cos)
// for the pairs (a, b) of the rotated columns [off, off + 2 pairs): b = a + pairs
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
// norm_rope_dw_kernel (norm_rope_sums.cuh), each in a fixed order: no atomics,
// the same bits every run for one GPU.
//
// Both are bound by HBM: every row is read once and written once. A task is a
// pair of 16-byte vectors of one row (for rotated columns the two halves of
// the same pairs, or two vectors of whole pairs when interleaved), so a rotation
// never leaves its lane; `lph` lanes (a power of two) share a row and
// 32 / lph rows are a group. A warp takes a token, or a share of its groups
// when there are few tokens: the query rows, the key rows, the values. It keeps
// the token's angles, multiplied by the weights, in registers and walks the
// groups by adding to pointers. Rows come through a ring in shared memory that
// every lane fills by cp.async for itself alone (it reads back what it asked
// for: no barrier); a cursor asks ahead of the arithmetic across sides and
// tokens, so a warp's stream never runs dry, at no cost in registers. A
// forward warp, alone in its CTA, walks its tokens (an equal share, or a short
// walk of many that are dealt out as warps end: see nr_plan_fwd), a CTA of the
// gradient an equal share, in batches; the next batch's angles are formed in
// shared memory, each once, before the current one's rows. Rows whose sizes,
// offsets or strides, or half of whose rotated columns, are no multiple of 16
// bytes run the same code with vectors of 4 bytes or of one element.
#pragma once

#include <cuda_fp16.h>

#include "cp_async.cuh"
#include "sm100.cuh"

namespace loza {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;

// Warps per SM: 16, unless a lane's share of a row takes more than half of the
// registers (rows of more than 32 tasks, and short vectors). The forward's CTAs
// are single warps: none waits for another at a barrier or at its end (CTAs of
// 8 warps: rotation of 64 x 64 heads of 576 5.3 against 4.8 us, norm of 8,192
// tokens with 64 + 64 heads of 192 212 against 198). The gradient's have 8, to
// sum the weights' gradients over.
__host__ __device__ constexpr int nr_warps_per_sm(int vec, int nv) { return nv * vec > 8 || nv > 4 ? 8 : 16; }
__host__ __device__ constexpr int nr_ctas_per_sm(int vec, int nv) { return nr_warps_per_sm(vec, nv) / kNrWarps; }

struct NrShape {
  int d, norm_dim, rope_off, pairs, interleaved, lph, lph_log, nrope, npass, ntasks;
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
  int page_shift, d_v;
  int walks;            // of `walk` tokens each or, if that is 0, equal shares of them
  int walk;
  int batch;            // tokens per step of a walk
  int wide_log;         // log2 of the warps (CTAs) that share a walk, when there are few tokens
  int vper_log;         // log2 of the vectors per value row, or -1
};

struct NrBwdParams {
  NrShape s;
  NrSide q, k;
  float* partial;       // [2][gridDim.x][norm_dim]
  int batch;            // tokens per step of a CTA
  int wide_log;
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

template <typename T> constexpr bool is_half = false;
template <> constexpr bool is_half<__half> = true;

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
      const bool next = VEC == 1 && s.interleaved;  // else the partner, or any vector of whole pairs, half a table on
      a = s.rope_off + (next ? 2 * t : t * VEC);
      b = next ? a + 1 : a + s.pairs;
    } else if (t < s.ntasks) {
      const int n = (s.npass + 1) >> 1, i = t - s.nrope;
      a = i * VEC;
      if (a >= s.rope_off) a += 2 * s.pairs;
      if (i + n < s.npass) {
        b = (i + n) * VEC;
        if (b >= s.rope_off) b += 2 * s.pairs;
      }
    }
  }
};

// cos and sin (times scale and sign) of the angles of tokens [tok0, tok0 + n), by the CTA's threads. Within a token,
// the VEC angles of task t are laid out so that the lanes of a row read consecutive 16 bytes: angle e is at
// (e / 2) (2 nrope) + 2 t + e % 2. They are those of pairs t VEC + e or, interleaved, of the VEC / 2 pairs of the
// task's first vector and the VEC / 2 of its second one, half the rotated columns on.
template <int VEC, bool INTER, int THREADS>
__device__ __forceinline__ void nr_angles(const NrShape& s, int64_t tok0, int n, float2* tab) {
  if (s.pairs == 0) return;
  // a thread keeps its pair (or few pairs) and walks the tokens, `per` of them at a time
  const int per = max(1, THREADS / s.pairs), i0 = s.pairs < THREADS ? threadIdx.x / s.pairs : 0;
  if (i0 >= per) return;
  for (int pair = threadIdx.x - i0 * s.pairs; pair < s.pairs; pair += THREADS) {
    const double freq = s.inv_freq[pair] * 0.15915494309189533577;  // turns: 1 / (2 pi)
    int t = pair / VEC, e = pair - t * VEC;
    if constexpr (INTER && VEC > 1) {
      const int second = pair >= s.pairs / 2, x = pair - second * (s.pairs / 2);
      t = x / (VEC / 2);
      e = x - t * (VEC / 2) + second * (VEC / 2);
    }
    const int at = VEC == 1 ? pair : (e >> 1) * (2 * s.nrope) + 2 * t + (e & 1);
    for (int i = i0; i < n; i += per) {
      double turns = (double)s.positions[tok0 + i] * freq;
      turns -= rint(turns);
      float sn, cs;
      sincospif(2.f * (float)turns, &sn, &cs);
      tab[i * s.pairs + at] = make_float2(cs * s.scale, sn * s.scale * s.sign);
    }
    if (s.pairs < THREADS) break;
  }
}

// 32-bit values of one vector: pairs in 64-bit registers, which the packed
// fp32x2 instructions take as they are (one element: a plain float).
template <int VEC> struct NrVals {
  static constexpr int N = VEC / 2;
  uint64_t p[N];
};
template <> struct NrVals<1> {
  static constexpr int N = 1;
  float p[1];
};
__device__ __forceinline__ uint64_t nr_pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 nr_split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t nr_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t nr_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t nr_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t nr_swap(uint64_t a) {
  const float2 v = nr_split(a);
  return nr_pair(v.y, v.x);
}
__device__ __forceinline__ float nr_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float nr_fma(float a, float b, float c) { return fmaf(a, b, c); }
template <int VEC> __device__ __forceinline__ auto nr_both(float x) {
  if constexpr (VEC == 1) return x; else return nr_pair(x, x);
}
template <int VEC> __device__ __forceinline__ NrVals<VEC> nr_fill(float x) {
  NrVals<VEC> r;
#pragma unroll
  for (int e = 0; e < r.N; ++e) r.p[e] = nr_both<VEC>(x);
  return r;
}
template <int VEC> __device__ __forceinline__ float nr_total(const NrVals<VEC>& a) {
  if constexpr (VEC == 1) {
    return a.p[0];
  } else {
    uint64_t s = a.p[0];
#pragma unroll
    for (int e = 1; e < a.N; ++e) s = nr_add(s, a.p[e]);
    const float2 v = nr_split(s);
    return v.x + v.y;
  }
}

// Memory form <-> 32-bit values.
template <typename T, int VEC>
__device__ __forceinline__ NrVals<VEC> nr_unpack(const Pack<T, VEC>& p) {
  NrVals<VEC> r;
  if constexpr (VEC == 1) {
    r.p[0] = Elt<T>::up(p.e[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) r.p[e] = nr_pair(p.e[2 * e], p.e[2 * e + 1]);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      if constexpr (is_half<T>) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
        r.p[e] = nr_pair(v.x, v.y);
      } else {
        r.p[e] = nr_pair(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
      }
    }
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> nr_pack(const NrVals<VEC>& f) {
  Pack<T, VEC> p;
  if constexpr (VEC == 1) {
    p.e[0] = Elt<T>::down(f.p[0]);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 v = nr_split(f.p[e]);
      if constexpr (sizeof(T) == 4) {
        w[2 * e] = __float_as_uint(v.x);
        w[2 * e + 1] = __float_as_uint(v.y);
      } else if constexpr (is_half<T>) {
        const __half2 h = __floats2half2_rn(v.x, v.y);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[e] = pack_bf16(v.x, v.y);
      }
    }
  }
  return p;
}

// The map of a token's pairs of one task (a rotation, transposed by the sign
// of the table's sines):
//   half layout   y_a = x_a ac + x_b bs, y_b = x_b bc + x_a as
//   interleaved   y_a = x_a ac + swap(x_a) as, y_b = x_b bc + swap(x_b) bs
//   not rotated   y_a = x_a ac, y_b = x_b bc
// Weights w are folded into the factors.
template <int VEC>
struct NrMap {
  NrVals<VEC> ac, as, bc, bs;
  template <bool INTER>
  __device__ __forceinline__ void load(const NrShape& s, bool rot, int t, const float2* tab) {
    ac = bc = nr_fill<VEC>(1.f);
    as = bs = nr_fill<VEC>(0.f);
    if (!rot) return;
    if constexpr (VEC == 1) {
      const float2 v = tab[t];
      ac.p[0] = bc.p[0] = v.x;
      as.p[0] = v.y;
      bs.p[0] = -v.y;
    } else {
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {  // the angles of pairs 2e and 2e + 1
        const float4 v = *reinterpret_cast<const float4*>(tab + 2 * e * s.nrope + 2 * t);
        if constexpr (INTER && VEC == 2) {  // one pair of each vector
          ac.p[0] = nr_pair(v.x, v.x);
          as.p[0] = nr_pair(-v.y, v.y);
          bc.p[0] = nr_pair(v.z, v.z);
          bs.p[0] = nr_pair(-v.w, v.w);
        } else if constexpr (INTER) {
          NrVals<VEC>&c = e < VEC / 4 ? ac : bc, &sn = e < VEC / 4 ? as : bs;
          const int at = e < VEC / 4 ? 2 * e : 2 * e - VEC / 2;
          c.p[at] = nr_pair(v.x, v.x);
          c.p[at + 1] = nr_pair(v.z, v.z);
          sn.p[at] = nr_pair(-v.y, v.y);
          sn.p[at + 1] = nr_pair(-v.w, v.w);
        } else {
          ac.p[e] = bc.p[e] = nr_pair(v.x, v.z);
          as.p[e] = nr_pair(v.y, v.w);
          bs.p[e] = nr_pair(-v.y, -v.w);
        }
      }
    }
  }
  // The weights of the input columns: they come before the rotation.
  template <bool INTER>
  __device__ __forceinline__ void weigh(const NrVals<VEC>& wa, const NrVals<VEC>& wb) {
#pragma unroll
    for (int e = 0; e < ac.N; ++e) {
      ac.p[e] = nr_mul(ac.p[e], wa.p[e]);
      bc.p[e] = nr_mul(bc.p[e], wb.p[e]);
      if constexpr (INTER && VEC > 1) {
        as.p[e] = nr_mul(as.p[e], nr_swap(wa.p[e]));
        bs.p[e] = nr_mul(bs.p[e], nr_swap(wb.p[e]));
      } else {
        as.p[e] = nr_mul(as.p[e], wa.p[e]);
        bs.p[e] = nr_mul(bs.p[e], wb.p[e]);
      }
    }
  }
  template <bool INTER>
  __device__ __forceinline__ void apply(bool rot, NrVals<VEC>& a, NrVals<VEC>& b) const {
    if (!rot) {
#pragma unroll
      for (int e = 0; e < ac.N; ++e) {
        a.p[e] = nr_mul(a.p[e], ac.p[e]);
        b.p[e] = nr_mul(b.p[e], bc.p[e]);
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < ac.N; ++e) {
      if constexpr (INTER && VEC > 1) {
        a.p[e] = nr_fma(a.p[e], ac.p[e], nr_mul(nr_swap(a.p[e]), as.p[e]));
        b.p[e] = nr_fma(b.p[e], bc.p[e], nr_mul(nr_swap(b.p[e]), bs.p[e]));
      } else {
        const auto x = a.p[e];
        a.p[e] = nr_fma(x, ac.p[e], nr_mul(b.p[e], bs.p[e]));
        b.p[e] = nr_fma(b.p[e], bc.p[e], nr_mul(x, as.p[e]));
      }
    }
  }
};

__device__ __forceinline__ float nr_row_sum(float v, int lph) {
  for (int o = lph >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's ring of groups: `STREAMS` tensors, NV tasks of two vectors each.
// Slot layout [slot][vector][lane]: neighbouring lanes are neighbouring
// addresses. Vectors of 2 bytes (which cp.async does not take) and the longest
// rows of single elements are read where they are used instead.
template <typename T, int VEC, int NV, int STREAMS>
struct NrRing {
  static constexpr int kVec = sizeof(T) * VEC;
  static constexpr bool kOn = kVec >= 4 && NV <= 8;
  static constexpr int kVectors = 2 * NV * STREAMS;
  static constexpr int kLine = 32 * kVec;  // one vector of all lanes
  static constexpr int kSlotBytes = kVectors * kLine;
  // 128 KB in flight on an SM
  static constexpr int kWarpBytes = !kOn ? 0 : 131072 / nr_warps_per_sm(VEC, NV);
  static constexpr int kSlots = kOn ? kWarpBytes / kSlotBytes : 2;
  static constexpr int kAhead = kSlots - 1;  // a slot is filled again one group after it was used
  static_assert(kSlots >= 2 && (kWarpBytes & (kWarpBytes - 1)) == 0, "the ring's offsets wrap by a mask");
};

// The tokens [begin, end) of a walk, of `walks` equal ones over them all (at
// most 2^30 tokens). The forward counts them in 32 bits, the backward in 64:
// each is what the register allocator made the faster kernel of (72 against 75
// us, 198 against 200).
template <typename I>
__device__ __forceinline__ void nr_share(const NrShape& s, int walk, int walks, I& begin, I& end) {
  begin = (I)(s.tokens * walk / walks);
  end = (I)(s.tokens * (walk + 1) / walks);
}

// NORM: a side has weights (else the kernel is the rotation alone); INTER: the
// interleaved layout (with one element per vector both are the same code).
template <typename T, int VEC, int NV, bool NORM, bool INTER>
__global__ void __launch_bounds__(32, nr_warps_per_sm(VEC, NV)) norm_rope_kernel(const NrFwdParams p) {
  using Ring = NrRing<T, VEC, NV, 1>;
  using P = Pack<T, VEC>;
  extern __shared__ __align__(16) uint8_t nr_bytes[];
  const NrShape& s = p.s;
  float2* const tables = reinterpret_cast<float2*>(nr_bytes + Ring::kWarpBytes);  // two batches' angles
  const int table_size = p.batch * s.pairs;
  const int lane = threadIdx.x;
  const uint8_t* ring = nr_bytes + lane * Ring::kVec;
  const uint32_t ring_addr = smem_u32(ring);
  int begin, end;
  if (p.walk) {
    begin = (int)blockIdx.x * p.walk;
    end = (int)min(s.tokens, (int64_t)begin + p.walk);
  } else {
    nr_share(s, blockIdx.x >> p.wide_log, p.walks, begin, end);
  }
  const int lph = 1 << s.lph_log, t0 = lane & (lph - 1), sub = lane >> s.lph_log, rows = 32 >> s.lph_log;
  NrTask<VEC> task[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) task[v] = NrTask<VEC>(s, t0 + v * lph);
  const int vper = p.d_v / VEC, nvec = p.k.heads * vper;
  const int share = blockIdx.x & ((1 << p.wide_log) - 1);  // of a token's groups

  // The cursor: the group asked for next. kind 0: queries, 1: keys, 2: values.
  int c_tok = begin - 1;
  int c_kind = 2, c_g = 0, c_end = 0, c_hop = 0;  // first row (values: first vector), their number, the next group's
  int64_t c_xhop = 0;
  const T* c_x = nullptr;
  int c_oa[NV], c_ob[NV], c_la[NV], c_lb[NV];  // offsets of this lane's vectors, and their rows (vectors) after c_g
  constexpr int kNone = 1 << 30;               // a row that is never there
  uint32_t in_at = 0, out_at = 0;
  auto ask = [&]() {
    if constexpr (Ring::kOn) {
      if (c_g >= c_end) {  // to the next side or token that has something for this warp
        while (c_g >= c_end && c_tok < end) {
          if (++c_kind == 3) {
            c_kind = 0;
            if (++c_tok >= end) break;
          }
          if (c_kind == 2) {
            c_g = share * 64;
            c_end = nvec;
            c_hop = 64;
            c_x = static_cast<const T*>(p.v) + c_tok * p.v_stride + (int64_t)(c_g + lane) * VEC;
            c_xhop = (int64_t)(64 << p.wide_log) * VEC;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              c_oa[v] = 0;
              c_ob[v] = 32 * VEC;
              c_la[v] = v == 0 ? lane : kNone;
              c_lb[v] = v == 0 ? lane + 32 : kNone;
            }
          } else {
            auto side = [&](const NrSide& sd) {
              c_g = share * rows;
              c_end = sd.heads;
              c_hop = rows;
              c_x = static_cast<const T*>(sd.x) + c_tok * sd.x_stride + (int64_t)(c_g + sub) * s.d;
              c_xhop = (int64_t)(rows << p.wide_log) * s.d;
#pragma unroll
              for (int v = 0; v < NV; ++v) {
                const bool on = task[v].rot || !sd.skip_pass;
                c_oa[v] = max(task[v].a, 0);  // no task: an aligned address that is not read
                c_ob[v] = max(task[v].b, 0);
                c_la[v] = on && task[v].a >= 0 ? sub : kNone;
                c_lb[v] = on && task[v].b >= 0 ? sub : kNone;
              }
            };
            if (c_kind == 0) side(p.q); else side(p.k);
          }
          c_hop <<= p.wide_log;
        }
      }
      if (c_g < c_end) {  // the same for the whole warp
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const uint32_t dst = ring_addr + in_at + v * 2 * Ring::kLine;
          cp_async<Ring::kVec>(dst, c_x + c_oa[v], c_g + c_la[v] < c_end ? Ring::kVec : 0);
          cp_async<Ring::kVec>(dst + Ring::kLine, c_x + c_ob[v], c_g + c_lb[v] < c_end ? Ring::kVec : 0);
        }
        in_at = (in_at + Ring::kSlotBytes) & (Ring::kWarpBytes - 1);
        c_g += c_hop;
        c_x += c_xhop;
      }
      cp_async_commit();
    }
  };
  // The next group of the ring, into registers; its slot is asked for again after the one that was used before it.
  auto take = [&](P (&a)[NV], P (&b)[NV]) {
    if constexpr (Ring::kOn) {
      cp_async_wait<Ring::kAhead - 1>();
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint8_t* at = ring + out_at + v * 2 * Ring::kLine;
        a[v] = *reinterpret_cast<const P*>(at);
        b[v] = *reinterpret_cast<const P*>(at + Ring::kLine);
      }
      out_at = (out_at + Ring::kSlotBytes) & (Ring::kWarpBytes - 1);
      ask();
    }
  };
  if constexpr (Ring::kOn) {
#pragma unroll 1
    for (int k = 0; k < Ring::kAhead; ++k) ask();
  }
  int64_t slot_next = p.slots && begin < end ? p.slots[begin] : -1;  // the next token's
  nr_angles<VEC, INTER, 32>(s, begin, min(p.batch, end - begin), tables);

  int turn = 0;
  for (int tok0 = begin; tok0 < end; tok0 += p.batch, turn ^= 1) {
    const int n = min(p.batch, end - tok0);
    __syncwarp();  // this batch's angles are there, and the other table's have been read
    if (tok0 + n < end)
      nr_angles<VEC, INTER, 32>(s, tok0 + n, min(p.batch, end - tok0 - n), tables + (turn ^ 1) * table_size);
    const float2* tab = tables + turn * table_size;
    for (int i = 0; i < n; ++i) {
      const int tok = tok0 + i;
      const int64_t slot = slot_next;
      if (p.slots) slot_next = tok + 1 < end ? p.slots[tok + 1] : -1;
      const bool pooled = slot >= 0 && slot < p.n_slots;  // else a padded row, or a page that is not there
      const int64_t page = slot >> p.page_shift, prow = slot & ((1 << p.page_shift) - 1);
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {  // unrolled: the sides' parameters at fixed places
        const NrSide& sd = kind == 0 ? p.q : p.k;
        const int heads = sd.heads, hop = rows << p.wide_log, g0 = share * rows, h = g0 + sub;
        if (g0 >= heads) continue;
        T *o = nullptr, *o2 = nullptr;
        int64_t ohop = 0, o2hop = 0;
        P xa[NV], xb[NV];
        const T* w = static_cast<const T*>(sd.w);
        const bool norm = NORM && w != nullptr;
        const T* x = static_cast<const T*>(sd.x) + tok * sd.x_stride + (int64_t)h * s.d;
        if (pooled && kind == 1) {
          o = static_cast<T*>(p.k_pool.base) + page * p.k_pool.page_stride + prow * p.k_pool.row_stride +
              h * p.k_pool.head_stride;
          ohop = hop * p.k_pool.head_stride;
        }
        if (sd.out) {  // its own rows, the pool or (rarely) both
          o2 = o;
          o2hop = ohop;
          o = static_cast<T*>(sd.out) + tok * sd.out_stride + (int64_t)h * s.d;
          ohop = (int64_t)hop * s.d;
        }
        // the lane's columns of each task: none where nothing changes in place
        int ca[NV], cb[NV];
        bool norm_a[NV], norm_b[NV];
        NrMap<VEC> map[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const bool on = task[v].rot || !sd.skip_pass;
          ca[v] = on ? task[v].a : -1;
          cb[v] = on ? task[v].b : -1;
          norm_a[v] = norm && (unsigned)ca[v] < (unsigned)s.norm_dim;
          norm_b[v] = norm && (unsigned)cb[v] < (unsigned)s.norm_dim;
          map[v].template load<INTER>(s, task[v].rot, t0 + v * lph, tab + i * s.pairs);
          if (norm) {
            NrVals<VEC> wa = nr_fill<VEC>(1.f), wb = wa;
            if (norm_a[v]) wa = nr_unpack<T, VEC>(*reinterpret_cast<const P*>(w + ca[v]));
            if (norm_b[v]) wb = nr_unpack<T, VEC>(*reinterpret_cast<const P*>(w + cb[v]));
            map[v].template weigh<INTER>(wa, wb);
          }
        }
        for (int g = g0; g < heads; g += hop) {
          const bool in = g + sub < heads;
          if constexpr (Ring::kOn) {
            take(xa, xb);
          } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              xa[v] = xb[v] = pack_zero<T, VEC>();
              if (in && ca[v] >= 0) xa[v] = *reinterpret_cast<const P*>(x + ca[v]);
              if (in && cb[v] >= 0) xb[v] = *reinterpret_cast<const P*>(x + cb[v]);
            }
            x += (int64_t)hop * s.d;
          }
          if (norm) {
            NrVals<VEC> fa[NV], fb[NV], sq = nr_fill<VEC>(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              fa[v] = nr_unpack<T, VEC>(xa[v]);
              fb[v] = nr_unpack<T, VEC>(xb[v]);
              if (norm_a[v])
#pragma unroll
                for (int e = 0; e < sq.N; ++e) sq.p[e] = nr_fma(fa[v].p[e], fa[v].p[e], sq.p[e]);
              if (norm_b[v])
#pragma unroll
                for (int e = 0; e < sq.N; ++e) sq.p[e] = nr_fma(fb[v].p[e], fb[v].p[e], sq.p[e]);
            }
            const float r = rsqrtf(fmaf(nr_row_sum(nr_total<VEC>(sq), lph), s.inv_norm, s.eps));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const auto ra = nr_both<VEC>(norm_a[v] ? r : 1.f), rb = nr_both<VEC>(norm_b[v] ? r : 1.f);
#pragma unroll
              for (int e = 0; e < sq.N; ++e) {
                fa[v].p[e] = nr_mul(fa[v].p[e], ra);
                fb[v].p[e] = nr_mul(fb[v].p[e], rb);
              }
              map[v].template apply<INTER>(task[v].rot, fa[v], fb[v]);
              xa[v] = nr_pack<T, VEC>(fa[v]);
              xb[v] = nr_pack<T, VEC>(fb[v]);
            }
          } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
              if (task[v].rot) {
                NrVals<VEC> fa = nr_unpack<T, VEC>(xa[v]), fb = nr_unpack<T, VEC>(xb[v]);
                map[v].template apply<INTER>(true, fa, fb);
                xa[v] = nr_pack<T, VEC>(fa);
                xb[v] = nr_pack<T, VEC>(fb);
              }
          }
          if (in && o) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (ca[v] >= 0) *reinterpret_cast<P*>(o + ca[v]) = xa[v];
              if (cb[v] >= 0) *reinterpret_cast<P*>(o + cb[v]) = xb[v];
              if (o2) {
                if (ca[v] >= 0) *reinterpret_cast<P*>(o2 + ca[v]) = xa[v];
                if (cb[v] >= 0) *reinterpret_cast<P*>(o2 + cb[v]) = xb[v];
              }
            }
          }
          if (o) o += ohop;
          if (o2) o2 += o2hop;
        }
      }
      if (nvec == 0) continue;
      T* dst = pooled ? static_cast<T*>(p.v_pool.base) + page * p.v_pool.page_stride + prow * p.v_pool.row_stride
                      : nullptr;
      auto v_at = [&](int x) {
        const int vh = p.vper_log >= 0 ? x >> p.vper_log : x / vper;
        return dst + vh * p.v_pool.head_stride + (int64_t)(x - vh * vper) * VEC;
      };
      if constexpr (Ring::kOn) {
        P va[NV], vb[NV];
        for (int g = share * 64; g < nvec; g += 64 << p.wide_log) {
          take(va, vb);
          if (dst && g + lane < nvec) *reinterpret_cast<P*>(v_at(g + lane)) = va[0];
          if (dst && g + lane + 32 < nvec) *reinterpret_cast<P*>(v_at(g + lane + 32)) = vb[0];
        }
      } else if (dst) {
        const T* src = static_cast<const T*>(p.v) + tok * p.v_stride;
        for (int x = share * 32 + lane; x < nvec; x += 32 << p.wide_log) *v_at(x) = src[x];
      }
    }
  }
}

// Every CTA walks its tokens twice, the query rows and then the key rows, so
// that a warp has one set of weight gradients in registers.
template <typename T, int VEC, int NV, bool INTER>
__global__ void __launch_bounds__(kNrThreads, nr_ctas_per_sm(VEC, NV)) norm_rope_backward_kernel(const NrBwdParams p) {
  using Ring = NrRing<T, VEC, NV, 2>;
  using P = Pack<T, VEC>;
  extern __shared__ __align__(16) uint8_t nr_bytes[];
  // two batches' angles; at the end of a side kNrWarps rows of norm_dim sums
  float2* const tables = reinterpret_cast<float2*>(nr_bytes + kNrWarps * Ring::kWarpBytes);
  const NrShape& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* ring = nr_bytes + warp * Ring::kWarpBytes + lane * Ring::kVec;
  const uint32_t ring_addr = smem_u32(ring);
  int64_t begin, end;
  nr_share(s, blockIdx.x, gridDim.x, begin, end);
  const int lph = s.lph, t0 = lane & (lph - 1), rows = 32 / lph, sub = lane / lph;
  const int share = warp & ((1 << p.wide_log) - 1), tok_first = warp >> p.wide_log, tok_step = kNrWarps >> p.wide_log;
  NrTask<VEC> task[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) task[v] = NrTask<VEC>(s, t0 + v * lph);

#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const NrSide& sd = side == 0 ? p.q : p.k;
    const int heads = sd.heads;
    if (heads == 0) continue;
    const int batch = p.batch;
    const int table_size = batch * s.pairs, hop = rows << p.wide_log, g0 = share * rows;
    const int64_t xhop = (int64_t)hop * s.d;
    const T* w = static_cast<const T*>(sd.w);
    const bool norm = w != nullptr;
    bool norm_a[NV], norm_b[NV];
    P wa[NV], wb[NV];
    NrVals<VEC> dwa[NV], dwb[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      norm_a[v] = norm && (unsigned)task[v].a < (unsigned)s.norm_dim;
      norm_b[v] = norm && (unsigned)task[v].b < (unsigned)s.norm_dim;
      wa[v] = wb[v] = pack_zero<T, VEC>();
      if (norm_a[v]) wa[v] = *reinterpret_cast<const P*>(w + task[v].a);
      if (norm_b[v]) wb[v] = *reinterpret_cast<const P*>(w + task[v].b);
      dwa[v] = dwb[v] = nr_fill<VEC>(0.f);
    }
    // The cursor: the group asked for next.
    int64_t c_tok = begin + tok_first - tok_step;
    int c_g = heads;
    const T *c_x = nullptr, *c_y = nullptr;
    uint32_t in_at = 0, out_at = 0;
    auto ask = [&]() {
      if constexpr (Ring::kOn) {
        if (c_g >= heads && g0 < heads && c_tok < end) {  // to the next token
          c_tok += tok_step;
          if (c_tok < end) {
            c_g = g0;
            c_x = static_cast<const T*>(sd.x) + c_tok * sd.x_stride + (int64_t)(g0 + sub) * s.d;
            c_y = static_cast<const T*>(sd.dy) + c_tok * sd.dy_stride + (int64_t)(g0 + sub) * s.d;
          }
        }
        if (c_g < heads) {  // the same for the whole warp
          const bool here = c_g + sub < heads;  // rows behind the last head are zeros: they add nothing
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const uint32_t dst = ring_addr + in_at + v * 4 * Ring::kLine;
            if (task[v].a >= 0) cp_async<Ring::kVec>(dst, c_y + task[v].a, here ? Ring::kVec : 0);
            if (task[v].b >= 0) cp_async<Ring::kVec>(dst + Ring::kLine, c_y + task[v].b, here ? Ring::kVec : 0);
            if (norm_a[v]) cp_async<Ring::kVec>(dst + 2 * Ring::kLine, c_x + task[v].a, here ? Ring::kVec : 0);
            if (norm_b[v]) cp_async<Ring::kVec>(dst + 3 * Ring::kLine, c_x + task[v].b, here ? Ring::kVec : 0);
          }
          in_at = (in_at + Ring::kSlotBytes) & (Ring::kWarpBytes - 1);
          c_g += hop;
          c_x += xhop;
          c_y += xhop;
        }
        cp_async_commit();
      }
    };
    if constexpr (Ring::kOn) {
#pragma unroll 1
      for (int k = 0; k < Ring::kAhead; ++k) ask();
    }
    __syncthreads();  // the other side's sums have been read
    nr_angles<VEC, INTER, kNrThreads>(s, begin, (int)min((int64_t)batch, end - begin), tables);

    int turn = 0;
    for (int64_t tok0 = begin; tok0 < end; tok0 += batch, turn ^= 1) {
      const int n = (int)min((int64_t)batch, end - tok0);
      __syncthreads();  // this batch's angles are there, and the other table's have been read
      if (tok0 + n < end)
        nr_angles<VEC, INTER, kNrThreads>(s, tok0 + n, (int)min((int64_t)batch, end - tok0 - n), tables + (turn ^ 1) * table_size);
      const float2* tab = tables + turn * table_size;
      for (int i = tok_first; i < n; i += tok_step) {
        const int h = g0 + sub;
        const int64_t tok = tok0 + i;
        const T* x = static_cast<const T*>(sd.x) + tok * sd.x_stride + (int64_t)h * s.d;
        const T* y = static_cast<const T*>(sd.dy) + tok * sd.dy_stride + (int64_t)h * s.d;
        T* o = static_cast<T*>(sd.out) + tok * sd.out_stride + (int64_t)h * s.d;
        NrMap<VEC> map[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v)
          map[v].template load<INTER>(s, task[v].rot, t0 + v * lph, tab + i * s.pairs);
        for (int g = g0; g < heads; g += hop) {
          const bool in = g + sub < heads;
          P xa[NV], xb[NV], ya[NV], yb[NV];
          if constexpr (Ring::kOn) {
            cp_async_wait<Ring::kAhead - 1>();
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const uint8_t* at = ring + out_at + v * 4 * Ring::kLine;
              ya[v] = *reinterpret_cast<const P*>(at);
              yb[v] = *reinterpret_cast<const P*>(at + Ring::kLine);
              xa[v] = *reinterpret_cast<const P*>(at + 2 * Ring::kLine);
              xb[v] = *reinterpret_cast<const P*>(at + 3 * Ring::kLine);
            }
            out_at = (out_at + Ring::kSlotBytes) & (Ring::kWarpBytes - 1);
            ask();
          } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              xa[v] = xb[v] = ya[v] = yb[v] = pack_zero<T, VEC>();
              if (in && task[v].a >= 0) ya[v] = *reinterpret_cast<const P*>(y + task[v].a);
              if (in && task[v].b >= 0) yb[v] = *reinterpret_cast<const P*>(y + task[v].b);
              if (in && norm_a[v]) xa[v] = *reinterpret_cast<const P*>(x + task[v].a);
              if (in && norm_b[v]) xb[v] = *reinterpret_cast<const P*>(x + task[v].b);
            }
            x += xhop;
            y += xhop;
          }
          NrVals<VEC> fa[NV], fb[NV];  // dn
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            fa[v] = nr_unpack<T, VEC>(ya[v]);
            fb[v] = nr_unpack<T, VEC>(yb[v]);
            if (task[v].rot) map[v].template apply<INTER>(true, fa[v], fb[v]);
          }
          if (norm) {
            NrVals<VEC> sq = nr_fill<VEC>(0.f), dot = sq;  // sums of x^2 and g x
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (norm_a[v]) {
                const NrVals<VEC> x_ = nr_unpack<T, VEC>(xa[v]), w_ = nr_unpack<T, VEC>(wa[v]);
#pragma unroll
                for (int e = 0; e < sq.N; ++e) {
                  sq.p[e] = nr_fma(x_.p[e], x_.p[e], sq.p[e]);
                  dot.p[e] = nr_fma(nr_mul(fa[v].p[e], w_.p[e]), x_.p[e], dot.p[e]);
                }
              }
              if (norm_b[v]) {
                const NrVals<VEC> x_ = nr_unpack<T, VEC>(xb[v]), w_ = nr_unpack<T, VEC>(wb[v]);
#pragma unroll
                for (int e = 0; e < sq.N; ++e) {
                  sq.p[e] = nr_fma(x_.p[e], x_.p[e], sq.p[e]);
                  dot.p[e] = nr_fma(nr_mul(fb[v].p[e], w_.p[e]), x_.p[e], dot.p[e]);
                }
              }
            }
            const float ms = nr_row_sum(nr_total<VEC>(sq), lph), mg = nr_row_sum(nr_total<VEC>(dot), lph);
            const float r1 = in ? rsqrtf(fmaf(ms, s.inv_norm, s.eps)) : 0.f;  // eps may be 0
            const auto r = nr_both<VEC>(r1), c = nr_both<VEC>(-mg * r1 * r1 * s.inv_norm);  // c: -mean(g u) / rms
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (norm_a[v]) {
                const NrVals<VEC> x_ = nr_unpack<T, VEC>(xa[v]), w_ = nr_unpack<T, VEC>(wa[v]);
#pragma unroll
                for (int e = 0; e < sq.N; ++e) {
                  const auto u = nr_mul(x_.p[e], r), g_ = nr_mul(fa[v].p[e], w_.p[e]);
                  dwa[v].p[e] = nr_fma(fa[v].p[e], u, dwa[v].p[e]);
                  fa[v].p[e] = nr_fma(g_, r, nr_mul(u, c));
                }
              }
              if (norm_b[v]) {
                const NrVals<VEC> x_ = nr_unpack<T, VEC>(xb[v]), w_ = nr_unpack<T, VEC>(wb[v]);
#pragma unroll
                for (int e = 0; e < sq.N; ++e) {
                  const auto u = nr_mul(x_.p[e], r), g_ = nr_mul(fb[v].p[e], w_.p[e]);
                  dwb[v].p[e] = nr_fma(fb[v].p[e], u, dwb[v].p[e]);
                  fb[v].p[e] = nr_fma(g_, r, nr_mul(u, c));
                }
              }
            }
          }
          if (in) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (task[v].a >= 0) *reinterpret_cast<P*>(o + task[v].a) = nr_pack<T, VEC>(fa[v]);
              if (task[v].b >= 0) *reinterpret_cast<P*>(o + task[v].b) = nr_pack<T, VEC>(fb[v]);
            }
          }
          o += xhop;
        }
      }
    }
    if constexpr (Ring::kOn) cp_async_wait<0>();  // nothing but empty groups is left
    if (!norm) continue;  // the same for the whole CTA
    __syncthreads();      // the last angles have been read
    float* sums = reinterpret_cast<float*>(tables);
    // a lane's sums of one vector: over the rows of the warp that share its columns, then to the CTA
    auto leave = [&](const NrVals<VEC>& dw, int col, bool on) {
#pragma unroll
      for (int e = 0; e < dw.N; ++e) {
        float v[VEC == 1 ? 1 : 2];
        if constexpr (VEC == 1) {
          v[0] = dw.p[0];
        } else {
          v[0] = nr_split(dw.p[e]).x;
          v[1] = nr_split(dw.p[e]).y;
        }
#pragma unroll
        for (int j = 0; j < (VEC == 1 ? 1 : 2); ++j) {
          for (int o = lph; o < 32; o <<= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
          if (sub == 0 && on) sums[warp * s.norm_dim + col + 2 * e + j] = v[j];
        }
      }
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      leave(dwa[v], task[v].a, norm_a[v]);
      leave(dwb[v], task[v].b, norm_b[v]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < s.norm_dim; c += kNrThreads) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kNrWarps; ++k) t += sums[k * s.norm_dim + c];
      p.partial[((size_t)side * gridDim.x + blockIdx.x) * s.norm_dim + c] = t;
    }
  }
  griddep_launch_dependents();
}

}  // namespace loza
