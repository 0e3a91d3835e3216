// norm_rope_launch.cuh - launches of the kernels of norm_rope.cuh: shared memory, and the instance for a call.
#pragma once

#include <algorithm>

#include "norm_rope.cuh"

namespace loza {

// Angles of a batch, per warp: 2 KB leave room on an SM for 16 warps with two batches and a ring each; one token of
// the longest table (512 pairs, 4 KB) always fits, beside 7 others (rows that long run 8 warps per SM anyway).
constexpr int64_t kNrTableBytes = 2048;

// Most bytes that an instance's table of one batch takes (see nr_batch): its share per warp, or one token per warp.
constexpr int64_t nr_most_table(int warps, int vec, int nv) {
  return warps * std::max(kNrTableBytes, std::min<int64_t>(512, 32 * vec * nv) * (int64_t)sizeof(float2));
}

template <typename T, int VEC, int NV, bool NORM, bool INTER>
bool nr_launch_fwd(const NrFwdParams& p, cudaStream_t st) {
  using Ring = NrRing<T, VEC, NV, 1>;
  static_assert(Ring::kWarpBytes + 2 * nr_most_table(1, VEC, NV) <= 48 * 1024, "no opt-in to more shared memory");
  const size_t smem = Ring::kWarpBytes + (size_t)2 * p.batch * p.s.pairs * sizeof(float2);
  norm_rope_kernel<T, VEC, NV, NORM, INTER><<<(unsigned)(p.walks << p.wide_log), 32, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess;
}

template <typename T, int VEC, int NV, bool INTER>
bool nr_launch_bwd(const NrBwdParams& p, int ctas, cudaStream_t st) {
  auto kernel = norm_rope_backward_kernel<T, VEC, NV, INTER>;
  using Ring = NrRing<T, VEC, NV, 2>;
  // The kernel's limit is the context's, and threads may launch other sizes of this instance at this moment: all of
  // them set the most that the instance can ask for. (What a CTA occupies is the launch's own size.)
  constexpr int64_t most =
      kNrWarps * Ring::kWarpBytes +
      std::max<int64_t>(2 * nr_most_table(kNrWarps, VEC, NV), kNrWarps * std::min(1024, 64 * VEC * NV) * sizeof(float));
  static_assert(most <= 227 * 1024, "shared memory of a CTA");
  const size_t smem = (size_t)kNrWarps * Ring::kWarpBytes +
                      std::max((size_t)2 * p.batch * p.s.pairs * sizeof(float2),
                               (size_t)kNrWarps * p.s.norm_dim * sizeof(float));
  if (most > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess)
    return false;
  kernel<<<(unsigned)ctas, kNrThreads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess;
}

// One element per vector: both layouts are one kernel, and the rotation alone is the kernel of the norm.
template <typename T, int VEC, int NV>
bool nr_launch(const NrFwdParams& p, int, cudaStream_t st) {
  const bool norm = p.q.w || p.k.w;
  if constexpr (VEC == 1) return nr_launch_fwd<T, VEC, NV, true, false>(p, st);
  else if (p.s.interleaved)
    return norm ? nr_launch_fwd<T, VEC, NV, true, true>(p, st) : nr_launch_fwd<T, VEC, NV, false, true>(p, st);
  else
    return norm ? nr_launch_fwd<T, VEC, NV, true, false>(p, st) : nr_launch_fwd<T, VEC, NV, false, false>(p, st);
}
template <typename T, int VEC, int NV>
bool nr_launch(const NrBwdParams& p, int ctas, cudaStream_t st) {
  if constexpr (VEC == 1) return nr_launch_bwd<T, VEC, NV, false>(p, ctas, st);
  else
    return p.s.interleaved ? nr_launch_bwd<T, VEC, NV, true>(p, ctas, st)
                           : nr_launch_bwd<T, VEC, NV, false>(p, ctas, st);
}

// The instance for a vector length and tasks per lane (see nr_vec and nr_tasks). Each type's are compiled in a file of
// their own (norm_rope_bf16.cu and its siblings), at the same time.
template <typename T, typename Params>
bool nr_run_type(const Params& p, int vec, int nv, int ctas, cudaStream_t st) {
  if constexpr (sizeof(T) == 4) {
    if (vec == 4)
      return nv == 1   ? nr_launch<T, 4, 1>(p, ctas, st)
             : nv == 2 ? nr_launch<T, 4, 2>(p, ctas, st)
                       : nr_launch<T, 4, 4>(p, ctas, st);
  } else {
    if (vec == 8) return nv == 1 ? nr_launch<T, 8, 1>(p, ctas, st) : nr_launch<T, 8, 2>(p, ctas, st);
    if (vec == 2) return nv == 4 ? nr_launch<T, 2, 4>(p, ctas, st) : nr_launch<T, 2, 8>(p, ctas, st);
  }
  return nv == 4 ? nr_launch<T, 1, 4>(p, ctas, st) : nr_launch<T, 1, 16>(p, ctas, st);
}
#define LOZA_NR_INSTANCES(PREFIX, T)                                                                 \
  PREFIX template bool nr_run_type<T, NrFwdParams>(const NrFwdParams&, int, int, int, cudaStream_t); \
  PREFIX template bool nr_run_type<T, NrBwdParams>(const NrBwdParams&, int, int, int, cudaStream_t)

}  // namespace loza
