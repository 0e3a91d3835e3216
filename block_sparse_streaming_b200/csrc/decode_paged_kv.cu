// decode_paged_kv.cu - launches of the paged K/V decode: the instance for a type, head dims and query heads per key head.
#include "decode_paged_kv.cuh"
#include "launch_after.cuh"

namespace loza {

template <typename T, int DQK, int DV, int NT>
bool pkv_launch(const PagedKvParams& p, cudaStream_t st) {
  auto kernel = decode_paged_kv_kernel<T, DQK, DV, NT>;
  constexpr int smem = PagedKvLayout<DQK, DV, NT>::kSmem;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return false;
  kernel<<<(unsigned)p.ctas, kPkvThreads, smem, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return false;
  return launch_after(decode_paged_join_kernel<T, DV>, dim3(p.ctas, p.chunk), 256, st, p);
}

template <typename T>
bool pkv_run(const PagedKvParams& p, int d_qk, cudaStream_t st) {
  const bool wide = p.chunk > 8;  // more than one tile of 8 query heads
  if (d_qk == 64) return wide ? pkv_launch<T, 64, 64, 2>(p, st) : pkv_launch<T, 64, 64, 1>(p, st);
  if (d_qk == 128) return wide ? pkv_launch<T, 128, 128, 2>(p, st) : pkv_launch<T, 128, 128, 1>(p, st);
  return wide ? pkv_launch<T, 192, 128, 2>(p, st) : pkv_launch<T, 192, 128, 1>(p, st);
}

template bool pkv_run<__nv_bfloat16>(const PagedKvParams&, int, cudaStream_t);
template bool pkv_run<__half>(const PagedKvParams&, int, cudaStream_t);

}  // namespace loza
