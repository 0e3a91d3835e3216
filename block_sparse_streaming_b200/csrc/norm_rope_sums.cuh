// norm_rope_sums.cuh - the weights' gradients of norm_rope.cuh, from the sums that its CTAs leave.
#pragma once

#include "sm100.cuh"

namespace loza {

// dw[side][c] = sum over the CTAs of partial[side][cta][c], in a fixed order:
// 8 columns per block, 64 threads per column each over every 64th CTA, so that
// the few loads of a thread are all in flight at once.
struct NrDwParams {
  const float* partial;
  float *dqw, *dkw;
  int norm_dim, ctas;
};
__global__ void __launch_bounds__(512) norm_rope_dw_kernel(const NrDwParams p) {
  __shared__ float part[64][9];
  const int x = threadIdx.x & 7, col = blockIdx.x * 8 + x, j = threadIdx.x >> 3;
  float* out = blockIdx.y == 0 ? p.dqw : p.dkw;
  griddep_wait();
  if (!out) return;
  const float* in = p.partial + (size_t)blockIdx.y * p.ctas * p.norm_dim;
  float t = 0.f;
  if (col < p.norm_dim) {
#pragma unroll 8
    for (int c = j; c < p.ctas; c += 64) t += in[(size_t)c * p.norm_dim + col];
  }
  part[j][x] = t;
  __syncthreads();
  if (j < 4) {  // 16 parts each, then the four
    t = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += part[j * 16 + k][x];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if (j == 0 && col < p.norm_dim) out[col] = t;
  }
}

}  // namespace loza
