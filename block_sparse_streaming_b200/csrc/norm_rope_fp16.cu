// norm_rope_fp16.cu - the norm and rotation kernels of one element type.
#include <cuda_bf16.h>

#include "norm_rope_launch.cuh"

namespace loza {
LOZA_NR_INSTANCES(, __half);
}
