// norm_bwd_fp32_odd.cu -- the norms' gradient (norm_bwd.cuh) for an fp32 stream, rows at any element.
#include "norm_bwd.cuh"

namespace moe {

cudaError_t launch_norm_bwd_fp32_odd(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  return launch_source<ROW_FP32, 1>(a, chunks, st, parts);
}

}  // namespace moe
