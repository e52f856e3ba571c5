// norm_bwd_bf16.cu -- the norms' gradient (norm_bwd.cuh) for a bf16 stream.
#include "norm_bwd.cuh"

namespace moe {

cudaError_t launch_norm_bwd_bf16(const NormArgs& a, int v, int chunks, cudaStream_t st, int* parts) {
  return v == 8 ? launch_source<ROW_BF16, 8>(a, chunks, st, parts) : launch_source<ROW_BF16, 1>(a, chunks, st, parts);
}

}  // namespace moe
