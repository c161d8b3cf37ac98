// Prompts of the linear attention (simple form): token after token.
#include "kda_linear.cuh"

namespace kda {
namespace {

__global__ void check_offsets_kernel(LinearProblem p) {
  for (int n = blockIdx.x * blockDim.x + threadIdx.x; n < p.n_seq; n += gridDim.x * blockDim.x)
    if (!offsets_good(p, n)) atomicExch(p.status, (int)KDA_ERR_INVALID_ARG);
}

}  // namespace

size_t linear_fwd_workspace_bytes(int, int, int, int, bool) { return 0; }

cudaError_t launch_linear_fwd(const LinearProblem& p, void*, cudaStream_t stream) {
  if (p.cu_seqlens) check_offsets_kernel<<<1, 256, 0, stream>>>(p);
  return launch_linear_tokens(p, stream);
}

}  // namespace kda
