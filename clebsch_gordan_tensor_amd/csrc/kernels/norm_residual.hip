// Normalisation of x + residual and its gradients (norm_kernels.h).
#include "norm_kernels.h"

namespace e3k {

hipError_t launch_norm_residual(bool bwd, const NormArgs& a, const NormBlock* blocks, int n_blocks,
                                int bf16, hipStream_t s) {
  return launch_mode<kNormResidual>(bwd, a, blocks, n_blocks, bf16, s);
}

}  // namespace e3k
