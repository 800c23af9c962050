// Normalisation with its results in 8 bits, with and without a residual
// (norm_kernels.h).
#include "norm_kernels.h"

namespace e3k {

hipError_t launch_norm_fp8(const NormArgs& a, const NormBlock* blocks, int n_blocks, int bf16,
                           hipStream_t s) {
  return a.add ? launch_mode<kNormResidual | kNormFp8>(false, a, blocks, n_blocks, bf16, s)
               : launch_mode<kNormFp8>(false, a, blocks, n_blocks, bf16, s);
}

}  // namespace e3k
