// Normalisation of irreps features and its gradients (norm_kernels.h).
#include "norm_kernels.h"

namespace e3k {

size_t norm_part_floats(int64_t n_rows, int dim, int C, const NormBlock* blocks, int n_blocks,
                        int esize) {
  NormArgs a{};
  a.n_rows = n_rows;
  a.dim = dim;
  a.C = C;
  const auto [scalars, top] = scalars_and_top(blocks, n_blocks);
  if (whole_rows(C, n_blocks, scalars, top, true, esize))
    return size_t(plan_whole(a, blocks, n_blocks, true)) * n_blocks * 2 * C;
  if (staged(C, dim, n_blocks))
    return size_t(plan_staged(a, blocks, n_blocks, esize)) * n_blocks * 2 * C;
  size_t most = 0;
  (void)for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, int top) {
    most = std::max(most, size_t(plan(a, run, m, top, true, esize)) * 2 * C);
    return hipSuccess;
  });
  return most;
}

hipError_t launch_norm(bool bwd, const NormArgs& a, const NormBlock* blocks, int n_blocks,
                       int bf16, hipStream_t s) {
  return a.add ? launch_norm_residual(bwd, a, blocks, n_blocks, bf16, s)
               : launch_mode<0>(bwd, a, blocks, n_blocks, bf16, s);
}

}  // namespace e3k
