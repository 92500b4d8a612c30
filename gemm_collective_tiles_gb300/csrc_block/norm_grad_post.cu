// The norm gradient's kernels with a post-norm.
#include "norm_grad.cuh"

int gct::block::norm_grad_post(const NormGradParams& p, const NormGradPlan& pl, int y_type, int x_type, cudaStream_t stream) {
    return launch_norm_grad<true>(p, pl, y_type, x_type, stream);
}
