// What the two files that hold the norm gradient's kernels share: those without a
// post-norm, and those with one (half the time to compile each).
#pragma once
#include "norm_host.cuh"

namespace gct {
namespace block {

struct NormGradPlan {
    RowShape r;
    // kept: rows come ahead, and the vectors lie in shared memory; all: so do those of x, dh
    // and dn, in pieces
    bool in_registers, vec, kept, all;
    int64_t ctas;
    size_t smem, part, total;
};
// the kernels with a post-norm
int norm_grad_post(const NormGradParams& p, const NormGradPlan& pl, int y_type, int x_type, cudaStream_t stream);

}  // namespace block
}  // namespace gct

namespace {

template <bool POST>
int launch_norm_grad(const NormGradParams& p, const NormGradPlan& pl, int y_type, int x_type, cudaStream_t stream) {
    return by_types(y_type, x_type, [&](auto ty, auto tx) {
        constexpr int TY = decltype(ty)::value, TX = decltype(tx)::value, W = TX == T_F32 ? 4 : 8;
        const bool one = pl.r.C == 1;
        const auto kernel = !pl.vec  ? (one ? norm_grad_kernel<TY, TX, 0, 1, POST, false> : norm_grad_kernel<TY, TX, 0, 2, POST, false>)
                            : pl.all ? (one ? norm_grad_kernel<TY, TX, W, 1, POST, true> : norm_grad_kernel<TY, TX, W, 2, POST, true>)
                            : one    ? norm_grad_kernel<TY, TX, W, 1, POST, false>
                                     : norm_grad_kernel<TY, TX, W, 2, POST, false>;
        const int rc = allow_smem(reinterpret_cast<const void*>(kernel), pl.smem);
        if (rc) return rc;
        cudaLaunchAttribute attr[2];
        return launch("norm gradient launch", kernel,
                      launch_config(static_cast<unsigned>(pl.ctas * p.parts), pl.r.T, pl.smem, p.parts, stream, attr), p);
    });
}

}  // namespace
