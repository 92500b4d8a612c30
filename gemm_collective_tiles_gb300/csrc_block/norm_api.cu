// Host side of norm_join, as declared in include/gemm_collective_tiles.h.
#include "norm_host.cuh"

namespace {

template <int TY, int TX, int W>
int launch_norm_w(NormParams p, bool words, int sms, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    // Few rows: the more threads a row the shorter its way; many: work for a thread
    // between two reductions
    RowShape r = row_shape(p.D, p.M < 2 * sms ? 1 : 2, NORM_MAX_T);
    if (p.D > 16 * NORM_MAX_T) r = RowShape{static_cast<int>(round_up(cdiv(p.D, 16), 32)), 2};
    // 512 threads an SM, for registers enough (16384 x 4096, 32-bit residual: 129 us,
    // with 1024 threads 186; 1537 x 5003 f16: 38 and 59), unless a row needs more
    const int threads = r.T <= NORM_MAX_T ? NORM_MAX_T : NORM_CTA;
    const int groups = static_cast<int>(std::min<int64_t>(std::min(16, threads / r.T), cdiv(p.M, sms)));
    const int64_t ctas = std::min<int64_t>(cdiv(p.M, groups), sms);
    size_t smem = 0;
    if (ctas * groups < p.M)  // several rows for a group
        smem = row_memory(p, r, groups, true, RowKind{W, words}, {TY, p.x.data ? TX : -1}, SM_SMEM);
    auto of = [&](auto queued) {
        constexpr bool Q = decltype(queued)::value;
        return threads == NORM_CTA ? norm_kernel<TY, TX, W, 2, NORM_CTA, Q>
               : r.C == 1          ? norm_kernel<TY, TX, W, 1, NORM_MAX_T, Q>
                                   : norm_kernel<TY, TX, W, 2, NORM_MAX_T, Q>;
    };
    const auto kernel = W || p.depth > 0 ? of(std::true_type()) : of(std::integral_constant<bool, W != 0>());
    const int rc = allow_smem(reinterpret_cast<const void*>(kernel), smem);
    if (rc) return rc;
    cudaLaunchConfig_t lc = launch_config(static_cast<unsigned>(ctas), r.T, smem, 1, stream, attr);
    lc.blockDim = dim3(r.T, groups);
    return launch("norm launch", kernel, lc, p);
}
template <int TY, int TX>
int launch_norm(const NormParams& p, bool vec, bool words, int sms, cudaStream_t stream) {
    if (p.D > NORM_LONGEST) {
        cudaLaunchAttribute attr[2];
        return launch("norm launch", norm_long_kernel<TY, TX>, launch_config(static_cast<unsigned>(p.M), NORM_MAX_T, 0, 1, stream, attr), p);
    }
    return vec ? launch_norm_w<TY, TX, TX == T_F32 ? 4 : 8>(p, false, sms, stream) : launch_norm_w<TY, TX, 0>(p, words, sms, stream);
}

}  // namespace

extern "C" {

int iris_b200_norm_join(const iris_b200_norm_join_args* g, cudaStream_t stream) {
    NormParams p;
    bool vec, words;
    if (!g) return IRIS_EINVAL;
    const int rc = set_norm(g, p, vec, words);
    if (rc) return rc;
    if ((g->pre != 0) != (g->n.data != nullptr) && g->M > 0 && g->D > 0) return IRIS_EINVAL;
    if (g->M == 0 || g->D == 0) return IRIS_OK;
    int sms;
    if (sm_count(&sms)) return IRIS_ECUDA;
    return by_types(g->y_dtype, g->x_dtype,
                    [&](auto ty, auto tx) { return launch_norm<decltype(ty)::value, decltype(tx)::value>(p, vec, words, sms, stream); });
}

}  // extern "C"
