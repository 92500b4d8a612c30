// Host side of norm_join_grad, as declared in include/gemm_collective_tiles.h, and
// its kernels without a post-norm.
#include "norm_grad.cuh"

namespace {

int norm_grad(const iris_b200_norm_join_grad_args* g, void* ws, size_t ws_bytes, cudaStream_t stream, size_t* need) {
    int rc;
    NormGradParams p;
    std::memset(&p, 0, sizeof(p));
    if (!g) return IRIS_EINVAL;
    const iris_b200_norm_join_args& f = g->f;
    bool vec, words;
    iris_b200_norm_join_args ff = f;
    ff.h.data = ff.n.data = nullptr;
    if ((rc = set_norm(&ff, p.f, vec, words))) return rc;
    const int64_t M = f.M, D = f.D, G = f.gate.data ? f.gate_rows : 0;
    const int ye = dtype_size(f.y_dtype), xe = dtype_size(f.x_dtype), ge = dtype_size(f.gate_dtype);
    if ((g->dn.data && !f.pre) || (g->dgate.data && !f.gate.data) || (M > 0 && D > 0 && !f.stats)) return IRIS_EINVAL;
    if (M > 0 && D > 0 && !g->dh.data && !g->dn.data) return IRIS_EINVAL;
    if ((g->dh.data && (rc = check_in(&g->dh, M, D, xe))) || (g->dn.data && (rc = check_in(&g->dn, M, D, ye))) ||
        (g->dy.data && (rc = check_out(&g->dy, M, D, ye))) || (g->dx.data && (rc = check_out(&g->dx, M, D, xe))) ||
        (g->dgate.data && (rc = check_out(&g->dgate, G, D, ge))))
        return rc;
    void* const vectors[4] = {g->dweight, g->dbias, g->dpost_weight, g->dpost_bias};
    const int types[4] = {f.weight_dtype, f.bias_dtype, f.post_weight_dtype, f.post_bias_dtype};
    const int kinds[4] = {f.pre, f.pre, f.post, f.post};
    NormFinishParams fin;
    std::memset(&fin, 0, sizeof(fin));
    for (int i = 0; i < 4; ++i) {
        p.slot[i] = -1;
        if (!vectors[i]) continue;
        if (!kinds[i]) return IRIS_EINVAL;
        if ((rc = check_vec(vectors[i], types[i]))) return rc;
        fin.out[p.slots] = vectors[i];
        fin.type[p.slots] = types[i];
        p.slot[i] = p.slots++;
    }
    // (no rows: a gate's gradient is a sum of nothing)
    p.gate_sums = g->dgate.data && G && (M == 0 || p.f.group_rows != 1);
    vec = vec && rows16(g->dh, M, D, xe) && rows16(g->dn, M, D, ye) && rows16(g->dy, M, D, ye) && rows16(g->dx, M, D, xe) &&
          rows16(g->dgate, G, D, ge);
    if (D == 0) {
        if (need) *need = WS_HEADER;
        return IRIS_OK;
    }
    int sms;
    if ((rc = sm_count(&sms))) return rc;
    NormGradPlan pl;
    // A row to a CTA, or, where it is too long for one's registers, to a cluster; also
    // where no rows that start anywhere fit beside the sums (4000 x 8001 bf16: 411 us
    // read where they lie, 279 shared by two)
    pl.in_registers = D <= 8 * NORM_GRAD_LONGEST;
    p.parts = 1;
    while (pl.in_registers && p.parts * NORM_GRAD_LONGEST < D) p.parts *= 2;
    words = words && unit(g->dh) && unit(g->dn);
    const bool held = f.post_weight || f.post_bias || f.weight || (f.gate.data && f.gate_rows == 1);
    // 16 elements a thread hide more of a reduction than 8 and leave two CTAs an SM
    // (16384 x 4096 bf16, rms: 128 us, with 8 154; layer norm and gate 165 and 184), where
    // their sums leave shared memory for the vectors and a row ahead (both norms and a gate
    // of one row, 16384 x 2048: 182 and 121 us) and rows do not come singly (16384 x 1003
    // f16: 205 and 119) or beside 32-bit ones (16384 x 4096 f32: 269 and 248)
    int per_sm, most = vec && f.x_dtype != IRIS_F32 && D >= 512 ? 2 : 1;
    for (;;) {
        pl.r = row_shape(cdiv(D, p.parts), most, NORM_MAX_T);
        // 512 threads' registers fill an SM; what shared memory the sums leave holds rows ahead
        per_sm = std::min(NORM_MAX_T / pl.r.T, 16);
        const size_t sums = pl.r.C == 1 ? 0 : static_cast<size_t>(p.slots + p.gate_sums) * 2 * pl.r.C * pl.r.T * 16;
        const size_t room = SM_SMEM / per_sm - 1024;  // five sums of 64 T bytes leave at least 2944 of it (T = 32)
        pl.smem = sums + row_memory(p.f, pl.r, 1, false, RowKind{!vec ? 0 : f.x_dtype == IRIS_F32 ? 4 : 8, words},
                                    {f.y_dtype, f.x.data ? f.x_dtype : -1, g->dh.data ? f.x_dtype : -1, g->dn.data ? f.y_dtype : -1}, room - sums);
        pl.kept = p.f.depth > 0 && (p.f.vec_bytes || !held);
        if (most == 2 && !pl.kept)
            most = 1;
        else if (vec || !words || !pl.in_registers || p.f.depth || p.parts == 8)
            break;
        else
            p.parts *= 2;
    }
    pl.vec = vec;
    pl.all = vec && f.x.data && g->dh.data && g->dn.data && pl.kept;
    pl.ctas = std::min<int64_t>(M, int64_t(sms) * (pl.in_registers ? per_sm : 1) / p.parts);
    pl.part = round_up(static_cast<size_t>(pl.ctas) * p.slots * D * 4, 256);
    pl.total = WS_HEADER + pl.part + (p.gate_sums ? static_cast<size_t>(pl.ctas) * 2 * D * 4 : 0);
    if (need) {
        *need = pl.total;
        return IRIS_OK;
    }
    if (p.slots || p.gate_sums) {
        if (!ws || ws_bytes < pl.total) return IRIS_ENOWS;
        if (!aligned16(ws)) return IRIS_EALIGN;
        p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEADER);
        p.gate_part = reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEADER + pl.part);
    }
    p.dh = mat_of(g->dh);
    p.dn = mat_of(g->dn);
    p.dy = mat_of(g->dy);
    p.dx = mat_of(g->dx);
    p.dgate = mat_of(g->dgate);
    p.ctas = pl.ctas;
    if (M > 0) {
        if (pl.in_registers)
            rc = f.post ? norm_grad_post(p, pl, f.y_dtype, f.x_dtype, stream)
                        : launch_norm_grad<false>(p, pl, f.y_dtype, f.x_dtype, stream);
        else
            rc = by_types(f.y_dtype, f.x_dtype, [&](auto ty, auto tx) {
                constexpr int TY = decltype(ty)::value, TX = decltype(tx)::value;
                cudaLaunchAttribute attr[2];
                return launch("norm gradient launch", norm_grad_long_kernel<TY, TX>,
                              launch_config(static_cast<unsigned>(pl.ctas), NORM_MAX_T, 0, 1, stream, attr), p);
            });
        if (rc) return rc;
    }
    if (!p.slots && !p.gate_sums) return IRIS_OK;
    fin.part = p.part;
    fin.gate_part = p.gate_part;
    fin.ctas = static_cast<int>(pl.ctas);
    fin.slots = p.slots;
    fin.D = static_cast<int>(D);
    fin.dgate = p.dgate;
    fin.gate_type = f.gate_dtype;
    fin.M = M;
    fin.group_rows = p.f.group_rows;
    fin.groups = p.gate_sums ? G : 0;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t lc = launch_config(static_cast<unsigned>(cdiv(D, 32)), 256, 0, 1, stream, attr);
    lc.gridDim.y = static_cast<unsigned>(std::min<int64_t>(fin.slots + fin.groups, 1024));
    return launch("norm sums launch", norm_finish_kernel<0>, lc, fin);
}

}  // namespace

extern "C" {

int iris_b200_norm_join_grad_workspace_size(const iris_b200_norm_join_grad_args* args, const iris_b200_config*, size_t* bytes) {
    return bytes ? norm_grad(args, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_norm_join_grad(const iris_b200_norm_join_grad_args* args, const iris_b200_config*, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    return norm_grad(args, workspace, workspace_bytes, stream, nullptr);
}

}  // extern "C"
