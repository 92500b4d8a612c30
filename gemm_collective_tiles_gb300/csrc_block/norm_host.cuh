// Argument checks and shapes that norm_join and its gradient share.
#pragma once
#include <initializer_list>

#include "block_host.cuh"
#include "block_norm.cuh"

namespace {

bool norm_ok(int k) { return k >= IRIS_NORM_NONE && k <= IRIS_NORM_LAYER; }

// rows of unit stride, or not there
bool unit(const iris_b200_mat& m) { return !m.data || m.col_stride == 1; }

// checks and parameters of a forward call; `vec`: every tensor so far has rows on 16
// bytes; `words`: those that are read have rows of unit stride
int set_norm(const iris_b200_norm_join_args* g, NormParams& p, bool& vec, bool& words) {
    int rc;
    std::memset(&p, 0, sizeof(p));
    if (!dims_ok(g->M, 0, g->D) || !dtype_ok(g->y_dtype) || !dtype_ok(g->x_dtype) || !norm_ok(g->post) || !norm_ok(g->pre) ||
        g->reserved || !(g->eps >= 0.0) || (g->x_dtype != g->y_dtype && g->x_dtype != IRIS_F32))
        return IRIS_EINVAL;
    const int64_t M = g->M, D = g->D;
    const int ye = dtype_size(g->y_dtype), xe = dtype_size(g->x_dtype);
    if ((rc = check_in(&g->y, M, D, ye)) || (g->x.data && (rc = check_in(&g->x, M, D, xe))) ||
        (g->h.data && (rc = check_out(&g->h, M, D, xe))) || (g->n.data && (rc = check_out(&g->n, M, D, ye))))
        return rc;
    p.group_rows = std::max<int64_t>(M, 1);
    p.gate_rows = 1;
    if (g->gate.data) {
        const int64_t G = g->gate_rows;  // 0 where there are no rows of y either
        if (G < (M > 0) || G > std::max<int64_t>(M, 1) || (G && M % G) || !dtype_ok(g->gate_dtype)) return IRIS_EINVAL;
        if ((rc = check_in(&g->gate, G, D, dtype_size(g->gate_dtype)))) return rc;
        if (M > 0) p.group_rows = M / G;
        p.gate_rows = G;
    }
    if (!g->post && (g->post_weight || g->post_bias)) return IRIS_EINVAL;
    if (!g->pre && (g->weight || g->bias)) return IRIS_EINVAL;
    if ((rc = check_vec(g->post_weight, g->post_weight_dtype)) || (rc = check_vec(g->post_bias, g->post_bias_dtype)) ||
        (rc = check_vec(g->weight, g->weight_dtype)) || (rc = check_vec(g->bias, g->bias_dtype)))
        return rc;
    if (!aligned(g->stats, 16)) return IRIS_EALIGN;
    p.y = mat_of(g->y);
    p.x = mat_of(g->x);
    p.gate = mat_of(g->gate);
    p.h = mat_of(g->h);
    p.n = mat_of(g->n);
    p.post_w = Vec{g->post_weight, g->post_weight_dtype};
    p.post_b = Vec{g->post_bias, g->post_bias_dtype};
    p.pre_w = Vec{g->weight, g->weight_dtype};
    p.pre_b = Vec{g->bias, g->bias_dtype};
    p.gate_type = g->gate_dtype;
    p.M = M;
    p.D = static_cast<int>(D);
    p.post = g->post;
    p.pre = g->pre;
    p.scale = static_cast<float>(g->scale);
    p.eps = static_cast<float>(g->eps);
    p.stats = reinterpret_cast<float4*>(g->stats);
    for (int& at : p.vec_at) at = -1;
    vec = D % 8 == 0 && rows16(g->y, M, D, ye) && rows16(g->x, M, D, xe) && rows16(g->h, M, D, xe) && rows16(g->n, M, D, ye) &&
          rows16(g->gate, g->gate_rows, D, dtype_size(g->gate_dtype)) && aligned16(g->post_weight) && aligned16(g->post_bias) &&
          aligned16(g->weight) && aligned16(g->bias);
    words = unit(g->y) && unit(g->x) && unit(g->gate);
    return IRIS_OK;
}

// dynamic shared memory of a kernel is allowed once per device
int allow_smem(const void* kernel, size_t bytes) {
    struct Entry {
        const void* kernel;
        uint64_t devices;
    };
    static Entry known[128];
    if (bytes <= 32768) return IRIS_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IRIS_ECUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    for (Entry& e : known) {
        if (e.kernel == kernel && (e.devices >> dev & 1)) return IRIS_OK;
        if (e.kernel && e.kernel != kernel) continue;
        const cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
        if (rc != cudaSuccess) return cuda_fail("cudaFuncSetAttribute (norms)", static_cast<int>(rc));
        e.kernel = kernel;
        e.devices |= uint64_t(1) << dev;
        return IRIS_OK;
    }
    return IRIS_ECUDA;
}

RowShape row_shape(int64_t D, int C, int most) {
    const int64_t chunks = cdiv(D, 8);
    while (C < 2 && cdiv(chunks, C) > most) C *= 2;
    return RowShape{static_cast<int>(std::min<int64_t>(most, round_up(cdiv(chunks, C), 32))), C};
}
constexpr size_t SM_SMEM = 222 * 1024;  // dynamic shared memory of an SM, beside the kernels' own

// How rows reach their threads: pieces of W elements (8 or 4) where all of them
// lie on 16 bytes; single elements, which rows of unit stride bring through shared
// memory too (`shared`), or which are read where they lie.
struct RowKind {
    int w;
    bool shared;
};
// What of `room` bytes the vectors (in fp32) and the rows ahead of `groups` rows'
// threads take: vectors first, then up to 4 rows each.  `types`: of the tensors
// whose rows come, -1: not there.
size_t row_memory(NormParams& p, RowShape r, int groups, bool bias, RowKind kind, std::initializer_list<int> types, size_t room) {
    const size_t piece = static_cast<size_t>(r.C) * r.T * 16;
    const void* all[5] = {p.post_w.data, p.post_b.data, p.pre_w.data, bias ? p.pre_b.data : nullptr, p.gate_rows == 1 ? p.gate.data : nullptr};
    int n = 0;
    for (int i = 0; i < 5; ++i) p.vec_at[i] = all[i] ? n++ : -1;
    p.vec_bytes = static_cast<unsigned>(n * 2 * piece);
    if (p.vec_bytes > room) {
        p.vec_bytes = 0;
        for (int& at : p.vec_at) at = -1;
    }
    size_t bytes = 0;
    auto add = [&](int type) {
        if (kind.w)
            bytes += piece * (kind.w == 4 || type == T_F32 ? 2 : 1);
        else
            bytes += 8 * r.C * r.T * dtype_size(type) + 32;
    };
    for (int type : types)
        if (type >= 0) add(type);
    if (p.gate.data && p.gate_rows > 1) add(p.gate_type);
    p.row_bytes = static_cast<unsigned>(bytes);
    p.depth = 0;
    if (kind.w || kind.shared) p.depth = static_cast<int>(std::min<size_t>(4, (room - p.vec_bytes) / (groups * bytes)));
    if (!kind.w && p.depth < 2) p.depth = 0;
    return p.vec_bytes + static_cast<size_t>(groups) * p.depth * p.row_bytes;
}
template <typename F>
int by_types(int y, int x, F f) {
    if (y == IRIS_F32) return f(std::integral_constant<int, T_F32>(), std::integral_constant<int, T_F32>());
    if (y == IRIS_F16)
        return x == IRIS_F32 ? f(std::integral_constant<int, T_F16>(), std::integral_constant<int, T_F32>())
                             : f(std::integral_constant<int, T_F16>(), std::integral_constant<int, T_F16>());
    return x == IRIS_F32 ? f(std::integral_constant<int, T_BF16>(), std::integral_constant<int, T_F32>())
                         : f(std::integral_constant<int, T_BF16>(), std::integral_constant<int, T_BF16>());
}

}  // namespace
