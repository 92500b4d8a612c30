// Host side of matmul_act, act_grad, dropout, norm_join and norm_join_grad, as
// declared in include/gemm_collective_tiles.h: argument checks, the choice of
// kernels, tensor maps and launches.
#include <cmath>
#include <initializer_list>

#include "../csrc_fp8/fp8_host.cuh"
#include "block_few.cuh"
#include "block_norm.cuh"

using namespace gct::block;

namespace {

// The kernels: a pair's 256 x 256 or 256 x 128 tile, a CTA's 128 x 128, and the
// ones for at most 16, 32 or 64 rows.
enum Variant { PAIR = 0, HALF = 1, CTA = 2, FEW16 = 3, FEW32 = 4, FEW64 = 5, VARIANTS = 6 };
bool is_pair(int v) { return v <= HALF; }
int few_rows(int v) { return v == FEW16 ? 16 : v == FEW32 ? 32 : 64; }

struct DeviceInfo {
    int sms;
    int clusters[VARIANTS][4];  // that run at once, by log2 of the cluster's CTAs
    bool done;
};
DeviceInfo g_dev[64];

template <int CG, int BN>
int setup_tiles(DeviceInfo& d, int v) {
    using G = Geo<CG, BN>;
    return setup_kernel(act_gemm_kernel<CG, BN>, d.clusters[v], CG == 2, CG == 2 ? 1 : 3, G::THREADS, G::BYTES, G::REGS_TOTAL, d.sms);
}
template <int NT>
int setup_few(DeviceInfo& d, int v) {
    return setup_kernel(act_few_kernel<NT>, d.clusters[v], 0, 3, FewGeo<NT>::THREADS, FewGeo<NT>::BYTES, 0, d.sms);
}
int device_info(DeviceInfo* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IRIS_ECUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceInfo& d = g_dev[dev];
    if (!d.done) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return IRIS_ECUDA;
        int rc;
        if ((rc = setup_tiles<2, 256>(d, PAIR)) || (rc = setup_tiles<2, 128>(d, HALF)) || (rc = setup_tiles<1, 128>(d, CTA)) ||
            (rc = setup_few<16>(d, FEW16)) || (rc = setup_few<32>(d, FEW32)) || (rc = setup_few<64>(d, FEW64)) ||
            (rc = find_encode()))
            return rc;
        d.done = true;
    }
    *out = d;
    return IRIS_OK;
}

bool act_ok(int a) { return a >= IRIS_ACT_NONE && a <= IRIS_ACT_SILU; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int set_drop(Drop& d, double p, const int64_t* rng) {
    if (!(p >= 0.0 && p <= 1.0)) return IRIS_EINVAL;
    d.least = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    d.limit = static_cast<uint32_t>((static_cast<uint64_t>(d.least) << 16) - 1);
    d.scale = d.least == 65536u ? 0.f : static_cast<float>(65536.0 / (65536.0 - d.least));
    d.rng = reinterpret_cast<const long long*>(rng);
    if (d.least && !rng) return IRIS_EINVAL;
    return d.least && !aligned(rng, 8) ? IRIS_EALIGN : IRIS_OK;
}
// an optional vector
int check_vec(const void* data, int type) {
    if (!data) return IRIS_OK;
    if (!dtype_ok(type)) return IRIS_EINVAL;
    return aligned(data, dtype_size(type)) ? IRIS_OK : IRIS_EALIGN;
}
Mat mat_of(const iris_b200_mat& m) { return Mat{m.data, m.row_stride, m.col_stride}; }
// rows of unit stride on 16 bytes
bool rows16(const iris_b200_mat& m, int64_t rows, int64_t cols, int elem) {
    return !m.data || (aligned16(m.data) && (m.col_stride == 1 || cols == 1) && (rows <= 1 || m.row_stride * elem % 16 == 0));
}

// ---------------------------------------------------------------- matmul_act
struct Plan {
    int variant, split, stages, m_blocks, n_blocks, group_m, grid;
    int tail_tiles, tail_parts;
};

// Estimated time in us of a variant: `slots` clusters run at once and take the
// tiles in turn; a tile costs its stages, what it adds at its end and, where a
// cluster shares it, the meeting of the parts; and no product is faster than its
// bytes at 5.6 TB/s.  Constants fitted to 70 shapes from 512 x 512 x 512 to 4096 x
// 4096 x 14336 in every variant and split (rms 6 to 12 %); the choice that they
// make is on average 2 % slower than the fastest one measured.   A tail costs a
// part's stages, an end, and the sums' way through global memory (5 to 11 us of 256
// columns, by the parts).
double estimate(int v, int slots, int64_t tiles, int64_t part, int split, int64_t stages, int tail_parts, double bytes) {
    static const double start[] = {5.4, 5.2, 4.7, 3.3, 3.7, 4.1}, stage[] = {0.292, 0.256, 0.259, 0.25, 0.253, 0.254},
                        end[] = {3.0, 1.4, 1.9, 1.8, 3.1, 4.3}, meet[] = {0, 0, 2.5, 0.9, 0, 0};
    const double tile = part * stage[v] + end[v] + (split > 1 ? meet[v] : 0.0);
    const double rounds = tail_parts ? static_cast<double>(tiles / slots) : static_cast<double>(cdiv(tiles, slots));
    const double tail = tail_parts ? stages * stage[v] / tail_parts + end[v] + (v == PAIR ? 3.0 * tail_parts - 1.0 : 3.5) : 0.0;
    return start[v] + std::max(rounds * tile + tail, bytes / 5.6e6);
}

constexpr size_t TAIL_SUMS = 32 * 4;  // bytes per column of an epilogue warp
size_t tail_flag_bytes(const Plan& pl) { return round_up(size_t(pl.tail_tiles) * (pl.tail_parts - 1) * 16 * 8, 256); }
size_t tail_bytes(const Plan& pl) {
    if (!pl.tail_tiles) return 0;
    const size_t columns = pl.variant == PAIR ? 128 : 64;
    return tail_flag_bytes(pl) + size_t(pl.tail_tiles) * (pl.tail_parts - 1) * 16 * columns * TAIL_SUMS;
}

int make_plan(Plan& pl, const iris_b200_config* cfg, const DeviceInfo& d, int64_t rows, int64_t cols, int64_t depth) {
    iris_b200_config z;
    std::memset(&z, 0, sizeof(z));
    if (!cfg) cfg = &z;
    const int tm = cfg->tile_m;
    if (tm != 0 && tm != 16 && tm != 32 && tm != 64 && tm != 128 && tm != 256) return IRIS_EINVAL;
    if (cfg->tile_n != 0 && cfg->tile_n != 128 && cfg->tile_n != 256) return IRIS_EINVAL;
    if (cfg->k_split != 0 && cfg->k_split != 1 && cfg->k_split != 2 && cfg->k_split != 4 && cfg->k_split != 8) return IRIS_EINVAL;
    if (cfg->group_m < 0 || cfg->debug_skip_flag < 0 || cfg->grid < 0 || cfg->grid > d.sms) return IRIS_EINVAL;
    const int64_t stages = cdiv(depth, DEPTH);
    const double bytes = 2.0 * (double(rows) * depth + double(depth) * cols + double(rows) * cols);
    double best = 0;
    pl.variant = -1;
    for (int v = PAIR; v < VARIANTS; ++v) {
        const int cg = is_pair(v) ? 2 : 1, bn = v == PAIR ? 256 : 128;
        if (tm && tm != (v >= FEW16 ? few_rows(v) : 128 * cg)) continue;
        if (cfg->tile_n && cfg->tile_n != bn) continue;
        if (v >= FEW16 && rows > few_rows(v)) continue;
        const int64_t mb = cdiv(rows, 128 * cg), nb = cdiv(cols, bn), tiles = mb * nb;
        if (tiles > 0x7FFFFFFF) continue;
        for (int lg = 0; lg < (cg == 2 ? 1 : 4); ++lg) {
            const int split = 1 << lg;
            const int64_t part = cdiv(stages, split);
            const int slots = std::min(d.clusters[v][cg == 2 ? 1 : lg], cfg->grid ? cfg->grid / (cg * split) : INT32_MAX);
            // every part has stages, unless the config asks for it (an empty one adds zeros)
            if (slots < 1 || (cfg->k_split ? split != cfg->k_split : split > stages)) continue;
            // Pairs: a last round with at most half of them at work is cut into 2, 3 or
            // 4 parts of at least 16 stages (4096 x 14336 x 4096, 3.4 rounds: 278 us whole, 254 in 2;
            // 1024 x 16384 x 1024, 16 tiles: 76, 48 in 2, 37 in 4)
            const int64_t last = tiles % slots;
            for (int parts = 0; parts <= 4; parts = parts ? parts + 1 : 2) {
                if (parts && (cg != 2 || last == 0 || parts * last > slots || stages < 16 * parts)) continue;
                const double t = estimate(v, slots, tiles, part, split, stages, parts, bytes);
                if (pl.variant >= 0 && t >= best) continue;
                best = t;
                pl.variant = v;
                pl.split = split;
                pl.m_blocks = static_cast<int>(mb);
                pl.n_blocks = static_cast<int>(nb);
                pl.tail_parts = parts;
                pl.tail_tiles = parts ? static_cast<int>(last) : 0;
                pl.grid = static_cast<int>(std::min<int64_t>(tiles + (parts ? (parts - 1) * last : 0), slots)) * cg * split;
                // one group holds all rows of tiles at most
                pl.group_m = std::min(cfg->group_m ? std::max(1, cfg->group_m / cg) : 32 / cg, pl.m_blocks);
            }
        }
    }
    pl.stages = static_cast<int>(stages);
    return pl.variant < 0 ? IRIS_EINVAL : IRIS_OK;
}

template <int CG, int BN>
int launch_tiles(const ActParams& p, int grid, cudaStream_t stream) {
    using G = Geo<CG, BN>;
    cudaLaunchAttribute attr[2];
    return launch("kernel launch (matmul_act)", act_gemm_kernel<CG, BN>,
                  launch_config(grid, G::THREADS, G::BYTES, CG * p.split, stream, attr), p);
}
template <int NT>
int launch_few(const ActParams& p, int grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    return launch("kernel launch (matmul_act)", act_few_kernel<NT>,
                  launch_config(grid, FewGeo<NT>::THREADS, FewGeo<NT>::BYTES, p.split, stream, attr), p);
}

int check_matmul_act(const iris_b200_matmul_act_args* g, Drop& drop) {
    int rc;
    if (!g || !dims_ok(g->M, g->N, g->K) || !dtype16(g->ab_dtype) || !dtype_ok(g->out_dtype) || !act_ok(g->act)) return IRIS_EINVAL;
    if ((rc = set_drop(drop, g->p, g->rng)) || (rc = check_vec(g->bias, g->bias_dtype))) return rc;
    const int e = dtype_size(g->out_dtype);
    if ((rc = check_in(&g->A, g->M, g->K, 2)) || (rc = check_in(&g->B, g->K, g->N, 2)) || (rc = check_out(&g->out, g->M, g->N, e)))
        return rc;
    if (g->residual.data && (rc = check_in(&g->residual, g->M, g->N, e))) return rc;
    return g->z.data ? check_out(&g->z, g->M, g->N, e) : IRIS_OK;
}

// `reserve`: bytes behind the workspace's header that are the caller's
int matmul_act(const iris_b200_matmul_act_args* g, const iris_b200_config* cfg, void* ws, size_t ws_bytes, cudaStream_t stream,
               size_t* need, size_t reserve = 0) {
    ActParams p;
    std::memset(&p, 0, sizeof(p));
    int rc = check_matmul_act(g, p.drop);
    if (rc) return rc;
    const int64_t M = g->M, N = g->N, K = g->K;
    if (M == 0 || N == 0) {
        if (need) *need = WS_HEADER + reserve;
        return IRIS_OK;
    }
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    Plan pl;
    if ((rc = make_plan(pl, cfg, d, M, N, std::max<int64_t>(K, 1)))) return rc;
    const bool few = pl.variant >= FEW16;
    const Operand none{nullptr, 0, 0, 0, false, false, 0};
    // few rows: the tokens are read K-major, of which there is little to copy
    Operand a = K == 0 ? none : resolve_operand(&g->A, M, K, 2, !few);
    Operand b = K == 0 ? none : resolve_operand(&g->B, K, N, 2, true);
    const size_t copies = WS_HEADER + reserve, total = copies + a.copy_bytes + b.copy_bytes + tail_bytes(pl);
    if (need) {
        *need = total;
        return IRIS_OK;
    }
    if (!ws || ws_bytes < total) return IRIS_ENOWS;
    if (!aligned16(ws)) return IRIS_EALIGN;

    const int e = dtype_size(g->out_dtype);
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.D = static_cast<int>(K);
    p.bias = g->bias;
    p.bias_type = g->bias_dtype;
    p.bias_near = g->bias && dtype16(g->bias_dtype) && aligned16(g->bias);
    p.type = g->out_dtype;
    p.act = g->act;
    p.out = g->out.data;
    p.out_rs = g->out.row_stride;
    p.out_cs = g->out.col_stride;
    p.residual = g->residual.data;
    p.res_rs = g->residual.row_stride;
    p.res_cs = g->residual.col_stride;
    p.z = g->z.data;
    p.z_rs = g->z.row_stride;
    p.z_cs = g->z.col_stride;
    auto by_tma = [&](const iris_b200_mat& m) { return m.data && tma_rows(m.data, m.row_stride, m.col_stride, M, N, e); };
    p.out_tma = by_tma(g->out);
    p.res_tma = by_tma(g->residual);
    p.z_tma = by_tma(g->z);
    if (K == 0) {
        const int64_t n = cdiv(M * cdiv(N, 4), 256);
        cudaLaunchAttribute attr[2];
        return launch("fill launch", act_fill_kernel<0>,
                      launch_config(static_cast<unsigned>(std::min<int64_t>(n, int64_t(d.sms) * 8)), 256, 0, 1, stream, attr), p);
    }
    char* w = static_cast<char*>(ws);
    if (a.copy && (rc = launch_repack<uint16_t>(&g->A, a, w + copies, d.sms, stream))) return rc;
    if (b.copy && (rc = launch_repack<uint16_t>(&g->B, b, w + copies + a.copy_bytes, d.sms, stream))) return rc;
    const int t = g->ab_dtype == IRIS_BF16;
    const CUtensorMapDataType t16 = t ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // MN-major: whole groups of 64 rows or columns come in one box a stage
    p.a_mn = !a.transposed ? 0 : a.cols % 64 == 0 ? 2 : 1;
    p.b_mn = b.transposed ? 0 : b.cols % 64 == 0 ? 2 : 1;
    // few rows: no more of a box than there are tokens; what lies in the others'
    // place reaches only sums that nobody reads
    const int a_rows = few ? static_cast<int>(M) : 128, b_rows = pl.variant == HALF ? 64 : 128;
    auto map_operand = [&](CUtensorMap* m, const Operand& o, int mn, int rows) {
        return mn == 2 ? make_map_groups(m, t16, o, rows / 64) : make_map_2d(m, t16, 2, o, 64, mn ? 64 : rows);
    };
    if ((rc = map_operand(&p.tmA, a, p.a_mn, a_rows)) || (rc = map_operand(&p.tmB, b, p.b_mn, b_rows))) return rc;
    // few rows: the weights are the MMA's first operand
    p.idesc = few ? idesc_of(t, t, p.b_mn != 0, 0, 128, few_rows(pl.variant))
                  : idesc_of(t, t, p.a_mn != 0, p.b_mn != 0, is_pair(pl.variant) ? 256 : 128, pl.variant == PAIR ? 256 : 128);
    auto store_map = [&](CUtensorMap* m, const iris_b200_mat& x) {
        return make_store_map(m, p.type, x.data, N, M, M == 1 ? packed_pitch(N, e) : x.row_stride);
    };
    if (!few && pl.split == 1 &&
        ((p.out_tma && (rc = store_map(&p.tmC, g->out))) || (p.res_tma && (rc = store_map(&p.tmR, g->residual))) ||
         (p.z_tma && (rc = store_map(&p.tmZ, g->z)))))
        return rc;
    p.stages_total = pl.stages;
    p.split = pl.split;
    p.m_blocks = pl.m_blocks;
    p.n_blocks = pl.n_blocks;
    p.group_m = pl.group_m;
    p.tail_tiles = pl.tail_tiles;
    p.tail_parts = pl.tail_parts;
    p.tail_first = pl.m_blocks * pl.n_blocks - pl.tail_tiles;
    p.n_units = p.tail_first + pl.tail_tiles * pl.tail_parts;
    char* const tail = w + copies + a.copy_bytes + b.copy_bytes;
    p.tail_flags = reinterpret_cast<unsigned long long*>(tail);
    p.tail_sums = reinterpret_cast<float*>(tail + (pl.tail_tiles ? tail_flag_bytes(pl) : 0));
    p.ws = reinterpret_cast<WsHeader*>(w);
    p.wait_ns = cfg && cfg->wait_ns ? cfg->wait_ns : DEFAULT_WAIT_NS;
    p.debug_skip = cfg ? static_cast<uint32_t>(cfg->debug_skip_flag) : 0u;
    switch (pl.variant) {
        case PAIR: return launch_tiles<2, 256>(p, pl.grid, stream);
        case HALF: return launch_tiles<2, 128>(p, pl.grid, stream);
        case CTA: return launch_tiles<1, 128>(p, pl.grid, stream);
        case FEW16: return launch_few<16>(p, pl.grid, stream);
        case FEW32: return launch_few<32>(p, pl.grid, stream);
        default: return launch_few<64>(p, pl.grid, stream);
    }
}

// ---------------------------------------------------------------- elements
int sm_count(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return IRIS_ECUDA;
    return IRIS_OK;
}

template <int T>
int launch_dropout(const DropParams& p, bool vec, unsigned grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    return launch("dropout launch", vec ? dropout_kernel<T, true> : dropout_kernel<T, false>,
                  launch_config(grid, 256, 0, 1, stream, attr), p);
}
template <int T>
int launch_act_grad(const ActGradParams& p, bool vec, unsigned grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    return launch("act_grad launch", vec ? act_grad_kernel<T, true> : act_grad_kernel<T, false>,
                  launch_config(grid, 256, 0, 1, stream, attr), p);
}

int act_grad(const iris_b200_act_grad_args* g, void* ws, size_t ws_bytes, cudaStream_t stream, size_t* need, size_t reserve = 0) {
    int rc;
    ActGradParams p;
    std::memset(&p, 0, sizeof(p));
    if (!g || !dims_ok(g->M, g->N, 0) || !dtype_ok(g->dtype) || !act_ok(g->act)) return IRIS_EINVAL;
    if ((rc = set_drop(p.drop, g->p, g->rng)) || (rc = check_vec(g->dbias, g->dbias_dtype))) return rc;
    const int64_t M = g->M, N = g->N;
    const int e = dtype_size(g->dtype);
    if ((rc = check_in(&g->dy, M, N, e)) || (g->act != IRIS_ACT_NONE && (rc = check_in(&g->z, M, N, e)))) return rc;
    if (g->dz.data && (!dtype_ok(g->dz_dtype) || (rc = check_out(&g->dz, M, N, dtype_size(g->dz_dtype))))) return rc ? rc : IRIS_EINVAL;
    p.segs = static_cast<unsigned>(cdiv(N, SEG));
    // Rows of a CTA: enough CTAs to fill the GPU several times, and few partial
    // sums beside the tensors.
    p.rows = static_cast<int>(std::min<int64_t>(256, std::max<int64_t>(16, round_up(cdiv(M * p.segs, 2048), 8))));
    const int64_t blocks = cdiv(M, p.rows);
    const size_t total = WS_HEADER + reserve + (g->dbias ? static_cast<size_t>(blocks) * N * 4 : 0);
    if (need) {
        *need = total;
        return IRIS_OK;
    }
    if (N == 0 || (!g->dz.data && !g->dbias)) return IRIS_OK;
    if (g->dbias) {
        if (!ws || ws_bytes < total) return IRIS_ENOWS;
        if (!aligned16(ws)) return IRIS_EALIGN;
        p.sums = reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEADER + reserve);
    }
    if (M > 0) {
        if (blocks * p.segs > 0x7FFFFFFF) return IRIS_EINVAL;
        p.dy = mat_of(g->dy);
        if (g->act != IRIS_ACT_NONE) p.z = mat_of(g->z);
        p.dz = mat_of(g->dz);
        p.M = M;
        p.N = static_cast<int>(N);
        p.type = g->dtype;
        p.dz_type = g->dz_dtype;
        p.act = g->act;
        const bool vec = N % 8 == 0 && rows16(g->dy, M, N, e) && (g->act == IRIS_ACT_NONE || rows16(g->z, M, N, e)) &&
                         (!g->dz.data || rows16(g->dz, M, N, dtype_size(g->dz_dtype)));
        const unsigned grid = static_cast<unsigned>(blocks * p.segs);
        rc = g->dtype == IRIS_F32   ? launch_act_grad<T_F32>(p, vec, grid, stream)
             : g->dtype == IRIS_F16 ? launch_act_grad<T_F16>(p, vec, grid, stream)
                                    : launch_act_grad<T_BF16>(p, vec, grid, stream);
        if (rc) return rc;
    }
    if (!g->dbias) return IRIS_OK;
    const ColumnSumParams c{p.sums, static_cast<int>(blocks), static_cast<int>(N), g->dbias, g->dbias_dtype};
    cudaLaunchAttribute attr[2];
    return launch("column sum launch", column_sum_kernel<0>,
                  launch_config(static_cast<unsigned>(cdiv(N, 32)), 256, 0, 1, stream, attr), c);
}

// ---------------------------------------------------------------- linear_act_grad
// act_grad, then the two products of its result, which lies in the workspace in
// rows of whole 16 bytes where it is anything but dy.
int linear_act_grad(const iris_b200_linear_act_grad_args* g, void* ws, size_t ws_bytes, cudaStream_t stream, size_t* need) {
    int rc;
    Drop drop;
    if (!g || !dims_ok(g->M, g->N, g->K) || !dtype16(g->dtype) || !act_ok(g->act) || g->reserved) return IRIS_EINVAL;
    if ((rc = set_drop(drop, g->p, g->rng))) return rc;
    const int64_t M = g->M, N = g->N, K = g->K;
    if ((rc = check_in(&g->dy, M, N, 2)) || (g->dx.data && ((rc = check_in(&g->weight, K, N, 2)) || (rc = check_out(&g->dx, M, K, 2)))) ||
        (g->dweight.data && ((rc = check_in(&g->x, M, K, 2)) || (rc = check_out(&g->dweight, K, N, 2)))))
        return rc;
    const bool products = g->dx.data || g->dweight.data, own = products && (g->act != IRIS_ACT_NONE || drop.least);
    iris_b200_mat dz = g->dy;
    size_t reserve = 0;
    iris_b200_act_grad_args a;
    std::memset(&a, 0, sizeof(a));
    if (own) {
        const int64_t pitch = packed_pitch(N, 2);
        reserve = round_up(static_cast<size_t>(M) * pitch * 2, 256);
        dz = iris_b200_mat{ws ? static_cast<char*>(ws) + WS_HEADER : reinterpret_cast<void*>(16), pitch, 1};
        a.dz = dz;
    }
    a.dy = g->dy;
    a.z = g->z;
    a.dbias = g->dbias;
    a.rng = g->rng;
    a.M = M;
    a.N = N;
    a.p = g->p;
    a.dtype = a.dz_dtype = g->dtype;
    a.dbias_dtype = g->dbias_dtype;
    a.act = g->act;
    iris_b200_matmul_act_args m[2];
    std::memset(m, 0, sizeof(m));
    auto transposed = [](const iris_b200_mat& x) { return iris_b200_mat{x.data, x.col_stride, x.row_stride}; };
    m[0].A = dz;  // dx = dz weight^T
    m[0].B = transposed(g->weight);
    m[0].out = g->dx;
    m[0].M = M;
    m[0].N = K;
    m[0].K = N;
    m[1].A = transposed(g->x);  // dweight = x^T dz
    m[1].B = dz;
    m[1].out = g->dweight;
    m[1].M = K;
    m[1].N = N;
    m[1].K = M;
    size_t total = WS_HEADER + reserve;
    for (int run = 0; run < 2; ++run) {  // sizes first: nothing is launched where one of the three would be refused
        size_t n = 0;
        size_t* const size = run ? nullptr : &n;
        if (run) {
            if (need) {
                *need = total;
                return IRIS_OK;
            }
            if (!ws || ws_bytes < total) return IRIS_ENOWS;
            if (!aligned16(ws)) return IRIS_EALIGN;
        }
        if (own || g->dbias) {
            if ((rc = act_grad(&a, ws, ws_bytes, stream, size, reserve))) return rc;
            total = std::max(total, n);
        }
        for (iris_b200_matmul_act_args& x : m) {
            if (!x.out.data) continue;
            x.ab_dtype = x.out_dtype = g->dtype;
            if ((rc = matmul_act(&x, nullptr, ws, ws_bytes, stream, size, reserve))) return rc;
            total = std::max(total, n);
        }
    }
    return IRIS_OK;
}

// ---------------------------------------------------------------- norms
bool norm_ok(int k) { return k >= IRIS_NORM_NONE && k <= IRIS_NORM_LAYER; }

// rows of unit stride, or not there
bool unit(const iris_b200_mat& m) { return !m.data || m.col_stride == 1; }

// checks and parameters of a forward call; `vec`: every tensor so far has rows on 16
// bytes; `shared`: those that are read have rows of unit stride
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
        if (g->gate_rows < 1 || g->gate_rows > std::max<int64_t>(M, 1) || M % g->gate_rows || !dtype_ok(g->gate_dtype)) return IRIS_EINVAL;
        if ((rc = check_in(&g->gate, g->gate_rows, D, dtype_size(g->gate_dtype)))) return rc;
        p.group_rows = std::max<int64_t>(M / g->gate_rows, 1);
        p.gate_rows = g->gate_rows;
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
        if (rc != cudaSuccess) return cuda_fail("cudaFuncSetAttribute (norm_join_grad)", static_cast<int>(rc));
        e.kernel = kernel;
        e.devices |= uint64_t(1) << dev;
        return IRIS_OK;
    }
    return IRIS_ECUDA;
}

// Threads T of a row at 8 C elements each.
struct RowShape {
    int T, C;
};
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
template <int TY, int TX, int W>
int launch_norm_w(NormParams p, bool words, int sms, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    // Few rows: the more threads a row the shorter its way; many: work for a thread
    // between two reductions
    RowShape r = row_shape(p.D, p.M < 2 * sms ? 1 : 2, NORM_MAX_T);
    if (p.D > 16 * NORM_MAX_T) r = RowShape{static_cast<int>(round_up(cdiv(p.D, 16), 32)), 2};
    // 512 threads an SM, for registers enough (16384 x 4096, 32-bit residual: 129 us,
    // with 1024 threads 186; 1537 x 5003 f16: 40 and 59), unless a row needs more
    const int threads = r.T <= NORM_MAX_T ? NORM_MAX_T : NORM_CTA;
    const int groups = static_cast<int>(std::min<int64_t>(std::min(16, threads / r.T), cdiv(p.M, sms)));
    const int64_t ctas = std::min<int64_t>(cdiv(p.M, groups), sms);
    size_t smem = 0;
    if (ctas * groups < p.M)  // several rows for a group
        smem = row_memory(p, r, groups, true, RowKind{W, words}, {TY, p.x.data ? TX : -1}, SM_SMEM);
    const auto kernel = threads == NORM_CTA ? norm_kernel<TY, TX, W, 2, NORM_CTA>
                        : r.C == 1          ? norm_kernel<TY, TX, W, 1, NORM_MAX_T>
                                            : norm_kernel<TY, TX, W, 2, NORM_MAX_T>;
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
template <typename F>
int by_types(int y, int x, F f) {
    if (y == IRIS_F32) return f(std::integral_constant<int, T_F32>(), std::integral_constant<int, T_F32>());
    if (y == IRIS_F16)
        return x == IRIS_F32 ? f(std::integral_constant<int, T_F16>(), std::integral_constant<int, T_F32>())
                             : f(std::integral_constant<int, T_F16>(), std::integral_constant<int, T_F16>());
    return x == IRIS_F32 ? f(std::integral_constant<int, T_BF16>(), std::integral_constant<int, T_F32>())
                         : f(std::integral_constant<int, T_BF16>(), std::integral_constant<int, T_BF16>());
}

struct GradPlan {
    RowShape r;
    bool in_registers;
    int64_t ctas;
    size_t smem, part, total;
};
template <int TY, int TX, int W>
int launch_norm_grad_w(const NormGradParams& p, const GradPlan& pl, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    const auto kernel = pl.r.C == 1 ? norm_grad_kernel<TY, TX, W, 1> : norm_grad_kernel<TY, TX, W, 2>;
    const int rc = allow_smem(reinterpret_cast<const void*>(kernel), pl.smem);
    return rc ? rc : launch("norm gradient launch", kernel, launch_config(static_cast<unsigned>(pl.ctas * p.parts), pl.r.T, pl.smem, p.parts, stream, attr), p);
}

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
    p.gate_sums = g->dgate.data && p.f.group_rows != 1;
    vec = vec && rows16(g->dh, M, D, xe) && rows16(g->dn, M, D, ye) && rows16(g->dy, M, D, ye) && rows16(g->dx, M, D, xe) &&
          rows16(g->dgate, G, D, ge);
    int sms;
    if ((rc = sm_count(&sms))) return rc;
    GradPlan pl;
    // A row to a CTA, or, where it is too long for one's registers, to a cluster; also
    // where no rows that start anywhere fit beside the sums (4000 x 8001 bf16: 411 us
    // read where they lie, 279 shared by two)
    pl.in_registers = D <= 8 * NORM_GRAD_LONGEST;
    p.parts = 1;
    while (pl.in_registers && p.parts * NORM_GRAD_LONGEST < D) p.parts *= 2;
    words = words && unit(g->dh) && unit(g->dn);
    int per_sm;
    for (;; p.parts *= 2) {
        // 16 elements a thread hide more of a reduction than 8 and leave two CTAs an SM
        // (16384 x 4096 bf16, rms: 158 us, with 8 199), but where a post-norm's values and
        // sums need registers too, where they come singly or beside 32-bit ones, 8 do
        // (16384 x 2048, both norms: 150 and 184; 16384 x 1003 f16: 119 and 205)
        pl.r = row_shape(cdiv(D, p.parts), vec && f.x_dtype != IRIS_F32 && !f.post && D >= 512 ? 2 : 1, NORM_MAX_T);
        // 512 threads' registers fill an SM; what shared memory the sums leave holds rows ahead
        per_sm = std::min(NORM_MAX_T / pl.r.T, 16);
        const size_t sums = pl.r.C == 1 ? 0 : static_cast<size_t>(p.slots + p.gate_sums) * 2 * pl.r.C * pl.r.T * 16;
        const size_t room = SM_SMEM / per_sm - 1024;
        pl.smem = sums;
        p.f.depth = 0;
        if (sums < room)
            pl.smem += row_memory(p.f, pl.r, 1, false, RowKind{!vec ? 0 : f.x_dtype == IRIS_F32 ? 4 : 8, words},
                                  {f.y_dtype, f.x.data ? f.x_dtype : -1, g->dh.data ? f.x_dtype : -1, g->dn.data ? f.y_dtype : -1}, room - sums);
        if (vec || !words || !pl.in_registers || p.f.depth || p.parts == 8) break;
    }
    if (pl.smem > SM_SMEM) return IRIS_EUNSUPPORTED;
    pl.ctas = std::min<int64_t>(M, int64_t(sms) * (pl.in_registers ? per_sm : 1) / p.parts);
    pl.part = round_up(static_cast<size_t>(pl.ctas) * p.slots * D * 4, 256);
    pl.total = WS_HEADER + pl.part + (p.gate_sums ? static_cast<size_t>(pl.ctas) * 2 * D * 4 : 0);
    if (need) {
        *need = pl.total;
        return IRIS_OK;
    }
    if (D == 0) return IRIS_OK;
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
        rc = by_types(f.y_dtype, f.x_dtype, [&](auto ty, auto tx) {
            constexpr int TY = decltype(ty)::value, TX = decltype(tx)::value;
            if (pl.in_registers)
                return vec ? launch_norm_grad_w<TY, TX, TX == T_F32 ? 4 : 8>(p, pl, stream) : launch_norm_grad_w<TY, TX, 0>(p, pl, stream);
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

int iris_b200_matmul_act_workspace_size(const iris_b200_matmul_act_args* args, const iris_b200_config* cfg, size_t* bytes) {
    return bytes ? matmul_act(args, cfg, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_matmul_act(const iris_b200_matmul_act_args* args, const iris_b200_config* cfg, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
    return matmul_act(args, cfg, workspace, workspace_bytes, stream, nullptr);
}
int iris_b200_act_grad_workspace_size(const iris_b200_act_grad_args* args, const iris_b200_config*, size_t* bytes) {
    return bytes ? act_grad(args, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_act_grad(const iris_b200_act_grad_args* args, const iris_b200_config*, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
    return act_grad(args, workspace, workspace_bytes, stream, nullptr);
}
int iris_b200_linear_act_grad_workspace_size(const iris_b200_linear_act_grad_args* args, const iris_b200_config*, size_t* bytes) {
    return bytes ? linear_act_grad(args, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_linear_act_grad(const iris_b200_linear_act_grad_args* args, const iris_b200_config*, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
    return linear_act_grad(args, workspace, workspace_bytes, stream, nullptr);
}

int iris_b200_dropout(const iris_b200_dropout_args* g, cudaStream_t stream) {
    int rc;
    DropParams p;
    std::memset(&p, 0, sizeof(p));
    if (!g || !dims_ok(g->M, g->N, 0) || !dtype_ok(g->dtype) || g->reserved) return IRIS_EINVAL;
    if ((rc = set_drop(p.drop, g->p, g->rng))) return rc;
    const int64_t M = g->M, N = g->N;
    const int e = dtype_size(g->dtype);
    if ((rc = check_in(&g->x, M, N, e)) || (rc = check_out(&g->out, M, N, e)) ||
        (g->residual.data && (rc = check_in(&g->residual, M, N, e))))
        return rc;
    if (M == 0 || N == 0) return IRIS_OK;
    const int64_t segs = cdiv(N, SEG);
    int sms;
    if ((rc = sm_count(&sms))) return rc;
    p.x = mat_of(g->x);
    p.residual = mat_of(g->residual);
    p.out = mat_of(g->out);
    p.M = M;
    p.N = static_cast<int>(N);
    p.type = g->dtype;
    p.segs = static_cast<unsigned>(segs);
    // a CTA takes 8 rows' pieces, or, of more than 64 CTAs an SM, every row_step-th 8
    const int64_t down = std::min<int64_t>(cdiv(M, 8), std::max<int64_t>(1, int64_t(sms) * 64 / segs));
    p.row_step = down * 8;
    const bool vec = N % 8 == 0 && rows16(g->x, M, N, e) && rows16(g->out, M, N, e) && rows16(g->residual, M, N, e);
    const unsigned grid = static_cast<unsigned>(down * segs);
    if (g->dtype == IRIS_F32) return launch_dropout<T_F32>(p, vec, grid, stream);
    if (g->dtype == IRIS_F16) return launch_dropout<T_F16>(p, vec, grid, stream);
    return launch_dropout<T_BF16>(p, vec, grid, stream);
}

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
int iris_b200_norm_join_grad_workspace_size(const iris_b200_norm_join_grad_args* args, const iris_b200_config*, size_t* bytes) {
    return bytes ? norm_grad(args, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_norm_join_grad(const iris_b200_norm_join_grad_args* args, const iris_b200_config*, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    return norm_grad(args, workspace, workspace_bytes, stream, nullptr);
}

}  // extern "C"
