// Host side of matmul_act, act_grad, linear_act_grad and dropout, as declared in
// include/gemm_collective_tiles.h: argument checks, the choice of kernels, tensor
// maps and launches.
#include <cmath>

#include "block_elem.cuh"
#include "block_few.cuh"
#include "block_host.cuh"

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
int set_drop(Drop& d, double p, const int64_t* rng) {
    if (!(p >= 0.0 && p <= 1.0)) return IRIS_EINVAL;
    d.least = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    d.limit = static_cast<uint32_t>((static_cast<uint64_t>(d.least) << 16) - 1);
    d.scale = d.least == 65536u ? 0.f : static_cast<float>(65536.0 / (65536.0 - d.least));
    d.rng = reinterpret_cast<const long long*>(rng);
    if (d.least && !rng) return IRIS_EINVAL;
    return d.least && !aligned(rng, 8) ? IRIS_EALIGN : IRIS_OK;
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

}  // extern "C"
