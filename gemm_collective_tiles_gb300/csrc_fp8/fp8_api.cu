// Host side of the block-scaled 8-bit float entry points declared in
// include/gemm_collective_tiles.h: argument checks, operand layouts, the
// choice of tile and split, tensor maps and launches.
#include "fp8_few.cuh"
#include "fp8_gemm.cuh"
#include "fp8_host.cuh"

using namespace gct;
using namespace gct::fp8;

namespace {

// The kernels: a pair's 256 x 256 tile, a CTA's 128 x 128, and the ones for at
// most 16 or 32 rows.
enum Variant { PAIR = 0, CTA = 1, FEW16 = 2, FEW32 = 3 };

// per device: SMs and how many clusters of a kernel run at once, by kind,
// variant and log2 of the cluster's CTAs (a pair, or the parts of a split)
struct DeviceInfo {
    int sms;
    int clusters[2][4][4];
    bool done;
};
DeviceInfo g_dev[64];

template <int KIND, int CG>
int setup_tiles(DeviceInfo& d) {
    using G = Geo<KIND, CG>;
    int* const clusters = d.clusters[KIND][CG == 2 ? PAIR : CTA];  // both forms hold the same registers and memory
    const int rc = setup_kernel(block_gemm_kernel<KIND, CG, false>, clusters, CG == 2, CG == 2 ? 1 : 3, G::THREADS, G::BYTES,
                                G::REGS_TOTAL, d.sms);
    return rc ? rc
              : setup_kernel(block_gemm_kernel<KIND, CG, true>, clusters, CG == 2, CG == 2 ? 1 : 3, G::THREADS, G::BYTES,
                             G::REGS_TOTAL, d.sms);
}
template <int NT>
int setup_few(DeviceInfo& d) {
    return setup_kernel(few_rows_kernel<NT>, d.clusters[KIND_MM][NT == 16 ? FEW16 : FEW32], 0, 3, FewGeo<NT>::THREADS,
                        FewGeo<NT>::BYTES, 0, d.sms);
}

int device_info(DeviceInfo* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IRIS_ECUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceInfo& d = g_dev[dev];
    if (!d.done) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return IRIS_ECUDA;
        int rc;
        if ((rc = setup_tiles<KIND_MM, 1>(d)) || (rc = setup_tiles<KIND_MM, 2>(d)) || (rc = setup_tiles<KIND_WG, 1>(d)) ||
            (rc = setup_tiles<KIND_WG, 2>(d)) || (rc = setup_few<16>(d)) || (rc = setup_few<32>(d)))
            return rc;
        if ((rc = find_encode())) return rc;
        d.done = true;
    }
    *out = d;
    return IRIS_OK;
}

// Tile, split and workspace of one product (rows x cols over depth).
struct Plan {
    Variant variant;
    int cg, split, part_stages, stages, m_blocks, n_blocks, group_m, grid;
    int tail_tiles;  // pairs: tiles of the last round that are cut in two
    size_t copy_a, copy_b, tail, total;  // workspace offsets
};

// Tail tiles: 2 CTAs x 8 promotion warps each hand over 32 x 128 fp32 sums.
constexpr size_t TAIL_SUMS = 32 * 128 * 4;
size_t tail_flag_bytes(int tiles) { return round_up(size_t(tiles) * 16 * 8, 256); }

// Estimated time in us of a variant: `slots` clusters run at once and take the
// tiles in turn; a tile costs `part` stages, its epilogue and, where its
// contraction is split, the meeting of the parts.  Constants measured on GB300
// (launch 4.5; e.g. 1 x 4096 x 1024: 12.3 us as 8 CTAs of 32 stages, 9.1 split
// over 8; 333 x 1000 x 1112: 8.0 us whole, 9.9 split over 2; 100 x 4096 x 4096:
// 12.7 us whole, 10.4 split over 4; weight gradients of 2000 tokens, 500 x 504:
// 16.2 us whole, 11.1 split over 4, and of 8192 tokens, 512 x 512: 57 us
// whole, 26 split over 4).  Outputs that no tensor store can reach cost a pair's
// tile 1.2 us per byte of an element (3000 x 512 x 4097 bf16: 22.9 us, with 4096
// columns 16.2, in three rounds), a CTA's half of that, a meeting 0.8.
double estimate(bool wg, Variant v, int slots, int64_t tiles, int64_t part, int split, bool direct, int out_elem, bool tail) {
    const double stage = wg ? (v == PAIR ? 0.47 : 0.35) : (v == PAIR ? 0.45 : v == CTA ? 0.32 : v == FEW16 ? 0.27 : 0.42);
    double tile = part * stage + (v == PAIR ? 2.0 : 1.0);
    if (split > 1)
        tile += v >= FEW16 ? 2.0 : (wg ? 3.3 : 2.7) + (direct ? 0.0 : 0.8);
    else if (!direct && v <= CTA)
        tile += (v == PAIR ? 1.2 : 0.6) * out_elem;
    if (tail) return 4.5 + tiles / slots * tile + part * stage / 2 + 8.0;
    return 4.5 + cdiv(tiles, slots) * tile;
}

int make_plan(Plan& pl, bool wg, const iris_b200_config* cfg, const DeviceInfo& d, const Operand& a, const Operand& b,
              bool direct, int out_elem, int64_t rows, int64_t cols, int64_t depth) {
    iris_b200_config z;
    std::memset(&z, 0, sizeof(z));
    if (!cfg) cfg = &z;
    if (cfg->tile_m != 0 && cfg->tile_m != 128 && cfg->tile_m != 256) return IRIS_EINVAL;
    if (cfg->k_split != 0 && cfg->k_split != 1 && cfg->k_split != 2 && cfg->k_split != 4 && cfg->k_split != 8) return IRIS_EINVAL;
    if (cfg->tile_m == 256 && (cfg->k_split > 1 || cfg->grid == 1)) return IRIS_EINVAL;
    if (cfg->group_m < 0 || cfg->debug_skip_flag < 0 || cfg->grid < 0 || cfg->grid > d.sms) return IRIS_EINVAL;
    if (cfg->grid && cfg->k_split > cfg->grid) return IRIS_EINVAL;
    const int64_t stages = cdiv(depth, wg ? 64 : 128);
    const int grid = cfg->grid ? cfg->grid : d.sms;
    double best = 0;
    pl.cg = 0;
    for (int i = PAIR; i <= FEW32; ++i) {
        const Variant v = static_cast<Variant>(i);
        const int cg = v == PAIR ? 2 : 1;
        if (cfg->tile_m && cfg->tile_m != 128 * cg) continue;
        if (v >= FEW16 && (wg || rows > (v == FEW16 ? 16 : 32))) continue;
        const int64_t mb = cdiv(rows, 128 * cg), nb = cdiv(cols, 128 * cg), tiles = mb * nb;
        if (tiles > 0x7FFFFFFF) continue;
        for (int lg = 0; lg < (cg == 2 ? 1 : 4); ++lg) {
            const int split = 1 << lg;
            const int64_t part = cdiv(stages, split);
            const int slots = std::min(d.clusters[wg][v][cg == 2 ? 1 : lg], grid / (cg * split));
            if (slots < 1) continue;
            // every part has stages (an empty one, where the config asks for it, adds zeros)
            if (cfg->k_split ? split != cfg->k_split : part * (split - 1) >= stages) continue;
            // A last round with at most half of the pairs at work: cut its
            // tiles in two, where half a tile's time outweighs handing over
            // the sums (weight gradient over 16384 tokens, 4096 x 4096: 3.4 rounds
            // in 401 us, whole in 448)
            const int64_t last = tiles % slots;
            const bool tail = v == PAIR && last > 0 && 2 * last <= slots && part >= 32;
            const double t = estimate(wg, v, slots, tiles, part, split, direct, out_elem, tail);
            if (pl.cg == 0 || t < best) {
                best = t;
                pl.cg = cg;
                pl.variant = v;
                pl.split = split;
                pl.part_stages = static_cast<int>(part);
                pl.m_blocks = static_cast<int>(mb);
                pl.n_blocks = static_cast<int>(nb);
                pl.tail_tiles = tail ? static_cast<int>(last) : 0;
                pl.grid = static_cast<int>(std::min<int64_t>(tiles + pl.tail_tiles, slots)) * cg * split;
            }
        }
    }
    if (pl.cg == 0) return IRIS_EINVAL;
    pl.stages = static_cast<int>(stages);
    // one group holds all rows of tiles at most: the same order, and its size times
    // the columns of tiles is no larger than their number
    pl.group_m = std::min(cfg->group_m ? std::max(1, cfg->group_m / pl.cg) : 16 / pl.cg, pl.m_blocks);
    pl.copy_a = WS_HEADER;
    pl.copy_b = pl.copy_a + a.copy_bytes;
    pl.tail = pl.copy_b + b.copy_bytes;
    pl.total = pl.tail + (pl.tail_tiles ? tail_flag_bytes(pl.tail_tiles) + size_t(pl.tail_tiles) * 16 * TAIL_SUMS : 0);
    return IRIS_OK;
}

template <int KIND, int CG>
int launch_tiles(const GemmParams& p, bool direct, int grid, cudaStream_t stream) {
    using G = Geo<KIND, CG>;
    cudaLaunchAttribute attr[2];
    return launch("kernel launch (8-bit product)", direct ? block_gemm_kernel<KIND, CG, true> : block_gemm_kernel<KIND, CG, false>,
                  launch_config(grid, G::THREADS, G::BYTES, CG * p.split, stream, attr), p);
}
template <int NT>
int launch_few(const GemmParams& p, int grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    return launch("kernel launch (8-bit product)", few_rows_kernel<NT>,
                  launch_config(grid, FewGeo<NT>::THREADS, FewGeo<NT>::BYTES, p.split, stream, attr), p);
}

// out (rows x cols) of one product: everything that both kinds share.
// `wg`: operand a is X (depth x rows codes), b is dY (depth x cols, 16-bit);
// else a is A (rows x depth codes), b is B (depth x cols codes).
int run_product(bool wg, const iris_b200_mat* ma, int a_type, const iris_b200_mat* sa, const iris_b200_mat* mb,
                int b_type /* fp8 type or 16-bit dtype */, const iris_b200_mat* sb, const void* bias, int bias_dtype,
                const iris_b200_mat* out, int out_dtype, int64_t rows, int64_t cols, int64_t depth,
                const iris_b200_config* cfg, void* ws, size_t ws_bytes, cudaStream_t stream, size_t* need) {
    int rc;
    if (rows == 0 || cols == 0) {
        if (need) *need = WS_HEADER;
        return IRIS_OK;
    }
    const int b_elem = wg ? 2 : 1;
    const Operand none{nullptr, 0, 0, 0, false, false, 0};
    Operand a = depth == 0 ? none : wg ? resolve_operand(ma, depth, rows, 1, false) : resolve_operand(ma, rows, depth, 1, false);
    Operand b = depth == 0 ? none : resolve_operand(mb, depth, cols, b_elem, !wg);
    const bool direct = tma_rows(out->data, out->row_stride, out->col_stride, rows, cols, dtype_size(out_dtype));
    DeviceInfo d;
    if ((rc = device_info(&d))) return rc;
    Plan pl;
    if ((rc = make_plan(pl, wg, cfg, d, a, b, direct, dtype_size(out_dtype), rows, cols, std::max<int64_t>(depth, 1)))) return rc;
    if (need) {
        *need = pl.total;
        return IRIS_OK;
    }
    if (!ws || ws_bytes < pl.total) return IRIS_ENOWS;
    if (!aligned16(ws)) return IRIS_EALIGN;

    GemmParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = static_cast<int>(rows);
    p.N = static_cast<int>(cols);
    p.D = static_cast<int>(depth);
    p.bias = bias;
    p.bias_type = bias_dtype;
    p.out = out->data;
    p.out_type = out_dtype;
    p.out_rs = out->row_stride;
    p.out_cs = out->col_stride;
    if (depth == 0) {
        const int64_t n = cdiv(rows * cols, 256);
        cudaLaunchAttribute attr[2];
        return launch("fill launch", fill_kernel,
                      launch_config(static_cast<unsigned>(std::min<int64_t>(n, int64_t(d.sms) * 8)), 256, 0, 1, stream, attr), p);
    }
    char* w = static_cast<char*>(ws);
    if (a.copy && (rc = launch_repack<uint8_t>(ma, a, w + pl.copy_a, d.sms, stream))) return rc;
    if (b.copy) {
        rc = wg ? launch_repack<uint16_t>(mb, b, w + pl.copy_b, d.sms, stream)
                : launch_repack<uint8_t>(mb, b, w + pl.copy_b, d.sms, stream);
        if (rc) return rc;
    }
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (wg) {
        const CUtensorMapDataType t16 = b_type == IRIS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if ((rc = make_map_2d(&p.tmA, u8, 1, a, 128, 64))) return rc;
        // one box of all of a CTA's columns where no 64-column group runs past
        // the end of a row, else a box per group
        p.b_chunked = cols % 64 == 0;
        if ((rc = p.b_chunked ? make_map_groups(&p.tmB, t16, b, 2)
                              : make_map_2d(&p.tmB, t16, 2, b, 64, 64)))
            return rc;
        const int t = b_type == IRIS_BF16;
        p.idesc = idesc_of(t, t, 1, 1, 128 * pl.cg, 128 * pl.cg);
        p.x_bf16 = t;
        p.codes_e5m2 = a_type == IRIS_E5M2;
    } else {
        p.b_mn = !b.transposed;
        const bool few = pl.variant >= FEW16;
        p.a_box = pl.variant == FEW16 ? 16 : pl.variant == FEW32 ? 32 : 128;
        if ((rc = make_map_2d(&p.tmA, u8, 1, a, 128, p.a_box))) return rc;
        if ((rc = make_map_2d(&p.tmB, u8, 1, b, 128, 128))) return rc;
        // few rows: the weights are the MMA's first operand
        p.idesc = few ? idesc_of(b_type, a_type, p.b_mn, 0, 128, p.a_box)
                      : idesc_of(a_type, b_type, 0, p.b_mn, 128 * pl.cg, 128 * pl.cg);
        p.sb = static_cast<const float*>(sb->data);
        p.sb_rs = sb->row_stride;
        p.sb_cs = sb->col_stride;
    }
    p.sa = static_cast<const float*>(sa->data);
    p.sa_rs = sa->row_stride;
    p.sa_cs = sa->col_stride;
    p.stages_total = pl.stages;
    p.part_stages = pl.part_stages;
    p.split = pl.split;
    p.m_blocks = pl.m_blocks;
    p.n_blocks = pl.n_blocks;
    p.group_m = pl.group_m;
    p.tail_tiles = pl.tail_tiles;
    p.tail_first = pl.m_blocks * pl.n_blocks - pl.tail_tiles;
    p.n_units = p.tail_first + 2 * pl.tail_tiles;
    p.tail_flag = reinterpret_cast<unsigned long long*>(w + pl.tail);
    p.tail_sums = reinterpret_cast<unsigned long long*>(w + pl.tail + tail_flag_bytes(pl.tail_tiles));
    p.ws = reinterpret_cast<WsHeader*>(w);
    p.wait_ns = cfg && cfg->wait_ns ? cfg->wait_ns : DEFAULT_WAIT_NS;
    p.debug_skip = cfg ? static_cast<uint32_t>(cfg->debug_skip_flag) : 0u;
    if (direct && pl.variant <= CTA && (rc = make_store_map(&p.tmC, out_dtype, out->data, cols, rows,
                                       rows == 1 ? packed_pitch(cols, dtype_size(out_dtype)) : out->row_stride)))
        return rc;
    if (wg) return pl.variant == PAIR ? launch_tiles<KIND_WG, 2>(p, direct, pl.grid, stream) : launch_tiles<KIND_WG, 1>(p, direct, pl.grid, stream);
    switch (pl.variant) {
        case PAIR: return launch_tiles<KIND_MM, 2>(p, direct, pl.grid, stream);
        case CTA: return launch_tiles<KIND_MM, 1>(p, direct, pl.grid, stream);
        case FEW16: return launch_few<16>(p, pl.grid, stream);
        default: return launch_few<32>(p, pl.grid, stream);
    }
}

int check_matmul(const iris_b200_matmul_fp8_args* g) {
    int rc;
    if (!g || !dims_ok(g->M, g->N, g->K) || !dtype_ok(g->out_dtype) || !fp8_ok(g->a_type) || !fp8_ok(g->b_type)) return IRIS_EINVAL;
    if (g->bias && !dtype_ok(g->bias_dtype)) return IRIS_EINVAL;
    const int64_t kb = cdiv(g->K, 128);
    if ((rc = check_in(&g->A, g->M, g->K, 1)) || (rc = check_in(&g->B, g->K, g->N, 1)) ||
        (rc = check_in(&g->a_scales, g->M, kb, 4)) || (rc = check_in(&g->b_scales, kb, cdiv(g->N, 128), 4)))
        return rc;
    if (g->bias && reinterpret_cast<uintptr_t>(g->bias) % dtype_size(g->bias_dtype)) return IRIS_EALIGN;
    return check_out(&g->out, g->M, g->N, dtype_size(g->out_dtype));
}
int check_wgrad(const iris_b200_weight_grad_fp8_args* g) {
    int rc;
    if (!g || !dims_ok(g->M, g->N, g->K) || !dtype16(g->dy_dtype) || !dtype_ok(g->out_dtype) || !fp8_ok(g->x_type) || g->reserved)
        return IRIS_EINVAL;
    if ((rc = check_in(&g->X, g->M, g->K, 1)) || (rc = check_in(&g->dY, g->M, g->N, 2)) ||
        (rc = check_in(&g->x_scales, g->M, cdiv(g->K, 128), 4)))
        return rc;
    return check_out(&g->out, g->K, g->N, dtype_size(g->out_dtype));
}
int product(const iris_b200_matmul_fp8_args* g, const iris_b200_config* cfg, void* ws, size_t ws_bytes, cudaStream_t stream,
            size_t* need) {
    const int rc = check_matmul(g);
    if (rc) return rc;
    return run_product(false, &g->A, g->a_type, &g->a_scales, &g->B, g->b_type, &g->b_scales, g->bias, g->bias_dtype, &g->out,
                       g->out_dtype, g->M, g->N, g->K, cfg, ws, ws_bytes, stream, need);
}
int product(const iris_b200_weight_grad_fp8_args* g, const iris_b200_config* cfg, void* ws, size_t ws_bytes,
            cudaStream_t stream, size_t* need) {
    const int rc = check_wgrad(g);
    if (rc) return rc;
    return run_product(true, &g->X, g->x_type, &g->x_scales, &g->dY, g->dy_dtype, nullptr, nullptr, IRIS_F32, &g->out,
                       g->out_dtype, g->K, g->N, g->M, cfg, ws, ws_bytes, stream, need);
}

template <int T>
int launch_quant(const QuantParams& q, bool vec, bool shift, bool tile, unsigned grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    return launch("quantize launch",
                  vec && shift ? (tile ? quantize_vec_kernel<T, true, true> : quantize_vec_kernel<T, false, true>)
                  : vec        ? (tile ? quantize_vec_kernel<T, true, false> : quantize_vec_kernel<T, false, false>)
                               : (tile ? quantize_any_kernel<T, true> : quantize_any_kernel<T, false>),
                  launch_config(grid, Q_THREADS, 0, 1, stream, attr), q);
}

}  // namespace

extern "C" {

int iris_b200_quantize_fp8(const iris_b200_quantize_fp8_args* g, cudaStream_t stream) {
    int rc;
    if (!g || !dims_ok(g->M, 0, g->K) || !dtype_ok(g->x_dtype) || !fp8_ok(g->type) || (g->block_rows != 1 && g->block_rows != 128))
        return IRIS_EINVAL;
    const iris_b200_mat *x = &g->x, *codes = &g->codes, *scales = &g->scales;
    const int64_t M = g->M, K = g->K, kb = cdiv(K, 128), sr = g->block_rows == 1 ? M : cdiv(M, 128);
    if ((rc = check_in(x, M, K, dtype_size(g->x_dtype))) || (rc = check_out(codes, M, K, 1)) ||
        (rc = check_out(scales, sr, kb, 4)))
        return rc;
    if (M == 0 || K == 0) return IRIS_OK;
    const bool tile = g->block_rows == 128;
    const int64_t blocks = kb * cdiv(M, tile ? Q_TILE : Q_ROWS);
    if (blocks > 0x7FFFFFFF) return IRIS_EINVAL;
    QuantParams q;
    q.x = x->data;
    q.codes = static_cast<uint8_t*>(codes->data);
    q.scales = static_cast<float*>(scales->data);
    q.x_rs = x->row_stride;
    q.x_cs = x->col_stride;
    q.c_rs = codes->row_stride;
    q.c_cs = codes->col_stride;
    q.s_rs = scales->row_stride;
    q.s_cs = scales->col_stride;
    q.M = M;
    q.K = K;
    q.kblocks = static_cast<unsigned>(kb);
    q.e5m2 = g->type == IRIS_E5M2;
    q.pow2 = g->pow2 != 0;
    q.fmax = q.e5m2 ? 57344.f : 448.f;
    q.rfmax = 1.f / q.fmax;
    // f16 input: with scales of at least 2^-15 (e5m2: 2^-8) the codes' finest
    // step is f16's own, 2^-24, so scaled codes are f16 values again and
    // nothing that f16 can hold is lost to the bound
    q.pmin = g->x_dtype == IRIS_F16 ? (q.e5m2 ? -8 : -15) : -100;
    const int e = dtype_size(g->x_dtype);
    // 16-byte reads and writes where rows are of unit stride and code rows start
    // on 16 bytes.  Rows of x that do not are shifted into place: 16384 x 4096
    // bf16 one element off 37 us, against 33 aligned and 90 element by element.
    const bool vec = (x->col_stride == 1 || K == 1) && (codes->col_stride == 1 || K == 1) && aligned16(codes->data) &&
                     (M == 1 || codes->row_stride % 16 == 0);
    const bool shift = !aligned16(x->data) || (M > 1 && x->row_stride * e % 16 != 0);
    const unsigned grid = static_cast<unsigned>(blocks);
    if (g->x_dtype == IRIS_F32) return launch_quant<T_F32>(q, vec, shift, tile, grid, stream);
    if (g->x_dtype == IRIS_F16) return launch_quant<T_F16>(q, vec, shift, tile, grid, stream);
    return launch_quant<T_BF16>(q, vec, shift, tile, grid, stream);
}

int iris_b200_matmul_fp8_workspace_size(const iris_b200_matmul_fp8_args* args, const iris_b200_config* cfg, size_t* bytes) {
    return bytes ? product(args, cfg, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_matmul_fp8(const iris_b200_matmul_fp8_args* args, const iris_b200_config* cfg, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
    return product(args, cfg, workspace, workspace_bytes, stream, nullptr);
}
int iris_b200_weight_grad_fp8_workspace_size(const iris_b200_weight_grad_fp8_args* args, const iris_b200_config* cfg,
                                             size_t* bytes) {
    return bytes ? product(args, cfg, nullptr, 0, nullptr, bytes) : IRIS_EINVAL;
}
int iris_b200_weight_grad_fp8(const iris_b200_weight_grad_fp8_args* args, const iris_b200_config* cfg, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
    return product(args, cfg, workspace, workspace_bytes, stream, nullptr);
}

int iris_b200_capture_id(cudaStream_t stream, unsigned long long* id) {
    if (!id) return IRIS_EINVAL;
    cudaStreamCaptureStatus status;
    if (cudaStreamGetCaptureInfo(stream, &status, id) != cudaSuccess) {
        cudaGetLastError();  // the legacy stream while another captures: not an error of a later call
        return IRIS_ECUDA;
    }
    if (status != cudaStreamCaptureStatusActive) *id = 0;
    return IRIS_OK;
}

}  // extern "C"
