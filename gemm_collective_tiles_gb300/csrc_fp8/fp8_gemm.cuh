// Persistent tensor-core kernel of the block-scaled 8-bit products.
//
//   KIND_MM  out[m][n] = sum_b sa[m][b] * sb[b][n / 128] * P_b[m][n] + bias[n],
//            P_b = the product of the 8-bit codes over the 128-deep K block b.
//   KIND_WG  out[k][n] = sum_m (codes[m][k] * sx[m][k / 128]) * dY[m][n]: the
//            weight gradient from an input kept as 8-bit codes and scales.
//
// Both are one loop over the contraction in chunks whose fp32 product the
// tensor cores leave in tensor memory; eight promotion warps add each chunk,
// times its scale, into fp32 registers.  In KIND_MM a chunk is one K block of
// 128, because its two scales hold for that block alone.  In KIND_WG the scale
// varies along the contraction, so eight more warps turn codes into scaled
// 16-bit operands on their way from shared memory to the MMA (exact for
// power-of-two scales: a code has at most 4 significant bits), and a chunk is
// WG_CHUNK stages long, which bounds the length of the sums that the tensor
// cores keep by themselves.  f16 operands of a chunk whose values would leave
// f16's range are held times a power of two (run_factors).
//
// CTA layout, one CTA per SM:
//   warp 0       TMA producer (lane 0); KIND_WG: of the codes
//   warp 1       MMA issuer; owns tensor memory
//   warp 2       KIND_WG: TMA producer of dY (lane 0)
//   warp 3       KIND_MM, CG = 1: second MMA issuer; KIND_WG, f16: the chunks'
//                powers of two
//   warps 4-11   promotion and epilogue: quadrant warp % 4 of the accumulator's
//                rows, column half (warp - 4) / 4
//   warps 12-19  KIND_WG: converters
// CG = 2: a cluster of two CTAs computes a 256 x 256 tile with
// tcgen05.mma.cta_group::2, each staging its 128 rows of A and 128 columns of
// B; the even CTA issues the MMAs.  CG = 1: 128 x 128 tiles, for fewer rows.
//
// CG = 1 can split the contraction: a cluster of 2, 4 or 8 CTAs takes a tile,
// each a part of its stages; the fp32 sums meet in shared memory, where each
// CTA adds a slice of every warp's rows over all parts in part order, so
// results do not depend on timing and nothing goes through global memory.
//
// Tiles are dealt out in a fixed order.  Every wait is bounded: one that gives
// up records where in the workspace header, stops the launch, and the roles
// drain and leave.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_ptx.cuh"
#include "fp8_quant.cuh"
#include "fp8_wait.cuh"

namespace gct {
namespace fp8 {

enum : int { KIND_MM = 0, KIND_WG = 1 };
constexpr int BM = 128;         // rows per CTA (tensor-memory lanes)
constexpr int WG_CHUNK = 8;     // KIND_WG: 64-deep stages per chunk
constexpr int MAX_SPLIT = 8;    // CTAs of a cluster that share a tile

struct GemmParams {
    CUtensorMap tmA;  // MM: codes {k, row}, box {128, a_box}; WG: codes {k, m}, box {128, 64}
    CUtensorMap tmB;  // MM: codes {k, n} or {n, k}, box {128, 128}; WG: dY {n, m}, box {64, 64}
    CUtensorMap tmC;  // out {n, row}, box {128 bytes, 32}
    int M, N;         // output rows and columns
    int D;            // contraction length
    int stages_total, part_stages, split;  // contraction in stages; stages per part; parts
    int m_blocks, n_blocks, group_m;
    int n_units;      // work units: tiles, and two halves of each tail tile (pairs)
    int tail_first, tail_tiles;
    int b_mn;         // MM: B has its columns contiguous
    int b_chunked;    // WG: tmB is {64, m, n / 64}, one box per stage
    int a_box;        // MM: rows of A that a stage loads
    uint32_t idesc;
    const float* sa;  // MM: scales of A (row, K block); WG: scales of X (m, K block)
    long long sa_rs, sa_cs;
    const float* sb;  // MM: scales of B (K block, column block)
    long long sb_rs, sb_cs;
    int codes_e5m2, x_bf16;  // WG: code type, 16-bit type
    const void* bias;
    int bias_type;
    void* out;
    int out_type;
    long long out_rs, out_cs;
    WsHeader* ws;
    unsigned long long* tail_flag;  // per (tail tile, CTA, promotion warp): a first half's sums are in tail_sums
    unsigned long long* tail_sums;  // 32 x 128 fp32 each, in pairs of columns, a lane per row
    unsigned long long wait_ns;
    uint32_t debug_skip;          // test hook: k > 0: tile k - 1 never reports its accumulator
};

template <int KIND, int CG>
struct Geo {
    static constexpr int BN = CG == 2 ? 256 : 128;     // tile columns (of the pair)
    static constexpr int COLS = BN / 2;                // accumulator columns of a promotion warp
    static constexpr int DEPTH = KIND == KIND_MM ? 128 : 64;  // contraction per stage
    static constexpr int UMMA_STEPS = 4;               // 128 / 32 or 64 / 16
    static constexpr uint32_t A_BYTES = BM * 128;      // rows x 128 bytes of contraction
    static constexpr uint32_t B_BYTES = (BN / CG) * 128;
    static constexpr uint32_t RAW_BYTES = KIND == KIND_WG ? 64 * 128 : 0;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    // a stage holds one A and one B box; KIND_WG: the converted A and B, and
    // the codes have a ring of their own (RAWS slots)
    static constexpr int STAGES = KIND == KIND_WG ? 4 : CG == 2 ? 5 : 6;
    static constexpr int RAWS = KIND == KIND_MM ? 0 : 4;
    static constexpr int FACTORS = KIND == KIND_MM ? 0 : 4;  // chunks whose powers of two are known ahead
    static constexpr int ISSUERS = KIND == KIND_MM && CG == 1 ? 2 : 1;  // warps that issue MMAs
    static constexpr int THREADS = KIND == KIND_MM ? 384 : 640;
    static constexpr int BOXES = KIND == KIND_MM && CG == 1 ? 1 : 2;  // staging per promotion warp, 32 x 128 bytes each
    static constexpr uint32_t OUT_BYTES = BOXES * 32 * 128;
    static constexpr int TMEM_COLS = 512;
    static constexpr int ACCS = TMEM_COLS / BN;        // accumulators under way
    // Two warps that take turns at a ring (issuers, converter groups) each own
    // every other slot: a wait by parity is only valid for one who sees every
    // phase of the barrier, and with an odd ring each would see every other.
    static_assert(ISSUERS == 1 || (STAGES % 2 == 0 && ACCS % 2 == 0), "issuers by parity of the slot");
    static_assert(KIND == KIND_MM || (STAGES % 2 == 0 && RAWS % 2 == 0), "converter groups by parity of the slot");
    static constexpr int NUM_BARS = 3 * STAGES + 2 * RAWS + 2 * FACTORS + 2 * ACCS + 2 * 8 + 2;
    static constexpr uint32_t TILES_BYTES = STAGES * STAGE_BYTES + RAWS * RAW_BYTES;
    static constexpr uint32_t BYTES = 1024 + TILES_BYTES + 8 * OUT_BYTES + NUM_BARS * 8 + 16 + FACTORS * 8 + 16;
    // registers: the launch's total (168 or 96 a thread) is shared out anew
    static constexpr int REGS_CTL = KIND == KIND_MM ? 40 : 48;
    static constexpr int REGS_PROMOTE = KIND == KIND_MM ? 232 : 152;
    static constexpr int REGS_CONVERT = KIND == KIND_MM ? 0 : 64;
    static constexpr int REGS_TOTAL = 128 * REGS_CTL + 256 * (REGS_PROMOTE + REGS_CONVERT);
};
static_assert(Geo<KIND_MM, 2>::REGS_TOTAL <= 384 * 168 && Geo<KIND_WG, 2>::REGS_TOTAL <= 640 * 96, "register split");

template <int KIND, int CG>
struct Smem {
    using G = Geo<KIND, CG>;
    uint8_t* base;  // tiles, codes, staging
    // shared-memory addresses.  Barriers per stage: full (KIND_MM: A and B have
    // landed; KIND_WG: A is converted), b_full (KIND_WG: B has landed), done
    // (its MMAs have run: the stage may be filled again); per slot of codes:
    // raw_full, raw_empty; per slot of factors: fac_full, fac_empty; per
    // accumulator: acc_full, acc_empty; per promotion warp: parts_in (every part's sums lie in shared memory), parts_out (every
    // part has read this CTA's)
    uint32_t tiles, raw_tiles, full, done, raw_full, raw_empty, fac_full, fac_empty, b_full, acc_full, acc_empty, parts_in, parts_out, final_bar;
    uint32_t *tmem_slot, *epoch_slot;
    float2* factors;  // per slot: what a chunk's scales are multiplied by, and what its sums are
    __device__ void carve(uint8_t* p) {
        base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
        tiles = smem_u32(base);
        raw_tiles = tiles + G::STAGES * G::STAGE_BYTES;
        full = tiles + G::TILES_BYTES + 8 * G::OUT_BYTES;
        done = full + 8 * G::STAGES;
        b_full = done + 8 * G::STAGES;
        raw_full = b_full + 8 * G::STAGES;
        raw_empty = raw_full + 8 * G::RAWS;
        fac_full = raw_empty + 8 * G::RAWS;
        fac_empty = fac_full + 8 * G::FACTORS;
        acc_full = fac_empty + 8 * G::FACTORS;
        acc_empty = acc_full + 8 * G::ACCS;
        parts_in = acc_empty + 8 * G::ACCS;
        parts_out = parts_in + 64;
        final_bar = parts_out + 64;
        tmem_slot = reinterpret_cast<uint32_t*>(base + (final_bar + 16 - tiles));
        epoch_slot = tmem_slot + 1;
        factors = reinterpret_cast<float2*>(tmem_slot + 4);
    }
    __device__ __forceinline__ uint32_t a(uint32_t s) const { return tiles + s * G::STAGE_BYTES; }
    __device__ __forceinline__ uint32_t b(uint32_t s) const { return tiles + s * G::STAGE_BYTES + G::A_BYTES; }
    __device__ __forceinline__ uint32_t raw(uint32_t s) const { return raw_tiles + s * G::RAW_BYTES; }
    __device__ __forceinline__ uint8_t* at(uint32_t addr) const { return base + (addr - tiles); }
    __device__ __forceinline__ uint8_t* out(int w) const { return base + G::TILES_BYTES + w * G::OUT_BYTES; }
};

// which half of a pair's tile this CTA works on
template <int CG>
__device__ __forceinline__ int half(const Ctl& ctl) {
    return CG == 2 ? ctl.rank : 0;
}

struct Unit {
    int mb, nb, lo, hi;  // tile and this CTA's stages of it
    int tail;            // pairs: half * tail_tiles + index of a tail tile, or -1
};
// Tiles in groups of group_m rows of tiles, so the tiles running at once share
// their operands in L2.  The tiles of a last round that would keep at most half
// of the pairs busy are cut into two halves of the contraction, all first
// halves before all second ones.
template <int CG>
__device__ __forceinline__ Unit unit_of(const GemmParams& p, const Ctl& ctl, int u) {
    Unit x;
    int t = u;
    x.tail = -1;
    if (CG == 2 && u >= p.tail_first) {
        x.tail = u - p.tail_first;
        t = p.tail_first + x.tail % p.tail_tiles;
    }
    const int per = p.group_m * p.n_blocks;
    const int g = t / per, first = g * p.group_m;
    const int rows = min(p.group_m, p.m_blocks - first), in = t - g * per;
    x.mb = first + in % rows;
    x.nb = in / rows;
    x.lo = CG == 1 ? ctl.rank * p.part_stages : 0;
    x.hi = min(p.stages_total, x.lo + p.part_stages);
    if (CG == 2 && x.tail >= 0) {
        if (x.tail < p.tail_tiles)
            x.hi = p.stages_total / 2;
        else
            x.lo = p.stages_total / 2;
    }
    return x;
}

// Loads.  KIND_MM: `which` 0 streams A and B.  KIND_WG: 0 streams the codes, 1
// streams dY.  The odd CTA's pair loads count on the even CTA's barrier, so to
// know that they have landed it waits until the MMA has read its last fill.
template <int KIND, int CG>
__device__ void run_tma(const GemmParams& p, const Ctl& ctl, Smem<KIND, CG>& sm, int which, int first, int step) {
    using G = Geo<KIND, CG>;
    if constexpr (KIND == KIND_MM) {
        Ring<G::STAGES> st;
        Fills fills;
        const uint32_t bytes = p.a_box * 128 + G::B_BYTES;
        bool ok = true;
        for (int u = first; u < p.n_units && ok; u += step) {
            const Unit x = unit_of<CG>(p, ctl, u);
            const int row = (x.mb * CG + half<CG>(ctl)) * BM;
            const int col = x.nb * G::BN + half<CG>(ctl) * (G::BN / CG);
            for (int s = x.lo; s < x.hi; ++s) {
                if (!wait_bar(ctl, sm.done + 8 * st.slot, st.phase ^ 1, WAIT_EMPTY)) {
                    ok = false;
                    break;
                }
                const int d = s * G::DEPTH;
                const int bc0 = p.b_mn ? col : d, bc1 = p.b_mn ? d : col;
                if (CG == 1) {
                    bar_expect_tx(sm.full + 8 * st.slot, bytes);
                    tma_load_2d(sm.a(st.slot), &p.tmA, d, row, sm.full + 8 * st.slot);
                    tma_load_2d(sm.b(st.slot), &p.tmB, bc0, bc1, sm.full + 8 * st.slot);
                } else {
                    if (half<CG>(ctl) == 0) bar_expect_tx(sm.full + 8 * st.slot, CG * bytes);
                    const uint32_t fb = map_to(sm.full + 8 * st.slot, 0);
                    tma_load_2d_pair(sm.a(st.slot), &p.tmA, d, row, fb);
                    tma_load_2d_pair(sm.b(st.slot), &p.tmB, bc0, bc1, fb);
                }
                fills.add(st.slot, st.phase);
                st.next();
            }
        }
        fills.drain(ctl, half<CG>(ctl) ? sm.done : sm.full, G::STAGES);
    } else if (which == 0) {
        Ring<G::RAWS> st;
        Fills fills;
        bool ok = true;
        for (int u = first; u < p.n_units && ok; u += step) {
            const Unit x = unit_of<CG>(p, ctl, u);
            const int row = (x.mb * CG + half<CG>(ctl)) * BM;
            for (int s = x.lo; s < x.hi; ++s) {
                if (!wait_bar(ctl, sm.raw_empty + 8 * st.slot, st.phase ^ 1, WAIT_EMPTY)) {
                    ok = false;
                    break;
                }
                bar_expect_tx(sm.raw_full + 8 * st.slot, G::RAW_BYTES);
                tma_load_2d(sm.raw(st.slot), &p.tmA, row, s * G::DEPTH, sm.raw_full + 8 * st.slot);
                fills.add(st.slot, st.phase);
                st.next();
            }
        }
        fills.drain(ctl, sm.raw_full, G::RAWS);
    } else {
        Ring<G::STAGES> st;
        Fills fills;
        bool ok = true;
        for (int u = first; u < p.n_units && ok; u += step) {
            const Unit x = unit_of<CG>(p, ctl, u);
            const int col = x.nb * G::BN + half<CG>(ctl) * (G::BN / CG);
            for (int s = x.lo; s < x.hi; ++s) {
                if (!wait_bar(ctl, sm.done + 8 * st.slot, st.phase ^ 1, WAIT_EMPTY)) {
                    ok = false;
                    break;
                }
                const int d = s * G::DEPTH;
                if (half<CG>(ctl) == 0) bar_expect_tx(sm.b_full + 8 * st.slot, CG * G::B_BYTES);
                const uint32_t fb = CG == 2 ? map_to(sm.b_full + 8 * st.slot, 0) : 0u;
                if (p.b_chunked) {
                    if (CG == 1)
                        tma_load_3d(sm.b(st.slot), &p.tmB, 0, d, col / 64, sm.b_full + 8 * st.slot);
                    else
                        tma_load_3d_pair(sm.b(st.slot), &p.tmB, 0, d, col / 64, fb);
                } else
                for (int c = 0; c < G::BN / CG / 64; ++c) {
                    if (CG == 1)
                        tma_load_2d(sm.b(st.slot) + c * 8192, &p.tmB, col + c * 64, d, sm.b_full + 8 * st.slot);
                    else
                        tma_load_2d_pair(sm.b(st.slot) + c * 8192, &p.tmB, col + c * 64, d, fb);
                }
                fills.add(st.slot, st.phase);
                st.next();
            }
        }
        fills.drain(ctl, half<CG>(ctl) ? sm.done : sm.b_full, G::STAGES);
    }
}

// MMAs.  The whole warp runs the loop, so that addresses and descriptors stay
// in uniform registers, where the tensor-core instructions take them from; one
// elected lane issues.  A stage has few MMAs (four), so whatever else the loop
// does per stage shows: with 128 x 128 tiles it takes longer than the MMAs, and
// two issuers take the chunks in turn (each chunk has its own accumulator).
template <int KIND, int CG>
__device__ void run_mma(const GemmParams& p, const Ctl& ctl, Smem<KIND, CG>& sm, uint32_t tmem, int issuer, int first,
                        int step) {
    using G = Geo<KIND, CG>;
    constexpr int CH = KIND == KIND_MM ? 1 : WG_CHUNK;
    // Descriptors.  K-major (A and B^T of KIND_MM): 8-row groups 1024 bytes
    // apart (stride offset), K steps of 32 codes 32 bytes further along the
    // swizzled rows.  MN-major: rows of 128 bytes per contraction index, 8-deep
    // groups 1024 bytes apart (stride offset), K steps of 32 or 16 rows;
    // KIND_WG's two 64-element columns are 8192 bytes apart (leading offset).
    const uint32_t a_adv = KIND == KIND_MM ? 2 : 128;
    const uint32_t b_adv = KIND == KIND_MM ? (p.b_mn ? 256 : 2) : 128;
    const uint32_t lead = KIND == KIND_MM ? 16 : 8192;
    const uint64_t a_desc = smem_desc(sm.a(0), lead, 1024), b_desc = smem_desc(sm.b(0), lead, 1024);
    const uint32_t idesc = p.idesc;
    Ring<G::STAGES> st;
    Ring<G::ACCS> acc;
    bool ok = true;
    for (int u = first; u < p.n_units && ok; u += step) {
        const Unit x = unit_of<CG>(p, ctl, u);
        const bool report = p.debug_skip != static_cast<uint32_t>(u) + 1;
        for (int s0 = x.lo; s0 < x.hi && ok; s0 += CH, acc.next()) {
            if (G::ISSUERS == 2 && (acc.slot & 1) != issuer) {
                st.next();
                continue;
            }
            if (!wait_bar(ctl, sm.acc_empty + 8 * acc.slot, acc.phase ^ 1, WAIT_ACC_EMPTY)) {
                ok = false;
                break;
            }
            const int end = min(x.hi, s0 + CH);
            const uint32_t d = tmem + acc.slot * G::BN;
            for (int s = s0; s < end; ++s, st.next()) {
                if (!wait_bar(ctl, sm.full + 8 * st.slot, st.phase, WAIT_FULL) ||
                    (KIND == KIND_WG && !wait_bar(ctl, sm.b_full + 8 * st.slot, st.phase, WAIT_FULL_B))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = a_desc + st.slot * (G::STAGE_BYTES / 16), bd = b_desc + st.slot * (G::STAGE_BYTES / 16);
                const uint32_t more = s > s0 ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < G::UMMA_STEPS; ++k) {
                        if (KIND == KIND_MM)
                            umma_f8<CG>(d, ad + k * a_adv, bd + k * b_adv, idesc, k > 0 ? 1u : more);
                        else
                            umma_f16<CG>(d, ad + k * a_adv, bd + k * b_adv, idesc, k > 0 ? 1u : more);
                    }
                    umma_commit_all<CG>(sm.done + 8 * st.slot);
                    if (s == end - 1 && report) umma_commit_all<CG>(sm.acc_full + 8 * acc.slot);
                }
                __syncwarp();
            }
        }
    }
    if (elect_one()) umma_commit_one<CG>(sm.final_bar + 8 * issuer);
    __syncwarp();
    wait_bar(ctl, sm.final_bar + 8 * issuer, 0, WAIT_DRAIN_MMA);
}

// 16 codes -> 16 scaled 16-bit values.  Codes go to f16 pairs (exact) and
// through fp32, times the scale, to the 16-bit type: one rounding, none for a
// power-of-two scale.  (Setting a code's bits into a bf16 number and scaling
// pairs of those takes as many instructions, all of them half rate.)
template <bool BF16, bool E5M2>
__device__ __forceinline__ void convert16(const uint4& c, float scale, uint32_t (&o)[8]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t h = cvt_f8x2_f16x2<E5M2>(w[j / 2], j & 1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        o[j] = pack16(f.x * scale, f.y * scale, BF16);
    }
}

__device__ __forceinline__ float load_bias(const GemmParams& p, int col) {
    if (!p.bias || col >= p.N) return 0.f;
    if (p.bias_type == T_F32) return load_elem<T_F32>(p.bias, col);
    return p.bias_type == T_F16 ? load_elem<T_F16>(p.bias, col) : load_elem<T_BF16>(p.bias, col);
}
__device__ __forceinline__ void store_out(const GemmParams& p, long long row, long long col, float v) {
    const long long i = row * p.out_rs + col * p.out_cs;
    if (p.out_type == T_F32)
        static_cast<float*>(p.out)[i] = v;
    else if (p.out_type == T_F16)
        static_cast<__half*>(p.out)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
}

// A promotion warp: sums and epilogue of its 32 rows x COLS columns of each
// tile, kept in fp32 registers.  DIRECT: tensor stores can write the output.
template <int KIND, int CG, bool DIRECT>
struct Worker {
    using G = Geo<KIND, CG>;
    static constexpr int COLS = G::COLS;
    const GemmParams& p;
    const Ctl& ctl;
    Smem<KIND, CG>& sm;
    const uint32_t tmem;
    const int w, lane, q, h;
    uint8_t* const stg;
    Ring<G::ACCS> from;  // the accumulator that the next chunk will be in
    uint32_t rounds = 0, stores = 0;
    unsigned long long acc[COLS / 2];  // pairs of fp32 sums

    __device__ __forceinline__ Worker(const GemmParams& p_, const Ctl& c_, Smem<KIND, CG>& s_, uint32_t t_, int w_, int lane_)
        : p(p_), ctl(c_), sm(s_), tmem(t_), w(w_), lane(lane_), q(w_ & 3), h(w_ >> 2), stg(s_.out(w_)) {
        clear();
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
    }

    // where this warp's part of a unit lies
    struct Place {
        int u;
        Unit x;
        int blk, row0;
        bool live;  // some of its rows and columns exist; otherwise it only keeps step
    };
    __device__ __forceinline__ Place place(int u) const {
        Place pl;
        pl.u = u;
        pl.x = unit_of<CG>(p, ctl, u);
        pl.blk = pl.x.mb * CG + half<CG>(ctl);
        pl.row0 = pl.blk * BM + q * 32;
        pl.live = pl.row0 < p.M && col_of(pl, 0) < p.N;
        return pl;
    }
    // first matrix column of the warp's c-th 32 columns
    __device__ __forceinline__ int col_of(const Place& pl, int c) const {
        return pl.x.nb * G::BN + h * COLS + c * 32;
    }

    // 32 columns' products times the scale, from the warp's column AT on
    template <int AT>
    __device__ __forceinline__ void add(const uint32_t (&r)[32], unsigned long long f2) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[AT / 2 + i] = fma_f32x2(pack_f32x2(r[2 * i], r[2 * i + 1]), f2, acc[AT / 2 + i]);
    }
    // acc += the next chunk's product * scale; the buffer is handed back as soon
    // as its last load has arrived.  Pairs read 32 columns while they add the
    // 32 before, and read rows and columns that do not exist as well: the loop
    // runs once per stage on the way from one MMA to the next but one, and fewer
    // instructions in it are worth more than idle warps (8192^3: 373 us; with 64
    // columns at a time, added in between, and a test of `live` 385).
    // Otherwise wide loads make few round trips to tensor memory.
    template <int LD>
    __device__ __forceinline__ bool promote(bool live, float scale) {
        const uint32_t buf = from.slot;
        if (!wait_bar(ctl, sm.acc_full + 8 * buf, from.phase, WAIT_ACC_FULL)) return false;
        from.next();
        __syncwarp();  // tensor-memory loads are for the converged warp
        tc_fence_after();
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2)
                    mbar_arrive_remote(map_to(sm.acc_empty + 8 * buf, 0));
                else
                    bar_arrive(sm.acc_empty + 8 * buf);
            }
        };
        constexpr bool PAIRS = KIND == KIND_MM && CG == 2;
        if (PAIRS || live) {
            const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::BN + h * COLS;
            const uint32_t f = __float_as_uint(scale);
            const unsigned long long f2 = pack_f32x2(f, f);
            if constexpr (PAIRS) {
                uint32_t r0[32], r1[32];
                tmem_ld_cols(base, r0);
                tmem_wait_regs(r0);
                tmem_ld_cols(base + 32, r1);
                add<0>(r0, f2);
                tmem_wait_regs(r1);
                tmem_ld_cols(base + 64, r0);
                add<32>(r1, f2);
                tmem_wait_regs(r0);
                tmem_ld_cols(base + 96, r1);
                add<64>(r0, f2);
                tmem_wait_regs(r1);
                release();
                add<96>(r1, f2);
            } else {
                uint32_t r[LD];
#pragma unroll
                for (int c = 0; c < COLS / LD; ++c) {
                    tmem_ld_cols(base + c * LD, r);
                    tmem_wait_regs(r);
                    if (c == COLS / LD - 1) release();
#pragma unroll
                    for (int i = 0; i < LD / 2; ++i)
                        acc[c * (LD / 2) + i] = fma_f32x2(pack_f32x2(r[2 * i], r[2 * i + 1]), f2, acc[c * (LD / 2) + i]);
                }
            }
        } else {
            release();
        }
        return true;
    }

    // A staged box to an output that no tensor store can reach.  Rows of unit
    // stride that start anywhere: box k of a warp's part of a row fills the 128
    // aligned bytes from its first byte's granule on, with what the box before
    // left over, eight lanes to a row, each shifting 16 bytes into place; only
    // what lies before the row's first granule and after its last goes by
    // elements.  Bound by the latency of its instructions (8 warps), hence fixed
    // shared addresses and, beside several boxes, edges in loops of their own
    // (333 x 1000 x 1111: 9.4 us, with such loops 9.7; weight gradient of 4
    // tokens, 6840 x 3567 f32: 48 us; a box at a time, edges and all, 66; with
    // 3568 columns and tensor stores 20).
    template <typename E>
    __device__ __forceinline__ void store_rows(int k, int row0, int c0) const {
        constexpr int SIZE = sizeof(E), ROW = G::BOXES == 1 ? 128 : COLS * SIZE;
        // columns are clipped before they become bytes, which may pass 2^31
        const int g = lane & 7, r0 = lane >> 3, rows = min(32, p.M - row0), bytes = min(ROW / SIZE, p.N - c0) * SIZE;
        const long long step = 4 * SIZE * p.out_rs;
        uint8_t* const to0 = static_cast<uint8_t*>(p.out) + ((row0 + r0) * p.out_rs + c0) * SIZE;
        // unit n of row r, units XORed with the row
        auto unit = [&](int n, int r) { return stg + (n >> 3) % G::BOXES * 4096 + r * 128 + (((n ^ r) & 7) << 4); };
        const uint8_t *const here = unit(8 * k + g, r0), *const before = unit(8 * k + g + 8 * G::BOXES - 1, r0);
        auto element = [&](uint8_t* row, int r, int b) {
            *reinterpret_cast<E*>(row + b) = *reinterpret_cast<const E*>(unit(b >> 4, r) + (b & 15));
        };
        auto head = [&](uint8_t* row, int r) {
            if (g * SIZE < min(-static_cast<int>(reinterpret_cast<uintptr_t>(row)) & 15, bytes)) element(row, r, g * SIZE);
        };
        auto tail = [&](uint8_t* row, int r) {
            const int first = -static_cast<int>(reinterpret_cast<uintptr_t>(row)) & 15;
            const int end = bytes - (static_cast<int>(reinterpret_cast<uintptr_t>(row + bytes)) & 15);
            const int b = max(first, end) + g * SIZE;
            if (g * SIZE < 16 && b < bytes) element(row, r, b);
        };
        uint8_t* to = to0;
#pragma unroll 2
        for (int i = 0; i < 8; ++i, to += step) {
            if (r0 + 4 * i >= rows) break;
            const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(to)) & 15, o = 128 * k + 16 * g - mis;
            // row r0 + 4 i: 512 bytes per i, and every other i flips bit 2 of the unit
            const uint8_t* const a = (mis ? before : here) + i * 512;
            const uint8_t* const b = here + i * 512;
            const uint4 lo = *reinterpret_cast<const uint4*>(stg + (static_cast<int>(a - stg) ^ (i & 1) << 6));
            const uint4 hi = *reinterpret_cast<const uint4*>(stg + (static_cast<int>(b - stg) ^ (i & 1) << 6));
            const uint32_t two[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t v[4];
            shift_granules<1>(two, (16 - mis) & 15, v);
            if (o >= 0 && o + 16 <= bytes) *reinterpret_cast<uint4*>(to + o) = make_uint4(v[0], v[1], v[2], v[3]);
            if (G::BOXES == 1) {
                head(to, r0 + 4 * i);
                tail(to, r0 + 4 * i);
            }
        }
        if (G::BOXES > 1 && k == 0) {
            to = to0;
#pragma unroll 2
            for (int r = r0; r < rows; r += 4, to += step) head(to, r);
        }
        if (G::BOXES > 1 && 128 * (k + 1) >= bytes) {
            to = to0;
#pragma unroll 2
            for (int r = r0; r < rows; r += 4, to += step) tail(to, r);
        }
    }
    // any strides: a lane per column
    template <typename E>
    __device__ __forceinline__ void store_elements(const uint8_t* box, int row0, int c0) const {
        constexpr int PER = 128 / (32 * sizeof(E));  // columns per lane
        const int rows = min(32, p.M - row0);
        E* to = static_cast<E*>(p.out) + row0 * p.out_rs + (c0 + lane) * p.out_cs;
#pragma unroll 2
        for (int r = 0; r < rows; ++r, to += p.out_rs) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int b = (lane + 32 * e) * static_cast<int>(sizeof(E));  // byte in the row
                if (c0 + lane + 32 * e < p.N)
                    to[32 * e * p.out_cs] = *reinterpret_cast<const E*>(box + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15));
            }
        }
    }

    // Split contraction over S CTAs: each warp lays its 32 x 64 sums into shared
    // memory, as many columns at a time as its staging holds (rows of units of
    // 16 bytes, XORed with the row), tells the same warp of every part, and adds
    // its part's rows of them over all parts in order.  The loads from the
    // other CTAs are all under way at once; neighbouring lanes hold neighbouring
    // columns of a row, so stores reach few rows each.  After its last tile a
    // CTA's stages are free, and hold all columns at once (48 x 14336 x
    // 4096, whose staging holds half of them: 18.1 -> 17.1 us).
    template <int S, int UNITS>
    __device__ __forceinline__ bool join(const Place& pl, bool more) {
        constexpr int ROUNDS = 16 / UNITS, SHARE = UNITS / S;
        uint8_t* const stg = UNITS * 512 <= G::OUT_BYTES ? this->stg : sm.at(sm.tiles) + w * UNITS * 512;
        static_assert(8 * UNITS * 512 <= G::STAGES * G::STAGE_BYTES, "all warps' sums fit the stages");
        const uint32_t row_at = lane * UNITS * 16;
        const int unit = lane % UNITS;
        auto share_row = [&](int i) { return ctl.rank * (32 / S) + i * (32 / UNITS) + lane / UNITS; };  // of the warp's 32
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            // the other parts have read what lay here before
            if (rounds > 0 && !wait_bar_cluster(ctl, sm.parts_out + 8 * w, (rounds - 1) & 1, WAIT_PARTS)) return false;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                float v[4];
                unpack_f32x2(acc[2 * (r * UNITS + j)], v[0], v[1]);
                unpack_f32x2(acc[2 * (r * UNITS + j) + 1], v[2], v[3]);
                *reinterpret_cast<float4*>(stg + row_at + ((j ^ (lane & (UNITS - 1))) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
            }
            __syncwarp();
            if (lane < S) mbar_arrive_cluster(map_to(sm.parts_in + 8 * w, lane));
            if (!wait_bar_cluster(ctl, sm.parts_in + 8 * w, rounds & 1, WAIT_PARTS)) return false;
            __syncwarp();
            ++rounds;
            const uint32_t all = smem_u32(stg);
            float4 t[SHARE][S];
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const uint32_t from_k = map_to(all, k);
#pragma unroll
                for (int i = 0; i < SHARE; ++i) {
                    const int at = share_row(i);
                    t[i][k] = ld_shared_cluster_f4(from_k + at * UNITS * 16 + ((unit ^ (at & (UNITS - 1))) << 4));
                }
            }
#pragma unroll
            for (int i = 0; i < SHARE; ++i) {
                float4 sum = t[i][0];
#pragma unroll
                for (int k = 1; k < S; ++k) {
                    sum.x += t[i][k].x;
                    sum.y += t[i][k].y;
                    sum.z += t[i][k].z;
                    sum.w += t[i][k].w;
                }
                const int row = pl.row0 + share_row(i), c = col_of(pl, 0) + (r * UNITS + unit) * 4;
                float v[4] = {sum.x, sum.y, sum.z, sum.w};
                if (KIND == KIND_MM && p.bias) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += load_bias(p, c + e);
                }
                if (row < p.M) {
                    if (DIRECT && c + 4 <= p.N) {  // unit stride, rows on 16 bytes
                        const long long o = row * p.out_rs + c;
                        if (p.out_type == T_F32)
                            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
                        else
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
                                make_uint2(pack16(v[0], v[1], p.out_type == T_BF16), pack16(v[2], v[3], p.out_type == T_BF16));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (c + e < p.N) store_out(p, row, c + e, v[e]);
                    }
                }
            }
            // the values above are in registers: the parts may lay their next
            // sums, if there are any: a CTA on its way out gets no more arrivals
            __syncwarp();
            if ((more || r + 1 < ROUNDS) && lane < S) mbar_arrive_cluster(map_to(sm.parts_out + 8 * w, lane));
        }
        return true;
    }

    template <int UNITS>
    __device__ __forceinline__ bool join_parts(const Place& pl, bool more) {
        return p.split == 2 ? join<2, UNITS>(pl, more) : p.split == 4 ? join<4, UNITS>(pl, more) : join<8, UNITS>(pl, more);
    }

    // Tail tiles: the first half's warps leave their sums in global memory, the
    // same warps of the second half take them up, first half first.  Both halves
    // run in the launch's last round, the first ones on the pairs that start
    // first.  A flag holds the launch's epoch.
    __device__ __forceinline__ bool tail(const Place& pl) {
        const int i = ((pl.x.tail % p.tail_tiles) * CG + ctl.rank) * 8 + w;
        unsigned long long* at = p.tail_sums + static_cast<size_t>(i) * (COLS / 2 * 32) + lane;
        const unsigned long long ready = static_cast<unsigned long long>(ctl.epoch) << 32 | 0x5A17F1A6u;
        if (pl.x.tail < p.tail_tiles) {
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j) at[j * 32] = acc[j];
            __threadfence();
            __syncwarp();
            if (lane == 0) st_release_gpu_u64(p.tail_flag + i, ready);
            return true;
        }
        bool there = ld_acquire_gpu_u64(p.tail_flag + i) == ready;
        const uint64_t t0 = global_timer_ns();
        while (!there) {
            __nanosleep(100);
            there = ld_acquire_gpu_u64(p.tail_flag + i) == ready;
            if (!there && (launch_aborted(ctl) || global_timer_ns() - t0 > ctl.limit)) {
                if (!launch_aborted(ctl)) raise_timeout(ctl, WAIT_TAIL, i);
                return false;
            }
        }
        __syncwarp();
        const unsigned long long one = pack_f32x2(0x3F800000u, 0x3F800000u);
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) acc[j] = fma_f32x2(acc[j], one, __ldcg(at + j * 32));
        return true;
    }

    __device__ __forceinline__ bool epilogue(const Place& pl, bool more) {
        if (CG == 2 && pl.x.tail >= 0) {
            if (pl.live && !tail(pl)) return false;
            if (pl.x.tail < p.tail_tiles) {  // the second half writes the output
                clear();
                return true;
            }
        }
        if (CG == 1 && p.split > 1) {
            // not live in one part: not live in any
            constexpr int STAGED = G::OUT_BYTES / 512;
            if (pl.live && !(more ? join_parts<STAGED>(pl, true) : join_parts<16>(pl, false))) return false;
            clear();
            return true;
        }
        // 32 rows x 128 bytes at a time through swizzled staging; the sums are
        // rounded here, once
        if (pl.live) {
            const bool wide = p.out_type == T_F32;
            const bool add_bias = KIND == KIND_MM && p.bias != nullptr;
#pragma unroll
            for (int c = 0; c < COLS / 32; ++c) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) unpack_f32x2(acc[c * 16 + i], v[2 * i], v[2 * i + 1]);
                if (add_bias) {
                    const float b = load_bias(p, col_of(pl, c) + lane);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, b, i);
                }
                if (wide || (c & 1) == 0) {  // a staging box is used anew
                    if (lane == 0) bulk_wait_read<G::BOXES - 1>();
                    __syncwarp();
                }
                uint8_t* box = stg + (DIRECT ? stores : wide ? c : c / 2) % G::BOXES * 4096;
                if (wide) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<float4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else {
                    const int bf = p.out_type == T_BF16;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(box + lane * 128 + (((j + (c & 1) * 4) ^ (lane & 7)) << 4)) =
                            make_uint4(pack16(v[8 * j], v[8 * j + 1], bf), pack16(v[8 * j + 2], v[8 * j + 3], bf),
                                       pack16(v[8 * j + 4], v[8 * j + 5], bf), pack16(v[8 * j + 6], v[8 * j + 7], bf));
                }
                if (wide || (c & 1) == 1) {
                    const int cc = col_of(pl, wide ? c : c - 1);
                    if constexpr (DIRECT) {  // a tensor store, which clips the ragged edges
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            if (cc < p.N) tma_store_2d(&p.tmC, box, cc, pl.row0);
                            bulk_commit();
                        }
                        ++stores;
                    } else {
                        __syncwarp();
                        // box k of the warp's part of a row, or of its own
                        const int k = G::BOXES == 1 ? 0 : wide ? c : c / 2, row_c = G::BOXES == 1 ? cc : col_of(pl, 0);
                        const bool rows = p.out_cs == 1;
                        if (cc >= p.N) {
                        } else if (rows && wide) {
                            store_rows<float>(k, pl.row0, row_c);
                        } else if (rows) {
                            store_rows<uint16_t>(k, pl.row0, row_c);
                        } else if (wide) {
                            store_elements<float>(box, pl.row0, cc);
                        } else {
                            store_elements<uint16_t>(box, pl.row0, cc);
                        }
                        __syncwarp();
                    }
                }
            }
        }
        clear();
        return true;
    }
};

// Promotion warps; false = a wait gave up.
template <int CG, bool DIRECT>
__device__ bool run_promote_mm(const GemmParams& p, const Ctl& ctl, Smem<KIND_MM, CG>& sm, uint32_t tmem, int w, int lane,
                            int first, int step) {
    Worker<KIND_MM, CG, DIRECT> wk(p, ctl, sm, tmem, w, lane);
    for (int u = first; u < p.n_units; u += step) {
        const auto pl = wk.place(u);
        // A stage's two scales are fetched AHEAD stages ahead, into registers
        // of their own (the loop is unrolled by as many), so that no load is
        // waited for: passing them from register to register would wait for
        // each within its stage.  Pairs do not unroll: two copies of their
        // longer loop do not run from the nearest instruction cache.
        // Rows below the last read its scales; past the last stage the last
        // one's are read.
        constexpr int AHEAD = CG == 2 ? 1 : 4;
        const float* pa = p.sa + min(pl.row0 + lane, p.M - 1) * p.sa_rs + pl.x.lo * p.sa_cs;
        const float* pb = p.sb + min(wk.col_of(pl, 0), p.N - 1) / 128 * p.sb_cs + pl.x.lo * p.sb_rs;
        int left = pl.x.hi - pl.x.lo;
        float a[AHEAD], b[AHEAD];
        auto fetch = [&](float& fa, float& fb) {
            fa = *pa;
            fb = *pb;
            if (--left > 0) {
                pa += p.sa_cs;
                pb += p.sb_rs;
            }
        };
        if (left > 0) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) fetch(a[j], b[j]);
        }
        for (int s = pl.x.lo; s < pl.x.hi; s += AHEAD) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (s + j >= pl.x.hi) break;
                const float scale = a[j] * b[j];
                fetch(a[j], b[j]);
                if (!wk.template promote<64>(pl.live, scale)) return false;
            }
        }
        if (!wk.epilogue(pl, u + step < p.n_units)) return false;
    }
    return true;
}

// f16 weight gradients: code * scale can be as large as fp32 holds, and f16 ends
// at 65504 (an f16 input close to that becomes 2^16 by its codes already).  So
// each chunk of WG_CHUNK stages has a power of two 2^-f, by which its scales are
// multiplied on their way into f16 and its sums divided again in fp32.  f is 0
// where the chunk's largest finite scale keeps every code within f16's range and
// the finest code step at f16's own, 2^-24, or above it: there a code times a
// power-of-two scale is exact.  Otherwise the largest scale is taken to the
// largest power of two that fits, and values are exact down to 2^(f - 24), 2^-39
// of the largest value that the chunk could hold.
// Warp 3, which has nothing else to do, is up to FACTORS chunks ahead: 16
// scales a lane, all loads in flight, beside some 3 us of MMAs per chunk.  What
// it costs is the converters' wait, once a chunk, and the first chunk's scales:
// 4096 x 4096 x 14336 f16 into f32 340 -> 350 us, 777 x 1000 x 1112 9.8 -> 10.4
// (with the power left out of the scales where it is 1; 355, 10.5 always in).
template <int CG>
__device__ void run_factors(const GemmParams& p, const Ctl& ctl, Smem<KIND_WG, CG>& sm, int lane, int first, int step) {
    using G = Geo<KIND_WG, CG>;
    constexpr int PER = WG_CHUNK * G::DEPTH / 32;
    Ring<G::FACTORS> fac;
    const float fmax = p.codes_e5m2 ? 57344.f : 448.f;
    const int top = p.codes_e5m2 ? 0 : 7;        // largest 2^top with fmax * 2^top <= 65504
    const int bottom = p.codes_e5m2 ? -8 : -15;  // 2^bottom times the codes' finest step is 2^-24
    for (int u = first; u < p.n_units; u += step) {
        const Unit x = unit_of<CG>(p, ctl, u);
        const int kblk = x.mb * CG + half<CG>(ctl);
        const bool live = kblk * BM < p.M;
        for (int s = x.lo; s < x.hi; s += WG_CHUNK, fac.next()) {
            const long long m0 = static_cast<long long>(s) * G::DEPTH + lane;
            const int left = live ? min(p.D, min(x.hi, s + WG_CHUNK) * G::DEPTH) - s * G::DEPTH - lane : 0;
            const float* at = p.sa + kblk * p.sa_cs + m0 * p.sa_rs;
            const long long apart = 32 * p.sa_rs;
            float v[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                v[i] = 32 * i < left ? *at : 0.f;
                at += apart;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = amax_finite(0.f, v[i]);
#pragma unroll
            for (int w = PER / 2; w > 0; w /= 2)
#pragma unroll
                for (int i = 0; i < w; ++i) v[i] = fmaxf(v[i], v[i + w]);
            // magnitudes order like their bits
            const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[0]));
            const float m = __uint_as_float(bits);
            // m <= 2^e (subnormal scales: 2^-126)
            const int e = max(static_cast<int>(bits >> 23), 1) - 127 + ((bits & 0x7FFFFFu) && bits >> 23 ? 1 : 0);
            int f = 0;
            if (bits != 0u && (m * fmax >= 65520.f || e < bottom)) f = max(-126, min(126, e - top));
            // all lanes leave or none: the reduction above is the whole warp's
            if (!__all_sync(0xFFFFFFFFu, wait_bar(ctl, sm.fac_empty + 8 * fac.slot, fac.phase ^ 1, WAIT_FACTOR_EMPTY))) return;
            if (lane == 0) {
                sm.factors[fac.slot] = make_float2(__int_as_float((127 - f) << 23), __int_as_float((127 + f) << 23));
                bar_arrive(sm.fac_full + 8 * fac.slot);
            }
            __syncwarp();
        }
    }
}
// The next chunk's factors, for a warp; each of the sixteen that use them tells
// warp 3 that it has them.
template <int CG>
__device__ __forceinline__ bool take_factor(const Ctl& ctl, Smem<KIND_WG, CG>& sm, Ring<Geo<KIND_WG, CG>::FACTORS>& fac, int lane,
                                            float2& f) {
    if (!wait_bar(ctl, sm.fac_full + 8 * fac.slot, fac.phase, WAIT_FACTOR)) return false;
    f = sm.factors[fac.slot];
    __syncwarp();
    if (lane == 0) bar_arrive(sm.fac_empty + 8 * fac.slot);
    fac.next();
    return true;
}

template <int CG, bool DIRECT, bool BF16>
__device__ bool run_promote_wg(const GemmParams& p, const Ctl& ctl, Smem<KIND_WG, CG>& sm, uint32_t tmem, int w, int lane,
                               int first, int step) {
    Worker<KIND_WG, CG, DIRECT> wk(p, ctl, sm, tmem, w, lane);
    Ring<Geo<KIND_WG, CG>::FACTORS> fac;
    for (int u = first; u < p.n_units; u += step) {
        const auto pl = wk.place(u);
        for (int s = pl.x.lo; s < pl.x.hi; s += WG_CHUNK) {
            float2 f = make_float2(1.f, 1.f);
            if (!BF16 && !take_factor(ctl, sm, fac, lane, f)) return false;
            if (!wk.template promote<16>(pl.live, f.y)) return false;
        }
        if (!wk.epilogue(pl, u + step < p.n_units)) return false;
    }
    return true;
}

// Conversion: 64 x 128 codes -> 16-bit values times their row's scale, in the
// MN-major swizzled layout (two columns of 64 k, rows of 128 bytes, 16-byte
// units XORed with the row; the codes lie swizzled alike).  Two groups of four
// warps take the stages in turn, so one stage's latencies (barrier, shared
// memory, fence) pass under the other's arithmetic.  A thread takes 16 codes
// of four rows, 16 apart.  Eight neighbouring threads take half of two rows
// whose numbers differ in bits 0 and 2: their codes' units and their results'
// units then are eight different ones, so no bank is asked twice.
template <int CG, bool BF16, bool E5M2>
__device__ void run_convert(const GemmParams& p, const Ctl& ctl, Smem<KIND_WG, CG>& sm, int t, int first, int step) {
    using G = Geo<KIND_WG, CG>;
    Ring<G::RAWS> rs;
    Ring<G::STAGES> st;
    Ring<G::FACTORS> fac;
    float2 factor = make_float2(1.f, 1.f);
    const int group = t >> 7, tt = t & 127;
    const int col = tt >> 3 & 1, j = tt & 3;                 // column of 64 k, quarter of it
    const int r0 = (tt >> 4) * 2 ^ ((tt & 4) ? 5 : 0);        // first row
    // offsets in a slot; rows r0 + 16 i have the same XOR
    const uint32_t from = r0 * 128 + (((col * 4 + j) ^ (r0 & 7)) << 4);
    const uint32_t to0 = col * 8192 + r0 * 128 + (((2 * j) ^ (r0 & 7)) << 4);
    const uint32_t to1 = col * 8192 + r0 * 128 + (((2 * j + 1) ^ (r0 & 7)) << 4);
    const long long apart = 16 * p.sa_rs;
    int turn = 0;  // stages so far, over all units
    for (int u = first; u < p.n_units; u += step) {
        const Unit x = unit_of<CG>(p, ctl, u);
        // this CTA's 128 output rows are one block of scales; a stage's are
        // fetched one turn (two stages) ahead.  Rows past the last count as 0.
        const int kblk = x.mb * CG + half<CG>(ctl);
        const int s0 = x.lo + ((turn & 1) != group);
        const float* at = p.sa + kblk * p.sa_cs + (static_cast<long long>(s0) * G::DEPTH + r0) * p.sa_rs;
        int left = kblk * BM < p.M ? min(p.D, x.hi * G::DEPTH) - s0 * G::DEPTH - r0 : 0;  // rows from `at` on
        float next[4];
        auto fetch = [&]() {
            const float* q = at;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                next[i] = 16 * i < left ? *q : 0.f;
                q += apart;
            }
            at += 8 * apart;
            left -= 2 * G::DEPTH;
        };
        fetch();
        for (int s = x.lo; s < x.hi; ++s, ++turn, rs.next(), st.next()) {
            // both groups take every chunk's factors, whether or not it has a stage of theirs
            if (!BF16 && (s - x.lo) % WG_CHUNK == 0 && !take_factor(ctl, sm, fac, t & 31, factor)) return;
            if ((turn & 1) != group) continue;
            float sc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[i] = next[i];
            if (!BF16 && factor.x != 1.f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[i] *= factor.x;
            }
            fetch();
            if (!wait_bar(ctl, sm.raw_full + 8 * rs.slot, rs.phase, WAIT_RAW)) return;
            if (!wait_bar(ctl, sm.done + 8 * st.slot, st.phase ^ 1, WAIT_A_EMPTY)) return;
            const uint8_t* src = sm.at(sm.raw(rs.slot)) + from;
            uint8_t* dst = sm.at(sm.a(st.slot));
            uint4 c4 = *reinterpret_cast<const uint4*>(src);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 c = c4;
                if (i < 3) c4 = *reinterpret_cast<const uint4*>(src + (i + 1) * 2048);
                uint32_t o[8];
                convert16<BF16, E5M2>(c, sc[i], o);
                *reinterpret_cast<uint4*>(dst + to0 + i * 2048) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dst + to1 + i * 2048) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if ((t & 31) == 0) {
                bar_arrive(sm.raw_empty + 8 * rs.slot);
                if (CG == 2)
                    mbar_arrive_remote(map_to(sm.full + 8 * st.slot, 0));
                else
                    bar_arrive(sm.full + 8 * st.slot);
            }
        }
    }
}

// DIRECT is a form of its own because the code of the other kind of stores,
// beside the pairs' promotion loop, costs that loop registers.
template <int KIND, int CG, bool DIRECT>
__global__ void __launch_bounds__(Geo<KIND, CG>::THREADS, 1) block_gemm_kernel(const __grid_constant__ GemmParams p) {
    using G = Geo<KIND, CG>;
    extern __shared__ uint8_t smem_raw[];
    Smem<KIND, CG> sm;
    sm.carve(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // CTAs per cluster: the pair, or the parts of the contraction
    const int csize = CG == 2 ? 2 : p.split;
    const int rank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            bar_init(sm.full + 8 * s, KIND == KIND_MM ? 1 : CG * 4);
            bar_init(sm.done + 8 * s, 1);
            bar_init(sm.b_full + 8 * s, 1);
        }
        for (int s = 0; s < G::RAWS; ++s) {
            bar_init(sm.raw_full + 8 * s, 1);
            bar_init(sm.raw_empty + 8 * s, 4);
        }
        for (int b = 0; b < G::ACCS; ++b) {
            bar_init(sm.acc_full + 8 * b, 1);
            bar_init(sm.acc_empty + 8 * b, CG * 8);
        }
        for (int i = 0; i < 8; ++i) {
            bar_init(sm.parts_in + 8 * i, csize);
            bar_init(sm.parts_out + 8 * i, csize);
        }
        bar_init(sm.final_bar, 1);
        bar_init(sm.final_bar + 8, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        if (DIRECT && p.split == 1) tma_prefetch_desc(&p.tmC);
        // for the whole CTA, which waits for this thread below
        grid_wait();
        grid_release();
        uint32_t e = *reinterpret_cast<volatile uint32_t*>(&p.ws->epoch) + 1u;
        *sm.epoch_slot = e == 0u ? 1u : e;
    }
    if (KIND == KIND_WG && threadIdx.x == 96 && !p.x_bf16)
        for (int s = 0; s < G::FACTORS; ++s) {
            bar_init(sm.fac_full + 8 * s, 1);
            bar_init(sm.fac_empty + 8 * s, 16);
        }
    if (warp == 1) tmem_alloc<G::TMEM_COLS, CG>(sm.tmem_slot);
    tc_fence_before();
    __syncthreads();
    if (csize > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    const Ctl ctl{p.ws, *sm.epoch_slot, p.wait_ns, rank};
    const int first = blockIdx.x / csize, step = gridDim.x / csize;

    if (warp < 4) {
        reg_dec<G::REGS_CTL>();
        if (warp == 0) {
            if (lane == 0) run_tma<KIND, CG>(p, ctl, sm, 0, first, step);
        } else if (KIND == KIND_WG && warp == 2) {
            if (lane == 0) run_tma<KIND, CG>(p, ctl, sm, 1, first, step);
        } else if (warp == 1) {
            if (CG == 1 || rank == 0) run_mma<KIND, CG>(p, ctl, sm, tmem, 0, first, step);
        }
        if (G::ISSUERS == 2 && warp == 3) run_mma<KIND, CG>(p, ctl, sm, tmem, 1, first, step);
        if constexpr (KIND == KIND_WG)
            if (warp == 3 && !p.x_bf16) run_factors<CG>(p, ctl, sm, lane, first, step);
        __syncwarp();
    } else if (warp < 12) {
        reg_inc<G::REGS_PROMOTE>();
        if constexpr (KIND == KIND_MM)
            run_promote_mm<CG, DIRECT>(p, ctl, sm, tmem, warp - 4, lane, first, step);
        else
            p.x_bf16 ? run_promote_wg<CG, DIRECT, true>(p, ctl, sm, tmem, warp - 4, lane, first, step)
                     : run_promote_wg<CG, DIRECT, false>(p, ctl, sm, tmem, warp - 4, lane, first, step);
        if (lane == 0) bulk_wait_all();  // its stores have left shared memory, stopped or not
        __syncwarp();
    } else if constexpr (KIND == KIND_WG) {
        reg_dec<G::REGS_CONVERT>();
        const int t = threadIdx.x - 384;
        if (p.x_bf16)
            p.codes_e5m2 ? run_convert<CG, true, true>(p, ctl, sm, t, first, step)
                         : run_convert<CG, true, false>(p, ctl, sm, t, first, step);
        else
            p.codes_e5m2 ? run_convert<CG, false, true>(p, ctl, sm, t, first, step)
                         : run_convert<CG, false, false>(p, ctl, sm, t, first, step);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // no CTA of a cluster leaves (or frees tensor memory) while another may
    // still signal its barriers or read its shared memory
    if (csize > 1) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<G::TMEM_COLS, CG>(tmem);
    }
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&p.ws->done_ctr, 1u) == gridDim.x - 1)
            *reinterpret_cast<uint4*>(p.ws) = make_uint4(ctl.epoch, 0u, 0u, 0u);
    }
}

// Empty contraction: out = bias, or zero.
__global__ void __launch_bounds__(256) fill_kernel(const __grid_constant__ GemmParams p) {
    grid_wait();
    grid_release();
    const long long n = static_cast<long long>(p.M) * p.N;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
        store_out(p, i / p.N, i % p.N, load_bias(p, static_cast<int>(i % p.N)));
}

}  // namespace fp8
}  // namespace gct
