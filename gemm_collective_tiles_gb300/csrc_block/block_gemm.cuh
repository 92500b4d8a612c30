// Persistent tensor-core kernel of the 16-bit product with its epilogue.
//
//   z[m][n] = sum_k A[m][k] B[k][n] + bias[n]
//   out[m][n] = residual[m][n] + drop(act(z[m][n]))
//
// A stage holds 64 of the contraction: an operand whose contraction is
// contiguous in memory lies there in rows of 128 bytes (K-major), one whose rows
// or columns are contiguous in two blocks of 64 of them by 64 of the contraction
// (MN-major); the tensor core takes either, so no operand is transposed and the
// products of a layer's backward pass (dz B^T, A^T dz) read the tensors as they
// are.  Sums stay in tensor memory until a tile is done; with two or four
// accumulators the next tile's MMAs run under this one's epilogue.
//
// Bound by the tensor cores, and before them by what the L2 delivers: a stage of a
// pair's 256 x 256 tile is 32 KB per SM for 512 cycles of MMA, one of a 128 x 128
// tile 32 KB for 256.  Measured, 4096 x 4096 x 14336: 247 us (1.95 PFLOP/s), with
// bias 249, gelu 254, gelu_tanh 250, z beside out 261, dropout 256; on 256 x 128
// tiles 405, on 128 x 128 455.
//
// CTA layout, one CTA per SM:
//   warp 0       TMA producer (lane 0)
//   warp 1       MMA issuer; owns tensor memory
//   warps 4-11   epilogue: quadrant warp % 4 of the accumulator's rows, column
//                half (warp - 4) / 4
// CG = 2: a cluster of two CTAs computes a 256 x BN tile with
// tcgen05.mma.cta_group::2, each staging its 128 rows of A and half of B's
// columns; the even CTA issues the MMAs.  CG = 1: 128 x 128 tiles, of which a
// cluster of 2, 4 or 8 CTAs may each take a part of the contraction; the fp32
// sums meet in shared memory and are added in the order of the parts.
//
// Every wait is bounded: one that gives up records where in the workspace
// header, stops the launch, and the roles drain and leave.
#pragma once
#include "../csrc_fp8/fp8_wait.cuh"
#include "act.cuh"

namespace gct {
namespace block {

using namespace gct::fp8;

constexpr int ROWS = 128;       // rows per CTA (tensor-memory lanes)
constexpr int DEPTH = 64;       // contraction per stage
constexpr int MOST_PARTS = 8;   // CTAs of a cluster that share a tile
constexpr int WAIT_RESIDUAL = 112;

struct ActParams {
    CUtensorMap tmA, tmB;  // K-major {k, row}, box {64, rows of a CTA}; MN-major {row, k}, box {64, 64}
    CUtensorMap tmC, tmR, tmZ;  // out, residual, z {n, row}, box {128 bytes, 32}
    int M, N, D;           // output rows and columns, contraction
    int stages_total, split;  // contraction in stages; CTAs that share a tile's
    int m_blocks, n_blocks, group_m, n_units;
    int a_mn, b_mn;        // MN-major operands; 2: their maps are {64, k, row / 64}, one box a stage
    int tail_first, tail_tiles, tail_parts;  // pairs: the last tiles are cut into parts of the contraction
    unsigned long long* tail_flags;  // per (part but the last, tail tile, CTA, epilogue warp): its sums are there
    float* tail_sums;                // 32 x COLS each, in fours of columns, 32 rows next to each other
    uint32_t idesc;
    const void* bias;
    int bias_type;
    int bias_near;         // of 16 bits, on 16 bytes
    void *out, *z;         // z may be absent
    const void* residual;  // may be absent
    int type;              // of out, z and residual
    int out_tma, z_tma, res_tma;
    long long out_rs, out_cs, z_rs, z_cs, res_rs, res_cs;
    int act;
    Drop drop;
    WsHeader* ws;
    unsigned long long wait_ns;
    uint32_t debug_skip;   // test hook: k > 0: tile k - 1 never reports its accumulator
};

__device__ __forceinline__ float bias_at(const ActParams& p, int col) {
    return p.bias && col < p.N ? load_any(p.bias, p.bias_type, col) : 0.f;
}

// A lane's four neighbouring columns (from a multiple of 4 on), for rows whose
// sums come through shared memory: the rest of the formula.  Their bias is
// fetched before the sums are there.
struct Four {
    int col;
    bool live, whole;  // some of them exist, all do
    float bias[4];
    __device__ __forceinline__ Four(const ActParams& p, int c) : col(c), live(c < p.N), whole(c + 4 <= p.N) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = bias_at(p, c + e);
    }
    __device__ __forceinline__ float4 residual(const ActParams& p, long long row) const {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!p.residual || !live || row >= p.M) return f;
        if (p.res_tma && whole) {  // unit stride, rows on 16 bytes
            if (p.type == T_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + row * p.res_rs + col);
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.residual) + row * p.res_rs + col);
            if (p.type == T_F16) {
                unpack16<T_F16>(u.x, f.x, f.y);
                unpack16<T_F16>(u.y, f.z, f.w);
            } else {
                unpack16<T_BF16>(u.x, f.x, f.y);
                unpack16<T_BF16>(u.y, f.z, f.w);
            }
            return f;
        }
        auto at = [&](int e) { return col + e < p.N ? load_any(p.residual, p.type, row * p.res_rs + (col + e) * p.res_cs) : 0.f; };
        return make_float4(at(0), at(1), at(2), at(3));
    }
    __device__ __forceinline__ void put(const ActParams& p, void* to, bool tma, long long rs, long long cs, long long row,
                                        const float (&v)[4]) const {
        if (tma && whole) {
            if (p.type == T_F32)
                *reinterpret_cast<float4*>(static_cast<float*>(to) + row * rs + col) = make_float4(v[0], v[1], v[2], v[3]);
            else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(to) + row * rs + col) =
                    make_uint2(pack16(v[0], v[1], p.type == T_BF16), pack16(v[2], v[3], p.type == T_BF16));
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < p.N) store_any(to, p.type, row * rs + (col + e) * cs, v[e]);
    }
    __device__ __forceinline__ void finish(const ActParams& p, const DropKey& key, long long row, float (&v)[4], const float4& res) const {
        if (!live || row >= p.M) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += bias[e];
        if (p.z) put(p, p.z, p.z_tma, p.z_rs, p.z_cs, row, v);
        apply_act(v, p.act);
        if (p.drop.least) {
            uint32_t w[4];
            philox8(key, static_cast<uint32_t>(col) >> 3, static_cast<uint32_t>(row), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t pair = (col & 4) ? w[2 + e / 2] : w[e / 2];
                v[e] = ((e & 1) ? pair : pair << 16) > p.drop.limit ? v[e] * p.drop.scale : 0.f;
            }
        }
        v[0] += res.x;
        v[1] += res.y;
        v[2] += res.z;
        v[3] += res.w;
        put(p, p.out, p.out_tma, p.out_rs, p.out_cs, row, v);
    }
};

template <int CG, int BN>
struct Geo {
    static constexpr int COLS = BN / 2;                // accumulator columns of an epilogue warp
    static constexpr int B_ROWS = BN / CG;             // B's columns in a CTA's shared memory
    static constexpr uint32_t A_BYTES = ROWS * 128, B_BYTES = B_ROWS * 128, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = B_ROWS == 128 ? 5 : 6;
    static constexpr int TMEM_COLS = 512, ACCS = TMEM_COLS / BN;
    static constexpr uint32_t BOX_BYTES = 32 * 128, OUT_BYTES = 2 * BOX_BYTES;  // staging of an epilogue warp
    static constexpr uint32_t TILES_BYTES = STAGES * STAGE_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 2 * 8 + 2 * 8 + 1;
    static constexpr uint32_t BYTES = 1024 + TILES_BYTES + 8 * OUT_BYTES + NUM_BARS * 8 + 16;
    static constexpr int THREADS = 384;
    static constexpr int REGS_CTL = 40, REGS_EPI = 232;  // of 168 a thread at launch
    static constexpr int REGS_TOTAL = 128 * REGS_CTL + 256 * REGS_EPI;
    static_assert(REGS_TOTAL <= THREADS * 168, "register split");
    static_assert(BYTES <= 232448, "shared memory");
};

template <int CG, int BN>
struct Smem {
    using G = Geo<CG, BN>;
    uint8_t* base;
    // barriers per stage: full, done (its MMAs have run); per accumulator: full,
    // empty; per epilogue warp: its two boxes' residuals have landed, every
    // part's sums lie in shared memory, every part has read this CTA's
    uint32_t tiles, full, done, acc_full, acc_empty, res_full, parts_in, parts_out, final_bar;
    uint32_t *tmem_slot, *epoch_slot;
    __device__ void carve(uint8_t* p) {
        base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
        tiles = smem_u32(base);
        full = tiles + G::TILES_BYTES + 8 * G::OUT_BYTES;
        done = full + 8 * G::STAGES;
        acc_full = done + 8 * G::STAGES;
        acc_empty = acc_full + 8 * G::ACCS;
        res_full = acc_empty + 8 * G::ACCS;
        parts_in = res_full + 128;
        parts_out = parts_in + 64;
        final_bar = parts_out + 64;
        tmem_slot = reinterpret_cast<uint32_t*>(base + (final_bar + 8 - tiles));
        epoch_slot = tmem_slot + 1;
    }
    __device__ __forceinline__ uint32_t a(uint32_t s) const { return tiles + s * G::STAGE_BYTES; }
    __device__ __forceinline__ uint32_t b(uint32_t s) const { return tiles + s * G::STAGE_BYTES + G::A_BYTES; }
    __device__ __forceinline__ uint8_t* out(int w) const { return base + G::TILES_BYTES + w * G::OUT_BYTES; }
};

struct Unit {
    int mb, nb, lo, hi;  // tile and this CTA's stages of it
    int tail, part;      // pairs: index of a tail tile and the part of it, or -1
};
// first stage of a part of the contraction; parts differ by one stage at most
__device__ __forceinline__ int part_start(const ActParams& p, int part) {
    return static_cast<int>(static_cast<long long>(p.stages_total) * part / p.split);
}
// Tiles in groups of group_m rows of tiles, so that the tiles running at once
// share their operands in L2.  The tiles of a last round that would leave half of
// the pairs idle or more are cut into parts of the contraction.
template <int CG>
__device__ __forceinline__ Unit unit_of(const ActParams& p, const Ctl& ctl, int u) {
    Unit x;
    x.tail = x.part = -1;
    if (CG == 2 && u >= p.tail_first) {  // all first parts before all second ones
        x.part = (u - p.tail_first) / p.tail_tiles;
        x.tail = u - p.tail_first - x.part * p.tail_tiles;
        u = p.tail_first + x.tail;
    }
    const int per = p.group_m * p.n_blocks;
    const int g = u / per, first = g * p.group_m;
    const int rows = min(p.group_m, p.m_blocks - first), in = u - g * per;
    x.mb = first + in % rows;
    x.nb = in / rows;
    x.lo = CG == 1 ? part_start(p, ctl.rank) : 0;
    x.hi = CG == 1 ? part_start(p, ctl.rank + 1) : p.stages_total;
    if (CG == 2 && x.tail >= 0) {
        x.lo = p.stages_total * x.part / p.tail_parts;
        x.hi = p.stages_total * (x.part + 1) / p.tail_parts;
    }
    return x;
}
template <int CG>
__device__ __forceinline__ int half(const Ctl& ctl) {
    return CG == 2 ? ctl.rank : 0;
}

// One operand's box or boxes of a stage: `n` of its rows from `row` on.
template <int CG>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* m, int mn, int row, int n, int d, uint32_t bar) {
    if (mn == 2) {
        CG == 1 ? tma_load_3d(dst, m, 0, d, row / 64, bar) : tma_load_3d_pair(dst, m, 0, d, row / 64, bar);
        return;
    }
    if (!mn) {
        CG == 1 ? tma_load_2d(dst, m, d, row, bar) : tma_load_2d_pair(dst, m, d, row, bar);
        return;
    }
    for (int c = 0; c < n; c += 64, dst += 8192)
        CG == 1 ? tma_load_2d(dst, m, row + c, d, bar) : tma_load_2d_pair(dst, m, row + c, d, bar);
}

// The odd CTA's pair loads count on the even CTA's barrier, so to know that they
// have landed it waits until the MMA has read its last fill.
template <int CG, int BN>
__device__ void run_tma(const ActParams& p, const Ctl& ctl, Smem<CG, BN>& sm, int first, int step) {
    using G = Geo<CG, BN>;
    Ring<G::STAGES> st;
    Fills fills;
    bool ok = true;
    for (int u = first; u < p.n_units && ok; u += step) {
        const Unit x = unit_of<CG>(p, ctl, u);
        const int row = (x.mb * CG + half<CG>(ctl)) * ROWS;
        const int col = x.nb * BN + half<CG>(ctl) * G::B_ROWS;
        for (int s = x.lo; s < x.hi; ++s) {
            if (!wait_bar(ctl, sm.done + 8 * st.slot, st.phase ^ 1, WAIT_EMPTY)) {
                ok = false;
                break;
            }
            if (half<CG>(ctl) == 0) bar_expect_tx(sm.full + 8 * st.slot, CG * G::STAGE_BYTES);
            const uint32_t bar = CG == 1 ? sm.full + 8 * st.slot : map_to(sm.full + 8 * st.slot, 0);
            load_operand<CG>(sm.a(st.slot), &p.tmA, p.a_mn, row, ROWS, s * DEPTH, bar);
            load_operand<CG>(sm.b(st.slot), &p.tmB, p.b_mn, col, G::B_ROWS, s * DEPTH, bar);
            fills.add(st.slot, st.phase);
            st.next();
        }
    }
    fills.drain(ctl, half<CG>(ctl) ? sm.done : sm.full, G::STAGES);
}

// MMAs.  The whole warp runs the loop, so that addresses and descriptors stay in
// uniform registers; one elected lane issues.
template <int CG, int BN>
__device__ void run_mma(const ActParams& p, const Ctl& ctl, Smem<CG, BN>& sm, uint32_t tmem, int first, int step) {
    using G = Geo<CG, BN>;
    // K-major: 8-row groups 1024 bytes apart (stride offset), a K step of 16 is 32
    // bytes further along the swizzled rows.  MN-major: rows of 128 bytes per
    // contraction index, 8-deep groups 1024 bytes apart (stride offset), blocks of
    // 64 rows 8192 bytes apart (leading offset), a K step is 16 rows of 128 bytes.
    const uint32_t a_adv = p.a_mn ? 128 : 2, b_adv = p.b_mn ? 128 : 2;
    const uint64_t a_desc = smem_desc(sm.a(0), p.a_mn ? 8192 : 16, 1024), b_desc = smem_desc(sm.b(0), p.b_mn ? 8192 : 16, 1024);
    const uint32_t idesc = p.idesc;
    Ring<G::STAGES> st;
    Ring<G::ACCS> acc;
    bool ok = true;
    for (int u = first; u < p.n_units && ok; u += step, acc.next()) {
        const Unit x = unit_of<CG>(p, ctl, u);
        if (x.lo == x.hi) break;  // a part without stages has none in any tile
        const bool report = p.debug_skip != static_cast<uint32_t>(u) + 1;
        if (!wait_bar(ctl, sm.acc_empty + 8 * acc.slot, acc.phase ^ 1, WAIT_ACC_EMPTY)) break;
        const uint32_t d = tmem + acc.slot * BN;
        for (int s = x.lo; s < x.hi; ++s, st.next()) {
            if (!wait_bar(ctl, sm.full + 8 * st.slot, st.phase, WAIT_FULL)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t at = st.slot * (G::STAGE_BYTES / 16);
            const uint32_t more = s > x.lo ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < DEPTH / 16; ++k)
                    umma_f16<CG>(d, a_desc + at + k * a_adv, b_desc + at + k * b_adv, idesc, k > 0 ? 1u : more);
                umma_commit_all<CG>(sm.done + 8 * st.slot);
                if (s == x.hi - 1 && report) umma_commit_all<CG>(sm.acc_full + 8 * acc.slot);
            }
            __syncwarp();
        }
    }
    if (elect_one()) umma_commit_one<CG>(sm.final_bar);
    __syncwarp();
    wait_bar(ctl, sm.final_bar, 0, WAIT_DRAIN_MMA);
}

// An epilogue warp: 32 rows x COLS columns of each tile, 32 columns at a time
// from tensor memory through two boxes of 32 rows x 128 bytes in shared memory
// (128-byte swizzle).  The residual is loaded into the box that its sum is
// stored from; with z, box 0 is z's and box 1 out's.
template <int CG, int BN>
struct Epilogue {
    using G = Geo<CG, BN>;
    const ActParams& p;
    const Ctl& ctl;
    Smem<CG, BN>& sm;
    const uint32_t tmem;
    const int w, lane, q, h;
    uint8_t* const stg;
    const DropKey key;
    Ring<G::ACCS> from;
    uint32_t uses = 0, joins = 0, phases = 0, pending = 0;  // boxes used; joins; residual barriers' phases; loads under way
    int row0 = 0, col0 = 0;

    __device__ __forceinline__ Epilogue(const ActParams& p_, const Ctl& c_, Smem<CG, BN>& s_, uint32_t t_, int w_, int lane_)
        : p(p_), ctl(c_), sm(s_), tmem(t_), w(w_), lane(lane_), q(w_ & 3), h(w_ >> 2), stg(s_.out(w_)), key(drop_key(p_.drop)) {}

    __device__ __forceinline__ uint8_t* box(uint32_t use) const { return stg + (use & 1) * G::BOX_BYTES; }
    // where 16-byte unit j of this lane's row lies in a box
    __device__ __forceinline__ uint32_t unit_at(int j) const { return lane * 128 + ((j ^ (lane & 7)) << 4); }

    // before a box is used anew: at most N of this warp's newer stores still read
    template <int N>
    __device__ __forceinline__ void box_free() {
        if (lane == 0) bulk_wait_read<N>();
        __syncwarp();
    }
    // residual columns from `col` on into a free box; lanes that cannot use the
    // tensor memory accelerator copy elements
    template <typename E>
    __device__ __forceinline__ void copy_in(uint8_t* b, int col) const {
        constexpr int PER = 128 / (32 * sizeof(E));
        const E* at = static_cast<const E*>(p.residual) + row0 * p.res_rs + (col + lane) * p.res_cs;
        const int rows = min(32, p.M - row0);
#pragma unroll 4
        for (int r = 0; r < rows; ++r, at += p.res_rs) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int o = (lane + 32 * e) * static_cast<int>(sizeof(E));
                if (col + lane + 32 * e < p.N)
                    *reinterpret_cast<E*>(b + r * 128 + (((o >> 4) ^ (r & 7)) << 4) + (o & 15)) = at[32 * e * p.res_cs];
            }
        }
    }
    __device__ __forceinline__ void fetch(uint32_t use, int col) {
        uint8_t* const b = box(use);
        if (!p.res_tma) {
            p.type == T_F32 ? copy_in<float>(b, col) : copy_in<uint16_t>(b, col);
            __syncwarp();
            return;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            const uint32_t bar = sm.res_full + (w * 2 + (use & 1)) * 8;
            bar_expect_tx(bar, G::BOX_BYTES);
            tma_load_2d(smem_u32(b), &p.tmR, col, row0, bar);
        }
        pending |= 1u << (use & 1);
    }
    __device__ __forceinline__ bool landed(uint32_t use, int where) {
        const uint32_t bit = 1u << (use & 1);
        if (!(pending & bit)) return true;
        if (!wait_bar(ctl, sm.res_full + (w * 2 + (use & 1)) * 8, (phases & bit) ? 1u : 0u, where)) return false;
        __syncwarp();
        phases ^= bit;
        pending ^= bit;
        return true;
    }
    // 32 columns of this lane's row: columns 32 .. 63 of a 16-bit box for c odd
    __device__ __forceinline__ void add_in(const uint8_t* b, int c, float (&v)[32]) const {
        if (p.type == T_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 f = *reinterpret_cast<const float4*>(b + unit_at(j));
                v[4 * j] += f.x;
                v[4 * j + 1] += f.y;
                v[4 * j + 2] += f.z;
                v[4 * j + 3] += f.w;
            }
            return;
        }
        const bool bf = p.type == T_BF16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 u = *reinterpret_cast<const uint4*>(b + unit_at(j + (c & 1) * 4));
            const uint32_t words[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo, hi;
                if (bf)
                    unpack16<T_BF16>(words[e], lo, hi);
                else
                    unpack16<T_F16>(words[e], lo, hi);
                v[8 * j + 2 * e] += lo;
                v[8 * j + 2 * e + 1] += hi;
            }
        }
    }
    __device__ __forceinline__ void lay(uint8_t* b, int c, const float (&v)[32]) const {
        if (p.type == T_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4*>(b + unit_at(j)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            return;
        }
        const int bf = p.type == T_BF16;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(b + unit_at(j + (c & 1) * 4)) =
                make_uint4(pack16(v[8 * j], v[8 * j + 1], bf), pack16(v[8 * j + 2], v[8 * j + 3], bf),
                           pack16(v[8 * j + 4], v[8 * j + 5], bf), pack16(v[8 * j + 6], v[8 * j + 7], bf));
    }
    // any strides: a lane per column
    template <typename E>
    __device__ __forceinline__ void copy_out(const uint8_t* b, void* dst, long long rs, long long cs, int col) const {
        constexpr int PER = 128 / (32 * sizeof(E));
        E* to = static_cast<E*>(dst) + row0 * rs + (col + lane) * cs;
        const int rows = min(32, p.M - row0);
#pragma unroll 4
        for (int r = 0; r < rows; ++r, to += rs) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int o = (lane + 32 * e) * static_cast<int>(sizeof(E));
                if (col + lane + 32 * e < p.N)
                    to[32 * e * cs] = *reinterpret_cast<const E*>(b + r * 128 + (((o >> 4) ^ (r & 7)) << 4) + (o & 15));
            }
        }
    }
    // a box goes out, as one bulk group
    __device__ __forceinline__ void send(uint8_t* b, const CUtensorMap* map, bool tma, void* dst, long long rs, long long cs,
                                         int col) {
        if (tma) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) tma_store_2d(map, b, col, row0);
        } else {
            __syncwarp();
            p.type == T_F32 ? copy_out<float>(b, dst, rs, cs, col) : copy_out<uint16_t>(b, dst, rs, cs, col);
            __syncwarp();
        }
        if (lane == 0) bulk_commit();
    }

    __device__ __forceinline__ void hand_back() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (CG == 2)
                mbar_arrive_remote(map_to(sm.acc_empty + 8 * from.slot, 0));
            else
                bar_arrive(sm.acc_empty + 8 * from.slot);
        }
        from.next();
    }
    __device__ __forceinline__ uint32_t acc_at(int c) const {
        return tmem + (static_cast<uint32_t>(q * 32) << 16) + from.slot * BN + h * G::COLS + c * 32;
    }
    __device__ __forceinline__ bool acc_ready() {
        if (!wait_bar(ctl, sm.acc_full + 8 * from.slot, from.phase, WAIT_ACC_FULL)) return false;
        __syncwarp();  // tensor-memory loads are for the converged warp
        tc_fence_after();
        return true;
    }

    // where the sums of a part of a tail tile lie, of this warp
    __device__ __forceinline__ int tail_slot(int tail, int part) const {
        return ((part * p.tail_tiles + tail) * 2 + ctl.rank) * 8 + w;
    }
    __device__ __forceinline__ unsigned long long tail_ready() const {
        return static_cast<unsigned long long>(ctl.epoch) << 32 | 0x7A115C0Du;
    }
    // All parts but the last leave their sums in global memory, for the same warp of
    // the last one's pair, which runs them in the order of the parts.
    __device__ __forceinline__ bool leave(const Unit& x) {
        if (!acc_ready()) return false;
        const int slot = tail_slot(x.tail, x.part);
        float4* at = reinterpret_cast<float4*>(p.tail_sums + static_cast<size_t>(slot) * (G::COLS * 32)) + lane;
#pragma unroll 1
        for (int c = 0; c < G::COLS / 32; ++c) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(acc_at(c), r);
            tmem_wait_regs(r);
            if (c == G::COLS / 32 - 1) hand_back();
#pragma unroll
            for (int j = 0; j < 8; ++j, at += 32)
                *at = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) st_release_gpu_u64(p.tail_flags + slot, tail_ready());
        return true;
    }
    __device__ __forceinline__ bool tail_there(int tail) {
        for (int part = 0; part < p.tail_parts - 1; ++part) {
            const unsigned long long* flag = p.tail_flags + tail_slot(tail, part);
            const uint64_t t0 = global_timer_ns();
            while (ld_acquire_gpu_u64(flag) != tail_ready()) {
                __nanosleep(100);
                if (launch_aborted(ctl)) return false;
                if (global_timer_ns() - t0 > ctl.limit) {
                    raise_timeout(ctl, WAIT_TAIL, tail);
                    return false;
                }
            }
        }
        __syncwarp();
        return true;
    }

    __device__ __forceinline__ bool whole(int tail) {
        const bool wide = p.type == T_F32;
        const int per = wide ? 1 : 2;  // 32-column groups of a box
        const int boxes = min(G::COLS / 32 / per, (p.N - col0 + 32 * per - 1) / (32 * per));
        const uint32_t stride = p.z ? 2 : 1, first = uses + stride - 1;  // the first box of out
        if (p.residual) {
            p.z ? box_free<0>() : box_free<1>();
            fetch(first, col0);
            if (!p.z && boxes > 1) {
                box_free<0>();
                fetch(first + 1, col0 + 32 * per);
            }
        }
        if (!acc_ready()) return false;
        if (CG == 2 && tail >= 0 && !tail_there(tail)) return false;
        const int groups = boxes * per;
#pragma unroll 1
        for (int c = 0; c < groups; ++c) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(acc_at(c), r);
            const int col = col0 + c * 32;
            const bool near = p.bias_near && col + 32 <= p.N;
            const float b = near ? 0.f : bias_at(p, col + lane);
            uint4 near_bias[4];  // the same for all lanes; 16-bit
            if (near) {
#pragma unroll
                for (int j = 0; j < 4; ++j) near_bias[j] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + col)[j];
            }
            tmem_wait_regs(r);
            if (c == groups - 1) hand_back();
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            if (CG == 2 && tail >= 0) {
                float sum[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] = 0.f;
#pragma unroll 1
                for (int part = 0; part < p.tail_parts - 1; ++part) {
                    const float4* at = reinterpret_cast<const float4*>(p.tail_sums + static_cast<size_t>(tail_slot(tail, part)) * (G::COLS * 32)) + c * 256 + lane;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 f = __ldcg(at + j * 32);
                        sum[4 * j] += f.x;
                        sum[4 * j + 1] += f.y;
                        sum[4 * j + 2] += f.z;
                        sum[4 * j + 3] += f.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += sum[i];
            }
            if (near) {
                const bool bf = p.bias_type == T_BF16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t words[4] = {near_bias[j].x, near_bias[j].y, near_bias[j].z, near_bias[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float lo, hi;
                        if (bf)
                            unpack16<T_BF16>(words[e], lo, hi);
                        else
                            unpack16<T_F16>(words[e], lo, hi);
                        v[8 * j + 2 * e] += lo;
                        v[8 * j + 2 * e + 1] += hi;
                    }
                }
            } else if (p.bias) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, b, i);
            }
            const bool begins = wide || (c & 1) == 0, ends = wide || (c & 1) == 1;
            const int box_col = ends && !wide ? col - 32 : col;
            if (p.z) {
                if (begins) box_free<1>();
                lay(box(uses), c, v);
                if (ends) send(box(uses), &p.tmZ, p.z_tma, p.z, p.z_rs, p.z_cs, box_col);
            }
            apply_act(v, p.act);
            if (p.drop.least) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    drop8(v + 8 * j, p.drop, key, static_cast<uint32_t>(col) / 8 + j, static_cast<uint32_t>(row0 + lane));
            }
            const uint32_t use = uses + stride - 1;
            if (begins) {
                // z's box of these columns has not gone out yet, so the newest store is this box's
                if (!p.residual)
                    p.z ? box_free<0>() : box_free<1>();
                else if (!landed(use, WAIT_RESIDUAL))
                    return false;
            }
            if (p.residual) add_in(box(use), c, v);
            lay(box(use), c, v);
            if (ends) {
                send(box(use), &p.tmC, p.out_tma, p.out, p.out_rs, p.out_cs, box_col);
                uses += stride;
                // the next residual that no box was free for
                const int next = c / per + (p.z ? 1 : 2);
                if (p.residual && next < boxes) {
                    box_free<0>();
                    fetch(use + 2, col0 + next * 32 * per);
                }
            }
        }
        return true;
    }

    // Split contraction over S CTAs: each warp lays its 32 x 64 sums into its
    // boxes (rows of units of 16 bytes, XORed with the row), tells the same warp of
    // every part, and adds its part's rows of them over all parts in order.  The
    // loads from the other CTAs are all under way at once; neighbouring lanes hold
    // neighbouring columns of a row, so stores reach few rows each.
    template <int S>
    __device__ __forceinline__ bool join(bool more) {
        constexpr int UNITS = 16, SHARE = UNITS / S;
        static_assert(UNITS * 512 <= G::OUT_BYTES || CG == 2, "a warp's sums fit its boxes");
        const bool empty = part_start(p, ctl.rank) == part_start(p, ctl.rank + 1);  // adds zeros
        const int unit = lane % UNITS;
        auto share_row = [&](int i) { return ctl.rank * (32 / S) + i * (32 / UNITS) + lane / UNITS; };
        const Four four(p, col0 + unit * 4);
        float4 res[SHARE];
#pragma unroll
        for (int i = 0; i < SHARE; ++i) res[i] = four.residual(p, row0 + share_row(i));
        if (!empty && !acc_ready()) return false;
        // the other parts have read what lay here before
        if (joins > 0 && !wait_bar_cluster(ctl, sm.parts_out + 8 * w, (joins - 1) & 1, WAIT_PARTS)) return false;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
            if (!empty) {
                tmem_ld_32x32b_x32(acc_at(c), r);
                tmem_wait_regs(r);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(stg + lane * UNITS * 16 + (((c * 8 + j) ^ (lane & (UNITS - 1))) << 4)) =
                    make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        }
        if (!empty) hand_back();
        __syncwarp();
        if (lane < S) mbar_arrive_cluster(map_to(sm.parts_in + 8 * w, lane));
        if (!wait_bar_cluster(ctl, sm.parts_in + 8 * w, joins & 1, WAIT_PARTS)) return false;
        __syncwarp();
        ++joins;
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
            float v[4] = {t[i][0].x, t[i][0].y, t[i][0].z, t[i][0].w};
#pragma unroll
            for (int k = 1; k < S; ++k) {
                v[0] += t[i][k].x;
                v[1] += t[i][k].y;
                v[2] += t[i][k].z;
                v[3] += t[i][k].w;
            }
            four.finish(p, key, row0 + share_row(i), v, res[i]);
        }
        // the values above are in registers: the parts may lay their next sums, if
        // there are any: a CTA on its way out gets no more arrivals
        __syncwarp();
        if (more && lane < S) mbar_arrive_cluster(map_to(sm.parts_out + 8 * w, lane));
        return true;
    }

    __device__ __forceinline__ void run(int first, int step) {
        for (int u = first; u < p.n_units; u += step) {
            const Unit x = unit_of<CG>(p, ctl, u);
            row0 = (x.mb * CG + half<CG>(ctl)) * ROWS + q * 32;
            col0 = x.nb * BN + h * G::COLS;
            if (row0 >= p.M || col0 >= p.N) {  // keeps step; not live in one part: not live in any
                if (x.lo == x.hi) continue;
                if (!acc_ready()) break;
                hand_back();
                continue;
            }
            if constexpr (CG == 1) {
                if (p.split > 1) {
                    const bool more = u + step < p.n_units;
                    if (!(p.split == 2 ? join<2>(more) : p.split == 4 ? join<4>(more) : join<8>(more))) break;
                    continue;
                }
            }
            if (CG == 2 && x.tail >= 0 && x.part < p.tail_parts - 1 ? !leave(x) : !whole(x.tail)) break;
        }
        for (uint32_t s = 0; s < 2; ++s) landed(s, WAIT_DRAIN_TMA);  // where the launch stopped
        if (lane == 0) bulk_wait_all();  // its stores have left shared memory
        __syncwarp();
    }
};

template <int CG, int BN>
__global__ void __launch_bounds__(Geo<CG, BN>::THREADS, 1) act_gemm_kernel(const __grid_constant__ ActParams p) {
    using G = Geo<CG, BN>;
    extern __shared__ uint8_t smem_raw[];
    Smem<CG, BN> sm;
    sm.carve(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int csize = CG == 2 ? 2 : p.split;  // CTAs per cluster
    const int rank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            bar_init(sm.full + 8 * s, 1);
            bar_init(sm.done + 8 * s, 1);
        }
        for (int b = 0; b < G::ACCS; ++b) {
            bar_init(sm.acc_full + 8 * b, 1);
            bar_init(sm.acc_empty + 8 * b, CG * 8);
        }
        for (int i = 0; i < 8; ++i) {
            bar_init(sm.res_full + 16 * i, 1);
            bar_init(sm.res_full + 16 * i + 8, 1);
            bar_init(sm.parts_in + 8 * i, csize);
            bar_init(sm.parts_out + 8 * i, csize);
        }
        bar_init(sm.final_bar, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        // for the whole CTA, which waits for this thread below
        grid_wait();
        grid_release();
        const uint32_t e = *reinterpret_cast<volatile uint32_t*>(&p.ws->epoch) + 1u;
        *sm.epoch_slot = e == 0u ? 1u : e;
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
            if (lane == 0) run_tma<CG, BN>(p, ctl, sm, first, step);
        } else if (warp == 1) {
            if (CG == 1 || rank == 0) run_mma<CG, BN>(p, ctl, sm, tmem, first, step);
        }
        __syncwarp();
    } else {
        reg_inc<G::REGS_EPI>();
        Epilogue<CG, BN>(p, ctl, sm, tmem, warp - 4, lane).run(first, step);
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

// An empty contraction: the sums are zero.
template <int DUMMY>
__global__ void __launch_bounds__(256) act_fill_kernel(const __grid_constant__ ActParams p) {
    grid_wait();
    grid_release();
    const DropKey key = drop_key(p.drop);
    const long long groups = (p.N + 3) / 4, n = p.M * groups;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        const Four four(p, static_cast<int>(i % groups) * 4);
        four.finish(p, key, i / groups, v, four.residual(p, i / groups));
    }
}

}  // namespace block
}  // namespace gct
