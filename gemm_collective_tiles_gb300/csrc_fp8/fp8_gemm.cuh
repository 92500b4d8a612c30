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
// varies along the contraction, so four converter warps turn codes into
// scaled 16-bit operands on their way from shared memory to the MMA (exact
// for power-of-two scales: a code has at most 4 significant bits), and a chunk
// is WG_CHUNK stages long, which bounds the length of the sums that the tensor
// cores keep by themselves.
//
// CTA layout, one CTA per SM:
//   warp 0       TMA producer (lane 0)
//   warp 1       MMA issuer (lane 0); owns tensor memory
//   warps 2, 3   none: they make the first warpgroup whole, which gives its
//                registers to the promotion warps
//   warps 4-11   promotion and epilogue: quadrant warp % 4 of the accumulator's
//                rows, column half (warp - 4) / 4
//   warps 12-15  KIND_WG: converters
// CG = 2: a cluster of two CTAs computes a 256 x 256 tile with
// tcgen05.mma.cta_group::2, each staging its 128 rows of A and 128 columns of
// B; the even CTA issues the MMAs.  CG = 1: 128 x 128 tiles, for few rows.
//
// Work units (tile, part of the contraction) are dealt out in a fixed order;
// with more than one part, the parts' fp32 sums go to the workspace and the
// last CTA to arrive adds them in part order, so results do not depend on
// timing.  Every wait is bounded: one that gives up records where in the
// workspace header, stops the launch, and the roles drain and leave.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_ptx.cuh"
#include "fp8_quant.cuh"

namespace gct {
namespace fp8 {

enum : int { KIND_MM = 0, KIND_WG = 1 };
constexpr int BM = 128;         // rows per CTA (tensor-memory lanes)
constexpr int WG_CHUNK = 8;     // KIND_WG: 64-deep stages per chunk
constexpr int MAX_SPLIT_SLOTS = 1024;  // (tile, CTA half) arrival counters in the workspace
constexpr int DEV_TIMEOUT = 1;

// where-codes recorded when a bounded wait gives up
enum : int {
    WAIT_EMPTY = 101,
    WAIT_FULL = 102,
    WAIT_CONVERTED = 103,
    WAIT_ACC_EMPTY = 104,
    WAIT_ACC_FULL = 105,
    WAIT_RAW = 106,
    WAIT_SYNC = 107,
    WAIT_DRAIN_TMA = 108,
    WAIT_DRAIN_MMA = 109,
};

// The library's workspace header (same layout for every op).
struct WsHeader {
    uint32_t epoch;        // epoch of the last completed launch
    uint32_t ctr[2];       // queue heads of other ops; zero between launches
    uint32_t done_ctr;     // CTAs finished in this launch
    int status;            // sticky first device error (0 = none)
    uint32_t abort_epoch;  // == current epoch while the launch is stopping
    int err_where;
    int err_index;
    uint32_t pad[56];
};
static_assert(sizeof(WsHeader) == 256, "workspace header is 256 bytes");

struct GemmParams {
    CUtensorMap tmA;  // MM: codes {k, row}, box {128, a_box}; WG: codes {k, m}, box {128, 64}, no swizzle
    CUtensorMap tmB;  // MM: codes {k, n} or {n, k}, box {128, 128}; WG: dY {n, m}, box {64, 64}
    CUtensorMap tmC;  // out or the parts' sums: {n, row, part}, box {128 bytes, 32, 1}
    int M, N;         // output rows and columns
    int D;            // contraction length
    int stages_total, part_stages, split;  // contraction in stages; stages per part; parts
    int m_blocks, n_blocks, group_m, n_units;
    int b_mn;         // MM: B has its columns contiguous
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
    unsigned long long* arrived;  // MAX_SPLIT_SLOTS epoch-tagged counters
    float* partial;               // split parts: [part][row][pitch]
    long long part_rs, part_stride;
    int staged;                   // the epilogue stores parts (or one fp32 copy) to `partial`
    unsigned long long wait_ns;
    uint32_t debug_skip;          // test hook: k > 0: unit k - 1 never reports its accumulator
};

struct Ctl {
    WsHeader* ws;
    uint32_t epoch;
    unsigned long long limit;
    int half;
};

__device__ __forceinline__ bool launch_aborted(const Ctl& c) {
    return *reinterpret_cast<volatile uint32_t*>(&c.ws->abort_epoch) == c.epoch;
}
__device__ __forceinline__ void raise_timeout(const Ctl& c, int where, int index) {
    if (atomicCAS(&c.ws->status, 0, DEV_TIMEOUT) == 0) {
        c.ws->err_where = where;
        c.ws->err_index = index;
    }
    __threadfence();
    atomicExch(&c.ws->abort_epoch, c.epoch);
}
__device__ __forceinline__ bool wait_bar(const Ctl& c, uint64_t* bar, uint32_t parity, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 0) {
            if (launch_aborted(c)) return false;
            if (global_timer_ns() - t0 > c.limit) {
                raise_timeout(c, where, -1);
                return false;
            }
        }
    }
}
// teardown: waits for asynchronous work already issued, also while stopping
__device__ __forceinline__ bool drain_bar(const Ctl& c, uint64_t* bar, uint32_t parity, int where) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > c.limit) {
            raise_timeout(c, where, -1);
            return false;
        }
    }
    return true;
}
// arrival count within this launch; a counter left by another launch restarts
__device__ __forceinline__ uint32_t arrive_count(unsigned long long* ctr, uint32_t epoch) {
    unsigned long long cur = *reinterpret_cast<volatile unsigned long long*>(ctr);
    while (true) {
        const unsigned long long want = (static_cast<uint32_t>(cur >> 32) == epoch)
                                            ? cur + 1
                                            : ((static_cast<unsigned long long>(epoch) << 32) | 1ull);
        const unsigned long long prev = atomicCAS(ctr, cur, want);
        if (prev == cur) return static_cast<uint32_t>(want);
        cur = prev;
    }
}

template <int KIND, int CG>
struct Geo {
    static constexpr int BN = CG == 2 ? 256 : 128;     // tile columns (of the pair)
    static constexpr int COLS = BN / 2;                // accumulator columns of a promotion warp
    static constexpr int DEPTH = KIND == KIND_MM ? 128 : 64;  // contraction per stage
    static constexpr int UMMA_STEPS = 4;               // 128 / 32 or 64 / 16
    static constexpr uint32_t A_BYTES = BM * 128;      // 128 rows x 128 bytes of contraction
    static constexpr uint32_t B_BYTES = (BN / CG) * 128;
    static constexpr uint32_t RAW_BYTES = KIND == KIND_WG ? 64 * 128 : 0;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + RAW_BYTES;
    static constexpr int STAGES = KIND == KIND_MM ? 6 : 4;
    static constexpr int THREADS = KIND == KIND_MM ? 384 : 512;
    static constexpr uint32_t OUT_BYTES = 32 * 128;    // staging per promotion warp
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int NUM_BARS = 4 * STAGES + 4 + 2;
    static constexpr uint32_t BYTES = 1024 + STAGES * STAGE_BYTES + 8 * OUT_BYTES + NUM_BARS * 8 + 32;
    // registers: the launch's total (168 or 128 a thread) is shared out anew
    static constexpr int REGS_CTL = KIND == KIND_MM ? 56 : 40;
    static constexpr int REGS_CONV = 96;
    static constexpr int REGS_PROMOTE = KIND == KIND_MM ? 224 : 184;
};
static_assert(128 * Geo<KIND_MM, 2>::REGS_CTL + 256 * Geo<KIND_MM, 2>::REGS_PROMOTE <= 384 * 168, "register split");
static_assert(128 * (Geo<KIND_WG, 2>::REGS_CTL + Geo<KIND_WG, 2>::REGS_CONV) + 256 * Geo<KIND_WG, 2>::REGS_PROMOTE <= 512 * 128,
              "register split");

template <int KIND, int CG>
struct Smem {
    using G = Geo<KIND, CG>;
    uint8_t *tiles, *out;
    uint64_t *full, *empty, *raw, *conv, *acc_full, *acc_empty, *sync, *final_bar;
    uint32_t *tmem_slot, *epoch_slot, *last;
    __device__ void carve(uint8_t* p) {
        tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
        out = tiles + G::STAGES * G::STAGE_BYTES;
        full = reinterpret_cast<uint64_t*>(out + 8 * G::OUT_BYTES);
        empty = full + G::STAGES;
        raw = empty + G::STAGES;
        conv = raw + G::STAGES;
        acc_full = conv + G::STAGES;
        acc_empty = acc_full + 2;
        sync = acc_empty + 2;
        final_bar = sync + 1;
        tmem_slot = reinterpret_cast<uint32_t*>(final_bar + 1);
        epoch_slot = tmem_slot + 1;
        last = tmem_slot + 2;
    }
    __device__ uint8_t* a(uint32_t s) const { return tiles + s * G::STAGE_BYTES; }
    __device__ uint8_t* b(uint32_t s) const { return tiles + s * G::STAGE_BYTES + G::A_BYTES; }
    __device__ uint8_t* raw_tile(uint32_t s) const { return tiles + s * G::STAGE_BYTES + G::A_BYTES + G::B_BYTES; }
};

struct Unit {
    int mb, nb, part, lo, hi;  // tile, part, its stages
};
// Tiles in groups of group_m rows of tiles, so the tiles running at once share
// their operands in L2; a tile's parts follow one another.
__device__ __forceinline__ Unit unit_of(const GemmParams& p, int u) {
    Unit x;
    const int t = u / p.split;
    x.part = u - t * p.split;
    const int per = p.group_m * p.n_blocks;
    const int g = t / per, first = g * p.group_m;
    const int rows = min(p.group_m, p.m_blocks - first), in = t - g * per;
    x.mb = first + in % rows;
    x.nb = in / rows;
    x.lo = x.part * p.part_stages;
    x.hi = min(p.stages_total, x.lo + p.part_stages);
    return x;
}

template <int KIND, int CG>
__device__ void run_tma(const GemmParams& p, const Ctl& ctl, Smem<KIND, CG>& sm, int first, int step) {
    using G = Geo<KIND, CG>;
    // bit s of `filled`: the phase of stage s's last fill
    uint32_t stage = 0, phase = 0, used = 0, filled = 0;
    bool ok = true;
    for (int u = first; u < p.n_units && ok; u += step) {
        const Unit x = unit_of(p, u);
        const int row = (x.mb * CG + ctl.half) * BM;
        const int col = x.nb * G::BN + ctl.half * (G::BN / CG);
        for (int s = x.lo; s < x.hi; ++s) {
            if (!wait_bar(ctl, &sm.empty[stage], phase ^ 1, WAIT_EMPTY)) {
                ok = false;
                break;
            }
            const int d = s * G::DEPTH;
            if constexpr (KIND == KIND_MM) {
                const uint32_t bytes = p.a_box * 128 + G::B_BYTES;
                const int bc0 = p.b_mn ? col : d, bc1 = p.b_mn ? d : col;
                if (CG == 1) {
                    mbar_arrive_expect_tx(&sm.full[stage], bytes);
                    tma_load_2d(sm.a(stage), &p.tmA, d, row, &sm.full[stage]);
                    tma_load_2d(sm.b(stage), &p.tmB, bc0, bc1, &sm.full[stage]);
                } else {
                    if (ctl.half == 0) mbar_arrive_expect_tx(&sm.full[stage], CG * bytes);
                    const uint32_t fb = mapa_shared(&sm.full[stage], 0);
                    tma_load_2d_pair(sm.a(stage), &p.tmA, d, row, fb);
                    tma_load_2d_pair(sm.b(stage), &p.tmB, bc0, bc1, fb);
                }
            } else {
                mbar_arrive_expect_tx(&sm.raw[stage], G::RAW_BYTES);
                tma_load_2d(sm.raw_tile(stage), &p.tmA, row, d, &sm.raw[stage]);
                if (CG == 1) {
                    mbar_arrive_expect_tx(&sm.full[stage], G::B_BYTES);
                    for (int c = 0; c < G::BN / CG / 64; ++c)
                        tma_load_2d(sm.b(stage) + c * 8192, &p.tmB, col + c * 64, d, &sm.full[stage]);
                } else {
                    if (ctl.half == 0) mbar_arrive_expect_tx(&sm.full[stage], CG * G::B_BYTES);
                    const uint32_t fb = mapa_shared(&sm.full[stage], 0);
                    for (int c = 0; c < G::BN / CG / 64; ++c)
                        tma_load_2d_pair(sm.b(stage) + c * 8192, &p.tmB, col + c * 64, d, fb);
                }
            }
            filled = (filled & ~(1u << stage)) | phase << stage;
            used |= 1u << stage;
            if (++stage == G::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    // every load has landed before the CTA leaves.  The odd CTA's loads count
    // on the even CTA's barrier: it waits until the MMA has read its last fill.
    bool left = true;
    for (int s = 0; s < G::STAGES; ++s)
        if ((used & (1u << s)) && left) {
            const uint32_t ph = filled >> s & 1u;
            left = drain_bar(ctl, ctl.half ? &sm.empty[s] : &sm.full[s], ph, WAIT_DRAIN_TMA);
            if (KIND == KIND_WG) left = left && drain_bar(ctl, &sm.raw[s], ph, WAIT_DRAIN_TMA);
        }
}

template <int KIND, int CG>
__device__ void run_mma(const GemmParams& p, const Ctl& ctl, Smem<KIND, CG>& sm, uint32_t tmem, int first, int step) {
    using G = Geo<KIND, CG>;
    constexpr int CH = KIND == KIND_MM ? 1 : WG_CHUNK;
    // per MMA step of K = 32 codes or 16 elements, in descriptor units of 16
    // bytes: 32 bytes along a K-major swizzled row, else 32 or 16 rows of 128
    const uint64_t a_adv = KIND == KIND_MM ? 2 : 128;
    const uint64_t b_adv = KIND == KIND_MM ? (p.b_mn ? 256 : 2) : 128;
    uint32_t stage = 0, phase = 0, chunk = 0;
    bool ok = true;
    for (int u = first; u < p.n_units && ok; u += step) {
        const Unit x = unit_of(p, u);
        for (int s0 = x.lo; s0 < x.hi && ok; s0 += CH, ++chunk) {
            const uint32_t buf = chunk & 1, use = chunk >> 1;
            if (!wait_bar(ctl, &sm.acc_empty[buf], (use & 1) ^ 1, WAIT_ACC_EMPTY)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + buf * G::BN;
            const int end = min(x.hi, s0 + CH);
            for (int s = s0; s < end; ++s) {
                if (!wait_bar(ctl, &sm.full[stage], phase, WAIT_FULL) ||
                    (KIND == KIND_WG && !wait_bar(ctl, &sm.conv[stage], phase, WAIT_CONVERTED))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // K-major: 8-row groups 1024 bytes apart (stride offset).
                // MN-major: 128-byte columns of 8-deep groups 1024 bytes
                // apart (stride offset); KIND_WG's two 64-element columns
                // 8192 bytes apart (leading offset).
                const uint64_t ad = smem_desc(smem_u32(sm.a(stage)), KIND == KIND_MM ? 16 : 8192, 1024);
                const uint64_t bd = smem_desc(smem_u32(sm.b(stage)), KIND == KIND_MM ? 16 : 8192, 1024);
#pragma unroll
                for (int k = 0; k < G::UMMA_STEPS; ++k) {
                    const uint32_t acc = (s > s0 || k > 0) ? 1u : 0u;
                    if (KIND == KIND_MM)
                        umma_f8<CG>(d, ad + k * a_adv, bd + k * b_adv, p.idesc, acc);
                    else
                        umma_f16<CG>(d, ad + k * a_adv, bd + k * b_adv, p.idesc, acc);
                }
                if (CG == 2)
                    umma_commit_pair_both(&sm.empty[stage]);
                else
                    umma_commit<1>(&sm.empty[stage]);
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (p.debug_skip == static_cast<uint32_t>(u) + 1) continue;
            if (CG == 2)
                umma_commit_pair_both(&sm.acc_full[buf]);
            else
                umma_commit<1>(&sm.acc_full[buf]);
        }
    }
    umma_commit<CG>(sm.final_bar);
    drain_bar(ctl, sm.final_bar, 0, WAIT_DRAIN_MMA);
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int bf16) {
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// bytes that are infinity or NaN, as a nonzero word (add: 4 or 1 in each byte)
__device__ __forceinline__ uint32_t special_codes(uint32_t w, uint32_t add) {
    return ((w & 0x7F7F7F7Fu) + add) & 0x80808080u;
}
// a power of two small enough for 2^120 times it to be a bf16 number, or zero
__device__ __forceinline__ bool simple_scale(float s) {
    return (__float_as_uint(s) & 0x7FFFFFu) == 0u && s <= 128.f;
}
// Converters: 64 x 128 codes of a stage -> 16-bit values times their row's
// scale, in the MN-major swizzled layout (two columns of 64 k, rows of 128
// bytes, 16-byte units XORed with the row).  A thread takes 16 codes of four
// rows; threads of the second column write their two units in the other
// order, so eight threads of a row touch all banks once.  The product is
// rounded once to the 16-bit type; a power-of-two scale makes it exact.
// bf16 with power-of-two scales, the usual case, needs no conversion
// instructions: a code's exponent and mantissa bits set into a bf16 number
// give its value times 2^-120 (e5m2: 2^-112), subnormal codes included, and
// one packed multiplication by scale * 2^120 is exact.  NaN and infinity do
// not follow that rule; a thread that meets one converts its codes one by one.
template <int CG>
__device__ void run_convert(const GemmParams& p, const Ctl& ctl, Smem<KIND_WG, CG>& sm, int t, int first, int step) {
    using G = Geo<KIND_WG, CG>;
    uint32_t stage = 0, phase = 0;
    const int seg = t & 7, row0 = t >> 3, col = seg >> 2;
    const int e5m2 = p.codes_e5m2;
    const uint32_t add = e5m2 ? 0x04040404u : 0x01010101u, mask = e5m2 ? 0x0FE00FE0u : 0x07F007F0u;
    const int shift = e5m2 ? 3 : 4;
    const float widen = __int_as_float((127 + (e5m2 ? 112 : 120)) << 23);
    for (int u = first; u < p.n_units; u += step) {
        const Unit x = unit_of(p, u);
        // this CTA's 128 output rows are one block of scales
        const int kblk = x.mb * CG + ctl.half;
        const bool live = kblk * BM < p.M;
        const float* sx = p.sa + kblk * p.sa_cs;
        float next[4];
        auto fetch = [&](int s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = s * G::DEPTH + row0 + 16 * i;
                next[i] = (live && m < p.D) ? __ldg(sx + m * p.sa_rs) : 0.f;
            }
        };
        fetch(x.lo);
        for (int s = x.lo; s < x.hi; ++s) {
            float sc[4];
            bool simple = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[i] = next[i];
                simple = simple && simple_scale(sc[i]);
            }
            if (s + 1 < x.hi) fetch(s + 1);
            if (!wait_bar(ctl, &sm.raw[stage], phase, WAIT_RAW)) return;
            const uint8_t* src = sm.raw_tile(stage);
            uint8_t* dst = sm.a(stage) + col * 8192;
            uint4 c4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c4[i] = *reinterpret_cast<const uint4*>(src + (row0 + 16 * i) * 128 + seg * 16);
            uint32_t special = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                special |= special_codes(c4[i].x, add) | special_codes(c4[i].y, add) | special_codes(c4[i].z, add) |
                           special_codes(c4[i].w, add);
            const bool fast = p.x_bf16 && simple && !special;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row0 + 16 * i;
                const uint32_t w[4] = {c4[i].x, c4[i].y, c4[i].z, c4[i].w};
                uint32_t o[8];
                if (fast) {
                    const __nv_bfloat162 f = __float2bfloat162_rn(sc[i] * widen);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t v = __byte_perm(w[j / 2], 0u, (j & 1) ? 0x3424u : 0x1404u);  // codes in bytes 1 and 3
                        const uint32_t b = (v & 0x80008000u) | ((v >> shift) & mask);
                        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), f);
                        o[j] = *reinterpret_cast<const uint32_t*>(&y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t h = cvt_f8x2_f16x2(w[j / 2] >> (16 * (j & 1)), p.codes_e5m2);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                        o[j] = pack16(f.x * sc[i], f.y * sc[i], p.x_bf16);
                    }
                }
                const uint4 v0 = make_uint4(o[0], o[1], o[2], o[3]), v1 = make_uint4(o[4], o[5], o[6], o[7]);
                const int j0 = (seg & 3) * 2;
                uint8_t* line = dst + r * 128;
                uint4* u0 = reinterpret_cast<uint4*>(line + ((j0 ^ (r & 7)) << 4));
                uint4* u1 = reinterpret_cast<uint4*>(line + (((j0 + 1) ^ (r & 7)) << 4));
                if (col) {
                    *u1 = v1;
                    *u0 = v0;
                } else {
                    *u0 = v0;
                    *u1 = v1;
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if ((t & 31) == 0) {
                if (CG == 2)
                    mbar_arrive_remote(mapa_shared(&sm.conv[stage], 0));
                else
                    mbar_arrive(&sm.conv[stage]);
            }
            if (++stage == G::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
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

// Promotion and epilogue of every unit; false = a wait gave up.
template <int KIND, int CG>
__device__ bool run_promote(const GemmParams& p, const Ctl& ctl, Smem<KIND, CG>& sm, uint32_t tmem, int w, int lane,
                            int first, int step) {
    using G = Geo<KIND, CG>;
    constexpr int COLS = G::COLS, CH = KIND == KIND_MM ? 1 : WG_CHUNK;
    const int q = w & 3, h = w >> 2;
    uint32_t chunk = 0, syncs = 0;
    uint8_t* stg = sm.out + w * G::OUT_BYTES;
    for (int u = first; u < p.n_units; u += step) {
        const Unit x = unit_of(p, u);
        const int blk = x.mb * CG + ctl.half;
        const int row0 = blk * BM + q * 32, row = row0 + lane;
        const int col0 = x.nb * G::BN + h * COLS;
        // rows or columns outside the matrix: nothing to add up, in step with the others
        const bool live = row0 < p.M && col0 < p.N;
        unsigned long long acc[COLS / 2];
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;

        const float* sa = p.sa + static_cast<long long>(row) * p.sa_rs;
        const float* sb = p.sb + (col0 / 128) * p.sb_cs;
        // the two scales of a stage are fetched two stages ahead and
        // multiplied where they are used, so that no load is waited for
        struct Scales {
            float a, b;
        };
        auto scales_of = [&](int s) {
            Scales v{0.f, 0.f};
            if (KIND == KIND_MM && live && s < x.hi) {
                if (row < p.M) v.a = __ldg(sa + s * p.sa_cs);
                v.b = __ldg(sb + s * p.sb_rs);
            }
            return v;
        };
        Scales s_cur = scales_of(x.lo), s_next = scales_of(x.lo + 1);
        for (int s0 = x.lo; s0 < x.hi; s0 += CH, ++chunk) {
            const uint32_t buf = chunk & 1;
            const Scales s_after = scales_of(s0 + 2);
            if (!wait_bar(ctl, &sm.acc_full[buf], (chunk >> 1) & 1, WAIT_ACC_FULL)) return false;
            tc_fence_after();
            if (live) {
                const float sc = KIND == KIND_MM ? s_cur.a * s_cur.b : 1.f;
                const unsigned long long sc2 = pack_f32x2(__float_as_uint(sc), __float_as_uint(sc));
                const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::BN + h * COLS;
                // KIND_MM promotes every stage: its next load runs under the
                // sums.  KIND_WG promotes every WG_CHUNK stages and has fewer
                // registers.
                constexpr int NB = KIND == KIND_MM ? 2 : 1;
                uint32_t r[NB][32];
                tmem_ld_32x32b_x32(base, r[0]);
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    tmem_wait_regs(r[c % NB]);
                    if (NB == 2 && c + 1 < COLS / 32) tmem_ld_32x32b_x32(base + (c + 1) * 32, r[(c + 1) % NB]);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[c * 16 + i] = fma_f32x2(pack_f32x2(r[c % NB][2 * i], r[c % NB][2 * i + 1]), sc2, acc[c * 16 + i]);
                    if (NB == 1 && c + 1 < COLS / 32) tmem_ld_32x32b_x32(base + (c + 1) * 32, r[0]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2)
                    mbar_arrive_remote(mapa_shared(&sm.acc_empty[buf], 0));
                else
                    mbar_arrive(&sm.acc_empty[buf]);
            }
            s_cur = s_next;
            s_next = s_after;
        }

        // epilogue: 32 rows x 128 bytes at a time through swizzled staging and
        // a tensor store, which clips the ragged edges.  Whole sums are
        // rounded here, once; parts stay fp32.
        if (live) {
            const bool wide = p.staged || p.out_type == T_F32;
            const bool add_bias = KIND == KIND_MM && p.bias != nullptr && !p.staged;
#pragma unroll
            for (int c = 0; c < COLS / 32; ++c) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) unpack_f32x2(acc[c * 16 + i], v[2 * i], v[2 * i + 1]);
                if (add_bias) {
                    const float b = load_bias(p, col0 + c * 32 + lane);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, b, i);
                }
                if (wide || (c & 1) == 0) {  // the staging buffer is used anew
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
                }
                if (wide) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<float4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else {
                    const int bf = p.out_type == T_BF16;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(stg + lane * 128 + (((j + (c & 1) * 4) ^ (lane & 7)) << 4)) =
                            make_uint4(pack16(v[8 * j], v[8 * j + 1], bf), pack16(v[8 * j + 2], v[8 * j + 3], bf),
                                       pack16(v[8 * j + 4], v[8 * j + 5], bf), pack16(v[8 * j + 6], v[8 * j + 7], bf));
                }
                if (wide || (c & 1) == 1) {
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        const int cc = col0 + (wide ? c : c - 1) * 32;
                        if (cc < p.N) tma_store_3d(&p.tmC, stg, cc, row0, p.staged ? x.part : 0);
                        bulk_commit();
                    }
                }
            }
        }

        if (p.staged) {
            // publish this part, then the last one of the tile adds them up in
            // part order and writes the output
            if (lane == 0) {
                bulk_wait_all();
                fence_proxy_async_global();
            }
            __syncwarp();
            __threadfence();
            auto sync = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.sync);
                const bool ok = wait_bar(ctl, sm.sync, syncs & 1, WAIT_SYNC);
                ++syncs;
                return ok;
            };
            if (!sync()) return false;
            if (w == 0 && lane == 0) {
                bool last = true;
                __threadfence();
                if (p.split > 1)
                    last = arrive_count(p.arrived + (u / p.split) * CG + ctl.half, ctl.epoch) == static_cast<uint32_t>(p.split);
                __threadfence();
                *reinterpret_cast<volatile uint32_t*>(sm.last) = last ? 1u : 0u;
            }
            if (!sync()) return false;
            if (*reinterpret_cast<volatile uint32_t*>(sm.last)) {
                __threadfence();
                const int rows = min(BM, p.M - blk * BM), tile_c = x.nb * G::BN;
                const int quads = (min(G::BN, p.N - tile_c) + 3) / 4;
                for (int i = w * 32 + lane; i < rows * quads; i += 256) {
                    const int r = blk * BM + i / quads, c = tile_c + (i % quads) * 4;
                    const float* src = p.partial + static_cast<long long>(r) * p.part_rs + c;
                    float4 sum = __ldcg(reinterpret_cast<const float4*>(src));
                    for (int k = 1; k < p.split; ++k) {
                        const float4 t = __ldcg(reinterpret_cast<const float4*>(src + k * p.part_stride));
                        sum.x += t.x;
                        sum.y += t.y;
                        sum.z += t.z;
                        sum.w += t.w;
                    }
                    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < p.N) store_out(p, r, c + e, v[e] + (KIND == KIND_MM ? load_bias(p, c + e) : 0.f));
                }
            }
            // the flag is read by all before the next unit may set it anew
            if (!sync()) return false;
        }
    }
    return true;
}

template <int KIND, int CG>
__global__ void __launch_bounds__(Geo<KIND, CG>::THREADS, 1) block_gemm_kernel(const __grid_constant__ GemmParams p) {
    using G = Geo<KIND, CG>;
    extern __shared__ uint8_t smem_raw[];
    Smem<KIND, CG> sm;
    sm.carve(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int half = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
            mbar_init(&sm.raw[s], 1);
            mbar_init(&sm.conv[s], CG * 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], CG * 8);
        }
        mbar_init(sm.sync, 8);
        mbar_init(sm.final_bar, 1);
        fence_mbar_init();
        uint32_t e = *reinterpret_cast<volatile uint32_t*>(&p.ws->epoch) + 1u;
        *sm.epoch_slot = e == 0u ? 1u : e;
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        tma_prefetch_desc(&p.tmC);
    }
    if (warp == 1) tmem_alloc<G::TMEM_COLS, CG>(sm.tmem_slot);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    const Ctl ctl{p.ws, *sm.epoch_slot, p.wait_ns, half};
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp < 4) {
        reg_dec<G::REGS_CTL>();
        if (warp == 0) {
            if (lane == 0) run_tma<KIND, CG>(p, ctl, sm, first, step);
        } else if (warp == 1) {
            if (lane == 0 && half == 0) run_mma<KIND, CG>(p, ctl, sm, tmem, first, step);
        }
        __syncwarp();
    } else if (warp < 12) {
        reg_inc<G::REGS_PROMOTE>();
        run_promote<KIND, CG>(p, ctl, sm, tmem, warp - 4, lane, first, step);
        if (lane == 0) bulk_wait_all();  // its stores have left shared memory, stopped or not
        __syncwarp();
    } else if constexpr (KIND == KIND_WG) {
        reg_dec<G::REGS_CONV>();
        run_convert<CG>(p, ctl, sm, threadIdx.x - 384, first, step);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // neither CTA of a pair leaves (or frees tensor memory) while the other
    // may still signal its barriers
    if (CG == 2) cluster_sync();
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
    const long long n = static_cast<long long>(p.M) * p.N;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
        store_out(p, i / p.N, i % p.N, load_bias(p, static_cast<int>(i % p.N)));
}

}  // namespace fp8
}  // namespace gct
