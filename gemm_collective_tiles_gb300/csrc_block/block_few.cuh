// The 16-bit product with its epilogue for at most 64 rows (decoding): the
// weights' columns take the MMA's 128 rows and the tokens its N.
//
// Such a product reads every weight once for a handful of multiplications and
// should run at the speed of memory: a tile needs no more of the tensor core
// than its tokens, a stage is 16 KB of weights and its tokens' 64 columns, and
// ten of them are under way per SM.
//
// Measured: one token 4096 x 14336 in 21.7 us (5.4 TB/s; as 128 x 128 tiles 42),
// 48 x 14336 x 4096 with its residual in 25.9 us.  Two CTAs an SM of five stages
// each instead of one of eleven: 24.4 us for the token.
//
// CTA layout (256 threads, one CTA per SM): warp 0 loads, warp 1 issues the
// MMAs, warps 4-7 are the epilogue: 32 columns of the output each.  A cluster of
// up to 8 CTAs shares a tile's contraction.  At the end every part's sums lie in
// shared memory as [token][column]; each CTA adds its share of the rows over them,
// in the order of the parts, and finishes them, four columns a lane.
#pragma once
#include "block_gemm.cuh"

namespace gct {
namespace block {

template <int NT>
struct FewGeo {
    static constexpr uint32_t W_BYTES = 128 * 128, X_BYTES = NT * 128, STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int STAGES = NT == 16 ? 11 : NT == 32 ? 9 : 7;
    static constexpr int ACCS = 2, TMEM_COLS = ACCS * NT;
    static constexpr uint32_t SUMS = NT * 128;  // fp32
    static constexpr uint32_t TILES_BYTES = STAGES * STAGE_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 3;
    static constexpr uint32_t BYTES = 1024 + TILES_BYTES + SUMS * 4 + NUM_BARS * 8 + 16;
    static constexpr int THREADS = 256;
    static_assert(BYTES <= 232448, "shared memory");
};

// 16, 32 or 64 columns at once
template <int NT>
__device__ __forceinline__ void load_sums(uint32_t from, uint32_t (&r)[NT]) {
    tmem_ld_cols(from, r);
    tmem_wait_regs(r);
}

template <int NT>
__global__ void __launch_bounds__(FewGeo<NT>::THREADS, 1) act_few_kernel(const __grid_constant__ ActParams p) {
    using G = FewGeo<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t tiles = smem_u32(base);
    float* const sums = reinterpret_cast<float*>(base + G::TILES_BYTES);
    const uint32_t full = tiles + G::TILES_BYTES + G::SUMS * 4, done = full + 8 * G::STAGES;
    const uint32_t acc_full = done + 8 * G::STAGES, acc_empty = acc_full + 8 * G::ACCS;
    const uint32_t parts_in = acc_empty + 8 * G::ACCS, parts_out = parts_in + 8, final_bar = parts_out + 8;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base + (final_bar + 8 - tiles));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int S = p.split;
    const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(done + 8 * s, 1);
        }
        for (int b = 0; b < G::ACCS; ++b) {
            bar_init(acc_full + 8 * b, 1);
            bar_init(acc_empty + 8 * b, 4);
        }
        bar_init(parts_in, 4 * S);
        bar_init(parts_out, 4 * S);
        bar_init(final_bar, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        // for the whole CTA, which waits for this thread below
        grid_wait();
        grid_release();
        const uint32_t e = *reinterpret_cast<volatile uint32_t*>(&p.ws->epoch) + 1u;
        tmem_slot[1] = e == 0u ? 1u : e;
    }
    if (warp == 1) tmem_alloc<G::TMEM_COLS, 1>(tmem_slot);
    tc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot[0];
    const Ctl ctl{p.ws, tmem_slot[1], p.wait_ns, rank};
    const int first = blockIdx.x / S, step = gridDim.x / S;
    const int lo = part_start(p, rank), hi = part_start(p, rank + 1);

    if (warp == 0) {
        if (lane == 0) {
            Ring<G::STAGES> st;
            Fills fills;
            bool ok = true;
            for (int u = first; u < p.n_units && ok; u += step)
                for (int s = lo; s < hi; ++s) {
                    if (!wait_bar(ctl, done + 8 * st.slot, st.phase ^ 1, WAIT_EMPTY)) {
                        ok = false;
                        break;
                    }
                    const uint32_t w = tiles + st.slot * G::STAGE_BYTES, bar = full + 8 * st.slot;
                    bar_expect_tx(bar, G::W_BYTES + p.M * 128);
                    load_operand<1>(w, &p.tmB, p.b_mn, u * 128, 128, s * DEPTH, bar);
                    tma_load_2d(w + G::W_BYTES, &p.tmA, s * DEPTH, 0, bar);
                    fills.add(st.slot, st.phase);
                    st.next();
                }
            fills.drain(ctl, full, G::STAGES);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t w_adv = p.b_mn ? 128 : 2;
        const uint64_t w_desc = smem_desc(tiles, p.b_mn ? 8192 : 16, 1024), x_desc = smem_desc(tiles + G::W_BYTES, 16, 1024);
        Ring<G::STAGES> st;
        Ring<G::ACCS> acc;
        bool ok = true;
        for (int u = first; u < p.n_units && ok && lo < hi; u += step, acc.next()) {
            const bool report = p.debug_skip != static_cast<uint32_t>(u) + 1;
            if (!wait_bar(ctl, acc_empty + 8 * acc.slot, acc.phase ^ 1, WAIT_ACC_EMPTY)) break;
            for (int s = lo; s < hi; ++s, st.next()) {
                if (!wait_bar(ctl, full + 8 * st.slot, st.phase, WAIT_FULL)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t at = st.slot * (G::STAGE_BYTES / 16);
                const uint32_t more = s > lo ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < DEPTH / 16; ++k)
                        umma_f16<1>(tmem + acc.slot * NT, w_desc + at + k * w_adv, x_desc + at + k * 2, p.idesc, k > 0 ? 1u : more);
                    umma_commit_all<1>(done + 8 * st.slot);
                    if (s == hi - 1 && report) umma_commit_all<1>(acc_full + 8 * acc.slot);
                }
                __syncwarp();
            }
        }
        if (elect_one()) umma_commit_one<1>(final_bar);
        __syncwarp();
        wait_bar(ctl, final_bar, 0, WAIT_DRAIN_MMA);
    } else if (warp >= 4) {
        const int q = warp - 4;
        const DropKey key = drop_key(p.drop);
        const int row_lo = p.M * rank / S, row_hi = p.M * (rank + 1) / S;  // this part's share of the outputs
        Ring<G::ACCS> acc;
        uint32_t tiles_done = 0;
        for (int u = first; u < p.n_units; u += step, ++tiles_done) {
            const Four four(p, u * 128 + lane * 4);
            float4 res[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) res[j] = four.residual(p, min(row_lo + q + 4 * j, p.M - 1));
            uint32_t r[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) r[i] = 0u;
            if (lo < hi) {  // a part without stages adds zeros
                if (!wait_bar(ctl, acc_full + 8 * acc.slot, acc.phase, WAIT_ACC_FULL)) break;
                __syncwarp();  // tensor-memory loads are for the converged warp
                tc_fence_after();
                load_sums<NT>(tmem + (static_cast<uint32_t>(q * 32) << 16) + acc.slot * NT, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(acc_empty + 8 * acc.slot);
                acc.next();
            }
            // every part has read what lay here before
            if (tiles_done > 0 && !wait_bar_cluster(ctl, parts_out, (tiles_done - 1) & 1, WAIT_PARTS)) break;
            float* const to = sums + q * 32 + lane;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i < p.M) to[i * 128] = __uint_as_float(r[i]);
            __syncwarp();
            if (S == 1) {
                if (lane == 0) bar_arrive(parts_in);
            } else if (lane < S) {
                mbar_arrive_cluster(map_to(parts_in, lane));
            }
            if (S == 1 ? !wait_bar(ctl, parts_in, tiles_done & 1, WAIT_PARTS)
                       : !wait_bar_cluster(ctl, parts_in, tiles_done & 1, WAIT_PARTS))
                break;
            __syncwarp();
            // this part's rows of the tile: four columns a lane, every 16th of them a warp
            // at once with the loads of four rows under way
            const uint32_t mine = smem_u32(sums) + lane * 16;
            for (int i = row_lo + q; i < row_hi; i += 16) {
                float4 part[4][MOST_PARTS];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < MOST_PARTS; ++k)
                        if (k < S && i + 4 * j < row_hi)
                            part[j][k] = ld_shared_cluster_f4((S == 1 ? mine : map_to(mine, k)) + (i + 4 * j) * 512);
                if (i > row_lo + q) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) res[j] = four.residual(p, min(i + 4 * j, p.M - 1));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (i + 4 * j >= row_hi) break;
                    float v[4] = {part[j][0].x, part[j][0].y, part[j][0].z, part[j][0].w};
#pragma unroll
                    for (int k = 1; k < MOST_PARTS; ++k)
                        if (k < S) {
                            v[0] += part[j][k].x;
                            v[1] += part[j][k].y;
                            v[2] += part[j][k].z;
                            v[3] += part[j][k].w;
                        }
                    four.finish(p, key, i + 4 * j, v, res[j]);
                }
            }
            // tell the parts that their sums have been read, unless none will write
            // again: a CTA on its way out gets no more arrivals
            __syncwarp();
            if (u + step < p.n_units) {
                if (S == 1) {
                    if (lane == 0) bar_arrive(parts_out);
                } else if (lane < S) {
                    mbar_arrive_cluster(map_to(parts_out, lane));
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // no CTA of a cluster leaves while another may still signal its barriers or
    // read its sums
    if (S > 1) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<G::TMEM_COLS, 1>(tmem);
    }
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&p.ws->done_ctr, 1u) == gridDim.x - 1)
            *reinterpret_cast<uint4*>(p.ws) = make_uint4(ctl.epoch, 0u, 0u, 0u);
    }
}

}  // namespace block
}  // namespace gct
